"""The ncu summary of the fused products says which sources it was taken of (no GPU)."""

import os
import re

from persistent_warp_specialized_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_summary_is_of_these_sources_or_says_so():
    with open(os.path.join(ROOT, "profiles", "fused_products.md")) as f:
        text = f.read()
    stamp = re.search(r"source_stamp:\s*`([0-9a-f]{64})`", text)
    assert stamp
    assert stamp.group(1) == _build.kernel_stamp("fused_products") or "of earlier sources" in text
