"""Shapes of the weight gradient that take each way through its kernel, and what is launched for them
with 76 resident CTA pairs: test_train_host.py holds the plans to it, test_wgrad_ways_gpu.py runs them."""

PAIRS = 76

# (rows, cols, outs): halves, ranges of tokens, units of half a tile, most units of one pair, TMA scales
WAYS = {
    # tiles of two N-halves
    (700, 2500, 2304): (2, 1, 0, 1, False),
    (1000, 4864, 4096): (2, 1, 0, 2, False),     # both accumulators handed back once
    (700, 5120, 8192): (2, 1, 32, 5, True),      # four times, then half tiles
    (520, 3000, 4608): (2, 1, 64, 2, False),     # half tiles leave accumulator 1 alone
    (1000, 2048, 7000): (2, 1, 72, 2, True),     # the last tile column is ragged
    (16384, 2048, 1024): (2, 4, 0, 1, True),
    (16000, 2000, 1000): (2, 4, 0, 1, False),    # ranges of 63, 63, 63 and 61 k-blocks
    # of one
    (130, 5000, 4096): (1, 1, 32, 5, False),
    (64, 4096, 5120): (1, 1, 32, 5, True),       # one k-block a unit
    (1024, 1536, 1024): (1, 1, 48, 1, True),
    (12000, 1536, 1024): (1, 3, 0, 1, True),
    (30000, 100, 64): (1, 53, 0, 1, False),      # the last range has one k-block
}
