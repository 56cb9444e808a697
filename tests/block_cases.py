"""Sizes of the block-scaled products' and the layer's GPU tests by the variant that they take; the CPU
tests check that they take it."""
from __future__ import annotations

# M, N, K, groups, how the groups end (tests.test_gpu_block.group_ends)
FORWARD = {
    "64x64": [(200, 1000, 1040, 2, "cuts"), (500, 999, 400, 3, "cuts"), (1, 8000, 272, 1, "even")],
    "128x64": [(1000, 1500, 400, 3, "cuts"), (900, 1408, 2064, 4, "empties"), (1333, 1111, 272, 7, "cuts")],
    "128x128": [(1900, 1511, 272, 5, "cuts"), (5000, 3500, 144, 6, "cuts"), (4700, 3600, 400, 5, "empties")],
    "256x256": [(4000, 4001, 400, 2, "cuts"), (8000, 4000, 144, 5, "empties"), (4096, 4096, 1040, 2, "cuts"), (16500, 4104, 144, 3, "cuts")],
}
# the same through the transposed weights: M, N (contraction), K
DATA_GRADIENT = {
    "128x64": [(1000, 400, 1500, 3, "cuts")],
    "128x128": [(1900, 272, 1511, 5, "empties")],
    "256x256": [(4000, 400, 4001, 2, "cuts"), (8000, 272, 4000, 5, "empties")],
}
# M, N, K, groups: outputs [groups, K, N]
WEIGHT_GRADIENT = {
    "64x64": [(1000, 500, 700, 1, "even"), (1333, 304, 264, 9, "empties")],
    "128x128": [(900, 704, 1032, 3, "cuts"), (900, 701, 1030, 3, "cuts")],
    "256x256": [(700, 1504, 1304, 9, "cuts"), (1100, 2048, 2056, 4, "empties"), (400, 1530, 1290, 12, "empties")],
}

# The layer: T, top_k, experts of the call, hidden, inner, and the experts that tokens may choose
# (the launch goes by the sizes alone).  Then (token tiles, tokens of a pass, parts) of the gate and up
# product and of the down product.
LAYERS = {
    # 33 blocks of the contraction and more than 64: a part's factors are read twice (four parts)
    "long contraction": ((3, 2, 2, 33280, 16, 2), (1, 4, 4), (1, 4, 1)),
    "long inner": ((2, 1, 3, 16, 33280, 3), (1, 2, 1), (1, 2, 4)),
    # two parts over passes of 32 tokens, three passes, chunks in turn
    "passes of 32": ((70, 1, 4, 1040, 528, 4), (2, 32, 4), (2, 32, 2)),
    # passes of 64 over 5 blocks and over 66, down over 4: chunks of two blocks and of one, in turn
    "passes of 64": ((40, 8, 8, 640, 4096, 8), (4, 64, 1), (2, 32, 2)),
    "passes of 64, long": ((40, 2, 64, 8336, 512, 3), (4, 64, 1), (4, 64, 1)),
    "two passes of 64": ((128, 1, 16, 2064, 2048, 2), (4, 64, 1), (2, 32, 2)),
}
