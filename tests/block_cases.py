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
