"""Sizes of the grouped products' and the 4-bit product's tests, with the kernel that the choosing rules send each to."""
from persistent_tile_scheduling_macro_amd import (PGEMM_GROUPED_ANY as ANY, PGEMM_GROUPED_FEW16 as FEW16,
                                                  PGEMM_GROUPED_FEW16_WIDE as FEW16_WIDE, PGEMM_GROUPED_FEW32_WIDE as FEW32,
                                                  PGEMM_GROUPED_FEW_GRAD as FEW_GRAD, PGEMM_GROUPED_PINGPONG as PINGPONG)

BODIES = (ANY, PINGPONG, FEW16, FEW16_WIDE, FEW32)

# rows of each expert, K, N, layout -> bodies of the product and of the rows' gradient, body and pieces of the weights'.
# Some expert is empty or has a row or two, last tiles are cut in rows, K and N, and steps of 64 are odd in number.
_BOTH = [
    ([3001, 0, 1100, 4099], 1000, 2056, PINGPONG, PINGPONG, (PINGPONG, 1)),
    ([1900, 1, 2100], 1024, 2048, PINGPONG, ANY, (PINGPONG, 1)),
    ([2600, 3400, 0], 1288, 1032, PINGPONG, PINGPONG, (PINGPONG, 2)),
    ([5000, 2, 3999, 0, 7001], 520, 512, PINGPONG, PINGPONG, (ANY, 5)),
    ([4100, 900], 64, 64, FEW32, FEW32, (PINGPONG, 13)),
    ([1300, 0, 2700], 1031, 1033, ANY, ANY, (ANY, 1)),
    ([8999, 1], 257, 131, ANY, ANY, (ANY, 23)),
    ([2500, 0, 600, 1900], 512, 776, ANY, ANY, (ANY, 4)),
    ([0, 700, 1, 499], 600, 600, FEW32, FEW32, (FEW_GRAD, 1)),
    ([5, 9, 1, 0, 3], 200, 136, FEW16, FEW16, (FEW_GRAD, 1)),
    ([5, 9, 1, 0, 3], 201, 137, FEW16, FEW16, (FEW_GRAD, 1)),
    ([4, 0, 7, 9, 1, 6, 2, 8] * 8, 1032, 1032, FEW16_WIDE, FEW16_WIDE, (FEW_GRAD, 1)),
    ([4, 0, 7, 9, 1, 6, 2, 8] * 8, 1031, 1033, FEW16_WIDE, FEW16_WIDE, (FEW_GRAD, 1)),
    ([60, 0, 75, 33], 4096, 1032, FEW32, FEW32, (FEW_GRAD, 1)),
    ([60, 0, 75, 33], 2047, 1031, FEW32, FEW32, (FEW_GRAD, 1)),
]
GROUPED = [(c, K, N, layout, y, dx, dw) for c, K, N, y, dx, dw in _BOTH for layout in ("kn", "nk")]

# rows, columns, K, experts (0: one matrix) -> rows at once and column blocks, on 256 CUs
W4 = [
    (3, 16390, 331, 0, (4, 2)), (13, 16390, 331, 0, (16, 2)), (37, 16390, 331, 0, (32, 2)),
    (4, 16384, 640, 0, (4, 2)), (16, 16384, 640, 0, (16, 2)), (32, 16384, 640, 0, (32, 2)),
    (60, 520, 331, 32, (4, 2)), (200, 520, 331, 32, (16, 2)), (450, 520, 331, 32, (32, 2)),
    (3, 70, 331, 0, (4, 1)), (13, 70, 331, 0, (16, 1)), (37, 70, 331, 0, (32, 1)),
    (20, 70, 331, 11, (4, 1)), (60, 70, 331, 11, (16, 1)), (130, 70, 331, 11, (32, 1)),
]
