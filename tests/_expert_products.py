"""Sizes of the 8-bit floating point products that reach every tile, whole and with K split, with remainders
in every direction and K of more blocks than a tile's ring holds."""
import ctypes

from weight_only_bit_moe_amd import binding

TILES = 7                   # of the plain product; -1: streamed
GROUPED_TILES = 5

# T, N, K of each (tile, slices of K)
PLAIN = {
    (0, 1): (2959, 2724, 1040), (1, 1): (2513, 2343, 1040), (2, 1): (2777, 2840, 1040), (3, 1): (1127, 921, 1040),
    (4, 1): (469, 520, 1040), (5, 1): (1426, 1426, 1056), (6, 1): (2177, 1795, 1040),
    (1, 2): (1541, 1742, 10448), (3, 2): (579, 782, 3296), (4, 2): (596, 409, 2192), (5, 2): (1393, 717, 4768),
    (6, 2): (1556, 1286, 4880),
    (0, 4): (8366, 195, 15648), (1, 4): (1289, 971, 12656), (2, 4): (5276, 257, 29008), (3, 4): (514, 454, 4448),
    (4, 4): (34, 18, 8480), (5, 4): (609, 777, 6480), (6, 4): (1130, 933, 5424),
    (0, 8): (4312, 217, 39648), (1, 8): (697, 997, 31296), (2, 8): (7720, 66, 75536), (3, 8): (271, 397, 13936),
    (4, 8): (34, 17, 8736), (5, 8): (321, 676, 19040), (6, 8): (905, 540, 14288),
    (1, 16): (655, 399, 91488), (3, 16): (262, 194, 46512), (4, 16): (33, 18, 35888), (5, 16): (335, 325, 64736),
    (6, 16): (459, 514, 44736),
}
# and streamed ones: ragged tokens and channels, K of several turns of the waves
STREAMED = [(1, 17, 4112), (8, 4100, 2064), (9, 300, 4112), (16, 4111, 2192), (31, 517, 3088), (64, 530, 2064),
            (150, 70, 1040)]

# tile, and E, R, N, K: experts of one, few and more than 64, that is more than one turn of the search
GROUPED = [
    (0, (1, 2464, 3359, 1056)), (0, (3, 7621, 1048, 1040)), (0, (17, 12129, 530, 1056)),
    (1, (2, 2763, 1458, 1040)), (1, (9, 6368, 521, 1072)), (1, (70, 14974, 131, 1056)),
    (2, (1, 1598, 1378, 1040)), (2, (9, 5457, 364, 1040)), (2, (70, 9018, 166, 1040)),
    (3, (2, 1265, 782, 1072)), (3, (17, 4968, 143, 1040)), (3, (70, 6080, 71, 1088)),
    (4, (3, 40, 530, 1040)), (4, (9, 300, 83, 2064)), (4, (70, 700, 150, 1040)),
]


class Plan(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("split", ctypes.c_int), ("workspace", ctypes.c_size_t)]


def plan(T, N, K):
    """The tile, the slices of K and the workspace of a plain product, as the library plans it."""
    f = binding.load_library()._ZN5wna1613gemm_fp8_planEiii
    f.restype, f.argtypes = Plan, [ctypes.c_int] * 3
    return f(T, N, K)


def grouped_tile(E, R, N, K):
    f = binding.load_library()._ZN5wna1621gemm_fp8_grouped_tileEiiii
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int] * 4
    return f(E, R, N, K)
