"""The plans that the library's launchers of the 8-bit row operators choose,
asked of the built library itself (host functions, by their C++ symbols)."""

import ctypes

from quantized_base_rank_amd import _lib


class _Pair(ctypes.Structure):
    _fields_ = [("a", ctypes.c_int32), ("b", ctypes.c_int32)]


def _host(symbol, res, n):
    f = getattr(_lib.lib(), symbol)
    f.restype, f.argtypes = res, [ctypes.c_int64] * n
    return f


def gemm_shape(M, N, K):
    """(64-row units of a tile, shares of K) of the product for many tokens."""
    p = _host("_ZN4qlin15w8a8_gemm_shapeElll", _Pair, 3)(M, N, K)
    return p.a, p.b


def few_shape(M, N, K):
    """(16-channel units of a workgroup, 16-token units, shares of K) of the product for few tokens."""
    tiles = _host("_ZN4qlin14w8a8_few_tilesElll", ctypes.c_int64, 3)(M, N, K)
    splits = _host("_ZN4qlin15w8a8_few_splitsElll", ctypes.c_int, 3)(M, N, K)
    rt = [t for t in (1, 2, 4) if -(-N // (16 * t)) == tiles]
    assert rt, (M, N, K, tiles)
    return rt[0], 1 if M <= 16 else 2 if M <= 32 else 4, splits


def token_shares(M, N, K, r):
    """(token shares of dB, of dA)."""
    f = _lib.lib()._ZN4qlin13tokens_sharesEllli
    f.restype, f.argtypes = _Pair, [ctypes.c_int64] * 3 + [ctypes.c_int]
    p = f(M, N, K, r)
    return p.a, p.b


def du_shape(M, N, r):
    """(columns a lane, 16-token units of a workgroup, shares of d_out) of du."""
    tiles = _host("_ZN4qlin8du_tilesEl", ctypes.c_int64, 1)(M)
    splits = _host("_ZN4qlin9du_splitsEll", ctypes.c_int, 2)(M, N)
    return 1 if r <= 16 else 2 if r <= 32 else 4 if r <= 64 else 8, 2 if tiles == -(-M // 32) else 4, splits


def dx_shares(M, N, K):
    """Shares of d_out for dX's last tiles (more than 16 tokens)."""
    return _host("_ZN4qlin14dx_gemm_sharesElll", ctypes.c_int, 3)(M, N, K)


# Sizes that between them take every path of the launchers (checked on the
# host), each at rows and columns that end inside a tile.

PRODUCTS = [
    # M, N, K: many tokens, tiles of 64, 128, 192, 256 rows, whole and in shares of K
    (200, 517, 400), (78, 17, 1168), (100, 301, 4096), (75, 12849, 1904), (459, 17, 25328), (128, 8191, 14336),
    (127, 8189, 28672), (263, 28241, 16), (333, 32003, 528), (333, 32003, 4096), (160, 8191, 28672), (1675, 17, 8512),
    (190, 6001, 12000), (202, 34501, 3600), (2047, 8191, 3600), (193, 20367, 11552),
    # few tokens: 16, 32, 64 channels by 16, 32, 64 tokens, whole and in shares
    (5, 17, 16), (3, 17, 2064), (24, 17, 48), (23, 333, 2112), (63, 17, 80), (51, 333, 2112), (9, 4105, 528),
    (19, 4123, 1040), (20, 7171, 4096), (58, 4105, 272), (50, 7171, 4096), (64, 7168, 4096), (9, 8341, 8352),
    (16, 14339, 8192), (8, 8159, 17184), (16, 8192, 28672), (21, 8797, 8384), (20, 14339, 8192), (30, 8191, 18208),
    (20, 8131, 28672), (46, 8221, 528), (40, 14339, 4096), (39, 8147, 16560),
]


def product_path(M, N, K):
    if M <= 64:
        rt, mt, s = few_shape(M, N, K)
        return "few", rt, mt, s > 1
    j, s = gemm_shape(M, N, K)
    return "many", j, s > 1


BACKWARDS = [
    # M, N, K, r, pool
    (50, 272, 576, 16, 1), (333, 1040, 64, 11, 1), (2136, 32, 64, 2, 1), (3495, 16, 64, 10, 32), (1601, 16, 128, 30, 1),
    (1967, 16, 64, 41, 1), (2338, 32, 64, 42, 32), (4096, 2048, 2176, 64, 1), (2048, 4096, 11008, 64, 32),
    (4778, 11024, 26432, 59, 1), (257, 272, 320, 80, 1), (300, 528, 1088, 96, 32), (1088, 16, 64, 69, 32),
    (1321, 16, 64, 85, 1), (3279, 704, 4928, 97, 1), (1253, 7920, 26176, 65, 1), (100, 1040, 448, 128, 1),
    (592, 32, 64, 110, 1), (866, 16, 64, 128, 32), (4096, 1024, 1024, 128, 1), (1506, 5840, 27776, 111, 32),
    (16401, 48, 64, 16, 1), (16401, 64, 128, 32, 32), (16401, 48, 192, 64, 1), (16401, 80, 64, 128, 1),
    (1, 1136, 128, 10, 1), (7, 1040, 64, 27, 1), (1, 1024, 64, 60, 32), (33, 1008, 64, 98, 1), (20, 48, 64, 20, 1),
    (20, 48, 64, 50, 1), (20, 48, 64, 99, 1),
]


def token_path(M, N, K, r):
    b, a = token_shares(M, N, K, r)
    return (r + 31) // 32, b > 1, a > 1


def du_path(M, N, r):
    fw, rt, s = du_shape(M, N, r)
    return fw, rt, s > 1
