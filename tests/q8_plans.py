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
    splits = _host("_ZN4qlin16w8a8_few_splitsElll", ctypes.c_int, 3)(M, N, K)
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
