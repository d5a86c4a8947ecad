"""Refusals of the attention operators and the cache, reported before anything
reaches a GPU, and their workspace sizes."""

import ctypes
import os

import pytest

from quantized_base_rank_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libqlin.so not built (run __graft_entry__.build())")

NULL_, SHAPE, ALIGN, WORKSPACE, OVERLAP = 1, 2, 3, 6, 8
BIG = 1 << 40
T, HQ, HKV, D, B = 40, 8, 2, 64, 3


def far(i):
    """Addresses 4 GiB apart."""
    return (i + 1) << 32


def swap(args, i, v):
    return [v if j == i else a for j, a in enumerate(args)]


def fwd_args():
    return [far(0), HQ * D, far(1), HKV * D, far(2), HKV * D, far(3), B, T, HQ, HKV, D, 0.125, far(4), far(5), None]


def bwd_args():
    return [far(0), HQ * D, far(1), HKV * D, far(2), HKV * D, far(3), far(4), far(5), far(6), B, T, HQ, HKV, D, 0.125,
            far(7), HQ * D, far(8), HKV * D, far(9), HKV * D, far(10), BIG, None]


SIZES = [(0, 0), (0, -1), (0, (1 << 20) + 1),             # batch
         (1, -1), (1, 1 << 31), (1, (1 << 31) // HQ),      # tokens
         (2, 0), (2, 9), (2, 1), (2, 8192), (2, 258),      # heads_q
         (3, 0), (3, 3), (3, 16),                          # heads_kv
         (4, 0), (4, 8), (4, 72), (4, 144)]                # dim


def test_prompt_refusals():
    f = _lib.lib().qlin_attn_fwd
    good = fwd_args()
    for i in (0, 2, 4, 6, 13):
        assert f(*swap(good, i, None)) == NULL_
    for i in (0, 2, 4, 13, 14):
        assert f(*swap(good, i, far(20) + 8)) == ALIGN
    assert f(*swap(good, 6, far(20) + 2)) == ALIGN
    for i, v in SIZES:
        assert f(*swap(good, 7 + i, v)) == SHAPE, (i, v)
    for i, row in ((1, HQ * D), (3, HKV * D), (5, HKV * D)):
        for v in (row - 8, row + 4, 0, -row, 1 << 23):
            assert f(*swap(good, i, v)) == SHAPE
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert f(*swap(good, 12, v)) == SHAPE
    assert f(*swap(good, 8, 0)) == 0  # no tokens


def test_gradient_refusals():
    f = _lib.lib().qlin_attn_bwd
    good = bwd_args()
    for i in (0, 2, 4, 6, 7, 8, 9, 16, 18, 20):
        assert f(*swap(good, i, None)) == NULL_
    for i in (0, 2, 4, 6, 7, 8, 16, 18, 20, 22):
        assert f(*swap(good, i, far(20) + 8)) == ALIGN
    for i, v in SIZES:
        assert f(*swap(good, 10 + i, v)) == SHAPE, (i, v)
    for i in (1, 3, 5, 17, 19, 21):
        assert f(*swap(good, i, 8)) == SHAPE
    assert f(*swap(good, 15, 0.0)) == SHAPE
    assert f(*swap(good, 22, None)) == WORKSPACE and f(*swap(good, 23, 64)) == WORKSPACE
    assert f(*swap(good, 11, 0)) == 0
    n = _lib.lib().qlin_attn_bwd_workspace_bytes
    assert n(B, T, HQ, HKV, D) > 0
    for i, v in SIZES:
        assert n(*swap([B, T, HQ, HKV, D], i, v)) == 0


def test_prompt_overlaps():
    f, b = _lib.lib().qlin_attn_fwd, _lib.lib().qlin_attn_bwd
    q, kv = 2 * T * HQ * D, 2 * T * HKV * D
    good = fwd_args()
    outs = {13: q, 14: 4 * T * HQ}
    for o, n in outs.items():
        for other, m in ((0, q), (2, kv), (4, kv), (6, 4 * (B + 1)), (27 - o, outs[27 - o])):
            for at in (good[other], good[other] + (m - 1) // 16 * 16, good[other] - (n - 1) // 16 * 16):
                assert f(*swap(good, o, at)) == OVERLAP, (o, other)
    good = bwd_args()
    need = _lib.lib().qlin_attn_bwd_workspace_bytes(B, T, HQ, HKV, D)
    ins = {0: q, 2: kv, 4: kv, 6: q, 7: 4 * T * HQ, 8: q, 9: 4 * (B + 1)}
    outs = {16: q, 18: kv, 20: kv, 22: need}
    for o, n in outs.items():
        for other, m in [*ins.items(), *((p, m) for p, m in outs.items() if p != o)]:
            at = good[other] + (m - 1) // 16 * 16
            assert b(*swap(good, o, at)) == OVERLAP, (o, other)


def test_alternating_parts():
    """dq, dk, dv as columns of one matrix: apart if their columns are."""
    b = _lib.lib().qlin_attn_bwd
    w = (HQ + 2 * HKV) * D

    def call(shift):
        a = bwd_args()
        a[11] = T
        base = far(30)
        a[16], a[17], a[18], a[19], a[20], a[21] = base, w, base + 2 * HQ * D, w, base + 2 * (HQ + HKV) * D + shift, w
        a[23] = 64  # (the workspace is looked at before, overlaps after it)
        return a

    n = _lib.lib().qlin_attn_bwd_workspace_bytes(B, T, HQ, HKV, D)
    for shift in (-16, 16, 2 * HKV * D):  # into dk, past the row's end into the next row's dq
        a = call(shift)
        a[23] = n
        assert b(*a) == OVERLAP
    # the same columns with inputs of another distance meet
    a = call(0)
    a[23], a[0] = n, far(30) + 16
    assert b(*a) == OVERLAP


def cache(**kw):
    f = dict(k_codes=far(0), v_codes=far(1), k_scale=far(2), v_scale=far(3), pages=10, heads=HKV, page=16, dim=D)
    f.update(kw)
    return _lib.KVCacheStruct(*f.values())


def batch(**kw):
    f = dict(cu=far(4), lens=far(5), table=far(6), batch=B, table_len=4, tokens=T)
    f.update(kw)
    return _lib.KVBatchStruct(*f.values())


def calls(c, s):
    """(name, status) of the three operators on a cache and a batch."""
    L = _lib.lib()
    c, s = ctypes.byref(c), ctypes.byref(s)
    return [("write", L.qlin_kv_write_q8(c, s, far(7), HKV * D, far(8), HKV * D, None)),
            ("read", L.qlin_kv_read_q8(c, s, far(7), far(8), None)),
            ("attn", L.qlin_attn_q8(c, s, far(7), HQ * D, HQ, 0.125, 64, far(8), far(9), BIG, None))]


@pytest.mark.parametrize("c,s,want", [
    *(({"pages": v}, {}, SHAPE) for v in (0, -1, (1 << 30) + 1)), *(({"heads": v}, {}, SHAPE) for v in (0, 1025)),
    *(({"page": v}, {}, SHAPE) for v in (0, 8, 24, 512, -16)), *(({"dim": v}, {}, SHAPE) for v in (0, 8, 72, 144)),
    *(({}, {"batch": v}, SHAPE) for v in (0, -1, (1 << 20) + 1)), *(({}, {"table_len": v}, SHAPE) for v in (0, (1 << 24) + 1)),
    *(({}, {"tokens": v}, SHAPE) for v in (-1, 1 << 31)),
    *(({n: None}, {}, NULL_) for n in ("k_codes", "v_codes", "k_scale", "v_scale")),
    *(({}, {n: None}, NULL_) for n in ("cu", "lens", "table")),
    *(({n: far(20) + 8}, {}, ALIGN) for n in ("k_codes", "v_codes", "k_scale", "v_scale")),
    *(({}, {n: far(20) + 2}, ALIGN) for n in ("cu", "lens", "table")),
    ({}, {"tokens": 0}, 0),
])
def test_cache_refusals(c, s, want):
    for name, got in calls(cache(**c), batch(**s)):
        assert got == want, name


def test_cache_call_refusals():
    L = _lib.lib()
    c, s = ctypes.byref(cache()), ctypes.byref(batch())
    w, r, a = L.qlin_kv_write_q8, L.qlin_kv_read_q8, L.qlin_attn_q8
    good_w, good_r = [c, s, far(7), HKV * D, far(8), HKV * D, None], [c, s, far(7), far(8), None]
    good_a = [c, s, far(7), HQ * D, HQ, 0.125, 64, far(8), far(9), BIG, None]
    for f, good, ptrs in ((w, good_w, (2, 4)), (r, good_r, (2, 3)), (a, good_a, (2, 7))):
        assert f(*swap(good, 0, None)) == NULL_ and f(*swap(good, 1, None)) == NULL_
        for i in ptrs:
            assert f(*swap(good, i, None)) == NULL_ and f(*swap(good, i, far(20) + 8)) == ALIGN
    for i in (3, 5):
        assert w(*swap(good_w, i, HKV * D - 8)) == SHAPE and w(*swap(good_w, i, HKV * D + 4)) == SHAPE
    for i, v in ((3, HQ * D + 4), (4, 0), (4, 7), (4, 4098), (5, 0.0), (5, float("nan")), (6, 0), (6, (1 << 30) + 1)):
        assert a(*swap(good_a, i, v)) == SHAPE, (i, v)
    assert a(*swap(good_a, 8, None)) == WORKSPACE and a(*swap(good_a, 9, 64)) == WORKSPACE
    assert a(*swap(good_a, 8, far(20) + 8)) == ALIGN
    n = L.qlin_attn_q8_workspace_bytes
    assert n(c, s, HQ, 64) > 0 and n(c, s, 7, 64) == 0 and n(c, s, HQ, 0) == 0 and n(None, s, HQ, 64) == 0


def test_cache_overlaps():
    L = _lib.lib()
    c, s = cache(), batch()
    codes, scales = 10 * HKV * 16 * D, 4 * 10 * HKV * 16
    memory = {"k_codes": codes, "v_codes": codes, "k_scale": scales, "v_scale": scales}
    arrays = {"cu": 4 * (B + 1), "lens": 4 * B, "table": 4 * B * 4}
    rows = 2 * T * HKV * D
    good_a = [ctypes.byref(c), ctypes.byref(s), far(7), HQ * D, HQ, 0.125, 64, far(8), far(9), BIG, None]
    need = L.qlin_attn_q8_workspace_bytes(good_a[0], good_a[1], HQ, 64)
    for x, n in [*memory.items(), *arrays.items()]:
        at = getattr(c if x in memory else s, x) + (n - 1) // 16 * 16
        assert L.qlin_kv_read_q8(ctypes.byref(c), ctypes.byref(s), at, far(8), None) == OVERLAP
        assert L.qlin_kv_read_q8(ctypes.byref(c), ctypes.byref(s), far(7), at, None) == OVERLAP
        assert L.qlin_attn_q8(*swap(good_a, 7, at)) == OVERLAP and L.qlin_attn_q8(*swap(good_a, 8, at)) == OVERLAP
    assert L.qlin_kv_read_q8(ctypes.byref(c), ctypes.byref(s), far(7), far(7) + rows - 16, None) == OVERLAP
    for at in (far(7) + 2 * T * HQ * D - 16, far(9) + (need - 1) // 16 * 16):
        assert L.qlin_attn_q8(*swap(good_a, 7, at)) == OVERLAP
    for x, n in memory.items():  # the cache over its inputs and over itself
        for other, m in ((far(7), rows), (far(8), rows), (far(4), 4 * (B + 1)), (far(5), 4 * B), (far(6), 16 * B),
                         *((getattr(c, y), k) for y, k in memory.items() if y != x)):
            bad = cache(**{x: other + (m - 1) // 16 * 16})
            assert L.qlin_kv_write_q8(ctypes.byref(bad), ctypes.byref(s), far(7), HKV * D, far(8), HKV * D, None) == OVERLAP


def test_launch_limits():
    """Sizes whose launches would pass 2^32 threads are refused, or not split further."""
    L = _lib.lib()
    n = L.qlin_attn_bwd_workspace_bytes
    assert n(1 << 20, 1 << 20, 4, 4, 64) > 0 and n(1 << 20, 1 << 20, 5, 5, 64) == 0
    assert n(1, (1 << 24) - 1, 64, 8, 64) > 0 and n(1, 1 << 24, 64, 8, 64) == 0
    assert L.qlin_attn_fwd(*swap(swap(fwd_args(), 7, 1 << 20), 10, HQ)) == SHAPE
    w = L.qlin_attn_q8_workspace_bytes

    def shares(b, tokens, heads, hq, length):
        c, s = cache(heads=heads, page=256), batch(batch=b, table_len=1 << 22, tokens=tokens)
        one = w(ctypes.byref(c), ctypes.byref(s), hq, 1)  # (not in shares)
        rest = w(ctypes.byref(c), ctypes.byref(s), hq, length) - one
        assert one > 0 and rest >= 0
        return max(1, rest // (tokens * hq * (D + 2) * 4))

    assert shares(1, 1, 1, 1, 1 << 30) > 1
    for b, tokens, heads, hq in ((32, 32, 8, 8), (1 << 10, 1 << 10, 8, 64), (1 << 17, 1 << 17, 8, 32), (1 << 20, 1 << 20, 4, 16),
                                 (1 << 20, 1 << 20, 4, 64), (1, 20000, 2, 64), (3, 1, 1, 128)):
        n = shares(b, tokens, heads, hq, 1 << 30)
        few = tokens * (hq // heads) <= 64 * b
        launched = (tokens * (hq // heads) // (32 if few else 256) + b) * heads * n
        assert launched < 1 << 24 and (n == 1 or (tokens * hq + 3) // 4 < 1 << 24), (b, tokens, n)
