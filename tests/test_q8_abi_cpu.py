"""Refusals of the 8-bit row operators, reported before anything reaches a
GPU, and their workspace sizes."""

import ctypes
import os

import pytest

from quantized_base_rank_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libqlin.so not built (run __graft_entry__.build())")

OK, BAD, BIG = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), 1 << 40
NULL_, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 5, 6


def _swap(args, i, v):
    return [v if j == i else a for j, a in enumerate(args)]


def test_quantize_refusals():
    f = _lib.lib().qlin_quantize_q8
    good = [OK, 1, 4, 100, OK, OK, OK, None]
    for i in (0, 4, 5):
        assert f(*_swap(good, i, None)) == NULL_
        assert f(*_swap(good, i, BAD)) == ALIGN
    assert f(*_swap(good, 6, BAD)) == ALIGN
    assert f(*_swap(good, 1, 3)) == UNSUPPORTED
    for i, v in ((2, 0), (2, -1), (2, (1 << 31) + 1), (3, 0), (3, 131073)):
        assert f(*_swap(good, i, v)) == SHAPE
    g = _lib.lib().qlin_dequant_q8
    good = [OK, OK, 4, 100, OK, None]
    for i in (0, 1, 4):
        assert g(*_swap(good, i, None)) == NULL_
        assert g(*_swap(good, i, BAD)) == ALIGN
    assert g(*_swap(good, 2, 0)) == SHAPE and g(*_swap(good, 3, 131073)) == SHAPE


def test_rmsnorm_refusals():
    f = _lib.lib().qlin_rmsnorm_q8
    good = [OK, OK, OK, 4, 100, 1e-5, OK, OK, OK, OK, OK, None]
    for i in (0, 2, 6, 7, 8):
        assert f(*_swap(good, i, None)) == NULL_
    for i in (0, 1, 2, 6, 7, 8, 9, 10):
        assert f(*_swap(good, i, BAD)) == ALIGN
    assert f(*_swap(good, 1, None)) == UNSUPPORTED  # h without a residual
    for i, v in ((3, 0), (4, 0), (4, 131073), (5, -1.0), (5, float("nan")), (5, float("inf"))):
        assert f(*_swap(good, i, v)) == SHAPE
    b = _lib.lib().qlin_rmsnorm_bwd
    good = [OK, OK, OK, OK, OK, 4, 100, OK, OK, OK, BIG, None]
    for i in (0, 1, 2, 3, 7, 8):
        assert b(*_swap(good, i, None)) == NULL_
    for i in (0, 1, 2, 3, 4, 7, 8, 9):
        assert b(*_swap(good, i, BAD)) == ALIGN
    assert b(*_swap(good, 5, 0)) == SHAPE and b(*_swap(good, 6, 131073)) == SHAPE
    assert b(*_swap(good, 9, None)) == WORKSPACE and b(*_swap(good, 10, 64)) == WORKSPACE
    n = _lib.lib().qlin_rmsnorm_workspace_bytes
    assert n(4, 100) > 0 and n(0, 100) == 0 and n(4, 0) == 0 and n(4, 131073) == 0


def test_product_refusals():
    f = _lib.lib().qlin_w8a8_fwd
    good = [OK, OK, 5, OK, OK, 77, 96, OK, OK, BIG, None]
    for i in (0, 1, 3, 4, 7):
        assert f(*_swap(good, i, None)) == NULL_
        assert f(*_swap(good, i, BAD)) == ALIGN
    for i, v in ((2, 0), (5, 0), (6, 0), (6, 8), (6, 100), (6, 131072)):
        assert f(*_swap(good, i, v)) == SHAPE
    assert f(*_swap(good, 8, None)) == WORKSPACE and f(*_swap(good, 9, 64)) == WORKSPACE
    assert f(*_swap(good, 8, BAD)) == ALIGN
    n = _lib.lib().qlin_w8a8_workspace_bytes
    assert n(5, 77, 96) > 0 and n(0, 77, 96) == 0 and n(5, 77, 100) == 0 and n(5, 77, 131072) == 0


def _qw(fmt=2, block=32, dq=0, d_out=64, d_in=128):
    p = 0x1000
    return _lib.QWeightStruct(fmt, block, dq, 0, d_out, d_in, p, p, p, p, p)


def test_backward_refusals():
    f = _lib.lib().qlin_bwd_q8
    w = _qw()
    good = [ctypes.byref(w), OK, OK, 20, OK, OK, 8, 2.0, 32, OK, OK, OK, OK, OK, OK, BIG, None]
    assert f(*_swap(good, 0, None)) == NULL_
    for i in (1, 2, 4, 5, 9, 10, 12, 13):
        assert f(*_swap(good, i, None)) == NULL_
        assert f(*_swap(good, i, BAD)) == ALIGN
    assert f(*_swap(good, 11, BAD)) == ALIGN
    for i, v in ((3, 0), (6, 0), (6, 129), (7, float("inf"))):
        assert f(*_swap(good, i, v)) == SHAPE
    assert f(*_swap(good, 8, 16)) == UNSUPPORTED
    assert f(*_swap(good, 0, ctypes.byref(_qw(fmt=1, block=64, dq=256)))) == UNSUPPORTED  # pooled needs INT4
    assert f(*_swap(good, 14, None)) == WORKSPACE and f(*_swap(good, 15, 64)) == WORKSPACE
    # dX beyond its 32-bit offsets: 256 rows of dY, the packed codes
    for m, d_out, d_in in ((256, 1 << 22, 64), (300, 1 << 23, 64), (20, 1 << 17, 1 << 16)):
        big = [ctypes.byref(_qw(d_out=d_out, d_in=d_in)), *good[1:]]
        big[3], big[15] = m, 1 << 50
        assert f(*big) == SHAPE
    n = _lib.lib().qlin_bwd_q8_workspace_bytes
    assert n(ctypes.byref(w), 20, 8, 32) > 0
    assert n(ctypes.byref(w), 20, 0, 32) == 0 and n(ctypes.byref(w), 0, 8, 32) == 0
    assert n(ctypes.byref(_qw(d_in=100)), 20, 8, 1) == 0
