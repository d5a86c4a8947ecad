"""Outputs that overlap an input, another output or the workspace are refused
by the 8-bit row operators before anything reaches a GPU: their kernels read
rows again after parts of the outputs are stored."""

import ctypes
import os

import pytest

from quantized_base_rank_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libqlin.so not built (run __graft_entry__.build())")

OVERLAP = 8
M, D, N, R = 6, 128, 64, 8


def far(i):
    """Addresses 4 GiB apart."""
    return (i + 1) << 32


def qw():
    p = far(40)
    return _lib.QWeightStruct(2, 32, 0, 0, N, D, p, p, p, p, p)


# entry point -> (arguments, {position of an output: bytes}, {position of an input: bytes})
def cases():
    L = _lib.lib()
    w = qw()
    rms_ws = L.qlin_rmsnorm_workspace_bytes(M, D)
    mul_ws = L.qlin_w8a8_workspace_bytes(M, N, D)
    bwd_ws = L.qlin_bwd_q8_workspace_bytes(ctypes.byref(w), M, R, 1)
    return {
        "qlin_quantize_q8": ([far(0), 2, M, D, far(1), far(2), far(3), None],
                             {4: M * D, 5: 4 * M, 6: 2 * M * D}, {0: 4 * M * D}),
        "qlin_dequant_q8": ([far(0), far(1), M, D, far(2), None], {4: 2 * M * D}, {0: M * D, 1: 4 * M}),
        "qlin_rmsnorm_q8": ([far(0), far(1), far(2), M, D, 1e-5, far(3), far(4), far(5), far(6), far(7), None],
                            {6: 2 * M * D, 7: M * D, 8: 4 * M, 9: 4 * M, 10: 2 * M * D},
                            {0: 2 * M * D, 1: 2 * M * D, 2: 2 * D}),
        "qlin_rmsnorm_bwd": ([far(0), far(1), far(2), far(3), far(4), M, D, far(5), far(6), far(7), rms_ws, None],
                             {7: 2 * M * D, 8: 4 * D, 9: rms_ws},
                             {0: 2 * M * D, 1: 2 * D, 2: 4 * M, 3: 2 * M * D, 4: 2 * M * D}),
        "qlin_w8a8_fwd": ([far(0), far(1), M, far(2), far(3), N, D, far(4), far(5), mul_ws, None],
                          {7: 2 * M * N, 8: mul_ws}, {0: M * D, 1: 4 * M, 3: N * D, 4: 4 * N}),
        "qlin_bwd_q8": ([ctypes.pointer(w), far(0), far(1), M, far(2), far(3), R, 2.0, 1, far(4), far(5), far(6), far(7),
                         far(8), far(9), bwd_ws, None],
                        {11: 2 * M * D, 12: 2 * R * D, 13: 2 * N * R, 14: bwd_ws},
                        {1: M * D, 2: 4 * M, 4: 2 * R * D, 5: 2 * N * R, 9: 2 * M * N, 10: 4 * M * R}),
    }


@pytest.mark.parametrize("name", ["qlin_quantize_q8", "qlin_dequant_q8", "qlin_rmsnorm_q8", "qlin_rmsnorm_bwd",
                                  "qlin_w8a8_fwd", "qlin_bwd_q8"])
def test_overlapping_outputs_are_refused(name):
    f = getattr(_lib.lib(), name)
    args, outs, ins = cases()[name]
    assert all(n > 16 for n in [*outs.values(), *ins.values()])
    for o, n in outs.items():
        for other, m in [*ins.items(), *((p, m) for p, m in outs.items() if p != o)]:
            # the same start; the last 16 bytes of one in the first 16 of the other
            for at in (args[other], args[other] + (m - 1) // 16 * 16, args[other] - (n - 1) // 16 * 16):
                bad = list(args)
                bad[o] = at
                assert f(*bad) == OVERLAP, (name, o, other)


def test_status_has_a_text():
    assert b"overlap" in _lib.lib().qlin_status_string(OVERLAP)
