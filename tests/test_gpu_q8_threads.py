"""Host threads that issue calls of several launches on one stream, each
through the binding's workspace: every result equals the one computed alone."""

import threading

import numpy as np
import pytest

from tests.gpu_util import to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_base_rank_amd as qb
    qb._lib.lib()
    return qb


def _bf16(a):
    from quantized_base_rank_amd.inputs import bf16_bits
    return to_dev_bf16(bf16_bits(np.asarray(a, np.float32)))


def test_threads_on_one_stream(qb):
    import torch
    rng = np.random.default_rng(21)

    def norm_gradient():
        M, d = 300, 1000
        h, dy = _bf16(rng.standard_normal((M, d))), _bf16(rng.standard_normal((M, d)))
        gamma, rstd = _bf16(rng.standard_normal(d)), to_dev_f32(rng.uniform(0.5, 2, M).astype(np.float32))
        return lambda: qb.qlin_rmsnorm_bwd(h, gamma, rstd, dy)

    def product(M, N, K):
        def rows(n):
            return qb.Q8Rows(torch.from_numpy(rng.integers(-127, 128, (n, K)).astype(np.int8)).cuda(),
                             to_dev_f32(rng.uniform(0.5, 2, n).astype(np.float32)))
        x, w = rows(M), rows(N)
        return lambda: (qb.qlin_w8a8_fwd(x, w),)

    def backward():
        M, N, K, r = 700, 512, 768, 24
        w = qb.qlin_quantize_int4_group(to_dev_f32((rng.standard_normal((N, K)) * 0.02).astype(np.float32)), 32)
        x = qb.qlin_quantize_q8(_bf16(rng.standard_normal((M, K))))
        A, B = _bf16(rng.standard_normal((r, K)) * 0.1), _bf16(rng.standard_normal((N, r)) * 0.1)
        dy, u = _bf16(rng.standard_normal((M, N))), to_dev_f32(rng.standard_normal((M, r)).astype(np.float32))
        return lambda: qb.qlin_bwd_q8(w, x, A, B, r, 2.0, dy, u)

    work = [norm_gradient(), norm_gradient(), product(100, 512, 4096), product(3, 70, 8192), backward(), backward()]
    alone = [[t.clone() for t in f()] for f in work]
    torch.cuda.synchronize()
    got, errors = [None] * len(work), []

    def body(i):
        try:
            got[i] = [work[i]() for _ in range(40)]
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=body, args=(i,)) for i in range(len(work))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, want in enumerate(alone):
        for out in got[i]:
            for a, b in zip(want, out):
                assert torch.equal(a, b), i
