"""The 8-bit row operators on memory of one buffer: neighbouring tensors are
taken, an output in the place of an input is refused."""

import numpy as np
import pytest

from tests.gpu_util import to_dev_bf16

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


def test_in_place_is_refused(qb):
    import torch
    rng = np.random.default_rng(1)
    M, d = 5, 96
    x, res, dh = (_bf16(rng.standard_normal((M, d))) for _ in range(3))
    gamma, rstd = _bf16(np.ones(d)), torch.ones(M, device="cuda")
    for call in (lambda: qb.qlin_rmsnorm_q8(x, gamma, 1e-5, residual=res, h=res),
                 lambda: qb.qlin_rmsnorm_q8(x, gamma, 1e-5, residual=res, h=x),
                 lambda: qb.qlin_rmsnorm_q8(x, gamma, 1e-5, values=x),
                 lambda: qb.qlin_rmsnorm_bwd(x, gamma, rstd, res, dh=dh, dx=dh),
                 lambda: qb.qlin_rmsnorm_bwd(x, gamma, rstd, res, dx=res),
                 lambda: qb.qlin_quantize_q8(x, values=x)):
        before = [t.clone() for t in (x, res, dh)]
        with pytest.raises(qb.QlinError) as e:
            call()
        assert e.value.status == 8
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, (x, res, dh)))


def test_neighbours_in_one_buffer_are_taken(qb):
    import torch
    rng = np.random.default_rng(2)
    M, d = 8, 64
    buf = torch.zeros(4 * M * d, dtype=torch.bfloat16, device="cuda")
    x, res, h, v = (buf[i * M * d:(i + 1) * M * d].view(M, d) for i in range(4))
    x.copy_(_bf16(rng.standard_normal((M, d))))
    res.copy_(_bf16(rng.standard_normal((M, d))))
    gamma = _bf16(1 + 0.1 * rng.standard_normal(d))
    want = qb.qlin_rmsnorm_q8(x.clone(), gamma, 1e-5, residual=res.clone(), want_values=True)
    got = qb.qlin_rmsnorm_q8(x, gamma, 1e-5, residual=res, h=h, values=v)
    for a, b in zip((want[0], want[1].codes, want[1].scale, want[2], want[3]),
                    (got[0], got[1].codes, got[1].scale, got[2], got[3])):
        assert torch.equal(a, b)
