"""A row of scale NaN (it held NaN or an infinity) in the backward pass from
an 8-bit checkpoint: sums over the rows take it up, everything else does not."""

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


@pytest.mark.parametrize("M,r,pool", [(3, 5, 1), (16, 16, 32), (70, 33, 1), (300, 64, 32), (1200, 100, 1)])
def test_backward_from_a_row_of_scale_nan(qb, M, r, pool):
    import torch
    rng = np.random.default_rng(M + r)
    N, K = 272, 576
    w = qb.qlin_quantize_int4_group(to_dev_f32((rng.standard_normal((N, K)) * 0.02).astype(np.float32)), 32)
    x = rng.standard_normal((M, K)).astype(np.float32)
    args = (_bf16(rng.standard_normal((r, K // pool)) * 0.1), _bf16(rng.standard_normal((N, r)) * 0.1), r, 2.0,
            _bf16(rng.standard_normal((M, N))), to_dev_f32(rng.standard_normal((M, r)).astype(np.float32)))
    dx, dA, dB = qb.qlin_bwd_q8(w, qb.qlin_quantize_q8(_bf16(x)), *args, pool=pool)
    assert bool(torch.isfinite(dA.float()).all())
    for bad in (np.nan, np.inf):
        x[M // 2, 7] = bad
        q = qb.qlin_quantize_q8(_bf16(x))
        assert bool(torch.isnan(q.scale[M // 2])) and int(torch.isnan(q.scale).sum()) == 1
        dxb, dAb, dBb = qb.qlin_bwd_q8(w, q, *args, pool=pool)
        assert torch.equal(dxb, dx) and torch.equal(dBb, dB)   # neither reads x
        assert bool(torch.isnan(dAb.float()).all())            # every element sums over the rows


@pytest.mark.parametrize("d", [5, 64, 1000, 4096, 40000])
def test_norm_of_rows_below_the_normal_range(qb, d):
    """With eps = 0, a mean square below fp32's normal numbers (2^-126) has lost its bits: a non-finite row, like one
    of zeros.  At 2^-126 and above, and with an eps that covers it, the row is as exact as any: the squares' sum is
    off by at most d roundings of 2^-150, which is 2^-24 of d 2^-126, besides its own."""
    tiny = np.full((4, d), 1.0, np.float32)
    tiny *= np.float32([2.0 ** -70, 2.0 ** -64, 2.0 ** -63, 2.0 ** -40])[:, None]
    tiny[:, 1:] *= np.float32([1.0, 1.0, -1.0, 1.0])[:, None]
    gamma = _bf16(np.ones(d))
    h, q, rstd, v = qb.qlin_rmsnorm_q8(_bf16(tiny), gamma, 0.0, want_values=True)
    assert list(np.isnan(rstd.cpu().numpy())) == [True, True, False, False]
    assert list(np.isnan(q.scale.cpu().numpy())) == [True, True, False, False]
    assert int(q.codes[:2].count_nonzero()) == 0 and bool((q.codes[2:].abs() == 127).all())
    u = 2.0 ** -24
    bound = (d / 64 + 32) * u / 2 + 5 * u   # half of the sum's error, then mean, root, reciprocal
    want = np.float64([2.0 ** 63, 2.0 ** 40])
    assert (np.abs(rstd.cpu().numpy()[2:] - want) <= want * bound).all()
    # eps = 2^-60 covers the first two
    _, q, rstd, _ = qb.qlin_rmsnorm_q8(_bf16(tiny), gamma, 2.0 ** -60)
    want = 1 / np.sqrt(np.float64([2.0 ** -140, 2.0 ** -128, 2.0 ** -126, 2.0 ** -80]) + 2.0 ** -60)
    assert (np.abs(rstd.cpu().numpy() - want) <= want * bound).all()
    assert bool((q.codes.abs() == 127).all())
