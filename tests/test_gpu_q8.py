"""8-bit row operators on the GPU against the float64 oracle: rows to 8 bits,
the norm with an 8-bit output and its gradient, the 8-bit product and the
layer's backward pass from an 8-bit checkpoint.

Tolerances come from the arithmetic the operators state.  u = 2^-24 is the
relative error of one fp32 rounding and 2^-8 that of one bf16 rounding (8 significant bits); a sum
of n fp32 terms, taken by threads of one wave or more, has at most n / 64 + 32
roundings on any path (SUM below)."""

import numpy as np
import pytest

from oracle import q8_oracle as Q
from tests import parity
from tests.gpu_util import bf16_host_bits, host, to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def SUM(n):
    return (n / 64 + 32) * U


@pytest.fixture(scope="module")
def qb():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_base_rank_amd as qb
    qb._lib.lib()
    return qb


def bf16(a):
    from quantized_base_rank_amd.inputs import bf16_bits
    return bf16_bits(a)


def val(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def rows(rng, M, d, outliers=True):
    """Gaussian rows with a few large columns, one row of zeros when M > 3."""
    x = rng.standard_normal((M, d)).astype(np.float32)
    if outliers and d > 8:
        x[:, rng.integers(0, d, max(1, d // 500))] *= 20
    if M > 3:
        x[M // 2] = 0
    return x


def same_codes(q, codes, scale):
    assert np.array_equal(host(q.codes), codes)
    assert np.array_equal(host(q.scale).view(np.uint32)[np.isfinite(scale)], scale.view(np.uint32)[np.isfinite(scale)])
    assert np.array_equal(np.isnan(host(q.scale)), np.isnan(scale))


def values_of(codes, scale):
    """bf16 bits of the fp32 product of code and scale."""
    return bf16(codes.astype(np.float32) * scale.astype(np.float32)[:, None])


# ------------------------------------------------------------ rows to 8 bits

SIZES = [(1, 1), (3, 7), (1, 4096), (5, 64), (257, 5003), (130, 8192), (2, 28672), (2, 131072), (9, 1001),
         (1000, 48), (33, 520), (4, 16392), (3, 40001), (3, 1500), (3, 6144), (5, 11008), (3, 12290), (2, 20000),
         (3, 24575), (2, 32768)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_to_8_bits(qb, M, d, dtype):
    import torch
    print(f"[q8] {M}x{d} {dtype}", flush=True)
    rng = np.random.default_rng(M * 7 + d)
    x = rows(rng, M, d)
    if dtype == "bf16":
        x = val(bf16(x))
        # the largest magnitude halved is an exact tie (63.5)
        if d > 2:
            x[:, d // 2] = x[np.arange(M), np.abs(x).argmax(axis=1)] / 2
        dev = to_dev_bf16(bf16(x))
    else:
        dev = to_dev_f32(x)
    v = torch.full((M, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q = qb.qlin_quantize_q8(dev, values=v)
    codes, scale = Q.quantize_rows(x)
    same_codes(q, codes, scale)
    assert np.array_equal(bf16_host_bits(v), values_of(codes, scale))
    assert np.array_equal(bf16_host_bits(qb.qlin_dequant_q8(q)), values_of(codes, scale))
    q2 = qb.qlin_quantize_q8(dev)
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scale, q2.scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [33, 2048])
def test_rows_to_8_bits_special_values(qb, dtype, d):
    rng = np.random.default_rng(3)
    x = val(bf16(rng.standard_normal((12, d)).astype(np.float32)))
    x[0, 5], x[1, 0], x[2, d - 1], x[3, 7] = np.nan, np.inf, -np.inf, -np.nan
    x[4] = 0
    x[4, 9] = -0.0
    x[5] *= np.float32(2.0 ** 125)      # near the top of the range
    x[6] *= np.float32(2.0 ** -124)     # subnormal rows
    x[7] = 0
    x[7, 3] = np.float32(2.0 ** -133)   # smallest bf16
    x[8] = -3.0
    x[9] *= np.float32(2.0 ** -110)
    x[10, 0] = np.float32(3.3895e38)    # largest bf16
    x = val(bf16(x))
    q = qb.qlin_quantize_q8(to_dev_bf16(bf16(x)) if dtype == "bf16" else to_dev_f32(x))
    codes, scale = Q.quantize_rows(x)
    assert np.array_equal(host(q.codes)[:7], codes[:7])
    same_codes(q, codes, scale)


def test_rows_past_32_bit_offsets(qb):
    """More than 2^32 elements: the last rows are where a 32-bit offset would go wrong."""
    import torch
    M, d = 32800, 131072
    x = torch.zeros((M, d), dtype=torch.bfloat16, device="cuda")
    tail = rows(np.random.default_rng(0), 3, d)
    x[-3:] = to_dev_bf16(bf16(tail))
    q = qb.qlin_quantize_q8(x)
    codes, scale = Q.quantize_rows(val(bf16(tail)))
    same_codes(qb.Q8Rows(q.codes[-3:], q.scale[-3:]), codes, scale)
    assert int(q.codes[0].count_nonzero()) == 0 and float(q.scale[:-3].abs().max()) == 0
    back = qb.qlin_dequant_q8(q)
    assert np.array_equal(bf16_host_bits(back[-3:]), values_of(codes, scale))


# -------------------------------------------------------------------- norm

def check_norm(qb, x, res, gamma, eps, want_values=True):
    M, d = x.shape
    h, q, rstd, v = qb.qlin_rmsnorm_q8(to_dev_bf16(bf16(x)), to_dev_bf16(bf16(gamma)), eps,
                                       residual=None if res is None else to_dev_bf16(bf16(res)),
                                       want_values=want_values)
    h64, r64, y64 = Q.rmsnorm(x, gamma, eps, res)
    ok = np.isfinite(y64).all(axis=1)
    if res is None:
        assert h is None
    else:
        got = val(bf16_host_bits(h)).astype(np.float64)
        assert (np.abs(got - h64)[ok] <= np.abs(h64)[ok] * (BF + 2 * U) + 2.0 ** -134).all()
    e_r = SUM(d) / 2 + 4 * U     # half the relative error of the sum of squares, then mean, eps, root, reciprocal
    e_y = e_r + 4 * U            # the sum's rounding, two products
    assert (np.abs(host(rstd) - r64)[ok] <= r64[ok] * e_r).all()
    a = np.abs(y64).max(axis=1)
    s = host(q.scale).astype(np.float64)
    codes = host(q.codes).astype(np.float64)
    assert np.isnan(s[~ok]).all() and (codes[~ok] == 0).all() and np.isnan(host(rstd)[~ok]).all()
    assert (np.abs(s - a / 127)[ok] <= a[ok] / 127 * (e_y + 2 * U)).all()
    safe = np.where(a > 0, a, 1)[:, None]
    assert (np.abs(codes - 127 * np.where(ok[:, None], y64, 0) / safe)[ok] <= 0.5 + 127 * (2 * e_y + 4 * U)).all()
    if want_values:
        assert np.array_equal(bf16_host_bits(v)[ok], values_of(host(q.codes), host(q.scale))[ok])
        assert np.isnan(val(bf16_host_bits(v))[~ok]).all()
    else:
        assert v is None


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("res", [False, True])
def test_norm(qb, M, d, res):
    print(f"[norm] {M}x{d} res={res}", flush=True)
    rng = np.random.default_rng(M + 3 * d)
    x = val(bf16(rows(rng, M, d)))
    r = val(bf16(rows(rng, M, d))) if res else None
    gamma = val(bf16(1 + 0.2 * rng.standard_normal(d)))
    check_norm(qb, x, r, gamma, 1e-5, want_values=(M + d) % 2 == 0)


@pytest.mark.parametrize("d", [24, 1000, 4096])
def test_norm_special_values(qb, d):
    rng = np.random.default_rng(d)
    x = val(bf16(rng.standard_normal((9, d))))
    res = val(bf16(rng.standard_normal((9, d))))
    gamma = val(bf16(1 + 0.2 * rng.standard_normal(d)))
    gamma[3] = 0
    x[0, 1], x[1, 2], res[2, 0] = np.nan, np.inf, -np.inf
    x[3], res[3] = 0, 0
    x[4] = -res[4]                       # a sum of zeros
    x[5] *= np.float32(2.0 ** -60)
    res[5] = 0
    x[6] *= np.float32(2.0 ** 50)
    with np.errstate(all="ignore"):
        check_norm(qb, x, res, gamma, 1e-5)
        check_norm(qb, x[5:], res[5:], gamma, 0.0)
    # eps = 0 on a row of zeros, and squares past fp32's range: non-finite rows
    z = np.zeros((2, d), np.float32)
    z[1] = val(bf16(np.full(d, 2.0 ** 70)))
    h, q, rstd, v = qb.qlin_rmsnorm_q8(to_dev_bf16(bf16(z)), to_dev_bf16(bf16(gamma)), 0.0, want_values=True)
    assert np.isnan(host(q.scale)).all() and (host(q.codes) == 0).all() and np.isnan(host(rstd)).all()


@pytest.mark.parametrize("M,d", SIZES + [(700, 300), (4096, 40)])
@pytest.mark.parametrize("dh", [False, True])
def test_norm_gradient(qb, M, d, dh):
    import torch
    print(f"[norm bwd] {M}x{d} dh={dh}", flush=True)
    rng = np.random.default_rng(M * 5 + d)
    h = val(bf16(rows(rng, M, d)))
    dy = val(bf16(rng.standard_normal((M, d))))
    e = val(bf16(rng.standard_normal((M, d)))) if dh else None
    gamma = val(bf16(1 + 0.2 * rng.standard_normal(d)))
    rstd = (1 / np.sqrt((h.astype(np.float64) ** 2).mean(axis=1) + 1e-5)).astype(np.float32)
    args = (to_dev_bf16(bf16(h)), to_dev_bf16(bf16(gamma)), to_dev_f32(rstd), to_dev_bf16(bf16(dy)))
    dhd = to_dev_bf16(bf16(e)) if dh else None
    dx, dg = qb.qlin_rmsnorm_bwd(*args, dh=dhd)
    dx64, dg64 = Q.rmsnorm_backward(h, gamma, rstd, dy, e)
    xh = np.abs(h.astype(np.float64)) * rstd[:, None]
    g = np.abs(dy * gamma.astype(np.float64))
    size = rstd[:, None] * (g + xh * (g * xh).mean(axis=1, keepdims=True)) + (0 if e is None else np.abs(e))
    tol = np.abs(dx64) * BF + size * (SUM(d) + 10 * U)
    assert (np.abs(val(bf16_host_bits(dx)) - dx64) <= tol).all()
    tol = np.abs(dy * xh).sum(axis=0) * (M + 32) * U
    assert (np.abs(host(dg) - dg64) <= tol).all()
    dx2, dg2 = qb.qlin_rmsnorm_bwd(*args, dh=dhd)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_norm_gradient_non_finite_row(qb):
    """A NaN reciprocal norm spoils its own row of dx and no other."""
    rng = np.random.default_rng(2)
    M, d = 6, 512
    h, dy = (val(bf16(rng.standard_normal((M, d)))) for _ in range(2))
    rstd = np.ones(M, np.float32)
    rstd[2] = np.nan
    gamma = np.ones(d, np.float32)
    dx, dg = qb.qlin_rmsnorm_bwd(to_dev_bf16(bf16(h)), to_dev_bf16(bf16(gamma)), to_dev_f32(rstd), to_dev_bf16(bf16(dy)))
    bad = np.isnan(val(bf16_host_bits(dx))).all(axis=1)
    assert list(bad) == [m == 2 for m in range(M)] and not np.isnan(val(bf16_host_bits(dx))[~bad]).any()
    assert np.isnan(host(dg)).all()


# ----------------------------------------------------------------- product

def codes_of(rng, M, K, full=False):
    if full:
        return rng.integers(-128, 128, (M, K)).astype(np.int8)
    return np.clip(np.rint(rng.standard_normal((M, K)) * 31), -127, 127).astype(np.int8)


def dev_rows(qb, codes, scale):
    import torch
    return qb.Q8Rows(torch.from_numpy(codes).cuda(), to_dev_f32(scale))


PRODUCTS = [(1, 1, 16), (1, 4096, 4096), (2, 333, 112), (16, 512, 1024), (17, 129, 2064), (5, 5000, 11008),
            (33, 1003, 528), (64, 256, 256), (100, 300, 80), (129, 257, 4096), (256, 256, 128), (257, 513, 400),
            (300, 1030, 1040), (513, 2001, 192), (700, 96, 8192), (8, 70, 28672), (40, 40, 131056), (1, 32003, 64),
            (1024, 1024, 512), (48, 8200, 1024), (3, 16, 65536), (24, 24, 384)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(qb, M, N, K):
    import torch
    print(f"[w8a8] {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    xq, wq = codes_of(rng, M, K, full=K < 1000), codes_of(rng, N, K)
    xs, ws = (rng.uniform(0.5, 2, n).astype(np.float32) * np.float32(0.01) for n in (M, N))
    x, w = dev_rows(qb, xq, xs), dev_rows(qb, wq, ws)
    # a canary after y: rows and columns past the edges stay untouched
    buf = torch.full((M * N + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = qb.qlin_w8a8_fwd(x, w, y=buf[: M * N].view(M, N))
    ref = Q.product(xq, xs, wq, ws)
    got = val(bf16_host_bits(y)).astype(np.float64)
    assert (np.abs(got - ref) <= np.abs(ref) * (BF + 4 * U)).all(), np.abs(got - ref).max()
    assert bool((buf[M * N:] == 3.0).all())
    assert torch.equal(qb.qlin_w8a8_fwd(x, w), y)


@pytest.mark.parametrize("M,N", [(100, 300), (1000, 4096), (700, 11008), (2048, 8192)])
def test_product_depths(qb, M, N):
    """Every remainder of the depth over the turn of the ring that the operands stream through, at each tile height
    (64, 128, 192, 256 rows), and lengths that end inside a step; at (100, 300) also depths in several shares."""
    import torch
    print(f"[w8a8 depths] {M}x{N}", flush=True)
    rng = np.random.default_rng(M)
    K0 = 4000
    xq, wq = (torch.from_numpy(codes_of(rng, n, K0)).cuda() for n in (M, N))
    xs, ws = (to_dev_f32(rng.uniform(0.5, 2, n).astype(np.float32) * np.float32(0.01)) for n in (M, N))
    # (the tallest tiles are taken from about 50 steps on)
    for K in [64 * h + 16 * (h % 4) for h in [*range(1, 22), *range(51, 62)]] + ([] if M > 100 else list(range(1392, 3200, 176))):
        x, w = qb.Q8Rows(xq[:, :K].contiguous(), xs), qb.Q8Rows(wq[:, :K].contiguous(), ws)
        got = qb.qlin_w8a8_fwd(x, w).double()
        ref = (x.codes.double() @ w.codes.double().t().contiguous()) * xs.double()[:, None] * ws.double()[None]
        assert bool(((got - ref).abs() <= ref.abs() * (BF + 4 * U)).all()), K


def test_product_extreme_codes(qb):
    """Every code at the format's ends: the integer sum is exact in int32."""
    for M, N in ((3, 70), (260, 270)):
        K = 131056
        xq = np.full((M, K), -128, np.int8)
        wq = np.full((N, K), -128, np.int8)
        wq[1] = 127
        one = np.ones(M, np.float32), np.ones(N, np.float32)
        got = val(bf16_host_bits(qb.qlin_w8a8_fwd(dev_rows(qb, xq, one[0]), dev_rows(qb, wq, one[1]))))
        ref = val(bf16(Q.product(xq, one[0], wq, one[1]).astype(np.float32)))
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (40, 300, 512), (300, 300, 512)])
def test_product_non_finite_row(qb, M, N, K):
    """A row of scale NaN or infinity gives NaN (infinity) there and nowhere else."""
    rng = np.random.default_rng(0)
    xq, wq = codes_of(rng, M, K), codes_of(rng, N, K)
    xs, ws = np.ones(M, np.float32), np.ones(N, np.float32)
    xs[M - 1] = np.nan
    xq[M - 1] = 0
    ws[7] = np.nan
    got = val(bf16_host_bits(qb.qlin_w8a8_fwd(dev_rows(qb, xq, xs), dev_rows(qb, wq, ws))))
    bad = np.zeros((M, N), bool)
    bad[M - 1] = True
    bad[:, 7] = True
    assert np.array_equal(np.isnan(got), bad)


def test_product_past_32_bit_offsets(qb):
    import torch
    M, N, K = 3, 70000, 32768  # 2.3 GB of weight codes
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(1)
    tail, xq = codes_of(rng, 40, K), codes_of(rng, M, K)
    w[-40:] = torch.from_numpy(tail).cuda()
    xs, ws = np.full(M, 0.01, np.float32), np.full(N, 0.01, np.float32)
    for m in (M, 65):
        x = np.repeat(xq, -(-m // M), axis=0)[:m]
        y = qb.qlin_w8a8_fwd(dev_rows(qb, x, np.full(m, 0.01, np.float32)), qb.Q8Rows(w, to_dev_f32(ws)))
        ref = Q.product(x, np.full(m, 0.01, np.float32), tail, ws[-40:])
        got = val(bf16_host_bits(y[:, -40:]))
        assert (np.abs(got - ref) <= np.abs(ref) * (BF + 4 * U)).all()
        assert float(y[:, :-40].abs().max()) == 0


def test_product_many_rows(qb):
    """More than 2^31 outputs."""
    import torch
    M, N, K = 66000, 33000, 16
    rng = np.random.default_rng(4)
    xq, wq = codes_of(rng, M, K), codes_of(rng, N, K)
    xs, ws = np.full(M, 0.01, np.float32), np.full(N, 0.01, np.float32)
    y = qb.qlin_w8a8_fwd(dev_rows(qb, xq, xs), dev_rows(qb, wq, ws))
    for sl in (slice(0, 70), slice(M // 2, M // 2 + 70), slice(M - 70, M)):
        ref = Q.product(xq[sl], xs[sl], wq, ws)
        got = val(bf16_host_bits(y[sl]))
        assert (np.abs(got - ref) <= np.abs(ref) * (BF + 4 * U)).all()


# ------------------------------------------- backward from an 8-bit checkpoint

def int4_weight(qb, oracle, rng, N, K):
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    w = qb.qlin_quantize_int4_group(to_dev_f32(W), 32)
    return w, oracle.bf16_bits_to_f64(oracle.dequant_int4_bf16(*oracle.quantize_int4_group(W, 32), 32))


def nf4_weight(qb, oracle, rng, N, K):
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    w = qb.qlin_quantize_nf4(to_dev_f32(W), 64, 256)
    return w, oracle.bf16_bits_to_f64(oracle.dequant_nf4_bf16(*oracle.quantize_nf4(W, 64, 256)))


BWD = [("nf4", 1, 64, 64, 4, 1), ("nf4", 5, 272, 576, 16, 1), ("int4", 9, 128, 1088, 33, 32), ("nf4", 16, 1024, 4096, 64, 1),
       ("int4", 16, 512, 128, 128, 1), ("nf4", 17, 256, 320, 8, 1), ("nf4", 200, 528, 4096, 16, 1),
       ("int4", 77, 256, 448, 100, 32), ("int4", 513, 1040, 768, 48, 32), ("nf4", 1000, 272, 1728, 64, 1),
       ("nf4", 2049, 64, 192, 5, 1), ("int4", 300, 64, 11008, 128, 32), ("nf4", 130, 48, 640, 127, 1),
       ("int4", 3, 16, 64, 1, 32)]


@pytest.mark.parametrize("fmt,M,N,K,r,pool", BWD)
def test_backward_from_checkpoint(qb, oracle, fmt, M, N, K, r, pool):
    import torch
    print(f"[bwd q8] {fmt} M={M} {N}x{K} r={r} pool={pool}", flush=True)
    rng = np.random.default_rng(M + N + K + r)
    w, Wd = (int4_weight if fmt == "int4" else nf4_weight)(qb, oracle, rng, N, K)
    x = val(bf16(rows(rng, M, K, outliers=False)))
    A = val(bf16(rng.uniform(-1, 1, (r, K // pool)) / np.sqrt(K // pool)))
    B = val(bf16(rng.standard_normal((N, r)) * 0.1))
    dy = val(bf16(rng.standard_normal((M, N))))
    q = qb.qlin_quantize_q8(to_dev_bf16(bf16(x)))
    xv = Q.rows_values(*Q.quantize_rows(x))
    u = oracle.pool_sum(xv, pool) @ A.T.astype(np.float64)
    u32 = u.astype(np.float32)
    args = (to_dev_bf16(bf16(A)), to_dev_bf16(bf16(B)), r, 2.0, to_dev_bf16(bf16(dy)), to_dev_f32(u32))
    dx, dA, dB = qb.qlin_bwd_q8(w, q, *args, pool=pool)
    dX_ref, dA_ref, dB_ref, _ = oracle.lora_backward(Wd, xv, A, B, 2.0, dy, pool, u=u32.astype(np.float64))
    parity.check({"dX": (val(bf16_host_bits(dx)), dX_ref), "dA": (val(bf16_host_bits(dA)), dA_ref),
                  "dB": (val(bf16_host_bits(dB)), dB_ref)})
    none, dA2, dB2 = qb.qlin_bwd_q8(w, q, *args, pool=pool, need_dx=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)


@pytest.mark.parametrize("fmt,M,N,K,pool", [("int4", 17, 4096, 320, 32), ("nf4", 100, 2064, 576, 1), ("nf4", 257, 1168, 256, 1),
                                            ("int4", 300, 720, 128, 1), ("nf4", 40, 11008, 64, 1), ("nf4", 33, 272, 4160, 1),
                                            ("int4", 513, 1040, 22144, 32)])
def test_backward_input_gradient_in_shares(qb, oracle, fmt, M, N, K, pool):
    """dX of few tiles, or of the few left after whole rounds: the sum over the output features split between
    workgroups, last shares that end inside a step, and a non-finite dY row that stays in its token; the same bits
    from run to run."""
    import torch
    print(f"[bwd q8 shares] {fmt} M={M} {N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    r = 12
    w, Wd = (int4_weight if fmt == "int4" else nf4_weight)(qb, oracle, rng, N, K)
    xv = Q.rows_values(*Q.quantize_rows(val(bf16(rng.standard_normal((M, K))))))
    q = qb.qlin_quantize_q8(to_dev_bf16(bf16(val(bf16(xv)))))
    A = val(bf16(rng.uniform(-1, 1, (r, K // pool)) / np.sqrt(K // pool)))
    B = val(bf16(rng.standard_normal((N, r)) * 0.1))
    dy = val(bf16(rng.standard_normal((M, N))))
    u = rng.standard_normal((M, r)).astype(np.float32)
    args = (to_dev_bf16(bf16(A)), to_dev_bf16(bf16(B)), r, 2.0, to_dev_bf16(bf16(dy)), to_dev_f32(u))
    dx, _, _ = qb.qlin_bwd_q8(w, q, *args, pool=pool)
    du = 2.0 * (dy.astype(np.float64) @ B)
    ref = dy.astype(np.float64) @ Wd + np.repeat(du @ A.astype(np.float64), pool, axis=1)
    parity.check({"dX": (val(bf16_host_bits(dx)), ref)})
    assert torch.equal(qb.qlin_bwd_q8(w, q, *args, pool=pool)[0], dx)
    bad = dy.copy()
    bad[M // 2, N - 1] = np.inf
    dxb, _, _ = qb.qlin_bwd_q8(w, q, args[0], args[1], r, 2.0, to_dev_bf16(bf16(bad)), args[5], pool=pool)
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(dxb[keep], dx[keep]) and not bool(torch.isfinite(dxb[M // 2].float()).all())


def test_backward_checkpoint_gradient_by_differences(qb, oracle):
    """dA against central differences of <dY, y> in the oracle's forward on
    the checkpoint's values: linear in A, so differences are exact up to
    rounding and only the bf16 rounding of dA remains."""
    rng = np.random.default_rng(8)
    M, N, K, r, pool = 40, 64, 256, 6, 32
    w, Wd = int4_weight(qb, oracle, rng, N, K)
    q = qb.qlin_quantize_q8(to_dev_bf16(bf16(rng.standard_normal((M, K)))))
    xv = Q.rows_values(host(q.codes), host(q.scale))
    A = val(bf16(rng.standard_normal((r, K // pool)) * 0.1)).astype(np.float64)
    B = val(bf16(rng.standard_normal((N, r)) * 0.1)).astype(np.float64)
    dy = val(bf16(rng.standard_normal((M, N)))).astype(np.float64)
    _, u = oracle.lora_forward(Wd, xv, A, B, 2.0, pool)
    _, dA, dB = qb.qlin_bwd_q8(w, q, to_dev_bf16(bf16(A)), to_dev_bf16(bf16(B)), r, 2.0, to_dev_bf16(bf16(dy)),
                               to_dev_f32(u.astype(np.float32)), pool=pool)
    f = lambda A, B: (dy * oracle.lora_forward(Wd, xv, A, B, 2.0, pool)[0]).sum()  # noqa: E731
    dA, dB = val(bf16_host_bits(dA)), val(bf16_host_bits(dB))
    scale = np.abs(dA).max()
    for j in range(r):
        for g in range(K // pool):
            E = np.zeros_like(A); E[j, g] = 1.0
            assert abs((f(A + E, B) - f(A - E, B)) / 2 - dA[j, g]) <= 4 * BF * max(abs(dA[j, g]), 1e-3 * scale)
    E = np.zeros_like(B); E[5, 3] = 1.0
    assert abs((f(A, B + E) - f(A, B - E)) / 2 - dB[5, 3]) <= 4 * BF * abs(dB[5, 3])


# --------------------------------------------------- streams, graphs, chains

def test_other_stream_and_graph(qb, oracle):
    """The chain norm -> product -> layer backward -> norm gradient, eagerly,
    on another stream, and captured in a graph and replayed with the program's
    own work in between: bit-identical."""
    import torch
    rng = np.random.default_rng(11)
    M, N, K, r = 150, 512, 1024, 16
    w, _ = nf4_weight(qb, oracle, rng, N, K)
    x, res = (to_dev_bf16(bf16(rows(rng, M, K))) for _ in range(2))
    gamma = to_dev_bf16(bf16(1 + 0.2 * rng.standard_normal(K)))
    w8 = qb.qlin_quantize_q8(to_dev_f32((rng.standard_normal((300, K)) * 0.02).astype(np.float32)))
    A = to_dev_bf16(bf16(rng.uniform(-1, 1, (r, K)) / 32))
    B = to_dev_bf16(bf16(rng.standard_normal((N, r)) * 0.1))
    dy = to_dev_bf16(bf16(rng.standard_normal((M, N))))
    need = max(qb.qlin_workspace_bytes(w, M, r), 1 << 22)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def step():
        h, q, rstd, v = qb.qlin_rmsnorm_q8(x, gamma, 1e-5, residual=res, want_values=True)
        y8 = qb.qlin_w8a8_fwd(q, w8, ws=ws)
        y, u = qb.qlin_fwd(w, v, A, B, r, 2.0, ws=ws)
        dv, dA, dB = qb.qlin_bwd_q8(w, q, A, B, r, 2.0, dy, u, ws=ws)
        dx, dg = qb.qlin_rmsnorm_bwd(h, gamma, rstd, dv, dh=res, ws=ws)
        return h, q.codes, q.scale, y8, y, dA, dB, dx, dg

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(4):
        for t in out:
            t.zero_()
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, out):
            assert torch.equal(a, b)


def test_graph_with_the_binding_s_workspace(qb):
    """Captured without a workspace of the caller's: the graph keeps its own,
    and eager calls in between that make the stream's grow leave it alone."""
    import torch
    rng = np.random.default_rng(12)
    x = dev_rows(qb, codes_of(rng, 4, 8192), np.ones(4, np.float32))
    w = dev_rows(qb, codes_of(rng, 64, 8192), np.ones(64, np.float32))  # K in shares: counters and sums
    big = dev_rows(qb, codes_of(rng, 200, 4096), np.ones(200, np.float32))
    bigw = dev_rows(qb, codes_of(rng, 3000, 4096), np.ones(3000, np.float32))
    eager = qb.qlin_w8a8_fwd(x, w).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = qb.qlin_w8a8_fwd(x, w)
    first = qb.qlin_w8a8_fwd(big, bigw).clone()
    for _ in range(4):
        y.zero_()
        assert torch.equal(qb.qlin_w8a8_fwd(x, w), eager)
        g.replay()
        assert torch.equal(qb.qlin_w8a8_fwd(big, bigw), first)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


@pytest.mark.parametrize("d", [9000, 16384, 20000, 32768])
def test_norm_gradient_wide_rows(qb, d):
    rng = np.random.default_rng(d)
    M = 37
    h, dy = (val(bf16(rng.standard_normal((M, d)))) for _ in range(2))
    gamma = val(bf16(1 + 0.2 * rng.standard_normal(d)))
    rstd = (1 / np.sqrt((h.astype(np.float64) ** 2).mean(axis=1) + 1e-5)).astype(np.float32)
    dx, dg = qb.qlin_rmsnorm_bwd(to_dev_bf16(bf16(h)), to_dev_bf16(bf16(gamma)), to_dev_f32(rstd), to_dev_bf16(bf16(dy)))
    dx64, dg64 = Q.rmsnorm_backward(h, gamma, rstd, dy)
    xh = np.abs(h.astype(np.float64)) * rstd[:, None]
    gy = np.abs(dy * gamma.astype(np.float64))
    size = rstd[:, None] * (gy + xh * (gy * xh).mean(axis=1, keepdims=True))
    assert (np.abs(val(bf16_host_bits(dx)) - dx64) <= np.abs(dx64) * BF + size * (SUM(d) + 10 * U)).all()
    assert (np.abs(host(dg) - dg64) <= np.abs(dy * xh).sum(axis=0) * (M + 32) * U).all()


def test_binding_refuses(qb):
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q = qb.qlin_quantize_q8(x)
    for bad in (x.half(), x[:, ::2], x.cpu(), x[0]):
        with pytest.raises(ValueError):
            qb.qlin_quantize_q8(bad)
    with pytest.raises(ValueError):
        qb.qlin_rmsnorm_q8(x, x[0, :32], 1e-5)
    with pytest.raises(ValueError):
        qb.qlin_w8a8_fwd(q, qb.Q8Rows(q.codes[:, :32].contiguous(), q.scale))
    with pytest.raises(qb.QlinError):
        qb.qlin_quantize_q8(x[:0])
    with pytest.raises(qb.QlinError):
        qb.qlin_w8a8_fwd(qb.qlin_quantize_q8(torch.zeros((2, 24), dtype=torch.bfloat16, device="cuda")),
                         qb.qlin_quantize_q8(torch.zeros((2, 24), dtype=torch.bfloat16, device="cuda")))
