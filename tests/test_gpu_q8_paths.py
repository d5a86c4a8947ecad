"""Every path that the launchers of the 8-bit row operators can take (tile
heights, shares, waves, ranks; tests/q8_plans.py lists the sizes and the host
tests check that they take them all) against float64 on the same inputs, and
the backward pass from 8-bit rows on every format of the frozen weight.

The product's bound: its integer sum is exact; one fp32 rounding of it and one
for each scale (2^-24 each), one to bf16 (2^-8).  The gradients: the bounds of
tests/parity.py for one rounding to bf16; its bound against the unrounded
reference, 2e-3, lies above the rounding's own error only for outputs of many
elements (twenty correctly rounded ones can be off by 2.04e-3 together), so
here it is that or the rounded reference's own error and the one-rounding
bound, whichever is larger."""

import pytest

from tests import parity
from tests import q8_plans as P
from tests.gpu_util import host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def qb():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_base_rank_amd as qb
    qb._lib.lib()
    return qb


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    import torch
    return torch.randn(shape, generator=g, device="cuda")


def code_rows(qb, g, n, K):
    import torch
    return qb.Q8Rows(torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8),
                     0.01 * (0.5 + 1.5 * torch.rand(n, generator=g, device="cuda")))


def val(t):
    return t.float().cpu().numpy()


def check(outputs):
    """outputs: {name: (tensor, float64 tensor)}."""
    for name, (got, ref) in outputs.items():
        got, ref = val(got), host(ref)
        e = parity.report(got, ref)
        own = parity._rel(parity.bf16_round(ref), ref)
        assert e["spec"] <= max(parity.SPEC, own + parity.ONE_BF16), (name, e, own)
        assert e["one"] <= parity.ONE_BF16 and e["local"] <= parity.LOCAL_BF16, (name, e)


# ----------------------------------------------------------------- product

@pytest.mark.parametrize("M,N,K", P.PRODUCTS)
def test_product_paths(qb, M, N, K):
    import torch
    print(f"[w8a8 path] {M}x{N}x{K} {P.product_path(M, N, K)}", flush=True)
    g = gen(M + N + K)
    x, w = code_rows(qb, g, M, K), code_rows(qb, g, N, K)
    buf = torch.full((M * N + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = qb.qlin_w8a8_fwd(x, w, y=buf[: M * N].view(M, N))
    ref = (x.codes.double() @ w.codes.double().t().contiguous()) * x.scale.double()[:, None] * w.scale.double()[None]
    off = (y.double() - ref).abs() > ref.abs() * (BF + 4 * U)
    assert not bool(off.any()), off.nonzero()[:4].tolist()
    assert bool((buf[M * N:] == 3.0).all())
    assert torch.equal(qb.qlin_w8a8_fwd(x, w), y)


# ---------------------------------------------------------------- backward

class Backward:
    """Inputs of one backward pass on random INT4 codes, and its float64 gradients."""

    def __init__(self, qb, M, N, K, r, pool):
        import torch
        g = gen(M + 3 * N + 5 * K + r)
        self.r, self.pool = r, pool
        self.w = qb.QWeight(qb.QLIN_FMT_INT4_GROUP, 32, 0, N, K,
                            torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                            scale=torch.full((N, K // 32), 0.005, dtype=torch.float16, device="cuda"),
                            zero=torch.full((N, K // 32), -0.0375, dtype=torch.float16, device="cuda"))
        self.x = qb.qlin_quantize_q8(randn(g, M, K).to(torch.bfloat16))
        self.A = (randn(g, r, K // pool) * (K // pool) ** -0.5).to(torch.bfloat16)
        self.B = (randn(g, N, r) * 0.1).to(torch.bfloat16)
        self.dy = randn(g, M, N).to(torch.bfloat16)
        self.u = randn(g, M, r)

    def run(self, qb, need_dx=False, ws=None):
        return qb.qlin_bwd_q8(self.w, self.x, self.A, self.B, self.r, 2.0, self.dy, self.u, pool=self.pool,
                              need_dx=need_dx, ws=ws)

    def exact(self):
        xv = self.x.codes.double() * self.x.scale.double()[:, None]
        xv = xv.view(xv.shape[0], -1, self.pool).sum(2)
        dy = self.dy.double()
        du = 2.0 * (dy @ self.B.double())
        return du, (du.t().contiguous() @ xv), 2.0 * (dy.t().contiguous() @ self.u.double())


@pytest.mark.parametrize("M,N,K,r,pool", P.BACKWARDS)
def test_backward_paths(qb, M, N, K, r, pool):
    import torch
    print(f"[bwd q8 path] {M} {N}x{K} r={r} pool={pool} {P.token_path(M, N, K, r)} {P.du_path(M, N, r)}", flush=True)
    b = Backward(qb, M, N, K, r, pool)
    none, dA, dB = b.run(qb)
    _, dA64, dB64 = b.exact()
    assert none is None
    check({"dA": (dA, dA64), "dB": (dB, dB64)})
    _, dA2, dB2 = b.run(qb)
    assert torch.equal(dA, dA2) and torch.equal(dB, dB2)


def test_backward_shapes_in_turn_on_one_workspace(qb):
    """Shapes whose tickets and partial sums lie differently, one after the other on one workspace."""
    import ctypes

    import torch
    cases = [Backward(qb, *c) for c in [(4096, 2048, 2176, 64, 1), (1321, 16, 64, 85, 1), (3495, 16, 64, 10, 32),
                                        (4096, 1024, 1024, 128, 1), (100, 1040, 448, 128, 1), (3279, 704, 4928, 97, 1)]]
    need = max(qb._lib.lib().qlin_bwd_q8_workspace_bytes(ctypes.byref(c.w.struct()), c.x.codes.shape[0], c.r, c.pool)
               for c in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = [c.run(qb, ws=ws)[1:] for c in cases]
    for order in ([5, 4, 3, 2, 1, 0], [2, 0, 4, 1, 5, 3]):
        for i in order:
            _, dA, dB = cases[i].run(qb, ws=ws)
            assert torch.equal(dA, first[i][0]) and torch.equal(dB, first[i][1]), i
    assert int(ws[: 1 << 16].count_nonzero()) == 0


# -------------------------------------------------- formats of the weight

FORMATS = [("nf", 3, 64, 256), ("nf", 2, 32, 0), ("nf", 4, 32, 256), ("nf", 3, 256, 0), ("nf", 2, 64, 256), ("nf4", 0, 64, 0),
           ("nf4", 0, 64, 256)]
DX = [(1, 512, 1024, 16), (5, 272, 768, 7), (16, 2064, 4352, 64), (100, 2064, 768, 33), (257, 1168, 256, 12),
      (40, 11008, 256, 4), (300, 720, 256, 100), (513, 1040, 22272, 16)]


@pytest.mark.parametrize("M,N,K,r", DX)
@pytest.mark.parametrize("fmt,bits,block,dq", FORMATS)
def test_backward_on_every_format(qb, fmt, bits, block, dq, M, N, K, r):
    """dX streamed, in shares, and whole rounds with the rest in shares; NormalFloat-k weights through their transcoded
    form, NF4 with and without double quantisation."""
    import torch
    print(f"[bwd q8 format] {fmt}{bits or ''} block={block} dq={dq} {M} {N}x{K} r={r}", flush=True)
    b = Backward(qb, M, N, K, r, 1)
    W = randn(gen(N + K), N, K) * 0.02
    b.w = qb.qlin_quantize_nf4(W, block, dq) if fmt == "nf4" else qb.qlin_quantize_nf(W, bits, block, dq)
    dx, dA, dB = b.run(qb, need_dx=True)
    du64, dA64, dB64 = b.exact()
    dx64 = b.dy.double() @ qb.qlin_dequant_bf16(b.w).double() + du64 @ b.A.double()
    check({"dX": (dx, dx64), "dA": (dA, dA64), "dB": (dB, dB64)})
    again = b.run(qb, need_dx=True)
    assert all(torch.equal(s, t) for s, t in zip((dx, dA, dB), again))
    # a non-finite value of dY stays in its token's row of dX
    keep = torch.arange(M, device="cuda") != M // 2
    b.dy = b.dy.clone()
    b.dy[M // 2, N - 1] = float("inf")
    dxb = b.run(qb, need_dx=True)[0]
    assert torch.equal(dxb[keep], dx[keep]) and not bool(torch.isfinite(dxb[M // 2].float()).all())
