"""Attention and the cache as programs use them: the same bits from run to run,
captured graphs, other streams, host threads, memory of the caller's own, many
sequences, offsets past 32 bits."""

import threading

import numpy as np
import pytest
import torch

from oracle import attn_oracle as A
from tests import attn_util as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_base_rank_amd as qb
    qb._lib.lib()
    return qb


class Step:
    """A prompt's attention and gradient, its rows into the cache, and tokens
    over it (few rows in shares, or many rows)."""

    def __init__(self, qb, seed, lens, Hq, Hkv, D, new, ctx):
        n = sum(lens)
        self.qb = qb
        self.q, self.k, self.v, self.do = (T.heads(seed + i, n, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
        self.cu = T.cu_of(lens)
        self.c = T.Paged(qb, seed + 5, ctx, new, Hkv, D, 32)
        m = sum(new)
        self.q2, self.k2, self.v2 = (T.heads(seed + i, m, h, D) for i, h in ((6, Hq), (7, Hkv), (8, Hkv)))
        self.max_len = max(ctx)

    def __call__(self):
        qb, c = self.qb, self.c
        o, lse = qb.qlin_attn_fwd(self.q, self.k, self.v, self.cu)
        dq, dk, dv = qb.qlin_attn_bwd(self.q, self.k, self.v, o, lse, self.do, self.cu)
        qb.qlin_kv_write_q8(c.cache, c.batch, self.k2, self.v2)
        o2 = qb.qlin_attn_q8(self.q2, c.cache, c.batch, max_len=self.max_len)
        k, v = qb.qlin_kv_read_q8(c.cache, c.batch, self.q2.shape[0])
        return [o, lse, dq, dk, dv, o2, k, v]


STEPS = [
    (1, [90, 33, 150], 4, 2, 128, [1, 1, 1], [700, 90, 1500]),     # few rows, shares joined
    (20, [257], 2, 2, 64, [300, 5], [900, 40]),                    # many rows
    (40, [64, 0, 7], 16, 1, 96, [20], [2100]),                     # many rows in shares
]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("case", STEPS, ids=lambda c: str(c[0]))
def test_same_bits(qb, case):
    s = Step(qb, *case)
    first = [t.clone() for t in s()]
    for _ in range(3):
        assert same(first, s())


@pytest.mark.parametrize("case", STEPS, ids=lambda c: str(c[0]))
def test_graphs(qb, case):
    """Two captured graphs, replayed in turns with the program's own work between
    them, against the eager results."""
    seeds = [case[0], case[0] + 100]
    steps = [Step(qb, s, *case[1:]) for s in seeds]
    eager = [[t.clone() for t in s()] for s in steps]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in steps:
            s()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s())
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            for t in outs[i]:
                t.zero_()
            scratch = torch.randn(1 << 18, device="cuda").sum()
            assert same(eager[1 - i], steps[1 - i]())  # eager work of the same operators
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(eager[i], outs[i]), f"replay {rep} of graph {i}"
            del scratch


def test_other_stream(qb):
    """Calls on a stream of their own while the default one is busy."""
    s = Step(qb, *STEPS[0])
    want = [t.clone() for t in s()]
    big = torch.randn((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        big = big @ big * 1e-4
    with torch.cuda.stream(side):
        got = s()
    side.synchronize()
    assert same(want, got)
    torch.cuda.synchronize()


def test_threads(qb):
    """Host threads on one stream and on streams of their own."""
    steps = [Step(qb, 200 + 20 * i, *STEPS[i % 3][1:]) for i in range(4)]
    want = [[t.clone() for t in s()] for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream() if i >= 2 else torch.cuda.default_stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got = steps[i]()
                    stream.synchronize()
                    if not same(want[i], got):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


@pytest.mark.parametrize("new,ctx,Hq,Hkv", [([1, 1], [1000, 300], 8, 2), ([40], [1500], 8, 1)])
def test_own_workspace(qb, new, ctx, Hq, Hkv):
    """A workspace of just the size that is asked for: used, never passed."""
    import ctypes
    c = T.Paged(qb, 3, ctx, new, Hkv, 64, 16)
    q = T.heads(1, sum(new), Hq, 64)
    cs, bs, _ = qb._kv_structs(c.cache, c.batch, sum(new))
    need = qb._lib.lib().qlin_attn_q8_workspace_bytes(ctypes.byref(cs), ctypes.byref(bs), Hq, max(ctx))
    assert need > 65536  # (in shares)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    o = qb.qlin_attn_q8(q, c.cache, c.batch, max_len=max(ctx), ws=ws[:need])
    c.check(q, o, 0.125)
    assert bool((ws[need:] == 0x5A).all())
    with pytest.raises(qb.QlinError):
        qb.qlin_attn_q8(q, c.cache, c.batch, max_len=max(ctx), ws=ws[:need - 16])
    lens = [70, 30]
    k, v, do = (T.heads(i, 100, h, 64) for i, h in ((2, Hkv), (3, Hkv), (4, Hq)))
    q = T.heads(5, 100, Hq, 64)
    o, lse = qb.qlin_attn_fwd(q, k, v, T.cu_of(lens))
    need = qb._lib.lib().qlin_attn_bwd_workspace_bytes(2, 100, Hq, Hkv, 64)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    dq, dk, dv = qb.qlin_attn_bwd(q, k, v, o, lse, do, T.cu_of(lens), ws=ws[:need])
    T.check_gradient(lens, Hq, Hkv, 64, q, k, v, do, dq, dk, dv, 0.125)
    assert bool((ws[need:] == 0x5A).all())


def test_many_short_sequences(qb):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, size=700).tolist()
    n, Hq, Hkv, D = sum(lens), 4, 2, 32
    q, k, v, do = (T.heads(i, n, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    cu = T.cu_of(lens)
    o, lse = qb.qlin_attn_fwd(q, k, v, cu)
    T.check_prompt(lens, Hq, Hkv, D, q, k, v, o, lse, D ** -0.5)
    dq, dk, dv = qb.qlin_attn_bwd(q, k, v, o, lse, do, cu)
    T.check_gradient(lens, Hq, Hkv, D, q, k, v, do, dq, dk, dv, D ** -0.5)
    ctx = [x + int(rng.integers(0, 60)) for x in lens]
    c = T.Paged(qb, 2, ctx, lens, Hkv, D, 16)
    c.check(q, qb.qlin_attn_q8(q, c.cache, c.batch), D ** -0.5)


@pytest.mark.parametrize("new", [[1, 1], [90, 7]])
def test_cache_past_32_bits(qb, new):
    """Codes of more than 4 GiB, sequences in its last pages."""
    H, D, page, pages = 8, 128, 64, 66000
    cache = qb.KVCache.empty(pages, H, D, page)
    assert cache.k_codes.numel() > 1 << 32
    lens = [300, 130]
    table = torch.tensor([[pages - 1, pages - 7, 65537, pages - 3, 65600], [65999 - 10, pages - 2, pages - 30, -1, -1]],
                         dtype=torch.int32, device="cuda")
    k, v = T.heads(1, sum(lens), H, D), T.heads(2, sum(lens), H, D)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    whole = qb.KVBatch(T.cu_of(lens), ln, table)
    qb.qlin_kv_write_q8(cache, whole, k, v)
    kr, vr = qb.qlin_kv_read_q8(cache, whole, sum(lens))
    kv = []
    for x, r in ((k, kr), (v, vr)):
        codes, scale = A.quantize_rows(T.f64(x))
        kv.append(codes.astype(np.float64) * scale.astype(np.float64)[..., None])
        assert torch.equal(r.cpu(), torch.from_numpy((codes * scale[..., None]).astype(np.float32)).to(torch.bfloat16))
    assert int((cache.k_scale != 0).sum()) == sum(lens) * H
    q = T.heads(3, sum(new), 2 * H, D)
    o = qb.qlin_attn_q8(q, cache, qb.KVBatch(T.cu_of(new), ln, table))
    s, t = T.starts(new), T.starts(lens)
    for b in range(2):
        for h in (0, 5, 15):
            r = A.attend(T.f64(q)[s[b]:s[b + 1], h], kv[0][t[b]:t[b + 1], h // 2], kv[1][t[b]:t[b + 1], h // 2],
                         lens[b] - new[b], D ** -0.5, cached=True)
            T.within(f"o of sequence {b} head {h}", T.f64(o)[s[b]:s[b + 1], h], r["o"], r["o_bound"] * (1 + 4 * A.F))


def test_rows_far_apart(qb):
    """Rows 16 MiB apart: a tile's offsets pass 2^30 bytes."""
    ld, n, Hq, Hkv, D = (1 << 23) - 8, 131, 2, 1, 64
    buf = torch.zeros(ld * n, dtype=torch.bfloat16, device="cuda").view(n, ld)
    x = T.heads(1, n, Hq + 2 * Hkv, D)
    w = (Hq + 2 * Hkv) * D
    buf[:, 64:64 + w] = x.view(n, w)
    part = buf[:, 64:64 + w].unflatten(1, (Hq + 2 * Hkv, D))
    q, k, v = part.split([Hq, Hkv, Hkv], 1)
    do, cu = T.heads(2, n, Hq, D), T.cu_of([n])
    o, lse = qb.qlin_attn_fwd(q, k, v, cu)
    want = qb.qlin_attn_fwd(*(t.contiguous() for t in (q, k, v)), cu)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = [buf[:, 1024 + i * 512:1024 + i * 512 + h * D].unflatten(1, (h, D)) for i, h in enumerate((Hq, Hkv, Hkv))]
    qb.qlin_attn_bwd(q, k, v, o, lse, do, cu, dq=g[0], dk=g[1], dv=g[2])
    for a, b in zip(g, qb.qlin_attn_bwd(*(t.contiguous() for t in (q, k, v)), o, lse, do, cu)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv", [(256, 2), (4096, 64)])
def test_many_heads(qb, Hq, Hkv):
    lens, D = [5, 3], 16
    q, k, v, do = (T.heads(i, 8, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    cu = T.cu_of(lens)
    o, lse = qb.qlin_attn_fwd(q, k, v, cu)
    T.check_prompt(lens, Hq, Hkv, D, q, k, v, o, lse, 0.25)
    T.check_gradient(lens, Hq, Hkv, D, q, k, v, do, *qb.qlin_attn_bwd(q, k, v, o, lse, do, cu), 0.25)
    c = T.Paged(qb, 2, [9, 40], lens, Hkv, D, 256)
    c.check(q, qb.qlin_attn_q8(q, c.cache, c.batch), 0.25)


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page", [
    ([3000], [150], 4, 2, 128, 64),             # many rows in shares
    ([3000], [150], 4, 2, 64, 16),
    ([1500], [300], 128, 128, 16, 32),          # many rows, every key in one workgroup
    ([1500], [300], 128, 128, 80, 128),
    ([20000, 40, 1, 700], [1, 1, 1, 1], 64, 64, 16, 64),  # few rows, the longest shares there are
])
def test_holes_in_long_sequences(qb, lens, new, Hq, Hkv, D, page):
    """Pages that are not there between whole steps, and steps that nothing cuts
    again behind them; NaN in every page of nobody."""
    c = T.Paged(qb, 11, lens, new, Hkv, D, page, spare=9)
    for b in range(len(lens)):
        held = -(-lens[b] // page)
        for i in [held // 3, held // 3 + 1, *range(held // 2, held, 13)]:
            if 0 < i < held - 1:
                c.table[b, i] = -1 if i % 2 else 1 << 30
    used = {int(p) for p in c.table.flatten() if 0 <= int(p) < c.cache.k_codes.shape[0]}
    for p in set(range(c.cache.k_codes.shape[0])) - used:
        c.cache.k_scale[p] = c.cache.v_scale[p] = float("nan")
    q = T.heads(3, sum(new), Hq, D)
    o = qb.qlin_attn_q8(q, c.cache, qb.KVBatch(c.batch.cu, c.batch.lens, c.table.cuda()), max_len=max(lens))
    c.check(q, o, D ** -0.5)
