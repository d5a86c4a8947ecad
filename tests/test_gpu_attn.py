"""Attention against the fp64 oracle, element by element within bounds derived
from its roundings: prompts and their gradient, and new tokens over the paged
8-bit cache, at sizes around the tiles and masks that leave rows empty."""

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


PROMPTS = [
    ([1], 1, 1, 64),
    ([1], 8, 1, 128),
    ([2, 1, 3], 4, 2, 16),
    ([31, 33, 0, 1, 64], 2, 2, 80),
    ([63, 65], 3, 1, 128),
    ([127, 129, 128], 2, 1, 96),
    ([0, 200, 0], 2, 2, 128),
    ([255], 4, 4, 64),
    ([257, 7], 7, 1, 112),
    ([300], 8, 2, 128),
    ([513], 2, 1, 32),
    ([40], 128, 1, 48),
    ([5, 17, 90, 2, 2, 61], 12, 4, 128),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPTS)
def test_prompts_and_gradient(qb, lens, Hq, Hkv, D):
    n, scale = sum(lens), 1 / D ** 0.5
    q, k, v, do = (T.heads(i + 7 * D, n, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    cu = T.cu_of(lens)
    o, lse = qb.qlin_attn_fwd(q, k, v, cu)
    T.check_prompt(lens, Hq, Hkv, D, q, k, v, o, lse, scale)
    dq, dk, dv = qb.qlin_attn_bwd(q, k, v, o, lse, do, cu)
    T.check_gradient(lens, Hq, Hkv, D, q, k, v, do, dq, dk, dv, scale)


def test_long_prompt(qb):
    """Many steps of every loop, a scale of its own."""
    lens, Hq, Hkv, D = [1500], 2, 1, 128
    q, k, v, do = (T.heads(i, 1500, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    o, lse = qb.qlin_attn_fwd(q, k, v, T.cu_of(lens), scale=0.03)
    T.check_prompt(lens, Hq, Hkv, D, q, k, v, o, lse, 0.03)
    dq, dk, dv = qb.qlin_attn_bwd(q, k, v, o, lse, do, T.cu_of(lens), scale=0.03)
    T.check_gradient(lens, Hq, Hkv, D, q, k, v, do, dq, dk, dv, 0.03)


def test_scores_far_apart(qb):
    """Scores of some hundreds: one key takes all, running maxima move by much."""
    lens, D = [333], 64
    q, k, v, do = (T.heads(i, 333, 2, D, big=40.0 if i < 3 else 1.0) for i in range(1, 5))
    o, lse = qb.qlin_attn_fwd(q, k, v, T.cu_of(lens))
    T.check_prompt(lens, 2, 2, D, q, k, v, o, lse, D ** -0.5)
    dq, dk, dv = qb.qlin_attn_bwd(q, k, v, o, lse, do, T.cu_of(lens))
    T.check_gradient(lens, 2, 2, D, q, k, v, do, dq, dk, dv, D ** -0.5)


def test_gradient_against_differences(qb):
    """The directional derivative of sum(o * do) in fp64."""
    n, Hq, Hkv, D, scale = 70, 4, 2, 64, 0.125
    q, k, v, do = (T.heads(i, n, h, D, big=1.0) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    o, lse = qb.qlin_attn_fwd(q, k, v, T.cu_of([n]))
    grads = qb.qlin_attn_bwd(q, k, v, o, lse, do, T.cu_of([n]))
    x = [T.f64(t) for t in (q, k, v)]
    don = T.f64(do)
    rng = np.random.default_rng(0)

    def loss(qn, kn, vn):
        return sum((A.attend(qn[:, h], kn[:, h // 2], vn[:, h // 2], 0, scale)["o"] * don[:, h]).sum() for h in range(Hq))

    for i in range(3):
        bound = 0.0
        u = rng.standard_normal(x[i].shape)
        e = 1e-5
        plus, minus = list(x), list(x)
        plus[i], minus[i] = x[i] + e * u, x[i] - e * u
        want = (loss(*plus) - loss(*minus)) / (2 * e)
        for h in range(Hq):
            _, b = A.gradient(x[0][:, h], x[1][:, h // 2], x[2][:, h // 2], don[:, h], scale)
            bound += (b[("dq", "dk", "dv")[i]] * np.abs(u[:, h if i == 0 else h // 2])).sum()
        got = (T.f64(grads[i]) * u).sum()
        # (central differences: e^2 of a third derivative of order |want|)
        assert abs(got - want) <= bound + 1e-6 * abs(want) + 1e-6


def test_parts_of_one_matrix(qb):
    """q, k, v from one product's output, gradients into one matrix."""
    lens, Hq, Hkv, D = [70, 59], 4, 2, 96
    n, w = sum(lens), Hq + 2 * Hkv
    qkv = T.heads(3, n, w + 1, D)[:, :w]
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    do, cu = T.heads(4, n, Hq, D), T.cu_of(lens)
    o, lse = qb.qlin_attn_fwd(q, k, v, cu)
    o2, lse2 = qb.qlin_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    d = torch.zeros((n, w, D), dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = d.split([Hq, Hkv, Hkv], 1)
    qb.qlin_attn_bwd(q, k, v, o, lse, do, cu, dq=dq, dk=dk, dv=dv)
    T.check_gradient(lens, Hq, Hkv, D, q, k, v, do, dq, dk, dv, D ** -0.5)
    for a, b in zip((dq, dk, dv), qb.qlin_attn_bwd(q, k, v, o, lse, do, cu)):
        assert torch.equal(a, b)


def test_rows_of_no_sequence(qb):
    """Rows before the first and behind the last sequence are neither used nor
    written: NaN there reaches nothing."""
    lens, Hq, Hkv, D, front, back = [37, 100], 4, 2, 64, 3, 80
    n = sum(lens)
    q, k, v, do = (T.heads(i, front + n + back, h, D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    for t in (q, k, v, do):
        t[:front] = float("nan")
        t[front + n:] = float("inf")
    cu = T.cu_of(lens) + front
    o = torch.full_like(q, 7)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    qb.qlin_attn_fwd(q, k, v, cu, out=o, lse=lse)
    mid = slice(front, front + n)
    T.check_prompt(lens, Hq, Hkv, D, q[mid], k[mid], v[mid], o[mid], lse[mid], D ** -0.5)
    g = [torch.full_like(t, 7) for t in (q, k, v)]
    qb.qlin_attn_bwd(q, k, v, o, lse, do, cu, dq=g[0], dk=g[1], dv=g[2])
    T.check_gradient(lens, Hq, Hkv, D, q[mid], k[mid], v[mid], do[mid], *(t[mid] for t in g), D ** -0.5)
    for t in (o, lse, *g):
        assert bool((t[:front] == 7).all()) and bool((t[front + n:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_what_the_mask_hides(qb, bad, D):
    """A token whose key and value are not finite: the queries before it, and the
    next sequence, are as without it."""
    lens, H = [150, 60], 2
    q, k, v = (T.heads(i, 210, H, D) for i in (1, 2, 3))
    o, lse = qb.qlin_attn_fwd(q, k, v, T.cu_of(lens))
    for at in (0, 31, 70, 149):
        k2, v2 = k.clone(), v.clone()
        k2[at, 0, 5], v2[at, :, 3] = bad, bad
        o2, lse2 = qb.qlin_attn_fwd(q, k2, v2, T.cu_of(lens))
        assert torch.equal(o[:at], o2[:at]) and torch.equal(lse[:at], lse2[:at])
        assert torch.equal(o[150:], o2[150:]) and torch.equal(lse[150:], lse2[150:])
        assert not torch.isfinite(o2[at:150, 1, 3]).any()  # (where it counts it shows)


CHUNKS = [
    # lens, new, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 2, 0], [1, 1, 0], 8, 1, 128, 16),
    ([17, 64, 65, 300], [1, 1, 1, 1], 8, 8, 128, 64),
    ([129, 1000], [1, 1], 16, 2, 128, 32),
    ([700, 3], [1, 1], 7, 1, 80, 16),
    ([500], [5], 4, 1, 96, 256),
    ([33, 520, 90], [33, 9, 2], 12, 4, 64, 16),
    ([270, 40], [130, 40], 6, 3, 128, 64),
    ([1100], [64], 8, 1, 128, 128),
    ([2100], [1], 128, 1, 128, 64),
    ([600, 1], [300, 1], 2, 2, 48, 16),
    ([4000, 77, 1500], [1, 1, 1], 4, 1, 128, 64),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page", CHUNKS)
def test_chunks_over_the_cache(qb, lens, new, Hq, Hkv, D, page):
    c = T.Paged(qb, 5, lens, new, Hkv, D, page)
    q = T.heads(1, sum(new), Hq, D)
    for kw in ({}, {"max_len": max(lens)}):
        o = qb.qlin_attn_q8(q, c.cache, c.batch, **kw)
        c.check(q, o, D ** -0.5)


def test_chunk_masks(qb):
    """Pages that are not there, sequences shorter than their new tokens, rows
    of no sequence, and NaN wherever nothing counts."""
    lens, new, H, D, page = [200, 5, 90, 64], [70, 9, 1, 64], 2, 128, 16
    c = T.Paged(qb, 6, lens, new, H, D, page)
    c.table[0, 3], c.table[0, 12], c.table[2, :] = -1, 1 << 20, -5
    c.table[3, 0] = -1  # the first 16 queries of the last sequence see nothing
    table = c.table.cuda()
    used = {int(p) for p in c.table.flatten() if 0 <= int(p) < c.cache.k_codes.shape[0]}
    for s in (c.cache.k_scale, c.cache.v_scale):  # pages of nobody, rows behind a sequence's last
        for p in range(s.shape[0]):
            if p not in used:
                s[p] = float("nan")
        for b, L in enumerate(lens):
            for t in range(L, (L + page - 1) // page * page):
                if 0 <= int(c.table[b, t // page]) < s.shape[0]:
                    s[int(c.table[b, t // page]), :, t % page] = float("nan")
    n = sum(new)
    q = T.heads(1, n + 20, 2 * H, D)
    q[n:] = float("nan")
    o = torch.full_like(q, 7)
    qb.qlin_attn_q8(q, c.cache, qb.KVBatch(c.batch.cu, c.batch.lens, table), out=o)
    c.check(q[:n], o[:n], D ** -0.5)
    assert bool((o[n:] == 7).all())
    # sequence 1: 9 new tokens, 5 cached: the first 4 have no place
    assert bool((o[70:74] == 0).all()) and bool((o[79] == 0).all()) and bool((o[80:96] == 0).all())


def test_shared_pages(qb):
    """Two sequences over the same prefix."""
    lens, new, H, D, page = [100, 100], [4, 4], 2, 64, 32
    c = T.Paged(qb, 8, lens, new, H, D, page)
    c.table[1, :3] = c.table[0, :3]
    q = T.heads(2, 8, H, D)
    o = qb.qlin_attn_q8(q, c.cache, qb.KVBatch(c.batch.cu, c.batch.lens, c.table.cuda()))
    c.check(q, o, D ** -0.5)


def test_longer_than_said(qb):
    """max_len below a sequence's length: taken as that long."""
    c = T.Paged(qb, 9, [300], [2], 2, 64, 16)
    q = T.heads(2, 2, 2, 64)
    o = qb.qlin_attn_q8(q, c.cache, c.batch, max_len=190)
    c.lens = [190]
    c.check(q, o, 0.125)


@pytest.mark.parametrize("Hkv,D,page,new,lens", [(1, 64, 16, [1, 1, 1], [1, 33, 100]), (8, 128, 64, [5, 0, 200], [5, 7, 260]),
                                                 (3, 80, 32, [17, 40], [90, 40]), (2, 16, 16, [9, 3], [4, 300]),
                                                 (5, 48, 16, [3] * 9 + [0, 1, 70], [40] * 12), (9, 96, 16, [1] * 200, list(range(1, 201)))])
def test_cache_write_and_read(qb, Hkv, D, page, new, lens):
    """Codes and scales bit for bit as the oracle rounds them, all other rows of
    the cache as they were, and the rows read back."""
    c = T.Paged(qb, 11, lens, new, Hkv, D, page)
    n = sum(new)
    k, v = T.heads(1, n + 2, Hkv + 1, D)[:, :Hkv], T.heads(2, n + 2, Hkv, D)
    k[0, 0, :] = 0
    if n > 4:
        k[3, 0, 1], v[4, 0, 0] = float("nan"), float("-inf")
        v[2, 0, :] = 2.0 ** -133  # below fp32's normal numbers
    want = [t.cpu().numpy().copy() for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scale, c.cache.v_scale)]
    back = [np.full((n + 2, Hkv, D), 7.0), np.full((n + 2, Hkv, D), 7.0)]
    s = T.starts(new)
    for i, x in enumerate((k, v)):
        codes, scale = A.quantize_rows(T.f64(x))
        for b in range(len(new)):
            for t in range(new[b]):
                place = lens[b] - new[b] + t
                if place < 0:
                    back[i][s[b] + t] = 0
                    continue
                pg, row = int(c.table[b, place // page]), place % page
                want[i][pg, :, row] = codes[s[b] + t]
                want[2 + i][pg, :, row] = scale[s[b] + t]
                back[i][s[b] + t] = codes[s[b] + t].astype(np.float64) * scale[s[b] + t][:, None]
    qb.qlin_kv_write_q8(c.cache, c.batch, k, v)
    got = [t.cpu().numpy() for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scale, c.cache.v_scale)]
    for w, g_ in zip(want, got):
        assert np.array_equal(w.view(np.uint8 if w.dtype == np.int8 else np.uint32)[~np.isnan(w.astype(np.float64))],
                              g_.view(np.uint8 if g_.dtype == np.int8 else np.uint32)[~np.isnan(w.astype(np.float64))])
        assert np.array_equal(np.isnan(w.astype(np.float64)), np.isnan(g_.astype(np.float64)))
    ko, vo = (torch.full((n + 2, Hkv, D), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qb.qlin_kv_read_q8(c.cache, c.batch, n + 2, k=ko, v=vo)
    for w, g_ in zip(back, (ko, vo)):
        w32 = torch.from_numpy(w.astype(np.float32)).to(torch.bfloat16).double().numpy()
        assert np.array_equal(w32, T.f64(g_), equal_nan=True)


def test_reading_all_and_absent_pages(qb):
    c = T.Paged(qb, 12, [50, 20], [50, 20], 2, 32, 16)
    c.table[0, 1] = -1
    k, v = qb.qlin_kv_read_q8(c.cache, qb.KVBatch(c.batch.cu, c.batch.lens, c.table.cuda()), 70)
    for b, at in ((0, slice(0, 50)), (1, slice(50, 70))):
        kn, vn, there = c.rows(b)
        for got, x in ((k, kn), (v, vn)):
            want = torch.from_numpy((x * there[:, None, None]).astype(np.float32)).to(torch.bfloat16)
            assert torch.equal(got[at].cpu(), want)
    # writing to a page that is not there changes nothing
    before = [t.clone() for t in (c.cache.k_codes, c.cache.k_scale)]
    bad = qb.KVBatch(c.batch.cu, c.batch.lens, torch.full_like(c.batch.table, 1 << 29))
    qb.qlin_kv_write_q8(c.cache, bad, k, v)
    assert torch.equal(before[0], c.cache.k_codes) and torch.equal(before[1], c.cache.k_scale)


@pytest.mark.parametrize("what", ["huge", "backwards", "negative"])
def test_arrays_that_make_no_sense(qb, what):
    """Whatever the int32 arrays hold, nothing outside the tensors is touched:
    rows of the outputs beyond the packed ones keep their values."""
    lens, new, H, D = [60, 40], [20, 30], 2, 64
    c = T.Paged(qb, 13, lens, new, H, D, 16)
    cu = {"huge": [0, 1 << 30, 0x7FFFFFFF], "backwards": [50, 20, 0], "negative": [-5, -(1 << 31), 10]}[what]
    ln = {"huge": [0x7FFFFFFF, 1 << 30], "backwards": [10, 0], "negative": [-(1 << 31), -1]}[what]
    cu, ln = torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(ln, dtype=torch.int32, device="cuda")
    batch = qb.KVBatch(cu, ln, c.batch.table)
    n = 50
    whole = [torch.full((n + 64, H, D), 7, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    q, k, v = (T.heads(i, n, H, D) for i in (1, 2, 3))
    outs = [w[:n] for w in whole]
    qb.qlin_attn_q8(q, c.cache, batch, out=outs[0])
    qb.qlin_kv_write_q8(c.cache, batch, k, v)
    qb.qlin_kv_read_q8(c.cache, batch, n, k=outs[1], v=outs[2])
    o, lse = qb.qlin_attn_fwd(q, k, v, cu, out=torch.zeros_like(q), lse=torch.zeros((n, H), device="cuda"))
    qb.qlin_attn_bwd(q, k, v, o, lse, q, cu, dq=outs[3], dk=outs[4], dv=outs[5])
    torch.cuda.synchronize()
    for w in whole:
        assert bool((w[n:] == 7).all())


def test_no_tokens(qb):
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    o, lse = qb.qlin_attn_fwd(e, e, e, cu)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    assert all(t.shape == (0, 2, 64) for t in qb.qlin_attn_bwd(e, e, e, o, lse, e, cu))
    c = T.Paged(qb, 14, [10], [0], 2, 64, 16)
    qb.qlin_kv_write_q8(c.cache, c.batch, e, e)
    assert qb.qlin_kv_read_q8(c.cache, c.batch, 0)[0].shape == (0, 2, 64)
    assert qb.qlin_attn_q8(e, c.cache, c.batch).shape == (0, 2, 64)


def test_refused_tensors(qb):
    q = T.heads(1, 10, 2, 64)
    cu = T.cu_of([10])
    with pytest.raises(ValueError):
        qb.qlin_attn_fwd(q.float(), q, q, cu)
    with pytest.raises(ValueError):
        qb.qlin_attn_fwd(q, q[:9], q, cu)
    with pytest.raises(ValueError):
        qb.qlin_attn_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), q, q, cu)  # heads not contiguous
    with pytest.raises(ValueError):
        qb.qlin_attn_fwd(q, q, q, cu.long())
    with pytest.raises(ValueError):
        qb.qlin_attn_fwd(q, q.cpu(), q, cu)
    with pytest.raises(qb.QlinError):
        qb.qlin_attn_fwd(q, q, q, cu, scale=0.0)
    with pytest.raises(qb.QlinError):
        qb.qlin_attn_fwd(q, q, q, cu, out=q)
    odd = torch.zeros((10, 2, 72), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qb.QlinError):
        qb.qlin_attn_fwd(odd, odd, odd, cu)
    with pytest.raises(qb.QlinError):
        qb.qlin_attn_fwd(T.heads(1, 10, 3, 64), q, q, cu)


def test_together(qb):
    """As a model uses them: a prompt's attention, its keys and values written to
    the cache, then the tokens that follow one at a time and as a piece; both
    see what the prompt's attention saw, in 8-bit rows."""
    H, g, D, page, n, more = 2, 4, 128, 64, 150, 5
    q, k, v = T.heads(1, n + more, H * g, D), T.heads(2, n + more, H, D), T.heads(3, n + more, H, D)
    cache = qb.KVCache.empty(8, H, D, page)
    table = torch.tensor([[6, 1, 3, -1]], dtype=torch.int32, device="cuda")

    def batch(new, length):
        return qb.KVBatch(T.cu_of([new]), torch.tensor([length], dtype=torch.int32, device="cuda"), table)

    qb.qlin_kv_write_q8(cache, batch(n, n), k[:n], v[:n])
    steps = []
    for t in range(n, n + more):
        qb.qlin_kv_write_q8(cache, batch(1, t + 1), k[t:t + 1], v[t:t + 1])
        steps.append(qb.qlin_attn_q8(q[t:t + 1], cache, batch(1, t + 1), max_len=t + 1))
    piece = qb.qlin_attn_q8(q[n:], cache, batch(more, n + more))
    every = qb.qlin_attn_q8(q, cache, batch(n + more, n + more))
    kr, vr = qb.qlin_kv_read_q8(cache, batch(n + more, n + more), n + more)
    full, _ = qb.qlin_attn_fwd(q, kr, vr, T.cu_of([n + more]))
    # against the exact values of the cached rows, each within its own bound
    cn = {x: A.quantize_rows(T.f64(t)) for x, t in (("k", k), ("v", v))}
    kn, vn = (c.astype(np.float64) * s.astype(np.float64)[..., None] for c, s in (cn["k"], cn["v"]))
    qn = T.f64(q)
    for h in range(H * g):
        r = A.attend(qn[:, h], kn[:, h // g], vn[:, h // g], 0, D ** -0.5, cached=True)
        for name, x, at in (("steps", torch.cat(steps), slice(n, None)), ("piece", piece, slice(n, None)),
                            ("every", every, slice(0, None))):
            T.within(f"{name} head {h}", T.f64(x)[:, h], r["o"][at], r["o_bound"][at] * (1 + 4 * A.F))
    # and the prompt's attention over the rows read back, within theirs
    T.check_prompt([n + more], H * g, H, D, q, kr, vr, full, _, D ** -0.5)
