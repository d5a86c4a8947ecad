"""Inputs and oracle results of the attention tests: packed sequences, a paged
cache with pages in a shuffled order."""

from __future__ import annotations

import numpy as np
import torch

from oracle import attn_oracle as A


def starts(lens):
    return [0, *np.cumsum(lens).tolist()]


def cu_of(lens, device="cuda"):
    return torch.tensor(starts(lens), dtype=torch.int32, device=device)


def heads(seed, T, H, D, big=4.0):
    """bf16 [T][H][D] Gaussians, one column of each head `big` times as large."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    x[..., seed % D] *= big
    return x.to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def within(name, got, want, bound, floor=1e-30):
    """Every element within its bound (and NaN nowhere)."""
    d = np.abs(got - want)
    worst = np.nanmax(d / (bound + floor)) if d.size else 0.0
    assert np.isfinite(got).all(), f"{name}: not finite"
    assert (d <= bound + floor).all(), f"{name}: {worst:.2f} of its bound, largest difference {d.max():.3e}"
    return worst


def check_prompt(lens, Hq, Hkv, D, q, k, v, o, lse, scale):
    g, s = Hq // Hkv, starts(lens)
    qn, kn, vn, on, ln = f64(q), f64(k), f64(v), f64(o), f64(lse)
    for b in range(len(lens)):
        at = slice(s[b], s[b + 1])
        for h in range(Hq):
            r = A.attend(qn[at, h], kn[at, h // g], vn[at, h // g], 0, scale)
            within(f"o of sequence {b} head {h}", on[at, h], r["o"], r["o_bound"])
            within(f"lse of sequence {b} head {h}", ln[at, h], r["lse"], r["lse_bound"])


def check_gradient(lens, Hq, Hkv, D, q, k, v, do, dq, dk, dv, scale):
    g, s = Hq // Hkv, starts(lens)
    qn, kn, vn, don, dqn, dkn, dvn = (f64(t) for t in (q, k, v, do, dq, dk, dv))
    for b in range(len(lens)):
        at = slice(s[b], s[b + 1])
        for hk in range(Hkv):
            sums = {x: 0.0 for x in ("dk", "dv", "dk_bound", "dv_bound")}
            for h in range(hk * g, hk * g + g):
                out, bound = A.gradient(qn[at, h], kn[at, hk], vn[at, hk], don[at, h], scale)
                within(f"dq of sequence {b} head {h}", dqn[at, h], out["dq"], bound["dq"])
                for x in ("dk", "dv"):
                    sums[x] = sums[x] + out[x]
                    sums[x + "_bound"] = sums[x + "_bound"] + bound[x]
            # (U |sum| <= the sum of the heads' U |dk|: the bounds add up)
            within(f"dk of sequence {b} head {hk}", dkn[at, hk], sums["dk"], sums["dk_bound"])
            within(f"dv of sequence {b} head {hk}", dvn[at, hk], sums["dv"], sums["dv_bound"])


class Paged:
    """A cache of random rows for sequences of the given lengths, the last
    new[b] of each the batch's."""

    def __init__(self, qb, seed, lens, new, H, D, page, spare=3, extra=2):
        g = torch.Generator().manual_seed(seed)
        used = [-(-L // page) for L in lens]
        pages = sum(used) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        self.lens, self.new, self.H, self.D, self.page = lens, new, H, D, page
        table = torch.full((len(lens), max(max(used, default=0), 1) + extra), -1, dtype=torch.int32)
        for b, n in enumerate(used):
            for i in range(n):
                table[b, i] = perm.pop()
        self.table = table
        codes = [torch.randint(-127, 128, (pages, H, page, D), generator=g, dtype=torch.int8) for _ in range(2)]
        scale = [(0.01 + 0.02 * torch.rand((pages, H, page), generator=g)) for _ in range(2)]
        self.cache = qb.KVCache(*(t.cuda() for t in codes), *(t.cuda() for t in scale))
        self.batch = qb.KVBatch(cu_of(new), torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda())

    def rows(self, b):
        """Keys and values of sequence b, fp64 [L][H][D], and which are there."""
        L, table = self.lens[b], self.table[b].numpy()
        t = np.arange(L)
        pg = np.where(t // self.page < len(table), table[np.minimum(t // self.page, len(table) - 1)], -1)
        there = (pg >= 0) & (pg < self.cache.k_codes.shape[0])
        at, row = np.where(there, pg, 0), t % self.page
        out = []
        for c, s in ((self.cache.k_codes, self.cache.k_scale), (self.cache.v_codes, self.cache.v_scale)):
            c, s = c.cpu().numpy(), s.cpu().numpy()
            out.append(c[at, :, row].astype(np.float64) * s[at, :, row].astype(np.float64)[..., None])
        return out[0], out[1], there

    def check(self, q, o, scale):
        Hq = q.shape[1]
        g, s, qn, on = Hq // self.H, starts(self.new), f64(q), f64(o)
        for b in range(len(self.lens)):
            k, v, there = self.rows(b)
            at = slice(s[b], s[b + 1])
            for h in range(Hq):
                r = A.attend(qn[at, h], k[:, h // g], v[:, h // g], self.lens[b] - self.new[b], scale, there, cached=True)
                # (a value's scale multiplies p in fp32 before that is rounded)
                within(f"o of sequence {b} head {h}", on[at, h], r["o"], r["o_bound"] * (1 + 4 * A.F))
