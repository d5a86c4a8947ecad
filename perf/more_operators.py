"""Timing cases of the attention operators: a paged cache of keys and values in
8-bit rows (written, and read back), attention of a chunk of new tokens over
that cache, and causal attention over whole packed prompts with its gradient.

`run` computes a case either with elementary torch operations in fp32 (the
plain form, `own = False`) or through the library (`own = True`); `exact`
computes the same outputs in fp64 from the definitions.

Rows are packed: the tokens of sequence b are rows cu[b] .. cu[b + 1] - 1.
Query head h reads key head h // (Hq / Hkv).  With scale = 1 / sqrt(D),
    s[i][j] = scale q_i . k_j  over the keys j at or before token i's place,
    p = softmax_j(s),  o_i = sum_j p[i][j] v_j,  lse_i = log sum_j exp s[i][j],
    dv_j = sum_i p[i][j] do_i,   ds[i][j] = p[i][j] (do_i . v_j - do_i . o_i),
    dq_i = scale sum_j ds[i][j] k_j,   dk_j = scale sum_i ds[i][j] q_i
(dk and dv summed over the query heads that share a key head).

The cache holds each key and value row (one token, one head, D elements) as
int8 codes and an fp32 scale: a = max |x|, scale = a / 127, code =
round_half_even(127 x / a).  Token t of a sequence sits in row t % page of the
page that the sequence's table names at t // page; a batch's new tokens are
the last of their sequences.
"""

import math
import random

import torch

own = False


def listed():
    return [
        # a decoding step of 64 sequences: one token each into the cache, and back
        {"name": "cache_step", "op": "cache", "B": 64, "new": 1, "ctx": 2048, "ragged": True, "Hkv": 8, "D": 128, "page": 64},
        # four prompts of 4096 tokens written to the cache and read back for a restart
        {"name": "cache_prompts", "op": "cache", "B": 4, "new": 4096, "ctx": 4096, "ragged": False, "Hkv": 8, "D": 128, "page": 64},
        # ragged prompts behind earlier turns, an odd width of head, small pages
        {"name": "cache_ragged", "op": "cache", "B": 11, "new": 777, "ctx": 2500, "ragged": True, "Hkv": 5, "D": 80, "page": 16},
        # one token of one conversation: pure latency
        {"name": "chunk_token", "op": "chunk", "B": 1, "new": 1, "ctx": 4096, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "page": 64},
        # decoding 64 conversations of up to 8192 tokens, eight query heads to a key head
        {"name": "chunk_decode", "op": "chunk", "B": 64, "new": 1, "ctx": 8192, "ragged": True, "Hq": 64, "Hkv": 8, "D": 128, "page": 64},
        # drafted tokens and short follow-ups, a key head to every query head, odd lengths
        {"name": "chunk_ragged", "op": "chunk", "B": 9, "new": 33, "ctx": 3001, "ragged": True, "Hq": 12, "Hkv": 12, "D": 96, "page": 16},
        # a long prompt taken in pieces: 2048 tokens behind 30000
        {"name": "chunk_prefill", "op": "chunk", "B": 1, "new": 2048, "ctx": 32048, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "page": 128},
        # one short prompt
        {"name": "prompt_short", "op": "prompt", "B": 1, "T": 250, "ragged": False, "Hq": 32, "Hkv": 32, "D": 128},
        # sixteen packed prompts of different lengths, narrow heads
        {"name": "prompt_packed", "op": "prompt", "B": 16, "T": 8191, "ragged": True, "Hq": 32, "Hkv": 8, "D": 64},
        # a short fine-tuning sequence: forward and gradients
        {"name": "train_short", "op": "train", "B": 1, "T": 200, "ragged": False, "Hq": 32, "Hkv": 32, "D": 128},
        # a fine-tuning batch of 4 x 1024 tokens
        {"name": "train_batch", "op": "train", "B": 4, "T": 4096, "ragged": False, "Hq": 32, "Hkv": 32, "D": 128},
        # a long document, eight query heads to a key head
        {"name": "train_long", "op": "train", "B": 1, "T": 8192, "ragged": False, "Hq": 64, "Hkv": 8, "D": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "chunk", "chunk", "prompt", "train"])
    while True:
        Hkv, g, D = _log(rng, 1, 32), rng.choice([1, 1, 2, 4, 7, 8]), rng.choice([64, 80, 96, 128, 128])
        if op in ("cache", "chunk"):
            ctx = _log(rng, 16, 32768)
            new = 1 if rng.random() < 0.4 else _log(rng, 1, min(ctx, 4096))
            c = {"op": op, "B": _log(rng, 1, 64), "new": new, "ctx": ctx, "ragged": rng.random() < 0.7}
            if op == "chunk":
                c["Hq"] = g * Hkv
            c.update({"Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128])})
        else:
            B = _log(rng, 1, 16)
            c = {"op": op, "B": B, "T": _log(rng, B, 8192), "ragged": rng.random() < 0.7, "Hq": g * Hkv, "Hkv": Hkv, "D": D}
        if op in ("cache", "chunk") and c["B"] * c["ctx"] * Hkv * D > 64 * 8192 * 8 * 128:
            continue
        if op == "cache" and c["B"] * c["new"] * Hkv * D > 4 * 4096 * 8 * 128:
            continue
        if op != "cache" and (c["Hq"] > 64 or work(c)["flops"] > 2e12):
            continue
        return c


# lengths of a case's sequences: they belong to the case, not to its inputs

def _lengths(case):
    """(new tokens, tokens in all) of each sequence."""
    B = case["B"]
    rng = random.Random(B * 1000003 + case.get("ctx", case.get("T")))
    if case["op"] in ("prompt", "train"):
        T = case["T"]
        if case["ragged"]:
            cuts = [0] + sorted(rng.sample(range(1, T), B - 1)) + [T] if B > 1 else [0, T]
        else:
            cuts = [T * b // B for b in range(B + 1)]
        n = [cuts[b + 1] - cuts[b] for b in range(B)]
        return n, n
    if not case["ragged"]:
        return [case["new"]] * B, [case["ctx"]] * B
    length = [rng.randint(-(-case["ctx"] // 4), case["ctx"]) for _ in range(B)]
    return [rng.randint(1, min(case["new"], L)) for L in length], length


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    new, length = _lengths(case)
    T = sum(new)
    if op == "cache":
        # bf16 rows read, codes and scales written, both read again, bf16 rows written
        return {"bytes": 2 * T * Hkv * (2 * D + 2 * (D + 4) + 2 * D), "flops": 6 * T * Hkv * D}
    Hq = case["Hq"]
    pairs = sum(n * L - n * (n - 1) // 2 for n, L in zip(new, length))
    if op == "chunk":
        return {"bytes": sum(length) * Hkv * 2 * (D + 4) + 4 * T * Hq * D, "flops": 4 * pairs * Hq * D}
    rows = 2 * T * D * (2 * Hq + 2 * Hkv) + 4 * T * Hq
    if op == "prompt":
        return {"bytes": rows, "flops": 4 * pairs * Hq * D}
    # the gradient: five products to the forward's two
    return {"bytes": rows + 2 * T * D * (2 * Hq + 2 * Hkv), "flops": 14 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs

def _heads(g, T, H, D):
    """bf16 rows of heads: unit Gaussians, in some heads a few columns several
    times as large (as keys have them)."""
    x = torch.randn((T, H, D), generator=g, device="cuda")
    big = torch.randint(0, D, (H, 2), generator=g, device="cuda")
    x.scatter_(2, big.expand(T, H, 2), 4 * x.gather(2, big.expand(T, H, 2)))
    return x.to(torch.bfloat16)


def _starts(n):
    out = [0]
    for v in n:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, Hkv, D, B = case["op"], case["Hkv"], case["D"], case["B"]
    new, length = _lengths(case)
    T = sum(new)
    st = {"case": case, "starts": _starts(new), "length": length, "max_len": max(length),
          "cu": torch.tensor(_starts(new), dtype=torch.int32, device="cuda")}
    if op in ("prompt", "train"):
        # one product gives q, k and v: rows of (Hq + 2 Hkv) heads
        st["q"], st["k"], st["v"] = _heads(g, T, case["Hq"] + 2 * Hkv, D).split([case["Hq"], Hkv, Hkv], 1)
        if op == "train":
            st["do"] = torch.randn((T, case["Hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        return st
    page = case["page"]
    used = [-(-L // page) for L in length]
    pages = sum(used) + 3  # a few free
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(used)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    st["table"], st["lens"] = table, torch.tensor(length, dtype=torch.int32, device="cuda")
    shape = (pages, Hkv, page)
    for name in ("k", "v"):
        if op == "cache":
            st[name] = _heads(g, T, Hkv, D)
            st[name + "_codes"] = torch.zeros((*shape, D), dtype=torch.int8, device="cuda")
            st[name + "_scale"] = torch.zeros(shape, device="cuda")
        else:
            # rows of Gaussians; keys twice as long as values
            a = 2.6 + 0.3 * torch.randn(shape, generator=g, device="cuda").clamp_(-3, 3)
            q = torch.randn((*shape, D), generator=g, device="cuda").mul_((127 / a)[..., None])
            st[name + "_codes"] = q.round_().clamp_(-127, 127).to(torch.int8)
            st[name + "_scale"] = a * ((2 if name == "k" else 1) / 127)
            del q
    if op == "chunk":
        st["q"] = _heads(g, T, case["Hq"], D)
    return st


# ------------------------------------------------------- the library's calls

def _run_own(st):
    import quantized_base_rank_amd as qb
    op = st["case"]["op"]
    if op in ("prompt", "train"):
        o, lse = qb.qlin_attn_fwd(st["q"], st["k"], st["v"], st["cu"])
        if op == "prompt":
            return {"o": o, "lse": lse}
        dq, dk, dv = qb.qlin_attn_bwd(st["q"], st["k"], st["v"], o, lse, st["do"], st["cu"])
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    cache = qb.KVCache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    batch = qb.KVBatch(st["cu"], st["lens"], st["table"])
    if op == "chunk":
        return {"o": qb.qlin_attn_q8(st["q"], cache, batch, max_len=st["max_len"])}
    qb.qlin_kv_write_q8(cache, batch, st["k"], st["v"])
    k, v = qb.qlin_kv_read_q8(cache, batch, st["starts"][-1])
    return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


# --------------------------------------------------------- the plain form

_BLOCK = 1024  # queries at a time


def _attend(q, k, v, first, do=None):
    """Queries q [n][Hq][D] at places first, first + 1, ... over keys and
    values [L][Hkv][D], all fp32.  Returns o, lse and, for do, dq, dk, dv."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    g, c = Hq // Hkv, 1 / math.sqrt(D)
    kt, vt = k.permute(1, 0, 2).contiguous(), v.permute(1, 0, 2).contiguous()
    o, lse = torch.empty_like(q), q.new_empty(n, Hq)
    grads = None
    if do is not None:
        grads = torch.empty_like(q), torch.zeros_like(kt), torch.zeros_like(vt)

    def rows(x, a, b):  # [b - a][Hq][D] -> [Hkv][g (b - a)][D]
        return x[a:b].view(b - a, Hkv, g, D).permute(1, 2, 0, 3).reshape(Hkv, g * (b - a), D)

    def back(x, m):
        return x.view(Hkv, g, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D)

    for a in range(0, n, _BLOCK):
        b = min(n, a + _BLOCK)
        m, e = b - a, min(L, first + b)
        qb, ke, ve = rows(q, a, b), kt[:, :e], vt[:, :e]
        s = torch.matmul(qb, ke.transpose(1, 2).contiguous()).mul_(c).view(Hkv, g, m, e)
        place = torch.arange(first + a, first + b, device=q.device)
        s.masked_fill_(torch.arange(e, device=q.device) > place[:, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(total).view(Hkv, g * m, e)
        ob = torch.matmul(p, ve)
        o[a:b] = back(ob, m)
        lse[a:b] = (top + total.log()).view(Hkv, g, m).permute(2, 0, 1).reshape(m, Hq)
        if do is not None:
            dob = rows(do, a, b)
            grads[2][:, :e] += torch.matmul(p.transpose(1, 2).contiguous(), dob)
            ds = torch.matmul(dob, ve.transpose(1, 2).contiguous())
            ds = ds.sub_((dob * ob).sum(-1, keepdim=True)).mul_(p).mul_(c)
            grads[0][a:b] = back(torch.matmul(ds, ke), m)
            grads[1][:, :e] += torch.matmul(ds.transpose(1, 2).contiguous(), qb)
    if do is None:
        return o, lse
    return o, lse, grads[0], grads[1].permute(1, 0, 2), grads[2].permute(1, 0, 2)


def _slots(st, b, first, end):
    """Pages and rows within them of a sequence's places first .. end - 1."""
    t = torch.arange(first, end, device="cuda")
    page = st["case"]["page"]
    return st["table"][b, torch.div(t, page, rounding_mode="floor")].long(), t % page


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op, bf, starts, length = c["op"], torch.bfloat16, st["starts"], st["length"]
    T, B, D = starts[-1], c["B"], c["D"]
    if op == "cache":
        out = {}
        where = [_slots(st, b, length[b] - (starts[b + 1] - starts[b]), length[b]) for b in range(B)]
        pg, row = torch.cat([w[0] for w in where]), torch.cat([w[1] for w in where])
        for name in ("k", "v"):
            x = st[name].double()  # the quotient next to a tie
            a = x.abs().amax(2, keepdim=True)
            q = torch.where(a > 0, torch.round(127 * x / a), torch.zeros_like(x))
            st[name + "_codes"][pg, :, row] = q.to(torch.int8)
            st[name + "_scale"][pg, :, row] = (a[..., 0] / 127).float()
            out[name] = (st[name + "_codes"][pg, :, row].float() * st[name + "_scale"][pg, :, row][..., None]).to(bf)
            out[name + "_scale"] = st[name + "_scale"]
        return out
    if op == "chunk":
        o = torch.empty((T, c["Hq"], D), dtype=bf, device="cuda")
        for b in range(B):
            i, j = starts[b], starts[b + 1]
            pg, row = _slots(st, b, 0, length[b])
            k, v = (st[x + "_codes"][pg, :, row].float() * st[x + "_scale"][pg, :, row][..., None] for x in ("k", "v"))
            o[i:j] = _attend(st["q"][i:j].float(), k, v, length[b] - (j - i))[0].to(bf)
        return {"o": o}
    names = ["o", "lse"] if op == "prompt" else ["o", "lse", "dq", "dk", "dv"]
    parts = []
    for b in range(B):
        at = slice(starts[b], starts[b + 1])
        parts.append(_attend(st["q"][at].float(), st["k"][at].float(), st["v"][at].float(), 0,
                             st["do"][at].float() if op == "train" else None))
    out = {x: torch.cat([p[i] for p in parts]) for i, x in enumerate(names)}
    if op == "train":
        del out["lse"]
    return {x: t if x == "lse" else t.to(bf) for x, t in out.items()}


# ------------------------------------------------- the definition in 64 bits

def _head64(q, k, v, do, behind):
    """One head of one sequence: q [n][D] behind `behind` earlier tokens."""
    n, D = q.shape
    seen = torch.ones((n, k.shape[0]), dtype=torch.bool, device=q.device).tril(behind)
    s = torch.where(seen, (q @ k.t()) / D ** 0.5, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse.unsqueeze(1))
    o = p @ v
    if do is None:
        return o, lse
    dp = do @ v.t()
    ds = p * (dp - (p * dp).sum(1, keepdim=True)) / D ** 0.5
    return o, lse, ds @ k, ds.t() @ q, p.t() @ do


def exact(case, seed):
    st = prepare(case, seed)
    op, Hkv, D, B = case["op"], case["Hkv"], case["D"], case["B"]
    starts, length, T = st["starts"], st["length"], st["starts"][-1]

    def places(b, first):
        # (page, row) of each place of a sequence from `first` on
        t = torch.arange(first, length[b], device="cuda")
        return st["table"][b].long()[t // case["page"]], t % case["page"]

    if op == "cache":
        out = {}
        for name in ("k", "v"):
            x = st[name].double()
            big = torch.linalg.vector_norm(x, ord=math.inf, dim=2)
            scale = big / 127
            codes = torch.round(x * 127 / torch.where(big == 0, torch.ones_like(big), big)[..., None])
            # the stored scale is rounded to fp32 before it is read
            out[name] = codes * scale.float().double()[..., None]
            held = st[name + "_scale"].double()
            for b in range(B):
                n = starts[b + 1] - starts[b]
                pg, row = places(b, length[b] - n)
                held[pg, :, row] = scale[starts[b]:starts[b + 1]]
            out[name + "_scale"] = held
        return out
    Hq = case["Hq"]
    g = Hq // Hkv

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if op == "chunk":
        o = zeros(T, Hq, D)
        for b in range(B):
            pg, row = places(b, 0)
            at = slice(starts[b], starts[b + 1])
            for h in range(Hkv):
                k, v = (st[x + "_codes"][pg, h, row].double() * st[x + "_scale"][pg, h, row].double().unsqueeze(1) for x in "kv")
                for i in range(h * g, h * g + g):
                    o[at, i] = _head64(st["q"][at, i].double(), k, v, None, length[b] - (starts[b + 1] - starts[b]))[0]
        return {"o": o}
    o, lse, dq, dk, dv = zeros(T, Hq, D), zeros(T, Hq), zeros(T, Hq, D), zeros(T, Hkv, D), zeros(T, Hkv, D)
    for b in range(B):
        at = slice(starts[b], starts[b + 1])
        for i in range(Hq):
            f = [st[x][at, h].double() for x, h in (("q", i), ("k", i // g), ("v", i // g))]
            r = _head64(*f, st["do"][at, i].double() if op == "train" else None, 0)
            o[at, i], lse[at, i] = r[0], r[1]
            if op == "train":
                dq[at, i] = r[2]
                dk[at, i // g] += r[3]
                dv[at, i // g] += r[4]
    return {"o": o, "lse": lse} if op == "prompt" else {"o": o, "dq": dq, "dk": dk, "dv": dv}
