"""Timing cases of the 8-bit row operators: the root-mean-square norm with an
8-bit output and its gradient, the 8-bit integer product, and the layer's
backward pass from an 8-bit activation checkpoint.

`run` computes a case either with elementary torch operations in fp32 (the
plain form, `own = False`) or through the library (`own = True`); `exact`
computes the same outputs in fp64 from the definitions.

The 8-bit row format: codes q[m][k] in -127..127 and one fp32 scale per row,
    a = max_k |v[m][k]|,  scale[m] = a / 127,  q = round_half_even(127 v / a),
the row standing for q * scale (a row of zeros has scale 0 and codes 0).
"""

import math

import torch

own = False

EPS = 1e-5
S = 2.0  # adapter scale


def listed():
    return [
        # one token of a 4096-wide model between two layers: pure latency
        {"name": "norm_token", "op": "norm", "M": 1, "d": 4096, "res": True},
        # a training batch or prompt of 4096 tokens at width 8192
        {"name": "norm_prompt", "op": "norm", "M": 4096, "d": 8192, "res": True},
        # a short ragged prompt at an odd width, first norm of a network (no residual)
        {"name": "norm_ragged", "op": "norm", "M": 777, "d": 5003, "res": False},
        # gradient of the norm: one short sequence
        {"name": "normbwd_short", "op": "normbwd", "M": 250, "d": 4096, "res": False},
        # gradient of the norm: a training batch, the residual stream's gradient added
        {"name": "normbwd_batch", "op": "normbwd", "M": 4096, "d": 8192, "res": True},
        # one token through a square projection, its 8-bit row at hand from the norm
        {"name": "w8a8_token", "op": "w8a8", "M": 1, "N": 4096, "K": 4096, "pack": False},
        # sixteen decoding sequences through a large down projection, bf16 rows at hand
        {"name": "w8a8_decode", "op": "w8a8", "M": 16, "N": 8192, "K": 28672, "pack": True},
        # a ragged prompt into an odd number of output features (a vocabulary with added entries)
        {"name": "w8a8_ragged", "op": "w8a8", "M": 333, "N": 32003, "K": 4096, "pack": True},
        # a prompt of 4096 tokens through the large down projection
        {"name": "w8a8_prompt", "op": "w8a8", "M": 4096, "N": 8192, "K": 28672, "pack": True},
        # a short fine-tuning sequence, square projection, rank 16: row kept in 8 bits, then its backward
        {"name": "ckpt_short", "op": "ckpt", "M": 200, "N": 4096, "K": 4096, "r": 16, "pool": 1, "pack": True, "dx": False},
        # the large down projection with rank 64 in a training batch (adapter gradients)
        {"name": "ckpt_batch", "op": "ckpt", "M": 4096, "N": 8192, "K": 28672, "r": 64, "pool": 1, "pack": True, "dx": False},
        # group-pooled adapter on a 4-bit group-quantized weight, input gradient included
        {"name": "ckpt_pooled", "op": "ckpt", "M": 2048, "N": 4096, "K": 11008, "r": 64, "pool": 32, "pack": False, "dx": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "normbwd", "w8a8", "w8a8", "ckpt", "ckpt"])
    while True:
        M = _log(rng, 1, 4096)
        if op in ("norm", "normbwd"):
            d = _log(rng, 64, 16384)
            if M * d <= 4096 * 8192:
                return {"op": op, "M": M, "d": d, "res": rng.random() < 0.7}
        elif op == "w8a8":
            N, K = _log(rng, 100, 33000), 16 * _log(rng, 8, 1792)
            if M * N * K <= 4096 * 8192 * 28672:
                return {"op": op, "M": M, "N": N, "K": K, "pack": rng.random() < 0.5}
        else:
            N, K = 16 * _log(rng, 16, 688), 64 * _log(rng, 4, 448)
            if M * N * K <= 4096 * 8192 * 28672:
                return {"op": op, "M": M, "N": N, "K": K, "r": _log(rng, 4, 128), "pool": rng.choice([1, 1, 32]),
                        "pack": rng.random() < 0.5, "dx": rng.random() < 0.3}


def work(case):
    op, M = case["op"], case["M"]
    if op == "norm":
        d = case["d"]
        # x, residual, gamma read; h (with a residual), codes, values, scale and reciprocal norm written
        return {"bytes": M * d * (2 + (4 if case["res"] else 0) + 1 + 2) + 2 * d + 8 * M, "flops": 8 * M * d}
    if op == "normbwd":
        d = case["d"]
        return {"bytes": M * d * (2 + 2 + (2 if case["res"] else 0) + 2) + 2 * d + 4 * M + 4 * d, "flops": 11 * M * d}
    N, K = case["N"], case["K"]
    rows = M * K * (2 if case["pack"] else 1) + (0 if case["pack"] else 4 * M)
    if op == "w8a8":
        return {"bytes": rows + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    r, G = case["r"], K // case["pool"]
    w = {"bytes": rows + 2 * M * N + 2 * N * r + 4 * M * r + 2 * r * G + 2 * N * r, "flops": 4 * M * N * r + 2 * M * G * r}
    if case["pack"]:
        w["bytes"] += M * K + 4 * M  # the checkpoint written
    if case["dx"]:
        w["bytes"] += N * K // 2 + 4 * N * (K // 32) + 2 * r * G + 2 * M * K
        w["flops"] += 2 * M * N * K + 2 * M * G * r
    return w


# ------------------------------------------------------------------ inputs

def _rows(g, M, d):
    """bf16 activations: unit Gaussians, a few feature columns twenty times as
    large, and (in longer batches) padding tokens of zeros at the end."""
    x = torch.randn((M, d), generator=g, device="cuda", dtype=torch.bfloat16)
    big = torch.randint(0, d, (max(1, d // 1024),), generator=g, device="cuda")
    x[:, big] *= 20
    if M >= 200:
        x[M - M // 100:] = 0
    return x


def _codes(g, M, d, std):
    """8-bit rows of Gaussians of standard deviation `std`, as codes and scales."""
    a = 4.0 + 0.3 * torch.randn((M,), generator=g, device="cuda").clamp_(-3, 3)
    q = torch.randn((M, d), generator=g, device="cuda", dtype=torch.float32)
    q *= (127 / a)[:, None]
    q.round_().clamp_(-127, 127)
    return q.to(torch.int8), a * (std / 127)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M = case["op"], case["M"]
    st = {"case": case}
    if op in ("norm", "normbwd"):
        d = case["d"]
        st["gamma"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(torch.bfloat16)
        if op == "norm":
            st["x"] = _rows(g, M, d)
            st["res"] = _rows(g, M, d) if case["res"] else None
        else:
            st["h"] = _rows(g, M, d)
            st["rstd"] = torch.rsqrt(st["h"].float().square().mean(1) + EPS)
            st["dy"] = torch.randn((M, d), generator=g, device="cuda", dtype=torch.bfloat16)
            st["dh"] = torch.randn((M, d), generator=g, device="cuda", dtype=torch.bfloat16) if case["res"] else None
        return st
    N, K = case["N"], case["K"]
    if case["pack"]:
        st["x"] = _rows(g, M, K)
    else:
        st["xq"], st["xs"] = _codes(g, M, K, 1.0)
    if op == "w8a8":
        st["wq"], st["ws"] = _codes(g, N, K, 0.02)
        return st
    r, G = case["r"], K // case["pool"]
    # the frozen weight: 4-bit codes with an fp16 scale and zero per 32 columns
    st["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    st["scale"] = (0.005 + 0.001 * torch.rand((N, K // 32), generator=g, device="cuda")).to(torch.float16)
    st["zero"] = (-7.5 * st["scale"].float() + 0.002 * torch.randn((N, K // 32), generator=g, device="cuda")).to(torch.float16)
    st["A"] = ((2 * torch.rand((r, G), generator=g, device="cuda") - 1) / math.sqrt(G)).to(torch.bfloat16)
    st["B"] = (0.01 * torch.randn((N, r), generator=g, device="cuda")).to(torch.bfloat16)
    st["dy"] = torch.randn((M, N), generator=g, device="cuda", dtype=torch.bfloat16)
    # u = P A^T, which the forward pass returns: here Gaussians of its size
    st["u"] = torch.randn((M, r), generator=g, device="cuda") * math.sqrt(case["pool"] / 3)
    return st


# ------------------------------------------------------- the library's calls

def _run_own(st):
    import quantized_base_rank_amd as qb
    c = st["case"]
    op = c["op"]
    if op == "norm":
        h, q, rstd, y = qb.qlin_rmsnorm_q8(st["x"], st["gamma"], EPS, residual=st["res"], want_values=True)
        return {"h": h, "values": y, "scale": q.scale, "rstd": rstd}
    if op == "normbwd":
        dx, dgamma = qb.qlin_rmsnorm_bwd(st["h"], st["gamma"], st["rstd"], st["dy"], dh=st["dh"])
        return {"dx": dx, "dgamma": dgamma}
    q = qb.qlin_quantize_q8(st["x"]) if c["pack"] else qb.Q8Rows(st["xq"], st["xs"])
    if op == "w8a8":
        return {"y": qb.qlin_w8a8_fwd(q, qb.Q8Rows(st["wq"], st["ws"]))}
    w = qb.QWeight(qb.QLIN_FMT_INT4_GROUP, 32, 0, c["N"], c["K"], st["codes"], scale=st["scale"], zero=st["zero"])
    dx, dA, dB = qb.qlin_bwd_q8(w, q, st["A"], st["B"], c["r"], S, st["dy"], st["u"], pool=c["pool"], need_dx=c["dx"])
    return {"dx": dx, "dA": dA, "dB": dB, "scale": q.scale if c["pack"] else None}


# --------------------------------------------------------- the plain form

def _q8(v):
    """fp32 rows -> (codes as fp32, scale)."""
    a = v.abs().amax(1, keepdim=True)
    q = torch.where(a > 0, torch.round(v * 127 / a), torch.zeros_like(v))
    return q, a[:, 0] / 127


def _weight(st):
    """The frozen weight's bf16 values, [N][K]: element i of a run of 8 sits in
    nibble i // 4 of byte i % 4; value = bf16(scale * q + zero)."""
    b = st["codes"].view(st["codes"].shape[0], -1, 1, 4)
    q = torch.cat([b & 15, b >> 4], 2).view(st["codes"].shape[0], -1, 32)
    w = q.float() * st["scale"].float()[:, :, None] + st["zero"].float()[:, :, None]
    return w.to(torch.bfloat16).view(st["codes"].shape[0], -1)


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op = c["op"]
    bf = torch.bfloat16
    if op == "norm":
        h = st["x"].float()
        if st["res"] is not None:
            h = h + st["res"].float()
        rstd = torch.rsqrt((h * h).mean(1) + EPS)
        q, scale = _q8(h * rstd[:, None] * st["gamma"].float())
        return {"h": h.to(bf) if st["res"] is not None else None, "values": (q * scale[:, None]).to(bf), "scale": scale, "rstd": rstd}
    if op == "normbwd":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = st["h"].float() * rstd
        g = dy * st["gamma"].float()
        dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(bf), "dgamma": (dy * xh).sum(0)}
    if c["pack"]:
        q, scale = _q8(st["x"].float())
    else:
        q, scale = st["xq"].float(), st["xs"]
    if op == "w8a8":
        y = q @ st["wq"].float().t()
        return {"y": (y * scale[:, None] * st["ws"]).to(bf)}
    x = q * scale[:, None]
    dy = st["dy"].float()
    du = S * (dy @ st["B"].float())
    dB = S * (dy.t() @ st["u"])
    dA = du.t() @ x.view(c["M"], -1, c["pool"]).sum(2)
    dx = None
    if c["dx"]:
        dx = dy @ _weight(st).float() + (du @ st["A"].float()).repeat_interleave(c["pool"], 1)
        dx = dx.to(bf)
    return {"dx": dx, "dA": dA.to(bf), "dB": dB.to(bf), "scale": scale if c["pack"] else None}


# ------------------------------------------------- the definition in 64 bits

def _rows64(v):
    """fp64 rows -> (codes, scale): a zero row divides by one."""
    a = v.abs().max(dim=1).values
    q = torch.round(127 * v / torch.where(a == 0, torch.ones_like(a), a).unsqueeze(1))
    return q, a / 127


def exact(case, seed):
    st = prepare(case, seed)
    f = {k: (t.double() if torch.is_tensor(t) and t.dtype != torch.uint8 else t) for k, t in st.items()}
    op, M = case["op"], case["M"]
    if op == "norm":
        h = f["x"] if f["res"] is None else f["x"] + f["res"]
        rstd = 1 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["d"] + EPS)
        q, scale = _rows64(h * torch.outer(rstd, f["gamma"]))
        return {"h": None if f["res"] is None else h, "values": q * scale.unsqueeze(1), "scale": scale, "rstd": rstd}
    if op == "normbwd":
        # y_k = gamma_k h_k rho, d rho / d h_j = -rho^3 h_j / d
        rho = f["rstd"].unsqueeze(1)
        t = (f["dy"] * f["gamma"] * f["h"]).sum(1, keepdim=True)
        dx = rho * f["dy"] * f["gamma"] - rho ** 3 / case["d"] * t * f["h"]
        return {"dx": dx if f["dh"] is None else dx + f["dh"], "dgamma": (f["dy"] * f["h"]).t() @ f["rstd"]}
    if case["pack"]:
        q, scale = _rows64(f["x"])
    else:
        q, scale = f["xq"], f["xs"]
    if op == "w8a8":
        return {"y": torch.outer(scale, f["ws"]) * (q @ f["wq"].t())}
    N, K, pool = case["N"], case["K"], case["pool"]
    du = S * (f["dy"] @ f["B"])
    # d/dA of s (P A^T) B^T against dY; P sums each group of `pool` columns
    dA = (du * scale.unsqueeze(1)).t() @ q.reshape(M, K // pool, pool).sum(-1)
    out = {"dx": None, "dA": dA, "dB": S * (f["dy"].t() @ f["u"]), "scale": scale if case["pack"] else None}
    if case["dx"]:
        col = torch.arange(K, device="cuda")
        byte = st["codes"][:, (col // 8) * 4 + col % 4]
        q4 = torch.where(col % 8 < 4, byte % 16, byte // 16).double()
        del byte
        w = (q4 * f["scale"][:, col // 32] + f["zero"][:, col // 32]).float().bfloat16().double()
        out["dx"] = f["dy"] @ w + du @ f["A"][:, col // pool]
    return out
