"""A pre-norm block around one adapted 4-bit layer, trained from 8-bit
activations and then served in 8 bits.

    python examples/adapted_block.py [--tokens 1000] [--steps 20]

One training step is
    h, q, rstd, v = rmsnorm(x + residual)    8-bit rows q; v their bf16 values
    y, u          = layer(v)                 frozen NF4 weight + adapter
    dv, dA, dB    = layer backward           from q (v is not kept)
    dx, dgamma    = norm backward
so that between the passes the layer keeps M (d_in + 4) bytes of its input
instead of 2 M d_in.  For serving, the weight with the adapter merged in is
held as 8-bit rows and the norm's rows go straight into the 8-bit product.
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantized_base_rank_amd as qb  # noqa: E402


def main(tokens: int = 1000, d_in: int = 1024, d_out: int = 1536, r: int = 16, steps: int = 20, lr: float = 2e-3):
    g = torch.Generator(device="cuda").manual_seed(0)
    bf = torch.bfloat16

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s, eps = 2.0, 1e-5
    w = qb.qlin_quantize_nf4(0.02 * randn(d_out, d_in))
    A, B = randn(r, d_in) / d_in ** 0.5, torch.zeros((d_out, r), device="cuda")
    gamma = torch.ones(d_in, device="cuda")
    x, residual = randn(tokens, d_in).to(bf), randn(tokens, d_in).to(bf)
    # the layer to imitate: another scale per feature and a rank-r change of the weight
    target_gamma = 1 + 0.1 * randn(d_in)
    change = 0.05 * randn(d_out, r) @ randn(r, d_in) / d_in ** 0.5
    h = x.float() + residual.float()
    y64 = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * target_gamma
    target = y64 @ (qb.qlin_dequant_bf16(w).float() + change).t()

    opt = torch.optim.Adam([A, B, gamma], lr=lr)
    losses, kept = [], 0
    for _ in range(steps):
        gb, Ab, Bb = gamma.to(bf), A.to(bf), B.to(bf)
        h, q, rstd, v = qb.qlin_rmsnorm_q8(x, gb, eps, residual=residual, want_values=True)
        y, u = qb.qlin_fwd(w, v, Ab, Bb, r, s)
        del v
        kept = q.nbytes()
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        dy = (diff / tokens).to(bf)
        dv, dA, dB = qb.qlin_bwd_q8(w, q, Ab, Bb, r, s, dy, u)
        _, dgamma = qb.qlin_rmsnorm_bwd(h, gb, rstd, dv)
        A.grad, B.grad, gamma.grad = dA.float(), dB.float(), dgamma
        opt.step()

    # serving: merge the adapter, hold the weight as 8-bit rows
    merged = qb.qlin_dequant_bf16(w).float() + s * B.to(bf).float() @ A.to(bf).float()
    w8 = qb.qlin_quantize_q8(merged.contiguous())
    _, q, _, v = qb.qlin_rmsnorm_q8(x, gamma.to(bf), eps, residual=residual, want_values=True)
    y8 = qb.qlin_w8a8_fwd(q, w8).float()
    y, _ = qb.qlin_fwd(w, v, A.to(bf), B.to(bf), r, s)
    err = float((y8 - y.float()).norm() / y.float().norm())
    return {"first_loss": losses[0], "last_loss": losses[-1], "bytes_kept": kept, "bytes_bf16": 2 * tokens * d_in,
            "served_rel_difference": err}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    for k, v in main(tokens=a.tokens, steps=a.steps).items():
        print(f"{k}: {v:.6g}")
