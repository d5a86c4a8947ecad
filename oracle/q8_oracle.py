"""CPU oracle of the 8-bit row operators, in float64.

TEST INFRASTRUCTURE ONLY, as qlin_oracle.py: nothing here is imported by the
library, and nothing of the library is imported here.

* quantize_rows ...... absmax rows in 8 bits ([QLoRA] "Background: what is
                       quantization?": scale by the largest magnitude, round
                       to the nearest level; the block is one row).  Pinned
                       against exact rationals.
* rmsnorm / rmsnorm_backward ... the norm's formula and its gradient, the
                       latter pinned by central differences.
* product ............ integer product of 8-bit rows with both scales.
* The layer's backward pass from a checkpoint is qlin_oracle.lora_backward on
  the rows' values.
"""

from __future__ import annotations

import numpy as np


def quantize_rows(x):
    """(codes int8, scale float32): round_half_even(127 x / a) per row, a the
    row's largest magnitude, and a / 127 rounded once; zero rows give zeros,
    rows with a non-finite value scale NaN and codes 0.  127 x is exact in
    float64 (24 + 7 bits), and a quotient that is no tie lies further from one
    (at least 1 / (254 2^24) relative) than float64 rounds."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x).all(axis=1)
    a = np.abs(np.where(ok[:, None], x, 0.0)).max(axis=1)
    safe = np.where(a > 0, a, 1.0)
    codes = np.rint(127.0 * np.where(ok[:, None], x, 0.0) / safe[:, None]).astype(np.int8)
    scale = (a.astype(np.float32) / np.float32(127)).astype(np.float32)  # one IEEE division
    scale[~ok] = np.nan
    return codes, scale


def rows_values(codes, scale):
    return np.asarray(codes, np.float64) * np.asarray(scale, np.float64)[:, None]


def rmsnorm(x, gamma, eps, residual=None):
    """(h, rstd, y)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, rstd, h * rstd[:, None] * np.asarray(gamma, np.float64)


def rmsnorm_backward(h, gamma, rstd, dy, dh=None):
    """(dx, dgamma) of <dy, h rstd(h) gamma> + <dh, h>."""
    h, gamma, rstd, dy = (np.asarray(v, np.float64) for v in (h, gamma, rstd, dy))
    xh = h * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * xh).sum(axis=0)


def product(xq, xs, wq, ws):
    s = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T  # integers below 2^53: exact
    return s * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]
