"""Row operators around the experts, in float64 on the CPU: RMS norm with its gradient, int8 rows,
int8 products, and the gradients of route, combine and the row gather.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Plain numpy from the formulas:

  norm      n = h / sqrt(mean(h^2) + eps), y = n * w.  With g = dy * w, the gradient of sum(dy * y):
            dh = (g - n * mean(g * n)) / sqrt(mean(h^2) + eps), dw = sum over rows of dy * n.
  int8 rows s = fp32(amax / 127) per row (1 when amax = 0 or the quotient underflows; the next fp32
            up where amax / s would round past 127, s being subnormal), q = round(v / s).
  experts   h = silu(g) * u with g, u = (q_x s_x) (q_w s_w)^T; h's rows quantised as above; then the
            down product.  `slack` bounds what a code of h one step aside can do to y: codes whose
            exact quotient lies within `near` of a half step may round either way in fp32.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(h, w, eps):
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def rmsnorm_grad(dy, h, w, eps):
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, w))
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, g = h * r, dy * w
    return r * (g - n * (g * n).mean(-1, keepdims=True)), (dy * n).sum(0)


def quant_i8(v):
    """Codes (float64 whole numbers) and the fp32 scales of rows, as float64."""
    v = np.asarray(v, np.float64)
    amax = np.abs(v).max(-1)
    s = (amax / 127.0).astype(np.float32)
    s = np.where((s > 0) & (amax >= 127.5 * s.astype(np.float64)), np.nextafter(s, np.float32(np.inf)), s)
    s = np.where(s == 0, np.float32(1), s).astype(np.float64)
    return np.rint(v / s[..., None]), s


def gemm_i8(xq, xs, wq, ws):
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T  # whole numbers below 2^53
    return acc * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def expert_i8(xq, xs, W):
    """One expert's rows -> (y, slack); W: gate, up, down codes and s_gate, s_up, s_down."""
    g = gemm_i8(xq, xs, W["gate"], W["s_gate"])
    h = swiglu(g, gemm_i8(xq, xs, W["up"], W["s_up"]))
    q, s = quant_i8(h)
    y = gemm_i8(q, s, W["down"], W["s_down"])
    # fp32 error of h: five roundings, and the hardware exp2's argument |g| * log2(e) rounded once
    near = np.abs(h / s[:, None]) * (np.abs(g) + 16) * 2.0 ** -22
    t = np.abs(h / s[:, None])
    risky = np.abs(t - np.floor(t) - 0.5) <= near
    # the scale itself carries that error too (amax's), once per row
    down = np.abs(np.asarray(W["down"], np.float64)) * np.asarray(W["s_down"], np.float64)[:, None]
    rel = (np.abs(g).max(-1, keepdims=True) + 16) * 2.0 ** -22
    return y, (risky * s[:, None]) @ down.T + np.abs(q * s[:, None]) @ down.T * rel


def route_grad(ids, w, dw, E):
    ids, w, dw = np.asarray(ids), np.asarray(w, np.float64), np.asarray(dw, np.float64)
    v = w * (dw - (w * dw).sum(1, keepdims=True))
    out = np.zeros((ids.shape[0], E))
    for j in range(ids.shape[1]):
        np.add.at(out, (np.arange(ids.shape[0]), ids[:, j]), v[:, j])
    return out


def combine_grad(dout, y, slot, w):
    dout, y, w = (np.asarray(a, np.float64) for a in (dout, y, w))
    T, k = w.shape
    dy = np.zeros_like(y)
    dy[np.asarray(slot)] = (w[:, :, None] * dout[:, None]).reshape(T * k, -1)
    rows = y[np.asarray(slot)].reshape(T, k, -1)
    return dy, np.einsum("td,tkd->tk", dout, rows)


def permute_grad(dxp, slot, k, add=None):
    dxp = np.asarray(dxp, np.float64)
    n, d = dxp.shape
    out = dxp[np.asarray(slot)].reshape(n // k, k, d).sum(1)
    return out if add is None else out + np.asarray(add, np.float64)
