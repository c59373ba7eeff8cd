"""What surrounds the layer in a model's block, in float64 on the CPU: routing by scores, the norms
around a block with their gradients, and products with 4-bit weights.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Plain numpy from the formulas:

  route    s = sigmoid(l) or softmax over all experts; c = s + b, or the logits' own order without a
           bias; a logit of -inf makes c = -inf.  Groups are valued by the sum of their 1 or 2 largest
           c; the k largest c of the best groups are selected, ties to the lower index; w = scale * s,
           over the sum of the selected where renormalised (0 where that is 0).
  block    u = x / sqrt(mean(x^2) + eps) * post, h = rs * r + bs * gate * u, y = the norm of h.
  w4       W[n][k] = (code - zero) * scale.
"""
from __future__ import annotations

import numpy as np


def scores(l, sigmoid):
    l = np.asarray(l, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(np.isneginf(m), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
        t = e.sum(1, keepdims=True)
        return np.where(t > 0, e / np.where(t > 0, t, 1.0), 0.0)


def choices(l, bias, sigmoid):
    """What experts are compared by."""
    l = np.asarray(l, np.float64)
    c = l if bias is None else scores(l, sigmoid) + np.asarray(bias, np.float64)
    return np.where(np.isneginf(l), -np.inf, c)


def route_scored(l, k, bias=None, sigmoid=True, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    l = np.asarray(l, np.float64)
    T, E = l.shape
    s, c = scores(l, sigmoid), choices(l, bias, sigmoid)
    allowed = np.ones((T, groups), bool)
    if groups > 1:
        v = c if bias is not None or group_top == 1 else np.where(np.isneginf(l), -np.inf, s)
        best = np.sort(v.reshape(T, groups, -1), 2)[:, :, ::-1][:, :, :group_top].sum(2)
        allowed = np.zeros((T, groups), bool)
        for t in range(T):
            order = sorted(range(groups), key=lambda g: (-best[t, g], g))
            allowed[t, order[:top_groups]] = True
    ids = np.empty((T, k), np.int64)
    size = E // groups
    for t in range(T):
        left = [e for e in range(E) if allowed[t, e // size]]
        ids[t] = sorted(left, key=lambda e: (-c[t, e], e))[:k]
    w = np.take_along_axis(s, ids, 1)
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
    return ids, scale * w


def route_scored_grad(l, ids, w, dw, sigmoid=True, renorm=True, scale=1.0):
    """(gradient, the magnitude of what is summed for it)."""
    l, w, dw = (np.asarray(a, np.float64) for a in (l, w, dw))
    ids = np.asarray(ids)
    T, E = l.shape
    D = (w * dw).sum(1, keepdims=True)
    aD = np.abs(w * dw).sum(1, keepdims=True)
    v = w * dw - (w * D / scale if renorm else 0.0)
    a = np.abs(w * dw) + (np.abs(w) * aD / scale if renorm else 0.0)
    if sigmoid:
        with np.errstate(over="ignore"):
            f = 1.0 / (1.0 + np.exp(np.take_along_axis(l, np.clip(ids, 0, E - 1), 1)))
        v, a = v * f, a * f
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    if not sigmoid and not renorm:
        s = scores(l, False)
        out, mag = -s * D, s * aD
    for j in range(ids.shape[1]):
        ok = (ids[:, j] >= 0) & (ids[:, j] < E)
        np.add.at(out, (np.arange(T)[ok], ids[ok, j]), v[ok, j])
        np.add.at(mag, (np.arange(T)[ok], ids[ok, j]), a[ok, j])
    return out, mag


def _root(v, eps):
    return np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def block_norm(x, r, post, gate, pre, rs, bs, eps):
    """(h before its rounding, the magnitude of its two terms, a function from h to y)."""
    x, r = np.asarray(x, np.float64), np.asarray(r, np.float64)
    u = x if post is None else x / _root(x, eps) * np.asarray(post, np.float64)
    if gate is not None:
        u = np.asarray(gate, np.float64) * u
    return rs * r + bs * u, np.abs(rs * r) + np.abs(bs * u), \
        lambda h: np.asarray(h, np.float64) / _root(np.asarray(h, np.float64), eps) * np.asarray(pre, np.float64)


def block_norm_grad(dy, dh, x, h, post, gate, pre, rs, bs, eps):
    """Gradients and, under "e_" + name, the magnitudes that rounding errors of each scale with."""
    dy, x, h, pre = (np.asarray(a, np.float64) for a in (dy, x, h, pre))
    dh = np.zeros_like(dy) if dh is None else np.asarray(dh, np.float64)
    gt = np.float64(1.0) if gate is None else np.asarray(gate, np.float64)
    g, r2 = dy * pre, 1.0 / _root(h, eps)
    n2 = h * r2
    H = dh + r2 * (g - n2 * (g * n2).mean(-1, keepdims=True))
    eH = np.abs(dh) + r2 * (np.abs(g) + np.abs(n2) * np.abs(g * n2).mean(-1, keepdims=True))
    out = dict(dpre=(dy * n2).sum(0), e_dpre=np.abs(dy * n2).sum(0), dres=rs * H, e_dres=abs(rs) * eH)
    if post is None:
        n1, u = x, x
    else:
        r1 = 1.0 / _root(x, eps)
        n1 = x * r1
        u = n1 * np.asarray(post, np.float64)
    if gate is not None:
        dg, e = bs * H * u, np.abs(bs * eH * u)
        out.update(dgate=dg, e_dgate=e) if gt.ndim == 2 else out.update(dgate=dg.sum(0), e_dgate=e.sum(0))
    b, eb = bs * gt * H, np.abs(bs * gt * eH)
    if post is not None:
        out.update(dpost=(b * n1).sum(0), e_dpost=np.abs(eb * n1).sum(0))
        b, eb = b * np.asarray(post, np.float64), eb * np.abs(np.asarray(post, np.float64))
        b = r1 * (b - n1 * (b * n1).mean(-1, keepdims=True))
        eb = r1 * (eb + np.abs(n1) * np.abs(eb * n1).mean(-1, keepdims=True))
    out.update(dx=b, e_dx=eb)
    return out


def w4_values(codes, scales, zeros, group):
    """uint8 [N][K/2] (the even element in the low half), [N][K/group] -> [N][K]."""
    codes = np.asarray(codes)
    q = np.empty((codes.shape[0], 2 * codes.shape[1]))
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    z = 8.0 if zeros is None else np.repeat(np.asarray(zeros, np.float64), group, 1)
    return (q - z) * np.repeat(np.asarray(scales, np.float64), group, 1)


def gemm_w4(x, w, up=None):
    """(y, the magnitude that rounding errors of its sums scale with)."""
    x = np.asarray(x, np.float64)
    y, e = x @ w.T, np.abs(x) @ np.abs(w).T
    if up is None:
        return y, e
    u, eu = x @ up.T, np.abs(x) @ np.abs(up).T
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-y))
    # |d silu| <= 1.1
    return y * s * u, 1.1 * e * np.abs(u) + np.abs(y * s) * eu
