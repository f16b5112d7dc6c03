"""Plain 64-bit implementations of the 8-bit and block-norm operators, and the
error bounds their GPU results are held to.

Bounds count roundings: U32 = 2^-24 for each fp32 operation, half a step of
the output type for the final rounding."""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
F32, F16, BF16 = 0, 1, 2
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -133}  # half a subnormal step, at least


def levels(v):
    """(levels, scales): q = 127 v / a to even, s = a / 127."""
    a = np.abs(v).max(axis=1) if v.shape[1] else np.zeros(v.shape[0])
    bad = ~np.isfinite(a)
    a = np.maximum(np.where(bad, 1.0, a), 127.0 * 2.0 ** -126)
    with np.errstate(invalid="ignore"):
        q = np.rint(np.where(bad[:, None], 0.0, v) * 127.0 / a[:, None])
    return q.astype(np.int64), np.where(bad, np.nan, a / 127.0)


def product(q, sa, w, sw, bias=None, relu=False):
    """(C, |sum sa sw|) of the scaled integer product."""
    s = (q.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64)
    t = s * sa[:, None] * sw[None, :]
    c = t if bias is None else t + bias[None, :]
    return (np.where(c > 0, c, 0.0) if relu else c), np.abs(t)


def product_bound(c, t, dtype):
    """The sum's conversion and the product with sa round once each, the
    multiply-add with sw and the bias once, then the output."""
    e = 2.02 * U32 * t + 1.01 * U32 * np.abs(c)
    return e + HALF_STEP[dtype] * (np.abs(c) + e) + TINY[dtype]


def by_token(g, T, per):
    return g[np.arange(T) // per]


def forward(x, y, gate, gate_rows, w_post, w_pre, alpha, eps, post):
    """x_out before its rounding, and h of that x_out."""
    T = x.shape[0]
    r_post = None
    xo = x
    if y is not None:
        z = y
        if post:
            r_post = 1.0 / np.sqrt((y * y).mean(axis=1) + eps)
            z = y * r_post[:, None]
        if w_post is not None:
            z = z * w_post
        if gate is not None:
            z = z * by_token(gate, T, gate_rows)
        xo = alpha * x + z
    r_pre = 1.0 / np.sqrt((xo * xo).mean(axis=1) + eps)
    h = xo * r_pre[:, None] * (1.0 if w_pre is None else w_pre)
    return {"x_out": xo, "h": h, "r_post": r_post, "r_pre": r_pre}


# Longest chain of fp32 additions in a row's sum: 32 elements in a thread, six
# steps in a wave, sixteen waves, rounded up.
CHAIN = 64
# Relative error of r: half the sum's, the mean and eps, the reciprocal root
# (one step, 2^-23) and its use.
R_ERR = (CHAIN / 2 + 6) * U32


def forward_bound(x, y, z, xo, alpha, xt):
    """x_out: z = y r w g rounds three times after r; one multiply-add."""
    e = np.abs(z) * (R_ERR + 4 * U32) + 2 * U32 * np.abs(alpha * x) + U32 * np.abs(xo)
    return e + HALF_STEP[xt] * (np.abs(xo) + e) + TINY[xt]


def h_bound(h, bt):
    e = np.abs(h) * (R_ERR + 3 * U32)
    return e + HALF_STEP[bt] * (np.abs(h) + e) + TINY[bt]


def backward(x_new, dx_new, dh, y, gate, gate_rows, w_post, w_pre, r_post, r_pre, alpha, post,
             bounds=None):
    """Gradients from the formulas, with the given r's.  `bounds`: a dict that
    receives the fp32 error of each output (before an output's own rounding):
    sums of D terms err by CHAIN roundings of the sum of magnitudes, products
    of up to six factors by eight."""
    T, D = x_new.shape
    e32 = (CHAIN + 8) * U32
    out = {}
    d = np.zeros((T, D)) if dx_new is None else dx_new
    ad = np.abs(d)  # magnitudes behind d: its error is e32 of them
    if dh is not None:
        u = x_new * r_pre[:, None]
        p = dh if w_pre is None else dh * w_pre
        d = d + r_pre[:, None] * (p - u * (p * u).mean(axis=1, keepdims=True))
        ad = ad + r_pre[:, None] * (np.abs(p)
                                    + np.abs(u) * np.abs(p * u).mean(axis=1, keepdims=True))
        if w_pre is not None:
            out["dw_pre"] = (dh * u).sum(axis=0)
    out["dx"] = alpha * d
    b = {"dx": e32 * np.abs(alpha) * ad}
    steps = (T + 48) * U32  # a column sum's longest chain of additions
    if dh is not None and w_pre is not None:
        b["dw_pre"] = (steps + 4 * U32) * np.abs(dh * u).sum(axis=0)
    if y is not None:
        n = y * r_post[:, None] if post else y
        g = 1.0 if gate is None else by_token(gate, T, gate_rows)
        w1 = 1.0 if w_post is None else w_post
        if gate is not None:
            of = np.arange(T) // gate_rows
            out["dgate"] = np.zeros(gate.shape)
            np.add.at(out["dgate"], of, d * n * w1)
            b["dgate"] = np.zeros(gate.shape)
            np.add.at(b["dgate"], of, (e32 + steps) * ad * np.abs(n * w1))
        if w_post is not None:
            out["dw_post"] = (d * g * n).sum(axis=0)
            b["dw_post"] = ((e32 + steps) * ad * np.abs(g * n)).sum(axis=0)
        m = d * g * w1
        am = ad * np.abs(g * w1)
        if post:
            c1 = (m * n).mean(axis=1, keepdims=True)
            ac1 = (am * np.abs(n)).mean(axis=1, keepdims=True)
            out["dy"] = r_post[:, None] * (m - n * c1)
            b["dy"] = 2 * e32 * r_post[:, None] * (am + np.abs(n) * ac1)
        else:
            out["dy"] = m
            b["dy"] = e32 * am
    if bounds is not None:
        bounds.update(b)
    return out
