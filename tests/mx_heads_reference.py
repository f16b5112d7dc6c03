"""Plain 64-bit implementations of the microscaled linear path and of the head
norms with rotation, and the error bounds their GPU results are held to.

Bounds count roundings: U32 = 2^-24 for each fp32 operation, half a step of
the output type for the final rounding."""

from __future__ import annotations

import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
E2M1, E4M3 = 0, 1
E2M1_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_values():
    """Values of the 128 codes without a sign, from the field definition."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v  # code 127 is NaN


def table(fmt, device="cpu"):
    return torch.tensor(E2M1_VALUES if fmt == E2M1 else e4m3_values(), dtype=torch.float64,
                        device=device)


def quantise(x, fmt):
    """(codes without packing [M, Kp], scale bytes [M, Kp / 32]) of rows of x.  The
    element is found among the format's values: the nearest, of two equally near
    the one with an even code, the largest for all beyond it."""
    x = x.double()
    M, K = x.shape
    Kp = -(-K // 128) * 128
    v = torch.zeros((M, Kp), dtype=torch.float64, device=x.device)
    v[:, :K] = x
    b = v.view(M, Kp // 32, 32)
    a = b.abs().amax(dim=2)
    bad = ~torch.isfinite(b).all(dim=2)
    a = torch.where(bad, torch.ones_like(a), a)
    # floor(log2 a) from the exact mantissa and exponent
    e = torch.frexp(a)[1].to(torch.int64) - 1 - (2 if fmt == E2M1 else 8)
    e = torch.where(a == 0, torch.full_like(e, -127), e).clamp(min=-127)
    m = (torch.where(bad.unsqueeze(2), torch.zeros_like(b), b)
         * torch.exp2(-e.double()).unsqueeze(2)).abs()
    t = table(fmt, x.device)
    hi = torch.searchsorted(t, m.contiguous()).clamp(max=len(t) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - m, m - t[lo]
    code = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    code = torch.where(m >= t[-1], torch.full_like(code, len(t) - 1), code)
    sign = 8 if fmt == E2M1 else 128
    code = code + torch.where(torch.signbit(b) & ~bad.unsqueeze(2), sign, 0)
    s = torch.where(bad, torch.full_like(e, 255), e + 127)
    return code.view(M, Kp), s


def pack(codes, fmt):
    if fmt == E4M3:
        return codes.to(torch.uint8)
    return (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)


def unpack(q, fmt):
    q = q.to(torch.int64)
    if fmt == E4M3:
        return q
    return torch.stack([q & 15, q >> 4], dim=2).reshape(q.shape[0], -1)


def values(codes, s, fmt):
    """What codes (without packing) and scale bytes stand for."""
    t = table(fmt, codes.device)
    sign = 8 if fmt == E2M1 else 128
    top = len(t) - 1
    mag = t[(codes % sign).clamp(max=top)]
    mag = torch.where(codes % sign > top, torch.full_like(mag, float("nan")), mag)
    v = torch.where(codes >= sign, -mag, mag)
    p = torch.exp2(s.double() - 127.0)
    p = torch.where(s == 255, torch.full_like(p, float("nan")), p)
    return (v.view(v.shape[0], -1, 32) * p.unsqueeze(2)).view(v.shape)


def product(ca, sa, fa, cw, sw, bias=None, relu=False):
    """(C, bound on its error before the output's rounding) of the product of two
    matrices of blocks given as unpacked codes and scale bytes.

    Groups of 8 products are added in fixed point and their sums in fp32, each
    addition cutting off at most a step (2 U32) of what has been summed; the waves'
    sums and the bias come on top.  In E4M3 each product of a group is cut off at
    2^(e - 13), e the group's largest sum of exponents."""
    a, w = values(ca, sa, fa), values(cw, sw, E2M1)
    c = a @ w.t().contiguous()
    mag = a.abs() @ w.abs().t().contiguous()
    K = a.shape[1]
    if bias is not None:
        c = c + bias.double()
        mag = mag + bias.double().abs()
    err = 2 * (K // 8 + 16) * U32 * mag
    if fa == E4M3:
        # largest magnitudes by group; none counts less than its format's
        # smallest normal value
        big_a = torch.maximum(a.abs(), block_floor(sa, 2.0 ** -6)).view(a.shape[0], -1, 8).amax(2)
        big_w = torch.maximum(w.abs(), block_floor(sw, 1.0)).view(w.shape[0], -1, 8).amax(2)
        err = err + 8 * 2.0 ** -13 * (big_a @ big_w.t().contiguous())
    return (torch.where(c > 0, c, torch.zeros_like(c)) if relu else c), err


def block_floor(s, least):
    p = least * torch.exp2(s.double().clamp(max=254) - 127.0)
    return p.repeat_interleave(32, dim=1)


def assert_close(got, want, err, dtype, name=""):
    """|got - want| <= err and half a step of the result's type; NaN where NaN."""
    got, want = got.double(), want.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), "%s: NaN in other places" % name
    tol = err + HALF_STEP[dtype] * (want.abs() + err) + TINY[dtype]
    off = torch.where(nan, torch.zeros_like(got), (got - want).abs())
    bad = off > torch.where(nan, torch.zeros_like(tol), tol)
    assert not bad.any(), "%s: %d of %d outside; worst %g of its bound" % (
        name, int(bad.sum()), bad.numel(), float((off / tol)[bad].max()))


# --------------------------------------------------------------------------
# Head norms with rotation.
# --------------------------------------------------------------------------
# Longest chain of fp32 additions in a head's sum: 16 values in a lane and six
# steps in a wave, rounded up; relative error of r: half the sum's, then the mean,
# eps, root and reciprocal.
CHAIN = 32
R_ERR = (CHAIN / 2 + 6) * U32


def pairs(D, R, interleaved):
    first = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    return first, first + (1 if interleaved else R // 2)


def turn(v, cos, sin, R, interleaved, back=False):
    """(turned, turned magnitudes): v [T, H, D], cos and sin [T, R / 2]."""
    i, j = (p.to(v.device) for p in pairs(v.shape[2], R, interleaved))
    c = cos.double().unsqueeze(1)
    s = sin.double().unsqueeze(1) * (-1.0 if back else 1.0)
    out, mag = v.clone(), v.abs()
    a, b = v[:, :, i], v[:, :, j]
    out[:, :, i], out[:, :, j] = a * c - b * s, a * s + b * c
    mag[:, :, i] = a.abs() * c.abs() + b.abs() * s.abs()
    mag[:, :, j] = a.abs() * s.abs() + b.abs() * c.abs()
    return out, mag


def heads_forward(x, w, cos, sin, R, eps, interleaved):
    """(out, bound on its error before the output's rounding)."""
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps)
    y = x * r if w is None else x * r * w.double()
    out, mag = turn(y, cos, sin, R, interleaved)
    return out, mag * (R_ERR + 5 * U32)


def heads_backward(d, x, w, cos, sin, R, eps, interleaved):
    """(dx, dw, bounds of both)."""
    d, x = d.double(), x.double()
    T, H, D = x.shape
    r = 1.0 / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps)
    n = x * r
    dy, ady = turn(d, cos, sin, R, interleaved, back=True)
    wd = 1.0 if w is None else w.double()
    p, ap = dy * wd, ady * (1.0 if w is None else w.double().abs())
    dx = r * (p - n * (p * n).mean(dim=2, keepdim=True))
    e32 = 2 * R_ERR + (CHAIN + 8) * U32
    ex = e32 * r * (ap + n.abs() * (ap * n.abs()).mean(dim=2, keepdim=True))
    dw = (dy * n).sum(dim=(0, 1))
    ew = (e32 + (T * H + 48) * U32) * (ady * n.abs()).sum(dim=(0, 1))
    return dx, dw, ex, ew


def tables(P, pairs_, base=10000.0):
    i = torch.arange(pairs_, dtype=torch.float64)
    a = torch.arange(P, dtype=torch.float64)[:, None] * base ** (-i / max(pairs_, 1))[None, :]
    return torch.cos(a).float(), torch.sin(a).float()
