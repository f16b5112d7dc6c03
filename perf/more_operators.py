"""Measured cases of the microscaled 4-bit linear path and of the norms of query and key heads.

What stands between a block's norm and its attention, forward and backward, as a serving or
training program calls it:

* ``quant_mx``        rows (or columns) of a matrix to microscaled blocks: 32 elements of 4 or 8
                      bits and one power of two each, and the values they stand for;
* ``linear_mx``       C = epilogue(Q(X) W^T + bias), X quantised within the call, W in 4 bits;
* ``linear_mx_backward``  dX = Q(dY) Q(W), dW = Q(dY)^T Q(X), blocks along the summed axis, and
                      the bias' gradient;
* ``head_norm_rope``  every query and key head normed and rotated to its token's position;
* ``head_norm_rope_backward``  its gradients.

``run`` computes them from elementary torch operations (``own`` false) or through the library's
entry points (``own`` true).  Shapes: the 8192-wide layers of the benchmark's 4-bit workloads and
generic block and head sizes.
"""

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32
PAD = 128  # rows of codes are whole runs of 128 elements, zeros past the end

LARGEST_PRODUCT = 8192 ** 3
LARGEST_MATRIX = 8192 ** 2
LARGEST_HEADS = 8192 * 40 * 128


def _quant(name, M, K, dt, fmt, sides):
    # sides: "rows", "columns" or "both"
    return {"name": name, "op": "quant_mx", "M": M, "K": K, "type": dt, "fmt": fmt,
            "sides": sides}


def _linear(name, op, M, N, K, dt, fmt, bias=False, relu=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "type": dt, "fmt": fmt,
            "bias": bias, "relu": relu}


def _heads(name, op, T, Hq, Hk, D, R, dt, interleaved=False, order="run"):
    # order of positions: "run" (a prompt from some place on) or "any" (a decode batch)
    return {"name": name, "op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "type": dt,
            "interleaved": interleaved, "order": order}


def listed():
    return [
        # a layer's weights brought to 4 bits, and what they stand for
        _quant("quant_weights", 8192, 8192, "bf16", "e2m1", "rows"),
        # activations of a training step, blocks along both axes, odd sizes, 8 bits
        _quant("quant_both_odd", 1537, 2047, "f32", "e4m3", "both"),
        # one token of a small model, where latency counts
        _linear("linear_one_token", "linear_mx", 1, 1024, 1024, "bf16", "e2m1"),
        # a decode batch of 16 sequences through a wide layer, activations in 8 bits
        _linear("linear_decode_batch", "linear_mx", 16, 8192, 8192, "bf16", "e4m3", bias=True),
        # odd sizes in 32 bits
        _linear("linear_odd", "linear_mx", 1000, 1001, 1003, "f32", "e2m1", bias=True),
        # the largest product: a long prompt through a wide layer
        _linear("linear_long_prompt", "linear_mx", 8192, 8192, 8192, "bf16", "e2m1", relu=True),
        # the backward pass of a layer with a bias
        _linear("linear_train", "linear_mx_backward", 2048, 4096, 4096, "bf16", "e2m1", bias=True),
        # odd sizes, gradients in 8 bits
        _linear("linear_train_odd", "linear_mx_backward", 1000, 1001, 1003, "f16", "e4m3"),
        # one token before attention
        _heads("heads_one_token", "head_norm_rope", 1, 32, 8, 128, 128, "bf16", order="any"),
        # a long prompt before attention
        _heads("heads_prompt", "head_norm_rope", 8192, 32, 8, 128, 128, "bf16"),
        # the backward pass of that
        _heads("heads_train", "head_norm_rope_backward", 8192, 32, 8, 128, 128, "bf16"),
        # heads of an odd length in 32 bits, a part of them rotated, neighbours paired
        _heads("heads_train_odd", "head_norm_rope_backward", 1537, 12, 3, 99, 66, "f32",
               interleaved=True),
    ]


def _spread(rng, lo, hi):
    """A size, spread over the logarithm of [lo, hi]; a third of them as drawn, the others
    multiples of 64 where that is in the range (layers' widths are)."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.67 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quant_mx", "linear_mx", "linear_mx", "linear_mx", "linear_mx_backward",
                     "linear_mx_backward", "head_norm_rope", "head_norm_rope_backward"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    fmt = rng.choice(["e2m1", "e2m1", "e4m3"])
    if op == "quant_mx":
        K = _spread(rng, 32, 8192)
        M = min(_spread(rng, 1, 8192), LARGEST_MATRIX // K)
        return {"op": op, "M": M, "K": K, "type": dt, "fmt": fmt,
                "sides": rng.choice(["rows", "columns", "both"])}
    if op.startswith("linear"):
        if dt == "f32":
            fmt = "e2m1"  # a 32-bit model keeps what 4-bit products hold exactly
        c = {"op": op, "M": _spread(rng, 1, 8192), "N": _spread(rng, 128, 8192),
             "K": _spread(rng, 128, 8192), "type": dt, "fmt": fmt, "bias": rng.random() < 0.5,
             "relu": op == "linear_mx" and rng.random() < 0.5}
        if op == "linear_mx_backward":
            c["M"] = max(1, min(c["M"], LARGEST_PRODUCT // 4 // (c["N"] * c["K"])))
        return c
    D = rng.choice([64, 96, 128, 128, 256, rng.randint(16, 256)])
    R = rng.choice([D // 2 * 2, D // 2 * 2, D // 4 * 2, 2 * rng.randint(0, D // 2)])
    Hk = rng.choice([1, 2, 4, 8, rng.randint(1, 9)])
    Hq = Hk * rng.choice([1, 2, 4, rng.randint(1, 8)])
    T = min(_spread(rng, 1, 8192), LARGEST_HEADS // ((Hq + Hk) * D))
    return {"op": op, "T": max(1, T), "Hq": Hq, "Hk": Hk, "D": D, "R": R, "type": dt,
            "interleaved": rng.random() < 0.5, "order": rng.choice(["run", "any"])}


def _blocks(v):
    """Rows of v, zeros past the end up to a whole run of PAD, as blocks of 32, in 32 bits."""
    M, K = v.shape
    out = torch.zeros((M, -(-K // PAD) * PAD), dtype=torch.float32, device=v.device)
    out[:, :K] = v
    return out.view(M, -1, BLOCK)


def _mx(v, fmt):
    """Elements and powers of two of the rows of v in blocks of 32: the power is the one that
    brings the largest magnitude to the format's highest octave, what is still above the largest
    element becomes that.  Every step is exact but the rounding to the element, ties to even."""
    b = _blocks(v)
    top, octave, least = (6.0, 2, 0) if fmt == "e2m1" else (448.0, 8, -6)
    frac = 1 if fmt == "e2m1" else 3
    e = (torch.frexp(b.abs().amax(dim=2, keepdim=True))[1] - 1 - octave).clamp(-127, 127)
    e = torch.where(b.abs().amax(dim=2, keepdim=True) > 0, e, torch.full_like(e, -127))
    u = torch.ldexp(b, -e)
    step = torch.ldexp(torch.ones_like(u),
                       (torch.frexp(u)[1] - 1).clamp(min=least) - frac)
    return (torch.round(u / step) * step).clamp(-top, top), e


def _values(q, e):
    return torch.ldexp(q, e).view(q.shape[0], -1)


def _codes(q, e):
    """4-bit codes, two to a byte, and scale bytes, as a checkpoint holds them."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    c = torch.bucketize(q.abs(), table) + 8 * (q < 0)
    c = c.view(q.shape[0], -1, 2)
    return ((c[:, :, 0] | c[:, :, 1] << 4).to(torch.uint8),
            (e.view(q.shape[0], -1) + 127).to(torch.uint8))


def _decode(codes, scales, dtype):
    """What packed 4-bit codes and scale bytes stand for."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0, -0.5, -1.0, -1.5, -2.0,
                          -3.0, -4.0, -6.0], dtype=dtype, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=2).to(torch.int32)
    v = table[c].view(codes.shape[0], -1, BLOCK)
    return (v * torch.exp2(scales.to(dtype) - 127.0).unsqueeze(2)).view(codes.shape[0], -1)


def _activations(M, K, dt, g):
    """Activations with a few channels larger than the others."""
    spread = torch.exp(0.5 * torch.randn((1, K), generator=g, device="cuda"))
    return (torch.randn((M, K), generator=g, device="cuda") * spread).to(DT[dt])


def _angles(R, P, base=10000.0):
    """Cosines and sines of every position, from angles in 64 bits."""
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    a = (torch.arange(P, dtype=torch.float64, device="cuda")[:, None]
         * base ** (-2.0 * i / max(R, 1))[None, :])
    return torch.cos(a).float(), torch.sin(a).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dt = DT[case["type"]]
    randn = lambda *size: torch.randn(size, generator=g, device="cuda")
    if case["op"] == "quant_mx":
        s["X"] = _activations(case["M"], case["K"], case["type"], g)
        return s
    if case["op"] == "linear_mx":
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = _activations(M, K, case["type"], g)
        # a checkpoint's layer, laid out once
        s["Wq"], s["Ws"] = _codes(*_mx(randn(N, K) / K ** 0.5, "e2m1"))
        s["b"] = randn(N) if case["bias"] else None
        s["C"] = torch.empty((M, N), dtype=dt, device="cuda")  # kept by a serving program
        return s
    if case["op"] == "linear_mx_backward":
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = _activations(M, K, case["type"], g)
        s["dY"] = randn(M, N).to(dt)
        s["W"] = (randn(N, K) / K ** 0.5).to(dt)
        return s
    T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
    # the heads are slices of one projection's output, values behind them
    x = (2.0 * randn(T, (Hq + 2 * Hk) * D)).to(dt)
    s["q"] = x[:, :Hq * D].unflatten(1, (Hq, D))
    s["k"] = x[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    s["wq"], s["wk"] = ((1.0 + 0.2 * randn(D)).to(dt) for _ in range(2))
    P = 32768
    if case["order"] == "run":
        first = int(torch.randint(0, P - T + 1, (1,), generator=g, device="cuda"))
        s["pos"] = torch.arange(first, first + T, device="cuda")
    else:
        s["pos"] = torch.randint(0, P, (T,), generator=g, device="cuda")
    s["cos"], s["sin"] = _angles(R, P)
    if case["op"] == "head_norm_rope_backward":
        s["dqo"], s["dko"] = randn(T, Hq, D).to(dt), randn(T, Hk, D).to(dt)
    return s


def _rotate(v, s, sign):
    """The first R elements of every head as pairs, turned by the token's angles."""
    R, D = s["R"], v.shape[2]
    c = s["cos"][s["pos"]].unsqueeze(1)
    n = s["sin"][s["pos"]].unsqueeze(1) * sign
    if s["interleaved"]:
        a, b = v[:, :, 0:R:2], v[:, :, 1:R:2]
        turned = torch.stack([a * c - b * n, a * n + b * c], dim=3).flatten(2)
    else:
        a, b = v[:, :, :R // 2], v[:, :, R // 2:R]
        turned = torch.cat([a * c - b * n, a * n + b * c], dim=2)
    return torch.cat([turned, v[:, :, R:]], dim=2) if R < D else turned


def _normed(x):
    x = x.float()
    r = 1.0 / torch.sqrt((x * x).mean(dim=2, keepdim=True) + EPS)
    return x * r, r


def _heads_backward(x, w, d, s):
    n, r = _normed(x)
    dy = _rotate(d.float(), s, -1.0)
    dn = dy * w.float()
    dx = r * (dn - n * (dn * n).mean(dim=2, keepdim=True))
    return dx.to(x.dtype), (dy * n).sum(dim=(0, 1))


def _run_plain(s):
    op = s["op"]
    if op == "quant_mx":
        out, K, M = {}, s["K"], s["M"]
        if s["sides"] != "columns":
            out["rows"] = _values(*_mx(s["X"], s["fmt"]))[:, :K].to(s["X"].dtype)
        if s["sides"] != "rows":
            out["columns"] = _values(*_mx(s["X"].t(), s["fmt"]))[:, :M].to(s["X"].dtype)
        return out
    if op == "linear_mx":
        v = _values(*_mx(s["X"], s["fmt"])) @ _decode(s["Wq"], s["Ws"], torch.float32).t()
        if s["b"] is not None:
            v = v + s["b"][None, :]
        if s["relu"]:
            v = torch.where(v > 0, v, torch.zeros_like(v))
        return v.to(s["C"].dtype)
    if op == "linear_mx_backward":
        fmt, dt = s["fmt"], s["dY"].dtype
        M, N, K = s["M"], s["N"], s["K"]
        d, w = _values(*_mx(s["dY"], fmt)), _values(*_mx(s["W"].t(), "e2m1"))
        out = {"dx": (d @ w.t()).to(dt)}
        d, x = _values(*_mx(s["dY"].t(), fmt)), _values(*_mx(s["X"].t(), "e2m1"))
        out["dw"] = (d @ x.t()).to(dt)
        if s["bias"]:
            out["dbias"] = s["dY"].float().sum(dim=0)
        return out
    if op == "head_norm_rope":
        return {n: _rotate(_normed(s[n])[0] * s["w" + n].float(), s, 1.0).to(s[n].dtype)
                for n in ("q", "k")}
    out = {}
    for n in ("q", "k"):
        out["d" + n], out["dw" + n] = _heads_backward(s[n], s["w" + n], s["d%so" % n], s)
    return out


def _run_own(s):
    from tiled_dense_gemm_07_amd import binding
    op = s["op"]
    if "fmt" in s:
        fmt = binding.TG_MX_E2M1 if s["fmt"] == "e2m1" else binding.TG_MX_E4M3
    if op == "quant_mx":
        f = binding.quant_mx(s["X"], fmt, sides=s["sides"])
        out, dt = {}, s["X"].dtype
        if f.q is not None:
            out["rows"] = binding.dequant_mx(f.q, f.s, fmt, K=s["K"], dtype=dt)
        if f.qt is not None:
            out["columns"] = binding.dequant_mx(f.qt, f.st, fmt, K=s["M"], dtype=dt)
        return out
    if op == "linear_mx":
        return binding.linear_mx(s["X"], s["Wq"], s["Ws"], bias=s["b"], fmt=fmt, C=s["C"],
                                 epilogue="relu" if s["relu"] else None)
    if op == "linear_mx_backward":
        f = binding.linear_mx_backward(s["dY"], X=s["X"], W=s["W"], fmt=fmt, dbias=s["bias"])
        out = {"dx": f.dx, "dw": f.dw}
        if s["bias"]:
            out["dbias"] = f.dbias
        return out
    if op == "head_norm_rope":
        f = binding.head_norm_rope(s["q"], s["k"], s["wq"], s["wk"], cos=s["cos"], sin=s["sin"],
                                   positions=s["pos"], eps=EPS, interleaved=s["interleaved"])
        return {"q": f.q, "k": f.k}
    f = binding.head_norm_rope_backward(s["dqo"], s["dko"], s["q"], s["k"], s["wq"], s["wk"],
                                        cos=s["cos"], sin=s["sin"], positions=s["pos"], eps=EPS,
                                        interleaved=s["interleaved"])
    return {"dq": f.dq, "dwq": f.dw_q, "dk": f.dk, "dwk": f.dw_k}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _code_bytes(rows, K, fmt):
    return rows * -(-K // BLOCK) * (BLOCK // 2 + 1 if fmt == "e2m1" else BLOCK + 1)


def work(case):
    op, e = case["op"], SIZE[case["type"]]
    if op == "quant_mx":
        # the matrix in; codes, scales and the values they stand for out
        M, K = case["M"], case["K"]
        out = 0
        if case["sides"] != "columns":
            out += _code_bytes(M, K, case["fmt"]) + e * M * K
        if case["sides"] != "rows":
            out += _code_bytes(K, M, case["fmt"]) + e * M * K
        return {"bytes": e * M * K + out, "flops": 4 * M * K}
    if op == "linear_mx":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": e * M * K + _code_bytes(N, K, "e2m1") + (4 * N if case["bias"] else 0)
                + e * M * N, "flops": 2 * M * N * K}
    if op == "linear_mx_backward":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": e * (M * N + 2 * M * K + 2 * N * K) + (4 * N if case["bias"] else 0),
                "flops": 4 * M * N * K}
    T, D, R, H = case["T"], case["D"], case["R"], case["Hq"] + case["Hk"]
    shared = T * (4 * R + 8) + 2 * e * D
    if op == "head_norm_rope":
        return {"bytes": 2 * e * T * H * D + shared, "flops": 10 * T * H * D}
    return {"bytes": 3 * e * T * H * D + shared + 8 * D, "flops": 20 * T * H * D}


# The definitions in 64 bits, term by term, apart from the forms above.

def _exact_mx(v, fmt):
    """Rows of v (64 bits) as what their microscaled blocks stand for."""
    bits, top, high, low = (2, 6.0, 4.0, 1.0) if fmt == "e2m1" else (4, 448.0, 256.0, 2.0 ** -6)
    parts = []
    for b in v.split(BLOCK, dim=1):
        peak = b.abs().max(dim=1, keepdim=True).values
        # the power of two P with high <= peak / P < 2 high
        P = torch.exp2(torch.floor(torch.log2(peak.clamp(min=2.0 ** -126)))) / high
        P = torch.where(peak / P < high, P / 2, P)
        P = torch.where(peak / P >= 2 * high, P * 2, P)
        P = P.clamp(min=2.0 ** -127)
        m = (b / P).abs()
        octave = torch.exp2(torch.floor(torch.log2(m.clamp(min=low))))
        grid = octave * 2.0 ** (1 - bits)
        n = torch.floor(m / grid)
        left = m / grid - n
        n = n + ((left > 0.5) | ((left == 0.5) & (n % 2 == 1))).to(n.dtype)
        parts.append(torch.sign(b) * torch.minimum(n * grid, torch.full_like(m, top)) * P)
    return torch.cat(parts, dim=1)


def _exact_turn(v, s, back):
    """Every pair as a complex number, times the token's unit number (or its conjugate)."""
    R = s["R"]
    z = torch.complex(s["cos"].double(), s["sin"].double()).index_select(0, s["pos"])
    z = (z.conj() if back else z)[:, None, :]
    first = (torch.arange(0, R, 2, device="cuda") if s["interleaved"]
             else torch.arange(0, R // 2, device="cuda"))
    second = first + (1 if s["interleaved"] else R // 2)
    p = torch.complex(v[:, :, first].contiguous(), v[:, :, second].contiguous()) * z
    out = v.clone()
    out[:, :, first] = p.real
    out[:, :, second] = p.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f64, op = torch.float64, case["op"]
    if op == "quant_mx":
        x, out = s["X"].to(f64), {}
        if case["sides"] != "columns":
            out["rows"] = _exact_mx(x, case["fmt"])
        if case["sides"] != "rows":
            out["columns"] = _exact_mx(x.T.contiguous(), case["fmt"])
        return out
    if op == "linear_mx":
        w = _decode(s["Wq"], s["Ws"], f64)[:, :case["K"]]
        c = torch.mm(_exact_mx(s["X"].to(f64), case["fmt"]), w.T.contiguous())
        if s["b"] is not None:
            c += s["b"].to(f64)
        return c.clamp(min=0.0) if case["relu"] else c
    if op == "linear_mx_backward":
        d, x, w = s["dY"].to(f64), s["X"].to(f64), s["W"].to(f64)
        turn = lambda v, fmt: _exact_mx(v.T.contiguous(), fmt).T.contiguous()
        out = {"dx": torch.mm(_exact_mx(d, case["fmt"]), turn(w, "e2m1")),
               "dw": torch.mm(turn(d, case["fmt"]).T.contiguous(), turn(x, "e2m1"))}
        if case["bias"]:
            out["dbias"] = d.sum(0)
        return out
    out = {}
    for n in ("q", "k"):
        x, w = s[n].to(f64), s["w" + n].to(f64)
        inv = (x.square().sum(2, keepdim=True) / case["D"] + EPS).rsqrt()
        if op == "head_norm_rope":
            out[n] = _exact_turn(x * inv * w, s, False)
            continue
        dy = _exact_turn(s["d%so" % n].to(f64), s, True)
        # d(x r)/dx with r = (mean x^2 + eps)^(-1/2):  r I - r^3 x x^T / D
        p = dy * w
        out["d" + n] = inv * p - inv ** 3 * x * (p * x).sum(2, keepdim=True) / case["D"]
        out["dw" + n] = (dy * x * inv).sum((0, 1))
    return out
