"""The norms between blocks and their gradients on the GPU, through the C ABI,
against the plain 64-bit forms: every pair of types, odd row lengths, strides,
shared and per-token gates, left-out operands, special rows, streams, graphs."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import i8_norm_reference as ref
from gpu_helpers import BF16, F16, F32, bits_to_f64, say, to_host_bits, torch_dtype
from tiled_dense_gemm_07_amd import binding

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DNAME = {F32: "f32", F16: "f16", BF16: "bf16"}
PAIRS = [(BF16, BF16), (F16, F16), (F32, BF16), (F32, F16), (F32, F32)]
by_pair = pytest.mark.parametrize("xt,bt", PAIRS,
                                  ids=["%s_%s" % (DNAME[a], DNAME[b]) for a, b in PAIRS])
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def f64(t, dtype):
    return None if t is None else bits_to_f64(to_host_bits(t.contiguous(), dtype), dtype)


def rand(r, shape, dtype, scale=1.0, add=0.0):
    v = (add + scale * r.normal(size=shape)).astype(np.float32)
    return torch.from_numpy(v).to(torch_dtype(dtype)).to(DEV)


def strided(t, pad, shift):
    M, K = t.shape
    buf = torch.full((M * (K + pad) + shift + 1,), 9.0, dtype=t.dtype, device=DEV)
    out = buf[shift:shift + M * (K + pad)].view(M, K + pad)[:, :K]
    out.copy_(t)
    return out


def operands(T, D, xt, bt, gate_rows, post, seed, y=True):
    r = np.random.Generator(np.random.PCG64(seed))
    s = {"x": rand(r, (T, D), xt, 2.0), "w_pre": rand(r, (D,), bt, 0.2, 1.0)}
    s["y"] = rand(r, (T, D), bt) if y else None
    s["gate"] = rand(r, (-(-T // gate_rows), D), bt, 0.5) if gate_rows else None
    s["w_post"] = rand(r, (D,), bt, 0.2, 1.0) if post else None
    s["dx_new"], s["dh"] = rand(r, (T, D), xt), rand(r, (T, D), bt)
    return s


def within(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r against %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def check_forward(s, f, xt, bt, gate_rows, alpha, post):
    """x' against its formula, h against the formula on the stored x'."""
    x, y, gate = f64(s["x"], xt), f64(s["y"], bt), f64(s["gate"], bt)
    w1, w2 = f64(s["w_post"], bt), f64(s["w_pre"], bt)
    xo = x
    if y is not None:
        e = ref.forward(x, y, gate, gate_rows, w1, w2, alpha, EPS, post)["x_out"]
        xo = f64(f.x, xt)
        within(xo, e, ref.forward_bound(x, y, e - alpha * x, e, alpha, xt), "x'")
    h = ref.forward(xo, None, None, 0, None, w2, alpha, EPS, post)["h"]
    if f.h is not None and f.hs is None:
        within(f64(f.h, bt), h, ref.h_bound(h, bt), "h")
    elif f.h is not None:
        # levels of an h that is off by fp32 roundings: one level further at
        # the borders, and the scale off by those roundings
        q, sc = ref.levels(h)
        hs = f.hs.cpu().numpy().astype(np.float64)
        err = ref.R_ERR + 4 * ref.U32
        assert np.all(np.abs(hs - sc) <= sc * err)
        got = f.h.cpu().numpy().astype(np.float64)
        within(got, 127.0 * h / np.abs(h).max(axis=1, keepdims=True),
               0.5 + 127.0 * 2 * err, "levels")


@by_pair
@pytest.mark.parametrize("D", [1, 7, 8, 64, 500, 512, 513, 2047, 2048, 2056, 4096, 4099, 8192,
                               8200, 16384, 16385, 32768])
def test_forward_row_lengths(D, xt, bt):
    T = 3
    for post, gate_rows, out in ((True, 2, "h"), (False, 1, "i8")):
        s = operands(T, D, xt, bt, gate_rows, post, D)
        say("block_norm %dx%d %s/%s %s" % (T, D, DNAME[xt], DNAME[bt], out))
        f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                               w_post=s["w_post"], w_pre=s["w_pre"], alpha=0.75, eps=EPS,
                               post_norm=post, out=out, save=True)
        torch.cuda.synchronize()
        check_forward(s, f, xt, bt, gate_rows, 0.75, post)
        xo = f64(f.x, xt)
        r2 = 1.0 / np.sqrt((xo * xo).mean(axis=1) + EPS)
        assert np.all(np.abs(f.r_pre.cpu().numpy() - r2) <= r2 * ref.R_ERR)
        if post:
            y = f64(s["y"], bt)
            r1 = 1.0 / np.sqrt((y * y).mean(axis=1) + EPS)
            assert np.all(np.abs(f.r_post.cpu().numpy() - r1) <= r1 * ref.R_ERR)
        else:
            assert f.r_post is None


@pytest.mark.parametrize("T", [1, 2, 5, 64, 300, 1031])
@pytest.mark.parametrize("D", [96, 1000, 4096])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 5000])
def test_forward_tokens_and_gates(T, D, gate_rows):
    s = operands(T, D, BF16, BF16, gate_rows, True, T)
    say("block_norm %dx%d gate_rows=%d" % (T, D, gate_rows))
    f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                           w_post=s["w_post"], w_pre=s["w_pre"], alpha=-0.5, eps=EPS)
    torch.cuda.synchronize()
    check_forward(s, f, BF16, BF16, gate_rows, -0.5, True)


@by_pair
def test_forward_left_out_operands(xt, bt):
    """Only the norm, only the residual, no weights, a shared 1-D gate."""
    T, D = 9, 200
    s = operands(T, D, xt, bt, 0, True, 1)
    say("block_norm parts %s/%s" % (DNAME[xt], DNAME[bt]))
    f = binding.block_norm(s["x"], w_pre=s["w_pre"], eps=EPS)  # pre-norm alone
    check_forward({**s, "y": None}, f, xt, bt, 0, 1.0, True)
    assert f.x is s["x"]
    f = binding.block_norm(s["x"], eps=EPS)  # h in x's type, no weight
    check_forward({**s, "y": None, "w_pre": None}, f, xt, xt, 0, 1.0, True)
    f = binding.block_norm(s["x"], y=s["y"], out=None, eps=EPS)  # no weights, no h
    assert f.h is None
    check_forward({**s, "w_post": None, "w_pre": None}, f, xt, bt, 0, 1.0, True)
    f = binding.block_norm(s["x"], y=s["y"], post_norm=False, out=None)
    within(f64(f.x, xt), f64(s["x"], xt) + f64(s["y"], bt),
           ref.forward_bound(f64(s["x"], xt), None, f64(s["y"], bt),
                             f64(s["x"], xt) + f64(s["y"], bt), 1.0, xt), "x + y")
    g = s["w_post"]
    f = binding.block_norm(s["x"], y=s["y"], gate=g, w_pre=s["w_pre"], eps=EPS)
    check_forward({**s, "w_post": None, "gate": g[None]}, f, xt, bt, T, 1.0, True)


@by_pair
def test_forward_fused_equals_parts_and_in_place(xt, bt):
    """One call has the bits of two; x' in place of x; strided rows."""
    T, D = 37, 1000
    s = operands(T, D, xt, bt, 5, True, 3)
    kw = dict(y=s["y"], gate=s["gate"], gate_rows=5, w_post=s["w_post"], alpha=0.9, eps=EPS)
    say("block_norm fused and in place %s/%s" % (DNAME[xt], DNAME[bt]))
    f = binding.block_norm(s["x"], w_pre=s["w_pre"], **kw)
    a = binding.block_norm(s["x"], out=None, **kw)
    b = binding.block_norm(a.x, w_pre=s["w_pre"], eps=EPS,
                           h=torch.empty_like(s["y"]))
    assert torch.equal(f.x, a.x) and torch.equal(f.h, b.h)
    q = binding.block_norm(s["x"], w_pre=s["w_pre"], out="i8", **kw)
    p = binding.block_norm(a.x, w_pre=s["w_pre"], eps=EPS, out="i8")
    assert torch.equal(q.h, p.h) and torch.equal(q.hs, p.hs) and torch.equal(q.x, f.x)
    x = s["x"].clone()
    g = binding.block_norm(x, w_pre=s["w_pre"], x_out=x, **kw)
    assert g.x is x and torch.equal(x, f.x) and torch.equal(g.h, f.h)
    xs, ys = strided(s["x"], 7, 1), strided(s["y"], 3, 3)
    h = strided(torch.zeros_like(s["y"]), 5, 1)
    xo = strided(torch.zeros_like(s["x"]), 1, 2)
    kw["y"] = ys
    binding.block_norm(xs, w_pre=s["w_pre"], x_out=xo, h=h, **kw)
    torch.cuda.synchronize()
    assert torch.equal(xo, f.x) and torch.equal(h, f.h)
    base = xo.as_strided((T - 1,), (D + 1,), xo.storage_offset() + D)  # the gaps
    assert bool((base == 9.0).all())


def test_forward_special_rows():
    """A row of zeros, rows with an infinity or NaN: the others are untouched."""
    T, D = 8, 600
    s = operands(T, D, BF16, BF16, 1, True, 4)
    s["x"][1], s["y"][1] = 0, 0
    s["y"][2, 5] = float("nan")
    s["x"][3, 599] = float("inf")
    s["x"][4] = 0  # the row that is left is y's
    say("block_norm special rows")
    for out in ("h", "i8"):
        f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], w_post=s["w_post"],
                               w_pre=s["w_pre"], eps=EPS, out=out)
        torch.cuda.synchronize()
        ok = [i for i in range(T) if i not in (2, 3)]
        t = {k: (v[ok] if v is not None and v.dim() == 2 else v) for k, v in s.items()}
        g = binding.BlockNorm(f.x[ok], f.h[ok], None if f.hs is None else f.hs[ok], None, None)
        if out == "h":
            check_forward(t, g, BF16, BF16, 1, 1.0, True)
            assert not bool(f.h[1].any())
            assert bool(f.h[2].isnan().all()) and bool(f.h[3].isnan().any())
        else:
            assert not bool(f.h[1].any()) and f.hs[1].item() == 2.0 ** -126
            assert bool(f.hs[2:4].isnan().all()) and not bool(f.h[2:4].any())
            assert bool(f.hs[ok].isfinite().all())


def test_forward_empty():
    say("block_norm T = 0")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    f = binding.block_norm(x, y=x)
    assert f.x.shape == (0, 64) and f.h.shape == (0, 64)
    g = binding.block_norm_backward(x, x, x, y=x, w_pre=x.new_ones(64),
                                    w_post=x.new_ones(64), r_post=torch.zeros(0, device=DEV),
                                    r_pre=torch.zeros(0, device=DEV))
    torch.cuda.synchronize()
    assert not bool(g.dw_pre.any()) and not bool(g.dw_post.any())


def run_backward(s, f, xt, bt, gate_rows, alpha, post, **kw):
    return binding.block_norm_backward(
        f.x, kw.get("dx_new", s["dx_new"]), kw.get("dh", s["dh"]), y=s["y"], gate=s["gate"],
        gate_rows=gate_rows, w_post=s["w_post"], w_pre=s["w_pre"], r_post=f.r_post, r_pre=f.r_pre,
        alpha=alpha, post_norm=post)


def check_backward(s, f, g, xt, bt, gate_rows, alpha, post, dx_new=True, dh=True):
    b = {}
    want = ref.backward(
        f64(f.x, xt), f64(s["dx_new"], xt) if dx_new else None, f64(s["dh"], bt) if dh else None,
        f64(s["y"], bt), f64(s["gate"], bt), gate_rows, f64(s["w_post"], bt), f64(s["w_pre"], bt),
        None if f.r_post is None else f64(f.r_post, F32),
        None if f.r_pre is None else f64(f.r_pre, F32), alpha, post, bounds=b)
    for name, dt in (("dx", xt), ("dy", bt), ("dgate", F32), ("dw_post", F32), ("dw_pre", F32)):
        got = getattr(g, name)
        assert (got is None) == (name not in want), name
        if got is not None:
            e = b[name]
            within(f64(got, dt).reshape(want[name].shape), want[name],
                   e + ref.HALF_STEP[dt] * (np.abs(want[name]) + e) + ref.TINY[dt], name)


@by_pair
@pytest.mark.parametrize("D", [1, 9, 64, 512, 520, 2047, 2048, 4096, 4100, 8192, 16384, 16390,
                               32768])
def test_backward_row_lengths(D, xt, bt):
    T = 11
    for post, gate_rows in ((True, 4), (False, 1)):
        s = operands(T, D, xt, bt, gate_rows, post, D)
        say("block_norm_backward %dx%d %s/%s post=%d" % (T, D, DNAME[xt], DNAME[bt], post))
        f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                               w_post=s["w_post"], w_pre=s["w_pre"], alpha=0.75, eps=EPS,
                               post_norm=post, save=True)
        g = run_backward(s, f, xt, bt, gate_rows, 0.75, post)
        torch.cuda.synchronize()
        check_backward(s, f, g, xt, bt, gate_rows, 0.75, post)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 100, 511, 4099])
@pytest.mark.parametrize("gate_rows", [0, 1, 2, 3, 8, 13, 64, 1000, 9999])
def test_backward_tokens_and_gates(T, gate_rows):
    """Gate rows shared by parts of a workgroup's rows, by exactly them, and by
    many workgroups."""
    D = 160
    s = operands(T, D, F32, BF16, gate_rows, True, T + gate_rows)
    say("block_norm_backward %dx%d gate_rows=%d" % (T, D, gate_rows))
    f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                           w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, save=True)
    g = run_backward(s, f, F32, BF16, gate_rows, 1.0, True)
    torch.cuda.synchronize()
    check_backward(s, f, g, F32, BF16, gate_rows, 1.0, True)
    again = run_backward(s, f, F32, BF16, gate_rows, 1.0, True)
    torch.cuda.synchronize()
    for a, b in zip(g, again):  # sums in a fixed order
        assert a is None and b is None or torch.equal(a, b)


@by_pair
def test_backward_left_out_operands(xt, bt):
    T, D = 21, 300
    s = operands(T, D, xt, bt, 4, True, 8)
    kw = dict(y=s["y"], gate=s["gate"], gate_rows=4, w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS,
              save=True)
    f = binding.block_norm(s["x"], **kw)
    say("block_norm_backward parts %s/%s" % (DNAME[xt], DNAME[bt]))
    g = run_backward(s, f, xt, bt, 4, 1.0, True, dx_new=None)
    check_backward(s, f, g, xt, bt, 4, 1.0, True, dx_new=False)
    g = run_backward(s, f, xt, bt, 4, 1.0, True, dh=None)
    assert g.dw_pre is None
    check_backward(s, f, g, xt, bt, 4, 1.0, True, dh=False)
    # the norm alone
    f = binding.block_norm(s["x"], w_pre=s["w_pre"], eps=EPS, save=True)
    g = binding.block_norm_backward(f.x, s["dx_new"], s["dh"], w_pre=s["w_pre"], r_pre=f.r_pre)
    check_backward({**s, "y": None, "gate": None, "w_post": None}, f, g, xt, bt, 0, 1.0, True)
    # no weights, no gate
    t = {**s, "gate": None, "w_post": None, "w_pre": None}
    f = binding.block_norm(s["x"], y=s["y"], eps=EPS, save=True)
    g = run_backward(t, f, xt, bt, 0, 1.0, True)
    check_backward(t, f, g, xt, bt, 0, 1.0, True)


def test_backward_against_differences():
    """The GPU gradients against central differences of the 64-bit forward
    formulas, along random directions."""
    T, D, gate_rows, alpha = 12, 96, 5, 0.8
    s = operands(T, D, F32, F32, gate_rows, True, 21)
    f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                           w_post=s["w_post"], w_pre=s["w_pre"], alpha=alpha, eps=EPS, save=True)
    g = run_backward(s, f, F32, F32, gate_rows, alpha, True)
    torch.cuda.synchronize()
    v = {k: f64(t, F32) for k, t in s.items()}
    r = np.random.Generator(np.random.PCG64(0))

    def loss(v):
        o = ref.forward(v["x"], v["y"], v["gate"], gate_rows, v["w_post"], v["w_pre"], alpha, EPS,
                        True)
        return (v["dx_new"] * o["x_out"]).sum() + (v["dh"] * o["h"]).sum()

    for k, got in (("x", g.dx), ("y", g.dy), ("gate", g.dgate), ("w_post", g.dw_post),
                   ("w_pre", g.dw_pre)):
        step, e = r.normal(size=v[k].shape), 1e-5
        d = (loss({**v, k: v[k] + e * step}) - loss({**v, k: v[k] - e * step})) / (2 * e)
        got = f64(got, F32).reshape(step.shape)
        # fp32 gradients, each good to (CHAIN + 8) roundings of its terms
        assert abs(d - (got * step).sum()) <= 1e-6 * abs(d) + 1e-5 * np.abs(got * step).sum(), k


def test_backward_strides():
    T, D = 33, 250
    s = operands(T, D, BF16, BF16, 7, True, 5)
    f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=7, w_post=s["w_post"],
                           w_pre=s["w_pre"], eps=EPS, save=True)
    want = run_backward(s, f, BF16, BF16, 7, 1.0, True)
    t = {**s, "y": strided(s["y"], 3, 1), "dx_new": strided(s["dx_new"], 5, 0),
         "dh": strided(s["dh"], 0, 3)}
    say("block_norm_backward strided")
    got = run_backward(t, f._replace(x=strided(f.x, 1, 1)), BF16, BF16, 7, 1.0, True)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("gate_rows", [1, 30, 100])
def test_backward_workspace_contents_do_not_matter(gate_rows):
    T, D = 100, 200
    s = operands(T, D, BF16, BF16, gate_rows, True, 5)
    f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
                           w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, save=True)
    want = run_backward(s, f, BF16, BF16, gate_rows, 1.0, True)
    a = binding.BlockNormGradArgs()
    one = 0x1000  # sizes depend on which operands are there, not on where
    a.T, a.D, a.xtype, a.btype, a.gate_rows, a.post_norm = T, D, BF16, BF16, gate_rows, 1
    for k in ("y", "gate", "dgate", "dw_post", "dw_pre"):
        setattr(a, k, one)
    a.ldy = D
    n = ctypes.c_size_t()
    assert binding.load_library().tg_block_norm_backward_workspace_size(ctypes.byref(a),
                                                                        ctypes.byref(n)) == 0
    ws = torch.full((n.value + 512,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN
    say("block_norm_backward workspace gate_rows=%d" % gate_rows)
    got = binding.block_norm_backward(
        f.x, s["dx_new"], s["dh"], y=s["y"], gate=s["gate"], gate_rows=gate_rows,
        w_post=s["w_post"], w_pre=s["w_pre"], r_post=f.r_post, r_pre=f.r_pre,
        workspace=ws[:n.value])
    torch.cuda.synchronize()
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    assert bool((ws[n.value:] == 0xFF).all())


def test_refusals():
    x = torch.zeros((6, 32), dtype=torch.bfloat16, device=DEV)
    for y in (x.float(), x.half()):  # pairs of types that are not offered
        with pytest.raises(binding.TileGemmError) as e:
            binding.block_norm(x, y=y)
        assert e.value.status == 3
    with pytest.raises(TypeError, match="unsupported dtype"):
        binding.block_norm(x, y=x.double())
    with pytest.raises(ValueError, match="gate_rows is needed"):
        binding.block_norm(x, y=x, gate=x[:3].clone())
    with pytest.raises(ValueError, match="gate must be"):
        binding.block_norm(x, y=x, gate=x[:3].clone(), gate_rows=3)
    with pytest.raises(ValueError, match="dense vector"):
        binding.block_norm(x, w_pre=x[0, :16])
    with pytest.raises(ValueError, match="y must be"):
        binding.block_norm(x, y=x[:, :16])
    with pytest.raises(ValueError, match="overlap"):
        binding.block_norm(x[:1].expand(6, 32))
    with pytest.raises(binding.TileGemmError) as e:
        binding.block_norm(x, y=x, post_norm=False, w_post=x[0])
    assert e.value.status == 8
    with pytest.raises(binding.TileGemmError) as e:
        binding.block_norm_backward(x, x, x)  # dh without r_pre
    assert e.value.status == 1


def test_stream_and_graph():
    """Forward and backward captured and replayed with new inputs between
    eager calls; the same bits as the eager calls."""
    T, D = 130, 512
    sets = [operands(T, D, BF16, BF16, 50, True, i) for i in range(3)]

    def both(s, ws=None, stream=None, buf=None):
        f = binding.block_norm(s["x"], y=s["y"], gate=s["gate"], gate_rows=50, w_post=s["w_post"],
                               w_pre=s["w_pre"], eps=EPS, save=True, stream=stream)
        g = binding.block_norm_backward(
            f.x, s["dx_new"], s["dh"], y=s["y"], gate=s["gate"], gate_rows=50, w_post=s["w_post"],
            w_pre=s["w_pre"], r_post=f.r_post, r_pre=f.r_pre, workspace=ws, stream=stream)
        return [f.x, f.h, *g]

    want = [both(s) for s in sets]
    torch.cuda.synchronize()
    say("block_norm on a side stream")
    got = both(sets[0], stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    s = {k: v.clone() for k, v in sets[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(s)
    say("block_norm graph replays")
    for i in (0, 1, 2, 1):
        for k, v in s.items():
            v.copy_(sets[i][k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        again = both(sets[2 - i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want[2 - i]))


def test_offsets_past_31_bits():
    """Rows beyond 2^31 bytes of every matrix: the last rows have the bits of
    a call on them alone, and sums over all rows those of a plain sum."""
    T, D = 300000, 4096  # 2.4 GB a matrix
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn((T, D), dtype=torch.bfloat16, device=DEV, generator=g)
    y = torch.randn((T, D), dtype=torch.bfloat16, device=DEV, generator=g)
    gate = torch.randn((3, D), dtype=torch.bfloat16, device=DEV, generator=g)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    say("block_norm %dx%d" % (T, D))
    f = binding.block_norm(x, y=y, gate=gate, gate_rows=100000, w_post=w, w_pre=w, save=True)
    e = binding.block_norm(x[-64:], y=y[-64:], gate=gate[2:], w_post=w, w_pre=w)
    torch.cuda.synchronize()
    assert torch.equal(f.x[-64:], e.x) and torch.equal(f.h[-64:], e.h)
    say("block_norm_backward %dx%d" % (T, D))
    b = binding.block_norm_backward(f.x, x, y, y=y, gate=gate, gate_rows=100000, w_post=w, w_pre=w,
                                    r_post=f.r_post, r_pre=f.r_pre)
    c = binding.block_norm_backward(f.x[-64:], x[-64:], y[-64:], y=y[-64:], gate=gate[2:],
                                    w_post=w, w_pre=w, r_post=f.r_post[-64:], r_pre=f.r_pre[-64:])
    torch.cuda.synchronize()
    assert torch.equal(b.dx[-64:], c.dx) and torch.equal(b.dy[-64:], c.dy)
    u = torch.zeros(D, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(u)
    for at in range(0, T, 20000):
        t = y[at:at + 20000].double() * f.x[at:at + 20000].double() * f.r_pre[at:at + 20000, None]
        u += t.sum(0)
        mag += t.abs().sum(0)
    # the longest chain: a workgroup's rows, the partial rows of a lane, and the last sums
    chain = T // 256 + 256 // 32 + 48
    assert bool(((b.dw_pre - u).abs() <= chain * ref.U32 * mag).all())
