"""GPU tests of the microscaled linear path against its 64-bit forms: codes,
scales and values bit for bit, products and gradients within counted roundings."""

import numpy as np
import pytest
import torch

import mx_heads_reference as ref
from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FMTS = [ref.E2M1, ref.E4M3]


def rand(shape, seed, dtype, spread=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:  # neighbouring blocks of different size
        x = x * torch.exp(2.0 * torch.randn(shape, generator=g, device="cuda"))
    return x.to(dtype)


def check_rows(x, q, s, fmt, name):
    codes, scales = ref.quantise(x, fmt)
    assert q.shape == (x.shape[0], codes.shape[1] // (2 if fmt == ref.E2M1 else 1))
    assert torch.equal(s.to(torch.int64), scales), name + ": scales"
    assert torch.equal(ref.unpack(q, fmt), codes), name + ": codes"


QUANT_SHAPES = [(1, 1), (5, 2), (40, 3), (7, 4), (260, 5), (1, 32), (3, 33), (31, 7), (128, 128), (129, 127), (130, 257), (257, 1003),
                (2, 8200), (1000, 64), (640, 640)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", QUANT_SHAPES)
def test_quant_both_sides(M, K, dtype, fmt):
    say("quant_mx %d x %d %s %d" % (M, K, dtype, fmt))
    x = rand((M, K), M + K, dtype)
    rows = binding.quant_mx(x, fmt)
    check_rows(x, rows.q, rows.s, fmt, "rows")
    assert rows.qt is None and rows.st is None
    columns = binding.quant_mx(x, fmt, sides="columns")
    check_rows(x.t().contiguous(), columns.qt, columns.st, fmt, "columns")
    both = binding.quant_mx(x, fmt, sides="both")
    for a, b in ((both.q, rows.q), (both.s, rows.s), (both.qt, columns.qt), (both.st, columns.st)):
        assert torch.equal(a, b)
    v = binding.dequant_mx(both.q, both.s, fmt, K=K, dtype=dtype)
    want = ref.values(*ref.quantise(x, fmt), fmt)[:, :K].to(dtype)
    assert torch.equal(v, want)
    vt = binding.dequant_mx(both.qt, both.st, fmt, K=M, dtype=F32)
    assert torch.equal(vt, ref.values(*ref.quantise(x.t(), fmt), fmt)[:, :M].float())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quant_every_16_bit_value(dtype, fmt):
    # every bit pattern, in blocks of like size (sorted) and of any size (shuffled);
    # blocks with infinities and NaN among them
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    order = torch.argsort(torch.nan_to_num(x.float().abs(), nan=float("inf")))
    g = torch.Generator().manual_seed(3)
    mixed = x[torch.randperm(65536, generator=g)]
    near = x[order]
    x = torch.cat([x, near, mixed]).view(-1, 256).cuda()
    both = binding.quant_mx(x, fmt, sides="both")
    check_rows(x, both.q, both.s, fmt, "rows")
    check_rows(x.t().contiguous(), both.qt, both.st, fmt, "columns")
    assert torch.equal(binding.quant_mx(x, fmt).q, both.q)


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_32_bit_borders(fmt):
    # ties between elements and their neighbours, at every power of two; the least
    # and the largest magnitudes; blocks of zeros
    e = torch.arange(-149, 128, dtype=torch.float64)
    m = torch.arange(0, 32, dtype=torch.float64) / 4.0  # 0, 1/4 .. 7 3/4
    tie = (m[None, :] * torch.exp2(e - 2.0)[:, None]).float()
    up = torch.nextafter(tie, torch.full_like(tie, float("inf")))
    down = torch.nextafter(tie, torch.zeros_like(tie))
    x = torch.cat([tie, up, -down, tie * 0.0, tie * -0.0]).cuda()
    x = x[torch.isfinite(x).all(dim=1)]
    q = binding.quant_mx(x, fmt)
    check_rows(x, q.q, q.s, fmt, "rows")
    t = binding.quant_mx(x, fmt, sides="columns")
    check_rows(x.t().contiguous(), t.qt, t.st, fmt, "columns")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_rows_that_are_not_finite(dtype, fmt):
    x = rand((200, 300), 5, dtype)
    x[3, 7], x[3, 200], x[100, 0], x[199, 299] = (float("nan"), float("inf"), -float("inf"),
                                                  float("nan"))
    both = binding.quant_mx(x, fmt, sides="both")
    check_rows(x, both.q, both.s, fmt, "rows")
    check_rows(x.t().contiguous(), both.qt, both.st, fmt, "columns")
    v = binding.dequant_mx(both.q, both.s, fmt, K=300)
    assert torch.isnan(v[3, :32]).all() and not torch.isnan(v[3, 32:192]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_strides_offsets_and_kept_memory(dtype):
    big = rand((300, 700), 6, dtype)
    for view in (big[7:250, 3:518], big[::2, 1:640], big[:1, 5:6], big[5:6, ::1]):
        both = binding.quant_mx(view, ref.E2M1, sides="both")
        check_rows(view, both.q, both.s, ref.E2M1, "rows")
        check_rows(view.t(), both.qt, both.st, ref.E2M1, "columns")
    out = torch.full((243, 700), 7.0, dtype=dtype, device="cuda")
    f = binding.quant_mx(big[7:250, 3:518])
    binding.dequant_mx(f.q, f.s, K=515, X=out[:, 2:517])
    want = ref.values(*ref.quantise(big[7:250, 3:518], 0), 0)[:, :515].to(dtype)
    assert torch.equal(out[:, 2:517], want)
    assert (out[:, :2] == 7).all() and (out[:, 517:] == 7).all()
    # buffers of the caller, between guards
    raw = torch.full((128 + 243 * 320 + 128,), 0xA5, dtype=torch.uint8, device="cuda")
    q = raw[128:128 + 243 * 320].view(243, 320)
    binding.quant_mx(big[7:250, 3:518], q=q)
    assert torch.equal(q, f.q)
    assert (raw[:128] == 0xA5).all() and (raw[-128:] == 0xA5).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("fmt", FMTS)
def test_dequant_every_code_and_scale(fmt, dtype):
    # a block for every scale byte and 32 codes
    n = 16 if fmt == ref.E2M1 else 256
    codes = torch.arange(max(n, 128)) % n
    codes = codes.view(1, -1).expand(256, -1).contiguous()
    s = torch.arange(256).view(256, 1).expand(256, codes.shape[1] // 32).contiguous()
    v = ref.values(codes, s, fmt)
    got = binding.dequant_mx(ref.pack(codes, fmt).cuda(), s.to(torch.uint8).cuda(), fmt,
                             dtype=dtype).cpu()
    want = v.to(dtype)  # one rounding: fp32 holds each of these values or is beyond them
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


def test_offsets_past_32_bits():
    # more than 2^31 elements in, out and between; the ends are looked at
    M, K = 300001, 8192
    say("quant_mx and linear_mx %d x %d" % (M, K))
    x = torch.empty((M, K), dtype=BF16, device="cuda").normal_()
    both = binding.quant_mx(x, sides="both")
    end = x[-300:]
    check_rows(end, both.q[-300:], both.s[-300:], ref.E2M1, "rows")
    c, s = ref.quantise(x[-(M % 32) - 320:, -9:].t(), ref.E2M1)
    n = 320 + M % 32  # whole blocks from there on
    assert torch.equal(both.st[-9:, (M - n) // 32:(M + 31) // 32].long(), s[:, :(n + 31) // 32])
    assert torch.equal(ref.unpack(both.qt[-9:, (M - n) // 2:], 0)[:, :n], c[:, :n])
    v = binding.dequant_mx(both.q, both.s)
    assert torch.equal(v[-300:], ref.values(*ref.quantise(end, 0), 0).to(BF16))
    del v, both
    wq, ws = weights(8192, 128, 3)
    c = binding.linear_mx(x[:, 5:133], wq, ws)
    want, err = linear_want(end[:, 5:133], wq, ws, 0, None, False)
    ref.assert_close(c[-300:], want, err, BF16)


def test_quant_of_nothing():
    for shape in ((0, 64), (5, 0), (0, 0)):
        f = binding.quant_mx(torch.zeros(shape, device="cuda"), sides="both")
        assert f.q.numel() == 0 and f.qt.numel() == 0
        assert binding.dequant_mx(f.q, f.s, K=shape[1]).shape == shape


# --------------------------------------------------------------------------
# Linear layer.
# --------------------------------------------------------------------------
def weights(N, K, seed):
    w = rand((N, K), seed, F32, spread=False) / K ** 0.5
    f = binding.quant_mx(w)
    return f.q, f.s


def linear_want(x, wq, ws, fmt, bias, relu):
    cx, sx = ref.quantise(x, fmt)
    return ref.product(cx, sx, fmt, ref.unpack(wq, 0), ws.to(torch.int64), bias, relu)


def check_linear(M, N, K, dtype, fmt, bias, relu, seed=0, **kw):
    say("linear_mx %d x %d x %d %s fmt %d" % (M, N, K, dtype, fmt))
    x = rand((M, K), 10 + seed, dtype, spread=False)
    wq, ws = weights(N, K, 20 + seed)
    b = rand((N,), 30 + seed, F32, spread=False) if bias else None
    c = binding.linear_mx(x, wq, ws, bias=b, fmt=fmt, epilogue="relu" if relu else None, **kw)
    want, err = linear_want(x, wq, ws, fmt, b, relu)
    ref.assert_close(c, want, err, dtype, "linear")
    return c


LINEAR = [(1, 1, 1), (1, 16, 32), (1, 1024, 1024), (2, 130, 2048), (3, 17, 129), (5, 100, 250),
          (8, 64, 2048), (8, 256, 4096), (9, 33, 96), (16, 512, 384), (16, 1000, 8192), (17, 48, 640),
          (32, 300, 1003), (33, 64, 128), (64, 70, 1024), (100, 257, 900), (130, 130, 130),
          (257, 511, 1280), (512, 768, 2048), (1000, 1001, 1003)]


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("dtype,fmt", [(BF16, 0), (F32, 0), (F16, 1), (BF16, 1), (F32, 1), (F16, 0)])
def test_linear(M, N, K, dtype, fmt):
    check_linear(M, N, K, dtype, fmt, bias=(M + N) % 2 == 0, relu=(M + K) % 3 == 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(2048, 2048, 1024), (2048, 2304, 1152), (4100, 1999, 2048),
                                   (300, 4096, 4096), (1024, 8192, 256), (8192, 640, 128)])
def test_linear_large(M, N, K, dtype, fmt):
    check_linear(M, N, K, dtype, fmt, bias=True, relu=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(17, 8001, 200), (18, 5001, 2000), (32, 4097, 4200), (33, 6999, 384),
                                   (40, 6001, 1152), (48, 7011, 640), (49, 5001, 896), (64, 4097, 1500)])
def test_linear_some_tens_of_tokens(M, N, K, fmt):
    # 32 and 64 rows of weights to a workgroup, runs of 512 k and one to three steps
    check_linear(M, N, K, BF16, fmt, bias=M % 2 == 0, relu=M % 3 == 0)


def test_linear_is_the_product_of_its_parts():
    # bit for bit what quant_mx and gemm_mx give one after the other
    for M, K in ((48, 1024), (300, 2048)):
        x = rand((M, K), 1, BF16)
        wq, ws = weights(256, K, 2)
        for fmt in FMTS:
            f = binding.quant_mx(x, fmt)
            a = binding.gemm_mx(fmt, f.q, f.s, wq, ws).float()
            b = binding.linear_mx(x, wq, ws, fmt=fmt).float()
            assert (a - b).abs().max() <= 2.0 ** -7 * a.abs().max()


def test_linear_integer_sums_are_exact():
    # small integers: every partial sum is exact, so every order gives the same bits
    g = torch.Generator(device="cuda").manual_seed(4)
    pick = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()
    for M in (1, 7, 16, 40, 300):
        x, w = pick(M, 700), pick(200, 700)
        x[:, ::32], w[:, ::32] = 4.0, 4.0  # the same power of two for every block
        x[x.abs() == 3.5] = 0
        f = binding.quant_mx(w)
        for fmt in FMTS:
            c = binding.linear_mx(x, f.q, f.s, fmt=fmt)
            want, _ = linear_want(x, f.q, f.s, fmt, None, False)
            assert torch.equal(c.double(), want)


@pytest.mark.parametrize("M", [1, 3, 16, 100])
def test_linear_rows_that_are_not_finite(M):
    x = rand((M, 500), 3, BF16)
    x[0, 499] = float("inf")
    if M > 2:
        x[2, 40] = float("nan")
    wq, ws = weights(64, 500, 4)
    c = binding.linear_mx(x, wq, ws)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[0] = True
    bad[min(2, M - 1)] = M > 2 or M == 1
    assert torch.equal(torch.isnan(c).all(dim=1), bad)
    assert torch.equal(torch.isnan(c).any(dim=1), bad)
    assert (binding.linear_mx(x, wq, ws, epilogue="relu")[bad] == 0).all()


def test_linear_strides_and_kept_memory():
    for M in (2, 20, 150):
        big = rand((M + 3, 900), 5, F16)
        x = big[1:M + 1, 7:640]
        wq, ws = weights(77, 633, 6)
        out = torch.full((M + 2, 100), -3.0, dtype=F16, device="cuda")
        binding.linear_mx(x, wq, ws, C=out[1:M + 1, 11:88])
        want, err = linear_want(x, wq, ws, 0, None, False)
        ref.assert_close(out[1:M + 1, 11:88], want, err, F16)
        out[1:M + 1, 11:88] = -3.0
        assert (out == -3.0).all()


def test_linear_of_nothing():
    wq, ws = weights(8, 100, 7)
    x = torch.zeros((0, 100), device="cuda", dtype=BF16)
    assert binding.linear_mx(x, wq, ws).shape == (0, 8)
    x = torch.zeros((3, 100), device="cuda", dtype=BF16)
    assert binding.linear_mx(x, wq[:0], ws[:0]).shape == (3, 0)
    empty = torch.zeros((3, 0), device="cuda", dtype=BF16)
    b = torch.arange(-4.0, 4.0, device="cuda")
    none = torch.zeros((8, 0), dtype=torch.uint8, device="cuda")
    c = binding.linear_mx(empty, none, none, bias=b, epilogue="relu")
    assert torch.equal(c.float(), b.clamp(min=0).expand(3, 8))
    assert (binding.linear_mx(empty, none, none) == 0).all()


def test_linear_reuses_a_workspace_and_other_streams():
    M, N, K = 40, 128, 512
    need = binding.linear_mx_workspace_size(M, N, K, binding.TG_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    wq, wsc = weights(N, K, 8)
    xs = [rand((M, K), 40 + i, BF16) for i in range(3)]
    want = [binding.linear_mx(x, wq, wsc) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, w in zip(xs, want):
        c = binding.linear_mx(x, wq, wsc, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(c, w)


def test_two_graphs_with_a_workspace_each():
    # replayed in turn and at once, on two streams
    wq, ws = weights(256, 512, 9)
    graphs = []
    for i in range(2):
        x, c = rand((60, 512), 90 + i, BF16), torch.empty((60, 256), dtype=BF16, device="cuda")
        need = binding.linear_mx_workspace_size(60, 256, 512, binding.TG_BF16)
        w = torch.empty((need,), dtype=torch.uint8, device="cuda")
        binding.linear_mx(x, wq, ws, C=c, workspace=w)
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            binding.linear_mx(x, wq, ws, C=c, workspace=w)
        graphs.append((g, st, x, c))
    for _ in range(3):
        for g, st, x, c in graphs:
            c.zero_()
        torch.cuda.synchronize()
        for g, st, x, c in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for g, st, x, c in graphs:
            assert torch.equal(c, binding.linear_mx(x, wq, ws))


@pytest.mark.parametrize("M", [1, 40])
def test_linear_captured(M):
    wq, ws = weights(256, 1024, 9)
    x = rand((M, 1024), 10, BF16)
    c = torch.empty((M, 256), dtype=BF16, device="cuda")
    binding.linear_mx(x, wq, ws, C=c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.linear_mx(x, wq, ws, C=c)
    for i in range(4):
        x.copy_(rand((M, 1024), 50 + i, BF16))
        g.replay()
        torch.cuda.synchronize()
        got = c.clone()
        assert torch.equal(got, binding.linear_mx(x, wq, ws))


# --------------------------------------------------------------------------
# Gradients.
# --------------------------------------------------------------------------
def backward_want(dY, X, W, fmt):
    out = {}
    if W is not None:
        out["dx"] = ref.product(*ref.quantise(dY, fmt), fmt, *ref.quantise(W.t(), 0))
    if X is not None:
        out["dw"] = ref.product(*ref.quantise(dY.t(), fmt), fmt, *ref.quantise(X.t(), 0))
    return out


def check_backward(M, N, K, dtype, wtype, fmt, seed=0):
    say("linear_mx_backward %d x %d x %d %s %s fmt %d" % (M, N, K, dtype, wtype, fmt))
    dY = rand((M, N), 60 + seed, dtype, spread=False)
    X = rand((M, K), 61 + seed, dtype, spread=False)
    W = rand((N, K), 62 + seed, wtype, spread=False) / max(K, 1) ** 0.5
    g = binding.linear_mx_backward(dY, X=X, W=W, fmt=fmt, dbias=True)
    want = backward_want(dY, X, W, fmt)
    ref.assert_close(g.dx, *want["dx"], dtype, "dx")
    ref.assert_close(g.dw, *want["dw"], wtype, "dw")
    d = dY.double()
    ref.assert_close(g.dbias, d.sum(0), (M + 8) * ref.U32 * d.abs().sum(0), F32, "dbias")
    return dY, X, W, g


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 130), (7, 33, 65), (32, 128, 96),
                                   (129, 130, 131), (300, 200, 100), (1000, 1001, 1003),
                                   (512, 1024, 640)])
@pytest.mark.parametrize("dtype,wtype,fmt", [(BF16, BF16, 0), (BF16, F32, 1), (F16, F16, 1),
                                             (F32, F32, 0)])
def test_backward(M, N, K, dtype, wtype, fmt):
    check_backward(M, N, K, dtype, wtype, fmt)


def test_backward_parts_and_strides():
    dY, X, W, g = check_backward(200, 150, 260, BF16, BF16, 0)
    a = binding.linear_mx_backward(dY, W=W)
    assert torch.equal(a.dx, g.dx) and a.dw is None and a.dbias is None
    a = binding.linear_mx_backward(dY, X=X)
    assert torch.equal(a.dw, g.dw) and a.dx is None
    a = binding.linear_mx_backward(dY, dbias=True)
    assert torch.equal(a.dbias, g.dbias) and a.dw is None and a.dx is None
    a = binding.linear_mx_backward(dY, W=W, dbias=True)
    assert torch.equal(a.dx, g.dx) and torch.equal(a.dbias, g.dbias)
    wide = torch.zeros((200, 999), dtype=BF16, device="cuda")
    wide[:, 5:155], wide[:, 301:561] = dY, X
    a = binding.linear_mx_backward(wide[:, 5:155], X=wide[:, 301:561], W=W, dbias=True)
    for n in ("dx", "dw", "dbias"):
        assert torch.equal(getattr(a, n), getattr(g, n)), n
    for _ in range(2):  # a fixed order: the same bits
        b = binding.linear_mx_backward(dY, X=X, W=W, dbias=True)
        for n in ("dx", "dw", "dbias"):
            assert torch.equal(getattr(b, n), getattr(g, n)), n


def test_backward_of_nothing():
    z = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
    g = binding.linear_mx_backward(z(0, 8), X=z(0, 40), W=z(8, 40), dbias=True)
    assert g.dx.shape == (0, 40) and (g.dw == 0).all() and (g.dbias == 0).all()
    g = binding.linear_mx_backward(z(5, 0), X=z(5, 40), W=z(0, 40), dbias=True)
    assert (g.dx == 0).all() and g.dx.shape == (5, 40) and g.dw.shape == (0, 40)
    g = binding.linear_mx_backward(z(5, 8) + 1, X=z(5, 0), W=z(8, 0), dbias=True)
    assert g.dx.shape == (5, 0) and (g.dbias == 5).all()


def test_backward_differences():
    # where every operand is held exactly along both axes the products are those
    # of the values: gradients of sum(dY * (X W^T + b)) by differences of values
    # that stay exact (all magnitudes 0, 1, 2 or 4 of one octave's power of two)
    g = torch.Generator(device="cuda").manual_seed(11)
    pick = lambda *s: torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0, 4.0], device="cuda")[
        torch.randint(0, 6, s, generator=g, device="cuda")]
    M, N, K = 64, 96, 160
    dY, X, W = pick(M, N), pick(M, K), pick(N, K)
    for t in (dY, X, W):
        t[::32, :] = 4.0
        t[:, ::32] = 4.0
    out = binding.linear_mx_backward(dY, X=X, W=W, dbias=True)
    loss = lambda x, w: float((dY.double() * (x.double() @ w.double().t())).sum())
    f0 = loss(X, W)
    for i, j in ((0, 0), (3, 77), (63, 159), (31, 32)):
        d = torch.zeros_like(X)
        d[i, j] = 1.0
        assert loss(X + d, W) - f0 == float(out.dx[i, j])
    for i, j in ((0, 0), (95, 159), (40, 33)):
        d = torch.zeros_like(W)
        d[i, j] = 1.0
        assert loss(X, W + d) - f0 == float(out.dw[i, j])
    assert torch.equal(out.dbias.double(), dY.double().sum(0))


def test_backward_captured():
    M, N, K = 96, 160, 224
    dY, X, W = rand((M, N), 70, BF16), rand((M, K), 71, BF16), rand((N, K), 72, BF16)
    binding.linear_mx_backward(dY, X=X, W=W, dbias=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = binding.linear_mx_backward(dY, X=X, W=W, dbias=True)
    for i in range(4):
        dY.copy_(rand((M, N), 80 + i, BF16))
        g.replay()
        torch.cuda.synchronize()
        want = binding.linear_mx_backward(dY, X=X, W=W, dbias=True)
        for n in ("dx", "dw", "dbias"):
            assert torch.equal(getattr(out, n), getattr(want, n)), n


def test_no_k_and_more_results_than_one_pass():
    M, N = 70000, 4096
    say("linear %d x %d x 0" % (M, N))
    bias = torch.arange(N, dtype=torch.float32, device="cuda") - 2000
    none = torch.zeros((N, 0), dtype=torch.uint8, device="cuda")
    C = binding.linear_mx(torch.empty((M, 0), dtype=BF16, device="cuda"), none, none, bias,
                          epilogue="relu")
    assert (C == bias.clamp(min=0).to(BF16)).all()
