"""GPU tests of the head norms with rotation and of their gradients against the
64-bit forms, and of the projection into attention as it is used: block norm,
linear layer in microscaled blocks, head norms, and the way back."""

import pytest
import torch

import mx_heads_reference as ref
from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def rand(shape, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def case(T, Hq, Hk, D, R, dtype, seed=0, P=None):
    q, k = 2 * rand((T, Hq, D), seed, dtype), 0.5 * rand((T, Hk, D), seed + 1, dtype)
    wq, wk = ((1 + 0.3 * rand((D,), seed + 2 + i, F32)).to(dtype) for i in range(2))
    P = max(T, 50) if P is None else P
    cos, sin = (t.cuda() for t in ref.tables(P, R // 2))
    g = torch.Generator(device="cuda").manual_seed(seed)
    pos = torch.randint(0, P, (T,), generator=g, device="cuda")
    return q, k, wq, wk, cos, sin, pos


SHAPES = [(4, 3, 1, 3, 2), (7, 2, 1, 4, 2), (7, 2, 1, 5, 4), (3, 3, 2, 30, 6), (5, 2, 2, 129, 10), (3, 2, 1, 515, 514),
          (3, 2, 1, 1023, 6), (1, 1, 0, 1, 0), (1, 1, 1, 2, 2), (3, 2, 1, 7, 4), (5, 3, 2, 16, 16), (1, 32, 8, 128, 128),
          (2, 7, 3, 64, 64), (33, 5, 2, 80, 80), (20, 4, 4, 96, 32), (9, 9, 1, 99, 66),
          (17, 6, 2, 128, 64), (4, 3, 3, 127, 126), (6, 2, 2, 192, 64), (3, 2, 1, 256, 256),
          (2, 2, 2, 300, 100), (2, 3, 1, 512, 512), (2, 2, 1, 1000, 500), (2, 1, 1, 1024, 1024),
          (2, 1, 2, 1021, 1020), (700, 2, 1, 32, 32)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
def test_forward_and_backward(T, Hq, Hk, D, R, dtype, interleaved):
    say("heads %s %s %s" % ((T, Hq, Hk, D, R), dtype, interleaved))
    q, k, wq, wk, cos, sin, pos = case(T, Hq, Hk, D, R, dtype)
    kw = dict(w_q=wq, w_k=wk, cos=cos, sin=sin, positions=pos, eps=EPS, interleaved=interleaved)
    out = binding.head_norm_rope(q, k, **kw)
    c, s = cos[pos], sin[pos]
    for got, x, w in ((out.q, q, wq), (out.k, k, wk)):
        want, err = ref.heads_forward(x, w, c, s, R, EPS, interleaved)
        ref.assert_close(got, want, err, dtype, "forward")
    dq, dk = rand((T, Hq, D), 8, dtype), rand((T, Hk, D), 9, dtype)
    g = binding.head_norm_rope_backward(dq, dk, q, k, **kw)
    for d, x, w, gx, gw in ((dq, q, wq, g.dq, g.dw_q), (dk, k, wk, g.dk, g.dw_k)):
        dx, dw, ex, ew = ref.heads_backward(d, x, w, c, s, R, EPS, interleaved)
        ref.assert_close(gx, dx, ex, dtype, "dx")
        ref.assert_close(gw, dw, ew, F32, "dw")


def test_many_tokens():
    T, Hq, Hk, D = 5000, 8, 2, 128
    q, k, wq, wk, cos, sin, pos = case(T, Hq, Hk, D, D, BF16)
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    want, err = ref.heads_forward(q, wq, cos[pos], sin[pos], D, EPS, False)
    ref.assert_close(out.q, want, err, BF16)
    dq, dk = rand(q.shape, 8, BF16), rand(k.shape, 9, BF16)
    g = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for d, x, w, gx, gw in ((dq, q, wq, g.dq, g.dw_q), (dk, k, wk, g.dk, g.dw_k)):
        dx, dw, ex, ew = ref.heads_backward(d, x, w, cos[pos], sin[pos], D, EPS, False)
        ref.assert_close(gx, dx, ex, BF16, "dx")
        ref.assert_close(gw, dw, ew, F32, "dw")
    again = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for a, b in zip(g, again):  # a fixed order: the same bits
        assert torch.equal(a, b)


def test_without_weights_keys_tables_or_positions():
    q, k, wq, wk, cos, sin, pos = case(40, 3, 2, 64, 64, BF16)
    run = torch.arange(40, device="cuda")
    a = binding.head_norm_rope(q, k, wq, wk, cos, sin, None, EPS)
    b = binding.head_norm_rope(q, k, wq, wk, cos, sin, run, EPS)
    assert torch.equal(a.q, b.q) and torch.equal(a.k, b.k)
    c = binding.head_norm_rope(q, None, wq, None, cos, sin, None, EPS)
    assert torch.equal(c.q, a.q) and c.k is None
    one = torch.ones_like(wq)
    c = binding.head_norm_rope(q, k, cos=cos, sin=sin, eps=EPS)
    b = binding.head_norm_rope(q, k, one, one, cos, sin, eps=EPS)
    assert torch.equal(c.q, b.q) and torch.equal(c.k, b.k)
    c = binding.head_norm_rope(q, k, wq, wk, eps=EPS)  # norms only
    want, err = ref.heads_forward(q, wq, cos[:40, :0], sin[:40, :0], 0, EPS, False)
    ref.assert_close(c.q, want, err, BF16)
    dq, dk = rand(q.shape, 8, BF16), rand(k.shape, 9, BF16)
    g = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, None, EPS)
    h = binding.head_norm_rope_backward(dq, None, q, None, wq, None, cos, sin, None, EPS)
    assert torch.equal(g.dq, h.dq) and torch.equal(g.dw_q, h.dw_q) and h.dk is None
    h = binding.head_norm_rope_backward(dq, dk, q, k, None, wk, cos, sin, None, EPS)
    assert torch.equal(g.dk, h.dk) and torch.equal(g.dw_k, h.dw_k) and h.dw_q is None


def test_slices_in_place_and_other_orders():
    T, Hq, Hk, D = 37, 4, 2, 96
    qkv = rand((T, (Hq + 2 * Hk) * D + 8), 3, BF16)
    kept = qkv.clone()
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    _, _, wq, wk, cos, sin, pos = case(T, Hq, Hk, D, 48, BF16)
    want = binding.head_norm_rope(q.contiguous(), k.contiguous(), wq, wk, cos, sin, pos, EPS)
    got = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    assert torch.equal(got.q, want.q) and torch.equal(got.k, want.k)
    # a cache that holds a head's tokens together
    qc = torch.full((Hq, T + 5, D), 3.0, dtype=BF16, device="cuda")
    binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS, q_out=qc[:, 2:T + 2].transpose(0, 1))
    assert torch.equal(qc[:, 2:T + 2].transpose(0, 1), want.q)
    assert (qc[:, :2] == 3).all() and (qc[:, T + 2:] == 3).all()
    # heads at odd places
    odd = torch.zeros((T, Hq, D + 3), dtype=BF16, device="cuda")
    odd[:, :, 1:D + 1] = q
    got = binding.head_norm_rope(odd[:, :, 1:D + 1], None, wq, None, cos, sin, pos, EPS)
    assert torch.equal(got.q, want.q)
    # gradients of inputs and gradients that are slices, and of a gradient shared by all heads
    dq = rand((T, 1, D), 8, BF16).expand(T, Hq, D)
    dk = rand((T, Hk, D), 9, BF16)
    a = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    b = binding.head_norm_rope_backward(dq.contiguous(), dk, q.contiguous(), k.contiguous(), wq, wk,
                                        cos, sin, pos, EPS)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    # in place; what stands behind the heads stays
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS, q_out=q, k_out=k)
    assert out.q.data_ptr() == qkv.data_ptr()
    assert torch.equal(q, want.q) and torch.equal(k, want.k)
    assert torch.equal(qkv[:, (Hq + Hk) * D:], kept[:, (Hq + Hk) * D:])


@pytest.mark.parametrize("D,R,interleaved", [(64, 32, False), (64, 32, True), (33, 20, False)])
def test_positions_outside_the_tables_give_nan(D, R, interleaved):
    q, k, wq, wk, cos, sin, pos = case(6, 2, 1, D, R, F32)
    pos = pos.clone()
    pos[1], pos[2], pos[4] = -1, cos.shape[0], 2 ** 40
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS, interleaved)
    bad = torch.tensor([False, True, True, False, True, False], device="cuda")
    for t in out:
        assert torch.isnan(t[bad][:, :, :R]).all() and not torch.isnan(t[~bad]).any()
        assert not torch.isnan(t[bad][:, :, R:]).any()


def test_far_positions_and_extreme_values():
    # the last row of a long table; rows of zeros; the largest values
    q, k, wq, wk, cos, sin, _ = case(4, 2, 2, 64, 64, F16, P=100000)
    pos = torch.tensor([99999, 0, 65536, 99998], device="cuda")
    q = q.clone()
    q[1] = 0.0
    q[2] = 65504.0
    q[3] = 6e-8
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    want, err = ref.heads_forward(q, wq, cos[pos], sin[pos], 64, EPS, False)
    ref.assert_close(out.q, want, err, F16)
    q[0, 1, 3] = float("nan")
    q[2, 0, 0] = float("inf")
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    bad = torch.isnan(out.q).any(dim=2)
    assert torch.equal(bad.cpu(), torch.tensor([[False, True], [False, False], [True, False],
                                                [False, False]]))
    assert not torch.isnan(out.k).any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,P", [(1024, 2, 1), (300, 2, 3), (200, 6, 1), (64, 64, 1), (99, 66, 2),
                                   (70, 6, 2), (1024, 6, 1), (5, 2, 5)])
def test_ends_of_small_tables(D, R, P, interleaved):
    q, k, wq, wk, cos, sin, _ = case(5, 3, 1, D, R, F32, P=P)
    pos = torch.tensor([P - 1, 0, P - 1, 0, P // 2], device="cuda")
    # in the middle of a larger buffer of NaN: what is past a table's end has no part
    raw = torch.full((2, P * (R // 2) + 64), float("nan"), device="cuda")
    c, s = (raw[i, 32:32 + P * (R // 2)].view(P, R // 2) for i in range(2))
    c.copy_(cos)
    s.copy_(sin)
    out = binding.head_norm_rope(q, k, wq, wk, c, s, pos, EPS, interleaved)
    want, err = ref.heads_forward(q, wq, cos[pos], sin[pos], R, EPS, interleaved)
    ref.assert_close(out.q, want, err, F32)
    d = rand(q.shape, 4, F32)
    g = binding.head_norm_rope_backward(d, k, q, k, wq, wk, c, s, pos, EPS, interleaved)
    dx, dw, ex, ew = ref.heads_backward(d, q, wq, cos[pos], sin[pos], R, EPS, interleaved)
    ref.assert_close(g.dq, dx, ex, F32)
    ref.assert_close(g.dw_q, dw, ew, F32)


def test_offsets_past_32_bits():
    # more than 2^31 values; the last tokens are looked at
    T, H, D = 1100000, 8, 256
    say("heads of %d tokens" % T)
    q = torch.empty((T, H, D), dtype=BF16, device="cuda").normal_()
    _, k, wq, wk, cos, sin, _ = case(T, 1, 1, D, D, BF16, P=100)
    pos = torch.arange(T, device="cuda") % 100
    end = slice(T - 50, T)
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    want, err = ref.heads_forward(q[end], wq, cos[pos[end]], sin[pos[end]], D, EPS, False)
    ref.assert_close(out.q[end], want, err, BF16)
    g = binding.head_norm_rope_backward(out.q, out.k, q, k, wq, wk, cos, sin, pos, EPS)
    dx, _, ex, _ = ref.heads_backward(out.q[end], q[end], wq, cos[pos[end]], sin[pos[end]], D, EPS,
                                      False)
    ref.assert_close(g.dq[end], dx, ex, BF16)
    assert torch.isfinite(g.dw_q).all() and torch.isfinite(g.dw_k).all()


def test_more_tokens_than_waves():
    # a wave takes units of several tokens
    T, D = 2 ** 26 + 3, 4
    say("heads of %d tokens" % T)
    q = torch.empty((T, 1, D), dtype=BF16, device="cuda").normal_()
    w = rand((D,), 2, BF16)
    out = binding.head_norm_rope(q, w_q=w, eps=EPS)
    for part in (slice(0, 100), slice(2 ** 25 - 7, 2 ** 25 + 93), slice(T - 100, T), slice(5, T, 99991)):
        none = torch.zeros((q[part].shape[0], 0), device="cuda")
        want, err = ref.heads_forward(q[part], w, none, none, 0, EPS, False)
        ref.assert_close(out.q[part], want, err, BF16)


def test_heads_far_apart():
    # heads more than 32 bits of bytes from the first of their unit
    T, H, D, far = 3, 8, 64, 640 * 2 ** 20 // 2
    x = torch.empty(((H - 1) * far + T * D,), dtype=BF16, device="cuda")
    q = x.as_strided((T, H, D), (D, far, 1))
    _, k, wq, wk, cos, sin, pos = case(T, H, 2, D, D, BF16)
    q.copy_(rand((T, H, D), 3, BF16))
    a = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    b = binding.head_norm_rope(q.contiguous(), k, wq, wk, cos, sin, pos, EPS)
    want, err = ref.heads_forward(q, wq, cos[pos], sin[pos], D, EPS, False)
    for got in (a.q, b.q):
        ref.assert_close(got, want, err, BF16)
    d = rand((T, H, D), 4, BF16)
    g = binding.head_norm_rope_backward(d, k, q, k, wq, wk, cos, sin, pos, EPS)
    dx, dw, ex, ew = ref.heads_backward(d, q, wq, cos[pos], sin[pos], D, EPS, False)
    ref.assert_close(g.dq, dx, ex, BF16)
    ref.assert_close(g.dw_q, dw, ew, F32)


def test_nothing():
    q = torch.zeros((0, 4, 64), dtype=BF16, device="cuda")
    w = torch.ones((64,), dtype=BF16, device="cuda")
    cos, sin = (t.cuda() for t in ref.tables(8, 32))
    out = binding.head_norm_rope(q, q, w, w, cos, sin)
    assert out.q.shape == (0, 4, 64)
    g = binding.head_norm_rope_backward(q, q, q, q, w, w, cos, sin)
    assert (g.dw_q == 0).all() and (g.dw_k == 0).all()
    q = torch.ones((3, 2, 64), dtype=BF16, device="cuda")
    none = q[:, :0]
    out = binding.head_norm_rope(q, none, w, w, cos, sin)
    assert out.k.shape == (3, 0, 64)
    g = binding.head_norm_rope_backward(q, none, q, none, w, w, cos, sin)
    assert (g.dw_k == 0).all() and g.dk.shape == (3, 0, 64)


def test_streams_and_captured():
    q, k, wq, wk, cos, sin, pos = case(64, 4, 2, 128, 128, BF16)
    dq, dk = rand(q.shape, 8, BF16), rand(k.shape, 9, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS, stream=side)
    ga = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, stream=side)
    side.synchronize()
    b = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    gb = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for x, y in zip(tuple(a) + tuple(ga), tuple(b) + tuple(gb)):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
        ga = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for i in range(4):
        q.copy_(rand(q.shape, 20 + i, BF16))
        pos.copy_(pos.flip(0))
        g.replay()
        torch.cuda.synchronize()
        b = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
        gb = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
        for x, y in zip(tuple(a) + tuple(ga), tuple(b) + tuple(gb)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("T", [1, 50, 300])
def test_projection_into_attention(T):
    # block norm, projection in 4 bits, head norms; each stage against its 64-bit
    # form on what the stage before gave, and the gradients back through all of them
    say("projection %d" % T)
    width, Hq, Hk, D = 320, 4, 2, 64
    N = (Hq + 2 * Hk) * D
    x, y = rand((T, width), 1, BF16), rand((T, width), 2, BF16)
    w_pre = (1 + 0.1 * rand((width,), 3, F32)).to(BF16)
    W = (rand((N, width), 4, F32) / width ** 0.5).to(BF16)
    bias = rand((N,), 5, F32)
    _, _, wq, wk, cos, sin, pos = case(T, Hq, Hk, D, D, BF16, P=400)
    f = binding.block_norm(x, y=y, w_pre=w_pre, save=True)
    w4 = binding.quant_mx(W)
    qkv = binding.linear_mx(f.h, w4.q, w4.s, bias=bias)
    want, err = ref.product(*ref.quantise(f.h, 0), 0, *ref.quantise(W, 0), bias)
    ref.assert_close(qkv, want, err, BF16, "projection")
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    out = binding.head_norm_rope(q, k, wq, wk, cos, sin, pos, EPS)
    for got, v, w in ((out.q, q, wq), (out.k, k, wk)):
        want, err = ref.heads_forward(v, w, cos[pos], sin[pos], D, EPS, False)
        ref.assert_close(got, want, err, BF16, "heads")
    dq, dk, dv = rand(q.shape, 6, BF16), rand(k.shape, 7, BF16), rand(k.shape, 8, BF16)
    gh = binding.head_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for d, v, w, gx, gw in ((dq, q, wq, gh.dq, gh.dw_q), (dk, k, wk, gh.dk, gh.dw_k)):
        dx, dw, ex, ew = ref.heads_backward(d, v, w, cos[pos], sin[pos], D, EPS, False)
        ref.assert_close(gx, dx, ex, BF16, "dx")
        ref.assert_close(gw, dw, ew, F32, "dw")
    dqkv = torch.cat([gh.dq.flatten(1), gh.dk.flatten(1), dv.flatten(1)], dim=1)
    gl = binding.linear_mx_backward(dqkv, X=f.h, W=W, dbias=True)
    ref.assert_close(gl.dx, *ref.product(*ref.quantise(dqkv, 0), 0, *ref.quantise(W.t(), 0)), BF16)
    ref.assert_close(gl.dw, *ref.product(*ref.quantise(dqkv.t(), 0), 0,
                                         *ref.quantise(f.h.t(), 0)), BF16)
    gb = binding.block_norm_backward(f.x, None, gl.dx, y=y, w_pre=w_pre, r_post=f.r_post,
                                     r_pre=f.r_pre)
    assert gb.dx.shape == x.shape and torch.isfinite(gb.dx).all() and torch.isfinite(gb.dy).all()
