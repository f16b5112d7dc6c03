"""Host-side checks of the 8-bit integer and block-norm entry points (no GPU
needed, no kernel launched): every invalid-argument path returns its status
before any HIP call, workspace sizes, and the binding's refusals.  Also pins
the tests' 64-bit norm gradients by differences."""

import ctypes

import numpy as np
import pytest

import i8_norm_reference as ref
from tiled_dense_gemm_07_amd import binding

OK, NULLP, SHAPE, DTYPE, EPI, ALIAS, NOCFG, HIP, BADL, WSP, SCRATCH = range(11)
# fake, well-separated device addresses: validation never dereferences them
P = [0x10000000 * (i + 1) for i in range(16)]
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_quant_argument_errors(lib):
    q = lib.tg_quant_i8
    assert q(4, 8, 3, P[0], 8, P[1], 8, P[2], None) == DTYPE
    assert q(-1, 8, 2, P[0], 8, P[1], 8, P[2], None) == SHAPE
    assert q(4, -8, 2, P[0], 8, P[1], 8, P[2], None) == SHAPE
    assert q(4, 8, 2, P[0], 7, P[1], 8, P[2], None) == SHAPE
    assert q(4, 8, 2, P[0], 8, P[1], 7, P[2], None) == SHAPE
    assert q(1 << 31, 8, 2, P[0], 8, P[1], 8, P[2], None) == SHAPE
    for bad in ((None, P[1], P[2]), (P[0], None, P[2]), (P[0], P[1], None)):
        assert q(4, 8, 2, bad[0], 8, bad[1], 8, bad[2], None) == NULLP
    assert q(4, 8, 2, P[0], 8, P[0] + 63, 8, P[2], None) == ALIAS
    assert q(4, 8, 2, P[0], 8, P[1], 8, P[0], None) == ALIAS
    assert q(4, 8, 2, P[0], 8, P[1], 8, P[1], None) == ALIAS
    assert q(0, 8, 2, None, 8, None, 8, None, None) == OK


def gemm(lib, M=4, N=4, K=32, A=P[0], lda=None, sa=P[1], W=P[2], ldw=None, sw=P[3], bias=None,
         dt=BF16, C=P[4], ldc=None, epi=0):
    return lib.tg_gemm_i8(M, N, K, A, K if lda is None else lda, sa, W, K if ldw is None else ldw,
                          sw, bias, dt, C, N if ldc is None else ldc, epi, None)


def test_gemm_argument_errors(lib):
    assert gemm(lib, dt=3) == DTYPE
    assert gemm(lib, epi=2) == EPI
    for k in ("M", "N", "K"):
        assert gemm(lib, **{k: -1}) == SHAPE
        assert gemm(lib, **{k: 1 << 31}) == SHAPE
    assert gemm(lib, K=131072) == SHAPE  # 128 * 128 * K would leave 32 bits
    assert gemm(lib, lda=1 << 23) == SHAPE  # 256 rows of a tile within 31 bits
    assert gemm(lib, ldw=1 << 23) == SHAPE
    assert gemm(lib, lda=31) == SHAPE
    assert gemm(lib, ldw=31) == SHAPE
    assert gemm(lib, ldc=3) == SHAPE
    for k in ("A", "sa", "W", "sw", "C"):
        assert gemm(lib, **{k: None}) == NULLP
    assert gemm(lib, C=P[0] + 8) == ALIAS
    assert gemm(lib, C=P[2] + 8) == ALIAS
    assert gemm(lib, C=P[1]) == ALIAS
    assert gemm(lib, C=P[3]) == ALIAS
    assert gemm(lib, C=P[5], bias=P[5]) == ALIAS
    assert gemm(lib, M=0, A=None, sa=None, C=None) == OK
    assert gemm(lib, N=0, W=None, sw=None, C=None) == OK
    assert gemm(lib, K=0, A=None, W=None, C=None) == NULLP


def test_query_names_the_kernel():
    q = lambda *a: binding.query_config(binding.TG_OP_I8, *a)
    assert q(1, 8192, 8192).startswith("i8_gemv_16 grid=512x1 ")
    assert q(4096, 4096, 4096).startswith("i8_256x256x128")
    assert q(1000, 1001, 1003).startswith("i8_any_64x64")
    assert q(0, 64, 64).startswith("i8_")
    for bad, status in (((-1, 4, 4), SHAPE), ((4, 4, 131072), SHAPE), ((4, 4, 4, 9), DTYPE)):
        with pytest.raises(binding.TileGemmError) as e:
            q(*bad)
        assert e.value.status == status


def linear(lib, M=4, N=4, K=32, dt=BF16, X=P[0], ldx=None, W=P[1], ldw=None, sw=P[2], bias=None,
           C=P[3], ldc=None, epi=0, ws=P[4], nb=1 << 20):
    return lib.tg_linear_i8(M, N, K, dt, X, K if ldx is None else ldx, W, K if ldw is None else ldw,
                            sw, bias, C, N if ldc is None else ldc, epi, ws, nb, None)


def test_linear_argument_errors(lib):
    assert linear(lib, dt=7) == DTYPE
    assert linear(lib, epi=-1) == EPI
    assert linear(lib, K=131072) == SHAPE
    assert linear(lib, ldx=8) == SHAPE
    assert linear(lib, ldw=8) == SHAPE
    assert linear(lib, ldc=3) == SHAPE
    for k in ("X", "W", "sw", "C"):
        assert linear(lib, **{k: None}) == NULLP
    assert linear(lib, C=P[0]) == ALIAS
    assert linear(lib, C=P[1]) == ALIAS
    assert linear(lib, C=P[2]) == ALIAS
    assert linear(lib, C=P[5], bias=P[5]) == ALIAS
    M = 1000  # enough rows that the levels go through the workspace
    need = binding.linear_i8_workspace_size(M, 64, 100, BF16)
    assert need >= M * 112 + 4 * M
    assert linear(lib, M=M, K=100, ws=None) == WSP
    assert linear(lib, M=M, K=100, nb=need - 1) == WSP
    assert linear(lib, M=M, K=100, ws=P[4] + 8) == WSP
    for over in (P[0], P[1], P[2], P[3]):
        assert linear(lib, M=M, K=100, ws=over) == ALIAS
    assert linear(lib, M=0, X=None, C=None, ws=None, nb=0) == OK
    assert binding.linear_i8_workspace_size(0, 64, 100, BF16) == 0
    n = ctypes.c_size_t()
    f = lib.tg_linear_i8_workspace_size
    assert f(4, 4, 4, BF16, None) == NULLP
    assert f(4, 4, 4, 3, ctypes.byref(n)) == DTYPE
    assert f(-4, 4, 4, BF16, ctypes.byref(n)) == SHAPE


def norm_args(**kw):
    a = binding.BlockNormArgs()
    d = dict(T=4, D=16, xtype=BF16, btype=BF16, x=P[0], ldx=16, y=P[1], ldy=16, gate=P[2],
             gate_rows=4, w_post=P[3], w_pre=P[4], alpha=1.0, eps=1e-6, post_norm=1, x_out=P[5],
             ldx_out=16, h=P[6], ldh=16, hq=P[7], ldhq=16, hs=P[8], r_post=P[9], r_pre=P[10])
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return a


def test_norm_argument_errors(lib):
    def f(**kw):
        return lib.tg_block_norm(ctypes.byref(norm_args(**kw)), None)

    assert lib.tg_block_norm(None, None) == NULLP
    assert f(xtype=3) == DTYPE
    assert f(btype=-1) == DTYPE
    assert f(xtype=BF16, btype=F16) == DTYPE
    assert f(xtype=BF16, btype=F32) == DTYPE
    assert f(T=-1) == SHAPE
    assert f(T=(1 << 30) + 1) == SHAPE
    assert f(D=-1) == SHAPE
    assert f(D=32769) == SHAPE
    assert f(gate_rows=0) == SHAPE
    for k in ("ldx", "ldy", "ldx_out", "ldh", "ldhq"):
        assert f(**{k: 15}) == SHAPE
    assert f(x=None) == NULLP
    assert f(x_out=None) == NULLP  # y without x_out
    assert f(hs=None) == NULLP
    assert f(hq=None) == NULLP  # scales without levels
    alone = dict(y=None, gate=None, w_post=None, r_post=None, x_out=None)
    assert f(**alone, h=None, hq=None, hs=None, r_pre=None, w_pre=None) == NULLP
    for k in ("gate", "w_post", "r_post", "x_out"):
        assert f(**{**alone, k: P[11]}) == BADL
    assert f(post_norm=0, r_post=None) == BADL  # w_post without the norm
    assert f(post_norm=0, w_post=None) == BADL  # r_post without the norm
    assert f(h=None, hq=None, hs=None, r_pre=None) == BADL  # w_pre without h
    assert f(h=None, hq=None, hs=None, w_pre=None) == BADL
    # outputs over inputs and over each other; x_out over x only if it is x
    assert f(x_out=P[0] + 2) == ALIAS
    assert f(x_out=P[0], ldx_out=32) == ALIAS
    assert f(x_out=P[1]) == ALIAS
    assert f(h=P[1]) == ALIAS
    assert f(h=P[5]) == ALIAS
    assert f(hq=P[6]) == ALIAS
    assert f(hs=P[4]) == ALIAS
    assert f(r_pre=P[9] + 12) == ALIAS
    assert f(T=0, x=None) == OK
    assert f(D=0, x=None) == OK


def grad_args(**kw):
    a = binding.BlockNormGradArgs()
    d = dict(T=4, D=16, xtype=BF16, btype=BF16, x_new=P[0], ldx_new=16, y=P[1], ldy=16, gate=P[2],
             gate_rows=4, w_post=P[3], w_pre=P[4], alpha=1.0, post_norm=1, r_post=P[5],
             r_pre=P[6], dx_new=P[7], lddx_new=16, dh=P[8], lddh=16, dx=P[9], lddx=16, dy=P[10],
             lddy=16, dgate=P[11], dw_post=P[12], dw_pre=P[13])
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return a


def test_norm_backward_argument_errors(lib):
    def f(ws=P[14], nb=1 << 24, **kw):
        return lib.tg_block_norm_backward(ctypes.byref(grad_args(**kw)), ws, nb, None)

    assert lib.tg_block_norm_backward(None, P[14], 0, None) == NULLP
    assert f(xtype=5) == DTYPE
    assert f(xtype=F16, btype=BF16) == DTYPE
    assert f(T=-1) == SHAPE
    assert f(D=32769) == SHAPE
    assert f(gate_rows=-2) == SHAPE
    for k in ("ldx_new", "ldy", "lddx_new", "lddh", "lddx", "lddy"):
        assert f(**{k: 15}) == SHAPE
    assert f(dx_new=None, dh=None, dw_pre=None) == NULLP
    assert f(x_new=None) == NULLP
    assert f(r_pre=None) == NULLP
    assert f(r_post=None) == NULLP
    assert f(dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None) == NULLP
    none = dict(y=None, gate=None, w_post=None, dy=None, dgate=None, dw_post=None)
    for k in ("gate", "w_post", "dy", "dgate", "dw_post"):
        assert f(**{**none, k: P[15]}) == BADL
    assert f(post_norm=0) == BADL
    assert f(gate=None) == BADL
    assert f(w_post=None) == BADL
    assert f(w_pre=None) == BADL
    assert f(dh=None) == BADL
    assert f(ws=None) == WSP
    assert f(ws=P[14] + 4) == WSP
    assert f(nb=16) == WSP
    for k, at in (("dx", 0), ("dy", 1), ("dgate", 2), ("dw_post", 5), ("dw_pre", 8), ("dx", 10),
                  ("dy", 14), ("dgate", 12)):
        assert f(**{k: P[at]}) == ALIAS, k
    assert f(T=0) == OK
    n = ctypes.c_size_t()
    size = lib.tg_block_norm_backward_workspace_size
    assert size(None, ctypes.byref(n)) == NULLP
    assert size(ctypes.byref(grad_args()), None) == NULLP
    assert size(ctypes.byref(grad_args(T=0)), ctypes.byref(n)) == OK and n.value == 0


def test_interleaved_slices_do_not_alias(lib):
    """Column slices of one buffer share its byte range but no element: the
    argument check goes on to the next fault instead of reporting an overlap."""
    a = dict(T=8, D=16, ldx=64, ldy=64, ldx_out=64, x=P[0], y=P[0] + 32, x_out=P[0] + 64, h=P[6],
             hq=None, hs=P[8])
    f = lib.tg_block_norm
    assert f(ctypes.byref(norm_args(**a)), None) == NULLP  # hs without hq
    a.update(hs=None, hq=None, x_out=P[0] + 48)
    assert f(ctypes.byref(norm_args(**a)), None) == ALIAS


def test_forced_launch_failure(lib, monkeypatch):
    """A failed launch is reported as TG_ERR_HIP by every new entry point."""
    monkeypatch.setenv("TG_FAULT", "launch")
    assert lib.tg_quant_i8(4, 8, 2, P[0], 8, P[1], 8, P[2], None) == HIP
    assert gemm(lib) == HIP
    assert linear(lib) == HIP
    assert lib.tg_block_norm(ctypes.byref(norm_args()), None) == HIP
    assert lib.tg_block_norm_backward(ctypes.byref(grad_args()), P[14], 1 << 24, None) == HIP


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16)
    q = torch.zeros(4, 16, dtype=torch.int8)
    s = torch.zeros(4)
    for call in (lambda: binding.quant_i8(x), lambda: binding.gemm_i8(q, s, q, s),
                 lambda: binding.linear_i8(x, q, s), lambda: binding.block_norm(x),
                 lambda: binding.block_norm_backward(x, x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="out must be"):
        binding.block_norm(x, out="f8")


def test_levels_reference():
    """Ties to even, the exact half, a zero row, infinities and NaN."""
    v = np.array([[127.0, 63.5, 62.5, -0.5], [254.0, 127.0, 1.0, -3.0], [0, 0, 0, 0],
                  [1.0, np.inf, 0, 0], [np.nan, 1.0, 2.0, 3.0]])
    q, s = ref.levels(v)
    assert q[0].tolist() == [127, 64, 62, 0]
    assert q[1].tolist() == [127, 64, 0, -2]
    assert not q[2:].any()
    assert s[0] == 1.0 and s[1] == 2.0 and s[2] == 2.0 ** -126
    assert np.isnan(s[3]) and np.isnan(s[4])


@pytest.mark.parametrize("post,gate_rows", [(True, 3), (True, 1), (False, 7), (True, 0)])
def test_reference_gradients_by_differences(post, gate_rows):
    """The formulas the GPU gradients are compared with, against central
    differences of the forward formulas, all in 64 bits."""
    r = np.random.Generator(np.random.PCG64(5))
    T, D, eps, alpha = 7, 10, 1e-6, 0.7
    v = {"x": r.normal(size=(T, D)), "y": r.normal(size=(T, D)), "w_pre": r.normal(size=D)}
    if gate_rows:
        v["gate"] = r.normal(size=(-(-T // gate_rows), D))
    if post:
        v["w_post"] = r.normal(size=D)
    a, b = r.normal(size=(T, D)), r.normal(size=(T, D))

    def loss(v):
        f = ref.forward(v["x"], v["y"], v.get("gate"), gate_rows, v.get("w_post"), v["w_pre"],
                        alpha, eps, post)
        return (a * f["x_out"]).sum() + (b * f["h"]).sum()

    f = ref.forward(v["x"], v["y"], v.get("gate"), gate_rows, v.get("w_post"), v["w_pre"], alpha,
                    eps, post)
    g = ref.backward(f["x_out"], a, b, v["y"], v.get("gate"), gate_rows, v.get("w_post"),
                     v["w_pre"], f["r_post"], f["r_pre"], alpha, post)
    for k, name in (("x", "dx"), ("y", "dy"), ("w_pre", "dw_pre"), ("gate", "dgate"),
                    ("w_post", "dw_post")):
        if k not in v:
            continue
        step = r.normal(size=v[k].shape)
        e = 1e-5
        d = (loss({**v, k: v[k] + e * step}) - loss({**v, k: v[k] - e * step})) / (2 * e)
        # the difference's own error: e^2 times third derivatives, and 2^-52 / e
        assert abs(d - (g[name] * step).sum()) <= 1e-6 * max(1.0, abs(d)), name
