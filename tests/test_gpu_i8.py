"""8-bit integer quantisation, product and linear on the GPU, through the C
ABI, against the plain 64-bit forms: odd sizes, strides, addresses, empty and
single rows, every output type, special values, streams and graphs."""

from __future__ import annotations

import numpy as np
import pytest

import i8_norm_reference as ref
import oracle
from gpu_helpers import BF16, F16, F32, bits_to_f64, say, to_host_bits, torch_dtype
from tiled_dense_gemm_07_amd import binding

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DNAME = {F32: "f32", F16: "f16", BF16: "bf16"}
TYPES = pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=lambda d: DNAME[d])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


def values(t, dtype):
    return bits_to_f64(to_host_bits(t.contiguous(), dtype), dtype)


def strided(t, pad=0, shift=0):
    """t's values in a wider buffer: rows `pad` elements apart, the first
    `shift` elements in."""
    M, K = t.shape
    buf = torch.zeros(M * (K + pad) + shift + 1, dtype=t.dtype, device=DEV)
    out = buf[shift:shift + M * (K + pad)].view(M, K + pad)[:, :K]
    out.copy_(t)
    return out


def make_levels(r, M, K):
    """All 256 levels, the extremes more often."""
    q = r.integers(-128, 128, size=(M, K))
    q[r.random((M, K)) < 0.05] = -128
    q[r.random((M, K)) < 0.05] = 127
    return q.astype(np.int8)


def make_product(M, N, K, seed, bias=True):
    r = np.random.Generator(np.random.PCG64(seed))
    A, W = make_levels(r, M, K), make_levels(r, N, K)
    sa = np.exp(r.normal(size=M)).astype(np.float32) / np.float32(127.0)
    sw = np.exp(r.normal(size=N)).astype(np.float32) / np.float32(127.0 * max(K, 1) ** 0.5)
    b = r.normal(size=N).astype(np.float32) if bias else None
    return A, sa, W, sw, b


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_product(got, A, sa, W, sw, b, dtype, relu):
    c, t = ref.product(A, sa.astype(np.float64), W, sw.astype(np.float64),
                       None if b is None else b.astype(np.float64), relu)
    bad = ~(np.abs(got - c) <= ref.product_bound(c, t, dtype))
    assert not bad.any(), "%d of %d outside, first at %s" % (
        bad.sum(), bad.size, np.argwhere(bad)[:3].tolist())


SIZES = [
    # M, N, K: single rows and columns, every kernel's tile borders, odd tails
    (1, 1, 1), (1, 16, 16), (1, 17, 64), (3, 5, 7), (1, 1000, 2048), (2, 33, 4096), (7, 129, 255),
    (16, 64, 1024), (16, 31, 48), (17, 64, 512), (31, 200, 336), (33, 257, 1000), (48, 512, 4096),
    (64, 64, 128), (65, 100, 208), (100, 384, 640), (128, 256, 256), (130, 250, 384),
    (200, 1001, 1003), (255, 257, 512), (256, 256, 4096), (300, 520, 144), (513, 300, 2000),
    (1, 300, 70000), (40, 70, 33000),
]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_sizes(M, N, K):
    A, sa, W, sw, b = make_product(M, N, K, M * 31 + N * 7 + K)
    dA, dsa, dW, dsw, db = (dev(a) for a in (A, sa, W, sw, b))
    for dtype, relu, bias in ((BF16, True, False), (F32, False, True), (F16, False, False)):
        say("gemm_i8 %dx%dx%d %s relu=%d bias=%d" % (M, N, K, DNAME[dtype], relu, bias))
        C = torch.full((M, N), float("nan"), dtype=torch_dtype(dtype), device=DEV)
        binding.gemm_i8(dA, dsa, dW, dsw, bias=db if bias else None, C=C,
                        epilogue="relu" if relu else None)
        torch.cuda.synchronize()
        check_product(values(C, dtype), A, sa, W, sw, b if bias else None, dtype, relu)


@TYPES
@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (5, 70, 272), (64, 128, 512), (200, 300, 640),
                                   (256, 512, 1024)])
def test_product_bits(M, N, K, dtype):
    """Scales that are powers of two: one rounding from the exact sum, as the
    oracle rounds it."""
    r = np.random.Generator(np.random.PCG64(M + N + K))
    A = r.integers(-8, 9, size=(M, K)).astype(np.int8)  # sums below 2^24: exact in fp32
    W = r.integers(-128, 128, size=(N, K)).astype(np.int8)
    sa = (2.0 ** r.integers(-6, 2, size=M)).astype(np.float32)
    sw = (2.0 ** r.integers(-9, -3, size=N)).astype(np.float32)
    say("gemm_i8 bits %dx%dx%d %s" % (M, N, K, DNAME[dtype]))
    C = binding.gemm_i8(dev(A), dev(sa), dev(W), dev(sw), out_dtype=torch_dtype(dtype),
                        epilogue="relu")
    torch.cuda.synchronize()
    c, _ = ref.product(A, sa.astype(np.float64), W, sw.astype(np.float64), relu=True)
    assert np.array_equal(to_host_bits(C, dtype), oracle.encode(dtype, c))


@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (9, 100, 512), (40, 130, 256), (150, 260, 512)])
@pytest.mark.parametrize("pad,shift", [(16, 16), (16, 0), (1, 0), (0, 1), (5, 3), (8, 4)])
def test_product_strides_and_addresses(M, N, K, pad, shift):
    """Row strides and first addresses that are and are not multiples of 16."""
    A, sa, W, sw, b = make_product(M, N, K, 77)
    for where in ("A", "W", "C"):
        dA, dW = dev(A), dev(W)
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide = None
        if where == "A":
            dA = strided(dA, pad, shift)
        elif where == "W":
            dW = strided(dW, pad, shift)
        else:
            wide = torch.full((M * (N + pad) + shift,), 7.0, dtype=torch.bfloat16, device=DEV)
            C = wide[shift:].view(M, N + pad)[:, :N]
        say("gemm_i8 %dx%dx%d %s pad=%d shift=%d" % (M, N, K, where, pad, shift))
        binding.gemm_i8(dA, dev(sa), dW, dev(sw), bias=dev(b), C=C)
        torch.cuda.synchronize()
        check_product(values(C, BF16), A, sa, W, sw, b, BF16, False)
        if wide is not None:  # nothing else was written
            C.fill_(7.0)
            assert bool((wide == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(17, 4112, 512), (20, 4100, 1003), (33, 4097, 272),
                                   (32, 4200, 2050), (100, 1100, 700)])
@pytest.mark.parametrize("pad", [(0, 0), (16, 0), (0, 1), (1, 0), (2, 3), (4, 4)], ids=str)
def test_product_few_tokens(M, N, K, pad):
    """17 to 128 tokens, more workgroups than compute units: rows of A and of W
    at 16-byte, 4-byte and single-byte steps."""
    A, sa, W, sw, b = make_product(M, N, K, M + N + K)
    say("gemm_i8 %dx%dx%d pads %s" % (M, N, K, pad))
    dA, dW = strided(dev(A), pad[0], pad[0] // 2), strided(dev(W), pad[1], pad[1] // 2)
    C = torch.full((M, N), float("nan"), dtype=torch.float32, device=DEV)
    binding.gemm_i8(dA, dev(sa), dW, dev(sw), bias=dev(b), C=C)
    torch.cuda.synchronize()
    check_product(values(C, F32), A, sa, W, sw, b, F32, False)


@pytest.mark.parametrize("M,N,K,pad", [(1500, 2100, 385, 0), (1500, 2100, 384, 1),
                                       (2100, 2300, 515, 0), (2100, 2300, 512, 1),
                                       (2100, 2300, 130, 2), (600, 3000, 100, 0),
                                       (2000, 2050, 770, 0), (2000, 2050, 768, 3),
                                       (2050, 4100, 390, 0), (2050, 4100, 384, 1),
                                       (700, 900, 9, 0)])
def test_product_any_layout_tiles(M, N, K, pad):
    """Every tile of the kernels for any layout: rows with and without an end of
    less than a strip, rows shorter than a strip."""
    A, sa, W, sw, b = make_product(M, N, K, M + N + K)
    say("gemm_i8 %dx%dx%d pad %d" % (M, N, K, pad))
    C = binding.gemm_i8(strided(dev(A), pad, 1), dev(sa), strided(dev(W), pad, 1), dev(sw),
                        bias=dev(b), out_dtype=torch.bfloat16, epilogue="relu")
    torch.cuda.synchronize()
    check_product(values(C, BF16), A, sa, W, sw, b, BF16, True)


@pytest.mark.parametrize("M,N,K", [(4100, 4096, 1024), (4096, 4097, 1008), (4000, 4300, 640),
                                   (16385, 1024, 1024), (1000, 16640, 1024)])
def test_product_in_two_launches(M, N, K):
    """A few rows or columns more than whole rounds of the largest tiles."""
    assert " + " in binding.query_config(4, M, N, K)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    A = torch.randint(-128, 128, (M, K), dtype=torch.int8, device=DEV, generator=g)
    W = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sa = 2.0 ** torch.randint(-6, 2, (M,), device=DEV, generator=g).float()
    sw = 2.0 ** torch.randint(-9, -3, (N,), device=DEV, generator=g).float()
    b = torch.randint(-4, 5, (N,), device=DEV, generator=g).float()
    say("gemm_i8 %dx%dx%d" % (M, N, K))
    for bias in (None, b):
        C = binding.gemm_i8(A, sa, W, sw, bias=bias, out_dtype=torch.float32, epilogue="relu")
        torch.cuda.synchronize()
        # sums up to 2^24 and scales that are powers of two: exact in fp32 but
        # for the bias, one rounding of the sum
        want = (A.cpu().float() @ W.cpu().float().t()).double()
        want = want * sa.cpu().double()[:, None] * sw.cpu().double()
        if bias is not None:
            want = want + b.cpu().double()
        assert torch.equal(C.cpu(), want.clamp(min=0).float())


def test_product_largest_sums():
    """The largest magnitudes the sum can take: 128 * 128 * K near 2^31."""
    for M, K in ((3, 131071), (70, 131056)):
        N = 20
        A = np.full((M, K), -128, dtype=np.int8)
        W = np.full((N, K), -128, dtype=np.int8)
        W[1::2] = 127
        one_a, one_w = np.ones(M, np.float32), np.ones(N, np.float32)
        say("gemm_i8 largest sums M=%d K=%d" % (M, K))
        C = binding.gemm_i8(dev(A), dev(one_a), dev(W), dev(one_w), out_dtype=torch.float32)
        torch.cuda.synchronize()
        want = np.where(np.arange(N) % 2 == 0, 16384.0 * K, -16256.0 * K)
        assert np.array_equal(C.cpu().numpy(), np.broadcast_to(want.astype(np.float32), (M, N)))


def test_product_empty():
    A = torch.zeros((5, 0), dtype=torch.int8, device=DEV)
    W = torch.zeros((7, 0), dtype=torch.int8, device=DEV)
    sa, sw = torch.ones(5, device=DEV), torch.ones(7, device=DEV)
    b = torch.arange(7, device=DEV, dtype=torch.float32) - 3.0
    say("gemm_i8 K = 0")
    C = binding.gemm_i8(A, sa, W, sw, bias=b, epilogue="relu")
    torch.cuda.synchronize()
    assert torch.equal(C.float(), b.clamp(min=0).expand(5, 7))
    assert binding.gemm_i8(A[:0], sa[:0], W, sw).shape == (0, 7)
    assert binding.gemm_i8(A, sa, W[:0], sw[:0]).shape == (5, 0)


def test_product_special_scales():
    """A NaN or infinite scale stays in its own row or column; ReLU maps NaN to 0."""
    for M, N, K in ((6, 40, 96), (70, 130, 256), (256, 256, 256)):
        A, sa, W, sw, _ = make_product(M, N, K, 5, bias=False)
        sa[2], sw[3] = np.nan, np.nan
        say("gemm_i8 special scales %dx%dx%d" % (M, N, K))
        C = binding.gemm_i8(dev(A), dev(sa), dev(W), dev(sw)).float().cpu().numpy()
        nan = np.zeros((M, N), bool)
        nan[2], nan[:, 3] = True, True
        assert np.array_equal(np.isnan(C), nan)
        C = binding.gemm_i8(dev(A), dev(sa), dev(W), dev(sw), epilogue="relu")
        assert not bool(C.isnan().any()) and not bool(C[2].any())


def test_product_refusals():
    q = torch.zeros((4, 32), dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="inner dimensions"):
        binding.gemm_i8(q, s, q[:, :16], s)
    with pytest.raises(TypeError, match="int8"):
        binding.gemm_i8(q.float(), s, q, s)
    with pytest.raises(ValueError, match="unit stride"):
        binding.gemm_i8(q[:, ::2], s, q[:, ::2], s)
    with pytest.raises(ValueError, match="overlap"):
        binding.gemm_i8(q[:1].expand(4, 32), s, q, s)
    with pytest.raises(ValueError, match="dense vector"):
        binding.gemm_i8(q, s[:3], q, s)
    with pytest.raises(TypeError, match="float32"):
        binding.gemm_i8(q, s.double(), q, s)
    with pytest.raises(ValueError, match="one device|GPU tensor"):
        binding.gemm_i8(q, s.cpu(), q, s)
    with pytest.raises(TypeError, match="unsupported dtype"):
        binding.gemm_i8(q, s, q, s, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="C must be"):
        binding.gemm_i8(q, s, q, s, C=torch.empty((4, 5), device=DEV))
    with pytest.raises(TypeError, match="C must be"):
        binding.linear_i8(torch.zeros((4, 32), device=DEV), q, s,
                          C=torch.empty((4, 4), dtype=torch.float16, device=DEV))
    with pytest.raises(binding.TileGemmError) as e:
        binding.linear_i8(torch.zeros((1000, 32), device=DEV), q, s,
                          workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == 9


def activations(r, M, K, dtype):
    v = r.normal(size=(M, K)) * np.exp(0.5 * r.normal(size=(1, K)))
    return torch.from_numpy(v.astype(np.float32)).to(torch_dtype(dtype)).to(DEV)


ROWS = [1, 2, 7, 8, 9, 63, 64, 100, 511, 512, 513, 1003, 2048, 2056, 4096, 4097, 8192, 8200, 32768,
        32769, 40000]


@TYPES
@pytest.mark.parametrize("K", ROWS)
def test_quant_rows(K, dtype):
    r = np.random.Generator(np.random.PCG64(K))
    M = 5
    x = activations(r, M, K, dtype)
    v = values(x, dtype)
    q, s = ref.levels(v)
    for pad, shift in ((0, 0), (3, 1)):
        say("quant_i8 %dx%d %s pad=%d" % (M, K, DNAME[dtype], pad))
        Q = strided(torch.zeros((M, K), dtype=torch.int8, device=DEV), pad, shift)
        Q, S = binding.quant_i8(strided(x, pad, shift), Q)
        torch.cuda.synchronize()
        assert np.array_equal(Q.cpu().numpy(), q)
        # one division of an exact value by 127, rounded
        assert np.array_equal(S.cpu().numpy(), s.astype(np.float32))


@TYPES
def test_quant_ties(dtype):
    """Values on the border between two levels go to the even one: multiples
    of a half of the row's step, for every magnitude of 8 bits."""
    a = np.arange(128, 256, dtype=np.float64)
    v = np.concatenate([a[:, None], a[:, None] * np.array([0.5, -0.5, 0.25, -0.25, 1.0, -1.0])],
                       axis=1)
    # and rows of the step 1 and 2 with every half
    half = np.concatenate([[127.0], np.arange(-126.5, 127.0, 1.0)])
    x = torch.zeros((len(a) + 2, 300), dtype=torch.float64)
    x[:len(a), :v.shape[1]] = torch.from_numpy(v)
    x[len(a), :half.size] = torch.from_numpy(half)
    x[len(a) + 1, :half.size] = torch.from_numpy(half * 2)
    x = x.to(torch_dtype(dtype)).to(DEV)
    q, _ = ref.levels(values(x, dtype))
    say("quant_i8 ties %s" % DNAME[dtype])
    Q, _ = binding.quant_i8(x)
    torch.cuda.synchronize()
    assert np.array_equal(Q.cpu().numpy(), q)


@TYPES
def test_quant_special_rows(dtype):
    """Zeros, infinities, NaN, the type's smallest and largest values."""
    info = torch.finfo(torch_dtype(dtype))
    x = torch.randn((9, 70), device=DEV).to(torch_dtype(dtype))
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 69] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = info.max
    x[4, 3] = -info.max / 2
    x[5] = 0
    x[5, 3] = info.smallest_normal
    x[5, 4] = -info.smallest_normal / 2
    x[6] = 0
    x[6, 1] = info.smallest_normal / 8  # subnormal
    x[7] = info.min
    say("quant_i8 special rows %s" % DNAME[dtype])
    Q, S = binding.quant_i8(x)
    torch.cuda.synchronize()
    q, s = ref.levels(values(x, dtype))
    assert np.array_equal(Q.cpu().numpy(), q)
    assert np.array_equal(np.isnan(S.cpu().numpy()), np.isnan(s))
    ok = ~np.isnan(s)
    assert np.array_equal(S.cpu().numpy()[ok], s[ok].astype(np.float32))


def test_quant_empty():
    Q, S = binding.quant_i8(torch.zeros((3, 0), device=DEV))
    torch.cuda.synchronize()
    assert Q.shape == (3, 0) and S.tolist() == [2.0 ** -126] * 3
    assert binding.quant_i8(torch.zeros((0, 9), device=DEV))[0].shape == (0, 9)


@TYPES
@pytest.mark.parametrize("M,N,K", [(1, 64, 1024), (1, 65, 1000), (2, 100, 72), (4, 200, 4096),
                                   (8, 33, 520), (13, 96, 2048), (16, 300, 8192), (17, 64, 64),
                                   (33, 128, 1001), (100, 200, 256), (257, 130, 1040), (5, 6, 0)])
def test_linear_equals_its_parts(M, N, K, dtype):
    """linear_i8 has the bits of quant_i8 followed by gemm_i8."""
    r = np.random.Generator(np.random.PCG64(M * N + K))
    x = activations(r, M, K, dtype) if K else torch.zeros((M, 0), dtype=torch_dtype(dtype),
                                                          device=DEV)
    _, _, W, sw, b = make_product(1, N, K, 3)
    W, sw, b = dev(W), dev(sw), dev(b)
    for pad in (0, 5):
        say("linear_i8 %dx%dx%d %s pad=%d" % (M, N, K, DNAME[dtype], pad))
        xs = strided(x, pad, pad) if K else x
        C = binding.linear_i8(xs, W, sw, bias=b, epilogue="relu")
        Q, S = binding.quant_i8(x)
        D = binding.gemm_i8(Q, S, W, sw, bias=b, out_dtype=x.dtype, epilogue="relu")
        torch.cuda.synchronize()
        assert torch.equal(C.view(torch.uint8), D.view(torch.uint8))
    if K:
        v = values(x, dtype)
        q, s = ref.levels(v)
        check_product(values(C, dtype), q, s.astype(np.float32), W.cpu().numpy(),
                      sw.cpu().numpy(), b.cpu().numpy(), dtype, True)


@TYPES
@pytest.mark.parametrize("M,N,K", [(1, 33, 257), (1, 100, 2049), (3, 48, 1003), (8, 17, 1538),
                                   (5, 30, 15), (16, 50, 770), (40, 4100, 515), (150, 200, 333)])
def test_linear_rows_at_any_byte(M, N, K, dtype):
    """W's rows at 4-byte and at single-byte steps: the bits of quant_i8 followed
    by gemm_i8 on rows at 16-byte boundaries."""
    r = np.random.Generator(np.random.PCG64(M + N + K))
    x = activations(r, M, K, dtype)
    _, _, W, sw, b = make_product(1, N, K, 3)
    W, sw, b = dev(W), dev(sw), dev(b)
    q, s = binding.quant_i8(x)
    wide = (K + 15) // 16 * 16
    want = binding.gemm_i8(strided(q, wide - K), s, strided(W, wide - K), sw, bias=b,
                           out_dtype=torch_dtype(dtype))
    for pad, shift in ((0, 0), (1, 0), (2, 1), ((-K) % 4, 0), ((-K) % 4, 3), ((-K) % 16, 2)):
        say("linear_i8 %dx%dx%d %s pad=%d shift=%d" % (M, N, K, DNAME[dtype], pad, shift))
        got = binding.linear_i8(x, strided(W, pad, shift), sw, bias=b)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@TYPES
@pytest.mark.parametrize("M,N,K", [(300, 300, 2050), (1030, 2000, 1001), (1030, 301, 510),
                                   (257, 100, 5001), (200, 70, 9007), (130, 40, 33001)])
def test_linear_copies_weights(M, N, K, dtype):
    """Sizes where the rows of W are copied to 16-byte boundaries in the
    workspace: the bits of the product on W as it is, whatever the workspace
    held, and nothing past the workspace written."""
    r = np.random.Generator(np.random.PCG64(M + N + K))
    x = activations(r, M, K, dtype)
    _, _, W, sw, b = make_product(1, N, K, 3)
    W, sw, b = dev(W), dev(sw), dev(b)
    q, s = binding.quant_i8(x)
    want = binding.gemm_i8(q, s, W, sw, bias=b, out_dtype=torch_dtype(dtype))
    need = binding.linear_i8_workspace_size(M, N, K, dtype)
    assert need >= (M + N) * K
    for pad, shift in ((0, 0), (1, 0), ((-K) % 16, 0), (5, 3)):
        say("linear_i8 %dx%dx%d %s pad=%d shift=%d" % (M, N, K, DNAME[dtype], pad, shift))
        ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        got = binding.linear_i8(x, strided(W, pad, shift), sw, bias=b, workspace=ws[:need])
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert bool((ws[need:] == 0x7F).all())


def test_linear_workspace_contents_do_not_matter():
    """A workspace of the reported size, full of other bytes; the bytes after it
    stay."""
    M, N, K = 40, 96, 1000
    x = torch.randn((M, K), device=DEV, dtype=torch.bfloat16)
    _, _, W, sw, b = make_product(1, N, K, 3)
    W, sw, b = dev(W), dev(sw), dev(b)
    want = binding.linear_i8(x, W, sw, bias=b)
    need = binding.linear_i8_workspace_size(M, N, K, BF16)
    for fill in (0xFF, 0x7F):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device=DEV)
        say("linear_i8 workspace of %02x" % fill)
        got = binding.linear_i8(x, W, sw, bias=b, workspace=ws[:need])
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool((ws[need:] == fill).all())


def test_linear_rows_that_are_not_finite():
    for M in (1, 5, 40, 300):
        x = torch.randn((M, 512), device=DEV, dtype=torch.bfloat16)
        x[0, 3] = float("nan")
        if M > 1:
            x[M - 1, 500] = float("-inf")
        _, _, W, sw, _ = make_product(1, 96, 512, 3)
        say("linear_i8 not finite M=%d" % M)
        C = binding.linear_i8(x, dev(W), dev(sw))
        bad = C.isnan().all(dim=1).cpu().tolist()
        assert bad == [i == 0 or i == M - 1 for i in range(M)]
        assert not bool(C[1:M - 1].isnan().any())


@pytest.mark.parametrize("M,N,K", [(1, 256, 1024), (16, 256, 1024), (64, 256, 512),
                                   (300, 512, 512), (300, 300, 2050), (8, 100, 1003),
                                   (4100, 4096, 1024)])
def test_stream_and_graph(M, N, K):
    """On a side stream, and captured and replayed with new inputs between
    eager calls: the same bits as the eager call on the null stream."""
    r = np.random.Generator(np.random.PCG64(1))
    xs = [activations(r, M, K, BF16) for _ in range(3)]
    _, _, W, sw, b = make_product(1, N, K, 3)
    W, sw, b = dev(W), dev(sw), dev(b)
    want = [binding.linear_i8(x, W, sw, bias=b) for x in xs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    say("linear_i8 on a side stream M=%d" % M)
    got = binding.linear_i8(xs[0], W, sw, bias=b, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])
    x, C = xs[0].clone(), torch.zeros_like(want[0])
    need = binding.linear_i8_workspace_size(M, N, K, BF16)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.linear_i8(x, W, sw, bias=b, C=C, workspace=ws)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        C.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want[i])
        assert torch.equal(binding.linear_i8(xs[2 - i], W, sw, bias=b), want[2 - i])


@pytest.mark.parametrize("K", [4096, 4095])
def test_offsets_past_31_bits(K):
    """Operands and results beyond 2^31 bytes: the last rows have the bits of a
    call on them alone."""
    M, N = 540000, 2056  # A 2.2 GB, C 2.2 GB
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    A = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV, generator=g)
    W = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sa = torch.rand(M, device=DEV, generator=g)
    sw = torch.rand(N, device=DEV, generator=g)
    say("gemm_i8 %dx%dx%d" % (M, N, K))
    C = binding.gemm_i8(A, sa, W, sw)
    torch.cuda.synchronize()
    assert M * K > 1 << 31 and C.numel() * 2 > 1 << 31
    for at in (M - 300, (1 << 31) // K - 150):
        part = binding.gemm_i8(A[at:at + 300], sa[at:at + 300], W, sw)
        torch.cuda.synchronize()
        assert torch.equal(part, C[at:at + 300])
    del C
    x = A[:300000].to(torch.bfloat16)
    say("quant_i8 %dx%d" % tuple(x.shape))
    Q, S = binding.quant_i8(x)
    torch.cuda.synchronize()
    q, s = binding.quant_i8(x[-100:])
    torch.cuda.synchronize()
    assert torch.equal(Q[-100:], q) and torch.equal(S[-100:], s)
