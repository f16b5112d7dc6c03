"""GPU tests of the products in microscaled blocks: E4M3 activations whose small
elements stand beside large ones, and the same call again."""

import pytest
import torch

import mx_heads_reference as ref
from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def wide(M, K, seed):
    """Rows whose products with E2M1 elements have exact sums in fp32, though elements of
    one group of eight are up to 2^17 apart: in each block of 32 one element of 256 and,
    beside it and behind it, odd multiples of 2^-9 (E4M3's smallest steps) and some of
    1.75 to 30, all of them E4M3 values at the block's power of two, 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n: torch.randint(0, n, (M, K), generator=g, device="cuda")
    x = (2 * rnd(4) + 1).float() * 2.0 ** -9
    mid = torch.tensor([1.75, 1.875, 2.0, 2.25, 3.75, 15.0, 30.0, 0.0], device="cuda")[rnd(8)]
    x = torch.where(rnd(4) == 0, mid, x)
    x = torch.where(rnd(2) == 0, x, -x)
    x[:, 3::32] = 256.0
    return x


def weights(N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.tensor(ref.E2M1_VALUES, device="cuda")[
        torch.randint(0, 8, (N, K), generator=g, device="cuda")]
    w = torch.where(torch.randint(0, 2, (N, K), generator=g, device="cuda") == 0, t, -t)
    w[:, ::32] = 4.0  # the same power of two for every block
    w[:, 3::32] = torch.tensor([1.0, -1.0], device="cuda").repeat(K // 32 + 1)[:w[:, 3::32].shape[1]]
    return w


@pytest.mark.parametrize("K", [128, 256, 416])
@pytest.mark.parametrize("M", [1, 7, 16, 20, 40, 130, 300, 1500])
def test_e4m3_products_are_exact(M, K):
    # |sum| < K / 32 (256 + 31 * 180) < 2^17 in all, less than 2^14 in steps of 2^-10
    # for what these inputs give: every partial sum is exact in fp32, in any order
    say("e4m3 exact %d x %d" % (M, K))
    x, w = wide(M, K, M + K), weights(300, K, K)
    f = binding.quant_mx(w)
    assert (f.s[:, :K // 32] == 127).all()
    want = x.double() @ w.double().t()
    assert float((x.double().abs() @ w.double().abs().t()).max()) < 2.0 ** 14
    c = binding.linear_mx(x, f.q, f.s, fmt=ref.E4M3)
    assert torch.equal(c.double(), want)
    if M <= 16:  # x is exact in 16 bits, too
        for dtype in (BF16, F16):
            c = binding.linear_mx(x.to(dtype), f.q, f.s, fmt=ref.E4M3)
            assert torch.equal(c, want.to(dtype))


def test_e4m3_products_are_exact_in_gradients():
    M, N, K = 300, 160, 96
    d, w = wide(M, N, 5), weights(K, N, 6).t().contiguous()
    g = binding.linear_mx_backward(d, W=w, fmt=ref.E4M3)
    assert torch.equal(g.dx.double(), d.double() @ w.double())
    d, x = wide(N, M, 7).t().contiguous(), weights(K, M, 8).t().contiguous()
    g = binding.linear_mx_backward(d, X=x, fmt=ref.E4M3)
    assert torch.equal(g.dw.double(), d.double().t().contiguous() @ x.double())


@pytest.mark.parametrize("M,N,K", [(16, 8192, 8192), (64, 4096, 4096), (1000, 1001, 1003),
                                   (2048, 2048, 2048)])
@pytest.mark.parametrize("fmt", [ref.E2M1, ref.E4M3])
def test_the_same_call_gives_the_same_bits(M, N, K, fmt):
    say("again %d x %d x %d fmt %d" % (M, N, K, fmt))
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    other = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    w = binding.quant_mx(torch.randn((N, K), generator=g, device="cuda"))
    first = binding.linear_mx(x, w.q, w.s, fmt=fmt)
    for _ in range(8):
        binding.linear_mx(other, w.q, w.s, fmt=fmt)
        assert torch.equal(binding.linear_mx(x, w.q, w.s, fmt=fmt), first)


@pytest.mark.parametrize("fmt", [ref.E2M1, ref.E4M3])
@pytest.mark.parametrize("M,N,K", [(1, 200, 1003), (16, 100, 4100), (40, 300, 601), (300, 129, 130),
                                   (389, 2423, 1150), (1439, 5439, 200)])
def test_what_weights_hold_past_k_has_no_part(M, N, K, fmt):
    say("weights past k %d x %d x %d fmt %d" % (M, N, K, fmt))
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    w = binding.quant_mx(torch.randn((N, K), generator=g, device="cuda"))
    want = binding.linear_mx(x, w.q, w.s, fmt=fmt)
    codes, s = ref.unpack(w.q, ref.E2M1).clone(), w.s.clone()
    codes[:, K:] = torch.randint(0, 16, codes[:, K:].shape, generator=g, device="cuda")
    whole = -(-K // 32)  # blocks past the last one that holds values
    s[:, whole:] = torch.randint(0, 255, s[:, whole:].shape, generator=g, device="cuda",
                                 dtype=torch.uint8)
    assert torch.equal(binding.linear_mx(x, ref.pack(codes, ref.E2M1), s, fmt=fmt), want)
