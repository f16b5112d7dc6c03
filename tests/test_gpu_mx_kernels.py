"""GPU tests of every kernel that linear_mx chooses among: each with odd sizes and C rows,
all types of C, and K of every number of steps that its loop tells apart.  The kernels and
their costs stand in tg_mx_e2m1.hip and tg_mx_e4m3.hip; the sizes below are such that the
costs choose the kernel that is named, which the launch log confirms."""

import os
import re

import pytest
import torch

import mx_heads_reference as ref
from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FMT = {"E2M1": ref.E2M1, "E4M3": ref.E4M3}

# (kernel, M, N, K in steps of 128).  Strips of 256 k: every remainder of a chunk of 1024,
# before the first whole one and after it; streams: runs of 512 k shared out among four or
# eight waves, and one to three steps behind them.
CHUNKS = tuple(range(1, 17))
RUNS = (1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 16, 29, 30, 31, 64)
CASES = [
    ("mx_stream_MX_E2M1_n1_m1_st4_w4", 199, 615, RUNS),
    ("mx_stream_MX_E2M1_n1_m1_st4_w8", 17, 37, (10, 11, 16, 29, 30, 31, 64)),
    ("mx_stream_MX_E2M1_n2_m1_st4_w4", 17, 2259, RUNS),
    ("mx_stream_MX_E2M1_n2_m2_st4_w4", 19, 6259, RUNS),
    ("mx_stream_MX_E2M1_n4_m2_st4_w4", 65, 4413, RUNS[2:]),
    ("mx_linear_MX_E2M1_64x64_w2x2_s4_MX_S128", 301, 129, CHUNKS),
    ("mx_linear_MX_E2M1_128x128_w2x4_s2_MX_S256", 389, 2423, CHUNKS),
    ("mx_linear_MX_E2M1_256x128_w2x4_s2_MX_S256", 2961, 2581, CHUNKS),
    ("mx_linear_MX_E2M1_128x256_w2x4_s2_MX_S256", 1545, 4731, CHUNKS),
    ("mx_linear_MX_E2M1_256x256_w2x4_s4_MX_S128", 1439, 5439, (1, 2, 3, 4, 5, 6, 7, 9, 11, 15)),
    ("mx_linear_MX_E2M1_256x256_w2x4_s2_MX_S256_1024", 1439, 5439, (8, 16, 24)),
    ("mx_stream_MX_E4M3_n1_m1_st4_w4", 199, 615, RUNS[:11]),
    ("mx_stream_MX_E4M3_n1_m1_st4_w8", 17, 37, (16, 29, 30, 31, 64)),
    ("mx_stream_MX_E4M3_n2_m1_st4_w4", 17, 2259, RUNS),
    ("mx_stream_MX_E4M3_n2_m2_st4_w4", 19, 4477, RUNS),
    ("mx_stream_MX_E4M3_n4_m2_st4_w4", 65, 4413, RUNS[:10]),
    ("mx_linear_MX_E4M3_64x64_w2x2_s4_MX_S128", 301, 129, CHUNKS),
    ("mx_linear_MX_E4M3_128x128_w2x4_s2_MX_S256", 389, 2423, CHUNKS),
    ("mx_linear_MX_E4M3_128x256_w2x4_s2_MX_S256", 641, 5401, CHUNKS),
    # the decode batch and the training step that perf/more_operators.py measures
    ("mx_stream_MX_E2M1_n2_m1_st4_w4", 16, 8192, (64,)),
    ("mx_stream_MX_E4M3_n2_m1_st4_w4", 16, 8192, (64,)),
    ("mx_linear_MX_E2M1_128x256_w2x4_s2_MX_S256", 2048, 4096, (32,)),
]


def table_of(fmt):
    """Names of the kernels in a format's table."""
    root = os.path.dirname(os.path.abspath(binding.__file__))
    names = set()
    with open(os.path.join(root, "csrc", "tg_mx_%s.hip" % fmt.lower())) as f:
        for line in f:
            m = re.search(r"TG_MX_(TILE|STREAM)\((.*)\)", line)
            if not m:
                continue
            a = [v.strip() for v in m.group(2).split(",")]
            names.add("mx_linear_%s_%sx%s_w%sx%s_s%s_%s" % (*a[1:7], a[0]) if m.group(1) == "TILE"
                      else "mx_stream_%s_n%s_m%s_st%s_w%s" % tuple(a[:5]))
    return names


@pytest.mark.parametrize("fmt", sorted(FMT))
def test_no_kernel_is_left_out(fmt):
    assert table_of(fmt) == {c[0] for c in CASES if "_MX_%s_" % fmt in c[0]}


def inputs(M, N, K, seed):
    """X whose values all three types hold, blocks of different powers of two; weights, bias."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-127, 128, (M, K), generator=g, device="cuda").float() / 16
    x *= torch.exp2(torch.randint(-4, 4, (M, -(-K // 32)), generator=g, device="cuda").float()
                    ).repeat_interleave(32, dim=1)[:, :K]
    w = binding.quant_mx(torch.randn((N, K), generator=g, device="cuda"))
    return x, w, torch.randn((N,), generator=g, device="cuda")


def exact_products(ca, sa, fa, cw, sw, bias):
    """As ref.product where no product is cut off: each group of eight (E4M3: each half of
    one) is added with a cut of at most a step of what has been summed."""
    a, w = ref.values(ca, sa, fa), ref.values(cw, sw, ref.E2M1)
    wt = w.t().contiguous()
    mag = a.abs() @ wt.abs() + bias.double().abs()
    halves = 2 if fa == ref.E4M3 else 1
    return a @ wt + bias.double(), 2 * (halves * a.shape[1] // 8 + 16) * ref.U32 * mag


@pytest.mark.parametrize("name,M,N,steps", [pytest.param(n, M, N, s, id="%s-%d-%d-%d" % (n, M, N, s))
                                            for n, M, N, all_steps in CASES for s in all_steps])
def test_kernel(name, M, N, steps, monkeypatch, capfd):
    # K up to the end of the last step's first block, so that rows are odd as well
    K = 128 * steps if N % 2 == 0 else 128 * steps - 97
    fmt = FMT[name.split("_")[3]]
    say("%s %d x %d x %d" % (name, M, N, K))
    x, w, bias = inputs(M, N, K, steps)
    blocks = (*ref.quantise(x, fmt), fmt, ref.unpack(w.q, ref.E2M1), w.s.to(torch.int64), bias)
    exact = exact_products(*blocks)
    cut = ref.product(*blocks) if fmt == ref.E4M3 and name.startswith("mx_linear") else exact
    for dtype in (BF16, F16, F32):
        monkeypatch.setenv("TG_LOG", "1")
        capfd.readouterr()
        c = binding.linear_mx(x.to(dtype), w.q, w.s, bias=bias, fmt=fmt)
        monkeypatch.delenv("TG_LOG")
        log = capfd.readouterr().err
        assert "[tilegemm] %s " % name in log, "other sizes are needed: " + log
        ref.assert_close(c, *(exact if dtype == F32 else cut), dtype, name)


def test_fused_kernel_is_the_product_of_its_parts():
    # quantisation and product in one launch, and in two calls: small integers, whose sums
    # are exact in any order, give the same bits
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, K in ((1, 4096), (16, 2048), (7, 1003), (3, 129)):
        x = torch.randint(-8, 9, (M, K), generator=g, device="cuda").to(BF16)
        w = binding.quant_mx(torch.randint(-6, 7, (200, K), generator=g, device="cuda").float())
        assert binding.linear_mx_workspace_size(M, 200, K, binding.TG_BF16) == 0
        for fmt in FMT.values():
            f = binding.quant_mx(x, fmt)
            want = (ref.values(ref.unpack(f.q, fmt), f.s.long(), fmt)
                    @ ref.values(ref.unpack(w.q, 0), w.s.long(), 0).t().contiguous())
            c = binding.linear_mx(x.float(), w.q, w.s, fmt=fmt)
            assert torch.equal(c.double(), want)


@pytest.mark.parametrize("M,K", [(48, 1024), (300, 2048), (2048, 1024)])
@pytest.mark.parametrize("fmt", sorted(FMT))
def test_linear_is_quantisation_and_gemm_mx(M, K, fmt):
    # integers whose products and sums gemm_mx and linear_mx hold exactly: the same bits
    fmt = FMT[fmt]
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randint(-8, 9, (M, K), generator=g, device="cuda").to(BF16)
    w = binding.quant_mx(torch.randint(-6, 7, (256, K), generator=g, device="cuda").float())
    f = binding.quant_mx(x, fmt)
    assert torch.equal(binding.gemm_mx(fmt, f.q, f.s, w.q, w.s), binding.linear_mx(x, w.q, w.s, fmt=fmt))
