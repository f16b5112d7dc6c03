"""The 8-bit feed-forward stack: its operators run together as a serving program
runs them, against the same stack in fp32."""

from __future__ import annotations

import pytest

from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (7, 200, 333), (64, 512, 1024),
                                                 (300, 256, 640)])
def test_stack_against_fp32(tokens, width, hidden):
    """Each quantised operand is off by a level's rounding, 1 / sqrt(12) of 1/127
    of its row's largest value, which is up to five times its rms: 1.2% of it.
    A layer has four such operands (2.3% of y together), bf16 roundings of
    0.2% beside them, and adds y, half as large, to the residual stream: 1.2% a
    layer, 1.7% for two."""
    from tiled_dense_gemm_07_amd.int8_block import Int8Stack

    stack = Int8Stack(width, hidden, 2, seed=3)
    x = torch.randn((tokens, width), device="cuda").to(torch.bfloat16)
    say("int8 stack %dx%dx%d" % (tokens, width, hidden))
    got, want = stack.serve(x).float(), stack.plain(x)
    torch.cuda.synchronize()
    assert (got - want).norm() <= 0.017 * want.norm()


def test_stack_in_a_graph():
    from tiled_dense_gemm_07_amd.int8_block import Int8Stack

    stack = Int8Stack(512, 1024, 3)
    xs = [torch.randn((16, 512), device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = [stack.serve(x) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    say("int8 stack graph")
    with torch.cuda.graph(g):
        out = stack.serve(x)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(stack.serve(xs[2 - i]), want[2 - i])


def test_boundary_step():
    from tiled_dense_gemm_07_amd.int8_block import Int8Stack

    stack = Int8Stack(512, 1024, 2)
    x, y, dx, dh = (torch.randn((40, 512), device="cuda").to(torch.bfloat16) for _ in range(4))
    say("int8 stack boundary step")
    f, g = stack.boundary_step(x, y, dx, dh)
    torch.cuda.synchronize()
    assert f.h.shape == (40, 512) and g.dx.shape == (40, 512) and g.dy.shape == (40, 512)
    assert g.dgate.shape == (512,) and g.dw_post.shape == (512,) and g.dw_pre.shape == (512,)
    assert all(bool(t.isfinite().all()) for t in g)


def test_command(capsys):
    from tiled_dense_gemm_07_amd import int8_block

    assert int8_block.main(["--tokens", "16", "--width", "512", "--hidden", "512",
                            "--layers", "2"]) == 0
    assert "serving 16 tokens" in capsys.readouterr().out
