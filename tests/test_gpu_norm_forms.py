"""Forms of the block norms on the GPU beside the full boundary, against the 64-bit
forms."""

from __future__ import annotations

import pytest

from gpu_helpers import say
from test_gpu_block_norm import DNAME, EPS, by_pair, check_backward, check_forward, operands, run_backward
from tiled_dense_gemm_07_amd import binding

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()


# --------------------------------------------------------------------------
# the norm alone
# --------------------------------------------------------------------------
@by_pair
def test_norm_alone_has_no_alpha(xt, bt):
    """Without a block before, x' is x whatever alpha is, and its gradient is not
    scaled: a program may hand its layers' alpha to every call."""
    T, D, alpha = 13, 300, 0.75
    s = {**operands(T, D, xt, bt, 0, False, 31), "y": None}
    say("block_norm alone, alpha %g, %s/%s" % (alpha, DNAME[xt], DNAME[bt]))
    f = binding.block_norm(s["x"], w_pre=s["w_pre"], alpha=alpha, eps=EPS, save=True)
    g = run_backward(s, f, xt, bt, 0, alpha, False)
    torch.cuda.synchronize()
    check_forward(s, f, xt, bt, 0, 1.0, False)
    check_backward(s, f, g, xt, bt, 0, 1.0, False)
    same = run_backward(s, f, xt, bt, 0, 1.0, False)
    torch.cuda.synchronize()
    assert torch.equal(g.dx, same.dx) and torch.equal(g.dw_pre, same.dw_pre)
