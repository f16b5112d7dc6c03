"""GPU tests of calls whose outputs have no elements."""

import pytest
import torch

from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_gradients_that_are_empty_by_themselves(wtype):
    z = lambda *s, dtype=torch.bfloat16: torch.ones(s, dtype=dtype, device="cuda")
    W = z(8, 40, dtype=wtype)
    g = binding.linear_mx_backward(z(0, 8), W=W)  # a frozen layer without tokens
    assert g.dx.shape == (0, 40) and g.dw is None and g.dbias is None
    g = binding.linear_mx_backward(z(5, 8), X=z(5, 0))
    assert g.dw.shape == (8, 0) and g.dx is None
    g = binding.linear_mx_backward(z(5, 8), W=z(8, 0, dtype=wtype))
    assert g.dx.shape == (5, 0)
    g = binding.linear_mx_backward(z(5, 0), X=z(5, 40))
    assert g.dw.shape == (0, 40)
    g = binding.linear_mx_backward(z(0, 8), X=z(0, 40))
    assert g.dw.shape == (8, 40) and (g.dw == 0).all()
    g = binding.linear_mx_backward(z(5, 0), W=z(0, 40, dtype=wtype))
    assert g.dx.shape == (5, 40) and (g.dx == 0).all()
    g = binding.linear_mx_backward(z(0, 0), W=z(0, 40, dtype=wtype), dbias=True)
    assert g.dx.shape == (0, 40) and g.dbias.shape == (0,)
    torch.cuda.synchronize()


def test_heads_that_are_empty_by_themselves():
    q = torch.ones((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert binding.head_norm_rope(q).q.shape == (0, 4, 64)
    g = binding.head_norm_rope_backward(q, None, q)
    assert g.dq.shape == (0, 4, 64) and g.dw_q is None
    q = torch.ones((3, 0, 64), dtype=torch.bfloat16, device="cuda")
    assert binding.head_norm_rope(q).q.shape == (3, 0, 64)
    assert binding.head_norm_rope_backward(q, None, q).dq.shape == (3, 0, 64)
    torch.cuda.synchronize()
