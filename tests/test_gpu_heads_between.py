"""GPU tests of head norms whose queries and keys lie between each other."""

import pytest
import torch

import mx_heads_reference as ref
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("T,H,D", [(37, 4, 64), (1, 5, 33), (300, 3, 100)])
def test_queries_and_keys_in_turn(T, H, D, order):
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    cos, sin = (t.cuda() for t in ref.tables(T, D // 4))
    wq, wk = rnd(D), rnd(D)

    def buffer():  # a query's head, a key's and others behind them; or a token's of each
        x = rnd(T, H, 3, D) if order == "heads" else rnd(H, T, 3, D).transpose(0, 1)
        return x, x[:, :, 0], x[:, :, 1]

    x, q, k = buffer()
    want = binding.head_norm_rope(q.contiguous(), k.contiguous(), wq, wk, cos, sin, None, EPS)
    y, qo, ko = buffer()
    kept = y[:, :, 2].clone()
    binding.head_norm_rope(q, k, wq, wk, cos, sin, None, EPS, q_out=qo, k_out=ko)
    assert torch.equal(qo, want.q) and torch.equal(ko, want.k) and torch.equal(y[:, :, 2], kept)
    kept = x[:, :, 2].clone()
    binding.head_norm_rope(q, k, wq, wk, cos, sin, None, EPS, q_out=q, k_out=k)
    assert torch.equal(q, want.q) and torch.equal(k, want.k) and torch.equal(x[:, :, 2], kept)
