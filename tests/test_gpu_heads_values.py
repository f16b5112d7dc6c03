"""GPU tests of the head norms with rotation: what stands beside values that are not
finite, where a part of the head is turned or none."""

import pytest
import torch

import mx_heads_reference as ref
from gpu_helpers import say
from tiled_dense_gemm_07_amd import binding

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
INF, NAN = float("inf"), float("nan")

# R below D and none, both orders, heads in one chunk and in several, lengths that
# eight does not divide, fewer than four values, small tables
FORMS = [(64, 32, 9), (64, 0, 9), (128, 64, 9), (99, 66, 9), (99, 0, 9), (30, 6, 9), (7, 4, 9),
         (3, 2, 9), (3, 0, 9), (300, 100, 9), (1023, 6, 9), (515, 2, 1), (200, 6, 1), (96, 80, 9)]


def inputs(T, H, D, R, P, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    cos, sin = (t.cuda() for t in ref.tables(P, R // 2))
    pos = torch.randint(0, P, (T,), generator=g, device="cuda")
    return (2 * rnd(T, H, D)).to(dtype), (1 + 0.2 * rnd(D)).to(dtype), cos, sin, pos


def pair_of(i, R, interleaved):
    """The values that value i is turned with, itself among them."""
    if i >= R:
        return {i}
    if interleaved:
        return {i, i ^ 1}
    return {i, (i + R // 2) % R}


def places(D, R):
    """Values behind the turned ones, at their ends and in the middle, and a turned one."""
    return sorted({R, R + 1, (R + D) // 2, D - 2, D - 1} & set(range(R, D))) + ([R - 1] if R else [])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D,R,P", FORMS)
def test_a_weight_that_is_not_finite(D, R, P, dtype, interleaved):
    say("heads weight %d %d %s %s" % (D, R, dtype, interleaved))
    x, w, cos, sin, pos = inputs(4, 3, D, R, P, dtype, D + R)
    plain = binding.head_norm_rope(x, None, w, None, cos, sin, pos, EPS, interleaved).q
    for at in places(D, R):
        for value in (INF, NAN):
            bad = w.clone()
            bad[at] = value
            got = binding.head_norm_rope(x, None, bad, None, cos, sin, pos, EPS, interleaved).q
            touched = pair_of(at, R, interleaved)
            rest = [i for i in range(D) if i not in touched]
            assert torch.equal(got[:, :, rest], plain[:, :, rest]), at
            assert not torch.isfinite(got[:, :, at]).any(), at
            if at >= R:  # not turned: the value itself
                want = (x[:, :, at].float() * value).to(dtype)
                assert torch.equal(torch.isnan(got[:, :, at]), torch.isnan(want))
                assert torch.equal(got[:, :, at][~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D,R,P", FORMS)
def test_a_gradient_that_is_not_finite(D, R, P, dtype, interleaved):
    say("heads gradient %d %d %s %s" % (D, R, dtype, interleaved))
    x, w, cos, sin, pos = inputs(5, 3, D, R, P, dtype, D + R + 1)
    d = inputs(5, 3, D, R, P, dtype, 77)[0]
    plain = binding.head_norm_rope_backward(d, None, x, None, w, None, cos, sin, pos, EPS,
                                            interleaved)
    for at in places(D, R):
        for value in (INF, NAN):
            bad = d.clone()
            bad[2, 1, at] = value
            got = binding.head_norm_rope_backward(bad, None, x, None, w, None, cos, sin, pos, EPS,
                                                  interleaved)
            rest = [i for i in range(D) if i not in pair_of(at, R, interleaved)]
            assert torch.equal(got.dw_q[rest], plain.dw_q[rest]), at
            assert not torch.isfinite(got.dw_q[at])
            # that head alone: its mean takes the gradient
            keep = torch.ones((5, 3), dtype=torch.bool, device="cuda")
            keep[2, 1] = False
            assert torch.equal(got.dq[keep], plain.dq[keep])
            assert torch.isnan(got.dq[2, 1, at])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 32), (64, 0), (33, 20)])
def test_an_infinite_value(D, R, interleaved):
    # x is infinite at one place behind the turned ones: r is zero, so that place is NaN
    # and the others are zero
    x, w, cos, sin, pos = inputs(3, 2, D, R, 9, F32, 5)
    x[1, 1, D - 1] = INF
    got = binding.head_norm_rope(x, None, w, None, cos, sin, pos, EPS, interleaved).q
    assert (got[1, 1, :D - 1] == 0).all() and torch.isnan(got[1, 1, D - 1])
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1, 0]).all()
