"""Host-side checks of the block norms' forms (no GPU needed): the 64-bit
gradients that the GPU tests compare with, by differences, for the plain
residual (no post norm, no gate) and for the norm alone; empty batches with a
shared gate; outputs that a call would not write."""

import numpy as np
import pytest

import i8_norm_reference as ref
from tiled_dense_gemm_07_amd import binding


@pytest.mark.parametrize("alpha", [1.0, 0.7])
@pytest.mark.parametrize("alone", [False, True], ids=["residual", "alone"])
def test_reference_gradients_by_differences(alone, alpha):
    """x' = alpha x + y, h = norm(x') w; and h = norm(x) w, where there is no
    block before, x' is x and alpha has no part."""
    r = np.random.Generator(np.random.PCG64(6))
    T, D, eps = 7, 10, 1e-6
    v = {"x": r.normal(size=(T, D)), "w_pre": r.normal(size=D)}
    if not alone:
        v["y"] = r.normal(size=(T, D))
    a, b = r.normal(size=(T, D)), r.normal(size=(T, D))

    def forward(v):
        return ref.forward(v["x"], v.get("y"), None, 0, None, v["w_pre"], alpha, eps, False)

    def loss(v):
        f = forward(v)
        return (a * f["x_out"]).sum() + (b * f["h"]).sum()

    f = forward(v)
    g = ref.backward(f["x_out"], a, b, v.get("y"), None, 0, None, v["w_pre"], None, f["r_pre"],
                     1.0 if alone else alpha, False)
    for k, name in (("x", "dx"), ("y", "dy"), ("w_pre", "dw_pre")):
        if k not in v:
            continue
        step, e = r.normal(size=v[k].shape), 1e-5
        d = (loss({**v, k: v[k] + e * step}) - loss({**v, k: v[k] - e * step})) / (2 * e)
        # the difference's own error: e^2 times third derivatives, and 2^-52 / e
        assert abs(d - (g[name] * step).sum()) <= 1e-6 * max(1.0, abs(d)), name


class FakeGate:
    """What the argument check asks of a gate on the GPU."""

    is_cuda, dtype = True, "bf16"

    def __init__(self, *shape):
        self.shape = shape

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


def test_shared_gate_of_no_tokens():
    for shape in ((16,), (1, 16)):
        for rows in (None, 0, 4):
            p, per = binding._gate_arg(FakeGate(*shape), rows, 0, 16, "bf16")
            assert p == 0x1000 and per >= 1
    p, per = binding._gate_arg(FakeGate(0, 16), None, 0, 16, "bf16")
    assert per == 1
    with pytest.raises(ValueError, match="gate must be"):
        binding._gate_arg(FakeGate(15), None, 0, 16, "bf16")


def test_buffers_that_a_call_would_not_write():
    """h without an output for it, and scales without levels, are refused: their
    old contents would stand in the result."""
    torch = pytest.importorskip("torch")
    x, s = torch.zeros(4, 16), torch.zeros(4)
    with pytest.raises(ValueError, match="h is not written"):
        binding.block_norm(x, y=x, out=None, h=x)
    for out in ("h", None):
        with pytest.raises(ValueError, match="hs is not written"):
            binding.block_norm(x, y=x, out=out, hs=s)
