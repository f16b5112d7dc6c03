"""Host-side checks (no kernel launched): calls with nothing to write, and heads that lie
between each other's values."""

import ctypes
import os

import pytest

from tiled_dense_gemm_07_amd import binding

OK, NULLP, SHAPE, DTYPE, EPI, ALIAS, NOCFG, HIP = range(8)
P = [0x10000000 * (i + 1) for i in range(20)]
BF16 = 2


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


@pytest.fixture
def no_launch():
    """Every launch fails, after all checks of its arguments."""
    old = os.environ.get("TG_FAULT")
    os.environ["TG_FAULT"] = "launch"
    yield
    if old is None:
        del os.environ["TG_FAULT"]
    else:
        os.environ["TG_FAULT"] = old


def grad(lib, **kw):
    a = binding.LinearMxGradArgs()
    d = dict(M=40, N=48, K=56, dtype=BF16, wtype=BF16, fmt=0, dY=P[0], lddy=48, X=P[1], ldx=56,
             W=P[2], ldw=56, dX=P[3], lddx=56, dW=P[4], lddw=56, dbias=P[5])
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return lib.tg_linear_mx_backward(ctypes.byref(a), P[6], 1 << 20, None)


def test_gradients_that_are_all_empty(lib, no_launch):
    # an empty tensor has no address: a call that asks for such outputs alone is no mistake
    none = dict(dX=None, dW=None, dbias=None)
    assert grad(lib, M=0, dY=None, X=None, **none) == OK             # dX alone, no tokens
    assert grad(lib, M=0, dY=None, X=None, W=None, **none) == OK
    assert grad(lib, K=0, X=None, W=None, lddx=0, lddw=0, **none) == OK  # dX or dW alone, K 0
    assert grad(lib, N=0, dY=None, W=None, **none) == OK             # dW alone, no outputs
    assert grad(lib, M=0, N=0, K=0, dY=None, X=None, W=None, **none) == OK
    # no output where each of the three would have elements
    assert grad(lib, **none) == NULLP
    # outputs that are not empty are still written
    assert grad(lib, M=0, dY=None, X=None, dX=None) == HIP
    assert grad(lib, K=0, X=None, W=None, dX=None, dW=None) == HIP
