"""Host-side checks (no kernel launched) of head norms whose queries and keys lie between
each other: the same strides, other places."""

import ctypes
import os

import pytest

from tiled_dense_gemm_07_amd import binding

OK, NULLP, SHAPE, DTYPE, EPI, ALIAS, NOCFG, HIP = range(8)
BF16, ES = 2, 2
BASE, TABLES = 1 << 30, 1 << 40
T, H, D = 8, 4, 64


@pytest.fixture(autouse=True)
def no_launch():
    """Every launch fails, after all checks of its arguments."""
    old = os.environ.get("TG_FAULT")
    os.environ["TG_FAULT"] = "launch"
    yield
    if old is None:
        del os.environ["TG_FAULT"]
    else:
        os.environ["TG_FAULT"] = old


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def at(place):
    """Address of value `place` of one buffer."""
    return BASE + ES * place


def fill(a, heads, T=T, Hq=H, Hk=H, D=D, **more):
    d = dict(T=T, Hq=Hq, Hk=Hk, D=D, R=D, dtype=BF16, w_q=TABLES, w_k=TABLES + 4096, cos=TABLES + 8192,
             sin=TABLES + (1 << 16), P=100, positions=None, eps=1e-6, interleaved=0)
    for n, (place, t, h) in heads.items():
        d.update({n: at(place), n + "_t": t, n + "_h": h})
    d.update(more)
    for k, v in d.items():
        setattr(a, k, v)
    return a


def forward(lib, q, k, q_out, k_out, **kw):
    a = fill(binding.HeadNormRopeArgs(), dict(q=q, k=k, q_out=q_out, k_out=k_out), **kw)
    return lib.tg_head_norm_rope(ctypes.byref(a), None)


def backward(lib, q, k, dq_out, dk_out, dq, dk):
    a = fill(binding.HeadNormRopeGradArgs(), dict(q=q, k=k, dq_out=dq_out, dk_out=dk_out, dq=dq, dk=dk))
    return lib.tg_head_norm_rope_backward(ctypes.byref(a), None, 0, None)


FAR = 1 << 24  # another buffer


def test_heads_of_queries_and_keys_in_turn(lib):
    # [T][H][2][D]: a query's head, then a key's
    t, h = 2 * H * D, 2 * D
    q, k = (0, t, h), (D, t, h)
    assert forward(lib, q, k, q, k) == HIP  # in place
    assert forward(lib, q, k, (FAR, t, h), (FAR + D, t, h)) == HIP
    assert forward(lib, q, k, q, (D - 1, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + D + 1, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + D - 1, t, h)) == ALIAS
    # over the keys, or a head or a token further
    assert forward(lib, q, k, k, (FAR, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + h, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + t, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + T * t, t, h)) == HIP
    assert forward(lib, q, k, (FAR, t, h), (FAR + T * t - h, t, h)) == ALIAS
    # [T][H][3][D], values behind the keys; fewer keys than queries
    t, h = 3 * H * D, 3 * D
    q, k = (0, t, h), (D, t, h)
    assert forward(lib, q, k, q, k) == HIP
    assert forward(lib, q, k, q, k, Hk=1) == HIP
    assert forward(lib, q, (3 * D, t, h), q, (FAR, t, h), Hk=1) == ALIAS
    # one token: its stride says nothing
    assert forward(lib, (0, 5, h), (D, 7, h), (0, 5, h), (D, 7, h), T=1) == HIP
    assert forward(lib, (0, 5, h), (D, 7, h), (0, 5, h), (D - 1, 7, h), T=1) == ALIAS


def test_tokens_of_queries_and_keys_in_turn(lib):
    # [H][T][2][D]
    t, h = 2 * D, 2 * T * D
    q, k = (0, t, h), (D, t, h)
    assert forward(lib, q, k, q, k) == HIP
    assert forward(lib, q, k, q, (D + 1, t, h)) == ALIAS
    assert forward(lib, q, k, (FAR, t, h), (FAR + D, t, h)) == HIP
    assert forward(lib, q, k, (FAR, t, h), (FAR + t, t, h)) == ALIAS


def test_gradients_between_each_other(lib):
    t, h = 2 * H * D, 2 * D
    q, k, gq, gk = (0, t, h), (D, t, h), (FAR, t, h), (FAR + D, t, h)
    oq, ok = (2 * FAR, t, h), (2 * FAR + D, t, h)
    assert backward(lib, q, k, gq, gk, oq, ok) == HIP
    assert backward(lib, q, k, gq, gk, oq, (2 * FAR + D - 1, t, h)) == ALIAS
    # between the inputs' heads, too
    t3, h3 = 3 * H * D, 3 * D
    q, k, gq, gk = (0, t3, h3), (FAR, t3, h3), (3 * FAR, t, h), (3 * FAR + D, t, h)
    assert backward(lib, q, k, gq, gk, (D, t3, h3), (FAR + D, t3, h3)) == HIP
    assert backward(lib, q, k, gq, gk, (D, t3, h3), (2 * D, t3, h3)) == HIP
    assert backward(lib, q, k, gq, gk, (D, t3, h3), (2 * D + 1, t3, h3)) == ALIAS
    assert backward(lib, q, k, gq, gk, q, ok) == ALIAS  # no in-place form


def test_every_small_arrangement(lib):
    # against the sets of values themselves
    T, H, D = 3, 2, 4
    values = lambda p, t, h, n: {p + i * t + j * h + e for i in range(T) for j in range(n)
                                 for e in range(D)}
    far = (1 << 24, 64, 16)
    for t, h in ((24, 8), (16, 8), (25, 9), (8, 24), (5, 20), (4, 12)):
        a = values(0, t, h, H)
        for n in (1, H):
            for p in range(-60, 61):
                want = HIP if a.isdisjoint(values(p, t, h, n)) else ALIAS
                got = forward(lib, far, (2 << 24, 64, 16), (0, t, h), (p, t, h), T=T, Hq=H, Hk=n, D=D,
                              R=0, cos=None, sin=None)
                assert got == want, (t, h, n, p)
