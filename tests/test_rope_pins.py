"""The rotary and per-head-norm oracle (oracle/rope.py) pinned by hand-derived values,
closed forms and differences, and qsa_rope_frequencies (host arithmetic) against it."""
import ctypes
import math

import numpy as np
import pytest

import block_sparse_long_10_b200 as qsa
from block_sparse_long_10_b200 import build as qbuild
from oracle import rope


@pytest.fixture(scope="module", autouse=True)
def lib():
    qbuild.build()
    return qsa.load()


def test_quarter_turn_by_hand():
    # one position of a pair with frequency pi/2: (a, b) -> (-b, a)
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0]).reshape(1, 1, 1, 5)
    f = [math.pi / 2, math.pi]
    half = rope.rope(x, [[1]], f, "half")[0, 0, 0]
    assert np.allclose(half, [-3, -2, 1, -4, 5])        # pairs (1,3), (2,4)
    inter = rope.rope(x, [[1]], f, "interleaved")[0, 0, 0]
    assert np.allclose(inter, [-2, 1, -3, -4, 5])       # pairs (1,2), (3,4)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_transpose_inverts_and_products_depend_on_distance(layout):
    g = np.random.default_rng(0)
    f, _ = rope.frequencies(1e4, 16)
    x, y = g.normal(size=(2, 1, 1, 1, 24))
    turn = lambda z, p: rope.rope(z, [[p]], f, layout)
    assert np.allclose(rope.rope(turn(x, 77), [[77]], f, layout, transpose=True), x)
    assert np.isclose((turn(x, 5) * turn(y, 2)).sum(), (turn(x, 105) * turn(y, 102)).sum())


def test_norm_by_hand():
    x = np.array([3.0, 4.0]).reshape(1, 1, 1, 2)  # mean square 12.5
    assert np.allclose(rope.norm(x, [1.0, 2.0], 0.0), [3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients_against_differences(layout):
    g = np.random.default_rng(1)
    x, dy = g.normal(size=(2, 1, 2, 2, 16))
    w, pos = g.normal(size=16), [[3, 40]]
    f, _ = rope.frequencies(100.0, 8)
    loss = lambda x, w: (rope.norm_rope(x, w, 1e-3, pos, f, layout, 1.2) * dy).sum()
    dx, dw = rope.norm_rope_grad(dy, x, w, 1e-3, pos, f, layout, 1.2)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for d in range(16):
        e = np.zeros(16)
        e[d] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-7


@pytest.mark.parametrize("rot", [2, 4, 32, 64, 128])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("by-parts", 8.0), ("by-parts", 1.0)])
def test_frequencies(rot, scaling, factor):
    if scaling == "ntk" and rot < 4:
        with pytest.raises(qsa.QSAError):
            qsa.qsa_rope_frequencies(1e4, rot, scaling, factor)
        return
    f, m = qsa.qsa_rope_frequencies(1e4, rot, scaling, factor, 4096.0)
    ref, mref = rope.frequencies(1e4, rot, scaling, factor, 4096.0)
    assert f.numel() == rot // 2 and f[0] == (0.25 if scaling == "linear" else 1.0)
    # a pow, an exp and a log of relative error 2^-52 each, arguments up to 10
    assert np.allclose(f.numpy(), ref, rtol=1e-14, atol=0)
    assert abs(m - mref) <= abs(mref) * 2 ** -24


def test_frequencies_ends():
    # NTK: the slowest pair is divided by the factor exactly, the fastest kept
    f, _ = qsa.qsa_rope_frequencies(1e4, 64, "ntk", 8.0)
    p, _ = qsa.qsa_rope_frequencies(1e4, 64)
    assert abs(float(p[-1] / f[-1]) - 8.0) < 1e-12 and f[0] == p[0]
    # by parts: pairs with many turns are kept, pairs with less than one are divided
    f, _ = qsa.qsa_rope_frequencies(1e4, 64, "by-parts", 8.0, 4096.0)
    turns = p * 4096.0 / (2 * math.pi)
    assert bool((f[turns > 64] == p[turns > 64]).all())
    assert np.allclose((p / f)[turns < 0.5].numpy(), 8.0, rtol=1e-14)


def test_frequencies_refusals(lib):
    out = (ctypes.c_double * 8)()
    call = lambda base=1e4, rot=16, sc=0, fac=1.0, ol=0.0, bf=32.0, bs=1.0, p=out: \
        lib.qsa_rope_frequencies(base, rot, sc, fac, ol, bf, bs, p, None)
    assert call() == 0
    for kw in (dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(rot=0),
               dict(rot=15), dict(rot=-2), dict(sc=4), dict(sc=-1), dict(fac=0.5),
               dict(fac=float("nan")), dict(sc=3, ol=0.0), dict(sc=3, ol=10.0, bf=0.5),
               dict(sc=3, ol=10.0, bs=0.0), dict(p=None)):
        assert call(**kw) == 1, kw
    with pytest.raises(ValueError):
        qsa.qsa_rope_frequencies(1e4, 16, "cubic")
