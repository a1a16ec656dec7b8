"""The polynomial that takes part of the tree kernels' exponentials (csrc/tree_attn.cu,
exp2_fma), in emulated fp32 with the coefficients of the source: each fused multiply-add is
exact in the 64 bits of a long double's fraction (48 of the product, and an addend of like
size) and rounded once."""
import os
import re

import numpy as np
import pytest

from block_sparse_long_10_b200 import build as qbuild

F, X = np.float32, np.longdouble
BOUND = 2.0 ** -22.4


@pytest.fixture(scope="module")
def exp2():
    assert np.finfo(X).nmant >= 63
    text = open(os.path.join(qbuild.CSRC, "tree_attn.cu")).read()
    body = text[text.index("void exp2_fma("):]
    body = body[:body.index("\n}\n")]
    horner = body[body.index("uint64_t p = fma2"):]
    c = [F(a) for a, b in re.findall(r"pair\(([0-9.]+)f, ([0-9.]+)f\)", horner) if a == b]
    assert len(c) == 6 and c[-1] == 1 and "SHIFT = 12582912.f" in body

    def run(x):
        x = np.maximum(x.astype(F), F(-127))
        t = x + F(12582912)
        f = (x.astype(X) - (t - F(12582912)).astype(X)).astype(F)
        p = np.full_like(f, c[0])
        for k in c[1:]:
            p = (p.astype(X) * f.astype(X) + X(k)).astype(F)
        return (p.view(np.uint32) + (t.view(np.uint32) << np.uint32(23))).view(F)

    return run


def _worst(exp2, x):
    return float(np.abs(exp2(x).astype(X) / np.exp2(x.astype(X)) - 1).max())


@pytest.mark.parametrize("sign", [1, -1])
def test_fractions(exp2, sign):
    """Every fifth fp32 number from 2^-12 to a half (below, the rounding of 1 + f alone)."""
    lo, hi = (int(F(v).view(np.uint32)) for v in (2.0 ** -12, 0.5))
    bits = np.arange(lo, hi + 1, 5, dtype=np.uint32)
    assert max(_worst(exp2, x.view(F) * F(sign)) for x in np.array_split(bits, 16)) <= BOUND
    tiny = F(sign) * F(2.0) ** np.arange(-149, -12).astype(F)
    assert _worst(exp2, tiny) <= BOUND


def test_the_whole_range(exp2):
    x = np.random.default_rng(1).uniform(-126, 8, 2000000).astype(F)
    assert _worst(exp2, x) <= BOUND
    whole = np.arange(-126, 9).astype(F)
    assert (exp2(whole) == np.exp2(whole)).all()


def test_from_the_smallest_exponent_down(exp2):
    x = np.linspace(-127, -126, 100001).astype(F)
    y = exp2(x)
    assert (y >= 0).all() and (y <= 2.0 ** -126).all()
    gone = np.array([-127, -127.5, -128, -1e4, -3e38, -np.inf], F)
    assert (exp2(gone) == 0).all()
