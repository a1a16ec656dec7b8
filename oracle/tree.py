"""Attention for a tree of drafted tokens, CPU oracle -- TEST INFRASTRUCTURE, NOT PART
OF THE PRODUCT PATH.

Plain numpy, fp64, one row and head at a time over an explicit list of cache rows, as
``include/qsa.h`` defines qsa_dense_tree_decode and qsa_sparse_tree_decode.  Only
``tests/`` may import it.
"""
from __future__ import annotations

import numpy as np


def tokens(P, i, parent, sel=None, r=4):
    """Cache rows that draft i attends to: the prefix (or its selected blocks and the tail
    after the last complete one) and the chain."""
    if sel is None:
        out = list(range(P))
    else:
        whole = P // r
        out = [r * j + k for j in sel if 0 <= j < whole for k in range(r)]
        out += list(range(whole * r, P))
    while i >= 0:
        out.append(P + i)
        i = int(parent[i])
    return out


def attend(q, k, v, rows, scale):
    """q [Hq,D], k/v [L,Hkv,D] -> o [Hq,D], lse [Hq], and what bounds their errors:
    sum p |v| [Hq,D] and the largest scale * sum |q k| of a row [Hq]."""
    Hq, D = q.shape
    G = Hq // k.shape[1]
    o, mass = np.zeros((Hq, D)), np.zeros((Hq, D))
    lse, size = np.full(Hq, -np.inf), np.zeros(Hq)
    if not rows:
        return o, lse, mass, size
    for h in range(Hq):
        kk, vv = k[rows, h // G], v[rows, h // G]
        x = kk @ q[h] * scale
        top = x.max()
        p = np.exp(x - top)
        lse[h] = top + np.log(p.sum())
        p /= p.sum()
        o[h], mass[h] = p @ vv, p @ np.abs(vv)
        size[h] = (np.abs(kk) @ np.abs(q[h])).max() * abs(scale)
    return o, lse, mass, size
