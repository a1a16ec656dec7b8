"""Rotary positions and per-head norms, CPU oracle -- TEST INFRASTRUCTURE, NOT PART OF
THE PRODUCT PATH.

Plain numpy, fp64, from the definitions in ``include/qsa.h``: frequencies, the
rotation and its transpose, the norm with the rotation, and its gradients from the
Jacobian written out (not from the kernels' formulas).  Only ``tests/`` may import it.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(base, rot, scaling="none", factor=1.0, orig_len=0.0, beta_fast=32.0,
                beta_slow=1.0):
    """Radians per position of pair i < rot / 2, one pair at a time; and mscale."""
    out = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "linear":
            f = f / factor
        elif scaling == "ntk":
            f = math.exp(-2.0 * i / rot * (math.log(base) + rot / (rot - 2) * math.log(factor)))
        elif scaling == "by-parts":
            pair = lambda beta: rot * math.log(orig_len / (2 * math.pi * beta)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
            slow = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = slow * f / factor + (1 - slow) * f
        out.append(f)
    return np.array(out), 0.1 * math.log(factor) + 1.0 if scaling == "by-parts" else 1.0


def pairs(rot, layout):
    """Index arrays (a, b) of the dims that form pair i."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rope(x, pos, freq, layout="half", mscale=1.0, transpose=False):
    """x [B,T,H,D], pos [B,T] -> the rotated heads."""
    x = np.asarray(x, np.float64)
    freq = np.asarray(freq, np.float64)
    a, b = pairs(2 * len(freq), layout)
    angle = np.asarray(pos, np.float64)[..., None, None] * freq
    c, s = np.cos(angle) * mscale, np.sin(angle) * mscale * (-1 if transpose else 1)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def norm_rope(x, weight, eps, pos, freq, layout="half", mscale=1.0):
    return rope(norm(x, weight, eps), pos, freq, layout, mscale)


def norm_rope_grad(dy, x, weight, eps, pos, freq, layout="half", mscale=1.0):
    """(dx, dweight): dx through the Jacobian d xhat_i / d x_j = (delta_ij - xhat_i xhat_j
    / D) / size of the norm, size = sqrt(mean x^2 + eps)."""
    x = np.asarray(x, np.float64)
    dz = rope(dy, pos, freq, layout, mscale, transpose=True)
    if weight is None:
        return dz, None
    w = np.asarray(weight, np.float64)
    D = x.shape[-1]
    size = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x / size
    jac = (np.eye(D) - xh[..., :, None] * xh[..., None, :] / D) / size[..., None]
    return ((dz * w)[..., None, :] @ jac)[..., 0, :], (dz * xh).sum((0, 1, 2))
