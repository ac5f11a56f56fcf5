"""Norm, rotation by position, 4-bit storage and pages in fp64 (numpy), straight
from the definitions.

Test infrastructure only; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def pairs(R, interleaved):
    """Index pairs (a, b) that are rotated together."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, cos, sin, interleaved=False):
    """x [..., D] turned by angles with cos, sin [..., R / 2] (which broadcast)."""
    a, b = pairs(2 * cos.shape[-1], interleaved)
    y = np.array(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, w, cos, sin, eps, interleaved=False):
    """Rows x [..., D]; w [D] or None; cos, sin [..., R / 2] or None."""
    n = x if w is None else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return n if cos is None else rotate(n, cos, sin, interleaved)


def norm_rope_bwd(x, w, cos, sin, dy, eps, interleaved=False):
    """dx, dw (None without w), and bounds' absolute terms: of dx (its two terms),
    and of dw (the sum of absolute terms)."""
    g = dy if cos is None else rotate(dy, cos, -sin, interleaved)
    ag = np.abs(dy) if cos is None else rotate(np.abs(dy), np.abs(cos), np.zeros_like(sin), interleaved) \
        + np.abs(rotate(np.abs(dy), np.zeros_like(cos), np.abs(sin), interleaved) * rotated(x, cos, interleaved))
    if w is None:
        return g, None, ag, None
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, u = x * r, g * w
    dx = r * (u - xh * np.mean(u * xh, -1, keepdims=True))
    au = ag * np.abs(w)
    lead = tuple(range(x.ndim - 1))
    return (dx, np.sum(g * xh, lead), r * (au + np.abs(xh) * np.mean(au * np.abs(xh), -1, keepdims=True)),
            np.sum(ag * np.abs(xh), lead))


def rotated(x, cos, interleaved):
    """1 where a value of x is rotated, 0 elsewhere."""
    m = np.zeros(x.shape)
    for i in pairs(2 * cos.shape[-1], interleaved):
        m[..., i] = 1
    return m


def step_of(amax):
    """amax / 7 to 5 significant bits, half up."""
    m, e = np.frexp(amax / 7)
    return np.ldexp(np.floor(m * 32 + 0.5) / 32, e)


def quantise(x):
    """x [..., D] to codes [..., D] in [-7, 7] and steps [..., D / 32]."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    step = step_of(np.abs(g).max(-1))
    n = np.rint(g / np.where(step > 0, step, 1)[..., None]) * (step > 0)[..., None]
    return np.clip(n, -7, 7).reshape(x.shape), step


def values(codes, steps):
    """What bytes [..., D / 2] and steps [..., D / 32] stand for."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64) - 8
    return (n.reshape(*n.shape[:-1], -1, 32) * steps[..., None]).reshape(n.shape)
