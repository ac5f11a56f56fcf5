"""Attention and layer norm in fp64 (numpy), straight from the definitions.

Test infrastructure only; shares no code with the CUDA path.  One sequence and
one head at a time.  The attention gradients also return, per output, the sum
of the absolute values of their terms, from which tests derive how far the
rounding of a factor can move the result.
"""
from __future__ import annotations

import numpy as np


def visible(lq, lk):
    """[lq, lk]: query i sees the keys j <= i + lk - lq."""
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)


def _softmax(q, k, scale, see):
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = np.max(s, axis=1, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
    e = np.where(see, e, 0.0)
    l = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m + np.log(np.where(l > 0, l, 1.0)), -np.inf)
    return e / np.where(l > 0, l, 1.0)[:, None], lse


def attn_fwd(q, k, v, scale, see=None):
    """One head of one sequence: q [lq, D], k, v [lk, D].  Returns o, lse and
    a = sum_j p_ij |v_j|."""
    see = visible(len(q), len(k)) if see is None else see
    p, lse = _softmax(q, k, scale, see)
    return p @ v, lse, p @ np.abs(v)


def attn_bwd(q, k, v, do, scale, see=None):
    """Gradients (dq, dk, dv) of one head, and a dict of absolute sums:
    dq, dk, dv (of their terms); pk = scale sum_j p_ij |k_j| and, for dk,
    pq(d)[j] = scale sum_i p_ij |q_i| d_i; cq and ck, the sums of dq and dk with
    p_ij sum_c |do_ic v_jc| in the place of ds_ij."""
    see = visible(len(q), len(k)) if see is None else see
    p, _ = _softmax(q, k, scale, see)
    o = p @ v
    ds = p * (do @ v.T - np.sum(do * o, axis=1, keepdims=True))
    c = p * (np.abs(do) @ np.abs(v).T)
    ab = {"cq": scale * c @ np.abs(k), "ck": scale * c.T @ np.abs(q),
          "dq": scale * np.abs(ds) @ np.abs(k), "dk": scale * np.abs(ds).T @ np.abs(q),
          "dv": p.T @ np.abs(do), "pk": scale * p @ np.abs(k),
          "pq": lambda d: scale * p.T @ (np.abs(q) * d[:, None])}
    return scale * ds @ k, scale * ds.T @ q, p.T @ do, ab


def layer_norm_fwd(x, w, b, eps):
    """Rows x [n, D]: returns y, mean, rstd."""
    mean = x.sum(1) / x.shape[1]
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).sum(1) / x.shape[1] + eps)
    y = (x - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_bwd(x, w, dy, eps):
    """Returns dx, dw, db."""
    _, mean, rstd = layer_norm_fwd(x, w, None, eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
