"""fp64 reference of the norms around a block (see the package docstring).

  u = block rho(block) w1 (post), v = x + s g u, y = v rho(v) w2 (pre)
  rho(z) = 1 / sqrt(mean(z^2) + eps) over a row; offset is added to w1 and w2.
"""
from __future__ import annotations

import numpy as np

__all__ = ["block_norm", "block_norm_grads"]


def _rho(z, eps):
    return 1.0 / np.sqrt((z * z).mean(axis=1, keepdims=True) + eps)


def block_norm(x, block=None, w1=None, g=None, w2=None, scale=1.0, post=True, pre=True, eps=1e-6,
               offset=0.0):
    """(v, y); y is None without ``pre``."""
    v = np.asarray(x, np.float64)
    if block is not None:
        u = np.asarray(block, np.float64)
        if post:
            u = u * _rho(u, eps) * (1.0 if w1 is None else np.asarray(w1, np.float64) + offset)
        v = v + scale * (1.0 if g is None else np.asarray(g, np.float64)) * u
    y = None
    if pre:
        y = v * _rho(v, eps) * (1.0 if w2 is None else np.asarray(w2, np.float64) + offset)
    return v, y


def block_norm_grads(x, block, dy, dv, w1=None, g=None, w2=None, scale=1.0, post=True, pre=True,
                     eps=1e-6, offset=0.0):
    """dict of dx, dblock, dw1, dg, dw2 for the upstream gradients dy (of y) and
    dv (of v; None = zeros)."""
    H = np.asarray(x).shape[1]
    one = np.ones(H)
    a1 = one if w1 is None else np.asarray(w1, np.float64) + offset
    a2 = one if w2 is None else np.asarray(w2, np.float64) + offset
    ag = one if g is None else np.asarray(g, np.float64)
    v, _ = block_norm(x, block, w1, g, w2, scale, post, pre, eps, offset)
    out = {}
    dvv = np.zeros_like(v) if dv is None else np.asarray(dv, np.float64)
    if pre:
        dy = np.asarray(dy, np.float64)
        r = _rho(v, eps)
        t = dy * a2
        dvv = dvv + r * t - v * r ** 3 * (v * t).mean(axis=1, keepdims=True)
        out["dw2"] = (dy * v * r).sum(axis=0)
    out["dx"] = dvv
    if block is not None:
        b = np.asarray(block, np.float64)
        r = _rho(b, eps) if post else 1.0
        u = b * r * a1 if post else b
        out["dg"] = (scale * dvv * u).sum(axis=0)
        du = scale * ag * dvv
        if post:
            out["dw1"] = (du * b * r).sum(axis=0)
            t = du * a1
            out["dblock"] = r * t - b * r ** 3 * (b * t).mean(axis=1, keepdims=True)
        else:
            out["dblock"] = du
    return out
