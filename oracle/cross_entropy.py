"""fp64 reference of the label cross entropy over a fused projection.

TEST INFRASTRUCTURE ONLY -- see the package docstring.

  a = W h / T, log q = a - logsumexp(a), e = label smoothing, lam = z-loss
  l_r  = -(1 - e) log q_y - (e / V) sum_v log q_v + lam LSE_r^2
  loss = (1/D) sum over kept rows of w_r l_r, D = kept rows ("mean") or 1 ("sum")
  G_r  = k_r (q (1 + 2 lam LSE_r) - (1 - e) 1_y - e / V),  dH_r = G_r W / T,
  dW   = sum_r G_r^T h_r / T,  k_r = w_r / D, or the given row gradient.
Rows whose label is ignore_index, or outside [0, V), are left out; no kept row
gives loss 0 and zero gradients.
"""
from __future__ import annotations

import numpy as np

from .kl import log_softmax, widen_bf16

__all__ = ["cross_entropy"]


def cross_entropy(hidden, W, labels, row_weight=None, T=1.0, label_smoothing=0.0, z_loss=0.0,
                  ignore_index=-100, reduction="mean", row_grad=None):
    """Dict with loss, row_loss [N], lse [N], dH [N, H], dW [V, H], and the
    magnitudes |G| |W| / T and |G|^T |h| / T (dH_abs, dW_abs) that bound what a
    relative rounding of G's entries can change, and the same with the positive
    part k q (1 + 2 lam LSE) in G's place (dH_q, dW_q), for relative errors of
    q ahead of the subtraction.  ``row_grad`` replaces the rows' factors w_r / D
    in the gradients."""
    h = widen_bf16(hidden) if np.asarray(hidden).dtype == np.uint16 else np.asarray(hidden, np.float64)
    W = widen_bf16(W) if np.asarray(W).dtype == np.uint16 else np.asarray(W, np.float64)
    labels = np.asarray(labels, np.int64)
    N, V = h.shape[0], W.shape[0]
    keep = np.nonzero((labels != ignore_index) & (labels >= 0) & (labels < V))[0]
    w = np.ones(N) if row_weight is None else np.asarray(row_weight, np.float64)
    row_loss, lse = np.zeros(N), np.zeros(N)
    dH, dH_abs = np.zeros(h.shape), np.zeros(h.shape)
    dW, dW_abs = np.zeros(W.shape), np.zeros(W.shape)
    dH_q, dW_q = np.zeros(h.shape), np.zeros(W.shape)
    out = dict(loss=0.0, row_loss=row_loss, lse=lse, dH=dH, dW=dW, dH_abs=dH_abs, dW_abs=dW_abs,
               dH_q=dH_q, dW_q=dW_q)
    if keep.size == 0:
        return out
    D = float(keep.size) if reduction == "mean" else 1.0
    hk, y = h[keep], labels[keep]
    a = hk @ W.T / T
    logq = log_softmax(a)
    lse[keep] = (a - logq)[:, 0]
    at = (np.arange(keep.size), y)
    row_loss[keep] = (-(1 - label_smoothing) * logq[at] - label_smoothing * logq.mean(axis=1)
                      + z_loss * lse[keep] ** 2)
    out["loss"] = float((w[keep] * row_loss[keep]).sum() / D)
    k = (w / D if row_grad is None else np.asarray(row_grad, np.float64))[keep][:, None]
    Q = np.exp(logq) * (1 + 2 * z_loss * lse[keep])[:, None]
    G = Q - label_smoothing / V
    G[at] -= 1 - label_smoothing
    G *= k / T
    dH[keep] = G @ W
    dW += G.T @ hk
    dH_abs[keep] = np.abs(G) @ np.abs(W)
    dW_abs += np.abs(G).T @ np.abs(hk)
    Q = np.abs(Q * (k / T))
    dH_q[keep] = Q @ np.abs(W)
    dW_q += Q.T @ np.abs(hk)
    return out
