"""Float64 oracle of what stands beside the sLSTM in a block: layer norm and linear attention with
a decay for each head, each from its definition (step by step, no chunks), with the gradients'
formulas. Plain numpy; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


# ---- layer norm ---------------------------------------------------------------------------------
def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(x, g, mean, rstd, weight=None):
    """(dx, dweight, dbias) for the gradient g of y."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    xh = (x - mean[..., None]) * rstd[..., None]
    gw = g if weight is None else g * weight
    dx = rstd[..., None] * (gw - gw.mean(-1, keepdims=True) - xh * (gw * xh).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (g * xh).sum(axes), g.sum(axes)


# ---- linear attention ---------------------------------------------------------------------------
def linear_attention(q, k, v, log_decay, state0=None, scale=1.0):
    """(o (T, dv), states (T + 1, dk, dv)) of one sequence and head: S_t = e^{g_t} S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t; states[0] = state0. log_decay (T)."""
    T, dk = q.shape
    S = np.zeros((T + 1, dk, v.shape[1]))
    if state0 is not None:
        S[0] = state0
    o = np.zeros((T, v.shape[1]))
    for t in range(T):
        S[t + 1] = np.exp(log_decay[t]) * S[t] + np.outer(k[t], v[t])
        o[t] = scale * (S[t + 1].T @ q[t])
    return o, S


def linear_attention_backward(q, k, v, log_decay, g_out, state0=None, g_final=None, scale=1.0):
    """(dq, dk, dv, dlog_decay, dstate0) of one sequence and head, by the adjoint of the recurrence."""
    _, S = linear_attention(q, k, v, log_decay, state0, scale)
    T = q.shape[0]
    L = np.zeros(S.shape[1:]) if g_final is None else np.array(g_final, np.float64)
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(T)
    for t in range(T - 1, -1, -1):
        L = L + scale * np.outer(q[t], g_out[t])  # the gradient of S_{t+1}, the state after step t
        dq[t] = scale * (S[t + 1] @ g_out[t])
        dk[t] = L @ v[t]
        dv[t] = L.T @ k[t]
        a = np.exp(log_decay[t])
        dg[t] = a * np.sum(L * S[t])
        L = a * L
    return dq, dk, dv, dg, L

