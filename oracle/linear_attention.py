"""Causal linear attention with a decay for each head — test infrastructure only.

By the recurrence, token by token, per (batch, head), d = exp(log_decay[h]):
    S_t = d S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t.
The gradients follow the recurrence backwards; with G_t the gradient of S_t,
    G_t = scale q_t do_t^T + d G_{t+1},
    dq_t = scale S_t do_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_0 = d G_1.
All arithmetic float64; tensors [B, S, H, D], states [B, H, D, D] (row = feature of k).
"""
from __future__ import annotations

import numpy as np


def _decay(log_decay):
    with np.errstate(divide="ignore"):
        return np.exp(np.asarray(log_decay, np.float64))[None, :, None, None]


def forward(q, k, v, log_decay, scale, state=None):
    """(o, state after the last token)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, S, H, D = q.shape
    s = np.zeros((B, H, D, D)) if state is None else np.asarray(state, np.float64).copy()
    d = _decay(log_decay)
    o = np.empty_like(v)
    for t in range(S):
        s = d * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhk,bhkv->bhv", q[:, t], s)
    return o, s


def backward(q, k, v, log_decay, scale, do, state=None, dstate=None):
    """(dq, dk, dv, gradient of the first state); dstate: gradient of the last one."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    B, S, H, D = q.shape
    d = _decay(log_decay)
    s = np.zeros((B, H, D, D)) if state is None else np.asarray(state, np.float64).copy()
    dq, dk, dv = np.empty_like(q), np.empty_like(k), np.empty_like(v)
    for t in range(S):
        s = d * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", s, do[:, t])
    g = np.zeros((B, H, D, D)) if dstate is None else np.asarray(dstate, np.float64).copy()
    for t in reversed(range(S)):
        g = g + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = np.einsum("bhkv,bhv->bhk", g, v[:, t])
        dv[:, t] = np.einsum("bhkv,bhk->bhv", g, k[:, t])
        g = d * g
    return dq, dk, dv, g


def magnitudes(q, k, v, log_decay, scale, state=None):
    """Sums of absolute terms of (o, last state): what rounding errors are relative to."""
    return forward(*(np.abs(np.asarray(x, np.float64)) for x in (q, k, v)), log_decay, scale,
                   None if state is None else np.abs(state))


def magnitudes_backward(q, k, v, log_decay, scale, do, state=None, dstate=None):
    """The same of the gradients."""
    return backward(*(np.abs(np.asarray(x, np.float64)) for x in (q, k, v)), log_decay, scale, np.abs(do),
                    None if state is None else np.abs(state), None if dstate is None else np.abs(dstate))
