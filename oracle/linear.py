"""Float64 oracle of linear attention with a decay per head: the recurrence token by token,
and its gradient by the reversed recurrence.  One sequence at a time, [n, H, d] arrays."""
from __future__ import annotations

import numpy as np


def decay(log_decay) -> np.ndarray:
    """exp of the logarithms, those above 0 taken as 0, [H, 1, 1]."""
    g = np.asarray(log_decay, np.float64)
    return np.exp(np.where(g > 0, 0.0, np.nan_to_num(g, nan=0.0, neginf=-np.inf)))[:, None, None]


def forward(q, k, v, log_decay, scale, state=None):
    """(o [n, H, d], final state [H, d, d])."""
    n, H, d = q.shape
    lam = decay(log_decay)
    s = np.zeros((H, d, d)) if state is None else np.array(state, np.float64)
    o = np.zeros((n, H, d))
    for t in range(n):
        s = lam * s + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.einsum("hi,hij->hj", q[t], s)
    return o, s


def backward(q, k, v, do, log_decay, scale, state=None, dstate=None):
    """(dq, dk, dv, gradient of the starting state) of sum(do * o) + sum(dstate * final)."""
    n, H, d = q.shape
    lam = decay(log_decay)
    states = np.zeros((n + 1, H, d, d))
    states[0] = 0.0 if state is None else state
    for t in range(n):
        states[t + 1] = lam * states[t] + k[t][:, :, None] * v[t][:, None, :]
    ds = np.zeros((H, d, d)) if dstate is None else np.array(dstate, np.float64)
    dq, dk, dv = (np.zeros((n, H, d)) for _ in range(3))
    for t in range(n - 1, -1, -1):
        ds = ds + scale * q[t][:, :, None] * do[t][:, None, :]
        dq[t] = scale * np.einsum("hij,hj->hi", states[t + 1], do[t])
        dk[t] = np.einsum("hij,hj->hi", ds, v[t])
        dv[t] = np.einsum("hij,hi->hj", ds, k[t])
        ds = lam * ds
    return dq, dk, dv, ds
