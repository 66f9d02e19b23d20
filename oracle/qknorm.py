"""Float64 oracle of the query / key norm with position rotation, and of its gradient.

x [..., H, d]; positions int [axes, ...]; pad rows are the caller's to blank.  Angles are
taken in float64, from positions and inverse frequencies, pair by pair."""
from __future__ import annotations

import numpy as np


def angles(positions, inv_freq, sections) -> np.ndarray:
    """[..., pairs]: pair p turns by positions[axis of p] * inv_freq[p]."""
    axis = np.repeat(np.arange(len(sections)), sections)
    assert axis.size == len(inv_freq)
    return np.moveaxis(np.asarray(positions, np.float64)[axis], 0, -1) * np.asarray(inv_freq, np.float64)


def rotate(x, ang, interleaved: bool, way: float = 1.0) -> np.ndarray:
    """x [..., H, d] with its first 2 * pairs values turned by ang [..., pairs] (way -1: back)."""
    out = np.array(x, np.float64)
    if ang is None:
        return out
    n = ang.shape[-1]
    c, s = np.cos(ang)[..., None, :], way * np.sin(ang)[..., None, :]
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    a, b = x[..., i], x[..., j]
    out[..., i] = a * c - b * s
    out[..., j] = a * s + b * c
    return out


def forward(x, w=None, eps=1e-6, ang=None, interleaved=False, norm=True) -> np.ndarray:
    x = np.asarray(x, np.float64)
    u = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else x
    return rotate(u if w is None else u * w, ang, interleaved)


def backward(x, dy, w=None, eps=1e-6, ang=None, interleaved=False, norm=True):
    """(dx, dw) of sum(dy * forward(x)); dw sums over all rows and heads."""
    x = np.asarray(x, np.float64)
    g = rotate(dy, ang, interleaved, -1.0)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else np.ones(x.shape[:-1] + (1,))
    u = x * r
    dw = (g * u).reshape(-1, x.shape[-1]).sum(0)
    h = g if w is None else g * w
    return (r * (h - u * np.mean(h * u, -1, keepdims=True)) if norm else h), dw
