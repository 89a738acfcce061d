"""fp64 oracle of the query/key norm with rotation — TEST INFRASTRUCTURE ONLY.

For one row x (d values), weight w, position p and frequencies f_i:
    y = R (w * x / sqrt(mean(x^2) + eps)),
R turning the pair (a, b) of frequency i to (a cos - b sin, b cos + a sin) with
the angle p f_i.  R is built as a d x d matrix per token, so that its transpose
gives the backward: g = R^T dy, dx = r (w g - xh mean(w g xh)), dw = sum g xh.
It shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .decay import _f64


def rotation(d, inv_freq, positions, interleaved=False):
    """[tokens..., d, d] matrices R with y = R x."""
    p = np.asarray(positions, dtype=np.float64)
    R = np.broadcast_to(np.eye(d), p.shape + (d, d)).copy()
    if inv_freq is None:
        return R
    f = _f64(inv_freq)
    half = f.shape[0]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(p * f[i]), np.sin(p * f[i])
        R[..., a, a], R[..., a, b], R[..., b, a], R[..., b, b] = c, -s, s, c
    return R


def forward(x, w, R, eps):
    """x [..., N, d] with R [N, d, d] (or a batch of them that broadcasts)."""
    x, w = _f64(x), _f64(w)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return np.matmul(R, y[..., None])[..., 0]


def backward(dy, x, w, R, eps):
    """(dx, dw)."""
    dy, x, w = _f64(dy), _f64(x), _f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    g = np.matmul(np.swapaxes(R, -1, -2), dy[..., None])[..., 0]
    dx = r * (w * g - xh * (w * g * xh).mean(-1, keepdims=True))
    return dx, (g * xh).reshape(-1, x.shape[-1]).sum(0)
