"""fp64 reference of rotary positions with an optional norm per head, and of its
gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring). The plain definition over
NumPy arrays [B, H, N, d]:

    u = x                                  or  x (mean(x^2) + eps)^(-1/2) weight
    (y_a, y_b) = amplitude (u_a cos t - u_b sin t, u_b cos t + u_a sin t)
    t = positions[b, n] freqs[j], (a, b) = (j, j + r / 2) or (2j, 2j + 1)
"""

from __future__ import annotations

import numpy as np

__all__ = ["pairs", "turn", "rotary", "rotary_backward"]


def pairs(r, interleaved):
    """Elements a and b of the r / 2 pairs."""
    j = np.arange(r // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)


def turn(u, freqs, positions, interleaved, amplitude, back=False):
    a, b = pairs(2 * len(freqs), interleaved)
    t = (positions[:, :, None].astype(np.float64) * freqs)[:, None]
    c, s = amplitude * np.cos(t), amplitude * np.sin(t)
    if back:
        s = -s
    y = u.copy()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    return y


def rotary(x, freqs, positions, interleaved=False, weight=None, eps=1e-6, amplitude=1.0):
    u = x
    if weight is not None:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    return turn(u, freqs, positions, interleaved, amplitude)


def rotary_backward(dy, x, freqs, positions, interleaved=False, weight=None, eps=1e-6, amplitude=1.0):
    """(dx, dweight or None)."""
    g = turn(dy, freqs, positions, interleaved, amplitude, back=True)
    if weight is None:
        return g, None
    n = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dweight = (g * x * n).sum((0, 1, 2))
    wg = weight * g
    return n * (wg - x * n * (wg * x * n).mean(-1, keepdims=True)), dweight
