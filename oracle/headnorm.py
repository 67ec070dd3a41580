"""Norm and rotation of query and key heads in float64 -- test infrastructure (see the package
docstring).

    xh = x / sqrt(mean(x^2) + eps),   n = xh * (w + offset),   y = R(pos) n

over the last axis of x [tokens, heads, d]; R turns the pairs (i, i + rot/2), or (2i, 2i + 1), of the
first rot elements by the angles of the token's row of the tables. The backward is the chain rule
written out: R's transpose, the weight, then the projection of the norm.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(n, cos, sin, pos, rot, interleaved, sign=1.0):
    a, b = pairs(rot, interleaved)
    y = n.copy()
    if rot:
        c, s = _f64(cos)[pos][:, None, :], sign * _f64(sin)[pos][:, None, :]
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., a] * s + n[..., b] * c
    return y


def forward(x, w, cos, sin, pos, rot, eps, interleaved=False, offset=0.0):
    x, w = _f64(x), _f64(w) + offset
    inv = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return rotate(x * inv * w, cos, sin, pos, rot, interleaved)


def backward(g, x, w, cos, sin, pos, rot, eps, interleaved=False, offset=0.0):
    """(dx, dw)."""
    g, x, w = _f64(g), _f64(x), _f64(w) + offset
    inv = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xh = x * inv
    gn = rotate(g, cos, sin, pos, rot, interleaved, -1.0)
    gh = gn * w
    return inv * (gh - xh * (gh * xh).mean(-1, keepdims=True)), (gn * xh).sum((0, 1))
