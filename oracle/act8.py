"""Activations in 8 bits -- test infrastructure (see the package docstring).

Blocks of 64 along a row (the last may be short), a = max |x|: code = 127 x / a to the nearest integer, ties to
even; scale = fl32(a / 127), at most the largest float32 whose 127-fold is finite. The float64 quotient decides every float32 case: a quotient of 24-bit numbers
(times 127) that is not a half-integer is further than 2^-34 of itself from one, and a half-integer is
represented exactly.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
TOP = np.nextafter(np.finfo(np.float32).max / np.float32(127), np.float32(0))


def pack(x):
    """(codes int8 [m, kp], scale float32 [m, kp / 64]) of a float32 array [m, k]."""
    x = np.asarray(x, np.float32)
    m, k = x.shape
    b = np.pad(x, ((0, 0), (0, -k % BLOCK))).reshape(m, -1, BLOCK)
    bad = ~np.isfinite(b).all(2)
    a = np.where(bad, 0, np.abs(np.nan_to_num(b, posinf=0, neginf=0)).max(2)).astype(np.float32)
    a = np.where(a < 2.0 ** -119, np.float32(0), a)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(127.0 * b.astype(np.float64) / a.astype(np.float64)[..., None])
    codes = np.where((a > 0)[..., None], q, 0).astype(np.int8)
    scale = np.where(bad, np.float32(np.nan), np.minimum(a / np.float32(127), TOP)).astype(np.float32)
    return codes.reshape(m, -1), scale


def value(codes, scale, k):
    """What they stand for, float32 [m, k]."""
    m = codes.shape[0]
    return (codes.reshape(m, -1, BLOCK).astype(np.float32) * scale[..., None]).reshape(m, -1)[:, :k]
