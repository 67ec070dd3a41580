"""The QLoRA layer with an adapter of its own for every row, in float64 -- test infrastructure (see
the package docstring).

Row i goes through the layer of the adapter a = ids[i] of the stacked A [L, r, K], B [L, N, r] with
the scale s[a]; a row whose id lies outside [0, L) goes through the frozen base alone. One row at a
time:

    T_i = A_a X_i,   Y_i = deq(W) X_i + s_a B_a T_i
    U_i = B_a^T dY_i,   dX_i = deq(W)^T dY_i + s_a A_a^T U_i,   dA_a += s_a U_i X_i^T,   dB_a += s_a dY_i T_i^T
"""
from __future__ import annotations

import numpy as np

from . import qlora

_f64 = qlora._f64


def forward(X, Wd, A, B, s, ids):
    X, Wd, A, B, s = (_f64(t) for t in (X, Wd, A, B, s))
    Y = X @ Wd.T
    T = np.zeros((X.shape[0], A.shape[1]))
    for i, a in enumerate(np.asarray(ids)):
        if 0 <= a < A.shape[0]:
            T[i] = A[a] @ X[i]
            Y[i] += s[a] * (B[a] @ T[i])
    return Y, T


def backward(dY, X, Wd, A, B, s, ids):
    dY, X, Wd, A, B, s = (_f64(t) for t in (dY, X, Wd, A, B, s))
    dX = dY @ Wd
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for i, a in enumerate(np.asarray(ids)):
        if 0 <= a < A.shape[0]:
            T, U = A[a] @ X[i], B[a].T @ dY[i]
            dX[i] += s[a] * (A[a].T @ U)
            dA[a] += s[a] * np.outer(U, X[i])
            dB[a] += s[a] * np.outer(dY[i], T)
    return dX, dA, dB
