"""Distillation from a teacher's top logits in float64 -- test infrastructure (see the package
docstring).

Row by row, entry by entry: z = logits / tau, p = softmax of the teacher's kept logits / tau,
loss = sum_j p_j (log p_j - log softmax(z)[idx_j]) and its gradient (softmax(z) - sum of p_j at each
index) / tau. An entry outside [0, v) or of teacher logit -inf is left out; a row without entries
has loss 0 and gradient 0.
"""
from __future__ import annotations

import numpy as np


def rows(logits, idx, teacher, tau):
    """(loss [t], lse [t], gradient [t, v])."""
    logits, teacher = np.asarray(logits, np.float64), np.asarray(teacher, np.float64)
    t, v = logits.shape
    loss, lse, grad = np.zeros(t), np.zeros(t), np.zeros((t, v))
    for i in range(t):
        z = logits[i] / tau
        m = z.max()
        with np.errstate(invalid="ignore"):
            lse[i] = m + np.log(np.exp(z - m).sum())
        keep = [(j, y / tau) for j, y in zip(idx[i], teacher[i]) if 0 <= j < v and y != -np.inf]
        if not keep:
            continue
        y = np.array([b for _, b in keep])
        log_p = y - (y.max() + np.log(np.exp(y - y.max()).sum()))
        grad[i] = np.exp(z - lse[i]) / tau
        for (j, _), lp in zip(keep, log_p):
            if np.exp(lp) > 0:
                loss[i] += np.exp(lp) * (lp - (z[j] - lse[i]))
            grad[i, j] -= np.exp(lp) / tau
    return loss, lse, grad
