"""Choice of experts, token by token in float64 -- test infrastructure (see the package docstring).

For the logits x of a routed token: its choices are the `top` largest x, ties to the lower index, -inf
never; its gates are softmax(x) there, or the softmax over the choices alone. Over the n routed tokens and
their N choices: counts, places in (expert, token) order, balance = E sum (counts_e / N) mean_p_e and
z = mean (log sum exp x)^2. The gradient takes the counts as constants.
"""
from __future__ import annotations

import numpy as np


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def choose(x, top):
    """The experts of one token, best first."""
    order = sorted((e for e in range(len(x)) if x[e] > -np.inf), key=lambda e: (-x[e], e))
    return order[:top]


def forward(logits, top, keep=None, renormalize=True):
    """idx, gate [t, top]; place [t, top]; source [t top]; counts [E]; sizes (n, N); mean_p [E]; losses [2]."""
    x = np.asarray(logits, np.float64)
    t, E = x.shape
    idx, gate = np.full((t, top), -1), np.zeros((t, top))
    mean_p, z, n = np.zeros(E), 0.0, 0
    for i in range(t):
        mine = choose(x[i], top) if keep is None or keep[i] else []
        if not mine:
            continue
        p = softmax(x[i])
        g = softmax(x[i][mine]) if renormalize else p[mine]
        idx[i, :len(mine)], gate[i, :len(mine)] = mine, g
        mean_p += p
        z += (x[i].max() + np.log(np.exp(x[i] - x[i].max()).sum())) ** 2
        n += 1
    counts = np.array([(idx == e).sum() for e in range(E)])
    place, source = np.full((t, top), -1), np.full(t * top, -1)
    at = 0
    for e in range(E):
        for i, j in zip(*np.nonzero(idx == e)):
            place[i, j], source[at] = at, i
            at += 1
    if n:
        mean_p, z = mean_p / n, z / n
    balance = E * (mean_p * counts).sum() / at if at else 0.0
    return dict(idx=idx, gate=gate, place=place, source=source, counts=counts, sizes=np.array([n, at]), mean_p=mean_p,
                losses=np.array([balance, z]))


def backward(dgate, dlosses, logits, idx, renormalize=True):
    """dlogits, with the counts of idx."""
    x = np.asarray(logits, np.float64)
    t, E = x.shape
    counts = np.array([(idx == e).sum() for e in range(E)])
    n, dx = int((idx >= 0).any(1).sum()), np.zeros_like(x)
    for i in range(t):
        mine = [(j, e) for j, e in enumerate(idx[i]) if e >= 0]
        if not mine:
            continue
        j, e = (np.array(v) for v in zip(*mine))
        p = softmax(x[i])
        jac = lambda q: np.diag(q) - np.outer(q, q)         # of a softmax
        dx[i] += jac(p) @ (dlosses[0] * E * counts / (counts.sum() * n))
        dx[i] += dlosses[1] * 2 * (x[i].max() + np.log(np.exp(x[i] - x[i].max()).sum())) * p / n
        if renormalize:
            dx[i][e] += jac(softmax(x[i][e])) @ dgate[i][j]
        else:
            dx[i] += jac(p)[:, e] @ dgate[i][j]
    return dx


def combine(Z, place, gate=None, base=None):
    """base + sum_j gate_j Z[place_j], rows without a place left out."""
    Z, (t, top) = np.asarray(Z, np.float64), place.shape
    y = np.zeros((t, Z.shape[1])) if base is None else np.array(base, np.float64)
    for i in range(t):
        for j in range(top):
            if place[i, j] >= 0:
                y[i] += (1.0 if gate is None else float(gate[i, j])) * Z[place[i, j]]
    return y
