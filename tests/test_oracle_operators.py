"""The float64 oracles of the operators beside the layer, pinned on the CPU: gradients against central
differences, and against the single layer, closed forms and torch.

Central differences with step h in float64 are off by h^2 |f'''| / 6 + 2^-52 |f| / h; with h = 1e-5 and
functions and third derivatives of order 1 to 100 that is below 1e-8, taken as 1e-6 relative to the
largest gradient.
"""
import numpy as np
import pytest
import torch

from oracle import distill, headnorm, multi, qlora

H, TOL = 1e-5, 1e-6


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        at = x[i]
        x[i] = at + H
        up = f()
        x[i] = at - H
        g[i] = (up - f()) / (2 * H)
        x[i] = at
    return g


def near(got, ref):
    assert np.abs(got - ref).max() <= TOL * max(1.0, np.abs(ref).max())


def test_multi_is_the_single_layer_for_each_adapter():
    rng = np.random.default_rng(0)
    X, W, A, B = (rng.standard_normal(s) for s in ((9, 6), (5, 6), (3, 2, 6), (3, 5, 2)))
    s, ids, dY = np.array([0.5, 2.0, 1.0]), np.array([2, 0, -1, 0, 7, 2, 2, 0, -3]), rng.standard_normal((9, 5))
    Y, T = multi.forward(X, W, A, B, s, ids)
    dX, dA, dB = multi.backward(dY, X, W, A, B, s, ids)
    for a in range(3):
        rows = ids == a
        y, t = qlora.forward(X[rows], W, A[a], B[a], s[a])
        dx, da, db = qlora.backward(dY[rows], X[rows], W, A[a], B[a], s[a])
        for got, ref in ((Y[rows], y), (T[rows], t), (dX[rows], dx), (dA[a], da), (dB[a], db)):
            assert np.allclose(got, ref, rtol=1e-12, atol=1e-12)
    none = (ids < 0) | (ids >= 3)
    assert np.allclose(Y[none], X[none] @ W.T) and not T[none].any() and np.allclose(dX[none], dY[none] @ W)
    assert not dA[1].any() and not dB[1].any()          # no rows


def test_multi_gradient_by_differences():
    rng = np.random.default_rng(1)
    X, W, A, B = (rng.standard_normal(s) for s in ((5, 4), (3, 4), (2, 2, 4), (2, 3, 2)))
    s, ids, dY = np.array([0.5, 2.0]), np.array([1, 0, -1, 1, 0]), rng.standard_normal((5, 3))
    f = lambda: (multi.forward(X, W, A, B, s, ids)[0] * dY).sum()
    for got, x in zip(multi.backward(dY, X, W, A, B, s, ids), (X, A, B)):
        near(got, differences(f, x))


@pytest.mark.parametrize("d,rot,interleaved", [(8, 8, False), (8, 4, True), (10, 6, False), (6, 0, False), (2, 2, True)])
def test_head_norm_gradient_by_differences(d, rot, interleaved):
    rng = np.random.default_rng(2)
    x, w, g = rng.standard_normal((3, 2, d)), rng.standard_normal(d), rng.standard_normal((3, 2, d))
    ang = rng.uniform(-3, 3, (5, rot // 2))
    args = (np.cos(ang), np.sin(ang), np.array([4, 0, 2]), rot, 1e-3, interleaved, 0.5)
    f = lambda: (headnorm.forward(x, w, *args) * g).sum()
    for got, at in zip(headnorm.backward(g, x, w, *args), (x, w)):
        near(got, differences(f, at))


def test_head_norm_closed_forms():
    """Rotation keeps the length of each pair; a rotation by pi / 2 swaps it; equal elements of size c
    have norm 1 at eps 0."""
    x = np.full((1, 1, 4), 3.0)
    one = headnorm.forward(x, np.ones(4), np.zeros((1, 2)), np.ones((1, 2)), np.array([0]), 4, 0.0)
    assert np.allclose(one, [[[-1, -1, 1, 1]]])
    inter = headnorm.forward(x, np.array([1.0, 2, 3, 4]), np.zeros((1, 2)), np.ones((1, 2)), np.array([0]), 4, 0.0, True)
    assert np.allclose(inter, [[[-2, 1, -4, 3]]])


def test_distill_gradient_by_differences():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((4, 7))
    idx = np.array([[1, 5, 2], [0, 0, 6], [3, -1, 9], [-1, -1, 7]])       # repeated, padded, empty
    teacher = rng.standard_normal((4, 3))
    teacher[0, 1] = -np.inf
    f = lambda: distill.rows(z, idx, teacher, 1.7)[0].sum()
    near(distill.rows(z, idx, teacher, 1.7)[2], differences(f, z))


def test_distill_is_the_divergence_of_torch():
    """With every logit kept the loss is torch's divergence of the two softmaxes; it is 0 for equal
    logits, and the gradient of a row sums to 0."""
    rng = np.random.default_rng(4)
    z, y = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    idx = np.stack([rng.permutation(6) for _ in range(3)])
    loss, lse, grad = distill.rows(z, idx, np.take_along_axis(y, idx, 1), 2.0)
    zt, yt = torch.tensor(z) / 2, torch.tensor(y) / 2
    ref = torch.nn.functional.kl_div(zt.log_softmax(1), yt.log_softmax(1), log_target=True, reduction="none").sum(1)
    assert np.allclose(loss, ref.numpy()) and np.allclose(lse, zt.logsumexp(1).numpy())
    assert np.abs(grad.sum(1)).max() < 1e-14
    assert np.abs(distill.rows(z, idx, np.take_along_axis(z, idx, 1), 2.0)[0]).max() < 1e-14
