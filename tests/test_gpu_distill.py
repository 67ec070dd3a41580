"""Distillation from a teacher's top logits: the HIP path against the float64 oracle.

Tolerances, eps = 2^-24. x = (z - max) / tau is rounded three times and exp2 is good to a few units in
the last place, so an exponential is off by (4 + 3 |x|) eps of itself; the sum of v of them in a tree
whose longest run is 16 chunks of 8 and ten exchanges adds at most 160 eps (walked rows: v / 1024 + 40).
lse: 256 eps + 4 eps |lse|. loss: sum p (|log p| + |log q|) 16 eps + 256 eps + 4 eps |lse|. gradient:
w / tau of (q (300 + 4 |x|) eps + p 64 eps), |x| <= 100 here; plus half the last place in bf16, taken as 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import distill
from tests.gpu_helpers import f32, say
from tests.test_gpu_graph import _replay_check

pytestmark = pytest.mark.gpu

DEV, EPS = "cuda", 2.0 ** -24

CASES = [(1, 1, 1, 1.0), (3, 5, 3, 2.0), (2, 17, 16, 0.5), (5, 1000, 1, 1.0), (4, 4097, 33, 4.0), (3, 16384, 256, 2.0),
         (2, 16411, 64, 1.0), (2, 32003, 128, 2.0), (2, 65536, 7, 0.5), (2, 70001, 300, 2.0), (2, 140003, 1024, 1.0)]


def inputs(t, v, top, dt, seed=0):
    g = torch.Generator().manual_seed(seed + t + v + top)
    z = (torch.randn(t, v, generator=g) * 3).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    idx = torch.stack([torch.randperm(v, generator=g)[:top] if v >= top else torch.randint(0, v, (top,), generator=g)
                       for _ in range(t)]).to(torch.int32)
    teacher = torch.randn(t, top, generator=g) * 3
    w = torch.rand(t, generator=g) + 0.1
    return z, idx, teacher, w


def check(z, idx, teacher, w, tau, loss, lse, grad, skip=()):
    z64 = f32(z).astype(np.float64)
    rl, rs, rg = distill.rows(z64, idx.cpu().numpy(), f32(teacher), tau)
    t, v = z64.shape
    base = 256 + v / 1024
    rows = [i for i in range(t) if i not in skip]
    if lse is not None:
        assert (np.abs(f32(lse) - rs) <= EPS * (base + 4 * np.abs(rs)))[rows].all()
    if loss is not None:
        for i in rows:
            y = f32(teacher)[i].astype(np.float64) / tau
            ok = (idx[i].cpu().numpy() >= 0) & (idx[i].cpu().numpy() < v) & (y > -np.inf)
            size = 0.0
            if ok.any():
                lp = y[ok] - y[ok].max() - np.log(np.exp(y[ok] - y[ok].max()).sum())
                lq = z64[i][idx[i].cpu().numpy()[ok]] / tau - rs[i]
                used = np.exp(lp) > 0
                size = (np.exp(lp) * (np.abs(lp) + np.abs(lq)))[used].sum()
            assert abs(float(loss[i]) - rl[i]) <= EPS * (16 * size + base + 4 * abs(rs[i])), (i, float(loss[i]), rl[i])
    if grad is not None:
        wt = f32(w).astype(np.float64)[:, None]
        ref = rg * wt
        q = np.exp(z64 / tau - rs[:, None]) * wt / tau
        p = np.abs(ref - q)
        tol = EPS * (q * (base + 500) + 64 * p) + (2.0 ** -8 * np.abs(ref) if grad.dtype == torch.bfloat16 else 0)
        assert (np.abs(f32(grad) - ref) <= tol + 2.0 ** -126)[rows].all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,v,top,tau", CASES)
def test_parity(lib, t, v, top, tau, dt):
    say(f"distill t={t} v={v} top={top} tau={tau} {dt}")
    z, idx, teacher, w = (x.to(DEV) for x in inputs(t, v, top, dt))
    loss, lse = lib.distill_topk_fwd(z, idx, teacher, tau)
    check(z, idx, teacher, w, tau, loss, lse, lib.distill_topk_bwd(w, z, idx, teacher, tau, lse))
    loss2, grad = lib.distill_topk_step(z, idx, teacher, tau, w)
    assert torch.equal(loss, loss2)
    check(z, idx, teacher, w, tau, None, None, grad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("v", [37, 20001, 150001])
def test_entries_that_are_not_there(lib, v, dt):
    """Indices outside the vocabulary, teacher logits of -inf, repeated indices, rows without entries,
    rows of weight 0 that hold NaN, masked logits (-inf and the type's lowest value)."""
    z, idx, teacher, w = inputs(8, v, 12, dt)
    idx[0, 3], idx[0, 4], idx[0, 5] = -1, v, 2 ** 31 - 1
    teacher[1, ::2] = float("-inf")
    idx[2] = idx[2, 0]
    idx[3] = -1
    teacher[4] = float("-inf")
    z[5], w[5] = float("nan"), 0.0
    low = torch.finfo(z.dtype).min
    for i in (6, 7):
        keep = torch.zeros(v, dtype=torch.bool)
        keep[idx[i].long()] = True
        z[i][~keep] = float("-inf") if i == 6 else low
    z, idx, teacher, w = (x.to(DEV) for x in (z, idx, teacher, w))
    loss, grad = lib.distill_topk_step(z, idx, teacher, 2.0, w)
    assert not loss[3:6].any() and not grad[3:6].any()
    check(z, idx, teacher, w, 2.0, loss, None, grad, skip=(5,))
    fwd, lse = lib.distill_topk_fwd(z, idx, teacher, 2.0)
    back = lib.distill_topk_bwd(w, z, idx, teacher, 2.0, lse)
    check(z, idx, teacher, w, 2.0, fwd, lse, back, skip=(5,))
    assert not back[5].any()


@pytest.mark.parametrize("v", [999, 40001, 140001])
def test_strides_in_place_and_weights(lib, v):
    """Rows at odd addresses and strides, gradients laid out otherwise than the logits, in place, no
    weights."""
    t, top = 5, 20
    z, idx, teacher, w = (x.to(DEV) for x in inputs(t, v, top, "bf16"))
    want_l, want = lib.distill_topk_step(z, idx, teacher, 2.0, w)
    wide = torch.full((t, v + 7), 5.0, dtype=z.dtype, device=DEV)
    for at in (0, 1, 3):
        view = wide[:, at:at + v]
        view.copy_(z)
        loss, grad = lib.distill_topk_step(view, idx, teacher, 2.0, w)
        assert torch.allclose(loss, want_l, rtol=1e-5, atol=1e-5)       # the sum's order follows the alignment
        check(z, idx, teacher, w, 2.0, loss, None, grad)
        out = torch.full((t, v + 3), 9.0, dtype=z.dtype, device=DEV)
        _, got = lib.distill_topk_step(view, idx, teacher, 2.0, w, out=out[:, 2:2 + v])
        assert torch.equal(got, grad) and (out[:, :2] == 9).all() and (out[:, 2 + v:] == 9).all()
        lib.distill_topk_step(view, idx, teacher, 2.0, w, out=view)
        assert torch.equal(view, grad)
        wide.fill_(5.0)
    _, one = lib.distill_topk_step(z, idx, teacher, 2.0)
    _, ones = lib.distill_topk_step(z, idx, teacher, 2.0, torch.ones(t, device=DEV))
    assert torch.equal(one, ones)


def test_no_rows_autograd_and_graph(lib):
    z, idx, teacher, w = (x.to(DEV) for x in inputs(6, 5001, 9, "f32"))
    loss, lse = lib.distill_topk_fwd(z[:0], idx[:0], teacher[:0], 1.0)
    assert loss.shape == (0,) and lib.distill_topk_step(z[:0], idx[:0], teacher[:0], 1.0)[1].shape == (0, 5001)

    def step():
        loss, lse = lib.distill_topk_fwd(z, idx, teacher, 2.0)
        return (loss, lse, lib.distill_topk_bwd(w, z, idx, teacher, 2.0, lse)) + tuple(
            lib.distill_topk_step(z, idx, teacher, 2.0, w))

    _replay_check(step)
    x = z.clone().requires_grad_()
    (lib.DistillTopKFunction.apply(x, idx, teacher, 2.0) * w).sum().backward()
    assert torch.equal(x.grad, step()[2])
