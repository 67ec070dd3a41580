"""Choice of experts and its gradient against the float64 oracle.

Whole numbers have to be equal. With u = 2^-24, a float32 softmax probability of a logit x is off by at most
(|x - max| + 24) u of itself: the difference's rounding (which exp makes relative), an exponential and a
logarithm of at most 2 ulp each, a sum of E <= 256 terms in a tree of 20 levels, and a division. With logits within 40 of each
other that is below 64 u. Means add up to 64 terms in a row and 36 more levels (100 u). Gradients are sums of
products of such numbers: at most 256 u of the sum of their magnitudes; bfloat16 results add half a step
(2^-9 of a 9-bit significand, 2^-8 of the value).
"""
import numpy as np
import pytest
import torch

from oracle import route
from tests.gpu_helpers import f32, say

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24


def logits(t, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(t, E, generator=g) * spread).to(dtype)


def check(lib, x, top, keep=None, renorm=True, dev_x=None, dl=(0.7, 0.3)):
    """One forward and backward against the oracle; x on the CPU."""
    t, E = x.shape
    say(f"route t={t} E={E} top={top} {x.dtype} renorm={renorm}")
    xd = x.to(DEV) if dev_x is None else dev_x
    kd = None if keep is None else keep.to(DEV)
    r = lib.moe_route(xd, top, kd, renorm)
    ref = route.forward(f32(x), top, None if keep is None else keep.numpy(), renorm)
    for name in ("idx", "place", "source", "counts", "sizes"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), ref[name]), name
    fin = lambda a: np.where(np.isfinite(f32(a)), f32(a).astype(np.float64), 0)
    assert (np.abs(f32(r.gate) - ref["gate"]) <= 64 * U * ref["gate"] + 1e-38).all()
    assert (np.abs(f32(r.mean_p) - ref["mean_p"]) <= 164 * U * ref["mean_p"] + 1e-38).all()
    size = np.abs(fin(x)).max() + 6                       # of a logit and of lse
    assert abs(float(r.losses[0]) - ref["losses"][0]) <= 256 * U * ref["losses"][0]
    assert abs(float(r.losses[1]) - ref["losses"][1]) <= 256 * U * size ** 2
    g = torch.randn(t, top, generator=torch.Generator().manual_seed(9))
    dl = torch.tensor(dl) * t
    dx = lib.moe_route_bwd(g.to(DEV), dl.to(DEV), xd, r.idx, r.counts, r.sizes, renorm)
    want = route.backward(g.double().numpy(), dl.double().numpy(), f32(x), ref["idx"], renorm)
    assert dx.dtype is x.dtype
    n = max(1, ref["sizes"][0])
    mag = (np.abs(g.numpy()).max() + abs(float(dl[0])) * E * ref["counts"].max(initial=0) / max(1, ref["sizes"][1]) / n
           + 2 * abs(float(dl[1])) * size / n)
    half = 2.0 ** -8 if x.dtype is torch.bfloat16 else 0.0
    assert (np.abs(f32(dx) - want) <= half * np.abs(want) + 256 * U * 2 * mag).all()
    return r


@pytest.mark.parametrize("t", [1, 2, 16, 17, 63, 64, 65, 1000, 4096, 4097])
@pytest.mark.parametrize("E,top", [(1, 1), (8, 2), (60, 4), (128, 8), (256, 16)])
def test_route(lib, t, E, top):
    dtype = torch.bfloat16 if t % 2 else torch.float32            # bfloat16 brings ties
    check(lib, logits(t, E, dtype, t), top, renorm=(t + E) % 3 != 0)


@pytest.mark.parametrize("E,top", [(16, 16), (17, 3), (31, 1), (33, 6), (65, 12), (129, 2)])
def test_every_register_count(lib, E, top):
    check(lib, logits(70, E, torch.float32, E), top, renorm=False)
    check(lib, logits(70, E, torch.bfloat16, E), top)


def test_many_tokens(lib):
    """More tokens than the largest grid takes at once."""
    check(lib, logits(20001, 8, torch.float32, 3), 2, renorm=False)
    check(lib, logits(16500, 16, torch.bfloat16, 3), 16)            # all experts of every token, 80 tokens a block


@pytest.mark.parametrize("t", [5, 300])
def test_padding(lib, t):
    """Tokens that are not kept, NaN among their logits or not, count for nothing."""
    x = logits(t, 24, torch.float32, 1)
    keep = torch.rand(t, generator=torch.Generator().manual_seed(2)) < 0.6
    check(lib, x, 3, keep)
    hidden = x.clone()
    hidden[~keep] = float("nan")
    a, b = (lib.moe_route(y.to(DEV), 3, keep.to(DEV)) for y in (x, hidden))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    check(lib, x, 3, keep.to(torch.uint8) * 2, renorm=False)     # any value but 0
    r = check(lib, x, 3, torch.zeros(t, dtype=torch.bool))       # nothing is routed
    assert not r.counts.any() and not r.losses.any() and (r.source == -1).all()


def test_masked_experts(lib):
    """-inf is never chosen, and a token may have fewer choices than `top`, or none."""
    for t in (6, 200):
        x = logits(t, 10, torch.float32, 4)
        x[torch.rand(t, 10, generator=torch.Generator().manual_seed(5)) < 0.7] = -np.inf
        x[2] = -np.inf
        for renorm in (True, False):
            r = check(lib, x, 4, renorm=renorm)
            assert (r.idx[2] == -1).all() and not r.gate[2].any()


def test_lowest_values_and_ties(lib):
    low = torch.finfo(torch.float32).min
    x = torch.full((4, 20), low)
    x[1, 7] = 1.0
    x[2] = 0.0
    x[2, 3] = -0.0                         # equal to +0
    x[3, ::2] = 3.0
    r = lib.moe_route(x.to(DEV), 3)
    assert r.idx.tolist() == [[0, 1, 2], [7, 0, 1], [0, 1, 2], [0, 2, 4]]
    third = torch.full((3,), 1 / 3)
    assert torch.allclose(r.gate.cpu(), torch.stack((third, torch.tensor([1.0, 0, 0]), third, third)), rtol=4 * U, atol=0)
    dx = lib.moe_route_bwd(torch.ones(4, 3, device=DEV), None, x.to(DEV), r.idx, r.counts, r.sizes)
    assert dx.abs().max() <= 8 * U         # g (1 - sum g), the gates sum to 1 within 4 u


def test_nan_and_inf_stay_in_their_token(lib):
    """A token with NaN (or +inf) still has valid, different experts; its gates and gradient are NaN, the others'
    bits are not touched (its probabilities are in the mean, so the losses are NaN)."""
    for t in (9, 500):
        x = logits(t, 12, torch.float32, 6)
        ok = lib.moe_route(x.to(DEV), 4)
        bad = x.clone()
        bad[3, 5], bad[7, 0] = np.nan, np.inf
        r = lib.moe_route(bad.to(DEV), 4)
        rest = [i for i in range(t) if i not in (3, 7)]
        assert r.idx[3].tolist()[0] == 5 and sorted(set(r.idx[3].tolist())) == sorted(r.idx[3].tolist())
        assert r.gate[3].isnan().all() and r.gate[7].isnan().any() and r.losses.isnan().all()
        assert torch.equal(r.gate[rest], ok.gate[rest]) and torch.equal(r.idx[rest], ok.idx[rest])
        g = torch.ones(t, 4, device=DEV)
        a, b = (lib.moe_route_bwd(g, None, y.to(DEV), r.idx, r.counts, r.sizes) for y in (x, bad))
        assert torch.equal(a[rest], b[rest]) and b[3].isnan().all()


def test_strides_and_places(lib):
    """Logits inside a wider matrix (rows not 16-byte aligned), the gradient over the logits."""
    wide = logits(300, 77, torch.bfloat16, 7).to(DEV)
    inner = wide[:, 3:63]
    x = inner.cpu()
    r = check(lib, x, 5, dev_x=inner)
    g, dl = torch.randn(300, 5, device=DEV), torch.ones(2, device=DEV)
    want = lib.moe_route_bwd(g, dl, inner.contiguous(), r.idx, r.counts, r.sizes)
    edge = wide.clone()
    lib.moe_route_bwd(g, dl, inner, r.idx, r.counts, r.sizes, out=inner)
    assert torch.equal(inner, want)
    assert torch.equal(wide[:, :3], edge[:, :3]) and torch.equal(wide[:, 63:], edge[:, 63:])


def test_gradients_apart(lib):
    """Each gradient alone (the other None) and both add up; no tokens at all."""
    x = logits(100, 16, torch.float32, 8)
    r = lib.moe_route(x.to(DEV), 2)
    g, dl = torch.randn(100, 2), torch.tensor([3.0, -2.0])
    for dg, d in ((g, None), (None, dl), (None, None)):
        got = lib.moe_route_bwd(None if dg is None else dg.to(DEV), None if d is None else d.to(DEV), x.to(DEV), r.idx,
                                r.counts, r.sizes)
        want = route.backward(np.zeros((100, 2)) if dg is None else dg.numpy(), np.zeros(2) if d is None else d.numpy(),
                              x.numpy(), r.idx.cpu().numpy())
        assert (np.abs(f32(got) - want) <= 256 * U * 16).all()
    e = lib.moe_route(x[:0].to(DEV), 2)
    assert e.gate.shape == (0, 2) and not e.counts.any() and not e.sizes.any() and not e.losses.any()
    assert lib.moe_route_bwd(e.gate, None, x[:0].to(DEV), e.idx, e.counts, e.sizes).shape == (0, 16)


def test_by_differences(lib):
    """The gradient against differences of the forward in float64 arithmetic of its own outputs' oracle is
    pinned on the CPU; here the HIP forward itself: a step of 2^-6 in one logit moves the weighted outputs by the
    gradient times the step, up to a second-order term (below 2 * step^2 per unit) and float32 rounding."""
    x = logits(4, 8, torch.float32, 10)
    g, dl = torch.randn(4, 2, generator=torch.Generator().manual_seed(11)), torch.tensor([1.0, 0.1])
    f = lambda y: (lambda r: float((r.gate.cpu().double() * g).sum() + (r.losses.cpu().double() * dl).sum()))(
        lib.moe_route(y.to(DEV), 2))
    r = lib.moe_route(x.to(DEV), 2)
    dx = lib.moe_route_bwd(g.to(DEV), dl.to(DEV), x.to(DEV), r.idx, r.counts, r.sizes).cpu()
    h = 2.0 ** -6
    for i in range(4):
        for e in range(8):
            up, down = x.clone(), x.clone()
            up[i, e] += h
            down[i, e] -= h
            if any(not torch.equal(lib.moe_route(y.to(DEV), 2).idx, r.idx) for y in (up, down)):
                continue                   # a choice changes: no derivative there
            assert abs((f(up) - f(down)) / (2 * h) - float(dx[i, e])) <= 20 * h * h
