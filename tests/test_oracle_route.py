"""The float64 oracles of expert routing and of 8-bit activations, pinned on the CPU: gradients against central
differences (off by below 1e-8 at step 1e-5, taken as 1e-6), closed forms, and bounds of the 8-bit codes."""
import numpy as np
import pytest
import torch

from oracle import act8, route
from tests.test_oracle_operators import differences, near


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_by_differences(renorm):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 5))
    x[2, 3] = -np.inf                       # an expert that cannot be chosen
    keep = np.array([1, 1, 1, 0, 1, 1])
    dg, dl = rng.standard_normal((6, 3)), np.array([0.7, 0.3])
    f0 = route.forward(x, 3, keep, renorm)

    def f():                                # no choice changes within the steps, so the counts are constant
        o = route.forward(x, 3, keep, renorm)
        assert (o["idx"] == f0["idx"]).all()
        return (o["gate"] * dg).sum() + (o["losses"] * dl).sum()

    got = route.backward(dg, dl, x, f0["idx"], renorm)
    finite = np.isfinite(x)
    ref = np.zeros_like(x)
    for i in zip(*np.nonzero(finite)):
        at = x[i]
        x[i] = at + 1e-5
        up = f()
        x[i] = at - 1e-5
        ref[i] = (up - f()) / 2e-5
        x[i] = at
    near(got, ref)
    assert not got[3].any() and got[2, 3] == 0


def test_route_closed_forms():
    o = route.forward(np.zeros((4, 8)), 2)          # ties: the lowest experts; even probabilities
    assert (o["idx"] == [0, 1]).all() and np.allclose(o["gate"], 0.5) and np.allclose(o["mean_p"], 1 / 8)
    assert np.allclose(o["losses"], [1.0, np.log(8) ** 2])
    assert (o["place"] == [[0, 4], [1, 5], [2, 6], [3, 7]]).all() and (o["source"] == [0, 1, 2, 3] * 2).all()
    one = np.full((3, 4), -np.inf)
    one[:, 2] = [1.0, -1.0, 5.0]                    # one expert takes all: balance E, gate 1, lse its logit
    o = route.forward(one, 2)
    assert (o["idx"] == [2, -1]).all() and np.allclose(o["losses"], [4.0, 9.0]) and (o["sizes"] == [3, 3]).all()
    o = route.forward(one, 2, keep=[0, 0, 0])
    assert (o["sizes"] == 0).all() and (o["source"] == -1).all() and not o["losses"].any()


def test_route_places_are_a_stable_sort():
    rng = np.random.default_rng(1)
    o = route.forward(rng.standard_normal((50, 7)), 3, rng.random(50) < 0.8)
    flat = o["idx"].reshape(-1)
    order = np.argsort(np.where(flat < 0, 7, flat), kind="stable")[:(flat >= 0).sum()]
    assert (o["place"].reshape(-1)[order] == np.arange(order.size)).all()
    assert (o["source"][:order.size] == order // 3).all() and (o["source"][order.size:] == -1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_act8_bounds(dtype):
    """Every value is within half a step (a / 254) of its code's, up to the roundings of the scale and of the
    product (2^-24 a each), and the largest of a block has the code 127."""
    x = (torch.randn(40, 200, generator=torch.Generator().manual_seed(2)) * 3).to(dtype).float().numpy()
    codes, scale = act8.pack(x)
    v = act8.value(codes, scale, 200)
    b = np.pad(x, ((0, 0), (0, 56))).reshape(40, 4, 64)
    a = np.abs(b).max(2)
    assert (np.abs(codes.reshape(40, 4, 64)).max(2) == 127).all()
    err = np.abs(np.pad(v - x, ((0, 0), (0, 56))).reshape(40, 4, 64)).max(2)
    assert (err <= a / 254 + a * 2.0 ** -23).all()


def test_act8_borders():
    x = np.zeros((7, 64), np.float32)
    x[0, :3] = [2.0, 1.0, -1.0]                     # 63.5: to the even 64
    x[1, :4] = [254.0, 1.0, 3.0, 5.0]               # 0.5, 1.5, 2.5: to 0, 2, 2
    x[2, :2] = [np.inf, 1.0]
    x[3, :2] = [np.nan, 1.0]
    x[4, 0] = 2.0 ** -120
    x[5, :2] = [2.0 ** -119, -2.0 ** -120]
    codes, scale = act8.pack(x)
    assert codes[0, :3].tolist() == [127, 64, -64] and codes[1, :4].tolist() == [127, 0, 2, 2]
    assert np.isnan(scale[2:4]).all() and not codes[2:5].any() and scale[4, 0] == 0 and scale[6, 0] == 0
    assert codes[5, :2].tolist() == [127, -64]
