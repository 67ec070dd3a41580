"""Tokens into expert order and back against the float64 oracle.

gather moves values: equal. combine rounds each of top + 1 sums (u = 2^-24 of the sum of magnitudes each) and the
result once (half a step). dZ is one product, rounded to float32 and once more. dgate is a sum of d products: at
most d / 64 + 16 in a row on a lane or over lanes, u each of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import route
from tests.gpu_helpers import f32, say

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def routing(t, E, top, seed, pad=0.2):
    x = np.random.default_rng(seed).standard_normal((t, E))
    keep = np.random.default_rng(seed + 1).random(t) >= pad
    o = route.forward(x, top, keep)
    i32 = lambda a: torch.from_numpy(a.astype(np.int32)).to(DEV)
    return o, i32(o["place"]), i32(o["source"])


def rows(n, d, dtype, seed):
    return torch.randn(n, d, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check(lib, t, d, E, top, dtype, pad=0.2, shift=0):
    """shift: elements by which the token-side matrices are off their alignment, in wider rows."""
    say(f"rows t={t} d={d} E={E} top={top} {dtype} shift={shift}")
    o, place, source = routing(t, E, top, t + d, pad)
    wide = lambda x: torch.nn.functional.pad(x, (shift, shift)).to(DEV)[:, shift:shift + x.shape[1]] if shift else x.to(DEV)
    X, base, dY = (rows(t, d, dtype, s) for s in (1, 2, 3))
    Z = rows(t * top, d, dtype, 4)
    Z[int(o["sizes"][1]):] = float("nan")                # rows behind the last are not read
    gate = torch.rand(t, top, generator=torch.Generator().manual_seed(5))
    Zd, gd = Z.to(DEV), gate.to(DEV)
    G = lib.moe_gather(wide(X), place, source)
    want = np.where(o["source"][:, None] >= 0, f32(X)[o["source"]], 0)
    assert np.array_equal(f32(G), want)
    half, Zn = HALF[dtype], np.nan_to_num(f32(Z))
    for g, b in ((gate, base), (gate, None), (None, None)):
        Y = lib.moe_combine(Zd, place, None if g is None else gd, None if b is None else wide(b))
        gn, bn = None if g is None else g.numpy(), None if b is None else f32(b)
        want = route.combine(Zn, o["place"], gn, bn)
        mag = route.combine(np.abs(Zn), o["place"], gn, None if b is None else np.abs(bn))
        assert (np.abs(f32(Y) - want) <= half * np.abs(want) + (top + 2) * U * mag).all()
    dZ, dgate = lib.moe_combine_bwd(wide(dY), Zd, place, source, gd)
    dZ, dgate, y = f32(dZ), f32(dgate), f32(dY).astype(np.float64)
    at, live = o["place"], o["place"] >= 0
    tok, _ = np.nonzero(live)
    want = np.zeros((t * top, d))
    want[at[live]] = gate.numpy()[live][:, None] * y[tok]
    assert (np.abs(dZ - want) <= (half + U) * np.abs(want)).all()
    z = Zn[np.where(live, at, 0)].astype(np.float64)
    want, mag = (np.where(live, (p[:, None] * q).sum(2), 0) for p, q in ((y, z), (np.abs(y), np.abs(z))))
    assert (np.abs(dgate - want) <= (d / 64 + 16) * U * mag).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,d,E,top", [(1, 4096, 8, 2), (1, 1, 2, 1), (3, 8, 4, 4), (17, 257, 8, 5), (64, 1000, 60, 6),
                                       (300, 2048, 8, 1), (33, 5120, 128, 16), (2000, 72, 8, 3), (5, 7, 3, 2)])
def test_rows(lib, dtype, t, d, E, top):
    check(lib, t, d, E, top, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [512, 515])
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_rows(lib, dtype, d, shift):
    check(lib, 40, d, 8, 2, dtype, shift=shift)


def test_many_rows(lib):
    """Enough rows for four chunks a lane."""
    check(lib, 5000, 264, 8, 2, torch.bfloat16)
    check(lib, 5000, 263, 8, 2, torch.bfloat16)


def test_no_padding_and_all_padding(lib):
    check(lib, 50, 128, 8, 2, torch.bfloat16, pad=0.0)
    check(lib, 50, 128, 8, 2, torch.bfloat16, pad=1.1)


def test_places_outside_the_rows(lib):
    """Places and tokens outside their ranges are none: nothing is read or written there."""
    t, top, d = 6, 2, 64
    place = torch.tensor([[0, 12], [-5, 1], [2, 2 ** 31 - 1], [3, -2 ** 31], [4, 5], [6, 99]], dtype=torch.int32, device=DEV)
    source = torch.tensor([0, 1, 2, 3, 4, 4, 5, 6, -1, 2 ** 31 - 1, -7, 100], dtype=torch.int32, device=DEV)
    X, Z = rows(t, d, torch.float32, 1).to(DEV), rows(t * top, d, torch.float32, 2).to(DEV)
    G = lib.moe_gather(X, place, source)
    assert torch.equal(G[:7], X[source[:7].long()]) and not G[7:].any()
    live = (place >= 0) & (place < 12)
    Y = lib.moe_combine(Z, place)
    want = (Z[place.clamp(0, 11).long()] * live[..., None]).sum(1)
    assert torch.allclose(Y, want, rtol=0, atol=4 * U * 8)
    dZ, dgate = lib.moe_combine_bwd(X, Z, place, source, torch.ones(t, top, device=DEV))
    assert torch.equal(dZ[:7], X[source[:7].long()]) and not dZ[7:].any() and not dgate[~live].any()


def test_more_choices_than_lanes(lib):
    """The rows' calls take any number of choices: 70 for each of 5 tokens, in any order of rows."""
    t, top, d = 5, 70, 40
    perm = torch.randperm(t * top, generator=torch.Generator().manual_seed(1))
    place = perm.to(torch.int32).view(t, top)
    source = torch.empty(t * top, dtype=torch.int32)
    source[perm] = torch.arange(t, dtype=torch.int32).repeat_interleave(top)
    X, Z = rows(t, d, torch.float32, 1), rows(t * top, d, torch.float32, 2)
    gate = torch.rand(t, top, generator=torch.Generator().manual_seed(3))
    dev = [z.to(DEV) for z in (X, Z, place, source, gate)]
    assert torch.equal(lib.moe_gather(dev[0], dev[2], dev[3]).cpu(), X[source.long()])
    want, mag = (route.combine(f(Z.numpy()), place.numpy(), gate.numpy()) for f in (np.asarray, np.abs))
    assert (np.abs(f32(lib.moe_combine(dev[1], dev[2], dev[4])) - want) <= 80 * U * mag).all()
    dZ, dg = lib.moe_combine_bwd(dev[0], dev[1], dev[2], dev[3], dev[4])
    flat = torch.empty(t * top)
    flat[perm] = gate.reshape(-1)
    assert torch.equal(dZ.cpu(), flat[:, None] * X[source.long()])
    z = Z[perm].view(t, top, d).double()
    assert (dg.cpu().double() - (X.double()[:, None] * z).sum(2)).abs().max() <= 64 * U * d


def test_in_place(lib):
    """Y over base, and both directions at once on one buffer where the header allows it."""
    o, place, source = routing(100, 8, 2, 1, 0.1)
    for d in (256, 255):
        Z, base = rows(200, d, torch.bfloat16, 1).to(DEV), rows(100, d, torch.bfloat16, 2).to(DEV)
        gate = torch.rand(100, 2, device=DEV)
        want = lib.moe_combine(Z, place, gate, base)
        assert lib.moe_combine(Z, place, gate, base, out=base) is base and torch.equal(base, want)
        dY = rows(100, d, torch.bfloat16, 3).to(DEV)
        dZ, dg = lib.moe_combine_bwd(dY, Z, place, source, gate)
        c, dg2, raw = lib.library(), torch.empty_like(dg), torch.cuda.current_stream().cuda_stream
        assert c.moe_combine_bwd(dY.data_ptr(), 0, 100, d, d, Z.data_ptr(), place.data_ptr(), source.data_ptr(), 2,
                                 gate.data_ptr(), Z.data_ptr(), dg2.data_ptr(), raw) == 0      # dZ over Z
        assert torch.equal(Z, dZ) and torch.equal(dg, dg2)


def test_offsets_past_32_bits(lib):
    """More than 2^32 elements of grouped rows."""
    t, top, d = 70000, 8, 8192
    place = torch.arange(t * top, dtype=torch.int32, device=DEV).view(top, t).t().contiguous()
    source = torch.arange(t, dtype=torch.int32, device=DEV).repeat(top)
    X = torch.randn(t, d, device=DEV, dtype=torch.bfloat16)
    G = lib.moe_gather(X, place, source)
    assert all(torch.equal(G[j * t:(j + 1) * t], X) for j in range(top))
    gate = torch.zeros(t, top, device=DEV)
    gate[:, 7] = 1.0
    assert torch.equal(lib.moe_combine(G, place, gate), X)
    dZ, dgate = lib.moe_combine_bwd(X, G, place, source, gate)
    assert torch.equal(dZ[7 * t:], X) and not dZ[:7 * t].any()
    assert all(torch.equal(dgate[:, j], dgate[:, 0]) for j in range(top))


def test_no_tokens(lib):
    place, source = torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    X = torch.empty(0, 32, device=DEV)
    assert lib.moe_gather(X, place, source).shape == (0, 32) and lib.moe_combine(X, place).shape == (0, 32)
    dZ, dg = lib.moe_combine_bwd(X, X, place, source, torch.empty(0, 2, device=DEV))
    assert dZ.shape == (0, 32) and dg.shape == (0, 2)
