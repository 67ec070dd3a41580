"""Norm and rotation of query and key heads: the HIP path against the float64 oracle.

Tolerances. eps = 2^-24 is the float32 unit roundoff. An output is a cos -+ b sin of two normalised
elements, each the product of x, the inverse root and the weight: about 8 roundings and the sum of d
squares (at most d/lanes + 6 additions in a row, halved by the root), so the error is below 32 eps of
the pair's size, (|a| + |b|); a bf16 output adds half its last place, 2^-9 of it, taken as 2^-8. The
input gradient subtracts two terms of at most the size of max|gh|: below 64 eps of inv max|gh|. dw is a
sum of n terms added in order over a thread's, a workgroup's and all parts: the error is below
(n / parts + 100) eps, taken as 256 eps, of the sum of the terms' sizes.
"""
import numpy as np
import pytest
import torch

from oracle import headnorm
from tests.gpu_helpers import f32, say
from tests.test_gpu_graph import _replay_check

pytestmark = pytest.mark.gpu

DEV, EPS = "cuda", 2.0 ** -24

CASES = [  # m, heads q, heads k, d, rot, interleaved, dtype, weight dtype, positions
    (1, 1, 0, 2, 2, False, "f32", "f32", "i32"), (1, 32, 8, 128, 128, False, "bf16", "bf16", "i64"),
    (3, 5, 1, 80, 50, True, "bf16", "f32", "i32"), (17, 4, 4, 96, 64, True, "bf16", "bf16", "i32"),
    (64, 6, 2, 64, 0, False, "f32", "bf16", "i32"), (33, 3, 2, 10, 6, False, "bf16", "bf16", "i64"),
    (40, 0, 3, 256, 256, True, "f32", "f32", "i32"), (9, 2, 1, 512, 512, False, "bf16", "bf16", "i32"),
    (9, 2, 1, 510, 502, True, "bf16", "bf16", "i32"), (200, 7, 2, 192, 64, False, "bf16", "bf16", "i32"),
    (1000, 8, 2, 128, 128, True, "bf16", "bf16", "i32"), (129, 12, 3, 36, 20, False, "f32", "f32", "i64"),
    (5, 2, 2, 508, 8, False, "f32", "f32", "i32"), (2500, 4, 1, 128, 128, False, "f32", "f32", "i32")]


def inputs(m, hq, hk, d, rot, dt, wt, pt, places=300, packed=True):
    g = torch.Generator().manual_seed(m + d + rot)
    X = torch.bfloat16 if dt == "bf16" else torch.float32
    Wt = torch.bfloat16 if wt == "bf16" else torch.float32
    qkv = (torch.randn(m, hq + 2 * hk, d, generator=g) * 2).to(X).to(DEV)
    q, k = (qkv[:, :hq] if hq else None), (qkv[:, hq:hq + hk] if hk else None)
    wq, wk = ((1 + torch.randn(d, generator=g) * 0.3).to(Wt).to(DEV) for _ in range(2))
    ang = torch.rand(places, rot // 2, generator=g) * 6
    pos = torch.randint(0, places, (m,), generator=g, dtype=torch.int32 if pt == "i32" else torch.int64)
    gq = torch.randn(m, hq, d, generator=g).to(X).to(DEV) if hq else None
    gk = torch.randn(m, hk, d, generator=g).to(X).to(DEV) if hk else None
    table = (ang.cos().to(DEV), ang.sin().to(DEV), pos.to(DEV)) if rot else (None, None, None)
    return q, k, wq, wk, table, gq, gk


def pair_size(n, rot, interleaved):
    """|a| + |b| of each element's pair (|n| past rot)."""
    size = np.abs(n)
    if rot:
        a, b = headnorm.pairs(rot, interleaved)
        both = size[..., a] + size[..., b]
        size[..., a] = size[..., b] = both
    return size


@pytest.mark.parametrize("m,hq,hk,d,rot,inter,dt,wt,pt", CASES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_parity(lib, m, hq, hk, d, rot, inter, dt, wt, pt, offset):
    say(f"head norm m={m} heads={hq}/{hk} d={d} rot={rot} inter={inter} {dt} {wt} {pt}")
    q, k, wq, wk, table, gq, gk = inputs(m, hq, hk, d, rot, dt, wt, pt)
    kw = dict(eps=1e-5, interleaved=inter, weight_offset=offset)
    out = lib.qk_norm_rope_fwd(q, k, wq, wk, *table, **kw)
    grads = lib.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, *table, **kw)
    last = 2.0 ** -8 if dt == "bf16" else 0.0
    cos, sin = (f32(table[0]), f32(table[1])) if rot else (None, None)
    pos = table[2].cpu().numpy() if rot else None
    for x, w, y, g, dx, dw in ((q, wq, out[0], gq, grads[0], grads[2]), (k, wk, out[1], gk, grads[1], grads[3])):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        args = (f32(x), f32(w), cos, sin, pos, rot, 1e-5, inter, offset)
        ref = headnorm.forward(*args)
        n = headnorm.forward(f32(x), f32(w), None, None, None, 0, 1e-5, inter, offset)
        assert (np.abs(f32(y) - ref) <= last * np.abs(ref) + 32 * EPS * pair_size(n, rot, inter)).all()
        rx, rw = headnorm.backward(f32(g), *args)
        x64 = f32(x).astype(np.float64)
        inv = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-5)
        gn = headnorm.rotate(f32(g).astype(np.float64), cos, sin, pos, rot, inter, -1.0)
        size = inv * np.abs(pair_size(gn, rot, inter) * (np.abs(f32(w).astype(np.float64)) + offset)).max(-1, keepdims=True)
        assert (np.abs(f32(dx) - rx) <= last * np.abs(rx) + 64 * EPS * size * np.maximum(1, np.abs(x64 * inv))).all()
        assert (np.abs(f32(dw) - rw) <= 256 * EPS * np.abs(pair_size(gn, rot, inter) * x64 * inv).sum((0, 1))).all()


def test_strides_in_place_and_packed_gradients(lib):
    """Inputs and outputs as slices of packed tensors, heads or tokens outermost, and in place."""
    m, hq, hk, d = 37, 6, 2, 64
    q, k, wq, wk, table, gq, gk = inputs(m, hq, hk, d, d, "bf16", "bf16", "i32")
    want = lib.qk_norm_rope_fwd(q, k, wq, wk, *table)
    grads = lib.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, *table)
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, gq, gk)]
    assert heads_first[0].stride(0) == d
    got = lib.qk_norm_rope_fwd(*heads_first[:2], wq, wk, *table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    packed = torch.full((m, hq + 2 * hk, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = lib.qk_norm_rope_bwd(*heads_first[2:], *heads_first[:2], wq, wk, *table,
                               out=(packed[:, :hq], packed[:, hq:hq + hk]))
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    assert (packed[:, hq + hk:] == 7).all()
    odd = torch.empty(m * (hq * d + 1) + 1, dtype=torch.bfloat16, device=DEV)[1:]     # rows at odd addresses
    odd = odd.as_strided((m, hq, d), (hq * d + 1, d, 1))
    odd.copy_(q)
    got = lib.qk_norm_rope_fwd(odd, k, wq, wk, *table)
    assert torch.equal(got[0], want[0])
    both = torch.cat((q, k), 1)
    lib.qk_norm_rope_fwd(both[:, :hq], both[:, hq:], wq, wk, *table, out=(both[:, :hq], both[:, hq:]))
    assert torch.equal(both, torch.cat(want, 1))


def test_broadcast_input_and_shared_table(lib):
    """An expanded input (stride 0) is read as it is."""
    q, k, wq, wk, table, _, _ = inputs(8, 4, 2, 32, 32, "f32", "f32", "i32")
    wide = q[:, :1].expand(8, 4, 32)
    got, _ = lib.qk_norm_rope_fwd(wide, None, wq, None, *table)
    want, _ = lib.qk_norm_rope_fwd(wide.contiguous(), None, wq, None, *table)
    assert torch.equal(got, want)


def test_zero_rows_and_places_outside_the_table(lib):
    """Heads of zeros give zeros (eps > 0); a token whose position lies outside the table gets NaN and
    leaves the others as they are; no tokens at all is nothing to do, with dw zero."""
    q, k, wq, wk, table, gq, gk = inputs(12, 4, 2, 64, 32, "bf16", "bf16", "i64")
    want = lib.qk_norm_rope_fwd(q, k, wq, wk, *table)
    q[3] = 0
    pos = table[2].clone()
    pos[5], pos[6], pos[7] = -1, 300, 2 ** 40
    got = lib.qk_norm_rope_fwd(q, k, wq, wk, table[0], table[1], pos)
    assert (got[0][3] == 0).all()
    rest = [i for i in range(12) if i not in (3, 5, 6, 7)]
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest]) and a[5:8].isnan().all()
    none = lib.qk_norm_rope_bwd(gq[:0], gk[:0], q[:0], k[:0], wq, wk, table[0], table[1], pos[:0])
    assert none[0].shape == (0, 4, 64) and not none[2].any() and not none[3].any()
    assert lib.qk_norm_rope_fwd(q[:0], k[:0], wq, wk, table[0], table[1], pos[:0])[1].shape == (0, 2, 64)


def test_autograd_and_graph(lib):
    q, k, wq, wk, table, gq, gk = inputs(50, 4, 2, 64, 64, "f32", "f32", "i32")

    def step():
        return tuple(lib.qk_norm_rope_fwd(q, k, wq, wk, *table)) + tuple(
            lib.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, *table))

    _replay_check(step)
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    y, z = lib.QKNormRopeFunction.apply(*leaves, *table)
    torch.autograd.backward((y, z), (gq, gk))
    for got, want in zip((t.grad for t in leaves), step()[2:]):
        assert torch.equal(got, want)
