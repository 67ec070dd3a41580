"""Activations in 8 bits against the oracle: codes, scales and unpacked values have to be equal, bit for bit.

The layers' backward passes from them: what does not touch the kept activation equals the bf16 layer's up to
the order of sums, see close_rest. dA = s U^T X is checked against float64 sums: U times the scale as the matrix cores take it (rounded to bf16:
half a step, 2^-8 of every term), U's float32 sums (below 2^-14 of the terms in it), float32 sums (m 2^-24 of the magnitudes at most, taken as
2^-10 for m <= 2^14), and the result's half step 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import act8, swiglu
from tests.gpu_helpers import f32, say

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def act(m, k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(k, generator=g))
    size[::37] *= 30
    return (torch.randn(m, k, generator=g) * size).to(dtype)


def same(a, b):
    return np.array_equal(np.asarray(a, np.float32).view(np.uint32), np.asarray(b, np.float32).view(np.uint32))


def check(lib, x, dev=None):
    m, k = x.shape
    say(f"act8 m={m} k={k} {x.dtype}")
    q = lib.act8_pack(x.to(DEV) if dev is None else dev)
    codes, scale = act8.pack(f32(x))
    assert q.shape == (m, k) and np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(np.isnan(scale), np.isnan(f32(q.scale))) and same(np.nan_to_num(f32(q.scale)), np.nan_to_num(scale))
    v = act8.value(codes, scale, k)
    got = lib.act8_unpack(q, F32)
    assert np.array_equal(f32(got), v, equal_nan=True)
    assert torch.equal(lib.act8_unpack(q).cpu().view(torch.int16)[~np.isnan(v)],
                       torch.from_numpy(v).to(BF).view(torch.int16)[~np.isnan(v)])
    return q


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 64), (3, 63), (17, 4096), (5, 65), (128, 100), (33, 777), (1000, 72), (7, 14336)])
def test_pack_and_unpack(lib, dtype, m, k):
    check(lib, act(m, k, dtype, m + k))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_borders(lib, dtype):
    """Halves of the largest value, exact half-integers, and (float32) values a step from a border."""
    x = torch.zeros(64, 128, dtype=F32)
    a = torch.exp2(torch.randn(64, generator=torch.Generator().manual_seed(1)) * 8)
    a[:20] = 127 * 2.0 ** torch.arange(-10, 10)               # ties at every half-integer
    a = a.to(dtype).float()
    h = torch.arange(127).float() + 0.5
    x[:, 0] = a
    x[:, 1:128] = a[:, None] * h / 127
    x[1::2] *= -1
    x = x.to(dtype)
    x[:, 64] = x[:, 0]
    if dtype is F32:
        step = torch.randint(-2, 3, x.shape, generator=torch.Generator().manual_seed(2), dtype=torch.int32)
        step[:, 0] = step[:, 64] = 0
        x = (x.view(torch.int32) + step * (x != 0)).view(F32)
    check(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extremes(lib, dtype):
    """Zeros, the smallest and largest numbers, Inf and NaN, which stay in their blocks."""
    x = act(12, 192, dtype, 3)
    x[0] = 0
    x[1, :64] = 2.0 ** -126
    x[2, :64] = 2.0 ** -119
    x[3, :64] *= 0
    x[3, 5] = 2.0 ** -120
    x[4, 70] = float("inf")
    x[5, 0] = float("-inf")
    x[6, 191] = float("nan")
    x[7, :64] = torch.finfo(dtype).max
    x[8, :64] = torch.finfo(BF).max / 2
    x[9, 63] = 1e-40
    q = check(lib, x)
    v = lib.act8_unpack(q, F32).cpu()
    assert not v.isinf().any()
    assert v[4, 64:128].isnan().all() and v[5, :64].isnan().all() and v[6, 128:].isnan().all()
    assert int(v.isnan().sum()) == 192


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [128, 130])
def test_strides(lib, dtype, k):
    """Rows inside a wider matrix, at any alignment; unpacked into one, whose rest stays."""
    wide = act(50, k + 9, dtype, 4).to(DEV)
    inner = wide[:, 3:3 + k]
    q = check(lib, inner.cpu(), dev=inner)
    out = torch.full((50, k + 9), 5.0, dtype=dtype, device=DEV)
    lib.act8_unpack(q, out=out[:, 1:1 + k])
    assert torch.equal(out[:, 1:1 + k], lib.act8_unpack(q, dtype)) and (out[:, :1] == 5).all() and (out[:, 1 + k:] == 5).all()
    assert lib.act8_pack(inner[:0]).shape == (0, k)
    assert lib.act8_unpack(lib.act8_pack(inner[:0])).shape == (0, k)


def test_offsets_past_32_bits(lib):
    """More than 2^32 elements."""
    m, k = 70000, 65600
    x = torch.randn(64, k, device=DEV).bfloat16().repeat(m // 64 + 1, 1)[:m]
    q = lib.act8_pack(x)
    first = lib.act8_pack(x[:64])
    assert torch.equal(q.codes[-48:], first.codes[:48])                 # 70000 = 64 * 1093 + 48
    for lo in (0, 64 * 500, 64 * 1000):
        assert torch.equal(q.codes[lo:lo + 64], first.codes) and torch.equal(q.scale[lo:lo + 64], first.scale)
    del x
    out = lib.act8_unpack(q)
    want = lib.act8_unpack(first)
    assert all(torch.equal(out[lo:lo + 64], want) for lo in (0, 64 * 500, 64 * 1000, 64 * 1092))


def layer(lib, m, k, n, r, seed, stack=1, dq=256):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().to(DEV)
    q = lib.nf4_quantize(normal(stack * n, k, std=0.02), dq)
    return q, act(m, k, BF, seed).to(DEV), normal(stack * r, k, std=k ** -0.5), normal(stack * n, r, std=0.05), normal(m, n)


def close_dA(got, U, X, s):
    U, X = f32(U).astype(np.float64), f32(X).astype(np.float64)
    want, mag = s * (U.T @ X), abs(s) * (np.abs(U).T @ np.abs(X))
    say(f"  dA: rel err {np.linalg.norm(f32(got) - want) / np.linalg.norm(want):.2e}")
    assert (np.abs(f32(got) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * mag).all()


def close_rest(dX, dB, want, dY, W, A, B, T, s):
    """dX and dB against the bf16 layer's. dB above rank 64 is equal bit for bit; up to there U and dB are float32 sums
    taken in another order, U's within 2^-10 of the magnitudes' sum, so that its bf16 values differ by that twice and a
    step of 2^-7. dX differs by what s A makes of that, by the order of its own float32 sums, which are split for few
    tiles (n <= 2^14: within 2^-10 of the magnitudes), and a step. dB against float64 sums: 2^-10 of the magnitudes, half
    a step."""
    more = 0
    if A is not None:
        dY, A, B, T = (z.double() for z in (dY, A, B, T))
        more = abs(s) * (2.0 ** -11 * (dY @ B).abs() @ A.abs())
        if A.shape[0] > 64:
            assert torch.equal(dB, want[2])
        else:
            more = abs(s) * (2.0 ** -7 * (dY @ B).abs() + 2.0 ** -8 * dY.abs() @ B.abs()) @ A.abs()
            ref, mag = s * dY.t() @ T, abs(s) * dY.abs().t() @ T.abs()
            assert ((dB.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag).all()
    assert ((dX.double() - want[0].double()).abs() <=
            2.0 ** -7 * want[0].double().abs() + more + 2.0 ** -10 * dY.double().abs() @ W.double().abs()).all()


@pytest.mark.parametrize("m,k,n,r", [(1, 64, 8, 1), (17, 320, 72, 7), (64, 256, 256, 8), (300, 1088, 136, 16), (1000, 448, 264, 20),
                                     (257, 192, 64, 33), (500, 256, 512, 64), (130, 4096, 64, 100), (2100, 128, 64, 128),
                                     (257, 128, 8, 1), (1000, 64, 392, 31), (513, 64, 1032, 32), (2000, 192, 4104, 13), (256, 64, 6152, 24), (700, 64, 1000, 63),
                                     (1100, 64, 15256, 8), (1300, 64, 12912, 32), (2000, 64, 8392, 64)])
def test_linear(lib, m, k, n, r):
    q, X, A, B, dY = layer(lib, m, k, n, r, m)
    T = torch.randn(m, r, device=DEV).bfloat16()
    s = 0.5
    X8 = lib.act8_pack(X)
    dX, dA, dB = lib.qlora_bwd_act8(dY, X8, q, A, B, s, T)
    want = lib.qlora_bwd(dY, lib.act8_unpack(X8), q, A, B, s, T)
    close_rest(dX, dB, want, dY, lib.nf4_dequantize(q, F32), A, B, T, s)
    close_dA(dA, dY.double() @ B.double(), lib.act8_unpack(X8, F32), s)
    none, dA2, dB2 = lib.qlora_bwd_act8(dY, X8, q, A, B, s, T, need_dx=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)


def test_part_of_the_rows(lib):
    """Rows of a kept activation are one themselves: a micro-batch's backward from its part."""
    q, X, A, B, dY = layer(lib, 100, 1088, 72, 8, 3)
    T = torch.randn(100, 8, device=DEV).bfloat16()
    whole = lib.act8_pack(X)
    part = lib.Act8Tensor(whole.codes[37:90], whole.scale[37:90], whole.k)
    assert torch.equal(lib.act8_unpack(part), lib.act8_unpack(whole)[37:90])
    got = lib.qlora_bwd_act8(dY[37:90], part, q, A, B, 0.5, T[37:90])
    want = lib.qlora_bwd_act8(dY[37:90].clone(), lib.act8_pack(X[37:90]), q, A, B, 0.5, T[37:90].clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("form", ["nf4", "nf4 dq", "e2m1"])
@pytest.mark.parametrize("m,k,n,r", [(1, 64, 4096, 4), (17, 320, 2048, 8), (300, 576, 4096, 33), (513, 1088, 1000, 0),
                                     (1000, 1088, 2832, 16), (130, 256, 1608, 128), (50, 128, 64, 0), (2000, 1024, 520, 0)])
def test_few_tiles(lib, m, k, n, r, form):
    """dX of few tiles and a long reduction, which is split over workgroups, for each kind of weight."""
    q, X, A, B, dY = layer(lib, m, k, n, max(r, 1), n)
    if form != "nf4 dq":
        w = torch.randn(n, k, generator=torch.Generator().manual_seed(m)).bfloat16().to(DEV)
        q = lib.nf4_quantize(w, 0) if form == "nf4" else lib.fp4_quantize(w)
    A, B, T = (A, B, torch.randn(m, r, device=DEV).bfloat16()) if r else (None, None, None)
    X8 = lib.act8_pack(X)
    dX, dA, dB = lib.qlora_bwd_act8(dY, X8, q, A, B, 1.5, T)
    assert r or dA is None and dB is None
    close_rest(dX, dB, lib.qlora_bwd(dY, X, q, A, B, 1.5, T), dY, lib.nf4_dequantize(q, F32), A, B, T, 1.5)


@pytest.mark.parametrize("m,k,n,r", [(1, 64, 8, 1), (40, 128, 72, 8), (300, 320, 264, 16), (70, 256, 40, 0), (200, 192, 100 * 8, 64), (513, 128, 72, 32)])
def test_pair(lib, m, k, n, r):
    q, X, A, _, dH = layer(lib, m, k, n, max(r, 1), m, stack=2)
    g = torch.Generator().manual_seed(5)
    Bg, Bu = ((torch.randn(n, r, generator=g) * 0.05).bfloat16().to(DEV) for _ in range(2))
    Ygu = act(m, 2 * n, BF, 6).to(DEV)
    Tgu = torch.randn(m, 2 * r, device=DEV).bfloat16() if r else None
    X8, Y8 = lib.act8_pack(X), lib.act8_pack(Ygu)
    args = (A, Bg, Bu) if r else (None, None, None)
    dX, dA, dBg, dBu = lib.qlora_swiglu_bwd_act8(dH, X8, q, *args, 0.5, Y8, Tgu)
    y = f32(lib.act8_unpack(Y8, F32)).astype(np.float64)
    h = f32(dH).astype(np.float64)
    dg, du = h * y[:, n:] * swiglu.silu_grad(y[:, :n]), h * swiglu.silu(y[:, :n])
    W = f32(lib.nf4_dequantize(q, F32)).astype(np.float64)
    # every rounding to bf16 on the way (of dY, the weight or A, U, s B or s A) costs at most 2^-8 of each term,
    # the result's own half a step
    near = lambda got, want, mag: (np.abs(f32(got) - want) <= 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -8 * mag).all()
    both = lambda f: (f(dg, du, lambda z: z), f(abs(dg), abs(du), abs))
    U = lambda g, u, of: np.concatenate((g @ of(f32(Bg)), u @ of(f32(Bu))), 1)
    assert near(dX, *both(lambda g, u, of: np.concatenate((g, u), 1) @ of(W) + (0.5 * U(g, u, of) @ of(f32(A)) if r else 0)))
    if r:
        T = f32(Tgu).astype(np.float64)
        assert near(dBg, *both(lambda g, u, of: 0.5 * g.T @ of(T[:, :r])))
        assert near(dBu, *both(lambda g, u, of: 0.5 * u.T @ of(T[:, r:])))
        assert near(dA, *both(lambda g, u, of: 0.5 * U(g, u, of).T @ of(f32(lib.act8_unpack(X8, F32)).astype(np.float64))))


@pytest.mark.parametrize("t,k,n,E,top,r", [(1, 64, 8, 2, 1, 1), (40, 256, 72, 4, 2, 8), (500, 320, 136, 8, 2, 16),
                                           (300, 192, 64, 3, 3, 40), (2000, 128, 64, 16, 1, 4), (900, 64, 1160, 3, 2, 21),
                                           (150, 64, 72, 256, 2, 8), (1500, 64, 136, 2, 2, 64)])
@pytest.mark.parametrize("grouped", [False, True])
def test_moe(lib, t, k, n, E, top, r, grouped):
    """The tokens kept once (through the routing), or the grouped rows themselves; every eighth token is padding."""
    keep = torch.arange(t, device=DEV) % 8 != 3
    x = torch.randn(t, E, generator=torch.Generator().manual_seed(t)).to(DEV)
    x[:, 0] -= 20.0 * (E > 2)                                 # the first expert gets next to no rows
    ro = lib.moe_route(x, top, keep)
    m, N = t * top, int(ro.sizes[1])
    q, X, A, B, _ = layer(lib, t, k, n, r, t, stack=E)
    dY, T = (torch.randn(m, w, device=DEV).bfloat16() for w in (n, r))
    dY[N:], T[N:] = float("nan"), float("nan")               # rows behind the last count for nothing
    X8 = lib.act8_pack(X)
    Xg = lib.moe_gather(lib.act8_unpack(X8), ro.place, ro.source)
    if grouped:
        X8, source = lib.act8_pack(Xg), None
        Xg = lib.act8_unpack(X8)
    else:
        source = ro.source
    dX, dA, dB = lib.qlora_moe_bwd_act8(dY, X8, source, ro.counts, q, A, B, 2.0, T)
    ws = torch.empty(lib.moe_workspace_bytes_dev(m, E, n, k, r), dtype=torch.uint8, device=DEV)
    want = torch.empty(m, k, dtype=BF, device=DEV), torch.empty_like(A), torch.empty_like(B)
    lib.qlora_moe_bwd_dev(dY, Xg, ro.counts, q, A, B, 2.0, T, *want, ws)
    W = lib.nf4_dequantize(q, F32)
    lo, v = 0, f32(lib.act8_unpack(X8, F32))
    for e, c in enumerate(ro.counts.tolist()):
        rows = v[lo:lo + c] if grouped else v[ro.source[lo:lo + c].cpu().numpy()]
        mine = dA[e * r:(e + 1) * r]
        if c == 0:
            assert not mine.any()
            assert not dB[e * n:(e + 1) * n].any()
        else:
            b, a = B[e * n:(e + 1) * n], A[e * r:(e + 1) * r]
            close_rest(dX[lo:lo + c], dB[e * n:(e + 1) * n], (want[0][lo:lo + c], None, want[2][e * n:(e + 1) * n]),
                       dY[lo:lo + c], W[e * n:(e + 1) * n], a, b, T[lo:lo + c], 2.0)
            close_dA(mine, dY[lo:lo + c].double() @ B[e * n:(e + 1) * n].double(), torch.from_numpy(rows), 2.0)
        lo += c


def test_longest_rows_of_dy(lib):
    m, n, k, r, s = 2, 2 ** 22, 64, 4, 0.5
    rand = lambda *shape: torch.randn(*shape, device=DEV, generator=torch.Generator(DEV).manual_seed(n % 97)).bfloat16()
    q = lib.NF4Tensor.empty(n, k, 256, torch.device(DEV))       # the weight is not read without dX
    X, A, B, dY, T = rand(m, k), rand(r, k), rand(n, r), rand(m, n), rand(m, r)
    X8 = lib.act8_pack(X)
    none, dA, dB = lib.qlora_bwd_act8(dY, X8, q, A, B, s, T, need_dx=False)
    assert none is None
    ref, mag = s * dY.double().t() @ T.double(), s * dY.double().abs().t() @ T.double().abs()
    assert ((dB.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag).all()
    # U is the sum of 2^22 products in chains of at most 2^12 sums: within 2^-12 of its magnitudes' sum
    U, mag = dY.double() @ B.double(), dY.double().abs() @ B.double().abs()
    v = lib.act8_unpack(X8, F32).double()
    want, most = s * U.t() @ v, s * U.abs().t() @ v.abs()
    assert ((dA.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -20) * most
            + 2.0 ** -12 * s * mag.t() @ v.abs()).all()


def test_captured_linear_and_pair(lib):
    """Captured with few tiles and one pass over dY, replayed with other inputs: the eager call's bits every time."""
    m, k, n, r = 300, 576, 2048, 8
    q, X, A, B, dY = layer(lib, m, k, n, r, 1)
    q2, _, A2, _, _ = layer(lib, m, k, n, r, 2, stack=2)
    T, T2, Ygu = (torch.randn(m, w, device=DEV).bfloat16() for w in (r, 2 * r, 2 * n))
    X8, Y8 = lib.act8_pack(X), lib.act8_pack(Ygu)
    run = lambda: (*lib.qlora_bwd_act8(dY, X8, q, A, B, 0.5, T), *lib.qlora_swiglu_bwd_act8(dY, X8, q2, A2, B, B, 0.5, Y8, T2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(4):
        dY.copy_(torch.randn(m, n, device=DEV))
        T.copy_(torch.randn(m, r, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, run())), i


def test_moe_foreign_sources(lib):
    """A source outside the kept rows stands for zeros."""
    m, k, n, r = 20, 128, 64, 8
    q, X, A, B, _ = layer(lib, m, k, n, r, 1)
    dY, T = (torch.randn(m, w, device=DEV).bfloat16() for w in (n, r))
    source = torch.arange(m, dtype=torch.int32, device=DEV)
    source[3], source[9], source[15] = -1, 2 ** 31 - 1, 20
    counts = torch.tensor([m], device=DEV)
    zeros = X.clone()
    zeros[[3, 9, 15]] = 0
    a = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(X), source, counts, q, A, B, 1.0, T)
    b = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(zeros), None, counts, q, A, B, 1.0, T)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_nan_stays_in_its_expert(lib):
    E, top, t, k, n, r = 4, 1, 80, 128, 64, 8
    x = torch.full((t, E), -5.0, device=DEV)
    x[torch.arange(t), torch.arange(t) % E] = 5.0
    ro = lib.moe_route(x, top)
    q, X, A, B, _ = layer(lib, t, k, n, r, 2, stack=E)
    dY, T = (torch.randn(t, w, device=DEV).bfloat16() for w in (n, r))
    ok = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(X), ro.source, ro.counts, q, A, B, 1.0, T)
    X[6, 70] = float("nan")                                  # expert 2, columns 64 .. 127
    bad = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(X), ro.source, ro.counts, q, A, B, 1.0, T)
    assert torch.equal(ok[0], bad[0]) and torch.equal(ok[2], bad[2])
    dA, dN = ok[1].view(E, r, k), bad[1].view(E, r, k)
    others = [0, 1, 3]
    assert torch.equal(dA[others], dN[others]) and torch.equal(dA[2, :, :64], dN[2, :, :64]) and dN[2, :, 64:].isnan().all()


@pytest.mark.parametrize("t,r,unrouted", [(80, 8, False), (80, 8, True), (400, 7, False), (400, 100, True), (256, 64, True)])
def test_nan_of_the_first_token_stays_in_its_expert(lib, t, r, unrouted):
    """A NaN in token 0, the first row that is kept: its expert's dA alone has it, and nobody's where that token is padding.
    The experts' rows end inside a stage of 64, or their stages are odd in number."""
    E, k, n = 4, 192, 64
    x = torch.full((t, E), -5.0, device=DEV)
    x[torch.arange(t), torch.arange(t) % E] = 5.0
    keep = torch.arange(t, device=DEV) >= int(unrouted)
    ro = lib.moe_route(x, 1, keep)
    q, X, A, B, _ = layer(lib, t, k, n, r, 2, stack=E)
    dY, T = (torch.randn(t, w, device=DEV).bfloat16() for w in (n, r))
    ok = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(X), ro.source, ro.counts, q, A, B, 1.0, T)
    assert all(z[:int(ro.sizes[1])].isfinite().all() for z in ok)
    X[0, 70] = float("nan")                                  # columns 64 .. 127
    bad = lib.qlora_moe_bwd_act8(dY, lib.act8_pack(X), ro.source, ro.counts, q, A, B, 1.0, T)
    N = int(ro.sizes[1])
    assert torch.equal(ok[0][:N], bad[0][:N]) and torch.equal(ok[2], bad[2])
    dA, dN = ok[1].view(E, r, k), bad[1].view(E, r, k)
    assert torch.equal(dA[1:], dN[1:]) and torch.equal(dA[0, :, :64], dN[0, :, :64]) and torch.equal(dA[0, :, 128:], dN[0, :, 128:])
    assert torch.equal(dA[0], dN[0]) if unrouted else dN[0, :, 64:128].isnan().all()
