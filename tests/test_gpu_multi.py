"""An adapter of its own for every row: the HIP path against the float64 oracle, exactly where the
values allow it and within the layer's tolerance elsewhere.

Exact cases: a base that decodes to zero and small integers in X, A, B, dY and powers of two in s. Every
product and sum is then an integer (or a power of two of one) below 2^24, T and U are integers up to
256 (exact in bf16), and Y, dX, dA and dB are the exact value rounded once to bf16.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import fp4, multi, nf4
from tests.gpu_helpers import check_close, f32, say, u16
from tests.test_gpu_graph import _replay_check

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make_ids(kind, m, L, seed=0):
    rng = np.random.default_rng(seed + 17 * m + L)
    ids = {"one": lambda: np.full(m, L - 1), "none": lambda: np.full(m, -1), "each": lambda: np.arange(m) % L,
           "mixed": lambda: np.where(rng.random(m) < 0.2, -1, rng.integers(0, L, m)),
           "outside": lambda: rng.choice([-7, -1, L, L + 1, 2 ** 31 - 1, 0, L - 1], m),
           "runs": lambda: np.repeat(rng.integers(-1, L, m), rng.integers(1, 40, m))[:m]}[kind]()
    return torch.from_numpy(ids.astype(np.int32))


def quantise(lib, W, fmt):
    if fmt == "e2m1":
        return lib.fp4_quantize(W.to(DEV)), fp4.dequantize_f32(fp4.quantize(W.float().numpy()))
    dq = 256 if fmt == "nf4" else 0
    return lib.nf4_quantize(W.to(DEV), dq), nf4.dequantize_f32(nf4.quantize(W.float().numpy(), dq))


SHAPES = [(1, 64, 8, 1, 1, "one"), (1, 512, 136, 16, 4, "each"), (2, 256, 264, 8, 2, "each"), (5, 320, 72, 12, 3, "mixed"),
          (15, 256, 520, 64, 15, "each"), (16, 512, 136, 16, 16, "each"), (16, 1024, 264, 32, 2, "none"),
          (17, 512, 264, 16, 5, "outside"), (48, 256, 72, 128, 7, "mixed"), (49, 192, 136, 4, 49, "each"),
          (64, 512, 520, 33, 3, "runs"), (130, 320, 264, 16, 64, "mixed"), (257, 256, 264, 20, 300, "each"),
          (300, 64, 520, 64, 2, "one"), (600, 192, 72, 8, 1024, "mixed"), (1025, 128, 136, 48, 6, "runs"),
          (1100, 256, 264, 7, 40, "outside")]
# one shape for every height of the mid kernel's row blocks, with K a multiple of its step and not, and
# wide weights for the 16-row stream kernel
HEIGHTS = [(m, k, 264, 16, 3, "mixed") for m in (20, 40, 60, 75, 95, 110, 125, 260) for k in (512, 576)]
WIDE = [(16, 512, 14400, 16, 16, "each"), (9, 256, 14400, 128, 4, "mixed"), (3, 256, 14344, 8, 2, "one"),
        (16, 256, 14400, 40, 20, "outside")]
SHAPES += HEIGHTS + WIDE


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n,r,L,kind", SHAPES)
def test_low_rank_part_is_exact(lib, m, k, n, r, L, kind, fmt):
    say(f"multi exact m={m} k={k} n={n} r={r} L={L} {kind} {fmt}")
    rng = np.random.default_rng(m + k + r)
    sparse = lambda shape, p: (rng.integers(-2, 3, shape) * (rng.random(shape) < p)).astype(np.float32)
    X, A, dY, B = sparse((m, k), 0.5), sparse((L, r, k), 16 / k), sparse((m, n), 0.5), sparse((L, n, r), min(0.3, 16 / n))
    s = 2.0 ** rng.integers(-2, 3, L).astype(np.float32)
    ids = make_ids(kind, m, L)
    q, Wd = quantise(lib, torch.zeros(n, k, dtype=torch.bfloat16), fmt)
    assert not Wd.any()
    Yo, To = multi.forward(X, Wd, A, B, s, ids.numpy())
    dXo, dAo, dBo = multi.backward(dY, X, Wd, A, B, s, ids.numpy())
    U = np.abs(np.einsum("in,inr->ir", dY, B[np.clip(ids.numpy(), 0, L - 1)])).max()
    assert np.abs(To).max() <= 256 and U <= 256, "the inputs leave the exact range"
    b = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    sd, idd = torch.from_numpy(s).to(DEV), ids.to(DEV)
    Y, T = lib.qlora_multi_fwd(b(X), q, b(A), b(B), sd, idd)
    dX, dA, dB = lib.qlora_multi_bwd(b(dY), b(X), q, b(A), b(B), sd, idd, T)
    for name, got, ref in (("T", T, To), ("Y", Y, Yo), ("dX", dX, dXo), ("dA", dA, dAo), ("dB", dB, dBo)):
        assert np.array_equal(f32(got), f32(torch.from_numpy(ref).to(torch.bfloat16))), name
    again = lib.qlora_multi_bwd(b(dY), b(X), q, b(A), b(B), sd, idd, None, need_dx=False)
    assert again[0] is None and torch.equal(again[1], dA) and torch.equal(again[2], dB)


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n,r,L,kind", SHAPES)
def test_parity(lib, m, k, n, r, L, kind, fmt):
    say(f"multi m={m} k={k} n={n} r={r} L={L} {kind} {fmt}")
    X, W = wl.normal_bf16(1 + m, (m, k), 1.0), wl.normal_bf16(2 + m, (n, k), 0.02)
    A, B = wl.normal_bf16(3 + m, (L, r, k), k ** -0.5), wl.normal_bf16(4 + m, (L, n, r), 0.1)
    dY = wl.normal_bf16(5 + m, (m, n), 1.0)
    s = wl.uniform_f32(6 + m, (L,), 0.25, 2.0)
    ids = make_ids(kind, m, L)
    q, Wd = quantise(lib, W, fmt)
    Yo, To = multi.forward(f32(X), Wd, f32(A), f32(B), s.numpy(), ids.numpy())
    dXo, dAo, dBo = multi.backward(f32(dY), f32(X), Wd, f32(A), f32(B), s.numpy(), ids.numpy())
    X, A, B, dY, s, ids = (t.to(DEV) for t in (X, A, B, dY, s, ids))
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    dX, dA, dB = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    for name, got, ref in (("Y", Y, Yo), ("T", T, To), ("dX", dX, dXo), ("dA", dA, dAo), ("dB", dB, dBo)):
        check_close(name, f32(got), ref)


# one shape for every row tile height that the split of the mid kernel chooses, K a multiple of its step and not
TILES = [(37, 64, 14376), (69, 256, 8928), (53, 2176, 80), (64, 768, 240), (121, 576, 8800), (193, 256, 13616),
         (333, 576, 120), (197, 1792, 80), (1258, 64, 4216), (864, 256, 6480), (410, 64, 14696), (609, 128, 9968),
         (2219, 64, 3240), (2155, 128, 3288)]


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n", TILES)
def test_forward_of_every_height(lib, m, k, n, fmt):
    say(f"multi height m={m} k={k} n={n} {fmt}")
    r, L = 16, 5
    X, W = wl.normal_bf16(1 + m, (m, k), 1.0), wl.normal_bf16(2 + m, (n, k), 0.02)
    A, B = wl.normal_bf16(3 + m, (L, r, k), k ** -0.5), wl.normal_bf16(4 + m, (L, n, r), 0.1)
    s, ids = wl.uniform_f32(6 + m, (L,), 0.25, 2.0), make_ids("mixed", m, L)
    q, Wd = quantise(lib, W, fmt)
    Yo, To = multi.forward(f32(X), Wd, f32(A), f32(B), s.numpy(), ids.numpy())
    Y, T = lib.qlora_multi_fwd(*(t if t is q else t.to(DEV) for t in (X, q, A, B, s, ids)))
    check_close("Y", f32(Y), Yo)
    check_close("T", f32(T), To)


@pytest.mark.parametrize("m", [7, 40, 300])
def test_rows_do_not_touch_one_another(lib, m):
    """Infinities and NaN in one row of X, or in an adapter no row has, stay there."""
    k, n, r, L = 256, 136, 16, 4
    X, W = wl.normal_bf16(1, (m, k), 1.0).to(DEV), wl.normal_bf16(2, (n, k), 0.02).to(DEV)
    A, B = wl.normal_bf16(3, (L, r, k), 0.1).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    s, ids = torch.full((L,), 0.5, device=DEV), (torch.arange(m, device=DEV) % 3).int()
    q = lib.nf4_quantize(W, 256)
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    A2, B2, X2 = A.clone(), B.clone(), X.clone()
    A2[3], B2[3], X2[m // 2, 5] = float("nan"), float("inf"), float("nan")
    Y2, T2 = lib.qlora_multi_fwd(X2, q, A2, B2, s, ids)
    others = torch.arange(m, device=DEV) != m // 2
    assert torch.equal(Y[others], Y2[others]) and torch.equal(T[others], T2[others])
    assert Y2[m // 2].isnan().all()
    dY = wl.normal_bf16(5, (m, n), 1.0).to(DEV)
    dX, dA, dB = lib.qlora_multi_bwd(dY, X, q, A2, B2, s, ids, T)
    want = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    assert torch.equal(dX, want[0]) and torch.equal(dA, want[1]) and torch.equal(dB, want[2])
    assert not dA[3].any() and not dB[3].any()


def test_one_adapter_agrees_with_the_layer(lib):
    """Every row on one adapter is qlora_fwd's layer (T bit for bit in value, Y within the rounding of
    s B to bf16 that the single layer makes: none for a power of two)."""
    m, k, n, r = 300, 512, 264, 16
    X, W = wl.normal_bf16(1, (m, k), 1.0).to(DEV), wl.normal_bf16(2, (n, k), 0.02).to(DEV)
    A, B = wl.normal_bf16(3, (r, k), k ** -0.5).to(DEV), wl.normal_bf16(4, (n, r), 0.1).to(DEV)
    q = lib.nf4_quantize(W, 256)
    Y, T = lib.qlora_fwd(X, q, A, B, 0.5)
    ids = torch.zeros(m, dtype=torch.int32, device=DEV)
    Y2, T2 = lib.qlora_multi_fwd(X, q, A[None].contiguous(), B[None].contiguous(), torch.tensor([0.5], device=DEV), ids)
    check_close("Y", f32(Y2), f32(Y))
    check_close("T", f32(T2), f32(T))


def test_graph_replay_with_other_ids(lib):
    m, k, n, r, L = 70, 256, 136, 16, 5
    X, W = wl.normal_bf16(1, (m, k), 1.0).to(DEV), wl.normal_bf16(2, (n, k), 0.02).to(DEV)
    A, B = wl.normal_bf16(3, (L, r, k), 0.1).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    dY, s = wl.normal_bf16(5, (m, n), 1.0).to(DEV), torch.full((L,), 0.5, device=DEV)
    ids = make_ids("mixed", m, L).to(DEV)
    q = lib.nf4_quantize(W, 256)

    def step():
        Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
        return (Y, T) + tuple(lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T))

    _replay_check(step)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for kind in ("each", "none", "runs"):
        ids.copy_(make_ids(kind, m, L))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want), kind


def test_autograd_and_other_stream(lib):
    m, k, n, r, L = 33, 256, 72, 8, 3
    X, W = wl.normal_bf16(1, (m, k), 1.0).to(DEV), wl.normal_bf16(2, (n, k), 0.02).to(DEV)
    A, B = wl.normal_bf16(3, (L, r, k), 0.1).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    dY, s = wl.normal_bf16(5, (m, n), 1.0).to(DEV), torch.full((L,), 0.5, device=DEV)
    ids = make_ids("mixed", m, L).to(DEV)
    q = lib.nf4_quantize(W, 256)
    want = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x, a, b = (t.clone().requires_grad_() for t in (X, A, B))
        lib.QLoRAMultiFunction.apply(x, q, a, b, s, ids).backward(dY)
    side.synchronize()
    for got, ref in zip((x.grad, a.grad, b.grad), want):
        assert torch.equal(got, ref)
