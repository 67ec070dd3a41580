"""The adapters' gradients at ranks, stages and sizes on either side of the kernels' choices, against float64 sums.

dB = s dY^T T: float32 sums over m rows (m 2^-24 of the magnitudes' sum at most, taken as 2^-10 for m <= 2^14), and half a
step of bf16 of the result, 2^-8. dA = s U^T X: the same, and of U = dY B the sums over n <= 2^15 columns (2^-9 of their
magnitudes) and the rounding to bf16, 2^-8.
"""
import pytest
import torch

from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def near(got, want, allowed):
    return bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + allowed).all())


def check(dA, dB, dY, X, B, T, s):
    dY, X, B, T = (z.double() for z in (dY, X, B, T))
    U, most, x = dY @ B, dY.abs() @ B.abs(), X.abs()
    assert near(dB, s * dY.t() @ T, s * 2.0 ** -10 * (dY.abs().t() @ T.abs()))
    assert near(dA, s * U.t() @ X, s * ((2.0 ** -8 + 2.0 ** -10) * (U.abs().t() @ x) + 2.0 ** -9 * (most.t() @ x)))


@pytest.mark.parametrize("m,k,n,r", [
    (1, 64, 8, 1), (64, 64, 72, 7), (65, 128, 64, 33), (128, 64, 520, 100), (129, 192, 264, 127), (200, 4096, 64, 63),
    (200, 4096, 64, 64), (300, 2112, 8184, 9), (300, 64, 8192, 8), (700, 64, 8192, 33), (9000, 64, 128, 128),
    (9000, 64, 128, 100), (1000, 2048, 2048, 128), (1000, 2048, 2048, 101), (77, 64, 20000, 128), (77, 64, 20000, 65),
    (2500, 320, 1000, 31), (130, 64, 32768, 2)])
def test_one_layer(lib, m, k, n, r):
    say(f"adapter sums m={m} k={k} n={n} r={r}")
    g = torch.Generator(DEV).manual_seed(m + n + r)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(BF)
    X, A, B, dY, T = rand(m, k), rand(r, k), rand(n, r), rand(m, n), rand(m, r)
    q = lib.NF4Tensor.empty(n, k, 256, torch.device(DEV))       # the weight is not read without dX
    none, dA, dB = lib.qlora_bwd(dY, X, q, A, B, 0.5, T, need_dx=False)
    assert none is None
    check(dA, dB, dY, X, B, T, 0.5)


@pytest.mark.parametrize("counts,k,n,r", [((1, 64, 0, 65), 64, 72, 33), ((200, 129), 128, 4088, 7), ((200, 129), 128, 4096, 100),
                                          ((0, 1000, 63, 2, 191), 1024, 520, 101), ((30, 70), 2048, 64, 64)])
def test_grouped(lib, counts, k, n, r):
    say(f"adapter sums of experts {counts} k={k} n={n} r={r}")
    E, m = len(counts), sum(counts)
    g = torch.Generator(DEV).manual_seed(m + n + r)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(BF)
    X, A, B, dY, T = rand(m, k), rand(E * r, k), rand(E * n, r), rand(m, n), rand(m, r)
    q = lib.NF4Tensor.empty(E * n, k, 256, torch.device(DEV))
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    ws = torch.empty(lib.moe_workspace_bytes_dev(m, E, n, k, r), dtype=torch.uint8, device=DEV)
    lib.qlora_moe_bwd_dev(dY, X, torch.tensor(counts, device=DEV), q, A, B, 0.5, T, None, dA, dB, ws)
    lo = 0
    for e, c in enumerate(counts):
        check(dA[e * r:(e + 1) * r], dB[e * n:(e + 1) * n], dY[lo:lo + c], X[lo:lo + c], B[e * n:(e + 1) * n], T[lo:lo + c], 0.5)
        lo += c


@pytest.mark.parametrize("m,k,n,r", [(4100, 64, 4104, 33), (4000, 64, 4104, 33), (2100, 128, 8192, 63), (4100, 64, 4104, 40),
                                     (4100, 64, 4104, 31)])
def test_eight_bits(lib, m, k, n, r):
    """X in 8 bits, U and dB from one pass or two launches. U times a scale is rounded to bf16 in the place of U."""
    g = torch.Generator(DEV).manual_seed(m + n + r)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(BF)
    X, A, B, dY, T = lib.act8_pack(rand(m, k)), rand(r, k), rand(n, r), rand(m, n), rand(m, r)
    q = lib.NF4Tensor.empty(n, k, 256, torch.device(DEV))
    none, dA, dB = lib.qlora_bwd_act8(dY, X, q, A, B, 0.5, T, need_dx=False)
    assert none is None
    check(dA, dB, dY, lib.act8_unpack(X, torch.float32), B, T, 0.5)


@pytest.mark.parametrize("m,k,n,r", [(1, 64, 72, 128), (16, 128, 4096, 100), (5, 64, 520, 65), (17, 64, 8, 127)])
def test_eight_bits_few_rows_high_rank(lib, m, k, n, r):
    """The two launches with the rows of a decode batch, U in float32 beside its bf16 form."""
    test_eight_bits(lib, m, k, n, r)


@pytest.mark.parametrize("t,top,E,k,n,r", [(300, 2, 4, 192, 264, 100), (37, 1, 3, 64, 72, 128), (9, 3, 5, 128, 520, 65),
                                           (4200, 1, 2, 64, 4104, 33)])
@pytest.mark.parametrize("grouped", [False, True])
def test_experts_from_eight_bits_at_high_rank(lib, t, top, E, k, n, r, grouped):
    """The grouped layer's two launches, from the tokens' codes or the grouped rows'."""
    g = torch.Generator(DEV).manual_seed(t + n + r)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(BF)
    ro = lib.moe_route(torch.randn(t, E, generator=g, device=DEV), top, torch.arange(t, device=DEV) % 5 != 2)
    X, A, B, dY, T = rand(t, k), rand(E * r, k), rand(E * n, r), rand(t * top, n), rand(t * top, r)
    q = lib.NF4Tensor.empty(E * n, k, 256, torch.device(DEV))
    X8 = lib.act8_pack(lib.moe_gather(X, ro.place, ro.source) if grouped else X)
    none, dA, dB = lib.qlora_moe_bwd_act8(dY, X8, None if grouped else ro.source, ro.counts, q, A, B, 0.5, T, need_dx=False)
    assert none is None
    x, lo = lib.act8_unpack(X8, torch.float32), 0
    for e, c in enumerate(ro.counts.tolist()):
        rows = x[lo:lo + c] if grouped else x[ro.source[lo:lo + c].long()]
        check(dA[e * r:(e + 1) * r], dB[e * n:(e + 1) * n], dY[lo:lo + c], rows, B[e * n:(e + 1) * n], T[lo:lo + c], 0.5)
        lo += c
