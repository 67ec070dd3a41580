"""An adapter for every row at the sizes of prompts and training: more than 256 rows and 128 tiles of
256 x 256 (the large forward kernel), the sums over rows in several stages, ranks above 64, more rows
than the transposes look through for an adapter's use, and X and dY of nearly 4 GiB.

The float64 oracle goes row by row; at these sizes `reference` computes the same per adapter, and is itself
held against the oracle at a small size. Tolerances as in test_gpu_multi.py.
"""
import ctypes

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import multi
from tests.gpu_helpers import check_close, f32, say
from tests.test_gpu_multi import DEV, make_ids, quantise

pytestmark = pytest.mark.gpu


def reference(dY, X, Wd, A, B, s, ids):
    """(Y, T, dX, dA, dB) in float64, one product for each adapter's rows."""
    dY, X, Wd, A, B, s = (np.asarray(t, np.float64) for t in (dY, X, Wd, A, B, s))
    Y, dX = X @ Wd.T, dY @ Wd
    T, dA, dB = np.zeros((X.shape[0], A.shape[1])), np.zeros_like(A), np.zeros_like(B)
    for a in range(A.shape[0]):
        i = np.nonzero(ids == a)[0]
        T[i] = X[i] @ A[a].T
        U = dY[i] @ B[a]
        Y[i] += s[a] * (T[i] @ B[a].T)
        dX[i] += s[a] * (U @ A[a])
        dA[a], dB[a] = s[a] * (U.T @ X[i]), s[a] * (dY[i].T @ T[i])
    return Y, T, dX, dA, dB


def test_reference_is_the_oracle():
    rng = np.random.default_rng(3)
    X, dY, A, B, Wd = (rng.standard_normal(sh) for sh in ((40, 24), (40, 16), (5, 3, 24), (5, 16, 3), (16, 24)))
    s, ids = rng.standard_normal(5), make_ids("mixed", 40, 5).numpy()
    want = multi.forward(X, Wd, A, B, s, ids) + multi.backward(dY, X, Wd, A, B, s, ids)
    for got, ref in zip(reference(dY, X, Wd, A, B, s, ids), want):
        assert np.allclose(got, ref, rtol=1e-12, atol=1e-12)


# m, k, n, r, L, order of ids. The first five take the large forward (153, 140, 258, 129 and 900 tiles of 256 x 256,
# whole and with a remainder on either side), r a multiple of 8 and not, the last of them with one adapter for
# all rows, more than 8192 of them, and blocks of 448 rows in the sums. The others: ranks above 64 in the 64-row
# projection, adapters without rows, blocks of 64 and 128 rows.
SHAPES = [(2300, 128, 4104, 12, 5, "mixed"), (2305, 64, 3336, 64, 3, "runs"), (300, 192, 32776, 16, 4, "outside"),
          (10800, 64, 768, 8, 7, "each"), (9001, 64, 6152, 128, 3, "one"), (9001, 256, 1032, 64, 9, "mixed"),
          (2600, 576, 2056, 72, 300, "runs"), (5003, 128, 1160, 12, 40, "runs")]


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n,r,L,kind", SHAPES)
def test_parity(lib, m, k, n, r, L, kind, fmt):
    say(f"multi large m={m} k={k} n={n} r={r} L={L} {kind} {fmt}")
    X, W = wl.normal_bf16(1 + m, (m, k), 1.0), wl.normal_bf16(2 + m, (n, k), 0.02)
    A, B = wl.normal_bf16(3 + m, (L, r, k), k ** -0.5), wl.normal_bf16(4 + m, (L, n, r), 0.1)
    dY, s, ids = wl.normal_bf16(5 + m, (m, n), 1.0), wl.uniform_f32(6 + m, (L,), 0.25, 2.0), make_ids(kind, m, L)
    q, Wd = quantise(lib, W, fmt)
    want = reference(f32(dY), f32(X), Wd, f32(A), f32(B), s.numpy(), ids.numpy())
    X, A, B, dY, s, ids = (t.to(DEV) for t in (X, A, B, dY, s, ids))
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    grads = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    for name, got, ref in zip(("Y", "T", "dX", "dA", "dB"), (Y, T) + tuple(grads), want):
        check_close(name, f32(got), ref)
    again = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, None)
    for got, ref in zip(again, grads):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n,r,L,kind", SHAPES)
def test_low_rank_part_is_exact(lib, m, k, n, r, L, kind, fmt):
    """As in test_gpu_multi.py: a base of zeros and small integers, so that every value is exact before its one
    rounding to bf16. (T and U within 256: exact in bf16; sums over rows below 2^24.)"""
    say(f"multi large exact m={m} k={k} n={n} r={r} L={L} {kind} {fmt}")
    rng = np.random.default_rng(m + k + r)
    sparse = lambda shape, p: (rng.integers(-2, 3, shape) * (rng.random(shape) < p)).astype(np.float32)
    X, A, dY, B = sparse((m, k), 0.5), sparse((L, r, k), 16 / k), sparse((m, n), 0.5), sparse((L, n, r), min(0.3, 16 / n))
    s = 2.0 ** rng.integers(-2, 3, L).astype(np.float32)
    ids = make_ids(kind, m, L)
    q, Wd = quantise(lib, torch.zeros(n, k, dtype=torch.bfloat16), fmt)
    assert not Wd.any()
    want = reference(dY, X, np.zeros((n, k)), A, B, s, ids.numpy())
    U = max(np.abs(dY[i] @ B[a]).max(initial=0) for a in range(L) for i in [np.nonzero(ids.numpy() == a)[0]])
    assert np.abs(want[1]).max() <= 256 and U <= 256 and max(np.abs(w).max() for w in want) < 2 ** 22
    b = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    sd, idd = torch.from_numpy(s).to(DEV), ids.to(DEV)
    Y, T = lib.qlora_multi_fwd(b(X), q, b(A), b(B), sd, idd)
    dX, dA, dB = lib.qlora_multi_bwd(b(dY), b(X), q, b(A), b(B), sd, idd, T)
    for name, got, ref in zip(("Y", "T", "dX", "dA", "dB"), (Y, T, dX, dA, dB), want):
        assert np.array_equal(f32(got), f32(torch.from_numpy(ref).to(torch.bfloat16))), name


def test_sums_of_whole_blocks(lib):
    """dA and dB over blocks of 1024 rows, the most that a workgroup takes (as in a training batch), the last
    of an adapter odd in length."""
    m, k, n, r, L = 9001, 64, 14856, 72, 3
    g = torch.Generator(device=DEV).manual_seed(5)
    X, dY = (torch.randn(m, c, generator=g, device=DEV).bfloat16() for c in (k, n))
    A, B = wl.normal_bf16(3, (L, r, k), k ** -0.5).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    s, ids = wl.uniform_f32(6, (L,), 0.25, 2.0).to(DEV), make_ids("runs", m, L).to(DEV)
    q = lib.nf4_quantize(wl.normal_bf16(2, (n, k), 0.02).to(DEV), 256)
    _, dA, dB = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, None, need_dx=False)
    for a in range(L):
        i = ids == a
        x, y, A64, B64 = X[i].double(), dY[i].double(), A[a].double(), B[a].double()
        check_close("dA", f32(dA[a]), f32((s[a].double() * ((y @ B64).T @ x)).float()))
        check_close("dB", f32(dB[a]), f32((s[a].double() * (y.T @ (x @ A64.T))).float()))


@pytest.mark.parametrize("m", [100, 255, 256, 257])
@pytest.mark.parametrize("r", [8, 33, 57, 72, 96, 112, 128])
def test_many_rows_to_an_adapter(lib, m, r):
    """Two adapters, on either side of the 256 rows up to which a block of the sums is an adapter: every rank
    tile of the sums and of the row projections, in stages of 64 rows."""
    k, n, L = 320, 264, 2
    say(f"multi rank m={m} r={r}")
    X, W = wl.normal_bf16(1 + m, (m, k), 1.0), wl.normal_bf16(2 + m, (n, k), 0.02)
    A, B = wl.normal_bf16(3 + m, (L, r, k), k ** -0.5), wl.normal_bf16(4 + m, (L, n, r), 0.1)
    dY, s, ids = wl.normal_bf16(5 + m, (m, n), 1.0), wl.uniform_f32(6 + m, (L,), 0.25, 2.0), make_ids("mixed", m, L)
    q, Wd = quantise(lib, W, "nf4")
    want = reference(f32(dY), f32(X), Wd, f32(A), f32(B), s.numpy(), ids.numpy())
    X, A, B, dY, s, ids = (t.to(DEV) for t in (X, A, B, dY, s, ids))
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    for name, got, ref in zip(("Y", "T", "dX", "dA", "dB"), (Y, T) + lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T), want):
        check_close(name, f32(got), ref)


@pytest.mark.parametrize("m,k,n", [(520001, 4096, 72), (60000, 64, 35776)])
def test_offsets_past_31_bits(lib, m, k, n):
    """X (Y and dY) of nearly the 4293918720 bytes that the gathering copies reach. Y and dX at the first, the
    last and some random rows, dA and dB whole, against float64 on the device."""
    r, L = 8, 3
    assert 0.98 * 4293918720 < m * max(n, k) * 2 <= 4293918720
    g = torch.Generator(device=DEV).manual_seed(7)
    X, dY = (torch.randn(m, c, generator=g, device=DEV, dtype=torch.bfloat16) for c in (k, n))
    A, B = wl.normal_bf16(3, (L, r, k), k ** -0.5).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    s, ids = wl.uniform_f32(6, (L,), 0.25, 2.0).to(DEV), (torch.randperm(m, generator=g, device=DEV) % (L + 1) - 1).int()
    q = lib.nf4_quantize(wl.normal_bf16(2, (n, k), 0.02).to(DEV), 256)
    W = lib.nf4_dequantize(q, torch.float32).double()
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    dX, dA, dB = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    some = torch.cat((torch.arange(20, device=DEV), torch.arange(m - 20, m, device=DEV),
                      torch.randint(0, m, (200,), generator=g, device=DEV)))
    x, y, a = X[some].double(), dY[some].double(), ids[some].long()
    sa = torch.where(a >= 0, s[a].double(), 0.0)[:, None]
    t, u = (x[:, None] * A[a].double()).sum(2), (y[:, :, None] * B[a].double()).sum(1)
    check_close("Y", f32(Y[some]), (x @ W.T.contiguous() + sa * (B[a].double() * t[:, None]).sum(2)).cpu().numpy())
    check_close("dX", f32(dX[some]), (y @ W + sa * (A[a].double() * u[:, :, None]).sum(1)).cpu().numpy())
    check_close("T", f32(T[some]), torch.where(a[:, None] >= 0, t, 0.0).cpu().numpy())
    for a in range(L):
        dA64, dB64 = torch.zeros(r, k, device=DEV, dtype=torch.float64), torch.zeros(n, r, device=DEV, dtype=torch.float64)
        for i in (ids == a).nonzero()[:, 0].split(40000):
            x, y = X[i].double(), dY[i].double()
            dA64 += s[a].double() * ((y @ B[a].double()).T.contiguous() @ x)
            dB64 += s[a].double() * (y.T.contiguous() @ (x @ A[a].double().T.contiguous()))
        check_close("dA", f32(dA[a]), dA64.cpu().numpy())
        check_close("dB", f32(dB[a]), dB64.cpu().numpy())


@pytest.mark.parametrize("m,k,n,r,L", [(1, 256, 136, 12, 2), (16, 256, 14408, 16, 4), (130, 320, 264, 16, 64),
                                       (300, 512, 1032, 12, 5), (2300, 128, 4104, 12, 5), (9001, 64, 264, 72, 3)])
def test_workspace_is_kept_to(lib, m, k, n, r, L):
    """Nothing is written past the bytes that the library asks for, on any path; a workspace of another
    content gives the same results."""
    X, dY = wl.normal_bf16(1, (m, k), 1.0).to(DEV), wl.normal_bf16(2, (m, n), 1.0).to(DEV)
    A, B = wl.normal_bf16(3, (L, r, k), 0.1).to(DEV), wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    s, ids = torch.full((L,), 0.5, device=DEV), make_ids("mixed", m, L).to(DEV)
    q = lib.nf4_quantize(wl.normal_bf16(5, (n, k), 0.02).to(DEV), 256)
    W = lib._NF4TensorC(q.n, q.k, q.block, q.dq_block, q.codes.data_ptr(), q.absmax.data_ptr(), q.scale.data_ptr())
    c, p = lib.library(), lambda t: t.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    grads = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    for fill in (0, 255):
        wsb = c.qlora_multi_fwd_workspace_bytes(m, n, k, r, L)
        ws = torch.full((wsb + 4096,), fill, dtype=torch.uint8, device=DEV)
        Y2, T2 = torch.empty_like(Y), torch.empty_like(T)
        assert c.qlora_multi_fwd(p(X), m, ctypes.byref(W), p(A), p(B), p(s), p(ids), L, r, p(Y2), p(T2), p(ws), wsb,
                                 stream) == lib.NF4_OK
        assert torch.equal(Y2, Y) and torch.equal(T2, T) and (ws[wsb:] == fill).all()
        wsb = c.qlora_multi_bwd_workspace_bytes(m, n, k, r, L)
        ws = torch.full((wsb + 4096,), fill, dtype=torch.uint8, device=DEV)
        out = [torch.empty_like(g) for g in grads]
        assert c.qlora_multi_bwd(p(dY), p(X), m, ctypes.byref(W), p(A), p(B), p(s), p(ids), L, r, p(T), *(p(g) for g in out),
                                 p(ws), wsb, stream) == lib.NF4_OK
        assert all(torch.equal(a, b) for a, b in zip(out, grads)) and (ws[wsb:] == fill).all()
