"""Rows of different jobs in one batch stay apart: infinities and NaN in a row's X or dY, or in an adapter
that no row has, change no bit of another row's T, Y or dX, nor of another adapter's dA and dB; and those in
a weight row's constants stay in its column of Y.

n % 64 != 0 in most shapes: the last step of dX's reduction then reaches past the end of a row of dY.
"""
import pytest
import torch

import workloads as wl
from tests.gpu_helpers import say
from tests.test_gpu_multi import DEV, quantise

pytestmark = pytest.mark.gpu

# dX with 2, 4 and 8 row tiles a wave and its reduction split; not split; the 16-row stream kernel;
# the large forward (153 tiles of 256 x 256)
SHAPES = [(7, 256, 1032), (100, 256, 1032), (300, 256, 1032), (300, 256, 136), (9, 256, 14408), (2300, 128, 4104)]


def inputs(lib, m, k, n, fmt, r=16, L=4):
    X, A, dY = (wl.normal_bf16(i, sh, sd).to(DEV) for i, sh, sd in ((1, (m, k), 1.0), (3, (L, r, k), 0.1), (5, (m, n), 1.0)))
    B = wl.normal_bf16(4, (L, n, r), 0.1).to(DEV)
    q, _ = quantise(lib, wl.normal_bf16(2, (n, k), 0.02), fmt)
    return X, q, A, B, torch.full((L,), 0.5, device=DEV), (torch.arange(m, device=DEV) % 3).int(), dY


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_a_row_of_dy(lib, m, k, n, fmt):
    say(f"multi isolation dY m={m} k={k} n={n} {fmt}")
    X, q, A, B, s, ids, dY = inputs(lib, m, k, n, fmt)
    want = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, None)
    # rows of adapter 1, each with a row of another adapter before and after it; Inf at a row's start and NaN
    # throughout
    bad = torch.tensor([1, (m // 2) // 3 * 3 + 1, (m - 2) // 3 * 3 + 1], device=DEV).unique()
    assert (ids[bad] == 1).all()
    dY2, A2, B2 = dY.clone(), A.clone(), B.clone()
    dY2[bad] = float("nan")
    dY2[bad[0], :8] = float("inf")
    A2[3], B2[3] = float("nan"), float("inf")
    dX, dA, dB = lib.qlora_multi_bwd(dY2, X, q, A2, B2, s, ids, None)
    rest = torch.ones(m, dtype=torch.bool, device=DEV)
    rest[bad] = False
    assert torch.equal(dX[rest], want[0][rest])
    assert dX[bad].isnan().all()
    for got, ref in ((dA, want[1]), (dB, want[2])):
        assert torch.equal(got[[0, 2, 3]], ref[[0, 2, 3]])
        assert not got[1].isfinite().all()


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_a_row_of_x(lib, m, k, n, fmt):
    say(f"multi isolation X m={m} k={k} n={n} {fmt}")
    X, q, A, B, s, ids, dY = inputs(lib, m, k, n, fmt)
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    want = lib.qlora_multi_bwd(dY, X, q, A, B, s, ids, T)
    X2, A2, B2 = X.clone(), A.clone(), B.clone()
    at = (m // 2) // 3 * 3 + 1
    X2[at, 5], X2[at, -1] = float("nan"), float("inf")
    A2[3], B2[3] = float("nan"), float("inf")
    Y2, T2 = lib.qlora_multi_fwd(X2, q, A2, B2, s, ids)
    rest = torch.arange(m, device=DEV) != at
    assert torch.equal(Y2[rest], Y[rest]) and torch.equal(T2[rest], T[rest])
    assert Y2[at].isnan().all() and T2[at].isnan().all()
    dX, dA, dB = lib.qlora_multi_bwd(dY, X2, q, A2, B2, s, ids, T2)
    assert torch.equal(dX, want[0])
    for got, ref in ((dA, want[1]), (dB, want[2])):
        assert torch.equal(got[[0, 2, 3]], ref[[0, 2, 3]])
        assert got[1].isnan().any()


@pytest.mark.parametrize("fmt", ["nf4", "nf4f", "e2m1"])
@pytest.mark.parametrize("m", [3, 20, 40, 60, 75, 95, 110, 125, 300])
def test_a_weight_row(lib, m, fmt):
    """K = 320 is no multiple of the mid kernel's step at any height, so that a step reaches past the end of
    a weight row. Blocks of row 51 and on have a constant of NaN, none of row 50."""
    k, n = 320, 136
    say(f"multi isolation W m={m} {fmt}")
    X, q, A, B, s, ids, _ = inputs(lib, m, k, n, fmt)
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    q2 = q.clone()
    if fmt == "nf4":
        q2.scale[1] = float("nan")                    # of blocks 256 to 511: rows 51 to 102
    elif fmt == "nf4f":
        q2.absmax.view(n, -1)[51:103] = float("nan")
    else:
        q2.absmax.view(n, -1)[51:103] = 0x7F          # the E4M3 NaN
    Y2, T2 = lib.qlora_multi_fwd(X, q2, A, B, s, ids)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[51:103] = True
    assert torch.equal(Y2[:, ~bad], Y[:, ~bad]) and torch.equal(T2, T)
    assert Y2[:, bad].isnan().all()


@pytest.mark.parametrize("k", [128, 256, 640, 768])
@pytest.mark.parametrize("m", [3, 20, 40, 60, 75, 95, 110, 125, 300])
def test_a_run_of_weight_rows(lib, m, k):
    """As above where K is a multiple of the step but the waves that take turns along K are not as many: a
    wave whose turn lies past the end of a weight row. The run of the double quantisation that starts with a
    row has a scale of NaN; the row before it has none of it."""
    n, kblk = 520, k // 64
    row = next(r for r in range(1, n) if r * kblk % 256 == 0)       # first row that starts a run
    say(f"multi isolation run m={m} k={k} row={row}")
    X, q, A, B, s, ids, _ = inputs(lib, m, k, n, "nf4")
    Y, T = lib.qlora_multi_fwd(X, q, A, B, s, ids)
    q2 = q.clone()
    q2.scale[row * kblk // 256] = float("nan")
    Y2, T2 = lib.qlora_multi_fwd(X, q2, A, B, s, ids)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[row:-(-(row * kblk + 256) // kblk)] = True
    assert torch.equal(Y2[:, ~bad], Y[:, ~bad]) and torch.equal(T2, T)
    assert Y2[:, bad].isnan().all()
