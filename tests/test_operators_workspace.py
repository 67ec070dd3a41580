"""Device workspace of the layer with an adapter for every row (no GPU needed): no float32 copy of Y beside
the kernel that keeps its sums in registers, and a bounded number of remembered sizes."""
import pytest

import nf4_dequant_gemm_amd as m


@pytest.mark.parametrize("rows,n,k,r,L", [(8192, 11008, 4096, 64, 4), (16384, 28672, 8192, 16, 8), (2300, 4104, 128, 12, 5),
                                          (257, 16392, 4096, 16, 3)])
def test_large_forward_holds_no_copy_of_y(rows, n, k, r, L):
    """More than 256 rows and 128 tiles of 256 x 256: the rows' order, T's float sums (at most 1000 workgroups
    of up to 64 rows) and, for a rank that is no multiple of 8, padded copies of B and T."""
    rp = (r + 7) // 8 * 8
    order = 4 * (rows + 4 * (L + 2))
    sums = max(1000 * 64, rows) * rp * 4
    padded = 0 if rp == r else (L * n + rows) * rp * 2
    got = m.library().qlora_multi_fwd_workspace_bytes(rows, n, k, r, L)
    assert got <= order + sums + padded + 5 * 256
    assert got < rows * n * 4


@pytest.mark.parametrize("rows,n,k,r,L", [(1, 4096, 4096, 16, 8), (256, 65536, 512, 16, 4), (1111, 2952, 2880, 12, 5),
                                          (257, 16384, 256, 8, 1)])
def test_split_sums_have_their_place(rows, n, k, r, L):
    """Up to 256 rows or 128 tiles Y's float sums are in the workspace."""
    assert m.library().qlora_multi_fwd_workspace_bytes(rows, n, k, r, L) >= rows * n * 4


def test_remembered_sizes_are_bounded():
    """A server sees a new batch size in many of its steps: the sizes that the binding remembers do not grow
    with them."""
    for rows in range(1, 3000):
        m._bytes_of("qlora_multi_fwd_workspace_bytes", rows, 64, 64, 8, 2)
    assert m._bytes_of.cache_info().currsize <= 1024
