"""Refusals of expert routing, of rows in expert order and of 8-bit activations (no GPU needed): every call below
is invalid by construction, so the host's checks refuse it before a pointer is used or anything is launched."""
import ctypes

import pytest
import torch

import nf4_dequant_gemm_amd as m

FAKE, ODD, EVEN = ctypes.c_void_p(4096), ctypes.c_void_p(4097), ctypes.c_void_p(4100)
INVALID, UNSUPPORTED = m.NF4_EINVAL, m.NF4_EUNSUPPORTED


def route(**o):
    a = dict(x=FAKE, dt=m.NF4_F32, t=100, E=8, ld=8, keep=None, top=2, idx=FAKE, gate=FAKE, place=FAKE, source=FAKE,
             counts=FAKE, sizes=FAKE, mean_p=FAKE, losses=FAKE, ws=FAKE, wsb=None) | o
    lib = m.library()
    wsb = lib.moe_route_workspace_bytes(100, 8) if a["wsb"] is None else a["wsb"]
    return lib.moe_route(a["x"], a["dt"], a["t"], a["E"], a["ld"], a["keep"], a["top"], 1, a["idx"], a["gate"], a["place"],
                         a["source"], a["counts"], a["sizes"], a["mean_p"], a["losses"], a["ws"], wsb, None)


def route_bwd(**o):
    a = dict(x=FAKE, dt=m.NF4_F32, t=100, E=8, ld=8, top=2, idx=FAKE, counts=FAKE, sizes=FAKE, dgate=FAKE, dlosses=FAKE,
             dx=FAKE, ldd=8) | o
    return m.library().moe_route_bwd(a["x"], a["dt"], a["t"], a["E"], a["ld"], a["top"], 1, a["idx"], a["counts"],
                                     a["sizes"], a["dgate"], a["dlosses"], a["dx"], a["ldd"], None)


def test_route_refuses():
    lib = m.library()
    need = lib.moe_route_workspace_bytes(100, 8)
    assert need > 0 and lib.moe_route_workspace_bytes(0, 8) == 0 and lib.moe_route_workspace_bytes(100, 257) == 0
    for call in (route, route_bwd):
        for o in (dict(x=None), dict(x=ODD), dict(dt=2), dict(t=-1), dict(E=0), dict(E=257, ld=257), dict(ld=7), dict(top=0),
                  dict(top=9), dict(E=32, ld=32, top=17), dict(idx=None), dict(idx=ODD), dict(counts=None),
                  dict(counts=EVEN), dict(sizes=None), dict(sizes=EVEN)):
            assert call(**o) == INVALID, o
            assert lib.nf4_last_error()
        assert call(t=2 ** 30) == UNSUPPORTED
    for name in ("gate", "place", "source", "mean_p", "losses"):
        assert route(**{name: None}) == INVALID and route(**{name: ODD}) == INVALID, name
    assert route(wsb=need - 1) == INVALID and route(ws=None) == INVALID and route(ws=EVEN) == INVALID
    for o in (dict(dx=None), dict(dx=ODD), dict(ldd=7), dict(dgate=ODD), dict(dlosses=ODD)):
        assert route_bwd(**o) == INVALID, o
    assert route_bwd(t=0, x=None, idx=None, dx=None) == m.NF4_OK       # nothing to do


def test_rows_refuse():
    lib = m.library()
    base = dict(x=FAKE, dt=m.NF4_BF16, t=10, d=16, ld=16, place=FAKE, source=FAKE, top=2, gate=FAKE, z=FAKE, out=FAKE,
                dgate=FAKE, b=FAKE)

    def gather(**o):
        a = base | o
        return lib.moe_gather(a["x"], a["dt"], a["t"], a["d"], a["ld"], a["place"], a["source"], a["top"], a["out"], None)

    def combine(**o):
        a = base | o
        return lib.moe_combine(a["x"], a["dt"], a["t"], a["d"], a["place"], a["top"], a["gate"], a["b"], a["ld"], a["out"],
                               a["ld"], None)

    def bwd(**o):
        a = base | o
        return lib.moe_combine_bwd(a["x"], a["dt"], a["t"], a["d"], a["ld"], a["z"], a["place"], a["source"], a["top"],
                                   a["gate"], a["out"], a["dgate"], None)

    for call in (gather, combine, bwd):
        for o in (dict(x=None), dict(x=ODD), dict(dt=-1), dict(t=-1), dict(d=0), dict(top=0), dict(ld=15), dict(place=None),
                  dict(place=ODD), dict(out=None), dict(out=ODD)):
            assert call(**o) == INVALID, (call.__name__, o)
        assert call(t=2 ** 30) == UNSUPPORTED and call(d=2 ** 31, ld=2 ** 31) == UNSUPPORTED
        assert call(t=0, x=None, place=None, source=None, out=None, z=None, gate=None, dgate=None, b=None) == m.NF4_OK
    for call in (gather, bwd):
        assert call(source=None) == INVALID and call(source=ODD) == INVALID
    assert combine(gate=ODD) == INVALID and combine(b=ODD) == INVALID
    for name in ("gate", "dgate", "z"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: ODD}) == INVALID, name


def act8(codes=4096, scale=4096, rows=10, k=128):
    return m._ACT8_STRUCT.pack(codes, scale, rows, k)


def test_act8_refuses():
    lib = m.library()
    both = lambda q, x=FAKE, dt=m.NF4_BF16, ld=128: (lib.act8_pack(x, dt, ld, q, None), lib.act8_unpack(q, x, dt, ld, None))
    for q in (None, act8(codes=0), act8(codes=4100), act8(scale=0), act8(scale=4098), act8(rows=-1), act8(k=0)):
        assert both(q) == (INVALID, INVALID)
    for q, ld in ((act8(rows=2 ** 31), 128), (act8(k=2 ** 31), 2 ** 31), (act8(rows=2 ** 30, k=2 ** 14), 2 ** 14)):
        assert both(q, ld=ld) == (UNSUPPORTED, UNSUPPORTED)
    for o in (dict(x=None), dict(x=ODD), dict(dt=7), dict(ld=127)):
        assert both(act8(), **o) == (INVALID, INVALID), o
    assert both(act8(codes=0, scale=0, rows=0), x=None) == (m.NF4_OK, m.NF4_OK)


def weight(n=64, k=128):
    return ctypes.byref(m._NF4TensorC(n, k, 64, 0, FAKE, FAKE, None))


def test_act8_layers_refuse():
    lib = m.library()
    M, n, k, r, E = 10, 64, 128, 8, 2
    wb, wp = lib.qlora_bwd_act8_workspace_bytes(M, n, k, r), lib.qlora_swiglu_bwd_act8_workspace_bytes(M, n // 2, k, r)
    wm = lib.qlora_moe_bwd_act8_workspace_bytes(M, E, n // E, k, r)
    assert min(wb, wp, wm) > 0 and lib.qlora_bwd_act8_workspace_bytes(0, n, k, r) == 0
    assert lib.qlora_swiglu_bwd_act8_workspace_bytes(M, 0, k, r) == 0
    assert lib.qlora_moe_bwd_act8_workspace_bytes(M, 257, n, k, r) == 0

    def linear(**o):
        a = dict(dY=FAKE, X=act8(), W=weight(), A=FAKE, B=FAKE, r=r, T=FAKE, dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, wsb=wb) | o
        return lib.qlora_bwd_act8(a["dY"], a["X"], a["W"], a["A"], a["B"], a["r"], 1.0, a["T"], a["dX"], a["dA"], a["dB"],
                                  a["ws"], a["wsb"], None)

    def pair(**o):
        a = dict(dY=FAKE, X=act8(), W=weight(), A=FAKE, B=FAKE, r=r, T=FAKE, dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, wsb=wp,
                 Y=act8(k=n), B2=FAKE, dB2=FAKE) | o
        return lib.qlora_swiglu_bwd_act8(a["dY"], a["X"], a["W"], a["A"], a["B"], a["B2"], a["r"], 1.0, a["Y"], a["T"],
                                         a["dX"], a["dA"], a["dB"], a["dB2"], a["ws"], a["wsb"], None)

    def moe(**o):
        a = dict(dY=FAKE, X=act8(rows=5), source=FAKE, m=M, counts=FAKE, E=E, W=weight(), A=FAKE, B=FAKE, r=r, T=FAKE,
                 dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, wsb=wm) | o
        return lib.qlora_moe_bwd_dev_act8(a["dY"], a["X"], a["source"], a["m"], a["counts"], a["E"], a["W"], a["A"],
                                          a["B"], a["r"], 1.0, a["T"], a["dX"], a["dA"], a["dB"], a["ws"], a["wsb"], None)

    for call, need in ((linear, wb), (pair, wp), (moe, wm)):
        for name in ("dY", "A", "B", "dA", "dB", "ws"):
            assert call(**{name: None}) == INVALID and call(**{name: ODD}) == INVALID, (call.__name__, name)
        for o in (dict(X=None), dict(X=act8(codes=0)), dict(X=act8(k=64)), dict(T=None), dict(T=ODD), dict(dX=ODD),
                  dict(r=-1), dict(r=129), dict(wsb=need - 1)):
            assert call(**o) == INVALID, (call.__name__, o)
        assert call(X=act8(k=96), W=weight(k=96)) == UNSUPPORTED
    assert linear(X=act8(rows=0, codes=0, scale=0)) == INVALID
    for o in (dict(Y=None), dict(Y=act8(k=n, rows=9)), dict(Y=act8(k=n + 8)), dict(B2=None), dict(dB2=None), dict(r=65)):
        assert pair(**o) == INVALID, o
    for o in (dict(source=None), dict(source=ODD), dict(counts=None), dict(counts=EVEN), dict(E=0), dict(E=257),
              dict(E=3), dict(m=0)):
        assert moe(**o) == INVALID, o


def test_bindings_refuse():
    x, i32 = torch.zeros(4, 128), torch.int32
    place, source, gate = torch.zeros(4, 2, dtype=i32), torch.zeros(8, dtype=i32), torch.ones(4, 2)
    for call in (lambda: m.moe_route(x, 2), lambda: m.moe_gather(x, place, source), lambda: m.moe_combine(x, place, gate),
                 lambda: m.moe_combine_bwd(x, x, place, source, gate), lambda: m.act8_pack(x),
                 lambda: m.moe_route_bwd(gate, None, x, place, source, source)):
        with pytest.raises(ValueError, match="device|must be"):
            call()
    q = m.Act8Tensor(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 2), 128)
    assert q.shape == (4, 128)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        m.act8_unpack(q, torch.float16)
    w = m.NF4Tensor.empty(64, 192, 0, "cpu")
    with pytest.raises(ValueError, match="k = 192"):
        m.qlora_bwd_act8(x, q, w, None, None, 1.0, None)


def test_partials_stay_bounded():
    """Beside U (in bf16, in float32 and once more as a partial) and B transposed a workspace holds 1 GiB of partials at
    most, however many rows there are."""
    lib = m.library()
    for rows in (1, 256, 5000, 1 << 16, 1 << 20):
        for n, k, r in ((64, 64, 1), (4096, 14336, 32), (28672, 8192, 64), (14336, 4096, 128)):
            assert lib.qlora_bwd_act8_workspace_bytes(rows, n, k, r) <= 10 * rows * r + 2 * r * n + (1 << 30) + 1024


def test_grouped_rows_of_no_tokens():
    """The grouped layer's kept activation has a row at least, also where every source is foreign: there is no row to read
    in the place of one that is not there."""
    lib = m.library()
    M, n, k, r, E = 10, 64, 128, 8, 2
    wsb = lib.qlora_moe_bwd_act8_workspace_bytes(M, E, n // E, k, r)
    for codes in (0, 4096):
        assert lib.qlora_moe_bwd_dev_act8(FAKE, act8(codes=codes, rows=0), FAKE, M, FAKE, E, weight(), FAKE, FAKE, r, 1.0, FAKE,
                                          FAKE, FAKE, FAKE, FAKE, wsb, None) == INVALID
        assert b"row" in lib.nf4_last_error()


def test_workspaces_of_the_pair_and_of_experts():
    """The pair's workspace is the stacked layer's at twice the rank, the projections' gradients and two block diagonals; that of
    experts holds U (in bf16, in float32 and once more as a partial), at most 1 GiB of dB's partials, or those of their
    dA and dB (one copy each where there are many experts), B transposed where it is used, and a table."""
    lib = m.library()
    for rows in (1, 300, 1 << 16, 1 << 20):
        for n, k, r in ((64, 64, 0), (64, 64, 1), (11008, 4096, 16), (11008, 4096, 64), (28672, 8192, 33)):
            pair, one = lib.qlora_swiglu_bwd_act8_workspace_bytes(rows, n, k, r), lib.qlora_bwd_act8_workspace_bytes(rows, 2 * n, k, 2 * r)
            assert one + 4 * rows * n + 16 * n * r <= pair <= one + 4 * rows * n + 16 * n * r + 3 * 256
        for E in (1, 8, 256):
            for n, k, r in ((64, 64, 1), (2048, 7168, 128), (11008, 4096, 64)):
                assert lib.qlora_moe_bwd_act8_workspace_bytes(rows, E, n, k, r) <= (
                    10 * rows * r + 2 * r * E * n + (1 << 30) + 4 * r * E * (n + k) + (1 << 16))
