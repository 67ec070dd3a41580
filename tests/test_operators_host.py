"""Refusals of the operators beside the layer (no GPU needed): every call below is invalid by
construction, so the host's checks refuse it before a pointer is used or anything is launched."""
import ctypes

import pytest
import torch

import nf4_dequant_gemm_amd as m

FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)
INVALID, UNSUPPORTED = m.NF4_EINVAL, m.NF4_EUNSUPPORTED


def weight(n=64, k=128):
    return m._NF4TensorC(n, k, 64, 0, FAKE, FAKE, None)


def test_multi_refuses():
    lib = m.library()
    M, n, k, r, L = 100, 64, 128, 8, 3
    wf, wb = lib.qlora_multi_fwd_workspace_bytes(M, n, k, r, L), lib.qlora_multi_bwd_workspace_bytes(M, n, k, r, L)
    assert wf > 0 and wb > 0 and lib.qlora_multi_fwd_workspace_bytes(0, n, k, r, L) == 0
    assert wb >= 2 * M * r * 2 + L * r * (n + k) * 2        # U, T and both transposed factors

    def fwd(**o):
        a = dict(X=FAKE, m=M, W=weight(), A=FAKE, B=FAKE, s=FAKE, ids=FAKE, L=L, r=r, Y=FAKE, T=FAKE, ws=FAKE, wsb=wf) | o
        return lib.qlora_multi_fwd(a["X"], a["m"], ctypes.byref(a["W"]), a["A"], a["B"], a["s"], a["ids"], a["L"],
                                   a["r"], a["Y"], a["T"], a["ws"], a["wsb"], None)

    def bwd(**o):
        a = dict(dY=FAKE, X=FAKE, m=M, W=weight(), A=FAKE, B=FAKE, s=FAKE, ids=FAKE, L=L, r=r, T=FAKE, dX=FAKE, dA=FAKE,
                 dB=FAKE, ws=FAKE, wsb=wb) | o
        return lib.qlora_multi_bwd(a["dY"], a["X"], a["m"], ctypes.byref(a["W"]), a["A"], a["B"], a["s"], a["ids"],
                                   a["L"], a["r"], a["T"], a["dX"], a["dA"], a["dB"], a["ws"], a["wsb"], None)

    for call, outs, need in ((fwd, ("Y", "T"), wf), (bwd, ("dA", "dB"), wb)):
        for name in ("X", "A", "B", "s", "ids", "ws") + outs:
            assert call(**{name: None}) == INVALID, name
            assert call(**{name: ODD}) == INVALID, name
            assert lib.nf4_last_error()
        for o in (dict(m=0), dict(L=0), dict(L=1025), dict(r=0), dict(r=129), dict(wsb=need - 1)):
            assert call(**o) == INVALID, o
        assert call(W=weight(n=60)) == UNSUPPORTED and call(W=weight(k=96)) == UNSUPPORTED
        assert call(m=2 ** 24) == UNSUPPORTED               # X of 4 GiB: past the gathers' offsets
    assert bwd(dY=None) == INVALID and bwd(dX=ODD) == INVALID and bwd(T=ODD) == INVALID


def heads(data=FAKE, ts=512, hs=64, n=8):
    return m._HeadsC(data, ts, hs, n)


def test_head_norm_refuses():
    lib = m.library()
    base = dict(tokens=5, d=64, rot=32, interleaved=0, dtype=m.NF4_BF16, w_dtype=m.NF4_F32, wq=4096, wk=4096,
                w_offset=0.0, eps=1e-6, cos=4096, sin=4096, places=10, pos=4096, pos64=0)
    ws = lib.qk_norm_rope_bwd_workspace_bytes(64)
    assert ws > 0 and lib.qk_norm_rope_bwd_workspace_bytes(0) == 0

    def both(q=heads(), k=heads(), qo=heads(), ko=heads(), gq=heads(), gk=heads(), wsb=ws, wsp=FAKE, **o):
        p = m._HeadNormC(**(base | o))
        ref = ctypes.byref
        f = lib.qk_norm_rope_fwd(ref(p), ref(q), ref(k), ref(qo), ref(ko), None)
        b = lib.qk_norm_rope_bwd(ref(p), ref(gq), ref(gk), ref(q), ref(k), ref(qo), ref(ko), FAKE, FAKE, wsp, wsb, None)
        return f, b

    for o in (dict(tokens=-1), dict(dtype=3), dict(w_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(wq=None),
              dict(wk=4098), dict(cos=None), dict(sin=4098), dict(pos=None), dict(pos=4098), dict(pos=4100, pos64=1),
              dict(places=0), dict(q=heads(n=0), k=heads(n=0), qo=heads(n=0), ko=heads(n=0)), dict(q=heads(data=None)),
              dict(k=heads(data=ODD)), dict(q=heads(ts=-1)), dict(qo=heads(n=7)), dict(ko=heads(hs=-2)), dict(q=heads(n=-1))):
        assert both(**o) == (INVALID, INVALID), o
    for o in (dict(d=63), dict(d=0), dict(d=514), dict(rot=66), dict(rot=31), dict(rot=-2), dict(tokens=2 ** 28)):
        assert both(**o) == (UNSUPPORTED, UNSUPPORTED), o
    # arguments that the backward alone has (its calls below are refused too)
    for o in (dict(gq=heads(n=7)), dict(gk=heads(data=ODD)), dict(wsb=ws - 1), dict(wsp=None)):
        p = m._HeadNormC(**base)
        a = dict(gq=heads(), gk=heads(), wsb=ws, wsp=FAKE) | o
        h = heads()
        ref = ctypes.byref
        assert lib.qk_norm_rope_bwd(ref(p), ref(a["gq"]), ref(a["gk"]), ref(h), ref(h), ref(h), ref(h), FAKE, FAKE,
                                    a["wsp"], a["wsb"], None) == INVALID, o


def test_distill_refuses():
    lib = m.library()
    base = dict(z=FAKE, dt=m.NF4_BF16, t=4, v=100, ld=100, idx=FAKE, y=FAKE, top=8, tau=2.0)

    def calls(out=FAKE, ldd=100, loss=FAKE, lse=FAKE, w=FAKE, **o):
        a = base | o
        head = (a["z"], a["dt"], a["t"], a["v"], a["ld"], a["idx"], a["y"], a["top"], a["tau"])
        return (lib.distill_topk_fwd(*head, loss, lse, None), lib.distill_topk_bwd(*head, lse, w, out, ldd, None),
                lib.distill_topk_step(*head, w, loss, out, ldd, None))

    for o in (dict(z=None), dict(z=ODD), dict(idx=None), dict(idx=ctypes.c_void_p(4098)), dict(y=None), dict(dt=5), dict(t=-1),
              dict(v=0), dict(ld=99), dict(top=0), dict(top=1025), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
              dict(tau=float("inf")), dict(tau=1e-45)):
        assert calls(**o) == (INVALID,) * 3, o
    assert calls(t=2 ** 31) == (UNSUPPORTED,) * 3 and calls(v=2 ** 30, ld=2 ** 30) == (UNSUPPORTED,) * 3
    a = (FAKE, m.NF4_BF16, 4, 100, 100, FAKE, FAKE, 8, 2.0)
    assert lib.distill_topk_fwd(*a, None, FAKE, None) == INVALID
    assert lib.distill_topk_fwd(*a, FAKE, ODD, None) == INVALID
    assert lib.distill_topk_bwd(*a, None, FAKE, FAKE, 100, None) == INVALID
    assert lib.distill_topk_bwd(*a, FAKE, None, FAKE, 100, None) == INVALID
    for call, first in ((lib.distill_topk_bwd, (FAKE, FAKE)), (lib.distill_topk_step, (FAKE, FAKE))):
        assert call(*a, *first, None, 100, None) == INVALID
        assert call(*a, *first, ODD, 100, None) == INVALID
        assert call(*a, *first, FAKE, 99, None) == INVALID
    assert lib.distill_topk_step(*a, ODD, FAKE, FAKE, 100, None) == INVALID
    assert lib.distill_topk_step(*a, FAKE, None, FAKE, 100, None) == INVALID
    # nothing to do is no error and needs no memory
    assert lib.distill_topk_fwd(None, m.NF4_F32, 0, 100, 100, None, None, 8, 1.0, None, None, None) == m.NF4_OK


def test_binding_refuses():
    """The Python layer's own checks: device tensors, shapes, types, contiguous heads and rows."""
    x, ids = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    q = m.NF4Tensor.empty(64, 128, 0, "cpu")
    A, B, s = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16), torch.ones(2)
    with pytest.raises(ValueError, match="device"):
        m.qlora_multi_fwd(x, q, A, B, s, ids)
    with pytest.raises(ValueError, match=r"\[L, r, k\]"):
        m.qlora_multi_fwd(x, q, A[0], B, s, ids)
    h, w = torch.zeros(4, 2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="device"):
        m.qk_norm_rope_fwd(h, None, w, None, None, None, None)
    with pytest.raises(ValueError, match="must be given"):
        m.qk_norm_rope_fwd(None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        m.qk_norm_rope_fwd(h.half(), None, w, None, None, None, None)
    with pytest.raises(ValueError, match="device"):
        m.distill_topk_fwd(torch.zeros(2, 9), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), 1.0)
