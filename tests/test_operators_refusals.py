"""Refusals of the head norms' outputs and of the distillation's temperature (no GPU needed): every call below
is invalid by construction, so the host's checks refuse it before a pointer is used or anything is launched."""
import ctypes

import pytest

import nf4_dequant_gemm_amd as m
from tests.test_operators_host import heads

D = 64
FAKE = ctypes.c_void_p(4096)


def calls(q_out=None, k_out=None, tokens=5, hq=8, hk=8):
    """(forward, backward) of 5 tokens of 8 + 8 heads of 64 with these outputs."""
    p = m._HeadNormC(tokens=tokens, d=D, rot=0, interleaved=0, dtype=m.NF4_BF16, w_dtype=m.NF4_F32, wq=4096, wk=4096,
                     w_offset=0.0, eps=1e-6)
    q, k = heads(n=hq), heads(n=hk)
    r = ctypes.byref
    qo, ko = q_out or q, k_out or k
    lib = m.library()
    ws = lib.qk_norm_rope_bwd_workspace_bytes(D)
    return (lib.qk_norm_rope_fwd(r(p), r(q), r(k), r(qo), r(ko), None),
            lib.qk_norm_rope_bwd(r(p), r(q), r(k), r(q), r(k), r(qo), r(ko), FAKE, FAKE, FAKE, ws, None))


@pytest.mark.parametrize("ts,hs", [(0, 64), (512, 0), (0, 0), (63, 512), (512, 63), (64, 64), (512, 512)])
@pytest.mark.parametrize("side", ["q_out", "k_out"])
def test_overlapping_outputs(side, ts, hs):
    """Strides that put two heads of an output on the same place (expanded tensors among them)."""
    assert calls(**{side: heads(ts=ts, hs=hs)}) == (m.NF4_EINVAL, m.NF4_EINVAL)
    assert b"overlap" in m.library().nf4_last_error()


@pytest.mark.parametrize("ts,hs,tokens,n", [(0, 64, 1, 8), (512, 0, 5, 1), (0, 0, 1, 1), (64, 320, 5, 8)])
def test_strides_of_one(ts, hs, tokens, n):
    """The stride of a single token or head says nothing, and heads may lie outermost: such an output passes
    (the call is refused for its other output, so that nothing is launched)."""
    h = heads(ts=ts, hs=hs, n=n)
    assert calls(q_out=h, k_out=heads(data=ctypes.c_void_p(4097)), tokens=tokens, hq=n) == (m.NF4_EINVAL, m.NF4_EINVAL)
    assert b"overlap" not in m.library().nf4_last_error()


@pytest.mark.parametrize("tau", [3.0e-39, 3.5e-39, 4.2e-39])
def test_temperature_whose_scale_overflows(tau):
    """1 / tau is finite, log2(e) / tau is not: every probability would be NaN."""
    assert 1 / ctypes.c_float(tau).value < 3.4028234e38
    lib = m.library()
    head = (FAKE, m.NF4_BF16, 4, 100, 100, FAKE, FAKE, 8, tau)
    assert lib.distill_topk_fwd(*head, FAKE, FAKE, None) == m.NF4_EINVAL
    assert lib.distill_topk_bwd(*head, FAKE, FAKE, FAKE, 100, None) == m.NF4_EINVAL
    assert lib.distill_topk_step(*head, FAKE, FAKE, FAKE, 100, None) == m.NF4_EINVAL
