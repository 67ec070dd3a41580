"""Norm and rotation of heads through autograd with queries or keys alone, and past 32-bit offsets."""
import pytest
import torch

from tests.test_gpu_headnorm import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot", [64, 0])
@pytest.mark.parametrize("given", ["q", "k"])
def test_autograd_of_one_side(lib, given, rot):
    """q without k and k without q: the gradients are qk_norm_rope_bwd's, in the inputs' types, also where the
    gradient arrives expanded; the weight of the side that is not given may be None or a tensor."""
    q, k, wq, wk, table, gq, gk = inputs(9, 4, 2, 64, rot, "bf16", "bf16", "i32")
    side = 0 if given == "q" else 1
    x, w, g = ((q, wq, gq), (k, wk, gk))[side]
    pair = lambda t: (t, None) if side == 0 else (None, t)
    for grad in (g, torch.ones((), dtype=g.dtype, device=g.device).expand(g.shape)):
        for other in (None, wk if side == 0 else wq):
            xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
            weights = (wl, other) if side == 0 else (other, wl)
            out = lib.QKNormRopeFunction.apply(*pair(xl), *weights, *table)
            assert out[1 - side] is None
            out[side].backward(grad)
            want = lib.qk_norm_rope_bwd(*pair(grad.contiguous()), *pair(x), *pair(w), *table)
            assert torch.equal(xl.grad, want[side]) and torch.equal(wl.grad, want[2 + side].to(w.dtype))
            assert want[1 - side] is None and want[3 - side] is None


def test_offsets_past_32_bits(lib):
    """More than 2^32 bytes and 2^31 elements of q: the last tokens are those of a call for them alone."""
    m, h, d = 530000, 32, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, gq = (torch.randn(m, h, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    ang = torch.rand(100, d // 2, generator=g, device="cuda") * 6
    pos = torch.randint(0, 100, (m,), generator=g, device="cuda")
    y, _ = lib.qk_norm_rope_fwd(q, None, w, None, ang.cos(), ang.sin(), pos)
    dq, _, dw, _ = lib.qk_norm_rope_bwd(gq, None, q, None, w, None, ang.cos(), ang.sin(), pos)
    assert dw.isfinite().all()
    for rows in (slice(0, 5), slice(m - 5, m)):
        args = (q[rows], None, w, None, ang.cos(), ang.sin(), pos[rows])
        assert torch.equal(y[rows], lib.qk_norm_rope_fwd(*args)[0])
        assert torch.equal(dq[rows], lib.qk_norm_rope_bwd(gq[rows], None, *args)[0])
