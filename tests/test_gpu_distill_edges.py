"""Distillation from a teacher's top logits at the values and sizes where a running maximum and sum can
go wrong: NaN beside masked logits, rows whose mask leaves nothing, more rows than one dimension of a
launch."""
import pytest
import torch

from tests.gpu_helpers import say
from tests.test_gpu_distill import DEV, check, inputs

pytestmark = pytest.mark.gpu

# rows of each launch: one chunk a thread and less, in registers of 64, 256, 512 and 1024 threads, walked
LENGTHS = [9, 400, 1000, 8191, 20001, 50001, 140003]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("v", LENGTHS)
def test_nan_logits_are_not_hidden(lib, v, dt):
    """A NaN makes its row's loss, lse and whole gradient NaN wherever it lies: alone among ordinary
    logits, in a run that fills whole 16-byte chunks, and among logits that are otherwise masked with -inf
    (all but one, elsewhere in the row). The other rows keep their values bit for bit."""
    say(f"distill NaN v={v} {dt}")
    t, top = 12, 4
    z, idx, teacher, w = inputs(t, v, top, dt)
    idx[:] = torch.arange(top) + v - top              # the teacher's entries: the row's last logits
    clean = z.clone()
    bad = {0: v // 2, 1: 0, 2: v - top - 1, 3: min(16, v // 3)}
    for row, at in bad.items():
        z[row, at] = float("nan")
    z[4, :v // 2] = float("nan")
    z[5] = float("nan")
    for row, at in ((6, 0), (7, v // 2), (8, min(8 * 70, v - top - 1))):
        z[row] = float("-inf")
        z[row, at] = float("nan")
        z[row, v - top:] = 1.0
    clean, z, idx, teacher, w = (x.to(DEV) for x in (clean, z, idx, teacher, w))
    rest = torch.arange(9, t, device=DEV)
    loss, lse = lib.distill_topk_fwd(z, idx, teacher, 2.0)
    step_loss, step_grad = lib.distill_topk_step(z, idx, teacher, 2.0, w)
    back = lib.distill_topk_bwd(w, z, idx, teacher, 2.0, lse)
    for x in (loss, lse, step_loss):
        assert x[:9].isnan().all(), x[:9]
    for g in (step_grad, back):
        assert g[:9].isnan().all()
    want, want_lse = lib.distill_topk_fwd(clean, idx, teacher, 2.0)
    want_step, want_grad = lib.distill_topk_step(clean, idx, teacher, 2.0, w)
    assert torch.equal(loss[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
    assert torch.equal(step_loss[rest], want_step[rest]) and torch.equal(step_grad[rest], want_grad[rest])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.5, 2.0])
@pytest.mark.parametrize("v", LENGTHS)
def test_rows_far_from_zero(lib, v, tau, dt):
    """Rows masked throughout with the type's lowest value, with -1e9, -1e4 and -1e3, and rows of ordinary
    logits about 1e5 and 300 away from 0: a constant added to a row changes neither its loss nor its
    gradient, so both are held to the values of the row less its maximum (exact in float32 here), by every
    entry point. Only lse moves with the row: in float32 it has lost the sum there, and beside the
    lowest value at tau < 1 it is -inf."""
    say(f"distill far v={v} tau={tau} {dt}")
    z, idx, teacher, w = inputs(7, v, 3, dt)
    low = torch.finfo(z.dtype).min
    for row, x in enumerate((low, -1e9, -1e4, -1e3)):
        z[row] = x
    z[4] += 1e5
    z[5] -= 1e5
    z[6] -= 300
    near = (z.double() - z.double().amax(1, keepdim=True)).float()
    assert torch.equal(near.double(), z.double() - z.double().amax(1, keepdim=True))
    z, near, idx, teacher, w = (x.to(DEV) for x in (z, near, idx, teacher, w))
    loss, lse = lib.distill_topk_fwd(z, idx, teacher, tau)
    step_loss, step_grad = lib.distill_topk_step(z, idx, teacher, tau, w)
    assert torch.equal(loss, step_loss)
    check(near, idx, teacher, w, tau, loss, None, step_grad)
    check(near, idx, teacher, w, tau, None, None, lib.distill_topk_bwd(w, z, idx, teacher, tau, lse))
    x = z.clone().requires_grad_()
    (lib.DistillTopKFunction.apply(x, idx, teacher, tau) * w).sum().backward()
    check(near, idx, teacher, w, tau, None, None, x.grad)


def test_many_short_rows(lib):
    """More than 2^26 rows: with 64 threads a row their number passes 2^32. Rows repeat every 8 (in content and in
    alignment), and so do the results, bit for bit."""
    t, v = 2 ** 26 + 16, 3
    z, idx, teacher, w = (x.to(DEV) for x in inputs(8, v, 1, "bf16"))
    want = lib.distill_topk_fwd(z, idx, teacher, 2.0) + lib.distill_topk_step(z, idx, teacher, 2.0, w)
    want_back = lib.distill_topk_bwd(w, z, idx, teacher, 2.0, want[1])
    many = lambda x: x.repeat((t // 8,) + (1,) * (x.dim() - 1))
    same = lambda got, ref: bool((got.view(t // 8, *ref.shape) == ref).all())
    z, idx, teacher, w = (many(x) for x in (z, idx, teacher, w))
    loss, lse = lib.distill_topk_fwd(z, idx, teacher, 2.0)
    assert same(loss, want[0]) and same(lse, want[1])
    assert same(lib.distill_topk_bwd(w, z, idx, teacher, 2.0, lse), want_back)
    step_loss, grad = lib.distill_topk_step(z, idx, teacher, 2.0, w)
    assert same(step_loss, want[2]) and same(grad, want[3])


def test_offsets_past_32_bits(lib):
    """More than 2^32 bytes and 2^31 elements of logits: the last rows are those of a call for them alone."""
    t, v = 17000, 131073
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn(t, v, generator=g, device=DEV, dtype=torch.bfloat16)
    idx = torch.randint(0, v, (t, 8), generator=g, device=DEV).int()
    teacher, w = torch.randn(t, 8, generator=g, device=DEV), torch.rand(t, generator=g, device=DEV)
    loss, lse = lib.distill_topk_fwd(z, idx, teacher, 2.0)
    back = lib.distill_topk_bwd(w, z, idx, teacher, 2.0, lse)
    step_loss, grad = lib.distill_topk_step(z, idx, teacher, 2.0, w)
    for rows in (slice(0, 8), slice(t - 8, t)):        # rows of the same alignment
        want, want_lse = lib.distill_topk_fwd(z[rows], idx[rows], teacher[rows], 2.0)
        assert torch.equal(loss[rows], want) and torch.equal(lse[rows], want_lse) and torch.equal(step_loss[rows], want)
        assert torch.equal(grad[rows], lib.distill_topk_step(z[rows], idx[rows], teacher[rows], 2.0, w[rows])[1])
        assert torch.equal(back[rows], lib.distill_topk_bwd(w[rows], z[rows], idx[rows], teacher[rows], 2.0, want_lse))
