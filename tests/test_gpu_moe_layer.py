"""The operators of the mixture-of-experts layer together: their autograd functions against float64 autograd, the
captured and replayed run, other streams, and the example."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"


def layer(lib, t, d, hidden, E, top, r, seed):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)
    q = lib.nf4_quantize(normal(E * hidden, d, std=d ** -0.5).bfloat16())
    return (normal(t, d).bfloat16(), normal(E, d, std=d ** -0.5), q, normal(E * r, d, std=d ** -0.5).bfloat16(),
            normal(E * hidden, r, std=0.05).bfloat16(), normal(t, hidden).bfloat16())


def reference(lib, X, router, q, A, B, s, idx, dY, losses, renorm):
    """Loss and gradients in float64 of sum(dY * Y) + losses, with the choices idx."""
    E, top = router.shape[0], idx.shape[1]
    W = lib.nf4_dequantize(q, torch.float32).double().view(E, -1, q.k)
    X, router, A, B = (z.detach().double().requires_grad_() for z in (X, router, A, B))
    x = X @ router.t()
    p = x.softmax(1)
    live = idx[:, 0] >= 0
    at = idx.long().clamp(min=0)
    gate = torch.gather(x, 1, at).softmax(1) if renorm else torch.gather(p, 1, at)
    gate = gate * live[:, None]
    Ar, Br = A.view(E, -1, q.k), B.view(E, W.shape[1], -1)
    Y = torch.zeros(X.shape[0], W.shape[1], dtype=torch.double, device=DEV)
    for e in range(E):
        full = X @ W[e].t() + s * (X @ Ar[e].t()) @ Br[e].t()
        Y = Y + ((idx == e) * gate).sum(1, keepdim=True) * full
    n = live.sum()
    counts = torch.stack([(idx == e).sum() for e in range(E)]).double()
    balance = E * (counts / counts.sum() * (p * live[:, None]).sum(0) / n).sum()
    z = (x.logsumexp(1).square() * live).sum() / n
    total = (dY.double() * Y).sum() + losses[0] * balance + losses[1] * z
    return Y, torch.autograd.grad(total, (X, router, A, B))


@pytest.mark.parametrize("t,d,hidden,E,top,r,renorm,eight", [(1, 128, 64, 4, 1, 4, True, True), (200, 256, 136, 8, 2, 8, True, True),
                                                             (333, 192, 72, 5, 3, 16, False, False), (64, 64, 264, 16, 4, 8, False, True)])
def test_gradients(lib, t, d, hidden, E, top, r, renorm, eight):
    """Outputs and gradients within the bf16 roundings on the way: of the gathered weight, T, Y, Z's and dZ's rows,
    U and the kept activation, each 2^-8 relative at most and independent: 2^-7 in norm. The 8-bit form adds half
    a step of 127 (below 2^-6 of an element's size in norm) to dA alone."""
    say(f"moe layer t={t} d={d} E={E} top={top}")
    X, router, q, A, B, dY = layer(lib, t, d, hidden, E, top, r, t)
    keep = torch.arange(t, device=DEV) % 7 != 5
    leaves = [z.clone().requires_grad_() for z in (X, router, A, B)]
    x, w, a, b = leaves
    ro = lib.MoERouting(*lib.MoERouteFunction.apply(x.float() @ w.t(), top, keep, renorm))
    rows = lib.MoEGatherFunction.apply(x, ro.place, ro.source)
    kept = lib.act8_pack(X) if eight else None
    Z = lib.QLoRAMoEFunction.apply(rows, q, a, b, 1.5, ro.counts, kept, ro.source if eight else None)
    Y = lib.MoECombineFunction.apply(Z, ro.place, ro.source, ro.gate)
    coef = (3.0, 0.5)
    ((dY * Y).float().sum() + coef[0] * ro.losses[0] + coef[1] * ro.losses[1]).backward()
    want, grads = reference(lib, X, router, q, A, B, 1.5, ro.idx, dY, coef, renorm)
    near = lambda name, got, ref, tol: (lambda e: (say(f"  {name} {e:.1e}"), e)[1])(
        float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())) <= tol
    assert near("Y", Y, want, 2.0 ** -7) and not Y[~keep].any()
    for name, leaf, g in zip(("X", "router", "A", "B"), leaves, grads):
        assert near(name, leaf.grad, g, 2.0 ** -7 + (2.0 ** -6 if name == "A" and eight else 0)), name


def test_linear_and_pair_functions(lib):
    """The layers that keep their activations in 8 bits: outputs as the bf16 layers', gradients theirs from the
    unpacked activation."""
    g = torch.Generator().manual_seed(1)
    normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().to(DEV)
    m, k, n, r = 130, 192, 72, 8
    X, dY = normal(m, k), normal(m, n)
    q, q2 = lib.nf4_quantize(normal(n, k, std=0.05)), lib.nf4_quantize(normal(2 * n, k, std=0.05))
    A, B, Bu, Agu = normal(r, k, std=0.1), normal(n, r, std=0.1), normal(n, r, std=0.1), normal(2 * r, k, std=0.1)
    grad = lambda f, q, *a: (lambda z: (f.apply(z[0], q, *z[1:], 0.5), z))([x.clone().requires_grad_() for x in a])
    Y, z = grad(lib.QLoRALinearAct8Function, q, X, A, B)
    Y.backward(dY)
    Y0, T = lib.qlora_fwd(X, q, A, B, 0.5)
    want = lib.qlora_bwd_act8(dY, lib.act8_pack(X), q, A, B, 0.5, T)
    assert torch.equal(Y, Y0) and all(torch.equal(a.grad, b) for a, b in zip(z, want))
    H, z = grad(lib.QLoRASwiGLUAct8Function, q2, X, Agu, B, Bu)
    H.backward(dY)
    H0, Ygu, Tgu = lib.qlora_swiglu_fwd(X, q2, Agu, B, Bu, 0.5)
    want = lib.qlora_swiglu_bwd_act8(dY, lib.act8_pack(X), q2, Agu, B, Bu, 0.5, lib.act8_pack(Ygu), Tgu)
    assert torch.equal(H, H0) and all(torch.equal(a.grad, b) for a, b in zip(z, want))


def test_moe_function_forms(lib):
    """The grouped function with the rows themselves kept in 8 bits (no source), without adapters, and with an
    input that needs no gradient."""
    X, router, q, A, B, _ = layer(lib, 60, 128, 72, 4, 1, 8, 3)
    counts = torch.tensor([20, 0, 33, 7], device=DEV)
    dY = torch.randn(60, 72, device=DEV).bfloat16()
    leaves = [z.clone().requires_grad_() for z in (X, A, B)]
    kept = lib.act8_pack(X)
    lib.QLoRAMoEFunction.apply(leaves[0], q, leaves[1], leaves[2], 1.0, counts, kept).backward(dY)
    ws = torch.empty(lib.moe_workspace_bytes_dev(60, 4, 72, 128, 8), dtype=torch.uint8, device=DEV)
    Y, T = X.new_empty(60, 72), X.new_empty(60, 8)
    lib.qlora_moe_fwd_dev(X, counts, q, A, B, 1.0, Y, T, ws)
    want = lib.qlora_moe_bwd_act8(dY, kept, None, counts, q, A, B, 1.0, T)
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))
    x = X.clone().requires_grad_()
    for k in (None, kept):
        x.grad = None
        lib.QLoRAMoEFunction.apply(x, q, None, None, 1.0, counts, k).backward(dY)
        assert x.grad.isfinite().all() and (k is None or torch.equal(x.grad, first))
        first = x.grad
    a, b = (z.clone().requires_grad_() for z in (A, B))
    lib.QLoRAMoEFunction.apply(X, q, a, b, 1.0, counts).backward(dY)
    # dB from bf16 rows: the same products in another order of float32 sums (2^-10 of the magnitudes each), and a step
    rows = lambda z: [e.double().abs() for e in z[:60].split(counts.tolist())]
    mag = torch.cat([d.t() @ t for d, t in zip(rows(dY), rows(T))])
    assert ((b.grad.double() - want[2].double()).abs() <= 2.0 ** -7 * want[2].double().abs() + 2.0 ** -9 * mag).all()
    assert a.grad.isfinite().all()


def step(lib, st):
    """A training step's calls, all on the current stream: everything but the logits' product."""
    r = lib.moe_route(st["x"], 2, st["keep"])
    rows = lib.moe_gather(st["X"], r.place, r.source)
    kept = lib.act8_pack(st["X"])
    m, n = rows.shape[0], st["dY"].shape[1]
    Y, T = rows.new_empty(m, n), rows.new_empty(m, 8)
    lib.qlora_moe_fwd_dev(rows, r.counts, st["q"], st["A"], st["B"], 1.0, Y, T, st["ws"])
    out = lib.moe_combine(Y, r.place, r.gate)
    dZ, dgate = lib.moe_combine_bwd(st["dY"], Y, r.place, r.source, r.gate)
    dR, dA, dB = lib.qlora_moe_bwd_act8(dZ, kept, r.source, r.counts, st["q"], st["A"], st["B"], 1.0, T)
    dX = lib.moe_combine(dR, r.place)
    dx = lib.moe_route_bwd(dgate, st["dl"], st["x"], r.idx, r.counts, r.sizes)
    return (*r[:8], out, dA, dB, dX, dx, dgate, lib.act8_unpack(kept))


def state(lib, t, seed):
    E, d, n = 8, 256, 72
    X, router, q, A, B, dY = layer(lib, t, d, n, E, 2, 8, seed)
    return dict(X=X, x=(X.float() @ router.t()), keep=torch.arange(t, device=DEV) % 9 != 4, q=q, A=A, B=B, dY=dY,
                dl=torch.ones(2, device=DEV),
                ws=torch.empty(lib.moe_workspace_bytes_dev(2 * t, E, n, d, 8), dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("t", [40, 300])
def test_captured(lib, t):
    """Two graphs of the step, replayed in turn with other inputs and eager work between: every replay's outputs are
    the eager call's, bit for bit."""
    st = [state(lib, t, s) for s in (1, 2)]
    side, graphs = torch.cuda.Stream(), []
    for s in st:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(lib, s)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(lib, s)
        graphs.append((graph, outs))
    for turn in range(4):
        for s, (graph, outs) in zip(st, graphs):
            fresh = state(lib, t, 10 + turn)
            for name in ("X", "x", "dY"):
                s[name].copy_(fresh[name])
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            want = step(lib, s)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_other_streams(lib):
    """The step on two streams at once equals the step alone."""
    st = [state(lib, t, 5) for t in (3000, 700)]
    want = [step(lib, s) for s in st]
    torch.cuda.synchronize()
    st[1]["ws"] = st[1]["ws"].clone()
    streams = [torch.cuda.Stream() for _ in st]
    for _ in range(5):
        got = []
        for s, z in zip(st, streams):
            with torch.cuda.stream(z):
                got.append(step(lib, s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_example(lib):
    """The example runs, serves what it trained, and its gradients are those of the run that keeps bf16 rows, up to
    the 8-bit activations (half a step of 127 beside the bf16 roundings: within 2^-5 in norm)."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_experts.py")
    spec = importlib.util.spec_from_file_location("moe_experts", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model, losses = ex.train(3, say=lambda *a, **k: None)
    assert all(x == x for x in losses)
    # bf16 activations: a few roundings of 2^-8 per block, in another order of sums
    assert ex.serve(model) < 2.0 ** -5
    data = ex.batch(torch.Generator("cuda").manual_seed(4))
    grads = [torch.autograd.grad(model.loss(*data, eight_bits=e)[0], model.leaves()) for e in (True, False)]
    for a, b in zip(*grads):
        assert b.norm() > 0 and (a - b).norm() <= 2.0 ** -5 * b.norm()


@pytest.mark.parametrize("reduce", [lambda y: y.sum(0), lambda y: y.mean(0, keepdim=True), lambda y: y.sum(1), lambda y: y.sum()],
                         ids=["tokens", "mean of tokens", "columns", "both"])
def test_combine_of_broadcast_gradients(lib, reduce):
    """The gradient of a sum over tokens, over columns or over both comes as an expanded tensor (a stride of 0)."""
    t, d, E, top = 30, 72, 5, 2
    g = torch.Generator(DEV).manual_seed(6)
    ro = lib.moe_route(torch.randn(t, E, generator=g, device=DEV), top, torch.arange(t, device=DEV) % 7 != 5)
    Z, base = (torch.randn(n, d, generator=g, device=DEV) for n in (t * top, t))

    def grads(dense):
        z, b, w = (x.clone().requires_grad_() for x in (Z, base, ro.gate))
        y = lib.MoECombineFunction.apply(z, ro.place, ro.source, w, b)
        if dense is None:
            reduce(y).square().sum().backward()
        else:
            y.backward(dense)
        return y.detach(), z.grad, b.grad, w.grad
    y, *got = grads(None)
    x = y.clone().requires_grad_()
    reduce(x).square().sum().backward()
    _, *want = grads(x.grad.contiguous())
    assert all(a.abs().sum() > 0 and torch.equal(a, b) for a, b in zip(got, want))


def test_combine_without_gates(lib):
    """No gates are ones, in the gradient too; it flows to Z and base."""
    t, d, E, top = 30, 72, 5, 2
    g = torch.Generator(DEV).manual_seed(7)
    ro = lib.moe_route(torch.randn(t, E, generator=g, device=DEV), top, torch.arange(t, device=DEV) % 7 != 5)
    Z, base, dY = (torch.randn(n, d, generator=g, device=DEV) for n in (t * top, t, t))
    outs = []
    for gate in (None, torch.ones_like(ro.gate)):
        z, b = Z.clone().requires_grad_(), base.clone().requires_grad_()
        y = lib.MoECombineFunction.apply(z, ro.place, ro.source, gate, b)
        y.backward(dY)
        outs.append((y.detach(), z.grad, b.grad))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and not outs[0][1][int(ro.sizes[1]):].any()
    z = Z.clone().requires_grad_()
    lib.MoECombineFunction.apply(z, ro.place, ro.source, None).sum(0).backward(dY[0])
    assert torch.equal(z.grad, lib.moe_gather(dY[:1].expand(t, d).contiguous(), ro.place, ro.source))


def test_losses_scaled_in_place(lib):
    """What a caller does to the outputs in place: scaled losses reach the logits scaled; the mean probabilities (summed over
    processes, say) and the places of dropped rows are no part of the gradient."""
    x = torch.randn(30, 6, device=DEV, generator=torch.Generator(DEV).manual_seed(8))
    grads = []
    for in_place in (False, True):
        leaf = x.clone().requires_grad_()
        r = lib.MoERouting(*lib.MoERouteFunction.apply(leaf, 2))
        losses = r.losses
        if in_place:
            losses *= 0.5
            r.mean_p.mul_(2)
            r.place[3] = -1
            r.source.fill_(-1)
        else:
            losses = losses * 0.5
        (losses.sum() + r.gate.square().sum()).backward()
        grads.append(leaf.grad)
    assert grads[0].abs().sum() > 0 and torch.equal(*grads)
