#!/usr/bin/env python3
"""A small mixture-of-experts model on 4-bit bases: trained with a balance loss, its blocks' tokens kept in 8 bits,
then served token by token.

Every block sends a token to TOP of E experts, each a gate, an up and a down projection with a frozen NF4 base
and low-rank adapters. moe_route chooses the experts and gives the counts, moe_gather brings the tokens into
expert order, the grouped layers (QLoRAMoEFunction) run all experts at once, and moe_combine adds their outputs,
weighted by the gates, to the token. The gate and up projections keep for their backward pass not the gathered
rows but the tokens, once, in 8 bits; their outputs, and what the down projection and the gates need, stay in bf16. The loss is that of the next token plus the balance and z losses of the
routers.

    python examples/moe_experts.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nf4_dequant_gemm_amd as nq  # noqa: E402

VOCAB, MODEL, HIDDEN, E, TOP, RANK, BLOCKS, S = 500, 256, 192, 8, 2, 8, 2, 2.0
BALANCE, Z = 0.02, 0.001


def _rms(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Block:
    """The experts of one block: frozen bases, adapters, router."""

    def __init__(self, normal):
        shapes = {"gate": (HIDDEN, MODEL), "up": (HIDDEN, MODEL), "down": (MODEL, HIDDEN)}
        self.base = {n: nq.nf4_quantize(normal(E * o, i, std=i ** -0.5).bfloat16()) for n, (o, i) in shapes.items()}
        leaf = lambda x: x.requires_grad_()
        self.A = {n: leaf(normal(E * RANK, i, std=i ** -0.5)) for n, (o, i) in shapes.items()}
        self.B = {n: leaf(normal(E * o, RANK, std=0.02)) for n, (o, i) in shapes.items()}
        self.router = leaf(normal(E, MODEL, std=MODEL ** -0.5))

    def leaves(self):
        return [*self.A.values(), *self.B.values(), self.router]

    def experts(self, name, x, counts, kept=None, source=None):
        return nq.QLoRAMoEFunction.apply(x, self.base[name], self.A[name].bfloat16(), self.B[name].bfloat16(), S, counts,
                                         kept, source)

    def __call__(self, x, keep=None, eight_bits=True):
        """x [tokens, MODEL] -> (x plus its experts' outputs, the router's two losses); tokens whose keep is 0 pass
        through as they are."""
        h = _rms(x)
        r = nq.MoERouting(*nq.MoERouteFunction.apply(h.float() @ self.router.t(), TOP, keep))
        rows = nq.MoEGatherFunction.apply(h, r.place, r.source)
        kept = nq.act8_pack(h.detach()) if eight_bits else None
        source = r.source if eight_bits else None
        g, u = (self.experts(n, rows, r.counts, kept, source) for n in ("gate", "up"))
        z = self.experts("down", torch.nn.functional.silu(g) * u, r.counts)
        return nq.MoECombineFunction.apply(z, r.place, r.source, r.gate, x), r.losses


class Model:
    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        normal = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
        self.embed = normal(VOCAB, MODEL).bfloat16()
        self.head = normal(MODEL, VOCAB, std=MODEL ** -0.5).bfloat16()
        self.blocks = [Block(normal) for _ in range(BLOCKS)]

    def leaves(self):
        return [p for b in self.blocks for p in b.leaves()]

    def __call__(self, tokens, keep=None, eight_bits=True):
        """Logits [tokens, VOCAB] and the sum of the routers' losses [2]."""
        x, losses = self.embed[tokens], 0
        for b in self.blocks:
            x, more = b(x, keep, eight_bits)
            losses = losses + more
        return _rms(x) @ self.head, losses

    def loss(self, tokens, after, keep=None, eight_bits=True):
        logits, losses = self(tokens, keep, eight_bits)
        each = torch.nn.functional.cross_entropy(logits.float(), after, reduction="none")
        weight = torch.ones_like(each) if keep is None else keep.float()
        return (each * weight).sum() / weight.sum() + BALANCE * losses[0] + Z * losses[1], losses


def batch(g, n=512):
    """Tokens, the token that follows each (a fixed permutation of the vocabulary), and a mask of padding."""
    after = torch.randperm(VOCAB, generator=torch.Generator().manual_seed(7)).cuda()
    tokens = torch.randint(0, VOCAB, (n,), generator=g, device="cuda")
    return tokens, after[tokens], torch.rand(n, generator=g, device="cuda") < 0.9


def train(steps, say=print):
    model = Model(1)
    opt = torch.optim.Adam(model.leaves(), lr=2e-3)
    g = torch.Generator("cuda").manual_seed(2)
    losses = []
    for step in range(steps):
        loss, router = model.loss(*batch(g))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if step % 10 == 0 or step == steps - 1:
            say("step %3d  loss %.4f  balance %.3f" % (step, loss.item(), router[0].item() / BLOCKS), flush=True)
    return model, torch.stack(losses).tolist()


@torch.no_grad()
def serve(model, n=12):
    """Tokens one at a time against all of them at once: the largest difference of the logits, relative."""
    tokens = torch.randint(0, VOCAB, (n,), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    whole = model(tokens)[0].float()
    each = torch.cat([model(tokens[i:i + 1])[0] for i in range(n)]).float()
    return ((each - whole).norm() / whole.norm()).item()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=40)
    a = p.parse_args(argv)
    model, losses = train(a.steps)
    print("loss %.4f -> %.4f over %d steps" % (losses[0], losses[-1], a.steps))
    print("served token by token: logits within %.1e of the batch's" % serve(model))


if __name__ == "__main__":
    main()
