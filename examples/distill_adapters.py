#!/usr/bin/env python3
"""Several adapters distilled in one batch on one 4-bit base, then served together.

One attention layer and a vocabulary head share an NF4 base among a few jobs, each with a low-rank
adapter of its own for every projection. A batch mixes the rows of all jobs: the projections add each
row's own adapter (QLoRAMultiFunction), queries and keys go through their head norms and the rotation
(QKNormRopeFunction), and the loss is the distance to a teacher of which only the top logits are kept
(DistillTopKFunction). The teacher of a job is the base with an adapter that the student does not see.
Afterwards every job gets one request: its prompt in one call, then one token at a time, one row for
each request, and the logits are compared with those of the whole sequence.

    python examples/distill_adapters.py [--steps 60]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nf4_dequant_gemm_amd as nq  # noqa: E402

VOCAB, MODEL, HQ, HK, D, RANK, JOBS, TOP, TAU = 1000, 256, 4, 2, 64, 8, 3, 32, 1.0
SHAPES = {"q": (HQ * D, MODEL), "k": (HK * D, MODEL), "v": (HK * D, MODEL), "o": (MODEL, HQ * D), "head": (VOCAB, MODEL)}


def _rms(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Model:
    """The frozen base and the adapters of all jobs beside it."""

    def __init__(self, seed, base=None, b_std=0.0):
        g = torch.Generator("cuda").manual_seed(seed)
        normal = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std
        if base is None:
            self.embed = normal(VOCAB, MODEL, std=1.0).bfloat16()
            # a head four times as large gives logits that a few tokens dominate
            self.base = {n: nq.nf4_quantize(normal(*s, std=(4 if n == "head" else 1) * s[1] ** -0.5).bfloat16())
                         for n, s in SHAPES.items()}
            angle = torch.arange(512, device="cuda")[:, None] * 1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)
            self.cos, self.sin = angle.cos(), angle.sin()
        else:
            self.embed, self.base, self.cos, self.sin = base.embed, base.base, base.cos, base.sin
        self.s = torch.full((JOBS,), 2.0, device="cuda")
        leaf = lambda x: x.requires_grad_()
        self.A = {n: leaf(normal(JOBS, RANK, s[1], std=s[1] ** -0.5)) for n, s in SHAPES.items()}
        self.B = {n: leaf(normal(JOBS, s[0], RANK, std=b_std)) for n, s in SHAPES.items()}
        self.wq, self.wk = leaf(torch.ones(D, device="cuda")), leaf(torch.ones(D, device="cuda"))

    def leaves(self):
        return [*self.A.values(), *self.B.values(), self.wq, self.wk]

    def project(self, name, x, ids):
        return nq.QLoRAMultiFunction.apply(x, self.base[name], self.A[name].bfloat16(), self.B[name].bfloat16(),
                                           self.s, ids)

    def logits(self, tokens, ids, pos, cache=None):
        """Logits [sequences, rows, VOCAB] of tokens [sequences, rows] at positions pos [rows], with the job of
        each sequence; cache: keys and values of the positions before, extended in place."""
        n, t = tokens.shape
        rows = ids[:, None].expand(n, t).reshape(-1).contiguous()
        at = pos[None].expand(n, t).reshape(-1).contiguous()
        x = self.embed[tokens.reshape(-1)]
        h = _rms(x)
        q = self.project("q", h, rows).view(n * t, HQ, D)
        k = self.project("k", h, rows).view(n * t, HK, D)
        v = self.project("v", h, rows).view(n, t, HK, D)
        q, k = nq.QKNormRopeFunction.apply(q, k, self.wq, self.wk, self.cos, self.sin, at)
        q, k = q.view(n, t, HQ, D), k.view(n, t, HK, D)
        if cache is not None:
            if cache:
                k, v = torch.cat((cache["k"], k), 1), torch.cat((cache["v"], v), 1)
            cache["k"], cache["v"] = k, v
        # attention is not what this example shows: a plain one in 32 bits
        heads = lambda z: z.float().repeat_interleave(HQ // z.shape[2], 2).transpose(1, 2).contiguous()
        qf, kf, vf = heads(q), heads(k), heads(v)
        score = qf @ kf.transpose(2, 3).contiguous() / math.sqrt(D)
        hidden = torch.arange(kf.shape[2], device="cuda")[None] > pos[:, None]
        a = score.masked_fill(hidden, -math.inf).softmax(-1) @ vf
        a = a.transpose(1, 2).reshape(n * t, HQ * D).bfloat16()
        y = _rms(x + self.project("o", a, rows))
        return self.project("head", y, rows).view(n, t, VOCAB)


def train(steps, say=print):
    """Distils every job's teacher into its adapter; the mean loss of each step."""
    teacher = Model(1, b_std=0.1)
    student = Model(2, base=teacher)
    opt = torch.optim.Adam(student.leaves(), lr=3e-3)
    g = torch.Generator("cuda").manual_seed(3)
    pos = torch.arange(48, device="cuda", dtype=torch.int32)
    # a small training set, and the top of the teacher's logits for it
    tokens = torch.randint(0, VOCAB, (8, 48), generator=g, device="cuda")
    ids = torch.tensor([0, 2, 1, 1, 0, 2, 2, 0], device="cuda", dtype=torch.int32)
    with torch.no_grad():
        top, idx = teacher.logits(tokens, ids, pos).view(-1, VOCAB).float().topk(TOP)
    losses = []
    for step in range(steps):
        z = student.logits(tokens, ids, pos).view(-1, VOCAB)
        loss = nq.DistillTopKFunction.apply(z, idx.int(), top, TAU).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if step % 20 == 0 or step == steps - 1:
            say("step %3d  loss %.4f" % (step, loss.item()), flush=True)
    return student, torch.stack(losses).tolist()


@torch.no_grad()
def serve(model, prompt=20, more=6):
    """One request for every job, prompts in one call and then token by token: the largest difference of the
    logits from those of the whole sequences, relative to their size."""
    g = torch.Generator("cuda").manual_seed(4)
    tokens = torch.randint(0, VOCAB, (JOBS, prompt + more), generator=g, device="cuda")
    ids = torch.arange(JOBS, device="cuda", dtype=torch.int32)
    pos = torch.arange(prompt + more, device="cuda", dtype=torch.int32)
    whole = model.logits(tokens, ids, pos).float()
    cache = {}
    parts = [model.logits(tokens[:, :prompt], ids, pos[:prompt], cache)]
    for i in range(prompt, prompt + more):
        parts.append(model.logits(tokens[:, i:i + 1], ids, pos[i:i + 1], cache))
    return ((torch.cat(parts, 1).float() - whole).norm() / whole.norm()).item()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=60)
    a = p.parse_args(argv)
    student, losses = train(a.steps)
    print("loss %.4f -> %.4f over %d steps" % (losses[0], losses[-1], a.steps))
    print("served token by token: logits within %.1e of the whole sequence's" % serve(student))


if __name__ == "__main__":
    main()
