"""Cases, plain forms and 64-bit values of the operators around the grouped (mixture-of-experts) layer
and of training with 8-bit activation checkpoints, timed and checked together:

* route: the choice of experts for every token, their gates, the rows' places in expert order, the
  counts, the balance and the z loss; with the gradient of the logits;
* rows: tokens taken into expert order and the experts' outputs joined again; with their gradients;
* pack: an activation put into 8 bits and taken out again;
* linear8, pair8, moe8: the activation of a 4-bit layer (of the gate/up pair, of the grouped layer) put
  into 8 bits, and the layer's backward pass from it.

`own` False computes them with elementary torch operations in 32 bits, rounded once at the end (the 8-bit
codes of float32 values in 64, since a value next to the border of two codes takes either in 32); True
calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64      # elements with one scale

# The 16 NF4 levels: the float32 values that the format fixes.
LEVELS = [-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
          -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
          0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045,
          0.722956657409668, 1.0]


def listed():
    return [
        # one token of one request: the smallest call, latency only
        dict(name="route_token", op="route", t=1, E=128, top=8, dt="f32", renorm=True, pad=0.0, bwd=False),
        # a ragged batch with padding, an expert count that is no power of two, gates as they are
        dict(name="route_ragged", op="route", t=1023, E=60, top=4, dt="bf16", renorm=False, pad=0.1, bwd=True),
        # a training batch over many experts, forward and backward
        dict(name="route_train", op="route", t=16384, E=128, top=8, dt="f32", renorm=True, pad=0.0, bwd=True),
        # sixteen requests decoding at once
        dict(name="rows_decode", op="rows", t=16, d=4096, E=8, top=2, dt="bf16", base=True, pad=0.0, bwd=False),
        # a ragged batch with padding, rows that are no multiple of 16 bytes
        dict(name="rows_ragged", op="rows", t=1111, d=1023, E=60, top=6, dt="f32", base=False, pad=0.1, bwd=True),
        # the 8192 tokens and two of 8 experts of the grouped layer's workload, forward and backward
        dict(name="rows_train", op="rows", t=8192, d=4096, E=8, top=2, dt="bf16", base=False, pad=0.0, bwd=True),
        # a short prompt's activation
        dict(name="pack_short", op="pack", m=17, k=4096, dt="bf16"),
        # the input of the down projection in training
        dict(name="pack_down", op="pack", m=16384, k=14336, dt="bf16"),
        # the first trained layer of a stack (its input needs no gradient) on the mlp_up shape
        dict(name="linear8_mlp_up", op="linear8", m=8192, k=4096, n=11008, r=64, dx=False),
        # the down projection's adapter gradients
        dict(name="linear8_down", op="linear8", m=16384, k=14336, n=4096, r=32, dx=False),
        # a small gate/up pair with odd sizes, the whole backward pass
        dict(name="pair8_ragged", op="pair8", m=1000, k=1088, n=1416, r=8, dx=True),
        # the grouped layer's workload, its input kept once for each token
        dict(name="moe8_mlp_up", op="moe8", t=8192, k=4096, n=11008, E=8, top=2, r=16),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; the round sizes (multiples of 1024) are among the listed cases."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return x - (x % 1024 == 0)


def draw(rng):
    op = rng.choice(["route", "route", "rows", "rows", "pack", "linear8", "pair8", "moe8"])
    if op == "route":
        E = rng.choice([2, 8, 16, 30, 60, 64, 72, 128, 160, 256])
        return dict(op=op, t=_log(rng, 1, 16384), E=E, top=rng.randint(1, min(E, 12)), dt=rng.choice(["bf16", "f32"]),
                    renorm=rng.random() < 0.6, pad=rng.choice([0.0, 0.0, 0.2]), bwd=rng.random() < 0.6)
    if op == "rows":
        E = rng.choice([4, 8, 60, 128])
        top, dt = rng.randint(1, 4 if E < 60 else 8), rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([64, 257, 768, 1000, 2048, 2880, 4096, 5120])
        t = _log(rng, 1, min(8192, 8192 * 4096 * 2 // (d * top * (2 if dt == "f32" else 1))))
        return dict(op=op, t=t, d=d, E=E, top=top, dt=dt, base=rng.random() < 0.4, pad=rng.choice([0.0, 0.2]),
                    bwd=rng.random() < 0.6)
    if op == "pack":
        k, dt = rng.choice([64, 100, 777, 2048, 4096, 11008, 14336]), rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, m=_log(rng, 1, min(16384, 2 * 10 ** 8 // k)), k=k, dt=dt)
    k = 64 * rng.choice([4, 9, 17, 32, 45, 64, 80])
    n = 8 * rng.choice([32, 37, 101, 177, 256, 369, 512])
    if op == "moe8":
        return dict(op=op, t=_log(rng, 1, 4096), k=k, n=n, E=rng.choice([2, 5, 8, 16]), top=rng.randint(1, 2),
                    r=rng.choice([4, 8, 16, 32]))
    return dict(op=op, m=_log(rng, 1, 8192), k=k, n=n, r=rng.choice([4, 8, 16, 20, 32, 64]), dx=rng.random() < 0.5)


# ---------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _act(g, m, k, dtype=torch.bfloat16):
    """An activation: normal, its channels of different size, a few of them far larger."""
    size = torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))
    size = torch.where(torch.rand(k, generator=g, device=DEV) < 0.004, 12 * size, size)
    return (torch.randn(m, k, generator=g, device=DEV) * size).to(dtype)


def _nf4(g, n, k):
    """A normal weight in NF4: codes (first element in the high nibble), int8 block constants, run scales."""
    w = torch.randn(n * k // 64, 64, generator=g, device=DEV) * 0.02
    a = w.abs().amax(1)
    lv = torch.tensor(LEVELS, device=DEV)
    c = torch.bucketize(w / a[:, None], (lv[1:] + lv[:-1]) / 2, out_int32=True).to(torch.uint8).view(-1, 2)
    S = torch.nn.functional.pad(a, (0, (-a.numel()) % 256)).view(-1, 256).amax(1) / 127
    q = torch.round(a / S.repeat_interleave(256)[:a.numel()]).clamp(0, 127).to(torch.int8)
    return (c[:, 0] << 4) | c[:, 1], q, S


def _routing(g, t, E, top, pad):
    """The experts of every token (distinct, popular and rare ones; -1 where it is padding), the places of
    its rows in expert order, the token of every row (-1 behind the last) and the experts' counts."""
    taste = torch.randn(t, E, generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    idx = taste.topk(top, dim=1).indices
    if pad:
        gone = torch.rand(t, generator=g, device=DEV) < pad
        idx = torch.where(gone[:, None], -1, idx)
    return (idx,) + _order(idx, E)


def _order(idx, E):
    flat = torch.where(idx < 0, E, idx).reshape(-1)
    order = torch.sort(flat, stable=True).indices                # by expert, then by token
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    place = torch.where(flat < E, place, -1).view(idx.shape)
    source = torch.where(flat[order] < E, order // idx.shape[1], -1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    return place.to(torch.int32), source.to(torch.int32), counts


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    dt = torch.float32 if case.get("dt") == "f32" else torch.bfloat16
    if op == "route":
        t, E, top = case["t"], case["E"], case["top"]
        st["logits"] = (1.5 * torch.randn(t, E, generator=g, device=DEV)
                        + torch.randn(E, generator=g, device=DEV)).to(dt)
        st["keep"] = None
        if case["pad"]:      # padding, but for the first token
            st["keep"] = (torch.rand(t, generator=g, device=DEV) >= case["pad"]) | (torch.arange(t, device=DEV) == 0)
        if case["bwd"]:
            st["dgate"] = _normal(g, (t, top), 1.0, torch.float32)
            st["dlosses"] = torch.tensor([0.01, 0.001], device=DEV) * t      # beside a loss summed over tokens
    elif op == "rows":
        t, d, top = case["t"], case["d"], case["top"]
        _, st["place"], st["source"], _ = _routing(g, t, case["E"], top, case["pad"])
        st["X"] = _act(g, t, d, dt)
        st["Z"] = _normal(g, (t * top, d), 1.0, dt)
        st["gate"] = torch.softmax(torch.randn(t, top, generator=g, device=DEV), 1)
        st["bias"] = _normal(g, (t, d), 1.0, dt) if case["base"] else None      # what a shared expert gave
        if case["bwd"]:
            st["dY"] = _normal(g, (t, d), 1.0, dt)
            st["dXg"] = _normal(g, (t * top, d), 1.0, dt)
    elif op == "pack":
        st["X"] = _act(g, case["m"], case["k"], dt)
    elif op == "moe8":
        t, k, n, E, top, r = (case[x] for x in ("t", "k", "n", "E", "top", "r"))
        _, _, st["source"], st["counts"] = _routing(g, t, E, top, 0.0)
        m = t * top
        st["X"] = _act(g, t, k)
        st["W"] = _nf4(g, E * n, k)
        st["A"], st["B"] = _normal(g, (E * r, k), k ** -0.5), _normal(g, (E * n, r), 0.01)
        st["T"], st["dY"] = _normal(g, (m, r), 1.0), _normal(g, (m, n), 1.0)
        st["s"] = 2.0
    else:
        m, k, n, r = (case[x] for x in ("m", "k", "n", "r"))
        pair = op == "pair8"
        st["X"] = _act(g, m, k)
        st["W"] = _nf4(g, (2 if pair else 1) * n, k)
        st["A"] = _normal(g, ((2 if pair else 1) * r, k), k ** -0.5)
        st["T"] = _normal(g, (m, (2 if pair else 1) * r), 1.0)
        st["B"] = _normal(g, (n, r), 0.01)
        st["dY"] = _normal(g, (m, n), 1.0)
        st["s"] = 0.5
        if pair:
            st["B2"], st["Ygu"] = _normal(g, (n, r), 0.01), _act(g, m, 2 * n)
    return st


# ---------------------------------------------------------------------------------- one pass
def run(st):
    return _LIB[st["op"]](st) if own else _PLAIN[st["op"]](st)


def _lib_route(st):
    import nf4_dequant_gemm_amd as nq
    r = nq.moe_route(st["logits"], st["top"], st["keep"], st["renorm"])
    out = {"idx": r.idx, "gate": r.gate, "place": r.place, "source": r.source, "counts": r.counts, "sizes": r.sizes,
           "mean_p": r.mean_p, "losses": r.losses}
    if st["bwd"]:
        out["dlogits"] = nq.moe_route_bwd(st["dgate"], st["dlosses"], st["logits"], r.idx, r.counts, r.sizes, st["renorm"])
    return out


def _lib_rows(st):
    import nf4_dequant_gemm_amd as nq
    out = {"Xg": nq.moe_gather(st["X"], st["place"], st["source"]),
           "Y": nq.moe_combine(st["Z"], st["place"], st["gate"], st["bias"])}
    if st["bwd"]:
        out["dZ"], out["dgate"] = nq.moe_combine_bwd(st["dY"], st["Z"], st["place"], st["source"], st["gate"])
        out["dX"] = nq.moe_combine(st["dXg"], st["place"])
    return out


def _lib_pack(st):
    import nf4_dequant_gemm_amd as nq
    return nq.act8_unpack(nq.act8_pack(st["X"]), st["X"].dtype)


def _weight(st, rows):
    import nf4_dequant_gemm_amd as nq
    return nq.NF4Tensor(rows, st["k"], 256, *st["W"])


def _lib_linear8(st):
    import nf4_dequant_gemm_amd as nq
    dX, dA, dB = nq.qlora_bwd_act8(st["dY"], nq.act8_pack(st["X"]), _weight(st, st["n"]), st["A"], st["B"], st["s"],
                                   st["T"], need_dx=st["dx"])
    return {"dA": dA, "dB": dB, "dX": dX} if st["dx"] else {"dA": dA, "dB": dB}


def _lib_pair8(st):
    import nf4_dequant_gemm_amd as nq
    dX, dA, dB, dB2 = nq.qlora_swiglu_bwd_act8(st["dY"], nq.act8_pack(st["X"]), _weight(st, 2 * st["n"]), st["A"], st["B"],
                                               st["B2"], st["s"], nq.act8_pack(st["Ygu"]), st["T"], need_dx=st["dx"])
    return {"dA": dA, "dB": dB, "dB2": dB2, "dX": dX} if st["dx"] else {"dA": dA, "dB": dB, "dB2": dB2}


def _lib_moe8(st):
    import nf4_dequant_gemm_amd as nq
    _, dA, dB = nq.qlora_moe_bwd_act8(st["dY"], nq.act8_pack(st["X"]), st["source"], st["counts"],
                                      _weight(st, st["E"] * st["n"]), st["A"], st["B"], st["s"], st["T"], need_dx=False)
    return {"dA": dA, "dB": dB}


_LIB = {"route": _lib_route, "rows": _lib_rows, "pack": _lib_pack, "linear8": _lib_linear8, "pair8": _lib_pair8,
        "moe8": _lib_moe8}


def _plain_route(st):
    x, E, top = st["logits"].float(), st["E"], st["top"]
    keep = torch.ones(st["t"], dtype=torch.bool, device=DEV) if st["keep"] is None else st["keep"]
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    val, idx = val[:, :top], torch.where(keep[:, None], idx[:, :top], -1)
    e = (x - val[:, :1]).exp()
    lse = val[:, 0] + e.sum(1).log()
    p = e / e.sum(1, keepdim=True)
    chosen = (val - val[:, :1]).exp()
    gate = chosen / (chosen.sum(1, keepdim=True) if st["renorm"] else e.sum(1, keepdim=True))
    gate = torch.where(keep[:, None], gate, 0.0)
    place, source, counts = _order(idx, E)
    n = keep.sum()
    mean_p = torch.where(keep[:, None], p, 0.0).sum(0) / n
    share = counts.float() / counts.sum()
    losses = torch.stack(((share * mean_p).sum() * E, torch.where(keep, lse * lse, 0.0).sum() / n))
    out = {"idx": idx.to(torch.int32), "gate": gate, "place": place, "source": source, "counts": counts,
           "sizes": torch.stack((n, counts.sum())), "mean_p": mean_p, "losses": losses}
    if st["bwd"]:
        dp = (share * E * st["dlosses"][0] / n).expand_as(p)
        dg, at = st["dgate"], idx.clamp(min=0)
        if not st["renorm"]:
            dp = dp.scatter_add(1, at, dg)
        dx = p * (dp - (p * dp).sum(1, keepdim=True)) + p * (2 * st["dlosses"][1] / n * lse)[:, None]
        if st["renorm"]:
            dx = dx.scatter_add(1, at, gate * (dg - (gate * dg).sum(1, keepdim=True)))
        out["dlogits"] = torch.where(keep[:, None], dx, 0.0).to(st["logits"].dtype)
    return out


def _take(rows, at):
    """rows[at] in 32 bits, zeros where at is negative."""
    return torch.where((at < 0)[..., None], 0.0, rows[at.clamp(min=0).long()].float())


def _plain_rows(st):
    dt, gate = st["X"].dtype, st["gate"]
    y = torch.zeros(st["t"], st["d"], device=DEV) if st["bias"] is None else st["bias"].float()
    for j in range(st["top"]):
        y = y + gate[:, j, None] * _take(st["Z"], st["place"][:, j])
    out = {"Xg": _take(st["X"], st["source"]).to(dt), "Y": y.to(dt)}
    if st["bwd"]:
        live = st["place"] >= 0
        of = torch.zeros(st["t"] * st["top"], device=DEV)
        of[st["place"][live].long()] = gate[live]
        out["dZ"] = (of[:, None] * _take(st["dY"], st["source"])).to(dt)
        dY, dX, dg = st["dY"].float(), 0, []
        for j in range(st["top"]):
            dg.append((dY * _take(st["Z"], st["place"][:, j])).sum(1))
            dX = dX + _take(st["dXg"], st["place"][:, j])
        out["dgate"], out["dX"] = torch.stack(dg, 1), dX.to(dt)
    return out


def _held(x):
    """What the 8-bit form of x [m, k] stands for, in 32 bits."""
    m, k = x.shape
    dt = torch.float32 if x.dtype == torch.bfloat16 else torch.float64
    b = torch.nn.functional.pad(x, (0, (-k) % BLOCK)).view(m, -1, BLOCK)
    a = b.abs().amax(2, keepdim=True)
    a = torch.where(a < 2.0 ** -119, 0.0, a)
    code = torch.where(a > 0, torch.round(b.to(dt) * 127 / a.to(dt)), 0.0)       # ties to even
    return (code.float() * (a.float() / 127)).view(m, -1)[:, :k]


def _plain_pack(st):
    return _held(st["X"]).to(st["X"].dtype)


def _plain_weight(st):
    codes, absmax, scale = st["W"]
    c = torch.stack((codes >> 4, codes & 15), 1).view(-1)
    a = absmax.float() * scale.repeat_interleave(256)[:absmax.numel()]
    return (torch.tensor(LEVELS, device=DEV)[c.int()].view(-1, 64) * a[:, None]).view(-1, st["k"])


def _plain_linear8(st):
    X, dY, A, B, s = _held(st["X"]), st["dY"].float(), st["A"].float(), st["B"].float(), st["s"]
    U = dY @ B
    out = {"dA": (s * (U.t() @ X)).bfloat16(), "dB": (s * (dY.t() @ st["T"].float())).bfloat16()}
    if st["dx"]:
        out["dX"] = (dY @ _plain_weight(st) + s * (U @ A)).bfloat16()
    return out


def _plain_pair8(st):
    X, dH, A, s, n, r = _held(st["X"]), st["dY"].float(), st["A"].float(), st["s"], st["n"], st["r"]
    y = _held(st["Ygu"])
    g, u = y[:, :n], y[:, n:]
    sig = 1 / (1 + (-g).exp())
    dg, du = dH * u * sig * (1 + g * (1 - sig)), dH * g * sig
    T, B, B2 = st["T"].float(), st["B"].float(), st["B2"].float()
    U = torch.cat((dg @ B, du @ B2), 1)
    out = {"dA": (s * (U.t() @ X)).bfloat16(), "dB": (s * (dg.t() @ T[:, :r])).bfloat16(),
           "dB2": (s * (du.t() @ T[:, r:])).bfloat16()}
    if st["dx"]:
        out["dX"] = (torch.cat((dg, du), 1) @ _plain_weight(st) + s * (U @ A)).bfloat16()
    return out


def _plain_moe8(st):
    # every expert's ranks side by side, and each row keeps those of its own expert
    E, n, r, s = st["E"], st["n"], st["r"], st["s"]
    m = st["dY"].shape[0]
    of = torch.repeat_interleave(torch.arange(E, device=DEV), st["counts"], output_size=m)
    X = _held(st["X"])[st["source"].long()]
    dY, T = st["dY"].float(), st["T"].float()
    mine = torch.arange(E, device=DEV).repeat_interleave(r) == of[:, None]                   # [m, E r]
    U = torch.where(mine, dY @ st["B"].float().view(E, n, r).permute(1, 0, 2).reshape(n, E * r), 0.0)
    dA = s * (U.t() @ X)
    dB = s * (dY.t() @ torch.where(mine, T.repeat(1, E), 0.0))                               # [n, E r]
    return {"dA": dA.bfloat16(), "dB": dB.view(n, E, r).permute(1, 0, 2).reshape(E * n, r).bfloat16()}


_PLAIN = {"route": _plain_route, "rows": _plain_rows, "pack": _plain_pack, "linear8": _plain_linear8,
          "pair8": _plain_pair8, "moe8": _plain_moe8}


# ------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    e = 4 if case.get("dt") == "f32" else 2
    if op == "route":
        t, E, top = case["t"], case["E"], case["top"]
        by, fl = t * E * e + t * top * 16 + 12 * E, t * E * (8 + top)
        if case["bwd"]:
            by, fl = by + 2 * t * E * e + t * top * 8, fl + 16 * t * E
        return {"bytes": by, "flops": fl}
    if op == "rows":
        t, d, top = case["t"], case["d"], case["top"]
        by = e * t * d * (2 + 2 * top + (1 if case["base"] else 0)) + t * top * 12
        fl = 2 * t * top * d
        if case["bwd"]:     # dY, Z and the rows' gradients read, dZ and dX written
            by, fl = by + e * t * d * (2 + 3 * top) + t * top * 20, fl + 4 * t * top * d
        return {"bytes": by, "flops": fl}
    if op == "pack":
        m, k = case["m"], case["k"]
        return {"bytes": int(m * k * (2 * e + 2 * (1 + 4 / BLOCK))), "flops": 5 * m * k}
    k, n, r = case["k"], case["n"], case["r"]
    held = 2 * (1 + 4 / BLOCK)                                       # codes and scales written, and read again
    if op == "moe8":
        m, E = case["t"] * case["top"], case["E"]
        by = case["t"] * k * (2 + held) + 2 * m * (n + r) + 4 * m + 2 * E * r * (k + 2 * n)
        return {"bytes": int(by), "flops": 2 * m * r * (k + 2 * n)}
    m = case["m"]
    if op == "linear8":
        by = m * k * (2 + held) + 2 * m * (n + r) + 2 * r * (k + 2 * n)
        fl = 2 * m * r * (k + 2 * n)
        if case["dx"]:
            by, fl = by + n * k * (0.5 + 1 / 64) + 2 * m * k + 2 * r * k, fl + 2 * m * n * k + 2 * m * r * k
        return {"bytes": int(by), "flops": fl}
    by = m * (k + 2 * n) * (2 + held) + 2 * m * (n + 2 * r) + 4 * r * (k + 2 * n)
    fl = 2 * m * r * (2 * k + 4 * n) + 20 * m * n
    if case["dx"]:
        by, fl = by + 2 * n * k * (0.5 + 1 / 64) + 2 * m * k + 4 * r * k, fl + 4 * m * n * k + 4 * m * r * k
    return {"bytes": int(by), "flops": fl}


# ------------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_route(st):
    D = torch.float64
    x = st["logits"].to(D)
    t, E = x.shape
    rows = torch.arange(t, device=DEV) if st["keep"] is None else st["keep"].nonzero()[:, 0]
    n, top = rows.numel(), st["top"]
    x = x[rows]
    # a logit's rank: how many are larger, or equal with a lower index
    rank = torch.empty(n, E, dtype=torch.long, device=DEV)
    lower = torch.ones(E, E, dtype=torch.bool, device=DEV).tril(-1)              # [i, j]: j < i
    for lo in range(0, n, 256):
        a = x[lo:lo + 256]
        rank[lo:lo + 256] = ((a[:, None] > a[:, :, None]) | ((a[:, None] == a[:, :, None]) & lower)).sum(2)
    best = torch.empty(n, top, dtype=torch.long, device=DEV)
    r, c = (rank < top).nonzero(as_tuple=True)
    best[r, rank[r, c]] = c
    p = torch.softmax(x, 1)
    g = torch.take_along_dim(p, best, 1)
    if st["renorm"]:
        g = torch.softmax(torch.take_along_dim(x, best, 1), 1)
    lse = torch.logsumexp(x, 1)
    share = torch.zeros(E, dtype=D, device=DEV)
    share.index_put_((best.reshape(-1),), torch.ones(n * top, dtype=D, device=DEV), accumulate=True)
    share /= n * top
    gate = torch.zeros(t, top, dtype=D, device=DEV)
    gate[rows] = g
    out = {"idx": None, "gate": gate, "place": None, "source": None, "counts": None, "sizes": None, "mean_p": p.mean(0),
           "losses": torch.stack((E * (share * p.mean(0)).sum(), lse.pow(2).mean()))}
    if st["bwd"]:
        db, dz = st["dlosses"].to(D)
        dg = st["dgate"].to(D)[rows]
        dx = p * 2 * dz * lse[:, None] / n
        c = E * share * db / n
        dx += p * (c - (p @ c)[:, None])
        mean = (g * dg).sum(1, keepdim=True)
        at = torch.arange(n, device=DEV)[:, None].expand_as(best)
        if st["renorm"]:
            dx[at, best] += g * (dg - mean)
        else:
            dx -= p * mean
            dx[at, best] += g * dg
        out["dlogits"] = torch.zeros(t, E, dtype=D, device=DEV)
        out["dlogits"][rows] = dx
    return out


def _exact_rows(st):
    D, t, d, top = torch.float64, st["t"], st["d"], st["top"]
    place = st["place"].long()
    token = torch.arange(t, device=DEV)[:, None].expand_as(place)[place >= 0]
    at, gate = place[place >= 0], st["gate"].to(D)[place >= 0]
    out = {"Xg": torch.zeros(t * top, d, dtype=D, device=DEV), "Y": torch.zeros(t, d, dtype=D, device=DEV)}
    out["Xg"][at] = st["X"].to(D)[token]
    if st["bias"] is not None:
        out["Y"] += st["bias"].to(D)
    Z = st["Z"].to(D)
    out["Y"].index_add_(0, token, gate[:, None] * Z[at])
    if st["bwd"]:
        dY = st["dY"].to(D)
        out["dZ"] = torch.zeros_like(out["Xg"])
        out["dZ"][at] = gate[:, None] * dY[token]
        out["dgate"] = torch.zeros(t, top, dtype=D, device=DEV)
        out["dgate"][place >= 0] = torch.linalg.vecdot(dY[token], Z[at])
        out["dX"] = torch.zeros(t, d, dtype=D, device=DEV).index_add_(0, token, st["dXg"].to(D)[at])
    return out


def _exact_held(x):
    m, k = x.shape
    out = torch.empty(m, k, dtype=torch.float64, device=DEV)
    for lo in range(0, k, BLOCK):
        b = x[:, lo:lo + BLOCK].to(torch.float64)
        top = b.abs().max(1, keepdim=True).values
        out[:, lo:lo + BLOCK] = (127 * b / top).round() * (top / 127)
    return out


def _exact_pack(st):
    return _exact_held(st["X"])


def _exact_weight(st):
    D = torch.float64
    codes, absmax, scale = st["W"]
    e = torch.empty(codes.numel() * 2, dtype=torch.long, device=DEV)
    e[0::2], e[1::2] = codes.long() // 16, codes.long() % 16
    a = absmax.to(D) * scale.to(D)[torch.arange(absmax.numel(), device=DEV) // 256]
    return (torch.tensor(LEVELS, dtype=torch.float32, device=DEV).to(D)[e].view(-1, 64) * a[:, None]).reshape(-1, st["k"])


def _exact_linear8(st):
    D, s = torch.float64, st["s"]
    dY = st["dY"].to(D)
    U = s * (dY @ st["B"].to(D))
    out = {"dA": U.T @ _exact_held(st["X"]), "dB": s * (dY.T @ st["T"].to(D))}
    if st["dx"]:
        out["dX"] = dY @ _exact_weight(st) + U @ st["A"].to(D)
    return out


def _exact_pair8(st):
    D, s, n, r = torch.float64, st["s"], st["n"], st["r"]
    y, dH = _exact_held(st["Ygu"]), st["dY"].to(D)
    g, u = y[:, :n], y[:, n:]
    sig = torch.sigmoid(g)
    dg, du = dH * u * (sig + g * sig * (1 - sig)), dH * g * sig
    A, T, X = st["A"].to(D), st["T"].to(D), _exact_held(st["X"])
    Ug, Uu = s * (dg @ st["B"].to(D)), s * (du @ st["B2"].to(D))
    out = {"dA": torch.cat((Ug.T @ X, Uu.T @ X)), "dB": s * (dg.T @ T[:, :r]), "dB2": s * (du.T @ T[:, r:])}
    if st["dx"]:
        W = _exact_weight(st)
        out["dX"] = dg @ W[:n] + du @ W[n:] + Ug @ A[:r] + Uu @ A[r:]
    return out


def _exact_moe8(st):
    D, n, r, s = torch.float64, st["n"], st["r"], st["s"]
    X, lo = _exact_held(st["X"]), 0
    dA, dB = torch.zeros_like(st["A"], dtype=D), torch.zeros_like(st["B"], dtype=D)
    for e, c in enumerate(st["counts"].tolist()):
        g = st["dY"][lo:lo + c].to(D)
        u = s * (g @ st["B"][e * n:(e + 1) * n].to(D))
        dA[e * r:(e + 1) * r] = u.T @ X[st["source"][lo:lo + c].long()]
        dB[e * n:(e + 1) * n] = s * (g.T @ st["T"][lo:lo + c].to(D))
        lo += c
    return {"dA": dA, "dB": dB}


_EXACT = {"route": _exact_route, "rows": _exact_rows, "pack": _exact_pack, "linear8": _exact_linear8,
          "pair8": _exact_pair8, "moe8": _exact_moe8}
