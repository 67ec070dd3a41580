"""Cases, plain forms and 64-bit values of the operators around the 4-bit projection that are timed
and checked together:

* multi: a projection with one frozen 4-bit weight (NF4 or E2M1) and a low-rank adapter of its own
  for every row (the requests of a serving batch, or the jobs of a training batch), forward and
  forward with backward;
* qk: the norm of every query and key head and the position rotation behind the q and k
  projections, forward and forward with backward;
* distill: the loss that trains a student on its teacher's top logits, and its gradient.

`own` False computes them with elementary torch operations in 32 bits, rounded once at the end;
True calls the library.
"""
import math

import torch

own = False

DEV = "cuda"

# The 16 NF4 levels: the float32 values that the format fixes.
LEVELS = [-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
          -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
          0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045,
          0.722956657409668, 1.0]
# The 8 magnitudes of an E2M1 code; bit 3 of the code is the sign.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # one token of one request through a 4096 x 4096 projection: the smallest call, latency only
        dict(name="multi_one_token", op="multi", m=1, k=4096, n=4096, r=16, L=8, fmt="nf4", rows="mixed", bwd=False),
        # sixteen requests decoding at once, each with its own adapter, on the repository's decode shape
        dict(name="multi_decode16", op="multi", m=16, k=8192, n=28672, r=16, L=16, fmt="nf4", rows="each", bwd=False),
        # a larger serving batch, 200 requests over 64 adapters (some with none), on the mlp_up weight
        dict(name="multi_batch200", op="multi", m=200, k=4096, n=11008, r=16, L=64, fmt="nf4", rows="mixed", bwd=False),
        # prompts of several requests in one batch on the q_proj shape: ragged runs of rows
        dict(name="multi_prefill", op="multi", m=4096, k=4096, n=4096, r=16, L=8, fmt="nf4", rows="runs", bwd=False),
        # a ragged prefill with the E2M1 weight and a rank that is no multiple of 8
        dict(name="multi_prefill_e2m1", op="multi", m=1111, k=2880, n=2952, r=12, L=5, fmt="e2m1", rows="runs", bwd=False),
        # four adapters trained in one batch on the mlp_up shape, forward and backward: the largest
        dict(name="multi_train", op="multi", m=8192, k=4096, n=11008, r=64, L=4, fmt="nf4", rows="runs", bwd=True),
        # the heads of a decode step of 16 requests, q and k as slices of one packed projection
        dict(name="qk_decode16", op="qk", m=16, hq=32, hk=8, d=128, rot=128, inter=False, dt="bf16", bwd=False),
        # the heads of a 4096-token prompt, rotation of part of each head, interleaved pairs
        dict(name="qk_prefill", op="qk", m=4096, hq=24, hk=6, d=96, rot=64, inter=True, dt="bf16", bwd=False),
        # a training batch, forward and backward
        dict(name="qk_train", op="qk", m=8192, hq=32, hk=8, d=128, rot=128, inter=False, dt="bf16", bwd=True),
        # the loss and gradient of a short batch with an odd vocabulary
        dict(name="distill_small", op="distill", t=17, v=32003, top=16, tau=2.0, dt="bf16", bwd=True),
        # evaluation of the loss alone on float32 logits
        dict(name="distill_eval", op="distill", t=1024, v=50001, top=64, tau=1.0, dt="f32", bwd=False),
        # a training batch with a large vocabulary
        dict(name="distill_train", op="distill", t=4096, v=128000, top=64, tau=2.0, dt="bf16", bwd=True),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; the round sizes (multiples of 1024) are among the listed cases."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return x - (x % 1024 == 0)


def draw(rng):
    op = rng.choice(["multi", "multi", "qk", "distill"])
    if op == "multi":
        m = _log(rng, 1, 8192)
        k = 64 * rng.choice([4, 5, 9, 16, 25, 32, 45, 64, 67, 80, 112, 128])
        n = 8 * rng.choice([32, 37, 101, 128, 256, 369, 512, 640, 1001, 1376, 1792, 3584])
        bwd = rng.random() < 0.4
        while m * k * n * (3 if bwd else 1) > 3 * 8192 * 4096 * 11008:
            n = 8 * max(32, n // 16)
        r = rng.choice([4, 8, 16, 16, 20, 32, 64, 128])
        L = max(1, min(_log(rng, 1, 64), 4096 // r))
        return dict(op=op, m=m, k=k, n=n, r=r, L=L, fmt=rng.choice(["nf4", "nf4", "nf4f", "e2m1"]),
                    rows=rng.choice(["each", "mixed", "runs", "runs"]), bwd=bwd)
    if op == "qk":
        d = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 5, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        m = _log(rng, 1, 8192)
        rot = d if rng.random() < 0.6 else 2 * rng.randint(1, d // 2)
        return dict(op=op, m=m, hq=hq, hk=hk, d=d, rot=rot, inter=rng.random() < 0.4,
                    dt=rng.choice(["bf16", "bf16", "f32"]), bwd=rng.random() < 0.5)
    v = _log(rng, 1000, 160000)
    t = _log(rng, 1, min(8192, 4096 * 128000 // v // 2))
    return dict(op=op, t=t, v=v, top=rng.randint(1, 256), tau=rng.choice([0.5, 1.0, 2.0, 4.0]),
                dt=rng.choice(["bf16", "bf16", "f32"]), bwd=rng.random() < 0.6)


# ---------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _row_ids(case, g):
    """The adapter of every row; -1 where a request has none."""
    m, L = case["m"], case["L"]
    if case["rows"] == "each":          # every row a request of its own
        return (torch.randperm(max(m, L), generator=g, device=DEV)[:m] % L).to(torch.int32)
    if case["rows"] == "mixed":         # any adapter, one row in eight without
        ids = torch.randint(0, L, (m,), generator=g, device=DEV)
        return torch.where(torch.rand(m, generator=g, device=DEV) < 0.125, -1, ids).to(torch.int32)
    # runs of rows (prompts, training jobs), about two for each adapter, in any order
    cuts = torch.rand(m, generator=g, device=DEV) < (2.0 * L / m)
    of_run = torch.randint(0, L, (m,), generator=g, device=DEV)
    return of_run[torch.cumsum(cuts, 0) % m].to(torch.int32)


def _nf4(g, n, k, dq):
    """A normal weight in NF4: codes (first element in the high nibble), block constants, run scales."""
    w = torch.randn(n * k // 64, 64, generator=g, device=DEV) * 0.02
    a = w.abs().amax(1)
    lv = torch.tensor(LEVELS, device=DEV)
    c = torch.bucketize(w / a[:, None], (lv[1:] + lv[:-1]) / 2, out_int32=True).to(torch.uint8).view(-1, 2)
    codes = (c[:, 0] << 4) | c[:, 1]
    if not dq:
        return codes, a, None
    pad = (-a.numel()) % 256
    S = torch.nn.functional.pad(a, (0, pad)).view(-1, 256).amax(1) / 127
    q = torch.round(a / S.repeat_interleave(256)[:a.numel()]).clamp(0, 127).to(torch.int8)
    return codes, q, S


def _e2m1(g, n, k):
    """A normal weight in E2M1: codes, an E4M3 scale (as its byte) per group of 16, the tensor scale."""
    w = torch.randn(n * k // 16, 16, generator=g, device=DEV) * 0.02
    S = (w.abs().max() / 2688).reshape(1)
    s8 = (w.abs().amax(1) / (6 * S)).clamp(max=448).to(torch.float8_e4m3fn)
    v = w / (s8.float() * S).clamp(min=1e-30)[:, None]
    mag = torch.tensor(E2M1, device=DEV)
    i = torch.bucketize(v.abs(), (mag[1:] + mag[:-1]) / 2, out_int32=True)
    c = (i + 8 * (v < 0)).to(torch.uint8).view(-1, 2)
    scale = torch.zeros(4, device=DEV)
    scale[0:1] = S
    return (c[:, 0] << 4) | c[:, 1], s8.view(torch.uint8), scale


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "multi":
        m, k, n, r, L = (case[x] for x in ("m", "k", "n", "r", "L"))
        st["codes"], st["absmax"], st["scale"] = (_e2m1(g, n, k) if case["fmt"] == "e2m1"
                                                  else _nf4(g, n, k, case["fmt"] == "nf4"))
        st["X"] = _normal(g, (m, k), 1.0)
        st["A"] = _normal(g, (L, r, k), k ** -0.5)
        st["B"] = _normal(g, (L, n, r), 0.01)
        st["s"] = torch.rand(L, generator=g, device=DEV) * 1.5 + 0.5      # alpha / rank of each adapter
        st["ids"] = _row_ids(case, g)
        if case["bwd"]:
            st["dY"] = _normal(g, (m, n), 1.0)
    elif case["op"] == "qk":
        m, hq, hk, d, rot = (case[x] for x in ("m", "hq", "hk", "d", "rot"))
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
        qkv = _normal(g, (m, hq + 2 * hk, d), 1.3, dt)                    # the packed projection's output
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        st["wq"] = (1 + _normal(g, (d,), 0.2, torch.float32)).to(dt)
        st["wk"] = (1 + _normal(g, (d,), 0.2, torch.float32)).to(dt)
        places = max(4096, 2 * m)
        freq = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) / max(1, rot // 2))
        ang = torch.arange(places, device=DEV, dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = torch.randint(0, places, (m,), generator=g, device=DEV, dtype=torch.int32)
        if case["bwd"]:
            st["gq"], st["gk"] = _normal(g, (m, hq, d), 1.0, dt), _normal(g, (m, hk, d), 1.0, dt)
    else:
        t, v, top = case["t"], case["v"], case["top"]
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
        z = torch.randn(t, v, generator=g, device=DEV) * 2.5
        # the teacher: the student's logits with noise, its largest kept
        near = z[:, :min(v, 8 * top)] + torch.randn(t, min(v, 8 * top), generator=g, device=DEV) * 1.5
        val, idx = near.topk(top, dim=1)
        st["logits"] = z.to(dt)
        step = max(1, v // min(v, 8 * top))
        st["logits"][:, ::step][:, :near.shape[1]] += (near * 0.5).to(dt)
        st["idx"], st["teacher"] = (idx * step).to(torch.int32), val
        # a padded position in sixteen counts for nothing; the others weigh one over their number
        keep = (torch.rand(t, generator=g, device=DEV) >= 0.0625) | (torch.arange(t, device=DEV) == 0)
        st["weight"] = keep.float() / keep.sum()
    return st


# ---------------------------------------------------------------------------------- one pass
def run(st):
    return _LIB[st["op"]](st) if own else _PLAIN[st["op"]](st)


def _lib_multi(st):
    import nf4_dequant_gemm_amd as nq
    q = nq.NF4Tensor(st["n"], st["k"], 256 if st["fmt"] == "nf4" else 0, st["codes"], st["absmax"], st["scale"],
                     16 if st["fmt"] == "e2m1" else 64)
    Y, T = nq.qlora_multi_fwd(st["X"], q, st["A"], st["B"], st["s"], st["ids"])
    if not st["bwd"]:
        return {"Y": Y, "T": T}
    dX, dA, dB = nq.qlora_multi_bwd(st["dY"], st["X"], q, st["A"], st["B"], st["s"], st["ids"], T)
    return {"Y": Y, "T": T, "dX": dX, "dA": dA, "dB": dB}


def _lib_qk(st):
    import nf4_dequant_gemm_amd as nq
    args = (st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"])
    q, k = nq.qk_norm_rope_fwd(*args, eps=1e-6, interleaved=st["inter"])
    if not st["bwd"]:
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = nq.qk_norm_rope_bwd(st["gq"], st["gk"], *args, eps=1e-6, interleaved=st["inter"])
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _lib_distill(st):
    import nf4_dequant_gemm_amd as nq
    if not st["bwd"]:
        loss, lse = nq.distill_topk_fwd(st["logits"], st["idx"], st["teacher"], st["tau"])
        return {"loss": loss, "lse": lse}
    loss, grad = nq.distill_topk_step(st["logits"], st["idx"], st["teacher"], st["tau"], st["weight"])
    return {"loss": loss, "grad": grad}


_LIB = {"multi": _lib_multi, "qk": _lib_qk, "distill": _lib_distill}


def _weight(st):
    """The dequantised weight [n, k] in 32 bits."""
    c = st["codes"]
    c = torch.stack((c >> 4, c & 15), 1).view(-1)
    if st["fmt"] == "e2m1":
        mag = torch.tensor(E2M1, device=DEV)
        w = torch.cat((mag, -mag))[c.int()].view(-1, 16) * st["absmax"].view(torch.float8_e4m3fn).float()[:, None]
        return (w * st["scale"][0]).view(st["n"], st["k"])
    a = st["absmax"].float()
    if st["fmt"] == "nf4":
        a = a * st["scale"].repeat_interleave(256)[:a.numel()]
    return (torch.tensor(LEVELS, device=DEV)[c.int()].view(-1, 64) * a[:, None]).view(st["n"], st["k"])


def _plain_multi(st):
    # every adapter's ranks side by side, and each row keeps those of its own adapter
    m, k, n, r, L = (st[x] for x in ("m", "k", "n", "r", "L"))
    W, X = _weight(st), st["X"].float()
    A = st["A"].float().view(L * r, k)
    B = st["B"].float().permute(1, 0, 2).reshape(n, L * r)
    of = torch.arange(L, device=DEV).repeat_interleave(r)
    mine = of == st["ids"][:, None]                                       # [m, L r]
    s = st["s"].repeat_interleave(r)
    T = torch.where(mine, X @ A.t(), 0.0)
    Y = X @ W.t() + (T * s) @ B.t()
    out = {"Y": Y.bfloat16(), "T": T.view(m, L, r).sum(1).bfloat16()}
    if st["bwd"]:
        dY = st["dY"].float()
        U = torch.where(mine, dY @ B, 0.0) * s
        out["dX"] = (dY @ W + U @ A).bfloat16()
        out["dA"] = (U.t() @ X).view(L, r, k).bfloat16()
        out["dB"] = ((dY.t() @ T) * s).view(n, L, r).permute(1, 0, 2).contiguous().bfloat16()
    return out


def _turn(x, cos, sin, rot, inter):
    """x [m, h, d] with its first `rot` elements rotated in pairs by the row's angles."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_qk(st):
    rot, inter, out = st["rot"], st["inter"], {}
    cos, sin = st["cos"][st["pos"].long()][:, None], st["sin"][st["pos"].long()][:, None]

    def head(x, w, gy):
        x, w = x.float(), w.float()
        inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        y = _turn(x * inv * w, cos, sin, rot, inter)
        if gy is None:
            return y, None, None
        gn = _turn(gy.float(), cos, -sin, rot, inter)                     # the transposed rotation
        xh, gh = x * inv, gn * w
        dx = inv * (gh - xh * (gh * xh).mean(-1, keepdim=True))
        return y, dx, (gn * xh).sum((0, 1))

    dt = st["q"].dtype
    y, dx, dw = head(st["q"], st["wq"], st.get("gq"))
    z, dz, dv = head(st["k"], st["wk"], st.get("gk"))
    out["q"], out["k"] = y.to(dt), z.to(dt)
    if st["bwd"]:
        out["dq"], out["dk"], out["dwq"], out["dwk"] = dx.to(dt), dz.to(dt), dw, dv
    return out


def _plain_distill(st):
    z = st["logits"].float() / st["tau"]
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    lse = top[:, 0] + e.sum(1).log()
    y = st["teacher"].float() / st["tau"]
    y = y - y.amax(1, keepdim=True)
    log_p = y - y.exp().sum(1, keepdim=True).log()
    p, idx = log_p.exp(), st["idx"].long()
    loss = (p * (log_p - (z.gather(1, idx) - lse[:, None]))).sum(1)
    if not st["bwd"]:
        return {"loss": loss, "lse": lse}
    w = st["weight"][:, None] / st["tau"]
    grad = (w * (z - lse[:, None]).exp()).scatter_add(1, idx, -w * p)
    return {"loss": torch.where(st["weight"] != 0, loss, 0.0), "grad": grad.to(st["logits"].dtype)}


_PLAIN = {"multi": _plain_multi, "qk": _plain_qk, "distill": _plain_distill}


# ------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "multi":
        m, k, n, r, L = (case[x] for x in ("m", "k", "n", "r", "L"))
        used = min(L, m)
        per = {"nf4": 0.5 + 1 / 64 + 4 / 16384, "nf4f": 0.5 + 4 / 64, "e2m1": 0.5 + 1 / 16}[case["fmt"]]
        weight, adapters = n * k * per, 2 * used * r * (k + n)
        low = 2 * m * r * (k + n)
        by = weight + adapters + 2 * m * (k + n + r) + 4 * m
        fl = 2 * m * n * k + low
        if case["bwd"]:   # dY and X read, dX, dA, dB written; the weight and the adapters read again
            by += weight + adapters + 2 * m * (n + 2 * k + r) + 2 * L * r * (k + n)
            fl += 2 * m * n * k + 2 * low
        return {"bytes": int(by), "flops": int(fl)}
    if case["op"] == "qk":
        e = (2 if case["dt"] == "bf16" else 4) * case["m"] * (case["hq"] + case["hk"]) * case["d"]
        tab = case["m"] * (4 * case["rot"] + 4)
        n = case["m"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": (5 * e + 2 * tab) if case["bwd"] else 2 * e + tab, "flops": (22 if case["bwd"] else 7) * n}
    e = (2 if case["dt"] == "bf16" else 4) * case["t"] * case["v"]
    small = case["t"] * (8 * case["top"] + 8)
    return {"bytes": (2 if case["bwd"] else 1) * e + small, "flops": (8 if case["bwd"] else 5) * case["t"] * case["v"]}


# ------------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    return {"multi": _exact_multi, "qk": _exact_qk, "distill": _exact_distill}[case["op"]](prepare(case, seed))


def _exact_multi(st):
    n, k, L, D = st["n"], st["k"], st["L"], torch.float64
    hi, lo = st["codes"].long() // 16, st["codes"].long() % 16
    code = torch.empty(n * k, dtype=torch.long, device=DEV)
    code[0::2], code[1::2] = hi, lo
    if st["fmt"] == "e2m1":
        mag = torch.tensor(E2M1, dtype=D, device=DEV)[code % 8]
        W = torch.where(code >= 8, -mag, mag)
        W = W.view(-1, 16) * (st["absmax"].view(torch.float8_e4m3fn).to(D) * st["scale"][0].to(D))[:, None]
    else:
        a = st["absmax"].to(D)
        if st["fmt"] == "nf4":
            a = a * st["scale"].to(D)[torch.arange(a.numel(), device=DEV) // 256]
        W = torch.tensor(LEVELS, dtype=torch.float32, device=DEV).to(D)[code].view(-1, 64) * a[:, None]
    W = W.reshape(n, k)
    del code, hi, lo
    X, A, B, s = (st[x].to(D) for x in ("X", "A", "B", "s"))
    Y, T = X @ W.T, torch.zeros(st["m"], st["r"], dtype=D, device=DEV)
    dY = st["dY"].to(D) if st["bwd"] else None
    dX = dY @ W if st["bwd"] else None
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(L):
        rows = (st["ids"] == a).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        x = X[rows]
        t = x @ A[a].T
        T[rows] = t
        Y[rows] += s[a] * (t @ B[a].T)
        if st["bwd"]:
            g = dY[rows]
            u = s[a] * (g @ B[a])
            dX[rows] += u @ A[a]
            dA[a] = u.T @ x
            dB[a] = s[a] * (g.T @ t)
    return {"Y": Y, "T": T, "dX": dX, "dA": dA, "dB": dB} if st["bwd"] else {"Y": Y, "T": T}


def _exact_qk(st):
    D, rot, d = torch.float64, st["rot"], st["d"]
    half = rot // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if st["inter"] else (i, i + half)
    c, s = st["cos"].to(D)[st["pos"].long()], st["sin"].to(D)[st["pos"].long()]
    res = {}
    for name, x, w, g in (("q", st["q"], st["wq"], st.get("gq")), ("k", st["k"], st["wk"], st.get("gk"))):
        x, w = x.to(D), w.to(D)
        norm = (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
        u = x / norm
        v = u * w

        def rotated(a, sign):
            b = a.clone()
            p, q = a.index_select(-1, first), a.index_select(-1, second)
            b[..., first] = p * c[:, None] - sign * q * s[:, None]
            b[..., second] = q * c[:, None] + sign * p * s[:, None]
            return b

        res[name] = rotated(v, 1)
        if g is not None:
            t = rotated(g.to(D), -1)
            h = t * w
            res["d" + name] = (h - u * ((h * u).sum(-1, keepdim=True) / d)) / norm
            res["dw" + name] = (t * u).sum(1).sum(0)
    return res


def _exact_distill(st):
    D = torch.float64
    z = st["logits"].to(D) / st["tau"]
    lse = torch.logsumexp(z, 1)
    t = st["teacher"].to(D) / st["tau"]
    log_p = t - torch.logsumexp(t, 1)[:, None]
    at = st["idx"].long()
    loss = (log_p.exp() * (log_p - torch.take_along_dim(z, at, 1) + lse[:, None])).sum(1)
    if not st["bwd"]:
        return {"loss": loss, "lse": lse}
    grad = (z - lse[:, None]).exp()
    rows = torch.arange(st["t"], device=DEV)[:, None].expand_as(at)
    grad.index_put_((rows, at), -log_p.exp(), accumulate=True)
    return {"loss": loss * (st["weight"] != 0), "grad": grad * (st["weight"].to(D) / st["tau"])[:, None]}
