"""Cases of the many-tensor AdamW operators: the step with 32-bit and with 8-bit states, and the sum of squares of the
mean gradient that clipping needs. Each works on one data-parallel rank's rows of a list of parameters.

  adamw32   master, m, v in fp32
  adamw8    master in fp32; m and r = sqrt(v) as e4m3 codes with one power-of-two scale (e8m0) per 32 elements
  sumsq     sum over all elements of (mean over the replicas)^2, in fp64

`own` false: plain torch operations. `own` true: the calls of zero_partitioned_optimizer_flatten_amd.

In the state every parameter's piece starts on a multiple of PIECE elements, with zeros behind its last element; the
scales of PIECE consecutive elements lie together, those of m before those of r.
"""
import math

import numpy as np
import torch

own = False

PIECE, BLOCK = 2048, 32
BETAS, EPS = (0.9, 0.95), 1e-8
LR = 3e-4
MASK32 = 0xFFFFFFFF
DEV = "cuda"


# ---------------------------------------------------------------- the lists

def _gpt2(layers, d, vocab, context):
    s = [(vocab, d), (context, d)]
    s += [(d,), (d,), (d, 3 * d), (3 * d,), (d, d), (d,), (d,), (d,), (d, 4 * d), (4 * d,), (4 * d, d), (d,)] * layers
    return s + [(d,), (d,)]


def _llama(layers, d, ffn, vocab):
    return [(vocab, d)] + [(d, d), (d, d), (d, d), (d, d), (ffn, d), (ffn, d), (d, ffn), (d,), (d,)] * layers + [(d,), (vocab, d)]


def _ragged(count, most, seed):
    r = np.random.RandomState(seed)
    n = np.maximum(1, np.exp(r.uniform(0.0, math.log(most), count)).astype(np.int64))
    return [(int(k),) if k < 8 or i % 2 else (7, max(1, int(k) // 7)) for i, k in enumerate(n)]


def _shapes(c):
    if c["list"] == "gpt2":
        return _gpt2(c["layers"], c["d"], c["vocab"], c["context"])
    if c["list"] == "llama":
        return _llama(c["layers"], c["d"], c["ffn"], c["vocab"])
    return _ragged(c["count"], c["most"], c["lseed"])


def _local(c):
    """Elements of this rank's rows of every parameter."""
    out = []
    for s in _shapes(c):
        rows = -(-s[0] // c["world"])
        rows = max(0, min(s[0], (c["rank"] + 1) * rows) - c["rank"] * rows)
        out.append(rows * (s[1] if len(s) > 1 else 1))
    return out


def _padded(sizes):
    return [-(-n // PIECE) * PIECE for n in sizes]


# ---------------------------------------------------------------- the cases

def _case(op, replicas, grad, out="bf16", clip=False, gap=0, t=100, **where):
    return dict(op=op, replicas=replicas, grad=grad, out=out, clip=clip, gap=gap, t=t, **where)


GPT2 = dict(list="gpt2", layers=12, d=768, vocab=50257, context=1024)
LLAMA = dict(list="llama", layers=32, d=4096, ffn=11008, vocab=32000)


def listed():
    few = dict(list="ragged", count=11, most=700, lseed=3, world=1, rank=0)
    return [
        # a handful of tiny tensors (an adapter's or a head's own optimizer): the call's latency
        dict(_case("adamw32", 1, "fp32", "fp32", **few), name="adamw32 few tiny"),
        # GPT-2 small on one GPU, no sharding: 148 tensors in one call
        dict(_case("adamw32", 1, "bf16", world=1, rank=0, **GPT2), name="adamw32 gpt2 whole"),
        # a rank of eight with its peers' gradient rows still separate; clipped
        dict(_case("adamw32", 8, "bf16", clip=True, world=8, rank=3, **GPT2), name="adamw32 gpt2 rank 3 of 8"),
        # the 7B list on a rank of eight, its gradient rows already reduced in fp32; clipped: the largest
        dict(_case("adamw32", 1, "fp32", clip=True, world=8, rank=0, **LLAMA), name="adamw32 llama7b reduced"),
        # the same four with 8-bit states
        dict(_case("adamw8", 1, "bf16", **few), name="adamw8 few tiny"),
        dict(_case("adamw8", 8, "bf16", clip=True, world=8, rank=3, **GPT2), name="adamw8 gpt2 rank 3 of 8"),
        # odd widths, pieces that follow each other at odd elements, two fp32 replicas, fp32 parameters
        dict(_case("adamw8", 2, "fp32", "fp32", gap=1, t=7, list="llama", layers=4, d=1025, ffn=2731, vocab=16001, world=3, rank=1),
             name="adamw8 odd widths"),
        dict(_case("adamw8", 1, "bf16", clip=True, world=8, rank=0, **LLAMA), name="adamw8 llama7b reduced"),
        # the norm before each of these steps
        dict(_case("sumsq", 4, "fp32", **few), name="sumsq few tiny"),
        dict(_case("sumsq", 8, "bf16", world=8, rank=3, **GPT2), name="sumsq gpt2 rank 3 of 8"),
        dict(_case("sumsq", 3, "bf16", gap=3, list="llama", layers=4, d=1025, ffn=2731, vocab=16001, world=3, rank=1), name="sumsq odd widths"),
        dict(_case("sumsq", 1, "fp32", world=8, rank=0, **LLAMA), name="sumsq llama7b reduced"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = max(work(c)["bytes"] for c in listed())
    while True:
        c = _case(rng.choice(("adamw32", "adamw8", "sumsq")), rng.choice((1, 1, 2, 3, 4, 5, 8, 16)), rng.choice(("bf16", "bf16", "fp32")),
                  rng.choice(("bf16", "bf16", "fp32")), rng.random() < 0.5, rng.choice((0, 0, 1, 2, 5)), log(1, 20000))
        if rng.random() < 0.4:
            c.update(list="ragged", count=log(1, 400), most=log(10, 3_000_000), lseed=rng.randrange(1 << 20), world=rng.choice((1, 1, 2, 5)), rank=0)
        else:
            d = log(64, 4200)
            w = rng.choice((1, 2, 3, 8, 16))
            c.update(list="llama", layers=log(1, 33), d=d, ffn=int(d * rng.uniform(2, 4)), vocab=log(1000, 33000), world=w, rank=rng.randrange(w))
        n = sum(_local(c))
        if n and work(c)["bytes"] <= top and n * (c["replicas"] + 4) <= 4_500_000_000:
            return c


def work(c):
    n = sum(_local(c))
    g = n * c["replicas"] * (2 if c["grad"] == "bf16" else 4)
    o = n * (2 if c["out"] == "bf16" else 4)
    if c["op"] == "sumsq":
        return {"bytes": g + 8, "flops": n * (c["replicas"] + 1)}
    if c["op"] == "adamw32":
        return {"bytes": g + 24 * n + o, "flops": n * (c["replicas"] + 16)}
    return {"bytes": g + 8 * n + 4 * n + 4 * n / BLOCK + o, "flops": n * (c["replicas"] + 24)}


# ------------------------------------------------------------------- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _between(pieces, pads):
    """The pieces behind each other, each followed by its zeros."""
    z = torch.zeros(PIECE, dtype=pieces[0].dtype, device=pieces[0].device)
    return torch.cat([x for p, k in zip(pieces, pads) for x in (p.reshape(-1), z[:k])])


def _nearest(x):
    """(codes, scales) of x, rounded to nearest: what a state read from a checkpoint starts with."""
    e = ((x.abs().view(-1, BLOCK).amax(1).view(torch.int32) + 0x1FFFFF) >> 23).sub_(8).clamp_(min=1)
    inv = ((254 - e) << 23).view(torch.float32)
    return (x.view(-1, BLOCK) * inv[:, None]).view(-1).to(torch.float8_e4m3fn), e.to(torch.uint8)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    sizes = _local(c)
    pads = [p - n for p, n in zip(_padded(sizes), sizes)]
    n = sum(sizes)

    def normal(std, count=n):
        return torch.randn(count, generator=gen, device=DEV).mul_(std)

    def views(flat):
        at, got = c["gap"], []
        for k in sizes:
            got.append(flat[at:at + k])
            at += k + c["gap"]
        return got

    total = n + c["gap"] * (len(sizes) + 1)
    quiet = (torch.rand(-(-total // 256), generator=gen, device=DEV) < 0.05).repeat_interleave(256)[:total]  # rows no token touched
    grads = []
    for _ in range(c["replicas"]):
        flat = normal(1e-3, total).mul_(torch.rand(1, generator=gen, device=DEV) + 0.5)
        flat[quiet] = 0
        grads.append(views(flat.to(_dtype(c["grad"]))))
        del flat
    s = dict(case=c, sizes=sizes, pads=pads, grads=grads)
    if c["op"] == "sumsq":
        s["sumsq"] = torch.zeros(1, dtype=torch.float64, device=DEV)
    else:
        s["out"] = torch.zeros(total, dtype=_dtype(c["out"]), device=DEV)
        s["outs"] = views(s["out"])
        s["decay"] = [0.1 if len(x) > 1 else 0.0 for x in _shapes(c)]
        s["factor"] = [0.5] + [1.0] * (len(sizes) - 1)
        s["seed"] = seed & 0x7FFFFFFF
        # a norm over all ranks, of which this rank's share is one part
        s["sumsq"] = torch.rand(1, generator=gen, device=DEV, dtype=torch.float64).add_(0.5).mul_(2.0) if c["clip"] else None

        def state(flat):
            return _between(list(flat.split(sizes)), pads)

        s["master"] = state(normal(0.02))
        m = state(normal(2e-4))
        r = state(normal(5e-4).abs_().add_(1e-5))
        if c["op"] == "adamw32":
            s["m"], s["v"] = m, r.square_()
        else:
            s["m"], em = _nearest(m)
            s["r"], er = _nearest(r)
            s["scale"] = torch.stack((em.view(-1, PIECE // BLOCK), er.view(-1, PIECE // BLOCK)), 1).contiguous().view(torch.float8_e8m0fnu)
        del m, r
    if own:
        import zero_partitioned_optimizer_flatten_amd as zero
        bits = 8 if c["op"] == "adamw8" else 32
        h = zero.AdamWState(_shapes(c), c["world"], c["rank"], LR, BETAS, EPS, weight_decay=s.get("decay", 0.0), lr_scale=s.get("factor", 1.0),
                            state_bits=bits, seed=s.get("seed", 0))
        held = h.state_tensors()
        for k in ("master", "m", "v", "r", "scale"):
            if k in s:
                held[k].copy_(s[k])
                s[k] = held[k]
        h.bind([[g if g.numel() else None for g in q] for q in grads], None if c["op"] == "sumsq" else s["outs"])
        s["handle"] = h
    return s


# --------------------------------------------------------------- the passes

def run(state):
    s, c = state, state["case"]
    if own:
        h = s["handle"]
        if c["op"] == "sumsq":
            h.sumsq(out=s["sumsq"])
            return s["sumsq"]
        h.step(c["t"], sumsq=s["sumsq"], max_norm=1.0)
    elif c["op"] == "sumsq":
        _sumsq(s)
        return s["sumsq"]
    elif c["op"] == "adamw32":
        _adamw32(s)
    else:
        _adamw8(s)
    return {k: s[k] for k in ("out", "master", "m", "v", "r", "scale") if k in s}


def _sumsq(s):
    total = torch.cat(s["grads"][0]).double()
    for q in s["grads"][1:]:
        total += torch.cat(q)
    s["sumsq"].copy_(total.square_().sum() / s["case"]["replicas"] ** 2)


def _scalars(t):
    f = np.float32
    bc1, bc2 = f(1.0 - BETAS[0] ** t), f(1.0 - BETAS[1] ** t)
    return dict(b1=float(f(BETAS[0])), c1=float(f(1.0 - BETAS[0])), b2=float(f(BETAS[1])), c2=float(f(1.0 - BETAS[1])), lr=float(f(LR)),
                eps=float(f(EPS)), bc1=float(bc1), bc2=float(bc2), rs=float(f(1.0) / np.sqrt(bc2)))


def _gradient(s):
    """The mean over the replicas, clipped, laid out as the state."""
    n = s["case"]["replicas"]
    g = _between(s["grads"][0], s["pads"]).float()
    for q in s["grads"][1:]:
        g += _between(q, s["pads"])
    if n > 1:
        g /= n
    if s["sumsq"] is not None:
        g *= (1.0 / (s["sumsq"].sqrt() + 1e-6)).clamp(max=1.0).float()
    return g


def _rates(s, lr):
    """(learning rate, decay factor) of every element of the state."""
    lr = torch.tensor(s["factor"], device=DEV) * lr
    keep = 1.0 - lr * torch.tensor(s["decay"], device=DEV)
    return [torch.cat([x.expand(n) for x, n in zip(v.unbind(), _padded(s["sizes"]))]) for v in (lr, keep)]


def _write(s):
    """The parameters from the master copy, each in its place."""
    rows = [x[:n] for x, n in zip(s["master"].split(_padded(s["sizes"])), s["sizes"])]
    torch._foreach_copy_([o for o in s["outs"] if o.numel()], [x for x in rows if x.numel()])


def _adamw32(s):
    k, g = _scalars(s["case"]["t"]), _gradient(s)
    s["m"].mul_(k["b1"]).add_(g * k["c1"])
    s["v"].mul_(k["b2"]).add_(g.square_().mul_(k["c2"]))
    del g
    lr, keep = _rates(s, k["lr"])
    den = (s["v"] / k["bc2"]).sqrt_().add_(k["eps"])
    s["master"].mul_(keep).sub_((s["m"] / k["bc1"]).mul_(lr).div_(den))
    _write(s)


def _values(codes, e):
    return (codes.float().view(-1, BLOCK) * e[:, None]).view(-1)


def _noise(s):
    """32 bits for every element, from the seed, the step and the element's place in the state."""
    def mix(x):
        x = (x * 0x9E3B5A35) & MASK32
        x = x ^ (x >> 15)
        x = (x * 0x5D2C9E1B) & MASK32
        return x ^ (x >> 16)

    key = mix(mix(s["seed"]) ^ (s["case"]["t"] & MASK32))
    q = torch.arange(s["master"].numel() // 4, device=DEV)
    x = mix((q + (q >> 32) * 0x7F4A7C15 + key) & MASK32)
    return torch.stack([x, (x * 0xB5297A4D) & MASK32, (x * 0x68E31DA5) & MASK32, (x * 0x1B56C4E9) & MASK32], 1).view(-1)


def _encode(x, noise, floor):
    """(codes, scales): a carry from `noise` (16 bits) into the third mantissa bit, what is below it cut, then the e4m3 grid."""
    finite = x.abs() < math.inf
    top = torch.where(finite, x, 0.0).abs_().view(-1, BLOCK).amax(1).view(torch.int32)
    e = ((top + 0x1FFFFF) >> 23).sub_(8).clamp_(min=1)
    y = ((x.view(torch.int32) + (noise << 4).to(torch.int32)) & ~0xFFFFF).view(torch.float32)
    y = (y.view(-1, BLOCK) * ((254 - e) << 23).view(torch.float32)[:, None]).view(-1)
    if floor:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    return torch.where(finite, y, math.nan).to(torch.float8_e4m3fn), e.to(torch.uint8)


def _adamw8(s):
    def fma(a, b, c):  # one rounding to 32 bits: the product of two 32-bit numbers is whole in 64
        return (a.double() * b).add_(c).float()

    k, g = _scalars(s["case"]["t"]), _gradient(s)
    e = s["scale"].float()
    m = _values(s["m"], e[:, 0].reshape(-1))
    m = fma(g, k["c1"], m * k["b1"])
    r = _values(s["r"], e[:, 1].reshape(-1))
    v = fma(g * k["c2"], g, (r * r) * k["b2"])
    del g
    r = v.double().sqrt_().float()
    lr, keep = _rates(s, k["lr"])
    u = (lr / k["bc1"]).mul_(m).div_((r * k["rs"]).add_(k["eps"]))
    del lr, v
    s["master"].mul_(keep).sub_(u)
    del keep, u
    noise = _noise(s)
    codes, em = _encode(m, noise >> 16, False)
    s["m"].copy_(codes)
    codes, er = _encode(r, noise & 0xFFFF, True)
    s["r"].copy_(codes)
    s["scale"].view(torch.uint8).copy_(torch.stack((em.view(-1, PIECE // BLOCK), er.view(-1, PIECE // BLOCK)), 1))
    _write(s)


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The same from the definitions in 64 bits: one step from this seed's inputs."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, n = case, case["replicas"]
    pad = _padded(s["sizes"])
    at = np.cumsum([0] + pad[:-1])
    g = torch.zeros(sum(pad), dtype=torch.float64, device=DEV)
    for k, size in enumerate(s["sizes"]):
        for q in s["grads"]:
            g[at[k]:at[k] + size] += q[k]
    if c["op"] == "sumsq":
        return torch.dot(g, g).view(1) / (n * n)
    g /= n
    if c["clip"]:
        g *= min(1.0, 1.0 / (math.sqrt(float(s["sumsq"])) + 1e-6))
    b1, b2 = BETAS
    bc1, bc2 = 1.0 - b1 ** c["t"], 1.0 - b2 ** c["t"]
    wide = None
    if c["op"] == "adamw8":
        wide = torch.pow(2.0, s["scale"].view(torch.uint8).double() - 127.0)
        m = (s["m"].double().view(-1, BLOCK) * wide[:, 0].reshape(-1, 1)).view(-1)
        v = (s["r"].double().view(-1, BLOCK) * wide[:, 1].reshape(-1, 1)).view(-1).square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    del g
    p = s["master"].double()
    step = m / bc1 / ((v / bc2).sqrt() + EPS)
    for k, size in enumerate(pad):
        lr = LR * s["factor"][k]
        x = p[at[k]:at[k] + size]
        x.mul_(1.0 - lr * s["decay"][k]).sub_(step[at[k]:at[k] + size], alpha=lr)
    del step
    out = s["out"].double()
    where = c["gap"]
    for k, size in enumerate(s["sizes"]):
        out[where:where + size] = p[at[k]:at[k] + size]
        where += size + c["gap"]
    if c["op"] == "adamw32":
        return {"out": out, "master": p, "m": m, "v": v}
    noise = _noise(s)
    m, em = _code64(m, (noise >> 16).double() / 65536.0, 0.0)
    r, er = _code64(v.sqrt_(), (noise & 0xFFFF).double() / 65536.0, 2.0 ** -9)
    return {"out": out, "master": p, "m": m, "r": r, "scale": torch.stack((em.view(-1, PIECE // BLOCK), er.view(-1, PIECE // BLOCK)), 1)}


def _code64(x, chance, least):
    """(codes' values, scales' values): blocks scaled by the power of two that brings their largest into (224, 448], each
    element up to the next of 8 steps of its octave with the chance that its place between two steps gives it."""
    top = x.abs().view(-1, BLOCK).amax(1)
    half, octave = torch.frexp(top)  # top = half * 2^octave, half in [1/2, 1)
    e = (octave - 1 - 8 + (half > 0.875)).double().clamp_(min=-126.0)
    e = torch.where(top > 0, e, -126.0)
    scale = torch.pow(2.0, e)
    part, octave = torch.frexp(x)
    y = torch.floor(part.abs() * 16.0 + chance) * part.sign()
    y = torch.ldexp(y, octave.double() - 4.0)
    y = (y.view(-1, BLOCK) / scale[:, None]).view(-1)
    y = torch.where(y.abs() < 2.0 ** -6, torch.round(y * 512.0) / 512.0, y)
    if least:
        y = torch.where(x > 0, y.clamp(min=least), y)
    return y, scale
