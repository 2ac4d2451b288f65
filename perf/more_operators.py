"""Cases of the operators at both ends of a language model, next to the optimizer step that reads their gradients.

  embed       rows of a (vocab, width) table by token, scaled, plus rows of a position table, with dropout
  embed_grad  the table's gradient, written or added into its place in a flat gradient vector
  dropout     from a counter-based generator, alone or added to a residual
  head_loss   softmax cross entropy of hidden states against a (vocab, width) table; with gradients of both, or the loss alone

`own` false: plain torch operations. `own` true: the calls of zero_partitioned_optimizer_flatten_amd.

Dropout keeps an element where its 16 random bits are at least round(65536 p), and scales what it keeps by the inverse of
the share kept. The bits are those of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
1, 2, 3", 2011): key = seed, counter = (element // 8, offset), 64 bits each; element 8 b + k takes the k-th 16 bits of
block b's 128, counted from the lowest. Ids outside the table have a row of zeros and no gradient; targets outside it
have no loss and no gradient.
"""
import math

import torch

own = False

DEV = "cuda"
M32 = 0xFFFFFFFF
IGNORED = -100


# ---------------------------------------------------------------- the cases

def _embed(n, vocab, width, dtype="bf16", context=0, scale=1.0, p=0.0, gap=0):
    return dict(op="embed", n=n, vocab=vocab, width=width, dtype=dtype, context=context, scale=scale, p=p, gap=gap)


def _grad(n, vocab, width, dtype="bf16", scale=1.0, p=0.0, gap=0, add=False, same=0.0):
    return dict(op="embed_grad", n=n, vocab=vocab, width=width, dtype=dtype, scale=scale, p=p, gap=gap, add=add, same=same)


def _drop(n, width, dtype="bf16", p=0.1, add=False):
    return dict(op="dropout", n=n, width=width, dtype=dtype, p=p, add=add)


def _loss(n, vocab, width, dtype="bf16", grads=True, gap=0, ignored=0.0, weighted=False, mean=True):
    return dict(op="head_loss", n=n, vocab=vocab, width=width, dtype=dtype, grads=grads, gap=gap, ignored=ignored, weighted=weighted, mean=mean)


def listed():
    return [
        # GPT-2 small's input for one sequence: token and position rows, dropout
        dict(_embed(1024, 50257, 768, context=1024, p=0.1), name="embed gpt2 sequence"),
        # the 7B list's input for a batch of packed sequences, rows scaled by the root of the width
        dict(_embed(32768, 32000, 4096, scale=64.0), name="embed llama7b batch"),
        # a small fp32 table with odd rows at an odd place of the flat vector, added to: latency
        dict(_grad(37, 1000, 65, "fp32", gap=1, add=True), name="embed_grad few tokens"),
        # GPT-2 small, eight sequences; the tied table's place holds the loss's share already
        dict(_grad(8192, 50257, 768, p=0.1, add=True), name="embed_grad gpt2 tied"),
        # the 7B list, untied; three tokens in ten are the one that pads sequences
        dict(_grad(16384, 32000, 4096, same=0.3), name="embed_grad llama7b padded"),
        # the activations of one GPT-2 sequence: latency
        dict(_drop(1024, 768), name="dropout gpt2 sequence"),
        # a wide residual stream in fp32 with an odd count of elements
        dict(_drop(16383, 5121, "fp32", p=0.25, add=True), name="dropout residual fp32"),
        # a character model's or a test's head: latency
        dict(_loss(16, 1000, 64, "fp32"), name="head_loss few rows"),
        # GPT-2 small, eight sequences
        dict(_loss(8192, 50257, 768), name="head_loss gpt2"),
        # the 7B list, a batch with a prompt that is not learned from: the largest
        dict(_loss(8192, 32000, 4096, ignored=0.2), name="head_loss llama7b"),
        # odd sizes at an odd place of the flat vector in fp32, weighted and summed
        dict(_loss(1023, 16001, 1025, "fp32", gap=1, weighted=True, mean=False), name="head_loss odd sizes"),
        # scoring the answers of a 13B model: few rows, no gradient
        dict(_loss(129, 32000, 5120, grads=False, ignored=0.1), name="head_loss llama13b scores"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("embed", "embed_grad", "dropout", "head_loss", "head_loss"))
    top = [work(c) for c in listed() if c["op"] == op]
    while True:
        dtype, gap, p = rng.choice(("bf16", "bf16", "fp32")), rng.choice((0, 0, 1, 8)), rng.choice((0.0, 0.1, 0.25, 0.5))
        n, vocab, width = log(1, 33000), log(100, 130000), log(16, 8200)
        if rng.random() < 0.6:
            width = -(-width // 64) * 64
        if op == "embed":
            c = _embed(n, vocab, width, dtype, rng.choice((0, log(16, 4096))), rng.choice((1.0, math.sqrt(width))), p, gap)
        elif op == "embed_grad":
            c = _grad(n, vocab, width, dtype, rng.choice((1.0, math.sqrt(width))), p, gap, rng.random() < 0.5, rng.choice((0.0, 0.0, 0.1, 0.5)))
        elif op == "dropout":
            c = _drop(n, width, dtype, rng.choice((0.1, 0.25, 0.5)), rng.random() < 0.5)
        else:
            c = _loss(n, vocab, width, dtype, rng.random() < 0.7, gap, rng.choice((0.0, 0.2)), rng.random() < 0.3, rng.random() < 0.7)
        w = work(c)
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top) and n * vocab <= 450_000_000:
            return c


def _distinct(c):
    """How many of the table's rows a batch of prepare()'s tokens is expected to name."""
    k = torch.arange(1, c["vocab"] + 1, dtype=torch.float64)
    share = torch.log1p(1.0 / k) / math.log(c["vocab"] + 1.0) * (1.0 - c.get("same", 0.0))
    return min(c["n"], round(float((1.0 - (1.0 - share) ** c["n"]).sum())) + (c.get("same", 0.0) > 0))


def work(c):
    n, width, e = c["n"], c["width"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "dropout":
        return {"bytes": n * width * e * (3 if c["add"] else 2), "flops": n * width * 2}
    ids = 8 * n
    if c["op"] == "embed":
        # a row that several tokens name is read once
        rows = _distinct(c) + min(n, c["context"])
        return {"bytes": ids * (2 if c["context"] else 1) + (rows + n) * width * e, "flops": n * width * 2}
    if c["op"] == "embed_grad":
        out = 2 * _distinct(c) if c["add"] else c["vocab"]
        return {"bytes": ids + (n + out) * width * e, "flops": n * width * 2}
    both = 2 if c["grads"] else 1
    return {"bytes": ids + 4 * n + (n + c["vocab"]) * width * e * both, "flops": 2 * n * c["vocab"] * width * (3 if c["grads"] else 1)}


# ------------------------------------------------------------------- inputs

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c, dt = case, _dtype(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, width = c["n"], c["width"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    def placed(x):
        """x as a view of a flat vector, `gap` elements behind its start."""
        flat = torch.zeros(x.numel() + c["gap"], dtype=dt, device=DEV)
        flat[c["gap"]:] = x.reshape(-1)
        return flat[c["gap"]:].view(x.shape)

    def ids():
        """Tokens as text has them: the k-th most frequent about k times rarer than the first."""
        u = uniform(n).double()
        return (torch.exp(u * math.log(c["vocab"] + 1.0)) - 1.0).long().clamp_(0, c["vocab"] - 1)

    s = dict(case=c, seed=(seed * 0x9E3779B97F4A7C15 + 1) & ((1 << 64) - 1), offset=(7 << 32) + 1000 + seed % 1000)
    if c["op"] == "dropout":
        s["x"] = normal(n, width).to(dt)
        s["add"] = normal(n, width).mul_(4.0).to(dt) if c["add"] else None
    elif c["op"] == "embed":
        s["tokens"] = ids()
        s["table"] = placed(normal(c["vocab"], width).mul_(0.02))
        if c["context"]:
            s["positions"] = (torch.arange(n, device=DEV) + seed % 5) % c["context"]
            s["position_table"] = normal(c["context"], width).mul_(0.01).to(dt)
    elif c["op"] == "embed_grad":
        s["tokens"] = torch.where(uniform(n) < c["same"], 2 % c["vocab"], ids())
        s["grad_out"] = normal(n, width).mul_(1e-3).to(dt)
        s["grad_table"] = placed(normal(c["vocab"], width).mul_(1e-3))
    else:
        targets = ids()
        table = normal(c["vocab"], width).mul_(0.02)
        # logits spread by 2, and up to 8 more at the target in three rows of five: what a model in training has
        lift = torch.where(uniform(n) < 0.6, uniform(n) * 8.0, 0.0) / (0.02 ** 2 * width)
        s["hidden"] = (normal(n, width).mul_(100.0 / math.sqrt(width)) + table[targets] * lift[:, None]).to(dt)
        s["table"] = placed(table)
        s["targets"] = torch.where(uniform(n) < c["ignored"], IGNORED, targets)
        s["weights"] = uniform(n) if c["weighted"] else None
        if c["grads"]:
            s["grad_hidden"] = torch.empty_like(s["hidden"])
            s["grad_table"] = placed(torch.zeros_like(table))
    return s


# --------------------------------------------------------------- the passes

def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    if c["op"] == "embed":
        return _plain_embed(s, c)
    if c["op"] == "embed_grad":
        return _plain_grad(s, c)
    if c["op"] == "dropout":
        return _plain_dropout(s["x"].float(), s, c, s["add"]).to(_dtype(c))
    return _plain_loss(s, c)


def _own(s, c):
    import zero_partitioned_optimizer_flatten_amd as zero
    drop = zero.Dropout(c["p"], s["seed"], s["offset"]) if c.get("p") else None
    if c["op"] == "embed":
        return zero.embed(s["tokens"], s["table"], scale=c["scale"], positions=s.get("positions"), position_table=s.get("position_table"), dropout=drop)
    if c["op"] == "embed_grad":
        return zero.embed_grad(s["grad_out"], s["tokens"], s["grad_table"], scale=c["scale"], dropout=drop, accumulate=c["add"])
    if c["op"] == "dropout":
        return zero.dropout(s["x"], drop, add=s["add"])
    losses = torch.empty(c["n"], device=DEV)
    loss = zero.head_loss(s["hidden"], s["table"], s["targets"], weights=s["weights"], reduction="mean" if c["mean"] else "sum",
                          losses=losses, grad_hidden=s.get("grad_hidden"), grad_table=s.get("grad_table"))
    return {"loss": loss, "losses": losses} | {k: s[k] for k in ("grad_hidden", "grad_table") if k in s}


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _keep(s, c):
    """Whether dropout keeps each of (n, width) elements."""
    count = c["n"] * c["width"]
    i = torch.arange(-(-count // 8), device=DEV)
    x0, x1 = i & M32, i >> 32
    x2, x3 = torch.full_like(i, s["offset"] & M32), torch.full_like(i, s["offset"] >> 32)
    k0, k1 = s["seed"] & M32, s["seed"] >> 32
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((b >> 32) & M32) ^ x1 ^ k0, b & M32, ((a >> 32) & M32) ^ x3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    x = torch.stack((x0, x1, x2, x3), 1).view(-1, 4, 1)
    bits = torch.cat((x & 0xFFFF, x >> 16), 2).view(-1)
    return (bits[:count] >= _threshold(c["p"])).view(c["n"], c["width"])


def _plain_dropout(x, s, c, add=None):
    if c["p"]:
        x = torch.where(_keep(s, c), x * (65536.0 / (65536 - _threshold(c["p"]))), 0.0)
    return x if add is None else x + add.float()


def _plain_embed(s, c):
    x = s["table"][s["tokens"]].float() * c["scale"]
    if c["context"]:
        x += s["position_table"][s["positions"]].float()
    return _plain_dropout(x, s, c).to(_dtype(c))


def _plain_grad(s, c):
    g = _plain_dropout(s["grad_out"].float(), s, c)
    total = torch.zeros(c["vocab"], c["width"], device=DEV).index_add_(0, s["tokens"], g).mul_(c["scale"])
    if c["add"]:
        total += s["grad_table"].float()
    return s["grad_table"].copy_(total)


def _plain_loss(s, c):
    h, w, y = s["hidden"].float(), s["table"].float(), s["targets"]
    valid = (y >= 0) & (y < c["vocab"])
    at = torch.where(valid, y, 0)[:, None]
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    here = z.gather(1, at)[:, 0]
    e = z.sub_(top).exp_()
    total = e.sum(1)
    losses = torch.where(valid, total.log() + top[:, 0] - here, 0.0)
    share = valid.float() if s["weights"] is None else torch.where(valid, s["weights"], 0.0)
    if c["mean"]:
        whole = share.sum()
        share = share / torch.where(whole > 0, whole, 1.0)
    out = {"loss": (losses * share).sum().view(1), "losses": losses}
    if not c["grads"]:
        return out
    g = e.mul_((share / total)[:, None]).scatter_add_(1, at, -share[:, None])
    s["grad_hidden"].copy_(g @ w)
    s["grad_table"].copy_(g.t() @ h)
    return out | {"grad_hidden": s["grad_hidden"], "grad_table": s["grad_table"]}


# -------------------------------------------------------------------- exact

def _times(x, const):
    """(high, low) 32 bits of the products of 32-bit x by a 32-bit constant, through 16-bit halves."""
    xh, xl, ch, cl = x >> 16, x & 0xFFFF, const >> 16, const & 0xFFFF
    low, mid1, mid2 = xl * cl, xh * cl, xl * ch
    carry = (low >> 16) + (mid1 & 0xFFFF) + (mid2 & 0xFFFF)
    return xh * ch + (mid1 >> 16) + (mid2 >> 16) + (carry >> 16), (low & 0xFFFF) | ((carry & 0xFFFF) << 16)


def _kept_share(s, c):
    """What dropout multiplies each element by, in 64 bits."""
    count, limit = c["n"] * c["width"], round(c["p"] * 65536)
    x = torch.zeros(4, (count + 7) // 8, dtype=torch.int64, device=DEV)
    x[0] = torch.arange(x.shape[1], device=DEV) % (1 << 32)
    x[1] = torch.arange(x.shape[1], device=DEV) // (1 << 32)
    x[2], x[3] = s["offset"] % (1 << 32), s["offset"] // (1 << 32)
    key = [s["seed"] % (1 << 32), s["seed"] // (1 << 32)]
    for r in range(10):
        hi0, lo0 = _times(x[0], 0xD2511F53)
        hi1, lo1 = _times(x[2], 0xCD9E8D57)
        keys = [(key[0] + r * 0x9E3779B9) % (1 << 32), (key[1] + r * 0xBB67AE85) % (1 << 32)]
        x = torch.stack((hi1 ^ x[1] ^ keys[0], lo1, hi0 ^ x[3] ^ keys[1], lo0))
    halves = torch.empty(x.shape[1], 8, dtype=torch.int32, device=DEV)
    halves[:, 0::2] = (x % 65536).t()
    halves[:, 1::2] = (x // 65536).t()
    kept = halves.reshape(-1)[:count].reshape(c["n"], c["width"]) >= limit
    return kept.double() * (1.0 / (1.0 - limit / 65536.0))


def exact(case, seed):
    """The same from the definitions in 64 bits, from this seed's inputs."""
    c, s = case, prepare(case, seed)
    if c["op"] == "dropout":
        y = s["x"].double() * _kept_share(s, c)
        return y if s["add"] is None else y + s["add"].double()
    if c["op"] == "embed":
        y = c["scale"] * torch.index_select(s["table"], 0, s["tokens"]).double()
        if c["context"]:
            y = y + torch.index_select(s["position_table"], 0, s["positions"]).double()
        return y * _kept_share(s, c) if c["p"] else y
    if c["op"] == "embed_grad":
        order = torch.argsort(s["tokens"], stable=True)
        g = s["grad_out"].double()
        if c["p"]:
            g = g * _kept_share(s, c)
        run_sums = torch.cat((g.new_zeros(1, c["width"]), g[order].cumsum_(0)))
        ends = torch.bincount(s["tokens"], minlength=c["vocab"]).cumsum(0)
        starts = torch.cat((ends.new_zeros(1), ends[:-1]))
        total = (run_sums[ends] - run_sums[starts]) * c["scale"]
        return total + s["grad_table"].double() if c["add"] else total
    h, w, y = s["hidden"].double(), s["table"].double(), s["targets"]
    rows = torch.nonzero((y >= 0) & (y < c["vocab"]))[:, 0]
    part = torch.zeros(c["n"], dtype=torch.float64, device=DEV)
    part[rows] = 1.0 if s["weights"] is None else s["weights"][rows].double()
    if c["mean"]:
        part /= float(part.sum()) or 1.0
    logp = torch.log_softmax(torch.mm(h, w.t()), 1)
    losses = torch.zeros(c["n"], dtype=torch.float64, device=DEV)
    losses[rows] = -logp[rows, y[rows]]
    out = {"loss": torch.dot(losses, part).view(1), "losses": losses}
    if c["grads"]:
        d = logp.exp_()
        d[rows, y[rows]] -= 1.0
        d *= part[:, None]
        out["grad_hidden"], out["grad_table"] = torch.mm(d, w), torch.mm(d.t(), h)
    return out
