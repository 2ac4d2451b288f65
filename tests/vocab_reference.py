"""Plain 64-bit references of the vocabulary operators, on the CPU, and bounds
on how far binary32 arithmetic with one rounding of each output may be off."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24                  # half a step of binary32, relative
M32 = np.uint64(0xFFFFFFFF)


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def philox(counter, key):
    """Philox4x32-10: four uint64 arrays holding 32 bits each, from such."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(x) for x in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & M32, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(shape, p, seed, offset=0):
    """(keep, scale): which elements dropout keeps, and their factor."""
    n = int(np.prod(shape))
    limit = int(np.floor(p * 65536 + 0.5))
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    o = np.full_like(block, offset)
    s = np.uint64(32)
    x = philox((block & M32, block >> s, o & M32, o >> s), (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.empty((len(block), 8), dtype=np.int64)
    for k in range(4):
        bits[:, 2 * k] = x[k] & np.uint64(0xFFFF)
        bits[:, 2 * k + 1] = x[k] >> np.uint64(16)
    keep = torch.from_numpy(bits.reshape(-1)[:n] >= limit).view(shape)
    return keep, 65536.0 / (65536 - limit) if limit < 65536 else 0.0


def drop(x, p, seed, offset=0):
    keep, scale = kept(x.shape, p, seed, offset)
    return torch.where(keep, x * scale, torch.zeros((), dtype=x.dtype))


def lookup(ids, table):
    inside = (ids >= 0) & (ids < table.shape[0])
    return torch.where(inside[..., None], table[torch.where(inside, ids, 0)], 0.0)


def embed(ids, table, scale=1.0, positions=None, position_table=None, dropout=None):
    """(value, bound without the output's rounding)"""
    t, x = table.double(), lookup(ids.long(), table.double()) * scale
    size = x.abs()
    if positions is not None:
        r = lookup(positions.long(), position_table.double())
        x, size = x + r, size + r.abs()
    if dropout:
        x, size = drop(x, *dropout), drop(size, *dropout)
    return x, size * 6 * U32      # scale, product, sum, factor, product: five roundings


def embed_grad(grad, ids, rows, scale=1.0, dropout=None, old=None):
    """The same of the table's gradient: a sum of n numbers in any order is off
    by at most n - 1 roundings of the sum of their sizes."""
    g = grad.double().view(-1, grad.shape[-1])
    if dropout:
        g = drop(g.view(grad.shape), *dropout).view(g.shape)
    ids = ids.reshape(-1).long()
    on = (ids >= 0) & (ids < rows)
    total = torch.zeros(rows, g.shape[1], dtype=torch.float64).index_add_(0, ids[on], g[on]) * scale
    size = torch.zeros_like(total).index_add_(0, ids[on], g[on].abs()) * abs(scale)
    count = torch.bincount(ids[on], minlength=rows)[:, None]
    bound = size * (count + 5) * U32
    if old is not None:
        total, bound = total + old.double(), bound + (size + old.double().abs()) * 2 * U32
    return total, bound


def head(hidden, table, targets, weights=None, mean=True, grad_scale=1.0, accumulate=None, table_grad=None):
    """{name: (value, bound with the output's rounding)} of the loss and its gradients.

    A dot product of K terms in binary32 is off by at most K roundings of the
    sum of its terms' sizes (two half steps each, should the matrix cores cut
    instead of round). That moves z, and with it l by as much at most twice,
    and p by a factor of exp of twice that. e is a number of 11 bits (bf16
    operands) with a floor of 2^-40, G one of the operands' type."""
    dt, bf = hidden.dtype, hidden.dtype == torch.bfloat16
    h, w, y = hidden.double(), table.double(), targets.long()
    n, v = h.shape[0], w.shape[0]
    part = torch.ones(n, dtype=torch.float64) if weights is None else weights.double()
    on = (y >= 0) & (y < v) & (part != 0)
    part = torch.where(on, part, 0.0)
    if mean:
        part = part / (float(part.sum()) or 1.0)
    h = torch.where(on[:, None], h, 0.0)
    at = torch.where(on, y, 0)[:, None]
    z = h @ w.t()
    dz = (h.abs() @ w.abs().t()) * 2 * (h.shape[1] + 2) * U32 + z.abs() * 2 * U32
    dz = dz.amax(1, keepdim=True)
    lse = torch.logsumexp(z, 1, keepdim=True)
    losses = torch.where(on, (lse - z.gather(1, at))[:, 0], 0.0)
    few = 2 * (v + 32) * U32
    dl = torch.where(on, 2 * dz[:, 0] + few + losses.abs() * 4 * U32, 0.0)
    loss = (losses * part).sum()
    out = {"losses": (losses, dl), "loss": (loss.view(1), ((dl * part.abs()).sum() + abs(loss) * 4 * U32).view(1))}
    g = part[:, None] * grad_scale
    p = torch.exp(z - lse)
    onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
    G = g * (p - onehot)
    dp = p * (torch.expm1(2 * dz) + few + 16 * U32 + (2.0 ** -12 if bf else 0.0)) + (2.0 ** -40 if bf else 2.0 ** -126)
    dG = g.abs() * (dp + 4 * U32) + half_step(dt) * (G.abs() + g.abs() * dp)
    dG = torch.where(on[:, None], dG, 0.0)

    def bound(x, d_left, left, right, k, to):
        return d_left @ right.abs() + 2 * (k + 2) * U32 * (left.abs() @ right.abs()) + half_step(to) * x.abs()

    gh = G @ w
    b = bound(gh, dG, G, w, v, dt)
    out["grad_hidden"] = (gh, b * (1 + half_step(dt)))
    to = table_grad or dt
    gw = G.t() @ h
    b = bound(gw, dG.t(), G.t(), h, n, to)
    if accumulate is not None:
        gw = gw + accumulate.double()
        b = b + (accumulate.double().abs() + gw.abs()) * (2 * U32 + half_step(to))
    out["grad_table"] = (gw, b * (1 + half_step(to)))
    return out


def check(got, want, bound, what="", rounded=None):
    """|got - want| <= bound, plus half a step of `rounded`'s type."""
    got = got.detach().cpu()
    if rounded is not None:
        bound = bound + half_step(rounded) * (want.abs() + bound) + torch.finfo(rounded).tiny * half_step(rounded)
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), off[bad].max().item(), bound[bad].max().item(),
                           torch.nonzero(bad)[:3].tolist())
