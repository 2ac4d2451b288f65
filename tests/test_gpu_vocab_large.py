"""Places that 32 bits do not hold: tables, tensors and pieces past 2^32
elements or bytes."""
import numpy as np
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def kept_at(first, n, p, seed):
    """Which of the elements first..first + n dropout keeps (first a multiple of 8)."""
    block = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    zeros, s = np.zeros_like(block), np.uint64(32)
    x = ref.philox((block & ref.M32, block >> s, zeros, zeros), (seed, 0))
    bits = np.stack([b for w in x for b in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    return torch.from_numpy(bits.reshape(-1)[:n].astype(np.int64) >= int(np.floor(p * 65536 + 0.5)))


def test_dropout_past_32_bits():
    n, p, seed = (1 << 32) + 77, 0.3, 12345
    x = torch.ones(n, dtype=BF, device="cuda")
    zero.dropout(x, zero.Dropout(p, seed), out=x)
    for first in (0, (1 << 31) - 512, (1 << 32) - 512, n // 8 * 8 - 1024):
        part = x[first:first + 1024 + (n % 8 if first > 1 << 32 else 0)].cpu()
        keep = kept_at(first, len(part), p, seed)
        want = torch.where(keep, torch.tensor(65536.0 / (65536 - 19661)), 0.0).to(BF)
        assert torch.equal(part, want)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_table_past_32_bits(ids):
    rows, width = 1_100_000, 4096                  # 4.5e9 elements
    table = torch.zeros(rows, width, dtype=BF, device="cuda")
    tokens = torch.tensor([0, 524287, 524288, 1048575, 1048576, rows - 1, 524288], dtype=ids, device="cuda")
    g = torch.Generator().manual_seed(1)
    values = torch.randn(6, width, generator=g).to(BF)
    table[tokens[:6].long()] = values.cuda()
    out = zero.embed(tokens, table)
    assert torch.equal(out.cpu(), values[[0, 1, 2, 3, 4, 5, 2]])
    grad = torch.randn(7, width, generator=g).to(BF)
    sums = grad[:6].double()
    sums[2] += grad[6].double()
    for many in (1, 100):                          # by runs and by spans
        table.fill_(2.0)
        zero.embed_grad(grad.repeat(many, 1).cuda(), tokens.repeat(many), table)
        got = table[tokens[:6].long()].cpu()
        want = sums * many
        # at most 2 * many terms to a row, none larger than their own and the last row's
        bound = (2 * many) ** 2 * ref.U32 * (grad[:6].double().abs() + grad[6].double().abs())
        ref.check(got, want, bound, many, BF)
        table[tokens[:6].long()] = 0
        assert not table.view(-1).view(torch.int64).any()


def test_piece_past_32_bits():
    """4.8 GB of exponentials at once: the first, the middle and the last rows and
    entries against the formula, the sums over all in 64 bits on the device."""
    n, vocab, width = 20000, 120000, 64
    g = torch.Generator().manual_seed(2)
    table = (torch.randn(vocab, width, generator=g) * 0.1).to(BF)
    hidden = (torch.randn(n, width, generator=g) * 2).to(BF)
    targets = torch.randint(0, vocab, (n,), generator=g)
    losses = torch.empty(n, device="cuda")
    gh, gt = torch.empty(n, width, dtype=BF, device="cuda"), torch.empty(vocab, width, device="cuda")
    zero.head_loss(hidden.cuda(), table.cuda(), targets.cuda(), reduction="sum", losses=losses, grad_hidden=gh,
                   grad_table=gt, piece_rows=n)
    at = torch.cat([torch.arange(8), torch.arange(n // 2, n // 2 + 8), torch.arange(n - 8, n)])
    want = ref.head(hidden[at], table, targets[at], mean=False)
    ref.check(losses.cpu()[at], *want["losses"], "losses")
    ref.check(gh.cpu()[at], *want["grad_hidden"], "grad_hidden")

    h, w = hidden.cuda().double(), table.cuda().double()
    lse, top = [], []
    for k in range(0, n, 1000):
        z = h[k:k + 1000] @ w.t()
        lse.append(torch.logsumexp(z, 1))
        size = h[k:k + 1000].abs() @ w.abs().t()   # of a dot product's terms, as in the reference
        top.append((size * 2 * (width + 2) + z.abs() * 2).amax(1) * ref.U32)
        del z, size
    lse, dz = torch.cat(lse)[:, None], torch.cat(top)[:, None]
    v = torch.cat([torch.arange(16), torch.arange(vocab // 2, vocab // 2 + 16), torch.arange(vocab - 16, vocab)]).cuda()
    p = torch.exp(h @ w[v].t() - lse)
    G = p - (targets.cuda()[:, None] == v).double()
    few = 2 * (vocab + 32) * ref.U32
    dp = p * (torch.expm1(2 * dz) + few + 16 * ref.U32 + 2.0 ** -12) + 2.0 ** -40
    dG = dp + 4 * ref.U32 + ref.half_step(BF) * (G.abs() + dp)
    want = G.t() @ h
    bound = dG.t() @ h.abs() + 2 * (n + 2) * ref.U32 * (G.abs().t() @ h.abs()) + ref.U32 * want.abs()
    ref.check(gt[v], want.cpu(), (bound * (1 + ref.U32)).cpu(), "grad_table")
