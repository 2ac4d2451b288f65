"""Rows whose target is all but certain. Every logit is one product of two short
numbers, exact in binary32, so the losses and G are bounded by the softmax's own
arithmetic: losses are not negative, and the gradient at the target, p - 1, never
points the wrong way."""
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# 8 significant bits at most. As multiples of log 2 they are far from the next number
# of binary32, on either side: 63.5, 202 and 254 by as much as 14e-6, 232 the other way.
HEIGHTS = [8.125, 10.0, 17.25, 30.0, 57.0, 63.5, 100.0, 202.0, 232.0, 254.0]
# Additions of a row's sum that meet the largest entry's 1: 32 in a lane and 2 across,
# then a row's tiles (500 at most here) over 16 lanes or more, and 6 across.
ADDS = 32 + 2 + 32 + 6


def make(n, vocab, width, dtype):
    """Row i has its height in column i alone; there the table has a 1 for its
    target and sixteenths up to a quarter for the others."""
    g = torch.Generator().manual_seed(n + vocab)
    a = torch.tensor([HEIGHTS[i % len(HEIGHTS)] for i in range(n)])
    hidden = torch.zeros(n, width)
    hidden[torch.arange(n), torch.arange(n)] = a
    table = torch.randint(-16, 5, (vocab, width), generator=g) / 16.0
    targets = torch.randperm(vocab, generator=g)[:n]
    table[targets, torch.arange(n)] = 1.0
    for x in (hidden, table):
        assert torch.equal(x, x.to(dtype).float())
    return hidden.to(dtype), table.to(dtype), targets, a.double()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width,piece", [
    (20, 1000, 64, 0),            # all in the loss's own workgroup
    (20, 1000, 64, 8),            # in pieces: the softmax apart
    (200, 1000, 256, 0),
    (20, 16000, 64, 0), (60, 16000, 64, 0), (120, 16000, 128, 0), (190, 16000, 192, 0), (250, 16000, 256, 0),
    (600, 9000, 640, 0), (900, 16000, 960, 300)])
def test_confident_rows(n, vocab, width, piece, dtype):
    hidden, table, targets, a = make(n, vocab, width, dtype)
    h, t, y = hidden.cuda(), table.cuda(), targets.cuda()
    losses, gt = torch.empty(n, device="cuda"), torch.empty(vocab, width, device="cuda")
    zero.head_loss(h, t, y, reduction="sum", losses=losses, grad_hidden=torch.empty_like(h), grad_table=gt, piece_rows=piece)
    at = torch.arange(n)
    d = a * (1.0 - table[:, :n].double())         # (vocab, n): how far below the target
    others = torch.exp(-d)
    others[targets, at] = 0.0
    tail = others.sum(0)
    want = torch.log1p(tail)
    # exp: the product with log2 e, its constant and the exponential itself, relative
    tail_off = (others * (2 * d + 32)).sum(0) * ref.U32
    off = tail_off + (ADDS + 4) * ref.U32 * (1 + tail) + want * 8 * ref.U32
    got = losses.cpu().double()
    assert got.min().item() >= 0
    ref.check(losses, want, off, "losses")

    # one product makes each of the table's entries: G itself times the height
    G = gt.cpu().double()[:, :n] / a
    p = others / (1 + tail)
    short = ref.half_step(dtype)
    at_target = -(tail / (1 + tail))
    got = G[targets, at]
    assert got.max().item() <= 0
    ref.check(got, at_target, (off + 8 * ref.U32) * (1 + short) + at_target.abs() * (short + 2 * ref.U32), "G at the target")
    # the others: their tile's largest, rounded as a multiple of log2 e, comes in too
    loose = p * ((2 * d + 4 * a + 64) * ref.U32 + off) + (2.0 ** -40 if dtype == BF else 2.0 ** -126)
    loose = loose + p * (2.0 ** -11 if dtype == BF else 0.0)
    loose = loose * (1 + short) + p * (short + 2 * ref.U32)
    loose[targets, at] = float("inf")
    ref.check(G, p, loose, "G")
