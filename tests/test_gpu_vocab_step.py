"""The vocabulary operators as a training step uses them: lookup with dropout,
loss and gradients into the flat gradient vector, the lookup's gradient added
to the tied table's, and the optimizer's step on that vector. Each operator is
checked on what the one before it made, the step bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CONTEXT, ROWS, WIDTH, BATCH = 12, 301, 23, 4      # odd rows: tensors follow each other at odd places
SHAPES = [(5,), (ROWS, WIDTH), (CONTEXT, WIDTH), (7,)]
NUMEL = sum(int(np.prod(s)) for s in SHAPES)


def views(flat):
    at, out = 0, []
    for s in SHAPES:
        n = int(np.prod(s))
        out.append(flat[at:at + n].view(s))
        at += n
    return out


class Model:
    """Tokens to a loss through one table, as the smallest language model does."""

    def __init__(self, dtype, device="cuda"):
        g = torch.Generator().manual_seed(3)
        self.dtype = dtype
        self.flat = (torch.randn(NUMEL, generator=g) * 0.3).to(dtype).to(device)
        self.grad = torch.zeros(NUMEL, dtype=dtype, device=device)
        _, self.table, self.places, _ = views(self.flat)
        _, self.table_grad, self.places_grad, _ = views(self.grad)
        self.positions = torch.arange(CONTEXT, device=device).expand(BATCH, CONTEXT).contiguous()
        self.counter = torch.zeros(1, dtype=torch.int64, device=device)

    def drop(self):
        return zero.Dropout(0.2, 11, 5, self.counter)

    def backward(self, tokens, targets):
        d = self.drop()
        x = zero.embed(tokens, self.table, scale=2.0, positions=self.positions, position_table=self.places, dropout=d)
        gx = torch.empty_like(x)
        loss = zero.head_loss(x, self.table, targets, grad_hidden=gx, grad_table=self.table_grad)
        head = self.table_grad.clone()
        zero.embed_grad(gx, tokens, self.table_grad, scale=2.0, dropout=d, accumulate=True)
        zero.embed_grad(gx, self.positions, self.places_grad, dropout=d)
        return loss, x, gx, head


def batch(step):
    g = torch.Generator().manual_seed(100 + step)
    tokens = torch.randint(0, ROWS, (BATCH, CONTEXT + 1), generator=g)
    targets = tokens[:, 1:].clone()
    targets[0, :5] = -100
    return tokens[:, :-1].contiguous(), targets.contiguous()


def check(m, tokens, targets, made, step):
    loss, x, gx, head = [t.cpu() for t in made]
    table, places = m.table.cpu(), m.places.cpu()
    drop = (0.2, 11, 5 + step)
    positions = m.positions.cpu()
    ref.check(x, *ref.embed(tokens, table, 2.0, positions, places, drop), "x", m.dtype)
    want = ref.head(x.view(-1, WIDTH), table, targets.view(-1))
    ref.check(loss, *want["loss"], "loss")
    ref.check(gx.view(-1, WIDTH), *want["grad_hidden"], "grad_hidden")
    ref.check(head, *want["grad_table"], "grad_table")
    ref.check(m.table_grad, *ref.embed_grad(gx, tokens, ROWS, 2.0, drop, head), "tied", m.dtype)
    ref.check(m.places_grad, *ref.embed_grad(gx, positions, CONTEXT, 1.0, drop), "places", m.dtype)


def bits(t):
    t = t.detach().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == BF else t.numpy()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_of_a_tied_model(dtype):
    m = Model(dtype)
    with zero.ShardState(NUMEL, 1, 0, 1e-2) as st:
        st.load_master(m.flat)
        o = oracle.ShardOracle(NUMEL, 1, 0, 1e-2)
        o.load_master(bits(m.flat))
        out = bits(m.flat).copy()
        for step in range(3):
            tokens, targets = batch(step)
            made = m.backward(tokens.cuda(), targets.cuda())
            check(m, tokens, targets, made, step)
            assert not views(m.grad)[0].any() and not views(m.grad)[3].any()
            st.step([m.grad], step + 1, m.flat)
            o.step([bits(m.grad)], step + 1, out)
            assert np.array_equal(bits(m.flat), out)
            m.counter.add_(1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_step_replays_as_the_next_ones(dtype):
    """Forward, backward, AdamW with clipping and the dropout's counter in one
    graph; every replay equals the eager steps of a twin, bit for bit, with
    eager work of both between the replays."""
    models = [Model(dtype), Model(dtype)]
    tokens, targets = (t.cuda() for t in batch(0))
    states, losses = [], []
    for m in models:
        st = zero.AdamWState(SHAPES, 1, 0, 1e-2, weight_decay=0.1)
        st.load_master(views(m.flat))
        st.bind([views(m.grad)], views(m.flat))
        st.schedule(next_t=1)
        states.append(st)

    def step(k):
        m, st = models[k], states[k]
        loss = m.backward(tokens, targets)[0]
        st.step_sched(st.sumsq(), 1.0)
        m.counter.add_(1)
        return loss

    for k in range(2):
        step(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(1)
    for n in range(1, 4):
        for a, b in zip((tokens, targets), batch(n)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        losses.append((held.item(), step(0).item()))
        torch.cuda.synchronize()
        assert losses[-1][0] == losses[-1][1]
        for a, b in ((models[0].flat, models[1].flat), (models[0].grad, models[1].grad)):
            assert np.array_equal(bits(a), bits(b))
    for st in states:
        st.close()
