"""The loss against the vocabulary table where the tests by size do not go:
weights of either sign in one workgroup, in pieces and apart, logits that
overflow, rows that are not numbers, and calls at once."""
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero
from test_gpu_head_loss import BF, F32, make, run

pytestmark = pytest.mark.gpu


def weights_of(kind, n, g):
    w = torch.rand(n, generator=g)
    if kind == "signed":
        w = w - 0.4
    if kind == "cancelling":                      # exactly
        w[n // 2:2 * (n // 2)] = -w[:n // 2]
        w[2 * (n // 2):] = 0.0
    if kind == "negative":
        w = -w
    if kind == "wide":
        w = w * 2.0 ** torch.randint(-20, 20, (n,), generator=g).float()
    w[::7] = 0.0
    if kind == "cancelling":
        w[n // 2:2 * (n // 2)] = -w[:n // 2]
        assert float(w.double().sum()) == 0.0
    return w


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["positive", "signed", "cancelling", "negative", "wide"])
@pytest.mark.parametrize("n,vocab,piece", [(20, 400, 0), (20, 90, 0), (150, 400, 0), (150, 400, 40), (300, 700, 299)])
def test_weights_of_any_sign(n, vocab, piece, kind, dtype):
    hidden, table, targets, g = make(n, vocab, 64, dtype)
    w = weights_of(kind, n, g)
    for mean in (False, True):
        run(hidden, table, targets, weights=w, mean=mean, grad_scale=4.0, piece=piece, what=(kind, mean))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,piece", [(4, 0), (4, 3), (150, 0)])
def test_logits_that_overflow_downwards(n, piece, dtype):
    """Whole tiles of the vocabulary at minus infinity, of finite operands: p, G
    and their rows' gradients are 0, and the others as if those were not there."""
    hidden, table, targets, g = make(n, 256, 64, dtype)
    hidden = hidden.abs() + 1.0
    hidden, targets = hidden.to(dtype), targets % 256
    table = torch.cat((table, torch.full((444, 64), -3e38).to(dtype)))
    losses, gh, gt = torch.empty(n, device="cuda"), torch.empty_like(hidden, device="cuda"), torch.empty_like(table, device="cuda")
    loss = zero.head_loss(hidden.cuda(), table.cuda(), targets.cuda(), losses=losses, grad_hidden=gh, grad_table=gt, piece_rows=piece)
    want = ref.head(hidden, table[:256], targets)
    ref.check(loss, *want["loss"], "loss")
    ref.check(losses, *want["losses"], "losses")
    ref.check(gh, *want["grad_hidden"], "grad_hidden")
    ref.check(gt[:256], *want["grad_table"], "grad_table")
    assert not gt[256:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,piece", [(5, 0), (5, 2), (150, 0)])
@pytest.mark.parametrize("what", ["nan", "overflow"])
def test_rows_that_are_not_numbers(what, n, piece, dtype):
    """A row with a NaN, or with a logit of plus infinity, has a NaN loss and
    gradient; it makes the sum and the table's gradient NaN and no other row's."""
    hidden, table, targets, g = make(n, 700, 64, dtype)
    h = hidden.clone()
    if what == "nan":
        h[2, 5] = float("nan")
    else:
        h[2] = torch.finfo(dtype).max * torch.sign(table[300].float()).to(dtype)
    outs = []
    for x in (hidden, h):
        losses, gh, gt = torch.empty(n, device="cuda"), torch.empty_like(x, device="cuda"), torch.empty_like(table, device="cuda")
        loss = zero.head_loss(x.cuda(), table.cuda(), targets.cuda(), reduction="sum", losses=losses, grad_hidden=gh, grad_table=gt,
                              piece_rows=piece)
        outs.append((loss, losses, gh, gt))
    clean, got = outs
    others = torch.arange(n, device="cuda") != 2
    assert got[0].isnan().all() and got[1][2].isnan() and got[2][2].isnan().all()
    assert got[3].isnan().all() if what == "nan" else got[3].isnan().any()
    assert torch.equal(got[1][others], clean[1][others]) and torch.equal(got[2][others], clean[2][others])


@pytest.mark.parametrize("captured", [False, True])
def test_two_losses_at_once(captured):
    """Two calls on two streams, or two graphs of one call each, that run at the
    same time: a workspace each, and the bits of calls one after the other."""
    data = [[x.cuda() for x in make(n, 5000, 256, BF, seed=s, ignored=0.1)[:3]] for s, n in enumerate((900, 700))]

    def call(d, stream=None):
        out = dict(losses=torch.empty(d[0].shape[0], device="cuda"), grad_hidden=torch.empty_like(d[0]), grad_table=torch.empty_like(d[1]))
        out["loss"] = zero.head_loss(*d, stream=stream, **out)
        return out

    want = [call(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    if captured:
        graphs, held = [], []
        for d in data:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                held.append(call(d))
    for _ in range(5):
        if captured:
            for o in held:
                for x in o.values():
                    x.zero_()
            torch.cuda.synchronize()
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            got = held
        else:
            got = [call(d, s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in b:
                assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("contents", [0, 127, 255])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width,piece", [(3, 300, 40, 0), (70, 17000, 64, 0), (700, 3000, 200, 0), (700, 3000, 200, 128), (40, 60000, 64, 0)])
def test_workspace_may_hold_anything(monkeypatch, n, vocab, width, piece, dtype, contents):
    """Zeros, large numbers, NaN."""
    from zero_partitioned_optimizer_flatten_amd import vocab as binding
    plain = binding._Call.workspace
    monkeypatch.setattr(binding._Call, "workspace", lambda *a: plain(*a).fill_(contents))
    hidden, table, targets, g = make(n, vocab, width, dtype, ignored=0.3)
    run(hidden, table, targets, piece=piece, gap=1)
