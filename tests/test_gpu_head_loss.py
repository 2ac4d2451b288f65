"""Softmax cross entropy against the vocabulary table, and its gradients,
against a 64-bit reference with bounds from the arithmetic."""
import numpy as np
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero
from test_gpu_vocab import placed, untouched

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(n, vocab, width, dtype, seed=0, ignored=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed + 31 * n + vocab)
    table = (torch.randn(vocab, width, generator=g) * 0.1).to(dtype)
    hidden = torch.randn(n, width, generator=g) * (spread / 0.1 / width ** 0.5)
    targets = torch.randint(0, vocab, (n,), generator=g)
    hidden = (hidden + (torch.rand(n, 1, generator=g) * 6 / (0.01 * width)) * table[targets].float()).to(dtype)
    targets[torch.rand(n, generator=g) < ignored] = -100
    return hidden, table, targets, g


def run(hidden, table, targets, gap=0, weights=None, mean=True, grad_scale=1.0, piece=0, accumulate=None,
        table_grad=None, grads=True, device_ids=torch.int64, what=""):
    dt = hidden.dtype
    flat, t = placed(table, gap)
    losses = torch.full((hidden.shape[0],), 9.0, device="cuda")
    kw = {}
    if grads:
        to = table_grad or dt
        start = accumulate if accumulate is not None else torch.full_like(table, 5.0, dtype=to)
        gflat, gt = placed(start, gap)
        kw = dict(grad_hidden=torch.full_like(hidden, 3.0, device="cuda"), grad_table=gt, accumulate=accumulate is not None)
    loss = zero.head_loss(hidden.cuda(), t, targets.to(device_ids).cuda(), weights=None if weights is None else weights.cuda(),
                          reduction="mean" if mean else "sum", grad_scale=grad_scale, losses=losses, piece_rows=piece, **kw)
    want = ref.head(hidden, table, targets, weights, mean, grad_scale, accumulate, table_grad)
    ref.check(loss, *want["loss"], (what, "loss"))
    ref.check(losses, *want["losses"], (what, "losses"))
    if grads:
        assert untouched(gflat, gap, table.numel())
        ref.check(kw["grad_hidden"], *want["grad_hidden"], (what, "grad_hidden"))
        ref.check(gt, *want["grad_table"], (what, "grad_table"))
        kw["grad_table"] = gt
    return {"loss": loss, "losses": losses, **kw}


SIZES = [(1, 1, 1), (1, 2, 3), (1, 1000, 64), (2, 127, 8), (5, 128, 65), (16, 129, 64), (31, 300, 100), (32, 256, 128),
         (33, 257, 127), (64, 1000, 192), (100, 511, 64), (127, 513, 72), (128, 640, 256), (129, 2000, 33),
         (255, 1023, 320), (257, 1025, 129), (300, 5000, 64), (513, 777, 96)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width", SIZES)
def test_head_loss(n, vocab, width, dtype):
    hidden, table, targets, g = make(n, vocab, width, dtype)
    run(hidden, table, targets)
    run(hidden, table, targets, gap=1, mean=False, grad_scale=0.5, device_ids=torch.int32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width", [(3000, 7000, 136), (700, 33000, 64), (2100, 2500, 1000)])
def test_head_loss_over_large_tiles(n, vocab, width, dtype):
    hidden, table, targets, g = make(n, vocab, width, dtype, ignored=0.3)
    run(hidden, table, targets)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width", [(1, 16640, 128), (3, 16800, 30), (40, 60000, 64), (2, 33000, 129), (9000, 50, 64)])
def test_few_tiles_of_many_parts(n, vocab, width, dtype):
    """One tile's long axis is shared out, in parts that do not come out even."""
    hidden, table, targets, g = make(n, vocab, width, dtype)
    run(hidden, table, targets)


@pytest.mark.parametrize("n", [1, 32, 33, 64, 65, 128, 129, 192, 193, 256])
@pytest.mark.parametrize("vocab,width", [(17000, 40), (16999, 200), (32768, 320), (32769, 320)])
def test_few_rows_of_a_long_table(n, vocab, width):
    """Fewer stages than LDS has places for, as many, and more."""
    hidden, table, targets, g = make(n, vocab, width, BF, ignored=0.1 if n > 1 else 0.0)
    run(hidden, table, targets)
    run(hidden, table, targets, grads=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_than_a_grid_has_lines(dtype):
    hidden, table, targets, g = make(70001, 40, 16, dtype, ignored=0.01)
    run(hidden, table, targets)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,vocab,width", [(1, 50, 16), (70, 1000, 64), (200, 3000, 65)])
def test_loss_alone(n, vocab, width, dtype):
    hidden, table, targets, g = make(n, vocab, width, dtype, ignored=0.2)
    run(hidden, table, targets, grads=False)
    run(hidden, table, targets, grads=False, piece=17)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("piece", [1, 7, 64, 100, 299, 300, 1000])
def test_pieces(dtype, piece):
    hidden, table, targets, g = make(300, 700, 96, dtype, ignored=0.4)
    for table_grad in (BF, F32):
        run(hidden, table, targets, piece=piece, table_grad=table_grad, what=table_grad)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("table_grad", [BF, F32])
@pytest.mark.parametrize("piece", [0, 90])
def test_added_to_what_is_there(dtype, table_grad, piece):
    hidden, table, targets, g = make(200, 600, 72, dtype)
    old = (torch.randn(600, 72, generator=g) * 0.01).to(table_grad)
    run(hidden, table, targets, accumulate=old, table_grad=table_grad, gap=3, piece=piece)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights(dtype):
    hidden, table, targets, g = make(150, 400, 64, dtype, ignored=0.1)
    w = torch.rand(150, generator=g)
    w[::7] = 0.0
    for mean in (False, True):
        run(hidden, table, targets, weights=w, mean=mean, grad_scale=128.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("outside", [-100, -1, 300, 2 ** 40])
def test_no_row_takes_part(dtype, outside):
    hidden, table, targets, g = make(40, 300, 64, dtype)
    hidden[3] = float("nan")
    for mean in (False, True):
        got = run(hidden, table, torch.full((40,), outside), mean=mean)
        assert got["loss"].item() == 0 and not got["losses"].any()
        assert not got["grad_hidden"].any() and not got["grad_table"].any()
    old = torch.randn(300, 64, generator=g).to(dtype)
    got = run(hidden, table, torch.full((40,), outside), accumulate=old, piece=16)
    assert torch.equal(got["grad_table"].cpu(), old)


def test_no_rows():
    table = torch.randn(50, 16, device="cuda")
    gt, gh = torch.ones(50, 16, device="cuda"), torch.empty(0, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert zero.head_loss(gh, table, none, grad_hidden=gh.clone(), grad_table=gt, accumulate=True).item() == 0
    assert (gt == 1).all()
    zero.head_loss(gh, table, none, grad_table=gt)
    assert (gt == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_take_no_part_may_hold_anything(dtype):
    hidden, table, targets, g = make(90, 500, 64, dtype)
    targets[::4], clean = -100, hidden.clone()
    clean[::4] = 0.0
    w = torch.ones(90)
    w[1::4] = 0.0
    want = run(clean, table, targets, weights=w)
    dirty = clean.clone()
    dirty[::4], dirty[1::8], dirty[5::8] = float("nan"), float("inf"), torch.finfo(dtype).max
    got = run_dirty(dirty, table, targets, w)
    for k in want:
        if torch.is_tensor(want[k]):
            assert torch.equal(got[k], want[k]), k


def run_dirty(hidden, table, targets, w):
    losses = torch.empty(hidden.shape[0], device="cuda")
    gh, gt = torch.empty_like(hidden, device="cuda"), torch.empty_like(table, device="cuda")
    loss = zero.head_loss(hidden.cuda(), table.cuda(), targets.cuda(), weights=w.cuda(), losses=losses, grad_hidden=gh, grad_table=gt)
    return {"loss": loss, "losses": losses, "grad_hidden": gh, "grad_table": gt}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_logits(dtype):
    """Entries of the vocabulary whose logit is minus infinity have p = 0; a
    row with a NaN has a NaN loss and leaves the others' losses alone."""
    hidden = torch.ones(4, 64, dtype=dtype)
    table = torch.zeros(700, 64, dtype=dtype)
    table[256:] = float("-inf")          # whole tiles of them
    table[1] = 0.01
    targets = torch.tensor([0, 1, 2, 3])
    hidden[2, 5] = float("nan")
    losses = torch.empty(4, device="cuda")
    zero.head_loss(hidden.cuda(), table.cuda(), targets.cuda(), losses=losses)
    z = torch.zeros(256, dtype=torch.float64)
    z[1] = float(table[1, 0]) * 64
    want = torch.logsumexp(z, 0) - z[:4]
    got = losses.cpu().double()
    assert got[2].isnan()
    on = torch.tensor([0, 1, 3])
    # 64 products and their sum, 256 exponentials and theirs
    assert ((got - want)[on].abs() < 2 * (64 + 256 + 32) * ref.U32).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spread", [0.0, 30.0, 300.0])
def test_flat_and_steep_rows(dtype, spread):
    hidden, table, targets, g = make(70, 1500, 64, dtype, spread=spread)
    run(hidden, table, targets)


def test_same_call_same_bits():
    hidden, table, targets, g = make(1500, 4000, 128, BF, ignored=0.2)
    a, b = (run(hidden, table, targets, piece=p) for p in (0, 0))
    for k in ("loss", "losses", "grad_hidden", "grad_table"):
        assert torch.equal(a[k], b[k]), k


def test_gradient_against_differences():
    """Central differences of the loss in single entries of both operands, fp32:
    the quotient is off by the loss's own roundings over the step and by the
    third derivative, at most 2 |x|^3 step^2 with |x| the other operand's entries."""
    hidden, table, targets, g = make(6, 40, 8, F32)
    h, t, y = hidden.cuda(), table.cuda(), targets.cuda()
    gh, gt = torch.empty_like(h), torch.empty_like(t)
    zero.head_loss(h, t, y, reduction="sum", grad_hidden=gh, grad_table=gt)
    bound = ref.head(hidden, table, targets, mean=False)["loss"][1].item()
    for x, grad, other in ((h, gh, table.abs().max().item()), (t, gt, hidden.abs().max().item())):
        step = 2.0 ** -5 / max(1.0, other)
        for r, c in [(0, 0), (3, 5), (5, 7), (1, 2)]:
            old = x[r, c].item()
            values = []
            for s in (step, -step):
                x[r, c] = old + s
                values.append((zero.head_loss(h, t, y, reduction="sum").double().item(), x[r, c].item()))
            x[r, c] = old
            quotient = (values[0][0] - values[1][0]) / (values[0][1] - values[1][1])
            rows = 1 if x is h else 6
            assert abs(quotient - grad[r, c].item()) < 2 * bound / step + 2 * rows * other ** 3 * step ** 2 + 1e-6


def test_replayed_and_on_another_stream():
    hidden, table, targets, g = make(400, 3000, 128, BF, ignored=0.2)
    h, t, y = hidden.cuda(), table.cuda(), targets.cuda()

    def call(stream=None):
        out = dict(losses=torch.empty(400, device="cuda"), grad_hidden=torch.empty_like(h), grad_table=torch.empty_like(t))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out["loss"] = zero.head_loss(h, t, y, stream=stream, **out)
        return out

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    side = torch.cuda.Stream()
    for step in range(3):
        h.copy_((torch.randn(400, 128, generator=g) * 2).to(BF))
        y.copy_(torch.randint(-1, 3000, (400,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want, other = call(), call(side)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(held[k], want[k]), k
            assert torch.equal(other[k], want[k]), k


@pytest.mark.parametrize("seed", range(10))
def test_drawn_sizes(seed):
    r = np.random.RandomState(seed)
    n, vocab, width = (max(1, int(np.exp(r.uniform(0, np.log(m))))) for m in (1200, 9000, 500))
    dt = [BF, F32][seed % 2]
    hidden, table, targets, g = make(n, vocab, width, dt, seed, ignored=[0.0, 0.3][seed // 2 % 2])
    run(hidden, table, targets, gap=int(r.randint(0, 9)), piece=int(r.choice([0, max(1, n // 3)])), mean=bool(r.randint(2)),
        what=(n, vocab, width))
