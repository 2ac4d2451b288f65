"""Embedding lookup, its gradient and dropout against 64-bit references."""
import numpy as np
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def placed(x, gap, device="cuda"):
    """x as a view `gap` elements into a larger vector, filled with sevens around it."""
    flat = torch.full((x.numel() + 2 * gap + 16,), 7.0, dtype=x.dtype)
    flat[gap:gap + x.numel()] = x.reshape(-1)
    flat = flat.to(device)
    return flat, flat[gap:gap + x.numel()].view(x.shape)


def untouched(flat, gap, n):
    return bool((flat[:gap] == 7).all()) and bool((flat[gap + n:] == 7).all())


def gen(seed):
    return torch.Generator().manual_seed(seed)


def zipf(n, rows, g, wide=True):
    u = torch.rand(n, generator=g, dtype=torch.float64)
    ids = (torch.exp(u * np.log(rows + 1.0)) - 1).long().clamp_(0, rows - 1)
    return ids if wide else ids.int()


# ------------------------------------------------------------------- lookup

@pytest.mark.parametrize("table_dtype,out_dtype", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("shape,rows,width,gap,p", [
    ((1,), 1, 1, 0, 0.0), ((1,), 5, 8, 1, 0.5), ((3, 5), 11, 7, 3, 0.3), ((2, 64), 100, 64, 0, 0.1),
    ((129,), 50, 65, 1, 0.25), ((7, 33), 1000, 768, 0, 0.1), ((77,), 333, 1025, 5, 0.9),
    ((4, 9), 10, 3, 0, 0.5)])
def test_embed(table_dtype, out_dtype, shape, rows, width, gap, p):
    g = gen(rows + width)
    n = int(np.prod(shape))
    table = torch.randn(rows, width, generator=g).to(table_dtype)
    context = 6
    pos_table = torch.randn(context, width, generator=g).to(table_dtype)
    tokens = zipf(n, rows, g).view(shape)
    positions = torch.randint(0, context, shape, generator=g)
    flat, t = placed(table, gap)
    _, pt = placed(pos_table, gap + 1)
    for use_pos in (False, True):
        for prob in {0.0, p}:
            d = zero.Dropout(prob, 0xABCDEF0123456789, 5 << 40) if prob else None
            got = zero.embed(tokens.cuda(), t, scale=3.7, positions=positions.cuda() if use_pos else None,
                             position_table=pt if use_pos else None, dropout=d, dtype=out_dtype)
            assert got.shape == (*shape, width) and got.dtype == out_dtype
            want, bound = ref.embed(tokens, table, float(np.float32(3.7)), positions if use_pos else None,
                                    pos_table, (prob, 0xABCDEF0123456789, 5 << 40) if prob else None)
            ref.check(got, want, bound, (use_pos, prob), out_dtype)


@pytest.mark.parametrize("wide", [False, True])
def test_embed_ids_outside_the_table(wide):
    dt = torch.int64 if wide else torch.int32
    big = 2 ** 62 if wide else 2 ** 31 - 1
    tokens = torch.tensor([0, -1, 4, 5, 3, -big, big], dtype=dt)
    table = torch.randn(5, 24)
    got = zero.embed(tokens.cuda(), table.cuda(), positions=tokens.flip(0).cuda(), position_table=table.cuda())
    want, bound = ref.embed(tokens, table, 1.0, tokens.flip(0), table)
    ref.check(got, want, bound, rounded=F32)
    assert (got[1] == table[3].cuda() * 0 + ref.lookup(tokens.flip(0).long(), table)[1].cuda()).all()


def test_embed_without_tokens():
    out = zero.embed(torch.empty(0, 3, dtype=torch.int64, device="cuda"), torch.ones(4, 5, device="cuda"))
    assert out.shape == (0, 3, 5)


def test_embed_of_infinities_and_dropped_nans():
    table = torch.tensor([[float("inf"), float("-inf"), float("nan"), 1.0] * 16])
    tokens = torch.zeros(50, dtype=torch.int64)
    got = zero.embed(tokens.cuda(), table.cuda(), dropout=zero.Dropout(0.5, 3)).cpu()
    keep, scale = ref.kept((50, 64), 0.5, 3)
    want = torch.where(keep, table.expand(50, 64) * scale, torch.zeros(()))
    assert torch.equal(got.nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


# ----------------------------------------------------------------- gradient

GRAD_CASES = [
    # count, rows, width, gap, p, how tokens fall
    (1, 1, 1, 0, 0.0, "zipf"), (1, 3000, 8, 1, 0.0, "zipf"), (2, 2, 513, 0, 0.5, "same"),
    (7, 10, 7, 3, 0.3, "zipf"), (8, 4, 64, 0, 0.0, "same"), (9, 4, 64, 0, 0.0, "same"),
    (64, 700, 65, 1, 0.1, "zipf"), (500, 300, 768, 0, 0.1, "zipf"), (1000, 5, 20, 2, 0.0, "zipf"),
    (1025, 2000, 33, 0, 0.25, "same"), (4096, 70000, 16, 0, 0.0, "spread"), (4097, 131073, 9, 1, 0.0, "zipf"),
    (6000, 512, 24, 0, 0.0, "outside"), (10000, 257, 8, 0, 0.0, "half"), (20000, 1, 5, 0, 0.1, "same"),
    (70000, 9, 8, 0, 0.0, "half"),
]


def tokens_of(how, count, rows, g):
    if how == "same":
        return torch.full((count,), rows // 2)
    if how == "spread":
        return torch.randperm(rows, generator=g)[:count]
    ids = zipf(count, rows, g)
    if how == "half":
        ids[torch.rand(count, generator=g) < 0.5] = rows - 1
    if how == "outside":
        ids[torch.rand(count, generator=g) < 0.5] = -100
        ids[torch.rand(count, generator=g) < 0.2] = rows
    return ids


@pytest.mark.parametrize("grad_dtype,table_dtype", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("count,rows,width,gap,p,how", GRAD_CASES)
def test_embed_grad(grad_dtype, table_dtype, count, rows, width, gap, p, how):
    g = gen(count + width)
    tokens = tokens_of(how, count, rows, g)
    grad = torch.randn(count, width, generator=g).to(grad_dtype)
    old = torch.randn(rows, width, generator=g).to(table_dtype)
    d = zero.Dropout(p, 77, 2 ** 33) if p else None
    ids = tokens.cuda() if count % 2 else tokens.int().cuda()
    for accumulate in (False, True):
        flat, t = placed(old, gap)
        back = zero.embed_grad(grad.cuda(), ids, t, scale=1.5, dropout=d, accumulate=accumulate)
        assert back is t
        want, bound = ref.embed_grad(grad, tokens, rows, 1.5, (p, 77, 2 ** 33) if p else None, old if accumulate else None)
        ref.check(t, want, bound, accumulate, table_dtype)
        assert untouched(flat, gap, rows * width)
        # rows that no token names: zeros, or what was there, bit for bit
        idle = torch.ones(rows, dtype=torch.bool)
        idle[tokens[(tokens >= 0) & (tokens < rows)]] = False
        left = t.cpu()[idle]
        assert torch.equal(left, old[idle] if accumulate else torch.zeros_like(left))
        again = placed(old, gap)[1]
        zero.embed_grad(grad.cuda(), ids, again, scale=1.5, dropout=d, accumulate=accumulate)
        assert torch.equal(again.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("count", [1, 7, 8, 9, 63, 64, 65, 255, 256, 257])
@pytest.mark.parametrize("how", ["same", "half", "outside"])
def test_embed_grad_of_few_tokens(count, how):
    """Runs shorter and longer than one wave takes, up to the whole batch."""
    rows, width = 300, 520
    g = gen(count)
    tokens = tokens_of(how, count, rows, g)
    grad = torch.randn(count, width, generator=g).to(BF)
    old = torch.randn(rows, width, generator=g).to(BF)
    for accumulate in (False, True):
        flat, t = placed(old, 3)
        zero.embed_grad(grad.cuda(), tokens.cuda(), t, dropout=zero.Dropout(0.2, 5), accumulate=accumulate)
        want, bound = ref.embed_grad(grad, tokens, rows, 1.0, (0.2, 5, 0), old if accumulate else None)
        ref.check(t, want, bound, accumulate, BF)
        assert untouched(flat, 3, rows * width)


def test_embed_grad_without_tokens():
    empty, old = torch.empty(0, dtype=torch.int64, device="cuda"), torch.ones(300, 5, device="cuda")
    g = torch.empty(0, 5, device="cuda")
    assert (zero.embed_grad(g, empty, old.clone(), accumulate=True) == 1).all()
    assert (zero.embed_grad(g, empty, old.clone()) == 0).all()


def test_embed_grad_keeps_nan_to_its_row():
    tokens = torch.tensor([3, 1, 3, 2, -1])
    grad = torch.ones(5, 16)
    grad[1], grad[4] = float("nan"), float("inf")
    t = zero.embed_grad(grad.cuda(), tokens.cuda(), torch.zeros(6, 16, device="cuda")).cpu()
    assert t[1].isnan().all()
    assert torch.equal(t[[0, 2, 3, 4, 5]], torch.tensor([0.0, 1, 2, 0, 0])[:, None].expand(5, 16))


@pytest.mark.parametrize("seed", range(12))
def test_embed_grad_of_drawn_sizes(seed):
    r = np.random.RandomState(seed)
    g = gen(seed)
    count, rows, width = (int(np.exp(r.uniform(0, np.log(m)))) for m in (9000, 60000, 600))
    tokens = tokens_of(["zipf", "half", "outside"][seed % 3], count, rows, g)
    grad = torch.randn(count, width, generator=g).to([BF, F32][seed % 2])
    t = zero.embed_grad(grad.cuda(), tokens.cuda(), torch.empty(rows, width, device="cuda"))
    want, bound = ref.embed_grad(grad, tokens, rows)
    ref.check(t, want, bound, (count, rows, width), F32)


def test_embed_gradient_is_the_lookups():
    """Against differences of the lookup itself, in every table entry."""
    g = gen(4)
    tokens = torch.tensor([[0, 2, 2], [4, 0, 2]])
    table, up = torch.randn(5, 3, generator=g), torch.randn(2, 3, 3, generator=g)
    d = zero.Dropout(0.4, 9)

    def value(t):
        return (zero.embed(tokens.cuda(), t.cuda(), scale=2.0, dropout=d).double().cpu() * up.double()).sum()

    got = zero.embed_grad(up.cuda(), tokens.cuda(), torch.empty(5, 3, device="cuda"), scale=2.0, dropout=d).cpu()
    for r in range(5):
        for c in range(3):
            step = torch.zeros(5, 3)
            step[r, c] = 0.25
            # linear: the difference quotient is exact but for roundings of 18 numbers of size < 20
            quotient = (value(table + step) - value(table - step)) / 0.5
            assert abs(quotient - got[r, c]) < 18 * 20 * 8 * ref.U32 / 0.5


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("count", [1, 7, 8, 9, 255, 2048, 2049, 100003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 2.0 ** -17, 0.99999, 1.0])
def test_dropout(dtype, count, p):
    g = gen(count)
    x, add = (torch.randn(count, generator=g).to(dtype) for _ in range(2))
    seed, offset = 2 ** 64 - 3, 2 ** 64 - 1
    fx, dx = placed(x, 1)
    for residual in (None, add):
        flat, out = placed(torch.zeros_like(x), 3)
        got = zero.dropout(dx, zero.Dropout(p, seed, offset), add=None if residual is None else residual.cuda(), out=out)
        want = ref.drop(x.double(), p, seed, offset)
        size = want.abs()
        if residual is not None:
            want, size = want + residual.double(), size + residual.double().abs()
        ref.check(got, want, size * 4 * ref.U32, rounded=dtype)
        assert untouched(flat, 3, count)


def test_dropout_in_place_and_shape():
    x = torch.randn(5, 6, 7, device="cuda")
    d = zero.Dropout(0.3, 1, 2)
    want = zero.dropout(x, d, add=x)
    got = x.clone()
    assert zero.dropout(got, d, add=got, out=got) is got and torch.equal(got, want)
    assert zero.dropout(x[:0], d).shape == (0, 6, 7)


def test_dropout_drops_what_is_not_finite():
    x = torch.full((1000,), float("nan"), device="cuda")
    keep, _ = ref.kept((1000,), 0.5, 8)
    assert torch.equal(zero.dropout(x, zero.Dropout(0.5, 8)).isnan().cpu(), keep)


def test_dropout_shares_and_pairs():
    """Over 2^22 elements the share kept, and that of neighbours kept together,
    lie within five deviations of p's; other offsets and seeds are independent."""
    n, p = 1 << 22, 0.3
    x = torch.ones(n, device="cuda")
    a, b, c = (zero.dropout(x, zero.Dropout(p, s, o)) != 0 for s, o in ((1, 0), (1, 1), (2, 0)))
    q = 1 - round(p * 65536) / 65536
    for share, want in [(a, q), (a[1:] & a[:-1], q * q), (a[8:] & a[:-8], q * q), (a & b, q * q), (a & c, q * q)]:
        # neighbours' pairs are dependent in twos: three times the variance at most
        assert abs(share.double().mean().item() - want) < 5 * (3 * want * (1 - want) / n) ** 0.5


def test_dropout_counter_is_read_by_the_kernel():
    x = torch.ones(4096, device="cuda")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = zero.Dropout(0.5, 5, 100, counter)
    zero.dropout(x, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = zero.dropout(x, d)
        counter.add_(1)
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, zero.dropout(x, zero.Dropout(0.5, 5, 100 + step)))


# ------------------------------------------------------- streams and graphs

def test_on_a_stream_given_by_hand():
    tokens = zipf(3000, 400, gen(1)).cuda()
    table = torch.randn(400, 96, device="cuda")
    up = torch.randn(3000, 96, device="cuda")
    want = (zero.embed(tokens, table), zero.embed_grad(up, tokens, torch.empty_like(table)), zero.dropout(up, zero.Dropout(0.1, 1)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (zero.embed(tokens, table, stream=side), zero.embed_grad(up, tokens, torch.empty_like(table), stream=side),
           zero.dropout(up, zero.Dropout(0.1, 1), stream=side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_replayed_beside_eager_calls():
    """Two captured gradients with tokens of their own, replayed in turn among
    eager calls: each equals the eager result on the tokens it finds."""
    g = gen(2)
    tokens = [zipf(2000, 3000, g).cuda() for _ in range(2)]
    up = torch.randn(2000, 200, generator=g).cuda()
    zero.embed_grad(up, tokens[0], torch.empty(3000, 200, device="cuda"))
    graphs, outs = [], []
    for t in tokens:
        outs.append(torch.empty(3000, 200, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            zero.embed_grad(up, t, outs[-1])
    for step in range(3):
        for t, graph, out in zip(tokens, graphs, outs):
            t.copy_(zipf(2000, 3000, g).cuda())
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, zero.embed_grad(up, t, torch.empty_like(out)))


def test_two_streams_at_once():
    g = gen(3)
    tokens = [zipf(4000, 1000, g).cuda() for _ in range(2)]
    up = torch.randn(4000, 256, generator=g).cuda()
    want = [zero.embed_grad(up, t, torch.empty(1000, 256, device="cuda")) for t in tokens]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                outs[k].append(zero.embed_grad(up, tokens[k], torch.empty(1000, 256, device="cuda")))
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, want[k])
