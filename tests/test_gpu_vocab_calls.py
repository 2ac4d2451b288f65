"""Calls of the vocabulary operators that their documentation allows, beside
those of the tests by operator."""
import pytest
import torch

import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(0,), (3, 0), (0, 7)])
def test_no_tokens_with_positions(dtype, shape):
    none = torch.empty(shape, dtype=torch.int64, device="cuda")
    table, places = (torch.ones(n, 8, dtype=dtype, device="cuda") for n in (10, 4))
    d = zero.Dropout(0.5, 1)
    out = zero.embed(none, table, positions=none, position_table=places, dropout=d)
    assert out.shape == (*shape, 8) and out.dtype == dtype
    grad = torch.ones(4, 8, dtype=dtype, device="cuda")
    zero.embed_grad(out, none, grad, dropout=d)
    assert not grad.any()


@pytest.mark.parametrize("rows", [131071, 131072, 131073, 262144, 1 << 20])
@pytest.mark.parametrize("n,add", [(257, True), (9000, False)])
def test_sort_groups_at_their_limits(rows, n, add):
    """Tables that give a workgroup of the sort as many ids as it takes, one less and one more."""
    g = torch.Generator().manual_seed(rows + n)
    ids = torch.randint(0, rows, (n,), generator=g)
    ids[:3], ids[3:6], ids[6::5] = rows - 1, torch.tensor([0, -1, rows]), ids[7]
    grad = torch.randn(n, 5, generator=g)
    old = torch.randn(rows, 5, generator=g)
    got = zero.embed_grad(grad.cuda(), ids.cuda(), old.cuda(), scale=1.5, accumulate=add)
    ref.check(got, *ref.embed_grad(grad, ids, rows, 1.5, None, old if add else None), "grad_table", F32)
