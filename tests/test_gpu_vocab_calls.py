"""Calls of the vocabulary operators that their documentation allows, beside
those of the tests by operator."""
import pytest
import torch

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
