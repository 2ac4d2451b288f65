"""What the Python binding refuses or passes on before it calls the library."""
from types import SimpleNamespace

import pytest
import torch

import zero_partitioned_optimizer_flatten_amd as zero


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), torch.device("cpu", 0), "meta"])
@pytest.mark.parametrize("make", [
    lambda d: zero.ShardState(10, 1, 0, 1e-3, device=d),
    lambda d: zero.FsdpShardState([(4, 3)], 1, 0, 1e-3, device=d),
    lambda d: zero.AdamWState([(4, 3)], 1, 0, 1e-3, device=d),
])
def test_a_state_refuses_a_device_that_is_no_gpu(make, device):
    with pytest.raises(ValueError, match="cuda"):
        make(device)


def test_a_stream_may_be_anything_with_a_handle():
    """Streams of other libraries, which know no torch device."""
    device = torch.device("cuda", 0)
    assert zero._stream_handle(SimpleNamespace(cuda_stream=0x1234), device) == 0x1234
