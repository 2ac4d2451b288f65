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


# ------------------------------------------------ bound tensors and their streams

class _Tensor:
    """As much of a device tensor as bind asks for."""
    device, dtype = torch.device("cuda", 0), torch.float32

    def __init__(self):
        self.used_on = []

    def is_contiguous(self):
        return True

    def numel(self):
        return 6

    def data_ptr(self):
        return 4096

    def element_size(self):
        return 4

    def record_stream(self, stream):
        self.used_on.append(stream.cuda_stream)


@pytest.fixture
def state(monkeypatch):
    """An AdamWState of one (2, 3) and one empty parameter whose library takes
    every call; current[0] is the current stream, st.capturing[0] whether a
    call's stream is being captured."""
    current, capturing = [0], [False]
    fake = SimpleNamespace(zero_adamw_bind=lambda *a: 0, zero_adamw_sumsq=lambda *a: 0,
                           zero_adamw_step=lambda *a: 0, zero_destroy=lambda *a: None)
    monkeypatch.setattr(zero, "lib", lambda: fake)
    monkeypatch.setattr(zero, "_raw_stream", lambda index: current[0])
    monkeypatch.setattr(zero, "_capturing", lambda *a: capturing[0], raising=False)
    monkeypatch.setattr(zero, "_torch_stream",
                        lambda s, device: SimpleNamespace(cuda_stream=current[0]) if s is None else s,
                        raising=False)
    st = object.__new__(zero.AdamWState)
    st.device, st.shapes, st._sizes = _Tensor.device, [(2, 3), (0,)], [(6, 6, 0), (0, 0, 0)]
    st._h, st._bound, st._bound_on = SimpleNamespace(value=0), None, 0
    st._captured, st.capturing = [], capturing
    return st, current


SIDE = SimpleNamespace(cuda_stream=7)


@pytest.mark.parametrize("bound_on,rebound_on,stream,used", [
    (0, 0, None, []),           # one stream throughout: the allocator orders it
    (7, 7, None, []),
    (0, 0, SIDE, [7]),          # the calls run on a stream given by hand
    (0, 7, None, [7]),          # the calls moved to another current stream
    (7, 0, None, [0]),
])
def test_a_rebind_keeps_replaced_tensors_for_its_stream(state, bound_on, rebound_on, stream, used):
    """A step on the bind's stream may still be reading the tensors that the
    next bind lets go of: they are marked as used there."""
    st, current = state
    g, o, second = _Tensor(), _Tensor(), _Tensor()
    current[0] = bound_on
    st.bind([[g, None]], [o, None], stream=stream)
    assert g.used_on == o.used_on == []
    current[0] = rebound_on
    st.bind([[second, None]], [second, None], stream=stream)
    assert g.used_on == o.used_on == used
    assert second.used_on == []


def test_a_captured_bind_keeps_its_tensors_and_those_before(state):
    """Until the first replay the device holds the earlier binding, and any
    later replay uploads the captured one again: both live as long as the
    state."""
    import weakref
    st, _ = state
    alive = []
    for captured in (False, True, False, False):
        st.capturing[0] = captured
        g, o = _Tensor(), _Tensor()
        alive.append((weakref.ref(g), weakref.ref(o)))
        st.bind([[g, None]], [o, None])
        del g, o
    assert [[r() is not None for r in p] for p in alive] == [
        [True, True], [True, True], [False, False], [True, True]]
    st.close()
    assert not any(r() is not None for p in alive for r in p)
