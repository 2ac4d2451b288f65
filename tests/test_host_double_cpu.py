"""The library's host side without a GPU: calls that need a context, and what
they hand to the kernels. Each call runs in a process of its own, so that one
that overruns its stack ends that process alone."""
import os
import subprocess
import sys

import pytest

import host_double

TESTS = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(TESTS)

pytestmark = pytest.mark.skipif(not host_double.available(), reason="g++ or the HIP headers missing")


@pytest.fixture(scope="module")
def so(tmp_path_factory):
    return host_double.build(str(tmp_path_factory.mktemp("host")))


def run(so, body):
    """The lines that `body` prints; H is the library."""
    script = (f"import sys; sys.path[:0] = [{ROOT!r}, {TESTS!r}]\n"
              "import ctypes, host_double\n"
              "import zero_partitioned_optimizer_flatten_amd as zero\n"
              f"H = host_double.Host({so!r}); L = H.L\n" + body)
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return r.stdout.splitlines()


# --------------------------------------- the per-parameter step on AdamW's states

PER_PARAMETER_STEP = """
world = {world}
h = H.adamw([(2 * world, 3), (world, 5)], world=world, rank=world - 1)
grads = H.pointers([H.malloc(4 * n) for q in range(world) for n in (6 * world, 5 * world)])
outs = H.pointers([H.malloc(4 * n) for n in (6, 5)])
assert L.zero_schedule_init(h, 5, None) == zero.ZERO_OK
was = L.double_launches()
rc = [L.zero_fsdp_step(h, grads, world, 0, outs, 0, 1, None),
      L.zero_fsdp_step_sched(h, grads, world, 0, outs, 0, None)]
t = ctypes.c_int64()
assert L.zero_schedule_get(h, ctypes.byref(t), None) == zero.ZERO_OK
print(rc[0], rc[1], L.double_launches() - was, t.value)
"""


@pytest.mark.parametrize("world", [17, 64, 256])
def test_per_parameter_step_refuses_more_replicas_than_it_takes(so, world):
    """An AdamW context may have a world of up to 256, the per-parameter step
    takes 16 replicas: refused before anything is gathered, launched or
    counted as a step."""
    assert run(so, PER_PARAMETER_STEP.format(world=world)) == ["-4 -4 0 5"]


@pytest.mark.parametrize("world", [1, 16])
def test_per_parameter_step_takes_what_fits(so, world):
    """One launch, then the scheduled step's two."""
    assert run(so, PER_PARAMETER_STEP.format(world=world)) == ["0 0 3 6"]


# ------------------------------------------------------------ state in and out

STATE = """
h = H.adamw([(700, 3)], bits={bits})
n = ctypes.c_int64()
L.zero_shard_info(h, ctypes.byref(n), None, None)
bufs = [H.malloc(4 * n.value) for _ in range(3)]
for call in (L.zero_get_state, L.zero_set_state):
    was = L.double_launches(), L.double_copies()
    for k in range(3):
        bad = list(bufs)
        bad[k] += 256                         # 256 bytes past the allocation's end
        print(call(h, *bad, None), end=" ")
    print(L.double_launches() - was[0], L.double_copies() - was[1], call(h, *bufs, None))
"""


@pytest.mark.parametrize("bits", [32, 8])
def test_a_refused_state_call_has_written_nothing(so, bits):
    """Whichever of the three buffers is too short."""
    assert run(so, STATE.format(bits=bits)) == ["-1 -1 -1 0 0 0"] * 2


# ---------------------------------------------------------------- store policy

POLICY = """
for n in {sizes}:
    h = H.adamw([(n // 2048, 2048)], bits={bits})
    ptr = H.pointers([4096])                  # no known allocation: not looked into
    assert L.zero_adamw_bind(h, ptr, 1, 1, ptr, 1, None) == zero.ZERO_OK
    assert L.zero_adamw_step(h, 1, None, 0.0, None) == zero.ZERO_OK
    print(L.double_adamw_streams())
    L.zero_destroy(h)
"""


@pytest.mark.parametrize("bits,per_piece", [(32, 12 * 2048), (8, 6 * 2048 + 128)])
def test_a_state_larger_than_half_the_infinity_cache_streams(so, bits, per_piece):
    """128 MiB of the state's own bytes, either kind: 12 an element, or 6 and
    two scales per 32."""
    pieces = (128 << 20) // per_piece
    sizes = [2048 * pieces, 2048 * (pieces + 1)]
    assert run(so, POLICY.format(sizes=sizes, bits=bits)) == ["0", "1"]


# ------------------------------------------------------------- a captured bind

CAPTURED = """
h = H.adamw([(700, 3)], bits={bits})
ptr = H.pointers([4096])
bind = lambda: L.zero_adamw_bind(h, ptr, 1, 1, ptr, 1, None)
L.double_capturing(1)
was = L.double_launches()
print(bind(), L.double_launches() - was, L.zero_adamw_step(h, 1, None, 0.0, None))
L.double_capturing(0)
grads_only = L.zero_adamw_bind(h, ptr, 1, 1, None, 1, None)
L.double_capturing(1)
print(grads_only, bind())                  # its outputs would be the first
L.double_capturing(0)
print(bind())
L.double_capturing(1)
print(bind(), L.zero_adamw_step(h, 1, None, 0.0, None))
"""


@pytest.mark.parametrize("bits", [32, 8])
def test_a_first_bind_is_not_captured(so, bits):
    """Captured, it would reach the device only with a replay, and a step
    before that would follow null pointers."""
    assert run(so, CAPTURED.format(bits=bits)) == ["-1 0 -1", "0 -1", "0", "0 0"]
