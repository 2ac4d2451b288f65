"""8-bit states whose blocks hold numbers of very different size."""
import math

import numpy as np
import pytest
import torch

import zero_partitioned_optimizer_flatten_amd as zero
from gpu_harness import log
from test_gpu_adamw import Job, _gpu  # noqa: F401 (_gpu: the fixture)
from test_adamw_codes_cpu import frozen_factor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.95)])
def test_step_on_blocks_of_mixed_magnitudes(betas):
    """Every code against the reference over 2^27 of magnitudes in a block, so
    that many are below the 2^-6 scales where e4m3 loses its mantissa."""
    j = Job([(40, 2048), (999,)], 1, 0, 1, torch.float32, torch.float32, 8, betas=betas)
    for k in range(6):
        x = j.rng.standard_normal(j.gflat[0].numel()) * 2.0 ** j.rng.uniform(-27, 0, j.gflat[0].numel())
        j.gflat[0].copy_(torch.from_numpy(x.astype(np.float32)))
        j.check_step(label=f"mixed {k}")
    j.close()


def _run(n, exponent, betas, start, steps):
    """r / |g| after `steps` steps of a constant gradient 2^-exponent."""
    st = zero.AdamWState([(n,)], 1, 0, 0.0, betas, 1e-8, state_bits=8, seed=5)
    g = torch.ldexp(torch.ones(n, device="cuda"), -exponent)
    zeros = torch.zeros(n, device="cuda")
    st.set_state(zeros, zeros, (start * g).square())
    st.bind([[g]], [zeros.clone()])
    for t in range(1, steps + 1):
        st.step(t)
    v = st.get_state()[2]
    st.close()
    return (v.double().sqrt() / g.double()).cpu().numpy().reshape(-1, 32)


def test_r_follows_its_gradients_within_2_to_the_12_of_its_blocks_largest():
    """Elements of 2^0 to 2^-12 in every block, b2 = 0.999, from a quarter of
    their gradient, 200 steps. All have three mantissa bits: 2^-12 of a largest
    in (224, 448] scales, both up to a quarter off, is above 2^-5 scales. So
    each keeps the bounds of a block of equals: the mean of n
    r's is at least the exact r less 5 sigma, each step's sigma being at most
    half a code step (1/16 of r) over sqrt(n); and at most sqrt(1.082) = 1.041
    times the exact one, plus as much (a step adds to the mean of r^2 at most
    its movement times the code step, ln(0.48/0.25) / 8 = 8.2% in all)."""
    n = 1 << 20
    exponent = (torch.arange(n, device="cuda") % 32) % 13
    got = _run(n, exponent, (0.9, 0.999), 0.25, 200)
    v = 0.0625
    for _ in range(200):
        v = 0.999 * v + 0.001
    place = np.arange(32) % 13
    for e in range(13):
        x = got[:, place == e]
        sigma = 5 / 16 * math.sqrt(200 / x.size)
        ratio = x.mean() / math.sqrt(v)
        log(f"2^-{e}: {ratio:.4f}")
        assert 1 - sigma <= ratio <= 1.041 + sigma, (e, ratio)


@pytest.mark.parametrize("betas,steps", [((0.9, 0.95), 400), ((0.9, 0.999), 3000)])
def test_r_far_below_its_blocks_largest_stays_within_the_stated_factor(betas, steps):
    """Below 2^-6 scales r moves only where a step takes it far enough, and may
    stay too small by the factor that frozen_factor derives (5% added, within
    which a move has a chance of at least a few percent a step)."""
    n = 1 << 15
    lane = torch.arange(n, device="cuda") % 32
    exponent = torch.where(lane == 0, 0, 8 + lane % 14)
    got = _run(n, exponent, betas, 0.0, steps)
    # r of the smallest is the least code, 2^-9 scales, whatever its gradient
    floor = 2.0 ** -9 / 224
    e = exponent.cpu().numpy().reshape(-1, 32)
    worst = 0.0
    for k in range(8, 22):
        x = got[e == k]
        log(f"2^-{k}: r/|g| {x.min():.3f} to {x.max():.3f}")
        if 2.0 ** -k > floor:
            worst = max(worst, 1.0 / x.min())
    log(f"b2 {betas[1]}: too small by up to {worst:.2f}, stated {frozen_factor(betas[1]):.2f}")
    assert (got[:, 1:] >= 1.0 / (1.05 * frozen_factor(betas[1]))).all()
