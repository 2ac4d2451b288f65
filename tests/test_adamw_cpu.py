"""The many-tensor AdamW operators on a machine without a GPU: what the C ABI
refuses before it touches a device, and the reference of the GPU tests
against torch and against itself."""
import ctypes

import numpy as np
import pytest
import torch

import adamw_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero


def _init(dim0=(4,), row=(3,), world=2, rank=0, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, bits=32,
          n=None, null=False):
    h = ctypes.c_void_p()
    d = (ctypes.c_int64 * max(1, len(dim0)))(*dim0)
    r = (ctypes.c_int64 * max(1, len(row)))(*row)
    rc = zero.lib().zero_adamw_init(len(dim0) if n is None else n, None if null else d, r, world,
                                    rank, lr, b1, b2, eps, bits, 0, ctypes.byref(h))
    return rc, h


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(null=True), dict(dim0=(-1,)), dict(row=(0,)), dict(world=0), dict(rank=2),
    dict(rank=-1), dict(world=257), dict(b1=1.0), dict(b2=0.0), dict(eps=-1.0),
    dict(lr=float("inf")), dict(bits=16), dict(bits=0), dict(bits=4),
    dict(dim0=(1 << 62,), row=(4,)), dict(dim0=(1 << 62, 1 << 62), row=(1, 1)),
])
def test_init_refuses(kw):
    rc, h = _init(**kw)
    assert rc == zero.ZERO_EINVAL and not h.value
    assert zero.lib().zero_last_error()


@pytest.mark.parametrize("bits", [8, 32])
def test_init_refuses_more_than_one_launch_holds(bits):
    rc, h = _init(dim0=(1 << 36,), row=(1,), world=1, bits=bits)
    assert rc == zero.ZERO_EUNSUPPORTED and not h.value


def test_init_refuses_a_null_result():
    assert zero.lib().zero_adamw_init(1, None, None, 1, 0, 1e-3, 0.9, 0.9, 0.0, 32, 0,
                                      None) == zero.ZERO_EINVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("bits", [8, 32])
def test_init_without_device_reports_hip_error(bits):
    rc, h = _init(bits=bits)
    assert rc == zero.ZERO_EHIP and not h.value


def test_null_context_is_refused():
    L = zero.lib()
    p = ctypes.c_void_p()
    assert L.zero_adamw_groups(None, None, None, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_bind(None, None, 1, 0, None, 0, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_sumsq(None, None, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_step(None, 1, None, 1.0, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_step_sched(None, None, 1.0, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_state(None, ctypes.byref(p), None, None, None) == zero.ZERO_EINVAL


# ---------------------------------------------------------- the reference

def test_codes_are_e4m3_values():
    """Every stored value is an e4m3 value times its scale, at most one step
    from what it stands for. Below 2^-6 the step is 2^-9: there the cut takes
    less than a step of x's own octave, at most 2^-10, and rounding to the
    grid at most half of 2^-9, together one step again."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((4096, 32)) * 10.0 ** rng.uniform(-6, 2, (4096, 32)))
    n = rng.integers(0, 65536, x.shape).astype(np.float64)
    e = ref.scale_exponent(np.abs(x).max(1))[:, None]
    y = np.ldexp(ref.code_value(x, n, e, False), -e)
    assert np.abs(y).max() <= 448.0
    assert np.array_equal(torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy(), y)
    s = np.ldexp(x, -e)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(s), 2.0 ** -6))) - 3)
    assert np.all(np.abs(y - s) <= step)


def test_the_scale_is_the_least_that_holds_the_block():
    top = np.concatenate([2.0 ** np.arange(-120.0, 120.0), 1.75 * 2.0 ** np.arange(-120.0, 120.0),
                          np.nextafter(1.75, 2) * 2.0 ** np.arange(-120.0, 120.0)])
    e = ref.scale_exponent(top)
    assert np.all(top <= np.ldexp(448.0, e)) and np.all((top > np.ldexp(448.0, e - 1)) | (e == -126))
    assert ref.scale_exponent(np.zeros(1))[0] == -126


def test_rounding_is_unbiased():
    """Over all 65536 values of the noise the mean code is x itself, for x
    whose lowest bits the noise can resolve."""
    n = np.arange(65536.0)
    for x in (1.0, 1.06, 1.3, 200.123, 440.0, 0.02):
        x = np.ldexp(np.round(np.ldexp(np.frexp(x)[0], 20)), np.frexp(x)[1] - 20)   # 20 bits
        got = ref.code_value(np.full(65536, x), n, np.zeros(65536, int), False)
        assert abs(got.mean() - x) < 1e-12 * x


def test_noise_is_uniform_and_differs_by_element_step_and_seed():
    a, b = ref.noise(7, 100, 1 << 16)
    for x in (a, b):
        # mean of 65536 uniform 16-bit numbers: sigma 65536/sqrt(12)/256 = 73.9
        assert abs(x.mean() - 32767.5) < 5 * 73.9
        assert abs(np.corrcoef(x[:-1], x[1:])[0, 1]) < 5 / 256
        assert np.unique(x).size > 40000
    assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 256
    for other in (ref.noise(7, 101, 1 << 16), ref.noise(8, 100, 1 << 16)):
        assert abs(np.corrcoef(a, other[0])[0, 1]) < 5 / 256
    # a window is the window of the whole
    c, d = ref.noise(7, 100, 100, start=1234)
    assert np.array_equal(c, a[1234:1334]) and np.array_equal(d, b[1234:1334])


def test_steps_agree_with_torch():
    """The 64-bit step against torch.optim.AdamW in float64, and the 8-bit
    one before coding against the 32-bit one."""
    rng = np.random.default_rng(3)
    p0 = rng.standard_normal(500)
    w = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([w], lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(500), np.zeros(500)
    for t in range(1, 6):
        g = rng.standard_normal(500)
        w.grad = torch.from_numpy(g.copy())
        opt.step()
        sc = ref.scalars(3e-3, (0.9, 0.99), 1e-8, t)
        (p8, m8, r8), _ = ref.step8(p, m, np.sqrt(v), g, 0 * g, sc, 1.0, 0.1)
        (p, m, v), _ = ref.step32(p, m, v, g, 0 * g, sc, 1.0, 0.1)
        assert np.allclose(p, w.detach().numpy(), rtol=1e-12, atol=0)
        assert np.allclose(p, p8, rtol=1e-12, atol=0) and np.allclose(m, m8, rtol=1e-12, atol=0)
        assert np.allclose(v, r8 * r8, rtol=1e-12, atol=0)


def test_clipping_agrees_with_torch():
    rng = np.random.default_rng(4)
    g = rng.standard_normal(300)
    w = torch.nn.Parameter(torch.zeros(300, dtype=torch.float64))
    w.grad = torch.from_numpy(g.copy())
    total = torch.nn.utils.clip_grad_norm_([w], 0.5)
    got, _ = ref.mean_gradient([g], float(total) ** 2, 0.5)
    assert np.allclose(got, w.grad.numpy(), rtol=1e-12, atol=0)
