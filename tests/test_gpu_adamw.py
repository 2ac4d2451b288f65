"""AdamW over many tensors on the GPU, with 32- and 8-bit states, and the sum
of squares it clips by, against the 64-bit forms of adamw_reference.

Tolerances are the bounds that adamw_reference derives for the sequence of
32-bit operations; a bf16 output adds half a step, 2^-8 of the value. Codes
of 8-bit states must be those of some number within the bound."""
import ctypes
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import adamw_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero
from gpu_harness import bits, log

pytestmark = pytest.mark.gpu

RAGGED = [(5,), (33, 7), (1,), (2048,), (2049,), (513, 3), (0, 4), (31,), (7, 300), (64, 64), (3,)]
BETAS, EPS, LR = (0.9, 0.95), 1e-8, 1e-3


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available()
    zero.lib()
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _f64(t):
    return t.detach().double().cpu().numpy()


class Job:
    """A state with bound buffers: every gradient and output is a window of
    one flat buffer, `gap` elements behind the one before, so alignments vary,
    and the elements between are guards."""

    def __init__(self, shapes, world, rank, n, gdt, odt, state_bits, gap=0, seed=0, rseed=11,
                 wd=None, scale=None, betas=BETAS, eps=EPS, outs=True):
        self.shapes, self.n, self.t, self.bits = shapes, n, 0, state_bits
        self.rng = np.random.default_rng(seed)
        k = len(shapes)
        self.wd = [0.1 if len(s) > 1 else 0.0 for s in shapes] if wd is None else wd
        self.scale = [0.5] + [1.0] * (k - 1) if scale is None else scale
        self.betas, self.eps, self.rseed = betas, eps, rseed
        self.st = zero.AdamWState(shapes, world, rank, LR, betas, eps, weight_decay=self.wd,
                                  lr_scale=self.scale, state_bits=state_bits, seed=rseed)
        self.sizes = [self.st.local_numel(i) for i in range(k)]
        self.at = [gap + sum(self.sizes[:i]) + gap * i for i in range(k)]
        total = sum(self.sizes) + gap * (k + 1)
        self.gflat = [torch.zeros(total, dtype=gdt, device="cuda") for _ in range(n)]
        self.oflat = torch.full((total,), 7.0, dtype=odt, device="cuda")
        self.grads = [self._windows(f) for f in self.gflat]
        self.outs = self._windows(self.oflat)
        p = [torch.from_numpy((self.rng.standard_normal(s) * 0.02).astype(np.float32)).cuda()
             for s in shapes]
        self.st.load_master(p)
        self.st.bind(self.grads, self.outs if outs else None)
        self.inside = np.zeros(total, bool)
        for a, s in zip(self.at, self.sizes):
            self.inside[a:a + s] = True

    def _windows(self, flat):
        return [flat[a:a + s] for a, s in zip(self.at, self.sizes)]

    def fill(self, std=1e-3):
        for f in self.gflat:
            f.copy_(torch.from_numpy((self.rng.standard_normal(f.numel()) * std)
                                     .astype(np.float32)))

    def state(self):
        """(master, m, v or r values, exponents of m, of r) as float64."""
        s = self.st.state_tensors()
        if self.bits == 32:
            return _f64(s["master"]), _f64(s["m"]), _f64(s["v"])
        e = s["scale"].view(torch.uint8).cpu().numpy().astype(int) - 127
        em, er = e[:, 0].reshape(-1), e[:, 1].reshape(-1)
        m = np.ldexp(_f64(s["m"]).reshape(-1, 32), em[:, None]).reshape(-1)
        r = np.ldexp(_f64(s["r"]).reshape(-1, 32), er[:, None]).reshape(-1)
        return _f64(s["master"]), m, r, em, er

    def raw(self):
        """Everything a step writes, as bytes."""
        torch.cuda.synchronize()
        s = self.st.state_tensors()
        return [x.contiguous().view(torch.uint8).cpu().numpy().copy()
                for x in [*s.values(), self.oflat]]

    def spread(self, pieces):
        """Per-tensor arrays laid out as the state."""
        out = np.zeros(self.st.shard)
        for i, x in enumerate(pieces):
            off = self.st.local[i][2]
            out[off:off + len(x)] = x
        return out

    def per_element(self, values):
        return self.spread([np.full(s, v) for s, v in zip(self.sizes, values)])

    def check_step(self, sumsq=None, max_norm=None, label=""):
        """One step, compared with the reference on the state before it."""
        self.t += 1
        before = self.state()
        s = None if sumsq is None else torch.tensor([sumsq], dtype=torch.float64, device="cuda")
        self.st.step(self.t, sumsq=s, max_norm=max_norm)
        torch.cuda.synchronize()
        self.compare(before, sumsq, max_norm, label)

    def compare(self, before, sumsq, max_norm, label):
        after = self.state()
        reps = [self.spread([_f64(g) for g in gl]) for gl in self.grads]
        g, dg = ref.mean_gradient(reps, sumsq, max_norm)
        sc = ref.scalars(LR, self.betas, self.eps, self.t)
        factor, decay = self.per_element(self.scale), self.per_element(self.wd)
        with np.errstate(invalid="ignore", divide="ignore"):
            step = ref.step32 if self.bits == 32 else ref.step8
            new, err = step(before[0], before[1], before[2], g, dg, sc, factor, decay)
        used = self.per_element([1.0] * len(self.sizes)) > 0
        for x, e, got, name in zip(new, err, after, ("master", "m", "v")):
            assert not got[~used].any(), f"{label}: {name} behind the last element"
            if self.bits == 8 and name != "master":
                continue
            d = np.abs(got - x)
            assert np.all(d[used] <= e[used]), (
                f"{label} t={self.t}: {name} off by up to {np.max((d / np.maximum(e, 1e-300))[used])} bounds")
        if self.bits == 8:
            nm, nr = ref.noise(self.rseed, self.t, self.st.shard)
            x = [np.where(used, v, 0.0) for v in (new[1], new[2])]
            e = [np.where(used, v, 0.0) for v in (err[1], err[2])]
            ref.check_codes(after[1], after[3], x[0], e[0], nm, False, f"{label} t={self.t} m")
            ref.check_codes(after[2], after[4], x[1], e[1], nr, True, f"{label} t={self.t} r")
        # the output is the master rounded once; the guards are untouched
        got = _f64(self.oflat)
        assert np.all(got[~self.inside] == 7.0), f"{label}: written outside the outputs"
        for i, s in enumerate(self.sizes):
            off = self.st.local[i][2]
            want = self.st.state_tensors()["master"][off:off + s].to(self.oflat.dtype)
            assert torch.equal(self.outs[i], want), f"{label}: output {i}"

    def close(self):
        self.st.close()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("n,gdt,odt,gap,clip", [
    (1, torch.float32, torch.float32, 0, None),
    (1, torch.bfloat16, torch.bfloat16, 1, 0.5),
    (2, torch.bfloat16, torch.float32, 3, None),
    (2, torch.float32, torch.bfloat16, 1, 1e9),
    (3, torch.bfloat16, torch.bfloat16, 0, 0.1),
    (4, torch.bfloat16, torch.bfloat16, 8, None),
    (5, torch.float32, torch.float32, 2, 0.5),
    (8, torch.bfloat16, torch.bfloat16, 5, 0.5),
    (8, torch.float32, torch.bfloat16, 0, None),
    (16, torch.bfloat16, torch.float32, 7, 0.5),
])
def test_step(state_bits, n, gdt, odt, gap, clip):
    j = Job(RAGGED, 1, 0, n, gdt, odt, state_bits, gap, seed=n + gap)
    for _ in range(3):
        j.fill()
        # a norm of 1.3: max_norm below it scales, above it does not
        j.check_step(None if clip is None else 1.69, clip, f"N={n} {gdt}->{odt} gap {gap}")
    j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("world", [2, 5, 16])
def test_every_kind_of_rank(state_bits, world):
    """First, middle and last rank: fewer rows, and none at all."""
    for rank in sorted({0, world // 2, world - 1}):
        j = Job(RAGGED, world, rank, 2, torch.bfloat16, torch.bfloat16, state_bits, 1, seed=rank)
        for _ in range(2):
            j.fill()
            j.check_step(label=f"rank {rank} of {world}")
        j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("length", [1, 2, 3, 4, 5, 31, 32, 33, 255, 256, 257, 511, 512, 513,
                                    2047, 2048, 2049, 4096, 4097, 10_000])
def test_every_length(state_bits, length):
    j = Job([(length,)], 1, 0, 1, torch.bfloat16, torch.bfloat16, state_bits, length % 5,
            seed=length)
    for _ in range(2):
        j.fill()
        j.check_step(label=f"length {length}")
    j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_rank_without_rows(state_bits):
    """Rank 4 of 5 holds no row of a 4-row parameter: nothing to launch."""
    st = zero.AdamWState([(4, 3)], 5, 4, LR, state_bits=state_bits)
    assert st.shard == 0 and st.state_bytes() == 0
    st.load_master([torch.zeros(4, 3, device="cuda")])
    st.bind([[None]], [None])
    s = torch.full((1,), 5.0, dtype=torch.float64, device="cuda")
    st.sumsq(out=s)
    assert s.item() == 0.0
    st.step(1, sumsq=s, max_norm=1.0)
    st.schedule(1)
    st.step_sched()
    assert st.schedule_next_t() == 2
    assert all(x.numel() == 0 for x in st.state_tensors().values())
    assert all(x.numel() == 0 for x in st.get_state())
    st.close()


@pytest.mark.parametrize("world,rank", [(1, 0), (4, 3)])
@pytest.mark.parametrize("gdt,odt", [(torch.bfloat16, torch.bfloat16),
                                     (torch.float32, torch.float32)])
def test_without_decay_and_clipping_it_is_the_per_parameter_step(world, rank, gdt, odt):
    """Bit for bit zero_fsdp_step, from the whole gradients of `world`
    replicas, several steps on."""
    shapes = [s for s in RAGGED if 0 not in s]
    a = zero.FsdpShardState(shapes, world, rank, LR, BETAS, EPS)
    b = zero.AdamWState(shapes, world, rank, LR, BETAS, EPS)
    gen = torch.Generator(device="cuda").manual_seed(5)
    p = [torch.randn(s, generator=gen, device="cuda") * 0.02 for s in shapes]
    a.load_master(p)
    b.load_master(p)
    grads = [[torch.empty(s, dtype=gdt, device="cuda") for s in shapes] for _ in range(world)]
    outs = [[torch.zeros(max(1, x.local_numel(k)), dtype=odt, device="cuda")[:x.local_numel(k)]
             for k in range(len(shapes))] for x in (a, b)]
    b.bind(grads, outs[1])
    for t in range(1, 5):
        for gl in grads:
            for g in gl:
                g.copy_(torch.randn(g.shape, generator=gen, device="cuda") * 1e-3)
        a.step(grads, t, outs[0])
        b.step(t)
        for x, y in zip(outs[0], outs[1]):
            assert torch.equal(x, y)
    for x, y in zip(a.state_pieces(a.get_state()), b.state_pieces(b.get_state())):
        assert all(torch.equal(i, k) for i, k in zip(x, y))
    # and zero_fsdp_step itself runs on the 32-bit context
    a.step(grads, 5, outs[0])
    FsdpStep = zero.FsdpShardState.step
    FsdpStep(b, grads, 5, outs[1])
    assert all(torch.equal(x, y) for x, y in zip(outs[0], outs[1]))
    a.close()
    b.close()


# ----------------------------------------------------------- sum of squares

def _sum_bound(reps, n_elems):
    """Binary64 throughout: the fold of N replicas errs by (N-1) 2^-53 of
    their magnitudes, a square and its addition by 2^-53 of the sum each
    (every addition's partial sum is at most the whole)."""
    return 2.0 ** -53 * (2 * len(reps) + n_elems + 4)


@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_sumsq(n, gdt, gap):
    j = Job(RAGGED, 1, 0, n, gdt, torch.float32, 32, gap, seed=3 * n + gap, outs=False)
    for k in range(3):
        j.fill(10.0 ** (-k))
        # guards hold what must not be read
        for f in j.gflat:
            f[torch.from_numpy(~j.inside).cuda()] = float("nan")
        got = j.st.sumsq().item()
        reps = [np.concatenate([_f64(g) for g in gl]) for gl in j.grads]
        mean = sum(reps) / n
        mass = sum(np.abs(r) for r in reps) / n
        want = math.fsum(mean * mean)
        assert abs(got - want) <= _sum_bound(reps, mean.size) * math.fsum(mass * mass)
        assert j.st.sumsq().item() == got, "the same gradients, other bits"
    j.close()


@pytest.mark.parametrize("n", [1, 3, 9])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
def test_sumsq_of_every_last_piece(n, gdt):
    """Rows of 256 elements, 4, 2 and 1 at a time, and a last one in part:
    every combination, in tensors of less and of more than a piece."""
    ends = [256 * r + d for r in range(8) for d in (1, 3, 4, 129, 254, 255, 256)]
    for gap in (1, 4):
        for first in (0, 2048):
            j = Job([(first + e,) for e in ends], 1, 0, n, gdt, torch.float32, 32, gap,
                    seed=first + gap, outs=False)
            j.fill()
            for f in j.gflat:
                f[torch.from_numpy(~j.inside).cuda()] = float("nan")
            reps = [np.concatenate([_f64(g) for g in gl]) for gl in j.grads]
            mean = sum(reps) / n
            mass = sum(np.abs(r) for r in reps) / n
            got = j.st.sumsq().item()
            assert (abs(got - math.fsum(mean * mean))
                    <= _sum_bound(reps, mean.size) * math.fsum(mass * mass))
            # one tensor's elements alone, so that none hides in the others' sum
            # (a sum of ones is exact; the mean's square rounds a few times by 2^-53)
            for k in range(0, len(ends), 5):
                for f in j.gflat:
                    f[torch.from_numpy(j.inside).cuda()] = 0.0
                for gl in j.grads:
                    gl[k].fill_(1.0)
                assert j.st.sumsq().item() == pytest.approx(first + ends[k], rel=1e-12)
            j.close()


@pytest.mark.parametrize("pieces", [1, 3, 4, 5, 17, 63, 64, 65, 68, 1000, 2044, 2049])
def test_sumsq_for_every_number_of_workgroups(pieces):
    """One to 512 workgroups of four pieces each, more than once: the last one
    to finish is found whatever their number, and the count starts anew."""
    j = Job([(2048 * pieces - 5,)], 1, 0, 1, torch.bfloat16, torch.float32, 32, 1, seed=pieces,
            outs=False)
    j.fill()
    x = _f64(j.grads[0][0])
    want = math.fsum(x * x)
    for _ in range(4):
        assert abs(j.st.sumsq().item() / want - 1) <= _sum_bound([x], x.size)
    j.close()


def test_sumsq_of_a_long_list_and_of_large_and_small_numbers():
    """More pieces than workgroups, and squares that leave binary32."""
    shapes = [(2048 * 2500 + 77,), (3, 5)]      # 2501 pieces, 2048 waves
    j = Job(shapes, 1, 0, 1, torch.float32, torch.float32, 32, 1, outs=False)
    for std in (1.0, 1e30, 1e-30):
        j.fill(std)
        x = np.concatenate([_f64(g) for g in j.grads[0]])
        got, want = j.st.sumsq().item(), math.fsum(x * x)
        assert abs(got / want - 1) <= _sum_bound([x], x.size)
    for bad in (float("nan"), float("inf")):
        j.fill()
        j.grads[0][0][1234] = bad
        assert not math.isfinite(j.st.sumsq().item())
    j.fill()
    assert math.isfinite(j.st.sumsq().item())
    j.close()


# ------------------------------------------------- what is not finite, and 0

@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sum_that_is_not_finite_writes_nothing(state_bits, bad):
    j = Job(RAGGED, 1, 0, 2, torch.bfloat16, torch.bfloat16, state_bits, 1)
    j.fill()
    j.check_step()
    was = j.raw()
    j.fill()
    j.grads[1][3][7] = bad
    s = j.st.sumsq()
    assert not math.isfinite(s.item())
    j.st.step(2, sumsq=s, max_norm=1.0)
    assert all(np.array_equal(a, b) for a, b in zip(was, j.raw()))
    j.fill()
    j.check_step(1.69, 0.5, "after a skipped step")
    j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_one_bad_gradient_spoils_its_own_element_alone(state_bits, bad):
    jobs = [Job(RAGGED, 1, 0, 1, torch.float32, torch.float32, state_bits, seed=2)
            for _ in range(2)]
    for j in jobs:
        j.fill()
        j.check_step()
    for j in jobs:
        j.fill()
        for g in (j.grads[0][3], j.grads[0][5]):
            g[100] = 0.0
    for g in (jobs[1].grads[0][3], jobs[1].grads[0][5]):
        g[100] = bad
    places = [jobs[0].st.local[k][2] + 100 for k in (3, 5)]
    for t in (2, 3):
        for j in jobs:
            j.st.step(t)
        a, b = jobs[0].state(), jobs[1].state()
        for x, y in zip(a[:3], b[:3]):
            assert not np.isfinite(y[places]).any()
            x, y = x.copy(), y.copy()
            x[places] = y[places] = 0.0
            assert np.array_equal(x, y), "a neighbour changed"
    for j in jobs:
        j.close()


def test_a_stored_moment_at_the_end_of_the_range_stays_alone():
    """m near the largest binary32 rounds to a code whose value is infinite:
    its neighbours keep their codes' values."""
    st = zero.AdamWState([(4096,)], 1, 0, LR, BETAS, EPS, state_bits=8)
    g = torch.zeros(4096, device="cuda")
    out = torch.zeros(4096, device="cuda")
    m = torch.full((4096,), 1e-3, device="cuda")
    v = torch.full((4096,), 1e-6, device="cuda")
    m[7] = torch.finfo(torch.float32).max
    st.set_state(torch.zeros(4096, device="cuda"), m, v)
    st.bind([[g]], [out])
    st.state_tensors()["m"].view(torch.uint8)[:32] = 0x38          # 1.0 each
    st.state_tensors()["m"].view(torch.uint8)[7] = 0x7E            # 448 * 2^120: infinite
    st.state_tensors()["scale"].view(torch.uint8)[0, 0, 0] = 247
    st.step(1)
    _, m2, _ = st.get_state()
    assert not math.isfinite(m2[7].item())
    want = np.float32(2.0 ** 120) * np.float32(BETAS[0])           # the others decay
    got = m2[:32].cpu().numpy()
    # a code is at most a step, an eighth of its octave, off
    assert (np.abs(np.delete(got, 7) / want - 1) <= 0.125).all()
    st.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_zero_gradients_and_large_ones(state_bits):
    """All zero (masters move by decay alone, and 8-bit blocks are zero), then
    gradients at both ends of what binary32 squares, then zero again."""
    j = Job(RAGGED, 1, 0, 1, torch.float32, torch.float32, state_bits)
    j.check_step(label="zero")
    assert not j.state()[1].any() and not j.state()[2].any()
    for std in (1e15, 1e-12, 1.0):
        j.fill(std)
        j.check_step(label=f"std {std}")
    for f in j.gflat:
        f.zero_()
    for _ in range(3):
        j.check_step(label="zero again")
    j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_eps_zero(state_bits):
    """Elements behind the last one stay zero where 0/0 is NaN."""
    j = Job([(5,), (2049,)], 1, 0, 1, torch.float32, torch.float32, state_bits, eps=0.0)
    for _ in range(2):
        j.fill()
        j.check_step(label="eps 0")
    j.close()


# --------------------------------------------------------------- 8-bit states

def test_every_code_reads_as_its_value():
    """All 256 codes on several scales through zero_get_state."""
    st = zero.AdamWState([(2048,)], 1, 0, LR, state_bits=8)
    s = st.state_tensors()
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8)
    s["m"].view(torch.uint8).copy_(codes)
    s["r"].view(torch.uint8).copy_(codes & 0x7F)
    e = torch.arange(128, dtype=torch.uint8, device="cuda").add_(90).view(1, 2, 64)
    s["scale"].view(torch.uint8).copy_(e)
    _, m, v = st.get_state()
    em, er = (x.astype(int) - 127 for x in s["scale"].view(torch.uint8).cpu().numpy()[0])
    for got, c, e, square in ((m, codes, em, False), (v, codes & 0x7F, er, True)):
        want = np.ldexp(_f64(c.view(torch.float8_e4m3fn)).reshape(64, 32), e[:, None]).reshape(-1)
        with np.errstate(over="ignore"):        # the largest squares leave binary32: infinite
            want = (want * want if square else want).astype(np.float32)
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)
    st.close()


def test_state_conversion():
    """get_state -> set_state keeps every value; the steps after it are the
    same bits; set_state rounds to the nearest code."""
    j = Job(RAGGED, 1, 0, 1, torch.bfloat16, torch.float32, 8, 1)
    for _ in range(3):
        j.fill()
        j.check_step()
    master, m, v = j.st.get_state()
    a = j.state()
    assert np.array_equal(_f64(m), a[1]) and np.array_equal(_f64(v), a[2] ** 2)
    k = Job(RAGGED, 1, 0, 1, torch.bfloat16, torch.float32, 8, 1, seed=99)
    # at an odd place of the caller's memory
    odd = [torch.zeros(x.numel() + 1, device="cuda")[1:].copy_(x) for x in (master, m, v)]
    k.st.set_state(*odd)
    assert all(np.array_equal(x, y) for x, y in zip(j.state()[:3], k.state()[:3]))
    k.t = j.t
    j.fill()
    for f, g in zip(k.gflat, j.gflat):
        f.copy_(g)
    for x in (j, k):
        x.check_step()
    assert all(np.array_equal(x, y) for x, y in zip(j.state()[:3], k.state()[:3]))
    # arbitrary values: nearest, ties to even, the block's scale
    n = j.st.shard
    gen = np.random.default_rng(8)
    mv = [(gen.standard_normal(n) * 10.0 ** gen.uniform(-4, 1, n)).astype(np.float32) for _ in range(2)]
    mv[1] = mv[1] ** 2
    j.st.set_state(master, *[torch.from_numpy(x).cuda() for x in mv])
    got = j.state()
    for x, y, e in ((mv[0].astype(np.float64), got[1], got[3]),
                    (np.sqrt(mv[1].astype(np.float64)).astype(np.float32).astype(np.float64), got[2], got[4])):
        assert np.array_equal(e, ref.scale_exponent(np.abs(x.reshape(-1, 32)).max(1)))
        z = torch.from_numpy(np.ldexp(x.reshape(-1, 32), -e[:, None]))
        w = z.float().to(torch.float8_e4m3fn).double().numpy()
        w = np.where(x.reshape(-1, 32) > 0, np.maximum(w, 2.0 ** -9), w) if x is not mv[0] and (x >= 0).all() else w
        assert np.array_equal(np.ldexp(w, e[:, None]).reshape(-1), y)
    j.close()
    k.close()


def test_state_bytes():
    st = zero.AdamWState([(100, 3), (7,)], 1, 0, LR, state_bits=8)
    assert st.state_bytes() == 307 * 6 + 2 * (10 + 1)
    st.close()
    st = zero.AdamWState([(100, 3), (7,)], 1, 0, LR)
    assert st.state_bytes() == 307 * 12
    st.close()


def test_small_moments_survive_and_rounding_is_unbiased():
    """A constant gradient under b2 = 0.999: rounding to nearest would leave r
    at its start, a quarter of |g|; stochastic rounding follows. Its means
    over n = 65536 elements: m is linear, so its mean is exact but for a sigma
    of half a code step (12.5%) over sqrt(n), 0.025% a step and less than
    sqrt(20) of that in all. r -> sqrt(b2 r^2 + (1-b2) g^2) is convex, so the
    mean is at least the exact r (less 5 sigma, of 200 steps); and a step
    adds to the mean of r^2 at most its movement times the code step, all
    steps together ln(0.48/0.25) * 12.5% = 8.2%, so that the mean of r is at
    most sqrt(1.082) = 1.041 times the exact one."""
    n = 65536
    st = zero.AdamWState([(n,)], 1, 0, 0.0, (0.9, 0.999), 1e-8, state_bits=8, seed=5)
    g = torch.full((n,), 1.0, device="cuda")
    st.set_state(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),
                 torch.full((n,), 0.0625, device="cuda"))
    st.bind([[g]], [torch.zeros(n, device="cuda")])
    v, m = 0.0625, 0.0
    for t in range(1, 201):
        st.step(t)
        v, m = 0.999 * v + 0.001, 0.9 * m + 0.1
    _, gm, gv = st.get_state()
    ratio = gv.double().sqrt().mean().item() / math.sqrt(v)
    sigma = 0.00025
    assert 1 - 5 * sigma * math.sqrt(200) <= ratio <= 1.041 + 5 * sigma * math.sqrt(200), ratio
    assert abs(gm.double().mean().item() - m) < 5 * sigma * math.sqrt(20)
    # an element 2^-20 of its block's largest keeps a second moment
    x = torch.zeros(n, device="cuda")
    x[::32], x[1::32] = 1.0, 2.0 ** -20
    g.copy_(x)
    st.set_state(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),
                 torch.zeros(n, device="cuda"))
    st.step(1)
    _, _, gv = st.get_state()
    assert (gv[1::32] > 0).all() and (gv[2::32] == 0).all()
    st.close()


# ------------------------------------------------------- together, and graphs

def _twins(state_bits, **kw):
    return [Job(RAGGED, 4, 1, 4, torch.bfloat16, torch.bfloat16, state_bits, 1, **kw)
            for _ in range(2)]


@pytest.mark.parametrize("state_bits", [32, 8])
def test_norm_clip_and_step_together_eager_and_replayed(state_bits):
    """The training loop's part: the norm of the rank's gradient, a sum over
    ranks (here this rank's alone), the clipped step; captured once with the
    device schedule and replayed, with eager work between, against the same
    calls made eagerly with host step counts."""
    a, b = _twins(state_bits)
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    b.st.schedule(1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.st.sumsq(out=s)
        b.st.step_sched(sumsq=s, max_norm=0.02)
    for t in range(1, 7):
        a.fill()
        for f, g in zip(b.gflat, a.gflat):
            f.copy_(g)
        if t == 4:                      # a new learning rate and decay for both
            a.st.set_lr(2e-3)
            b.st.schedule_lr(2e-3)
            for x in (a, b):
                x.st.set_groups([0.3] * len(RAGGED), [1.0] * len(RAGGED))
        a.st.step(t, sumsq=a.st.sumsq(), max_norm=0.02)
        graph.replay()
        if t % 2:                       # eager work between replays
            torch.cuda.synchronize()
            torch.ones(1000, device="cuda").sum().item()
        assert s.item() == a.st.sumsq().item() and math.sqrt(s.item()) > 0.02
        assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw())), f"t={t}"
    assert b.st.schedule_next_t() == 7
    # other buffers under the same graph
    for x in (a, b):
        flat = [torch.randn(f.numel(), device="cuda", generator=torch.Generator("cuda").manual_seed(q))
                .mul_(1e-3).to(f.dtype) for q, f in enumerate(x.gflat)]
        x.gflat, x.grads = flat, [x._windows(f) for f in flat]
        x.st.bind(x.grads, x.outs)
    a.st.step(7, sumsq=a.st.sumsq(), max_norm=0.02)
    graph.replay()
    assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw())), "after another bind"
    del graph
    a.close()
    b.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_captured_bind(state_bits):
    """Bind, norm and step in one graph, against the same calls made eagerly;
    eager steps on other gradients between the replays, each of which binds
    the captured ones again. A first bind is not captured."""
    a, b = _twins(state_bits)
    st = zero.AdamWState([(40,)], 1, 0, LR, state_bits=state_bits)
    g = torch.zeros(40, device="cuda")
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    b.st.schedule(1)
    others = [[x.clone() for x in gl] for gl in a.grads]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _einval(st.bind, [[g]], [g])
        b.st.bind(b.grads, b.outs)
        b.st.sumsq(out=s)
        b.st.step_sched(sumsq=s, max_norm=0.02)
    _einval(st.step, 1)
    for k in range(4):
        a.fill()
        for f, x in zip(b.gflat, a.gflat):
            f.copy_(x)
        a.st.bind(a.grads, a.outs)
        a.st.step(2 * k + 1, sumsq=a.st.sumsq(), max_norm=0.02)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw())), f"replay {k}"
        for gl in others:
            for x in gl:
                x.copy_(torch.randn(x.shape, device="cuda") * 1e-3)
        a.st.bind(others, a.outs)
        b.st.bind(others, b.outs)
        a.st.step(2 * k + 2)
        b.st.step_sched()
        assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw())), f"eager {k}"
    del graph
    for x in (a, b, st):
        x.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_scheduled_step_means_over_what_is_bound(state_bits):
    """Reduced gradients (one replica) on a rank of a world of four."""
    j = Job(RAGGED, 4, 1, 1, torch.float32, torch.float32, state_bits, 1)
    j.st.schedule(1)
    for _ in range(2):
        j.fill()
        before = j.state()
        j.t += 1
        j.st.step_sched()
        torch.cuda.synchronize()
        j.compare(before, None, None, "scheduled")
    j.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_another_stream(state_bits):
    a, b = _twins(state_bits)
    side = torch.cuda.Stream()
    for t in (1, 2, 3):
        a.fill()
        for f, g in zip(b.gflat, a.gflat):
            f.copy_(g)
        s = a.st.sumsq()
        a.st.step(t, sumsq=s, max_norm=0.02)
        side.wait_stream(torch.cuda.current_stream())
        r = b.st.sumsq(stream=side)
        b.st.step(t, sumsq=r, max_norm=0.02, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert s.item() == r.item()
        assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw()))
    a.close()
    b.close()


@pytest.mark.parametrize("by_hand", [True, False])
def test_replaced_buffers_live_until_a_running_step_is_done(by_hand):
    """A long step on a side stream, its gradient let go of by the next bind
    while it runs, and the main stream asking for memory of that size and
    overwriting it: the step sees the gradient it was bound to."""
    n = 1 << 26
    st = zero.AdamWState([(n,)], 1, 0, LR, BETAS, EPS)
    out = torch.zeros(n, device="cuda")
    other = torch.zeros(n, device="cuda")
    g = torch.full((n,), 1e-3, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    where = side if by_hand else None
    st.bind([[g]], [out], stream=where)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(None if by_hand else side):
        for t in range(1, 21):                    # about 0.3 ms each
            st.step(t, stream=where)
        del g
        st.bind([[other]], [out], stream=where)
    again = torch.full((n,), 1e3, device="cuda")  # on the main stream, at once
    torch.cuda.synchronize()
    assert (again == 1e3).all()
    m = st.get_state()[1]
    want = 1e-3 * (1.0 - BETAS[0] ** 20)
    # 20 steps, each off by 3 roundings of m at most (beta, product, sum)
    assert (m.double() / want - 1).abs().max().item() <= 80 * 2.0 ** -24
    st.close()


def test_a_stream_that_only_carries_its_handle():
    """Every call takes it, the sum's own output among them."""
    a, b = _twins(8)
    side = torch.cuda.Stream()
    bare = SimpleNamespace(cuda_stream=side.cuda_stream)
    a.fill()
    for f, g in zip(b.gflat, a.gflat):
        f.copy_(g)
    torch.cuda.synchronize()
    s, r = a.st.sumsq(), b.st.sumsq(stream=bare)
    a.st.step(1, sumsq=s, max_norm=0.02)
    b.st.step(1, sumsq=r, max_norm=0.02, stream=bare)
    torch.cuda.synchronize()
    assert s.item() == r.item()
    assert all(np.array_equal(x, y) for x, y in zip(a.raw(), b.raw()))
    a.close()
    b.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_new_state_on_a_stream_of_its_own(state_bits):
    """Everything after the constructor on a side stream that waits for
    nothing: the constructor leaves no work behind on its own stream. Decay as
    an array, the device without its index."""
    side = torch.cuda.Stream()
    g = torch.randn(10_000, device="cuda") * 1e-3
    p = torch.randn(10_000, device="cuda") * 0.02
    outs = [torch.zeros(10_000, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    states = []
    for k in range(2):
        st = zero.AdamWState([(10_000,)], 1, 0, LR, weight_decay=np.array([0.3]),
                             state_bits=state_bits, device="cuda")
        assert st.device == torch.device("cuda", 0)
        stream = side if k else None
        st.load_master([p], stream=stream)
        st.bind([[g]], [outs[k]], stream=stream)
        for t in (1, 2):
            st.step(t, sumsq=st.sumsq(stream=stream), max_norm=0.05, stream=stream)
        states.append(st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and outs[0].any()
    (a, b) = (x.get_state() for x in states)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for st in states:
        st.close()


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("world,rank", [(3, 1), (64, 2)])
def test_load_master_takes_this_ranks_rows(state_bits, dtype, world, rank):
    """From whole parameters of either dtype (and of a world past the replica
    limit), one element off alignment; the moments start at zero again."""
    shapes = [(130, 7), (5,), (64, 2), (2049,)]
    st = zero.AdamWState(shapes, world, rank, LR, state_bits=state_bits)
    p = [torch.randn(math.prod(s) + 1, device="cuda").to(dtype)[1:].view(s) for s in shapes]
    full = torch.randn(st.shard, device="cuda")
    keep = torch.zeros(st.shard, device="cuda")
    for k in range(4):
        keep[st.local[k][2]:st.local[k][2] + st.local_numel(k)] = 1
    st.set_state(full * keep, full * keep, (full * keep).square())
    st.load_master(p)
    master, m, v = st.get_state()
    for k, x in enumerate(p):
        first, rows, off = st.local[k]
        assert torch.equal(master[off:off + st.local_numel(k)], x[first:first + rows].float().view(-1))
    assert not m.any() and not v.any() and not master[keep == 0].any()
    st.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_two_states_at_once(state_bits):
    """Two contexts on two streams, their launches interleaved, against the
    same calls one after the other."""
    shapes = [(700_000,), (3, 1001)]
    jobs = [Job(shapes, 1, 0, 1, torch.bfloat16, torch.bfloat16, state_bits, 1, seed=k // 2)
            for k in range(4)]
    for j in jobs:
        j.fill()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sums = [torch.zeros(1, dtype=torch.float64, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for t in range(1, 21):
        for k, stream in enumerate(streams):              # jobs 0 and 2 at once
            jobs[2 * k].st.sumsq(out=sums[2 * k], stream=stream)
            jobs[2 * k].st.step(t, sumsq=sums[2 * k], max_norm=0.1, stream=stream)
    torch.cuda.synchronize()
    for k in (1, 3):                                      # 1 and 3 alone
        for t in range(1, 21):
            jobs[k].st.sumsq(out=sums[k])
            jobs[k].st.step(t, sumsq=sums[k], max_norm=0.1)
        torch.cuda.synchronize()
        assert sums[k].item() == sums[k - 1].item()
        assert all(np.array_equal(x, y) for x, y in zip(jobs[k].raw(), jobs[k - 1].raw()))
    for j in jobs:
        j.close()


def test_the_same_gradient_bound_twice():
    """One tensor as the gradient of two parameters, and as two replicas."""
    shapes = [(1000,), (1000,)]
    j = Job(shapes, 1, 0, 2, torch.float32, torch.float32, 32)
    g = torch.randn(1000, device="cuda") * 1e-3
    j.grads = [[g, g], [g, g]]
    j.st.bind(j.grads, j.outs)
    x = _f64(g)
    assert abs(j.st.sumsq().item() / (2 * math.fsum(x * x)) - 1) <= 2000 * 2.0 ** -52
    j.check_step(label="shared")
    j.close()


def test_whole_gradients_of_a_rank():
    """bind takes the whole parameter's gradient and finds its rows."""
    shapes = [(10, 7), (5,), (1, 3)]
    for rank in range(4):
        st = zero.AdamWState(shapes, 4, rank, LR)
        g = [torch.randn(s, device="cuda") for s in shapes]
        st.bind([g])
        want = sum(_f64(x[f:f + r]).ravel().dot(_f64(x[f:f + r]).ravel())
                   for x, (f, r, _) in zip(g, st.local))
        assert abs(st.sumsq().item() - want) <= 1e-12 * max(want, 1e-300)
        st.close()


def test_gpt2_small_rank():
    """GPT-2 small's 148 parameters, rank 3 of 8, clipped, both kinds."""
    import synth
    for state_bits in (32, 8):
        j = Job(synth.gpt2_small_shapes(), 8, 3, 2, torch.bfloat16, torch.bfloat16, state_bits, 1)
        j.fill()
        j.check_step(1.69, 0.5, "gpt2")
        log(f"gpt2 rank 3 of 8, {state_bits} bits: checked")
        j.close()


@pytest.mark.parametrize("state_bits", [8, 32])
def test_places_past_32_bits(state_bits):
    """4.3e9 elements (2^32 of them and more, up to 52 GB of state) in a
    tensor behind a small one: the last elements against the reference, the
    middle against zero."""
    n = (1 << 32) + 4099
    st = zero.AdamWState([(3,), (n,)], 1, 0, LR, BETAS, EPS, weight_decay=0.1,
                         state_bits=state_bits, seed=9)
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    out = torch.full((n + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    small = torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    st.bind([[small, g]], [small.clone(), out[:n]])
    tail = torch.randn(5000, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 1e-3
    g[-5000:] = tail.to(torch.bfloat16)
    x = _f64(g[-5000:])
    assert abs(st.sumsq().item() / math.fsum(x * x) - 1) <= 5000 * 2.0 ** -52
    st.step(1)
    torch.cuda.synchronize()
    off = st.local[1][2] + n - 5000
    got = _f64(st.state_tensors()["master"][off:off + 5000])
    sc = ref.scalars(LR, BETAS, EPS, 1)
    z = np.zeros(5000)
    step = ref.step32 if state_bits == 32 else ref.step8
    new, err = step(z, z, z, x, z, sc, 1.0, 0.1)
    assert np.all(np.abs(got - new[0]) <= err[0])
    assert torch.equal(out[n - 5000:n], st.state_tensors()["master"][off:off + 5000].bfloat16())
    assert out[n].item() == 7.0 and not out[:n - 5000].any()
    assert (out[:10] == 0).all() and (got != 0).sum() > 4900
    log(f"{n} elements, {state_bits} bits: checked")
    st.close()


# ------------------------------------------------------------------ refusals

def _einval(fn, *a, **kw):
    with pytest.raises(zero.ZeroError) as e:
        fn(*a, **kw)
    assert e.value.code == zero.ZERO_EINVAL, e.value


def test_refusals():
    st = zero.AdamWState([(8, 4), (3,)], 2, 0, LR)
    g = [torch.zeros(16, device="cuda"), torch.zeros(2, device="cuda")]
    o = [torch.zeros(16, device="cuda"), torch.zeros(2, device="cuda")]
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    _einval(st.sumsq)                                    # nothing bound
    _einval(st.step, 1)
    _einval(st.bind, [])                                 # no replica
    _einval(st.bind, [g] * 17)
    st.bind([g])
    _einval(st.step, 1)                                  # no outputs yet
    st.bind([g], o)
    _einval(st.bind, [g, g], o)                          # another count
    _einval(st.bind, [[x.bfloat16() for x in g]], o)     # another dtype
    _einval(st.bind, [g], [x.bfloat16() for x in o])
    _einval(st.bind, [g])                                # outputs gone
    _einval(st.step, 0)
    _einval(st.step_sched)                               # no schedule
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        _einval(st.step, 1, sumsq=s, max_norm=bad)
    for kw in (dict(weight_decay=-0.1), dict(weight_decay=float("nan")),
               dict(weight_decay=1e300), dict(lr_scale=float("inf")), dict(lr_scale=-1e300)):
        _einval(st.set_groups, **kw)
    with pytest.raises(ValueError):
        st.step(1, sumsq=s)                              # no max_norm
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda"),
                torch.zeros(1, dtype=torch.float64)):
        with pytest.raises(ValueError):
            st.step(1, sumsq=bad, max_norm=1.0)
        with pytest.raises(ValueError):
            st.sumsq(out=bad)
    for gl in ([g[0]], [g[0], None], [g[0][:15], g[1]], [torch.zeros(16), g[1]],
               [torch.zeros(32, device="cuda")[::2], g[1]]):
        with pytest.raises(ValueError):
            st.bind([gl], o)
    with pytest.raises(ValueError):
        st.bind([g], [torch.zeros(32, device="cuda"), o[1]])    # an output is this rank's rows
    with pytest.raises(TypeError):
        st.bind([[g[0], g[1].bfloat16()]], o)
    with pytest.raises(TypeError):
        st.bind([[x.half() for x in g]], o)
    for bad in ([0.1], [0.1] * 3):
        with pytest.raises(ValueError):
            st.set_groups(bad)
    with pytest.raises(ValueError):
        zero.AdamWState([(3,)], 1, 0, LR, seed=-1)
    # through the C ABI: null entries, misaligned and short buffers
    L, P = zero.lib(), ctypes.c_void_p
    big = torch.zeros(64, device="cuda")
    for ptrs in ([big.data_ptr(), 0], [big.data_ptr() + 2, big.data_ptr()]):
        arr = (P * 2)(*ptrs)
        assert L.zero_adamw_bind(st._h, arr, 1, 0, (P * 2)(*[x.data_ptr() for x in o]), 0,
                                 None) == zero.ZERO_EINVAL
        assert L.zero_adamw_bind(st._h, (P * 2)(*[x.data_ptr() for x in g]), 1, 0, arr, 0,
                                 None) == zero.ZERO_EINVAL
    assert L.zero_adamw_bind(st._h, None, 1, 0, None, 0, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_bind(st._h, (P * 2)(*[x.data_ptr() for x in g]), 1, 5, None, 0,
                             None) == zero.ZERO_EINVAL
    assert L.zero_adamw_sumsq(st._h, None, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_sumsq(st._h, s.data_ptr() + 4, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_step(st._h, 1, s.data_ptr() + 4, 1.0, None) == zero.ZERO_EINVAL
    st.step(1)                                           # and it still works
    st.close()
    # contexts of the other calls, and the other way round
    f = zero.FsdpShardState([(8, 4)], 2, 0, LR)
    assert L.zero_adamw_sumsq(f._h, s.data_ptr(), None) == zero.ZERO_EINVAL
    assert L.zero_adamw_step(f._h, 1, None, 1.0, None) == zero.ZERO_EINVAL
    assert L.zero_adamw_groups(f._h, None, None, None) == zero.ZERO_EINVAL
    f.close()
    q = zero.AdamWState([(8, 4)], 2, 0, LR, state_bits=8)
    whole = [torch.zeros(8, 4, device="cuda")]
    _einval(zero.FsdpShardState.step, q, [whole] * 2, 1, [torch.zeros(16, device="cuda")])
    _einval(zero.ShardState.step, q, [torch.zeros(q.shard, device="cuda")] * 2, 1,
            torch.zeros(q.shard, device="cuda"))
    q.close()


def test_a_buffer_past_its_allocation_is_refused():
    n = 1 << 20
    st = zero.AdamWState([(n,)], 1, 0, LR)
    L, P = zero.lib(), ctypes.c_void_p
    whole = torch.zeros(32 << 20, device="cuda")         # 128 MB, an allocation of its own
    fits, past = whole.data_ptr(), whole.data_ptr() + 4 * whole.numel() - 4096
    for g, o in ((past, fits), (fits, past)):
        assert L.zero_adamw_bind(st._h, (P * 1)(g), 1, 0, (P * 1)(o), 0, None) == zero.ZERO_EINVAL
    assert b"past the end" in L.zero_last_error()
    st.close()
