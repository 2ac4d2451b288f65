"""AdamW over many tensors where the replicas of one gradient lie at different
places modulo an access's width, for every replica count, and what the sum of
squares promises about its bits."""
import math

import numpy as np
import pytest
import torch

import adamw_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero
from test_gpu_adamw import LR, Job, _f64, _gpu, _sum_bound  # noqa: F401 (_gpu: the fixture)

pytestmark = pytest.mark.gpu

# whole pieces of 2048 elements with and without a rest, and less than one
PIECES = [(5 * 2048 + 77,), (2048,), (3,), (2, 2048), (4097,), (513, 3)]


class ApartJob(Job):
    """A Job whose replica q lies `shifts[q]` elements further than the others'
    in its own buffer; what is between the gradients is NaN."""

    def __init__(self, shapes, n, shifts, gdt, odt, state_bits, gap=0, **kw):
        super().__init__(shapes, 1, 0, n, gdt, odt, state_bits, gap, outs=False, **kw)
        total = len(self.inside)
        self.gflat = [torch.zeros(total + s, dtype=gdt, device="cuda") for s in shifts]
        self.grads = [self._windows(f[s:]) for f, s in zip(self.gflat, shifts)]
        self.guards = []
        for s in shifts:
            out = np.ones(total + s, bool)
            out[s:] = ~self.inside
            self.guards.append(torch.from_numpy(out).cuda())
        self.st.bind(self.grads, self.outs)

    def fill(self, std=1e-3):
        super().fill(std)
        for f, out in zip(self.gflat, self.guards):
            f[out] = float("nan")

    def check_sum(self, label):
        reps = [np.concatenate([_f64(g) for g in gl]) for gl in self.grads]
        mean = sum(reps) / self.n
        mass = sum(np.abs(r) for r in reps) / self.n
        got = self.st.sumsq().item()
        assert (abs(got - math.fsum(mean * mean))
                <= _sum_bound(reps, mean.size) * math.fsum(mass * mass)), label


def _shifts(kind, n):
    return {"all": [q % 4 for q in range(n)],        # every phase
            "last": [0] * (n - 1) + [1],             # one replica off
            "first": [3] + [0] * (n - 1)}[kind]


@pytest.mark.parametrize("kind", ["all", "last", "first"])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [2, 3, 8, 9])
def test_replicas_at_different_places(n, gdt, kind):
    for state_bits in (32, 8):
        for gap in (0, 1):
            j = ApartJob(PIECES, n, _shifts(kind, n), gdt, torch.bfloat16, state_bits, gap,
                         seed=n + gap)
            for _ in range(2):
                j.fill()
                j.check_sum(f"{kind} N={n} gap {gap}")
                j.check_step(1.69, 0.5, f"{kind} N={n} gap {gap} {state_bits} bits")
            j.close()


@pytest.mark.parametrize("n", range(1, 17))
def test_every_replica_count(n):
    for state_bits, gdt in ((32, torch.bfloat16), (8, torch.float32)):
        j = ApartJob(PIECES, n, [0] * n, gdt, torch.float32, state_bits, 1, seed=n)
        for _ in range(2):
            j.fill()
            j.check_sum(f"N={n}")
            j.check_step(1.69, 0.5, f"N={n}")
        j.close()


# ------------------------------------------------------------ the sum's bits

@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 3])
def test_the_sums_bits_go_by_the_places_modulo_four_elements(n, gdt):
    """The same gradients in other buffers at the same places modulo four
    elements: the same bits, which a resumed run needs. At other places they
    are added in another order: the same number within the bound."""
    sizes = [3 * 2048 + 500, 2048, 40_004, 12]       # multiples of 4: one phase per list
    gen = torch.Generator(device="cuda").manual_seed(n)
    vals = [[(torch.randn(s, generator=gen, device="cuda") * 1e-3).to(gdt) for s in sizes]
            for _ in range(n)]
    reps = [np.concatenate([_f64(g) for g in gl]) for gl in vals]
    mean = sum(reps) / n
    mass = sum(np.abs(r) for r in reps) / n
    want, bound = math.fsum(mean * mean), _sum_bound(reps, mean.size) * math.fsum(mass * mass)

    def total(phases, further):
        st = zero.AdamWState([(s,) for s in sizes], 1, 0, LR)
        grads, keep = [], []
        for q, gl in enumerate(vals):
            at = [phases[q] + further + 4 * k + sum(sizes[:k]) for k in range(len(sizes))]
            flat = torch.full((at[-1] + sizes[-1] + 8,), float("nan"), dtype=gdt, device="cuda")
            keep.append(flat)
            grads.append([flat[a:a + s].copy_(g) for a, s, g in zip(at, sizes, gl)])
        st.bind(grads)
        got = [st.sumsq().item() for _ in range(3)]
        st.close()
        assert got[0] == got[1] == got[2]
        assert abs(got[0] - want) <= bound
        return got[0]

    for phase in range(4):
        assert len({total([phase] * n, d) for d in (0, 4, 8, 12)}) == 1, phase
    if n > 1:
        assert len({total([0, 1, 3], d) for d in (0, 4, 8)}) == 1
