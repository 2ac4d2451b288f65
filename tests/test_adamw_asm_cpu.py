"""The gfx950 assembly of the many-tensor AdamW kernels, compiled on the CPU:
no packed fp32 arithmetic, no scratch, no loop over the descriptors of a wave
(all are uniform), and streaming loads and stores of the state."""
import os
import re
import shutil

import pytest

from zero_partitioned_optimizer_flatten_amd import build as zb


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not (os.path.exists(zb.HIPCC) or shutil.which(zb.HIPCC)):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm")
    zb.asm(str(out))
    asm = (out / "adamw_kernels.s").read_text()
    found = []
    for m in re.finditer(r"^(_Z\w+):", asm, re.M):
        end = asm.index(".Lfunc_end", m.end())
        found.append((m.group(1), asm[m.end():end], asm[end:end + 4000]))
    return found


def test_every_variant_is_there(kernels):
    """Replica counts 1, 2, 4, 8 and any other, both gradient and both output
    dtypes, both states; the sum for 1-4, 8 and any other."""
    names = [n for n, _, _ in kernels]
    assert sum("adamw32_kernel" in n for n in names) == 20
    assert sum("adamw8_kernel" in n for n in names) == 20
    assert sum("sumsq_kernel" in n for n in names) == 12


def test_no_packed_fp32_and_no_scratch(kernels):
    for name, body, tail in kernels:
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", body), name
        assert int(re.search(r"; ScratchSize: (\d+)", tail).group(1)) == 0, name


def test_no_loops_over_descriptors(kernels):
    """Such a loop reads a descriptor lane by lane with readfirstlane and
    compares; the only readfirstlane here is the wave's index."""
    for name, body, _ in kernels:
        if "adamw32_kernel" in name:
            assert "v_readfirstlane" not in body, name
        if "adamw8_kernel" in name:
            assert body.count("v_readfirstlane") <= 1, name


def test_state_streams(kernels):
    """Every buffer access carries the streaming hint, and stores come plain
    and at device scope."""
    for name, body, _ in kernels:
        if "adamw32_kernel" in name or "adamw8_kernel" in name:
            lines = re.findall(r"buffer_(?:load|store)_dword\w* [^\n]*", body)
            assert lines and all(re.search(r"\bnt\b", x) for x in lines), name
            stores = [x for x in lines if x.startswith("buffer_store")]
            assert 2 * sum("sc1" in x for x in stores) == len(stores), name


def test_partial_sums_are_handed_over_at_device_scope(kernels):
    """The order of a workgroup's partial sum before its count rests on these
    instructions: the partial stored at device scope, waited for, then
    counted; the partials loaded at device scope by the one that joins them."""
    for name, body, _ in kernels:
        if "sumsq_kernel" not in name:
            continue
        lines = [x.strip() for x in body.splitlines()]
        count = next(i for i, x in enumerate(lines) if x.startswith("global_atomic_add"))
        stores = [i for i, x in enumerate(lines[:count]) if x.startswith("global_store")]
        assert len(stores) == 1 and "global_store_dwordx2" in lines[stores[0]], name
        assert re.search(r"\bsc1\b", lines[stores[0]]), name
        assert "s_waitcnt vmcnt(0)" in lines[stores[0]:count], name
        loads = [x for x in lines[count:] if x.startswith("global_load")]
        assert len(loads) >= 2 and all(re.search(r"\bsc1\b", x) for x in loads), name
