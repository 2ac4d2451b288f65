"""The gfx950 assembly of the vocabulary operators' kernels, compiled on the
CPU: no packed fp32 arithmetic, no scratch in a loop, matrix products fed by
loads to LDS."""
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
    zb.asm(str(out), ("vocab_kernels", "head_kernels"))
    found = []
    for name in ("vocab_kernels", "head_kernels"):
        asm = (out / (name + ".s")).read_text()
        for m in re.finditer(r"^(_Z\w+):", asm, re.M):
            end = asm.index(".Lfunc_end", m.end())
            found.append((m.group(1), asm[m.end():end], asm[end:end + 4000]))
    return found


def blocks(body):
    return re.split(r"^\.LBB\w+:", body, flags=re.M)


def test_no_packed_fp32(kernels):
    for name, body, _ in kernels:
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", body), name


def test_scratch_is_nowhere_but_in_epilogues(kernels):
    for name, body, tail in kernels:
        if "product_kernel" not in name:
            assert int(re.search(r"; ScratchSize: (\d+)", tail).group(1)) == 0, name
        for b in blocks(body):
            assert not ("v_mfma" in b and "scratch_" in b), name


def test_products_run_on_the_matrix_cores_from_lds(kernels):
    """Of every variant: the types' instruction, loads to LDS, transpose reads
    where a bf16 operand lies across the long axis, and no wait for the loads
    inside a stage but the one."""
    seen = 0
    for name, body, _ in kernels:
        m = re.search(r"product_kernelILb([01])ELi(\d)ELb([01])ELb([01])E", name)
        if not m:
            continue
        seen += 1
        bf16, across = m.group(1) == "1", "1" in m.group(3, 4)
        assert ("v_mfma_f32_16x16x32_bf16" if bf16 else "v_mfma_f32_16x16x4_f32") in body, name
        assert re.search(r"buffer_load_dwordx4 [^\n]* lds", body), name
        assert ("ds_read_b64_tr_b16" in body) == (bf16 and across), name
        deep = "ELi1ELi3EEEv" in name or "ELi1ELi4EEEv" in name       # three or four stages in LDS
        for b in blocks(body):
            if b.count("v_mfma") >= 16:
                assert len(re.findall(r"s_waitcnt vmcnt", b)) <= (3 if deep else 1), name
    # bf16: logits, grad_hidden, grad_table to bf16 and to fp32, in three tiles, and
    # logits in five more; fp32: the same in two
    assert seen == 4 * 3 + 5 + 4 * 2, seen
