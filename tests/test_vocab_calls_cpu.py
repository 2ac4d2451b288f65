"""Calls of the vocabulary operators that the documentation allows, or that are
refused, at the ends of their ranges, against the host code built with g++."""
import ctypes
import os
import subprocess

import pytest

import host_double
from test_vocab_cpu import INVALID, L, UNSUPPORTED, changed, head_args, malloc, needs_gpp, refused, size_of  # noqa: F401
import zero_partitioned_optimizer_flatten_amd as zero
from zero_partitioned_optimizer_flatten_amd import build as zb


@needs_gpp
def test_no_rows_have_no_position_ids(L):  # noqa: F811
    """An empty tensor of ids has no address; its table is checked all the same."""
    rows, width = 10, 8
    table = malloc(L, 2 * rows * width)
    args = dict(ids=None, id_bytes=8, count=0, table=table, rows=rows, width=width, dtype=1, scale=1.0, pos=None,
                ptable=table, prows=rows, drop=None, out=None, odt=1, stream=None)
    call = lambda **kw: (lambda: L.zero_embed(*changed(args, **kw)))  # noqa: E731
    assert call()() == zero.ZERO_OK, L.zero_last_error()
    refused(L, INVALID, call(prows=0), "rows")
    refused(L, INVALID, call(prows=11), "run past")
    refused(L, INVALID, call(pos=table, ptable=None), "together")
    refused(L, INVALID, call(count=1, ids=table, out=malloc(L, 2 * width)), "together")


@needs_gpp
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("piece", [0, 50])
def test_workspace_is_enough_for_a_table_off_16_bytes(L, dtype, piece):  # noqa: F811
    """Such a table is copied, also where its rows are whole stages; the size call
    does not see its address and has to count the copy."""
    vocab, width, es = 1000, 64, 2 if dtype else 4
    args, need = head_args(L, dtype, dtype, piece, count=300, vocab=vocab, width=width)
    t = malloc(L, es * (vocab * width + 1))
    assert t % 16 == 0
    used = {}
    for off in (0, es):
        assert L.zero_head_loss(*changed(args, t=t + off)) == zero.ZERO_OK, L.zero_last_error()
        used[off] = L.double_head_bytes()
        assert used[off] <= need
    assert used[es] == used[0] + es * vocab * width
    # with the losses' place in it too, it is what the size call says
    refused(L, INVALID, lambda: L.zero_head_loss(*changed(args, t=t + es, losses=None, bytes=need - 1)), "needs")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = os.path.join(str(tmp_path_factory.mktemp("rules")), "librules.so")
    subprocess.check_call(["g++", *host_double.FLAGS, "-x", "c++", *[os.path.join(zb.CSRC, n) for n in ("zero_api.hip", "vocab_api.hip")],
                           *[os.path.join(host_double.TESTS, n) for n in ("host_double.cpp", "vocab_double.cpp", "vocab_rules.cpp")],
                           "-o", so])
    lib = ctypes.CDLL(so)
    lib.rules_turned_with_loss.restype = ctypes.c_int64
    lib.rules_turned_with_loss.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_int64]
    return lib


@needs_gpp
def test_one_workgroup_turns_few_numbers(rules):
    """Zeros behind the rows count: a thread of the 1024 goes through six vectors of
    16 bytes at most, and a call too large for that has a kernel for it."""
    done = 0
    for bf16 in (0, 1):
        for count in (1, 2, 4, 8, 16, 31, 32, 63, 64, 65, 128, 200, 1000):
            for vocab in (1, 100, 128, 129, 256, 500, 1000, 4000, 8192, 16000, 16384, 50257):
                turned = rules.rules_turned_with_loss(count, vocab, 64, bf16, 0)
                assert turned <= 6 * 1024 * (8 if bf16 else 4), (bf16, count, vocab, turned)
                assert turned == 0 or turned == -(-count // 64) * 64 * (-(-vocab // 128) * 128)
                assert rules.rules_turned_with_loss(count, vocab, 64, bf16, 1) == (turned if count == 1 else 0)
                done += turned > 0
    assert done >= 20, done
