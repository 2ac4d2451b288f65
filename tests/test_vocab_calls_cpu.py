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
from zero_partitioned_optimizer_flatten_amd import vocab


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


@needs_gpp
def test_outputs_over_the_dropout_counter_are_refused(L):  # noqa: F811
    """Every workgroup reads it, at no certain time."""
    n, rows, width = 6, 10, 8
    ids, table, x = malloc(L, 8 * n), malloc(L, 4 * rows * width), malloc(L, 4 * n * width)
    need = size_of(L, L.zero_embed_grad_workspace, n, rows, width)
    out, ws, apart = malloc(L, 4 * rows * width), malloc(L, need), malloc(L, 8)
    drop = lambda at: ctypes.byref(vocab._Drop(0.5, 1, 2, at))  # noqa: E731
    calls = {
        out: [lambda d: L.zero_embed(ids, 8, n, table, rows, width, 0, 1.0, None, None, 0, d, out, 0, None),
              lambda d: L.zero_dropout(x, None, out, n * width, 0, d, None),
              lambda d: L.zero_embed_grad(x, 0, ids, 8, n, rows, width, 1.0, d, out, 0, 0, ws, need, None)],
        ws: [lambda d: L.zero_embed_grad(x, 0, ids, 8, n, rows, width, 1.0, d, out, 0, 0, ws, need, None)]}
    for at, of in calls.items():
        for call in of:
            assert call(drop(apart)) == zero.ZERO_OK, L.zero_last_error()
            refused(L, INVALID, lambda: call(drop(at)), "overlap")
            refused(L, INVALID, lambda: call(drop(at + 8 * (n - 1))), "overlap")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = os.path.join(str(tmp_path_factory.mktemp("rules")), "librules.so")
    subprocess.check_call(["g++", *host_double.FLAGS, "-x", "c++", *[os.path.join(zb.CSRC, n) for n in ("zero_api.hip", "vocab_api.hip")],
                           *[os.path.join(host_double.TESTS, n) for n in ("host_double.cpp", "vocab_double.cpp", "vocab_rules.cpp")],
                           "-o", so])
    lib = ctypes.CDLL(so)
    lib.rules_turned_with_loss.restype = lib.rules_sort_groups.restype = ctypes.c_int64
    lib.rules_sort_groups.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
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


@needs_gpp
def test_sort_groups_are_no_more_than_the_ids_need(rules):
    ids = ctypes.c_int()
    for rows in (1, 255, 256, 257, 50257, 131071, 131072, 131073, 262144, 262145, 1 << 20, (1 << 30) - 1, 1 << 30):
        groups = rules.rules_sort_groups(1000, rows, ctypes.byref(ids))
        assert ids.value <= 512 and ids.value * groups >= rows
        assert groups == 256 or groups // 2 * 512 < rows, (rows, groups)


@needs_gpp
@pytest.mark.parametrize("rows,most", [(1 << 30, 1 << 21), (1 << 26, 1 << 25), ((1 << 22) + 1, 1 << 28), (1 << 20, (1 << 31) - 1)])
def test_sort_that_takes_the_device_for_long_is_refused(L, rows, most):  # noqa: F811
    """2^42 ids read, by rows / 512 workgroups; ordinary tables take any number."""
    n = ctypes.c_int64()
    size = L.zero_embed_grad_workspace
    assert size(most, rows, 1, ctypes.byref(n)) == zero.ZERO_OK, L.zero_last_error()
    if most < (1 << 31) - 1:
        assert size(most + 1, rows, 1, ctypes.byref(n)) == UNSUPPORTED
        p = malloc(L, 4096)
        refused(L, UNSUPPORTED, lambda: L.zero_embed_grad(p, 0, p, 8, most + 1, rows, 1, 1.0, None, p, 0, 1, p, 1 << 50, None),
                "more than one call")
