"""Calls of the vocabulary operators that the documentation allows, or that are
refused, at the ends of their ranges, against the host code built with g++."""
from test_vocab_cpu import INVALID, L, UNSUPPORTED, changed, malloc, needs_gpp, refused, size_of  # noqa: F401
import zero_partitioned_optimizer_flatten_amd as zero


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
