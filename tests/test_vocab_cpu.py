"""The vocabulary operators on a machine without a GPU: what the library and
the binding refuse, workspace sizes, and the references the GPU tests use."""
import ctypes
import os
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import host_double
import vocab_reference as ref
import zero_partitioned_optimizer_flatten_amd as zero
from zero_partitioned_optimizer_flatten_amd import build as zb
from zero_partitioned_optimizer_flatten_amd import vocab

needs_gpp = pytest.mark.skipif(not host_double.available(), reason="g++ or the HIP headers missing")


# ------------------------------------------------------------ the generator

def test_philox_known_answers():
    """The two extreme vectors published with the generator."""
    one = np.array([0xFFFFFFFF], dtype=np.uint64)
    zero_ = np.array([0], dtype=np.uint64)
    got = [int(x[0]) for x in ref.philox([zero_] * 4, (0, 0))]
    assert got == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    got = [int(x[0]) for x in ref.philox([one] * 4, (0xFFFFFFFF, 0xFFFFFFFF))]
    assert got == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_reference_gradients_are_the_formulas():
    """The 64-bit references against automatic differentiation in 64 bits."""
    g = torch.Generator().manual_seed(1)
    h, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((9, 5), (7, 5)))
    y = torch.tensor([0, 6, 3, -100, 2, 2, 7, 1, 0])
    weights = torch.rand(9, generator=g)
    for mean in (False, True):
        a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
        on = (y >= 0) & (y < 7)
        part = weights.double() * on
        nll = -torch.log_softmax(a @ b.t(), 1).gather(1, torch.where(on, y, 0)[:, None])[:, 0]
        loss = (nll * part).sum() / (part.sum() if mean else 1.0)
        (3.0 * loss).backward()
        want = ref.head(h, w, y, weights, mean, 3.0)
        assert torch.allclose(want["loss"][0], loss.detach(), rtol=1e-13)
        assert torch.allclose(want["grad_hidden"][0], a.grad, rtol=1e-12, atol=1e-15)
        assert torch.allclose(want["grad_table"][0], b.grad, rtol=1e-12, atol=1e-15)
    t = torch.randn(7, 5, generator=g, dtype=torch.float64).requires_grad_()
    ids, up = torch.tensor([[0, 3, 3], [6, -1, 9]]), torch.randn(2, 3, 5, generator=g)
    x, _ = ref.embed(ids, t, 2.0, dropout=(0.4, 9, 1))
    x.backward(up.double())
    assert torch.allclose(ref.embed_grad(up, ids, 7, 2.0, (0.4, 9, 1))[0], t.grad, rtol=1e-12, atol=1e-15)


# ------------------------------------------------- the library's host side

@pytest.fixture(scope="module")
def L(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("vocab"))
    so = os.path.join(out, "libvocab_host.so")
    tests = host_double.TESTS
    subprocess.check_call(["g++", *host_double.FLAGS, "-x", "c++", os.path.join(zb.CSRC, "zero_api.hip"),
                           os.path.join(zb.CSRC, "vocab_api.hip"), os.path.join(tests, "host_double.cpp"),
                           os.path.join(tests, "vocab_double.cpp"), "-o", so])
    lib = host_double.load(so)
    was = zero._lib, vocab._declared
    zero._lib, vocab._declared = lib, None
    try:
        vocab._lib()
    finally:
        zero._lib, vocab._declared = was
    lib.double_drop_limit.restype = ctypes.c_uint32
    lib.double_drop_scale.restype = ctypes.c_float
    lib.double_head_bytes.restype = lib.double_head_pieces.restype = ctypes.c_int64
    return lib


def malloc(L, nbytes):
    p = ctypes.c_void_p()
    assert L.hipMalloc(ctypes.byref(p), max(1, nbytes)) == 0
    return p.value


def refused(L, code, call, *text):
    before = L.double_vocab_launches()
    assert call() == code, L.zero_last_error()
    assert L.double_vocab_launches() == before
    said = L.zero_last_error().decode()
    for t in text:
        assert t in said, said


def changed(args, **kw):
    return list({**args, **kw}.values())


INVALID, UNSUPPORTED = zero.ZERO_EINVAL, zero.ZERO_EUNSUPPORTED


@needs_gpp
def test_embed_refuses(L):
    n, rows, width = 6, 10, 8
    args = dict(ids=malloc(L, 8 * n), id_bytes=8, count=n, table=malloc(L, 2 * rows * width), rows=rows, width=width, dtype=1,
                scale=1.0, pos=None, ptable=None, prows=0, drop=None, out=malloc(L, 2 * n * width), odt=1, stream=None)
    call = lambda **kw: (lambda: L.zero_embed(*changed(args, **kw)))  # noqa: E731
    assert call()() == zero.ZERO_OK
    for kw, text in [(dict(ids=None), "ids is null"), (dict(table=None), "table is null"), (dict(out=None), "out is null"),
                     (dict(id_bytes=2), "4 or 8"), (dict(dtype=7), "dtype"), (dict(odt=-1), "dtype"), (dict(count=-1), "count"),
                     (dict(rows=0), "rows"), (dict(width=0), "rows and columns"), (dict(scale=float("nan")), "finite"),
                     (dict(scale=1e39), "finite"), (dict(table=args["table"] + 1), "aligned"), (dict(ids=args["ids"] + 4), "aligned"),
                     (dict(rows=1000), "run past"), (dict(count=1000), "run past"), (dict(out=args["table"]), "overlap"),
                     (dict(pos=args["ids"]), "together"), (dict(ptable=args["table"]), "together"),
                     (dict(pos=args["ids"], ptable=args["table"], prows=0), "rows"),
                     (dict(pos=args["ids"], ptable=args["table"], prows=11), "run past")]:
        refused(L, INVALID, call(**kw), text)
    refused(L, UNSUPPORTED, call(count=2 ** 31), "more than one call")
    refused(L, UNSUPPORTED, call(count=2 ** 30, width=2 ** 10), "more than one call")
    refused(L, UNSUPPORTED, call(rows=2 ** 30 + 1), "2^30")
    assert call(count=0, ids=None, out=None)() == zero.ZERO_OK
    assert call(pos=args["ids"], ptable=args["table"], prows=10)() == zero.ZERO_OK


@needs_gpp
@pytest.mark.parametrize("p,limit", [(0.0, 0), (1e-9, 0), (2.0 ** -17, 1), (0.1, 6554), (0.5, 32768), (0.99999, 65535), (1.0, 65536)])
def test_dropout_limit_and_scale(L, p, limit):
    x = malloc(L, 400)
    d = vocab._Drop(p, 1, 2, None)
    assert L.zero_dropout(x, None, x, 100, 0, ctypes.byref(d), None) == zero.ZERO_OK
    assert L.double_drop_limit() == limit
    want = np.float32(65536.0 / (65536 - limit)) if limit < 65536 else np.float32(0)
    assert L.double_drop_scale() == want


@needs_gpp
def test_dropout_refuses(L):
    x, y = malloc(L, 400), malloc(L, 400)
    good = vocab._Drop(0.5, 1, 2, None)
    args = dict(x=x, add=None, out=y, count=100, dtype=0, drop=ctypes.byref(good), stream=None)
    call = lambda **kw: (lambda: L.zero_dropout(*changed(args, **kw)))  # noqa: E731
    assert call()() == call(out=x)() == call(add=y)() == zero.ZERO_OK
    for kw, text in [(dict(x=None), "null"), (dict(out=None), "null"), (dict(drop=None), "null"), (dict(count=-1), "count"),
                     (dict(count=101), "run past"), (dict(dtype=2), "dtype"), (dict(x=x + 2), "aligned"),
                     (dict(out=x + 4, count=90), "overlap"), (dict(add=y + 4, count=90), "overlap")]:
        refused(L, INVALID, call(**kw), text)
    for p in (-0.1, 1.1, float("nan")):
        refused(L, INVALID, call(drop=ctypes.byref(vocab._Drop(p, 1, 2, None))), "p must")
    refused(L, INVALID, call(drop=ctypes.byref(vocab._Drop(0.5, 1, 2, x + 4))), "counter")
    refused(L, UNSUPPORTED, call(count=2 ** 36), "more than one call")


def size_of(L, f, *args):
    n = ctypes.c_int64()
    assert f(*args, ctypes.byref(n)) == zero.ZERO_OK, L.zero_last_error()
    return n.value


@needs_gpp
def test_embed_grad_refuses(L):
    n, rows, width = 6, 10, 8
    need = size_of(L, L.zero_embed_grad_workspace, n, rows, width)
    args = dict(g=malloc(L, 2 * n * width), gdt=1, ids=malloc(L, 4 * n), id_bytes=4, count=n, rows=rows, width=width, scale=1.0,
                drop=None, t=malloc(L, 4 * rows * width + 4096), tdt=0, acc=0, ws=malloc(L, need), bytes=need, stream=None)
    call = lambda **kw: (lambda: L.zero_embed_grad(*changed(args, **kw)))  # noqa: E731
    assert call()() == call(acc=1)() == zero.ZERO_OK
    for kw, text in [(dict(g=None), "grad_out is null"), (dict(t=None), "grad_table is null"), (dict(ids=None), "null"),
                     (dict(ws=None), "workspace is null"), (dict(bytes=need - 1), "needs"), (dict(ws=args["ws"] + 16), "aligned"),
                     (dict(id_bytes=1), "4 or 8"), (dict(gdt=3), "dtype"), (dict(tdt=3), "dtype"), (dict(rows=1000), "run past"),
                     (dict(g=args["t"], gdt=0), "overlap"), (dict(ws=args["t"]), "overlap"), (dict(count=-2), "count")]:
        refused(L, INVALID, call(**kw), text)
    refused(L, UNSUPPORTED, call(rows=2 ** 30 + 1), "2^30")
    n64 = ctypes.c_int64()
    assert L.zero_embed_grad_workspace(n, rows, width, None) == INVALID
    assert L.zero_embed_grad_workspace(-1, rows, width, ctypes.byref(n64)) == INVALID


HEAD = dict(count=20, vocab=50, width=16)


def head_args(L, dtype=1, tdt=1, piece=0, **sizes):
    s = {**HEAD, **sizes}
    n, v, w = s["count"], s["vocab"], s["width"]
    es, gs = (2 if dtype else 4), (2 if tdt else 4)
    need = size_of(L, L.zero_head_loss_workspace, n, v, w, dtype, 1, 1, tdt, piece)
    return dict(h=malloc(L, es * n * w), t=malloc(L, es * v * w), dtype=dtype, y=malloc(L, 8 * n), id_bytes=8, count=n, vocab=v,
                width=w, weights=malloc(L, 4 * n), mean=1, scale=1.0, loss=malloc(L, 4), losses=malloc(L, 4 * n),
                gh=malloc(L, es * n * w), gt=malloc(L, gs * v * w), tdt=tdt, acc=0, piece=piece, ws=malloc(L, need), bytes=need,
                stream=None), need


@needs_gpp
def test_head_loss_refuses(L):
    args, need = head_args(L)
    call = lambda **kw: (lambda: L.zero_head_loss(*changed(args, **kw)))  # noqa: E731
    assert call()() == call(weights=None, losses=None, gh=None, gt=None)() == call(acc=1, mean=0)() == zero.ZERO_OK
    for kw, text in [(dict(h=None), "hidden"), (dict(t=None), "table"), (dict(y=None), "targets"), (dict(loss=None), "loss"),
                     (dict(ws=None), "workspace"), (dict(ws=args["ws"] + 128), "aligned"), (dict(bytes=16), "needs"),
                     (dict(id_bytes=16), "4 or 8"), (dict(dtype=9), "dtype"), (dict(tdt=9), "dtype"), (dict(count=-1), "count"),
                     (dict(vocab=0), "rows"), (dict(width=0), "columns"), (dict(piece=-1), "piece_rows"),
                     (dict(scale=float("inf")), "grad_scale"), (dict(h=args["h"] + 1), "aligned"), (dict(gt=args["gt"] + 1), "aligned"),
                     (dict(gh=args["h"]), "overlap"), (dict(gt=args["t"]), "overlap"), (dict(losses=args["weights"]), "overlap"),
                     (dict(loss=args["losses"]), "overlap"), (dict(gh=args["ws"]), "")]:
        refused(L, INVALID, call(**kw), text)
    refused(L, UNSUPPORTED, call(vocab=2 ** 21), "4 MiB")
    refused(L, UNSUPPORTED, call(width=2 ** 21), "4 MiB")
    refused(L, UNSUPPORTED, call(count=2 ** 31), "more than one call")
    refused(L, UNSUPPORTED, call(count=2 ** 30, vocab=1000000, piece=2 ** 20), "64 GiB")
    n64 = ctypes.c_int64()
    assert L.zero_head_loss_workspace(20, 50, 16, 1, 1, 1, 1, 0, None) == INVALID
    assert L.zero_head_loss_workspace(20, 50, 16, 1, 1, 1, 5, 0, ctypes.byref(n64)) == INVALID
    assert L.zero_head_loss_workspace(2 ** 30, 50, 16, 1, 1, 1, 1, 2 ** 21, ctypes.byref(n64)) == UNSUPPORTED


@needs_gpp
def test_head_loss_workspace_covers_every_alignment(L):
    """What the size call gives is enough whatever the table's alignment, and
    grows with no more than one piece."""
    for dtype in (0, 1):
        for tdt in (0, 1):
            for sizes in (dict(count=1), dict(count=300, vocab=1000, width=64), dict(count=77, vocab=129, width=33), dict(count=0)):
                for piece in (0, 1, 50):
                    args, need = head_args(L, dtype, tdt, piece, **sizes)
                    for kw in (dict(), dict(gh=None), dict(gt=None), dict(losses=None)):
                        assert L.zero_head_loss(*changed(args, **kw)) == zero.ZERO_OK, L.zero_last_error()
                        assert L.double_head_bytes() <= need
    ask = lambda n: size_of(L, L.zero_head_loss_workspace, n, 128256, 4096, 1, 1, 1, 1, 0)  # noqa: E731
    assert ask(1 << 20) - ask(1 << 14) < (1 << 20) * 64


@needs_gpp
def test_parts_of_a_tile_are_never_empty(L):
    """Cut into about k, every part has a stage and the last one ends with the tile."""
    per = ctypes.c_int()
    for steps in [*range(1, 700), 1001, 1875, 4008, 65536]:
        for k in range(1, 65):
            parts = L.double_head_parts(steps, k, ctypes.byref(per))
            assert 1 <= parts <= k
            assert (parts - 1) * per.value < steps <= parts * per.value, (steps, k)


# -------------------------------------------------------------- the binding

class _Tensor(SimpleNamespace):
    """As much of a device tensor as the checks ask for."""

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096

    def numel(self):
        return int(np.prod(self.shape)) if self.shape else 1

    def get_device(self):
        return self.device.index if self.device.type == "cuda" else -1

    def new_empty(self, shape, dtype=None):
        return tensor((shape,) if isinstance(shape, int) else shape, dtype or self.dtype)

    def record_stream(self, s):
        self.used_on.append(s.cuda_stream)


def tensor(shape, dtype=torch.float32, device="cuda:0", contiguous=True):
    return _Tensor(shape=torch.Size(shape), dtype=dtype, device=torch.device(device), contiguous=contiguous, used_on=[])


@pytest.fixture
def binding(monkeypatch):
    called = []

    def size(*a):
        a[-1]._obj.value = 512
        return 0

    def took(name):
        return lambda *a: called.append(name) or 0

    fake = SimpleNamespace(zero_embed=took("embed"), zero_embed_grad=took("embed_grad"), zero_dropout=took("dropout"),
                           zero_head_loss=took("head_loss"), zero_embed_grad_workspace=size, zero_head_loss_workspace=size)
    monkeypatch.setattr(vocab, "_lib", lambda: fake)
    monkeypatch.setattr(vocab, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(vocab, "_current_device", lambda: 0)
    monkeypatch.setattr(vocab.torch, "empty_like", lambda x: tensor(x.shape, x.dtype))
    return called


I64, BF = torch.int64, torch.bfloat16


@pytest.mark.parametrize("error,call", [
    (ValueError, lambda: zero.embed(tensor((3,), I64, "cpu"), tensor((5, 4)))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4), device="cpu"))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4), device="cuda:1"))),
    (TypeError, lambda: zero.embed(tensor((3,), torch.int16), tensor((5, 4)))),
    (TypeError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4), torch.float16))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5,)))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4), contiguous=False))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), out=tensor((3, 5)))),
    (TypeError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), out=tensor((3, 4)), dtype=BF)),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), positions=tensor((3,), I64))),
    (TypeError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), positions=tensor((3,), torch.int32), position_table=tensor((2, 4)))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), positions=tensor((4,), I64), position_table=tensor((2, 4)))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), positions=tensor((3,), I64), position_table=tensor((2, 3)))),
    (TypeError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), positions=tensor((3,), I64), position_table=tensor((2, 4), BF))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), dropout=zero.Dropout(0.1, -1))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), dropout=zero.Dropout(0.1, 1, 1 << 64))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), dropout=zero.Dropout(0.1, 1, 0, tensor((2,), I64)))),
    (ValueError, lambda: zero.embed(tensor((3,), I64), tensor((5, 4)), dropout=zero.Dropout(0.1, 1, 0, tensor((1,), I64, "cpu")))),
    (ValueError, lambda: zero.embed_grad(tensor((3, 5)), tensor((3,), I64), tensor((5, 4)))),
    (ValueError, lambda: zero.embed_grad(tensor((3, 4)), tensor((3,), I64), tensor((5, 4), contiguous=False))),
    (TypeError, lambda: zero.embed_grad(tensor((3, 4)), tensor((3,), I64), tensor((5, 4), torch.float64))),
    (ValueError, lambda: zero.dropout(tensor((3, 4), device="cpu"), zero.Dropout(0.1, 1))),
    (ValueError, lambda: zero.dropout(tensor((3, 4)), zero.Dropout(0.1, 1), add=tensor((4, 3)), out=tensor((3, 4)))),
    (TypeError, lambda: zero.dropout(tensor((3, 4)), zero.Dropout(0.1, 1), out=tensor((3, 4), BF))),
    (ValueError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((3,), I64), reduction="none")),
    (ValueError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((4,), I64))),
    (ValueError, lambda: zero.head_loss(tensor((3, 3)), tensor((5, 4)), tensor((3,), I64))),
    (TypeError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4), BF), tensor((3,), I64))),
    (TypeError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((3,), I64), weights=tensor((3,), BF))),
    (ValueError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((3,), I64), losses=tensor((4,)))),
    (TypeError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((3,), I64), grad_hidden=tensor((3, 4), BF))),
    (ValueError, lambda: zero.head_loss(tensor((3, 4)), tensor((5, 4)), tensor((3,), I64), grad_table=tensor((4, 4)))),
])
def test_binding_refuses(binding, error, call):
    with pytest.raises(error):
        call()
    assert not binding


def test_dropout_is_fixed_and_says_what_it_is():
    d = zero.Dropout(0.25, 7, 9)
    assert (d.p, d.seed, d.offset, d.counter) == (0.25, 7, 9, None) and "0.25" in repr(d)
    with pytest.raises(AttributeError):
        d.p = 0.5


def test_signatures_are_the_users():
    import inspect
    for f in (zero.embed, zero.embed_grad, zero.dropout, zero.head_loss):
        names = list(inspect.signature(f).parameters)
        assert "call" not in names and names[-1] == "stream" and f.__doc__
    assert list(inspect.signature(zero.embed).parameters)[:2] == ["tokens", "table"]


def test_binding_passes_on(binding):
    zero.embed(tensor((2, 3), I64), tensor((5, 4)))
    zero.embed_grad(tensor((2, 3, 4)), tensor((2, 3), I64), tensor((5, 4), BF))
    zero.dropout(tensor((3, 4)), zero.Dropout(0.1, 1), out=tensor((3, 4)))
    zero.head_loss(tensor((2, 3, 4)), tensor((5, 4)), tensor((2, 3), I64))
    assert binding == ["embed", "embed_grad", "dropout", "head_loss"]


def test_binding_takes_every_argument_by_name(binding):
    zero.embed(table=tensor((5, 4)), tokens=tensor((2, 3), I64))
    zero.embed_grad(tokens=tensor((2, 3), I64), grad_table=tensor((5, 4)), grad_out=tensor((2, 3, 4)))
    zero.dropout(drop=zero.Dropout(0.1, 1), x=tensor((3, 4)))
    zero.head_loss(targets=tensor((2, 3), I64), hidden=tensor((2, 3, 4)), table=tensor((5, 4)))
    assert binding == ["embed", "embed_grad", "dropout", "head_loss"]
    with pytest.raises(TypeError, match="needs tokens"):
        zero.embed(table=tensor((5, 4)))
