"""MI355X (gfx950) ZeRO-2 shard step: Python binding of libzero.so.

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch supplies device memory (tensor storage) and streams; the
binding checks tensor device/dtype/size so that a mistake becomes a Python
error instead of an out-of-bounds GPU access, then calls the C ABI declared
in include/zero.h with raw pointers.

There is no CPU fallback: if libzero.so is missing or cannot be loaded, the
first call raises ZeroError.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "zero.h")

ZERO_F32, ZERO_BF16 = 0, 1
ZERO_OK, ZERO_EINVAL, ZERO_ENOMEM, ZERO_EHIP, ZERO_EUNSUPPORTED = 0, -1, -2, -3, -4
MAX_WORLD = 256

_CODES = {ZERO_EINVAL: "EINVAL", ZERO_ENOMEM: "ENOMEM", ZERO_EHIP: "EHIP",
          ZERO_EUNSUPPORTED: "EUNSUPPORTED"}


class ZeroError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"zero [{_CODES.get(code, code)}]: {msg}")
        self.code = code
        self.msg = msg


_lib = None


def lib():
    """Load libzero.so (built in-tree by build.py) and declare signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ZeroError(ZERO_EUNSUPPORTED,
                        f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                        "python -m zero_partitioned_optimizer_flatten_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, vp, dbl = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_double
    p64 = ctypes.POINTER(ctypes.c_int64)
    L.zero_last_error.restype = ctypes.c_char_p
    L.zero_shard_geometry.argtypes = [i64, i32, i32, p64, p64, p64]
    L.zero_shard_init.argtypes = [i64, i32, i32, dbl, dbl, dbl, dbl, ctypes.POINTER(vp)]
    L.zero_shard_info.argtypes = [vp, p64, p64, p64]
    L.zero_shard_state_bytes.argtypes = [vp, p64]
    L.zero_set_lr.argtypes = [vp, dbl]
    L.zero_load_master.argtypes = [vp, vp, ctypes.c_int, i64, vp]
    L.zero_flatten.argtypes = [vp, vp, vp, i32, ctypes.c_int, vp, vp]
    L.zero_unflatten.argtypes = [vp, vp, i32, vp, ctypes.c_int, vp, vp]
    L.zero_flatten_range.argtypes = [vp, vp, vp, i32, ctypes.c_int, vp, i64, i64, vp]
    L.zero_step.argtypes = [vp, vp, i32, ctypes.c_int, i64, vp, ctypes.c_int, i64, i64, vp]
    L.zero_step_range.argtypes = [vp, i64, i64, vp, i32, ctypes.c_int, i64, vp, ctypes.c_int,
                                  i64, i64, vp]
    L.zero_dim0_split.argtypes = [i64, i32, i32, p64, p64]
    L.zero_fsdp_init.argtypes = [i32, vp, vp, i32, i32, dbl, dbl, dbl, dbl, ctypes.POINTER(vp)]
    L.zero_fsdp_local.argtypes = [vp, i32, p64, p64, p64]
    L.zero_fsdp_load_master.argtypes = [vp, vp, ctypes.c_int, vp]
    L.zero_fsdp_step.argtypes = [vp, vp, i32, ctypes.c_int, vp, ctypes.c_int, i64, vp]
    L.zero_set_step_workgroups.argtypes = [vp, i32]
    L.zero_schedule_init.argtypes = [vp, i64, vp]
    L.zero_schedule_init_noalloc.argtypes = [vp, i64, vp]
    L.zero_schedule_lr.argtypes = [vp, dbl, vp]
    L.zero_schedule_get.argtypes = [vp, p64, vp]
    L.zero_step_begin.argtypes = [vp, vp]
    L.zero_step_sched.argtypes = [vp, vp, i32, ctypes.c_int, i64, vp, ctypes.c_int, i64, vp]
    L.zero_step_range_sched.argtypes = [vp, i64, i64, vp, i32, ctypes.c_int, i64, vp,
                                        ctypes.c_int, i64, vp]
    L.zero_fsdp_step_sched.argtypes = [vp, vp, i32, ctypes.c_int, vp, ctypes.c_int, vp]
    u32, pvp = ctypes.c_uint32, ctypes.POINTER(vp)
    L.zero_adamw_init.argtypes = [i32, vp, vp, i32, i32, dbl, dbl, dbl, dbl, i32, u32, pvp]
    L.zero_adamw_groups.argtypes = [vp, vp, vp, vp]
    L.zero_adamw_bind.argtypes = [vp, vp, i32, ctypes.c_int, vp, ctypes.c_int, vp]
    L.zero_adamw_sumsq.argtypes = [vp, vp, vp]
    L.zero_adamw_step.argtypes = [vp, i64, vp, dbl, vp]
    L.zero_adamw_step_sched.argtypes = [vp, vp, dbl, vp]
    L.zero_adamw_state.argtypes = [vp, pvp, pvp, pvp, pvp]
    L.zero_get_state.argtypes = [vp, vp, vp, vp, vp]
    L.zero_set_state.argtypes = [vp, vp, vp, vp, vp]
    L.zero_state_bytes.argtypes = [i32, dbl, dbl, ctypes.POINTER(dbl)]
    L.zero_destroy.argtypes = [vp]
    L.zero_destroy.restype = None
    _lib = L
    return L


def _check(rc: int):
    if rc != ZERO_OK:
        raise ZeroError(rc, lib().zero_last_error().decode(errors="replace"))


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return ZERO_BF16
    if dt == torch.float32:
        return ZERO_F32
    raise TypeError(f"only float32 and bfloat16 are supported, got {dt}")


def _resolve_device(device) -> torch.device:
    """The given device, or the current one; always with its index."""
    d = torch.device("cuda") if device is None else torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"a state lives on a cuda device, got {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


# torch's own lookup of a device's current stream handle: 0.1 us, where building
# the stream object costs 1.7 us of a 5.6 us step call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    """The given stream (anything that carries a `cuda_stream` handle), or
    `device`'s current one (whatever device is current in the caller)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    # other objects are taken at their word: they need not know a device
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, state is on {device}")
    return stream.cuda_stream


def _torch_stream(stream, device: torch.device) -> torch.cuda.Stream:
    """The given stream, or the current one, as torch's own object."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream, device=device)


def _capturing(stream, device: torch.device) -> bool:
    """Whether the given stream, or the device's current one, is captured."""
    if stream is None and torch.cuda.current_device() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.cuda.is_current_stream_capturing()


def _ptr_array(ptrs: Sequence[int]):
    return (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)


def shard_geometry(numel: int, world: int, rank: int) -> Tuple[int, int, int]:
    """(shard, lo, padded) for this rank (host computation in the library)."""
    s, lo, p = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().zero_shard_geometry(numel, world, rank, ctypes.byref(s),
                                     ctypes.byref(lo), ctypes.byref(p)))
    return s.value, lo.value, p.value


def state_bytes(stage: int, numel: float, world: float) -> float:
    """Model-state bytes per card for ZeRO stage 0..3."""
    out = ctypes.c_double()
    _check(lib().zero_state_bytes(stage, float(numel), float(world), ctypes.byref(out)))
    return out.value


class ShardState:
    """One data-parallel rank's ZeRO-2 optimizer state on the current GPU.

    Mirrors the pages' ZeroAdam(params, lr, betas, eps) for one rank: the
    library owns fp32 master/m/v of `shard` elements; gradients, flat
    buffers and streams belong to the caller. The step number t is passed
    explicitly (first step t = 1), or kept on the device with schedule()
    for the *_sched calls, which a captured HIP graph can replay.
    """

    def __init__(self, numel: int, world: int, rank: int, lr: float,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 device=None):
        self.device = _resolve_device(device)
        self.numel, self.world, self.rank = int(numel), int(world), int(rank)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().zero_shard_init(self.numel, self.world, self.rank, float(lr),
                                         float(betas[0]), float(betas[1]), float(eps),
                                         ctypes.byref(h)))
        self._h = h
        s, lo, p = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().zero_shard_info(self._h, ctypes.byref(s), ctypes.byref(lo),
                                     ctypes.byref(p)))
        self.shard, self.lo, self.padded = s.value, lo.value, p.value

    # ------------------------------------------------------------ helpers
    def _dev(self, t: torch.Tensor, what: str):
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, state is on {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().zero_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # ------------------------------------------------------------- calls
    def set_step_workgroups(self, per_cu: int):
        """Cap later flat-layout steps at per_cu workgroups per compute unit
        (0: uncapped); results are unchanged."""
        _check(lib().zero_set_step_workgroups(self._h, int(per_cu)))

    def state_bytes(self) -> int:
        """Bytes of fp32 master, m and v this rank holds (12 per element)."""
        out = ctypes.c_int64()
        _check(lib().zero_shard_state_bytes(self._h, ctypes.byref(out)))
        return out.value

    def set_lr(self, lr: float):
        _check(lib().zero_set_lr(self._h, float(lr)))

    def load_master(self, flat_params: torch.Tensor, flat_offset: Optional[int] = None,
                    stream=None):
        """master = fp32(flat_params[flat_offset : flat_offset+shard]); m = v = 0.
        flat_offset defaults to lo for a full padded buffer, 0 otherwise."""
        self._dev(flat_params, "flat_params")
        off = flat_offset
        if off is None:
            off = self.lo if flat_params.numel() >= self.padded else 0
        if flat_params.numel() < off + self.shard:
            raise ValueError(f"flat_params has {flat_params.numel()} elements, "
                             f"need {off + self.shard}")
        _check(lib().zero_load_master(self._h, flat_params.data_ptr(),
                                      _dtype_code(flat_params.dtype), off,
                                      _stream_handle(stream, self.device)))

    def flatten(self, tensors: Sequence[torch.Tensor], out: torch.Tensor, stream=None,
                window: Optional[Tuple[int, int]] = None):
        """out[:numel] = concatenation of the tensors; out[numel:padded] = 0.
        window=(begin, count) writes only flat elements [begin, begin+count)."""
        dt = out.dtype
        self._dev(out, "out")
        if out.numel() < self.padded:
            raise ValueError(f"out has {out.numel()} elements, need {self.padded}")
        for i, t in enumerate(tensors):
            self._dev(t, f"tensors[{i}]")
            if t.dtype != dt:
                raise TypeError(f"tensors[{i}] is {t.dtype}, out is {dt}")
        numels = (ctypes.c_int64 * max(1, len(tensors)))(*[t.numel() for t in tensors])
        ptrs = _ptr_array([t.data_ptr() for t in tensors])
        if window is None:
            _check(lib().zero_flatten(self._h, ptrs, numels, len(tensors), _dtype_code(dt),
                                      out.data_ptr(), _stream_handle(stream, self.device)))
        else:
            b, n = window
            _check(lib().zero_flatten_range(self._h, ptrs, numels, len(tensors), _dtype_code(dt),
                                            out.data_ptr(), int(b), int(n),
                                            _stream_handle(stream, self.device)))

    def unflatten(self, flat: torch.Tensor, tensors: Sequence[torch.Tensor], stream=None):
        """Copy flat[off_t : off_t + numel_t] into each tensor, in order."""
        dt = flat.dtype
        self._dev(flat, "flat")
        if flat.numel() < self.numel:
            raise ValueError(f"flat has {flat.numel()} elements, need {self.numel}")
        for i, t in enumerate(tensors):
            self._dev(t, f"tensors[{i}]")
            if t.dtype != dt:
                raise TypeError(f"tensors[{i}] is {t.dtype}, flat is {dt}")
        numels = (ctypes.c_int64 * max(1, len(tensors)))(*[t.numel() for t in tensors])
        ptrs = _ptr_array([t.data_ptr() for t in tensors])
        _check(lib().zero_unflatten(self._h, flat.data_ptr(), len(tensors), numels,
                                    _dtype_code(dt), ptrs, _stream_handle(stream, self.device)))

    def _step_args(self, replicas, param_out, grad_offset, param_offset):
        if len(replicas) != self.world:
            raise ValueError(f"need {self.world} replicas, got {len(replicas)}")
        gdt = replicas[0].dtype
        go = grad_offset
        if go is None:
            go = self.lo if replicas[0].numel() >= self.padded else 0
        po = param_offset
        if po is None:
            po = self.lo if param_out.numel() >= self.padded else 0
        for q, r in enumerate(replicas):
            self._dev(r, f"replicas[{q}]")
            if r.dtype != gdt:
                raise TypeError("replicas must share one dtype")
            if r.numel() < go + self.shard:
                raise ValueError(f"replicas[{q}] has {r.numel()} elements, need {go + self.shard}")
        self._dev(param_out, "param_out")
        if param_out.numel() < po + self.shard:
            raise ValueError(f"param_out has {param_out.numel()} elements, need {po + self.shard}")
        return _ptr_array([r.data_ptr() for r in replicas]), gdt, int(go), int(po)

    def _range_args(self, shard_begin, count, replicas, param_out, grad_offset, param_offset):
        if len(replicas) != self.world:
            raise ValueError(f"need {self.world} replicas, got {len(replicas)}")
        if shard_begin < 0 or count < 0 or shard_begin + count > self.shard:
            raise ValueError(f"range [{shard_begin}, {shard_begin + count}) outside the shard")
        gdt = replicas[0].dtype
        for q, r in enumerate(replicas):
            self._dev(r, f"replicas[{q}]")
            if r.dtype != gdt:
                raise TypeError("replicas must share one dtype")
            if r.numel() < grad_offset + count:
                raise ValueError(f"replicas[{q}] has {r.numel()} elements, need {grad_offset + count}")
        self._dev(param_out, "param_out")
        if param_out.numel() < param_offset + count:
            raise ValueError(f"param_out has {param_out.numel()} elements, need {param_offset + count}")
        return _ptr_array([r.data_ptr() for r in replicas]), gdt

    def step(self, replicas: Sequence[torch.Tensor], t: int, param_out: torch.Tensor,
             grad_offset: Optional[int] = None, param_offset: Optional[int] = None,
             stream=None):
        """One shard step. replicas[q][grad_offset + i] is rank q's gradient of
        slice element i; writes param_out[param_offset + i]. Offsets default
        to lo for full padded buffers and 0 for slice-sized ones."""
        ptrs, gdt, go, po = self._step_args(replicas, param_out, grad_offset, param_offset)
        _check(lib().zero_step(self._h, ptrs, len(replicas), _dtype_code(gdt), go,
                               param_out.data_ptr(), _dtype_code(param_out.dtype), po,
                               int(t), _stream_handle(stream, self.device)))

    def step_range(self, shard_begin: int, count: int, replicas: Sequence[torch.Tensor],
                   t: int, param_out: torch.Tensor, grad_offset: int = 0,
                   param_offset: int = 0, stream=None):
        """The step on shard elements [shard_begin, shard_begin+count):
        replicas[q][grad_offset + i] feeds element shard_begin + i, which is
        written to param_out[param_offset + i]. Disjoint ranges on different
        streams may run concurrently."""
        ptrs, gdt = self._range_args(shard_begin, count, replicas, param_out, grad_offset,
                                     param_offset)
        _check(lib().zero_step_range(self._h, int(shard_begin), int(count), ptrs, len(replicas),
                                     _dtype_code(gdt), int(grad_offset), param_out.data_ptr(),
                                     _dtype_code(param_out.dtype), int(param_offset), int(t),
                                     _stream_handle(stream, self.device)))

    # ------------------------------------------- device-resident schedule
    def schedule(self, next_t: int = 1, stream=None):
        """Keep the step count and lr on the device (created on first use,
        outside any graph capture): the next scheduled step is next_t."""
        with torch.cuda.device(self.device):
            _check(lib().zero_schedule_init(self._h, int(next_t),
                                            _stream_handle(stream, self.device)))

    def schedule_noalloc(self, next_t: int = 1, stream=None):
        """schedule() in the device's static block: allocates nothing (one
        such schedule per device at a time)."""
        with torch.cuda.device(self.device):
            _check(lib().zero_schedule_init_noalloc(self._h, int(next_t),
                                                    _stream_handle(stream, self.device)))

    def schedule_lr(self, lr: float, stream=None):
        """Learning rate of later scheduled steps (stream-ordered)."""
        _check(lib().zero_schedule_lr(self._h, float(lr), _stream_handle(stream, self.device)))

    def schedule_next_t(self, stream=None) -> int:
        """The next scheduled step count (waits for the stream)."""
        out = ctypes.c_int64()
        _check(lib().zero_schedule_get(self._h, ctypes.byref(out),
                                       _stream_handle(stream, self.device)))
        return out.value

    def step_begin(self, stream=None):
        """Begin the next scheduled step (before step_range_sched calls)."""
        _check(lib().zero_step_begin(self._h, _stream_handle(stream, self.device)))

    def step_sched(self, replicas: Sequence[torch.Tensor], param_out: torch.Tensor,
                   grad_offset: Optional[int] = None, param_offset: Optional[int] = None,
                   stream=None):
        """step() at the device schedule's next step count and lr; advances
        the count. Capturable in a HIP graph."""
        ptrs, gdt, go, po = self._step_args(replicas, param_out, grad_offset, param_offset)
        _check(lib().zero_step_sched(self._h, ptrs, len(replicas), _dtype_code(gdt), go,
                                     param_out.data_ptr(), _dtype_code(param_out.dtype), po,
                                     _stream_handle(stream, self.device)))

    def step_range_sched(self, shard_begin: int, count: int, replicas: Sequence[torch.Tensor],
                         param_out: torch.Tensor, grad_offset: int = 0, param_offset: int = 0,
                         stream=None):
        """step_range() at the step the last step_begin began."""
        ptrs, gdt = self._range_args(shard_begin, count, replicas, param_out, grad_offset,
                                     param_offset)
        _check(lib().zero_step_range_sched(self._h, int(shard_begin), int(count), ptrs,
                                           len(replicas), _dtype_code(gdt), int(grad_offset),
                                           param_out.data_ptr(), _dtype_code(param_out.dtype),
                                           int(param_offset), _stream_handle(stream, self.device)))

    def bucket_ranges(self, bucket_bounds: Sequence[int]) -> List[Tuple[int, int, int, int]]:
        """For gradient buckets given as flat-vector boundaries
        [b0=0, b1, ..., bk=padded], the part of each bucket this rank owns:
        (bucket index, shard_begin, count, offset of that part inside the
        bucket). Buckets that miss this rank's slice are left out."""
        out = []
        lo, hi = self.lo, self.lo + self.shard
        for k in range(len(bucket_bounds) - 1):
            a, b = int(bucket_bounds[k]), int(bucket_bounds[k + 1])
            s, e = max(a, lo), min(b, hi)
            if s < e:
                out.append((k, s - lo, e - s, s - a))
        return out

    def get_state(self, stream=None) -> List[torch.Tensor]:
        """Fresh fp32 copies of (master, m, v)."""
        out = [torch.empty(self.shard, dtype=torch.float32, device=self.device)
               for _ in range(3)]
        _check(lib().zero_get_state(self._h, out[0].data_ptr(), out[1].data_ptr(),
                                    out[2].data_ptr(), _stream_handle(stream, self.device)))
        return out

    def set_state(self, master: torch.Tensor, m: torch.Tensor, v: torch.Tensor, stream=None):
        for name, x in (("master", master), ("m", m), ("v", v)):
            self._dev(x, name)
            if x.dtype != torch.float32 or x.numel() != self.shard:
                raise ValueError(f"{name} must be float32 with {self.shard} elements")
        _check(lib().zero_set_state(self._h, master.data_ptr(), m.data_ptr(), v.data_ptr(),
                                    _stream_handle(stream, self.device)))


def dim0_split(dim0: int, world: int, rank: int) -> Tuple[int, int]:
    """(first row, rows) of this rank's dim-0 shard of a parameter."""
    f, r = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().zero_dim0_split(dim0, world, rank, ctypes.byref(f), ctypes.byref(r)))
    return f.value, r.value


class FsdpShardState(ShardState):
    """One rank of the per-parameter (FSDP2-style) layout: every parameter
    is split along dim 0 and this rank keeps fp32 master/m/v for its rows.
    Inherits get_state / set_state / set_lr / close from ShardState."""

    def __init__(self, shapes, world: int, rank: int, lr: float,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, device=None):
        self.device = _resolve_device(device)
        self.shapes = [tuple(int(d) for d in s) for s in shapes]
        self.world, self.rank = int(world), int(rank)
        n = len(self.shapes)
        dim0 = (ctypes.c_int64 * max(1, n))(*[s[0] if s else 1 for s in self.shapes])
        rown = (ctypes.c_int64 * max(1, n))(*[
            int(torch.Size(s[1:]).numel()) if len(s) > 1 else 1 for s in self.shapes])
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().zero_fsdp_init(n, dim0, rown, self.world, self.rank, float(lr),
                                        float(betas[0]), float(betas[1]), float(eps),
                                        ctypes.byref(h)))
        self._h = h
        self._read_layout()

    def _read_layout(self):
        """shard, numel and every parameter's (first row, rows, state offset)."""
        s_, lo, p = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().zero_shard_info(self._h, ctypes.byref(s_), ctypes.byref(lo), ctypes.byref(p)))
        self.shard, self.lo, self.padded = s_.value, lo.value, p.value
        self.numel = sum(int(torch.Size(s).numel()) for s in self.shapes)
        self.local = []
        for k in range(len(self.shapes)):
            f, r, off = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
            _check(lib().zero_fsdp_local(self._h, k, ctypes.byref(f), ctypes.byref(r),
                                         ctypes.byref(off)))
            self.local.append((f.value, r.value, off.value))

    def local_shape(self, k: int) -> Tuple[int, ...]:
        return (self.local[k][1],) + self.shapes[k][1:]

    def local_numel(self, k: int) -> int:
        return int(torch.Size(self.local_shape(k)).numel())

    def _check_full(self, ts, what):
        if len(ts) != len(self.shapes):
            raise ValueError(f"{what}: need {len(self.shapes)} tensors, got {len(ts)}")
        for k, x in enumerate(ts):
            if x is None:
                if self.local[k][1]:
                    raise ValueError(f"{what}[{k}] is None but this rank holds rows of it")
                continue
            self._dev(x, f"{what}[{k}]")
            if tuple(x.shape) != self.shapes[k] and x.numel() != torch.Size(self.shapes[k]).numel():
                raise ValueError(f"{what}[{k}] has shape {tuple(x.shape)}, need {self.shapes[k]}")

    def load_master(self, params: Sequence[torch.Tensor], stream=None):
        """master = this rank's rows of each full parameter; m = v = 0."""
        self._check_full(params, "params")
        dts = {p.dtype for p in params if p is not None}
        if len(dts) != 1:
            raise TypeError("params must share one dtype")
        ptrs = _ptr_array([p.data_ptr() if p is not None else 0 for p in params])
        _check(lib().zero_fsdp_load_master(self._h, ptrs, _dtype_code(dts.pop()),
                                           _stream_handle(stream, self.device)))

    def _fsdp_args(self, replica_grads, params_out):
        if len(replica_grads) != self.world:
            raise ValueError(f"need {self.world} replicas, got {len(replica_grads)}")
        gdts = set()
        for q, gl in enumerate(replica_grads):
            self._check_full(gl, f"replica_grads[{q}]")
            gdts |= {g.dtype for g in gl if g is not None}
        if len(gdts) != 1:
            raise TypeError("gradients must share one dtype")
        if len(params_out) != len(self.shapes):
            raise ValueError("need one output shard per parameter")
        pdts = set()
        for k, o in enumerate(params_out):
            if self.local[k][1] == 0:
                continue
            self._dev(o, f"params_out[{k}]")
            if o.numel() < self.local_numel(k):
                raise ValueError(f"params_out[{k}] has {o.numel()} elements, "
                                 f"need {self.local_numel(k)}")
            pdts.add(o.dtype)
        if len(pdts) > 1:
            raise TypeError("outputs must share one dtype")
        pdt = pdts.pop() if pdts else torch.float32
        gptrs = _ptr_array([g.data_ptr() if g is not None else 0
                            for gl in replica_grads for g in gl])
        optrs = _ptr_array([o.data_ptr() if (o is not None and self.local[k][1]) else 0
                            for k, o in enumerate(params_out)])
        return gptrs, gdts.pop(), optrs, pdt

    def step(self, replica_grads: Sequence[Sequence[torch.Tensor]], t: int,
             params_out: Sequence[torch.Tensor], stream=None):
        """replica_grads[q][k]: replica q's full gradient of parameter k;
        params_out[k]: this rank's local shard of parameter k (written)."""
        gptrs, gdt, optrs, pdt = self._fsdp_args(replica_grads, params_out)
        _check(lib().zero_fsdp_step(self._h, gptrs, self.world, _dtype_code(gdt), optrs,
                                    _dtype_code(pdt), int(t), _stream_handle(stream, self.device)))

    def step_sched(self, replica_grads: Sequence[Sequence[torch.Tensor]],
                   params_out: Sequence[torch.Tensor], stream=None):
        """step() at the device schedule's next step count and lr."""
        gptrs, gdt, optrs, pdt = self._fsdp_args(replica_grads, params_out)
        _check(lib().zero_fsdp_step_sched(self._h, gptrs, self.world, _dtype_code(gdt), optrs,
                                          _dtype_code(pdt), _stream_handle(stream, self.device)))

    def state_pieces(self, state: Sequence[torch.Tensor]):
        """Split (master, m, v) from get_state into per-parameter local pieces."""
        out = []
        for x in state:
            out.append([x[off:off + r * (int(torch.Size(self.shapes[k][1:]).numel())
                                          if len(self.shapes[k]) > 1 else 1)]
                        for k, (_, r, off) in enumerate(self.local)])
        return out


class _Memory:
    """Library memory as torch sees it: torch.as_tensor(_Memory(...)) shares
    the buffer and keeps `owner` alive."""

    def __init__(self, owner, ptr: int, count: int, typestr: str):
        self.owner = owner
        self.__cuda_array_interface__ = dict(shape=(count,), typestr=typestr,
                                             data=(ptr, False), version=2)


class AdamWState(FsdpShardState):
    """AdamW over many tensors at once, one rank of the per-parameter layout:
    decoupled weight decay and a learning-rate scale per parameter (a number
    for all, or one each), clipping by a norm that stays on the device, and
    states in 32 or 8 bits. Gradients and outputs are bound once; a step is
    one launch and can be captured in a HIP graph.

        st = AdamWState([p.shape for p in params], world, rank, lr, weight_decay=0.1)
        st.load_master(params)
        st.bind([[p.grad for p in params]], params_out)
        s = st.sumsq()                       # all_reduce(s) where ranks share a model
        st.step(t, sumsq=s, max_norm=1.0)

    Inherits get_state / set_state / state_bytes / set_lr / load_master and the
    schedule calls; calls on one state must be ordered among themselves."""

    def __init__(self, shapes, world: int, rank: int, lr: float,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.0, lr_scale=1.0, state_bits: int = 32, seed: int = 0,
                 device=None):
        self.device = _resolve_device(device)
        self.shapes = [tuple(int(d) for d in s) for s in shapes]
        self.world, self.rank, self.state_bits = int(world), int(rank), int(state_bits)
        if not 0 <= int(seed) < 1 << 32:
            raise ValueError(f"seed must be in [0, 2^32), got {seed}")
        n = len(self.shapes)
        dim0 = (ctypes.c_int64 * max(1, n))(*[s[0] if s else 1 for s in self.shapes])
        # a parameter without elements has no rows; the library wants rows of >= 1
        rown = [int(torch.Size(s[1:]).numel()) if len(s) > 1 else 1 for s in self.shapes]
        for k, r in enumerate(rown):
            if r == 0:
                dim0[k], rown[k] = 0, 1
        rown = (ctypes.c_int64 * max(1, n))(*rown)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().zero_adamw_init(n, dim0, rown, self.world, self.rank, float(lr),
                                         float(betas[0]), float(betas[1]), float(eps),
                                         self.state_bits, int(seed), ctypes.byref(h)))
        self._h = h
        self._bound = None
        self._bound_on = 0          # stream that was current at the last bind
        self._captured = []         # bindings that a captured bind keeps alive
        self._read_layout()
        # (elements of this rank, of the parameter, before this rank's first)
        self._sizes = []
        for k, (first, rows, _) in enumerate(self.local):
            local = self.local_numel(k)
            self._sizes.append((local, int(torch.Size(self.shapes[k]).numel()),
                                first * (local // rows) if rows else 0))
        self.set_groups(weight_decay, lr_scale)
        torch.cuda.current_stream(self.device).synchronize()    # for calls on any stream

    def set_groups(self, weight_decay=0.0, lr_scale=1.0, stream=None):
        """Weight decay and learning-rate scale of later steps: a number for
        every parameter, or a sequence with one each."""
        n = len(self.shapes)
        arrays = []
        for name, x in (("weight_decay", weight_decay), ("lr_scale", lr_scale)):
            x = [float(v) for v in x] if hasattr(x, "__len__") else [float(x)] * n
            if len(x) != n:
                raise ValueError(f"{name}: need {n} values, got {len(x)}")
            arrays.append((ctypes.c_double * max(1, n))(*x))
        _check(lib().zero_adamw_groups(self._h, *arrays, _stream_handle(stream, self.device)))

    def _pointers(self, xs: Sequence[Optional[torch.Tensor]], what: str, whole: bool) -> list:
        """Addresses of this rank's elements of every parameter in xs, whose
        tensors hold these alone or, for gradients (`whole`), the parameter."""
        ptrs = []
        for k, (x, (local, full, first)) in enumerate(zip(xs, self._sizes)):
            if local == 0:
                ptrs.append(0)
                continue
            if x is None:
                raise ValueError(f"{what}[{k}] is None but this rank holds rows of it")
            if x.device != self.device or not x.is_contiguous():
                self._dev(x, f"{what}[{k}]")
            n = x.numel()
            if n == local:
                ptrs.append(x.data_ptr())
            elif whole and n == full:
                ptrs.append(x.data_ptr() + first * x.element_size())
            else:
                raise ValueError(f"{what}[{k}] has {n} elements, need {local}"
                                 + (f" (this rank's) or {full}" if whole else ""))
        return ptrs

    def bind(self, grads: Sequence[Sequence[Optional[torch.Tensor]]],
             params_out: Optional[Sequence[Optional[torch.Tensor]]] = None, stream=None):
        """grads[q][k]: replica q's gradient of parameter k, this rank's rows
        or all of them; the mean is over the replicas given (one list for
        gradients that are reduced already). params_out[k]: this rank's rows,
        written by steps; None binds gradients alone (for sumsq). None is
        taken for parameters of which this rank holds no rows. The state
        keeps the tensors alive until the next bind, and that one on another
        stream than the current one, or than was current when they were bound,
        marks them as used there (Tensor.record_stream), so that calls still
        running find them whole; other tensors that were made on yet another
        stream are the caller's to mark, as for torch's own operations. A bind
        that is captured into a graph (never the first) uploads its pointers
        with every replay; the state then keeps its tensors, and those bound
        before it, alive until close(). A step
        reads these very buffers, so gradients stay in place
        (zero_grad(set_to_none=False)) or are bound again."""
        n = len(self.shapes)
        for q, gl in enumerate(grads):
            if len(gl) != n:
                raise ValueError(f"grads[{q}]: need {n} tensors, got {len(gl)}")
        if params_out is not None and len(params_out) != n:
            raise ValueError(f"params_out: need {n} tensors, got {len(params_out)}")
        held = [k for k in range(n) if self._sizes[k][0]]
        gdts = {gl[k].dtype for gl in grads for k in held if gl[k] is not None}
        pdts = {params_out[k].dtype for k in held if params_out[k] is not None} \
            if params_out is not None else set()
        if len(gdts) > 1 or len(pdts) > 1:
            raise TypeError("gradients must share one dtype, and outputs one")
        gptrs = _ptr_array([p for q, gl in enumerate(grads)
                            for p in self._pointers(gl, f"grads[{q}]", True)])
        optrs = None if params_out is None else _ptr_array(
            self._pointers(params_out, "params_out", False))
        gdt = _dtype_code(gdts.pop()) if gdts else ZERO_F32
        pdt = _dtype_code(pdts.pop()) if pdts else ZERO_F32
        handle, current = _stream_handle(stream, self.device), _stream_handle(None, self.device)
        _check(lib().zero_adamw_bind(self._h, gptrs, len(grads), gdt, optrs, pdt, handle))
        bound = ([list(gl) for gl in grads], None if params_out is None else list(params_out))
        if _capturing(stream, self.device):
            self._captured += [self._bound, bound]
        elif self._bound is not None and (handle != current or handle != self._bound_on):
            # a context's calls are ordered among themselves, so what this
            # stream has behind it includes every call that used them
            at = _torch_stream(stream, self.device)
            for xs in (*self._bound[0], self._bound[1] or ()):
                for x in xs:
                    if x is not None:
                        x.record_stream(at)
        self._bound = bound
        self._bound_on = current

    def close(self):
        super().close()             # waits for the device
        self._bound, self._captured = None, []

    def _sum_ptr(self, x: Optional[torch.Tensor], stream=None):
        if x is None:
            return None
        self._dev(x, "sumsq")
        if x.dtype != torch.float64 or x.numel() != 1:
            raise ValueError("sumsq must be one float64")
        if stream is not None:
            x.record_stream(_torch_stream(stream, self.device))
        return x.data_ptr()

    def sumsq(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Sum of squares of the mean gradient over this rank's elements, as
        one float64 on the device (its root is the norm); written to `out`,
        or to a new tensor of the call's stream. Its last bits go by the
        order of the additions, which the gradients' addresses modulo four
        elements decide as well as the sizes."""
        if out is None:
            at = None if stream is None else _torch_stream(stream, self.device)
            with torch.cuda.device(self.device), torch.cuda.stream(at):
                out = torch.empty(1, dtype=torch.float64, device=self.device)
        _check(lib().zero_adamw_sumsq(self._h, self._sum_ptr(out, stream),
                                      _stream_handle(stream, self.device)))
        return out

    def step(self, t: int, sumsq: Optional[torch.Tensor] = None,
             max_norm: Optional[float] = None, stream=None):
        """One step at step number t on the bound buffers. With sumsq (the
        sum over all ranks, on the device) the gradient is scaled by
        min(1, max_norm / (sqrt(sumsq) + 1e-6)), and a sum that is not finite
        makes the step write nothing."""
        if sumsq is not None and max_norm is None:
            raise ValueError("clipping needs max_norm")
        _check(lib().zero_adamw_step(self._h, int(t), self._sum_ptr(sumsq, stream),
                                     float(max_norm or 0.0), _stream_handle(stream, self.device)))

    def step_sched(self, sumsq: Optional[torch.Tensor] = None,
                   max_norm: Optional[float] = None, stream=None):
        """step() at the device schedule's next step count and lr; advances
        the count. Capturable in a HIP graph."""
        if sumsq is not None and max_norm is None:
            raise ValueError("clipping needs max_norm")
        _check(lib().zero_adamw_step_sched(self._h, self._sum_ptr(sumsq, stream),
                                           float(max_norm or 0.0),
                                           _stream_handle(stream, self.device)))

    def state_tensors(self) -> dict:
        """The state itself, sharing the library's memory (until close()):
        master, m, v in fp32, or with 8 bits master in fp32, m and r = sqrt(v)
        as float8_e4m3fn codes and scale as float8_e8m0fnu, shaped
        [shard / 2048, 2, 64]: of every 32 elements of m, then of r."""
        ptr = [ctypes.c_void_p() for _ in range(4)]
        _check(lib().zero_adamw_state(self._h, *[ctypes.byref(p) for p in ptr]))

        def share(p, count, typestr):
            if count == 0:
                dt = torch.float32 if typestr == "<f4" else torch.uint8
                return torch.empty(0, dtype=dt, device=self.device)
            return torch.as_tensor(_Memory(self, p.value, count, typestr), device=self.device)

        n = self.shard
        if self.state_bits == 32:
            return dict(zip(("master", "m", "v"), (share(p, n, "<f4") for p in ptr[:3])))
        return dict(master=share(ptr[0], n, "<f4"),
                    m=share(ptr[1], n, "|u1").view(torch.float8_e4m3fn),
                    r=share(ptr[2], n, "|u1").view(torch.float8_e4m3fn),
                    scale=share(ptr[3], n // 16, "|u1").view(torch.float8_e8m0fnu).view(-1, 2, 64))
