"""GB300 ZeRO-DP partitioned mixed-precision AdamW step: Python binding of libzero_shard.so.

Argument marshalling only: every function here converts tensors to raw pointers and the
current CUDA stream to a handle, calls the C entry point of the same name declared in
include/zero.h, and raises ZeroError on a non-zero status.  All computation happens in
the library's CUDA kernels; if the library has not been built, loading fails loudly
(there is no fallback).  Build it with ``zero_partitioned_optimizer_shard_gb300._build.build()``
or ``__graft_entry__.build()``.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzero_shard.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ENOMEM, ZERO_ECUDA, ZERO_ETIMEOUT = 0, -1, -2, -3, -4, -5
ZERO_F16, ZERO_BF16, ZERO_F32, ZERO_U8 = 1, 2, 3, 4
ZERO_STATE8_BLOCK = 256
ZERO_MAX_KERNEL_RANKS = 64
ZERO_TILE_ELEMS = 8192


class ZeroError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = _lib().zero_strerror(status).decode()
        super().__init__(f"{fn}: {msg} (status {status}" +
                         (f", cudaError {cuda_error})" if status == ZERO_ECUDA else ")"))


class Layout(C.Structure):
    _fields_ = [
        ("psi", C.c_uint64), ("shard", C.c_uint64), ("psi_padded", C.c_uint64), ("pad", C.c_uint64),
        ("bucket_elems", C.c_uint64), ("n_buckets", C.c_uint64), ("tiles_per_rank", C.c_uint64),
        ("n_tiles", C.c_uint64), ("bytes_per_rank", C.c_uint64 * 4),
        ("comm_elems_per_rank", C.c_uint64 * 4), ("n_ranks", C.c_uint32), ("stage", C.c_uint32),
        ("align", C.c_uint32), ("tile_elems", C.c_uint32),
    ]


class HParams(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float),
                ("weight_decay", C.c_float), ("max_grad_norm", C.c_float),
                ("params_dtype", C.c_uint32)]


class StepState(C.Structure):
    _fields_ = [
        ("sumsq", C.c_double), ("norm", C.c_double), ("clip_coef", C.c_float),
        ("loss_scale", C.c_float), ("inv_scale", C.c_float), ("step_size", C.c_float),
        ("rbc2", C.c_float), ("decay", C.c_float), ("overflow", C.c_uint32), ("skip", C.c_uint32),
        ("t", C.c_uint32), ("good_steps", C.c_uint32), ("growth_interval", C.c_uint32),
        ("dynamic", C.c_uint32), ("n_ranks", C.c_uint32), ("n_steps", C.c_uint32),
        ("n_skipped", C.c_uint32), ("error", C.c_uint32), ("arrivals", C.c_uint32),
        ("inv_scale_used", C.c_float), ("launch_arrivals", C.c_uint32),
        ("applied_c", C.c_float), ("adamw_next_chunk", C.c_uint64), ("adamw_done", C.c_uint32),
        ("reserved", C.c_uint32 * 5),
    ]


class Tensor(C.Structure):
    """One tensor of a list (zero_tensor_t)."""
    _fields_ = [
        ("elems", C.c_uint64), ("grad", C.c_void_p), ("master", C.c_void_p), ("m", C.c_void_p),
        ("v", C.c_void_p), ("exps", C.c_void_p), ("params", C.c_void_p),
        ("grad_dtype", C.c_uint32), ("state_dtype", C.c_uint32), ("params_dtype", C.c_uint32),
        ("lr_scale", C.c_float), ("weight_decay", C.c_float), ("reserved", C.c_uint32),
    ]


assert C.sizeof(StepState) == 128 and C.sizeof(Tensor) == 80
STATE_BYTES = C.sizeof(StepState)

_P = C.c_void_p
_L = None


def _lib() -> C.CDLL:
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                               "(zero_partitioned_optimizer_shard_gb300._build.build())")
        L = C.CDLL(LIB_PATH)
        L.zero_partition.argtypes = [C.c_uint64, C.c_uint32, C.c_uint32, C.c_uint32, C.c_uint64,
                                     C.POINTER(Layout)]
        L.zero_segment_map.argtypes = [C.POINTER(Layout), _P, C.c_uint64, _P, C.c_uint64,
                                       C.POINTER(C.c_uint64)]
        L.zero_workspace_bytes.argtypes = [C.POINTER(Layout)]
        L.zero_workspace_bytes.restype = C.c_size_t
        L.zero_step_state_init.argtypes = [C.POINTER(Layout), C.c_float, C.c_uint32, C.c_uint32,
                                           _P, _P, _P]
        L.zero_step_state_read.argtypes = [_P, C.POINTER(StepState), _P]
        L.zero_step_state_write.argtypes = [_P, C.POINTER(StepState), _P]
        L.zero_reduce_shard_unscale.argtypes = [C.POINTER(Layout), C.c_int, C.POINTER(_P),
                                                C.c_uint64, C.c_uint64, _P, _P, _P, _P]
        L.zero_grad_norm.argtypes = [C.POINTER(Layout), C.POINTER(HParams), _P, _P, _P]
        L.zero_adamw_cast_gather.argtypes = [C.POINTER(Layout), C.POINTER(HParams), _P, _P, _P, _P,
                                             _P, _P, _P]
        L.zero_adamw_cast_gather_host_state.argtypes = L.zero_adamw_cast_gather.argtypes
        L.zero_step.argtypes = [C.POINTER(Layout), C.POINTER(HParams), C.c_int, C.POINTER(_P), _P,
                                _P, _P, _P, _P, _P, _P, _P]
        L.zero_step_host.argtypes = [C.POINTER(Layout), C.POINTER(HParams), C.c_int, C.POINTER(_P),
                                     _P, C.c_uint64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.zero_reduce_shard_unscale_local.argtypes = [C.POINTER(Layout), C.c_int, C.c_uint32,
                                                      C.c_uint32, C.POINTER(_P), C.c_uint64,
                                                      C.c_uint64, _P, _P, _P, _P]
        L.zero_adamw_cast_gather_local.argtypes = [C.POINTER(Layout), C.POINTER(HParams),
                                                   C.c_uint32, C.c_uint32, _P, _P, _P, _P, _P,
                                                   _P, _P]
        L.zero_step_launches.argtypes = [C.POINTER(Layout), C.c_int]
        L.zero_step_static_workspace.argtypes = [C.POINTER(Layout), C.POINTER(HParams), C.c_int,
                                                 C.POINTER(_P), _P, _P, _P, _P, _P, _P, _P]
        L.zero_tensors_workspace_bytes.argtypes = [C.c_uint64]
        L.zero_tensors_workspace_bytes.restype = C.c_size_t
        L.zero_tensors_state_init.argtypes = [C.c_uint32, C.c_float, C.c_uint32, C.c_uint32, _P, _P]
        L.zero_tensors_grad_norm.argtypes = [_P, C.c_uint64, C.POINTER(HParams), _P, _P, _P]
        L.zero_tensors_adamw.argtypes = [_P, C.c_uint64, C.POINTER(HParams), _P, _P]
        L.zero_tensors_adamw8.argtypes = [_P, C.c_uint64, C.POINTER(HParams), C.c_uint64, _P, _P]
        L.zero_tensors_state8_read.argtypes = [_P, _P, C.c_uint64, _P]
        L.zero_tensors_state8_write.argtypes = L.zero_tensors_state8_read.argtypes
        u32, u64, f32 = C.c_uint32, C.c_uint64, C.c_float
        L.zero_layernorm.argtypes = [C.c_int, u64, u32, _P, u64, _P, _P, C.c_int, f32, _P, u64, _P, _P, _P]
        L.zero_layernorm_workspace_bytes.argtypes = [u64, u32]
        L.zero_layernorm_backward.argtypes = [C.c_int, u64, u32, _P, u64, _P, C.c_int, _P, _P, _P, u64, _P, u64,
                                              _P, _P, C.c_int, u32, _P, _P]
        L.zero_embedding.argtypes = [C.c_int, u64, u32, u32, _P, u32, _P, f32, _P, u64, _P]
        L.zero_embedding_workspace_bytes.argtypes = [u64, u32, u32]
        L.zero_embedding_backward.argtypes = [C.c_int, u64, u32, u32, _P, u32, _P, u64, f32, _P, C.c_int, u32, _P,
                                              _P]
        L.zero_head_workspace_bytes.argtypes = [u64, u32, u32]
        L.zero_head_loss.argtypes = [C.c_int, u64, u32, u32, _P, u64, _P, _P, u32, _P, _P, _P, _P]
        L.zero_head_loss_backward.argtypes = [C.c_int, u64, u32, u32, _P, u64, _P, _P, u32, _P, f32, _P, _P, _P, u64,
                                              _P, C.c_int, u32, _P, _P]
        for name in ("layernorm", "embedding", "head"):
            getattr(L, f"zero_{name}_workspace_bytes").restype = C.c_size_t
        L.zero_strerror.argtypes = [C.c_int]
        L.zero_strerror.restype = C.c_char_p
        L.zero_last_cuda_error.argtypes = []
        for name in ("zero_partition", "zero_segment_map", "zero_step_state_init", "zero_step_state_read",
                     "zero_step_state_write", "zero_reduce_shard_unscale", "zero_grad_norm",
                     "zero_adamw_cast_gather", "zero_adamw_cast_gather_host_state", "zero_step",
                     "zero_step_host", "zero_last_cuda_error", "zero_reduce_shard_unscale_local",
                     "zero_adamw_cast_gather_local", "zero_step_launches",
                     "zero_step_static_workspace", "zero_tensors_state_init",
                     "zero_tensors_grad_norm", "zero_tensors_adamw", "zero_tensors_adamw8",
                     "zero_tensors_state8_read", "zero_tensors_state8_write", "zero_layernorm",
                     "zero_layernorm_backward", "zero_embedding", "zero_embedding_backward", "zero_head_loss",
                     "zero_head_loss_backward"):
            getattr(L, name).restype = C.c_int
        _L = L
    return _L


def lib() -> C.CDLL:
    """The loaded library (raises if it has not been built)."""
    return _lib()


def _check(fn: str, status: int) -> None:
    if status != ZERO_OK:
        raise ZeroError(fn, status, _lib().zero_last_cuda_error() if status == ZERO_ECUDA else 0)


def _ptr(x) -> int | None:
    """Tensor, int address or None -> address."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        # the current stream's handle without building a Stream object: 0.1 against 2.9 us
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr_array(xs: Sequence) -> C.Array:
    return (_P * len(xs))(*[_ptr(x) for x in xs])


def hparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
            max_grad_norm=1.0, params_dtype=0) -> HParams:
    """params_dtype: 0 or ZERO_BF16 for bf16 gathered parameters, ZERO_F16 for fp16."""
    return HParams(lr, beta1, beta2, eps, weight_decay, max_grad_norm, params_dtype)


# --------------------------------------------------------------------------------------
# entry points (same names as include/zero.h)
# --------------------------------------------------------------------------------------
def zero_partition(psi: int, n_ranks: int, stage: int = 2, align: int = 1,
                   bucket_elems: int = 0) -> Layout:
    lay = Layout()
    _check("zero_partition", _lib().zero_partition(psi, n_ranks, stage, align, bucket_elems,
                                                   C.byref(lay)))
    return lay


class Segment(C.Structure):
    """One piece of a model tensor inside one rank's shard (zero_segment_t)."""
    _fields_ = [("tensor", C.c_uint64), ("rank", C.c_uint64), ("tensor_offset", C.c_uint64),
                ("shard_offset", C.c_uint64), ("count", C.c_uint64)]


def zero_segment_map(layout: Layout, tensor_elems: Sequence[int]) -> list:
    """Each tensor's piece on each rank, in flat order: a list of Segment."""
    n_t = len(tensor_elems)
    sizes = (C.c_uint64 * max(n_t, 1))(*tensor_elems)
    n = C.c_uint64()
    _check("zero_segment_map", _lib().zero_segment_map(C.byref(layout), sizes, n_t, None, 0,
                                                       C.byref(n)))
    out = (Segment * max(n.value, 1))()
    _check("zero_segment_map", _lib().zero_segment_map(C.byref(layout), sizes, n_t, out, n.value,
                                                       C.byref(n)))
    return list(out[:n.value])


def zero_workspace_bytes(layout: Layout) -> int:
    return _lib().zero_workspace_bytes(C.byref(layout))


def zero_step_state_init(layout: Layout, loss_scale: float, dynamic: bool, growth_interval: int,
                         st, partials, stream=None) -> None:
    _check("zero_step_state_init", _lib().zero_step_state_init(
        C.byref(layout), loss_scale, int(bool(dynamic)), growth_interval, _ptr(st), _ptr(partials),
        _stream(stream)))


def zero_step_state_read(st, stream=None) -> StepState:
    out = StepState()
    _check("zero_step_state_read", _lib().zero_step_state_read(_ptr(st), C.byref(out), _stream(stream)))
    return out


def zero_step_state_write(st, state: StepState, stream=None) -> None:
    _check("zero_step_state_write", _lib().zero_step_state_write(_ptr(st), C.byref(state),
                                                                 _stream(stream)))


def zero_reduce_shard_unscale(layout: Layout, dtype: int, replicas: Sequence, begin: int, count: int,
                              g, partials, st, stream=None) -> None:
    _check("zero_reduce_shard_unscale", _lib().zero_reduce_shard_unscale(
        C.byref(layout), dtype, _ptr_array(replicas), begin, count, _ptr(g), _ptr(partials),
        _ptr(st), _stream(stream)))


def zero_grad_norm(layout: Layout, hp: HParams, partials, st, stream=None) -> None:
    _check("zero_grad_norm", _lib().zero_grad_norm(C.byref(layout), C.byref(hp), _ptr(partials),
                                                   _ptr(st), _stream(stream)))


def zero_adamw_cast_gather(layout: Layout, hp: HParams, g, master, m, v, params, st,
                           stream=None) -> None:
    _check("zero_adamw_cast_gather", _lib().zero_adamw_cast_gather(
        C.byref(layout), C.byref(hp), _ptr(g), _ptr(master), _ptr(m), _ptr(v), _ptr(params),
        _ptr(st), _stream(stream)))


def zero_adamw_cast_gather_host_state(layout: Layout, hp: HParams, g, master, m, v, params, st,
                                      stream=None) -> None:
    """master, m, v: page-locked host buffers (e.g. torch pin_memory tensors)."""
    _check("zero_adamw_cast_gather_host_state", _lib().zero_adamw_cast_gather_host_state(
        C.byref(layout), C.byref(hp), _ptr(g), _ptr(master), _ptr(m), _ptr(v), _ptr(params),
        _ptr(st), _stream(stream)))


def zero_reduce_shard_unscale_local(layout: Layout, dtype: int, rank_begin: int, rank_count: int,
                                    replicas: Sequence, begin: int, count: int, g_local, partials,
                                    st, stream=None) -> None:
    """g_local holds flat [rank_begin*S, (rank_begin+rank_count)*S) from index 0."""
    f = _lib().zero_reduce_shard_unscale_local
    _check("zero_reduce_shard_unscale_local", f(
        C.byref(layout), dtype, rank_begin, rank_count, _ptr_array(replicas), begin, count,
        _ptr(g_local), _ptr(partials), _ptr(st), _stream(stream)))


def zero_adamw_cast_gather_local(layout: Layout, hp: HParams, rank_begin: int, rank_count: int,
                                 g_local, master_local, m_local, v_local, params_local, st,
                                 stream=None) -> None:
    f = _lib().zero_adamw_cast_gather_local
    _check("zero_adamw_cast_gather_local", f(
        C.byref(layout), C.byref(hp), rank_begin, rank_count, _ptr(g_local), _ptr(master_local),
        _ptr(m_local), _ptr(v_local), _ptr(params_local), _ptr(st), _stream(stream)))


def zero_step(layout: Layout, hp: HParams, dtype: int, replicas: Sequence, g, partials, master, m,
              v, params, st, stream=None) -> None:
    """replicas: n_buckets * N device buffers (or addresses), bucket-major."""
    _check("zero_step", _lib().zero_step(
        C.byref(layout), C.byref(hp), dtype, _ptr_array(replicas), _ptr(g), _ptr(partials),
        _ptr(master), _ptr(m), _ptr(v), _ptr(params), _ptr(st), _stream(stream)))


def zero_step_launches(layout: Layout, dtype: int) -> int:
    """Kernel launches of one zero_step call for this layout: 1 (single-launch step) or
    n_buckets + 2."""
    f = _lib().zero_step_launches
    n = f(C.byref(layout), dtype)
    if n < 0:
        _check("zero_step_launches", n)
    return n


def zero_step_host(layout: Layout, hp: HParams, dtype: int, host_replicas: Sequence, staging,
                   staging_bytes: int, g, partials, master, m, v, params, st,
                   host_state_out=None, stream=None, copy_stream=None) -> None:
    """host_replicas: N pinned host buffers (or addresses) of psi_padded elements each."""
    _check("zero_step_host", _lib().zero_step_host(
        C.byref(layout), C.byref(hp), dtype, _ptr_array(host_replicas), _ptr(staging),
        staging_bytes, _ptr(g), _ptr(partials), _ptr(master), _ptr(m), _ptr(v), _ptr(params),
        _ptr(st), _ptr(host_state_out), _stream(stream), _stream(copy_stream)))


def zero_step_static_workspace(layout: Layout, hp: HParams, dtype: int, replicas: Sequence, g,
                               master, m, v, params, st, stream=None) -> None:
    """zero_step without a caller workspace: for callers that cannot allocate device
    memory.  The per-tile partials live in the library's static device array (8 MiB per
    GPU); calls must not overlap on the GPU.  See include/zero.h."""
    f = _lib().zero_step_static_workspace
    _check("zero_step_static_workspace", f(
        C.byref(layout), C.byref(hp), dtype, _ptr_array(replicas), _ptr(g), _ptr(master), _ptr(m),
        _ptr(v), _ptr(params), _ptr(st), _stream(stream)))


# --------------------------------------------------------------------------------------
# lists of tensors
# --------------------------------------------------------------------------------------
_CODES = {}
_ID_BYTES = {}


def _dtype_codes() -> dict:
    """torch dtypes to zero_dtype_t; 16-bit integers to 0 (parameters' bit patterns)."""
    if not _CODES:
        import torch
        _ID_BYTES.update({torch.int32: 4, torch.int64: 8})
        _CODES.update({torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32,
                       torch.uint8: ZERO_U8, torch.int16: 0, torch.uint16: 0})
    return _CODES


def _order(t) -> tuple:
    """Where a tensor's elements lie: a dimension of one element has no say in it."""
    return t.shape, [s for n, s in zip(t.shape, t.stride()) if n > 1]


class TensorList:
    """A list of tensors for the zero_tensors_* calls: the C array of zero_tensor_t, built
    once and used for as long as the tensors stay where they are.

    Every argument is a sequence with one entry per tensor, or None where no call on this
    list needs it; all are CUDA tensors of one device.  A tensor's arrays are contiguous, or
    dense in one and the same other order (channels last, a transposed weight).  grad: fp16,
    bf16 or fp32; master: fp32; m, v: fp32, or uint8 codes with exps, uint8 of
    2*ceil(elems/256) (bf16 m and v only as a target of zero_tensors_state8_read); params:
    bf16 or fp16, or 16-bit integers, whose type is then the hyperparameters'.  lr_scale,
    weight_decay: one number, or one per tensor; without a weight_decay each call takes its
    hyperparameters'.  The list keeps its tensors alive; set_grad() takes gradients that have
    moved.  The calls write the tensors in place, past autograd, and one step state serves one
    stream at a time."""

    _TYPES = {"grad": (ZERO_F16, ZERO_BF16, ZERO_F32), "master": (ZERO_F32,), "exps": (ZERO_U8,),
              "m": (ZERO_F32, ZERO_BF16, ZERO_U8), "v": (ZERO_F32, ZERO_BF16, ZERO_U8),
              "params": (ZERO_F16, ZERO_BF16, 0)}

    def __init__(self, grad=None, master=None, m=None, v=None, exps=None, params=None, lr_scale=1.0,
                 weight_decay=None):
        arrays = {"master": master, "m": m, "v": v, "grad": grad, "params": params, "exps": exps}
        self.tensors = {k: list(x) for k, x in arrays.items() if x is not None}
        if not self.tensors or list(self.tensors) == ["exps"]:
            raise ValueError("a list of tensors needs at least one of grad, master, m, v, params")
        if ("m" in self.tensors) != ("v" in self.tensors):
            raise ValueError("m and v come together")
        first = next(iter(self.tensors.values()))
        self.elems = [t.numel() for t in first]
        self.device = first[0].get_device() if first else -1
        self._work_bytes = None    # zero_tensors_workspace_bytes, once a norm needs it
        self._other_order = set()  # where the arrays besides the gradient are not contiguous
        n = len(first)
        for k, x in self.tensors.items():
            if len(x) != n:
                raise ValueError(f"{k} has {len(x)} tensors, the list {n}")
        codes = {k: self._check(k, x) for k, x in self.tensors.items()}
        if codes.get("m") != codes.get("v"):
            i = next(i for i, (a, b) in enumerate(zip(codes["m"], codes["v"])) if a != b)
            raise ValueError(f"m[{i}] and v[{i}] differ in type")
        # the decay that the array holds where it is the hyperparameters', else None
        self._hp_decay = 0.0 if weight_decay is None else None
        none = [None] * n
        ptr = {k: [t.data_ptr() for t in x] for k, x in self.tensors.items()}
        zeros = [0] * n
        self.array = (Tensor * max(n, 1))()
        for i, row in enumerate(zip(
                self.elems, *(ptr.get(k, none) for k in ("grad", "master", "m", "v", "exps", "params")),
                *(codes.get(k, zeros) for k in ("grad", "m", "params")), self._numbers(lr_scale),
                self._numbers(0.0 if weight_decay is None else weight_decay))):
            self.array[i] = row

    def __len__(self) -> int:
        return len(self.elems)

    def _take_decay(self, decay: float) -> None:
        self._hp_decay = decay
        for a in self.array:
            a.weight_decay = decay

    def _numbers(self, x) -> list:
        x = list(x) if hasattr(x, "__len__") else [x] * len(self)
        if len(x) != len(self):
            raise ValueError("lr_scale and weight_decay: one number, or one per tensor")
        return x

    def _check(self, name: str, xs: list) -> list:
        """The tensors' type codes, once every one of them is what the kernels take."""
        known, types, device, codes = _dtype_codes(), self._TYPES[name], self.device, []
        other = self._other_order if name != "exps" else set()  # exps have an order of their own
        for i, (t, n) in enumerate(zip(xs, self.elems)):
            want = 2 * -(-n // ZERO_STATE8_BLOCK) if name == "exps" else n
            if t.numel() != want:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements, not {want}")
            if not t.is_cuda or t.get_device() != device:
                raise ValueError(f"{name}[{i}] is not a CUDA tensor of the list's device")
            if not t.is_contiguous() or (other and i in other):
                self._check_order(name, i, t)
                if name != "grad":
                    other.add(i)
            code = known.get(t.dtype, -1)
            if code not in types:
                raise ValueError(f"{name}[{i}] has type {t.dtype}")
            codes.append(code)
        return codes

    def _check_order(self, name: str, i: int, t) -> None:
        """A tensor some array of which is not contiguous: dense, and every array of it in the
        same order."""
        n = 1
        for size, stride in sorted(zip(t.shape, t.stride()), key=lambda x: x[1]):
            if size > 1 and stride != n:
                raise ValueError(f"{name}[{i}] is not contiguous, nor dense in another order")
            n *= size
        for k, xs in self.tensors.items():
            if k != "exps" and (name == "exps" or _order(xs[i]) != _order(t)):
                raise ValueError(f"{name}[{i}] and {k}[{i}] differ in order")

    def set_grad(self, grad: Sequence) -> None:
        """The same tensors' gradients at new addresses, in the order of the other arrays."""
        grad = list(grad)
        if len(grad) != len(self):
            raise ValueError(f"grad has {len(grad)} tensors, the list {len(self)}")
        old = self.tensors.get("grad")
        self.tensors["grad"] = grad
        try:
            codes = self._check("grad", grad)
        except BaseException:  # the addresses in use stay those of tensors that are kept
            self.tensors["grad"] = old
            if old is None:
                del self.tensors["grad"]
            raise
        for a, g, code in zip(self.array, grad, codes):
            a.grad, a.grad_dtype = g.data_ptr(), code


_TORCH_C = None


def _list_stream(tensors: TensorList, stream) -> int | None:
    """The stream of a call on a list: by default the current one, of the list's device."""
    global _TORCH_C
    if stream is not None:
        return _stream(stream)
    if _TORCH_C is None:
        import torch
        torch.cuda.current_device()  # CUDA is initialised from here on
        _TORCH_C = torch._C
    current = _TORCH_C._cuda_getDevice()
    if tensors.device not in (current, -1):
        raise ValueError(f"the list is on device {tensors.device}, the current device is {current}")
    return _TORCH_C._cuda_getCurrentRawStream(current)


def _alike(a: TensorList, b: TensorList) -> int:
    """The length of two lists whose states lie alike."""
    if len(a.elems) != len(b.elems):
        raise ValueError(f"lists of {len(a)} and {len(b)} tensors")
    if a.device != b.device:
        raise ValueError(f"lists of devices {a.device} and {b.device}")
    if a._other_order or b._other_order:
        for i in a._other_order | b._other_order:
            if "m" in a.tensors and "m" in b.tensors and _order(a.tensors["m"][i]) != _order(b.tensors["m"][i]):
                raise ValueError(f"the lists' m[{i}] differ in order")
    return len(a.elems)


def zero_tensors_workspace_bytes(n_tensors: int) -> int:
    return _lib().zero_tensors_workspace_bytes(n_tensors)


def zero_tensors_state_init(n_ranks: int, loss_scale: float, dynamic: bool, growth_interval: int, st,
                            stream=None) -> None:
    """n_ranks: how many copies the gradients are sums of (1: already averaged)."""
    _check("zero_tensors_state_init", _lib().zero_tensors_state_init(
        n_ranks, loss_scale, int(bool(dynamic)), growth_interval, _ptr(st), _stream(stream)))


def zero_tensors_grad_norm(tensors: TensorList, hp: HParams, workspace, st, stream=None) -> None:
    """Norm, clip coefficient, skip decision and the step's scalars over the list's gradients
    (of this list alone: a rank's shard has its own norm, not the run's).
    workspace: of zero_tensors_workspace_bytes(len(tensors)) bytes; a tensor that is smaller is
    refused (ZERO_ENOMEM), the size behind a plain address is the caller's word."""
    need = tensors._work_bytes
    if need is None:
        need = tensors._work_bytes = zero_tensors_workspace_bytes(len(tensors.elems))
    if getattr(workspace, "nbytes", need) < need:
        raise ZeroError("zero_tensors_grad_norm", ZERO_ENOMEM)
    status = _lib().zero_tensors_grad_norm(tensors.array, len(tensors.elems), C.byref(hp), _ptr(workspace),
                                           _ptr(st), _list_stream(tensors, stream))
    if status:
        _check("zero_tensors_grad_norm", status)


def zero_tensors_adamw(tensors: TensorList, hp: HParams, st, stream=None) -> None:
    """AdamW over the list, fp32 states."""
    if tensors._hp_decay is not None and tensors._hp_decay != hp.weight_decay:
        tensors._take_decay(hp.weight_decay)
    status = _lib().zero_tensors_adamw(tensors.array, len(tensors.elems), C.byref(hp), _ptr(st),
                                       _list_stream(tensors, stream))
    if status:
        _check("zero_tensors_adamw", status)


def zero_tensors_adamw8(tensors: TensorList, hp: HParams, seed: int, st, stream=None) -> None:
    """AdamW over the list, 8-bit states; seed: of their stochastic rounding."""
    if tensors._hp_decay is not None and tensors._hp_decay != hp.weight_decay:
        tensors._take_decay(hp.weight_decay)
    status = _lib().zero_tensors_adamw8(tensors.array, len(tensors.elems), C.byref(hp), seed, _ptr(st),
                                        _list_stream(tensors, stream))
    if status:
        _check("zero_tensors_adamw8", status)


def zero_tensors_state8_read(source: TensorList, to: TensorList, stream=None) -> None:
    """The values of source's 8-bit states into to's fp32 or bf16 m and v, which lie in the
    same order."""
    status = _lib().zero_tensors_state8_read(source.array, to.array, _alike(source, to),
                                             _list_stream(source, stream))
    if status:
        _check("zero_tensors_state8_read", status)


def zero_tensors_state8_write(to: TensorList, source: TensorList, stream=None) -> None:
    """source's fp32 m and v into to's 8-bit states, to the nearest code; both lie in the same
    order."""
    status = _lib().zero_tensors_state8_write(to.array, source.array, _alike(to, source),
                                              _list_stream(to, stream))
    if status:
        _check("zero_tensors_state8_write", status)


# --------------------------------------------------------------------------------------
# beside the matrix products
# --------------------------------------------------------------------------------------
_FLOATS = (ZERO_F16, ZERO_BF16, ZERO_F32)


def _current() -> int:
    """The current device."""
    global _TORCH_C
    if _TORCH_C is None:
        import torch
        torch.cuda.current_device()  # CUDA is initialised from here on
        _TORCH_C = torch._C
    if not _CODES:
        _dtype_codes()
    return _TORCH_C._cuda_getDevice()


def _here(stream, device: int) -> int | None:
    return _TORCH_C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _type_of(name: str, t, device: int, types=None) -> int:
    """The type code of a CUDA tensor of the current device."""
    if t.get_device() != device:
        raise ValueError(f"{name} is not a CUDA tensor of the current device, {device}")
    code = _CODES.get(t.dtype, -1)
    if types is not None and code not in types:
        raise ValueError(f"{name} has type {t.dtype}")
    return code


def _rows(name: str, t, dim: int, device: int, types) -> tuple:
    """Type code, number of rows and their stride: the last dimension holds a row, the others
    count rows at one distance from each other."""
    code = _type_of(name, t, device, types)
    shape = t.shape
    if not shape or not dim or shape[-1] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, not rows of {dim}")
    if t.is_contiguous():
        return code, t.numel() // dim, dim
    n, stride = 1, 0
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s rows are not contiguous")
    for size, step in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if n > 1 and step != n * stride:
            raise ValueError(f"{name}'s rows are not at one distance from each other")
        stride = stride if n > 1 else step
        n *= size
    if stride < dim and n > 1:
        raise ValueError(f"{name}'s rows overlap")
    return code, n, stride if n > 1 else dim


def _whole(name: str, t, shape: tuple, device: int, types) -> int:
    """The type code of a contiguous tensor of the given shape."""
    code = _type_of(name, t, device, types)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return code


def _per_row(name: str, t, n: int, device: int) -> int:
    """The address of fp32 numbers, one per row, in any shape."""
    _type_of(name, t, device, (ZERO_F32,))
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, not {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t.data_ptr()


def _ids(name: str, t, device: int, n: int | None = None) -> tuple:
    """How many ids, and their bytes: int32 or int64."""
    _type_of(name, t, device)
    size = _ID_BYTES.get(t.dtype)
    if size is None:
        raise ValueError(f"{name} has type {t.dtype}, not int32 or int64")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    count = t.numel()
    if n is not None and count != n:
        raise ValueError(f"{name} has {count} elements, not {n}")
    return count, size


def _space(fn: str, t, need: int, device: int) -> int:
    """A workspace's address: a tensor that is smaller than needed is refused, the size behind a
    plain address is the caller's word."""
    if isinstance(t, int):
        return t
    _type_of("workspace", t, device)
    if not t.is_contiguous():
        raise ValueError("workspace is not contiguous")
    if t.nbytes < need:
        raise ZeroError(fn, ZERO_ENOMEM)
    return t.data_ptr()


def zero_layernorm_workspace_bytes(rows: int, dim: int) -> int:
    return _lib().zero_layernorm_workspace_bytes(rows, dim)


def zero_layernorm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias over x's last dimension.  x, y: fp16, bf16 or fp32;
    weight, bias (or None): x's type or fp32; mean, rstd: fp32 per row, kept for the backward
    pass, or None."""
    device, dim = _current(), weight.numel()
    code, n, xs = _rows("x", x, dim, device, _FLOATS)
    param = _whole("weight", weight, (dim,), device, (code, ZERO_F32))
    if bias is not None:
        _whole("bias", bias, (dim,), device, (param,))
    _, ny, ys = _rows("y", y, dim, device, (code,))
    if ny != n:
        raise ValueError(f"x has {n} rows, y {ny}")
    status = _lib().zero_layernorm(
        code, n, dim, x.data_ptr(), xs, weight.data_ptr(), _ptr(bias), param, eps, y.data_ptr(), ys,
        None if mean is None else _per_row("mean", mean, n, device),
        None if rstd is None else _per_row("rstd", rstd, n, device), _here(stream, device))
    if status:
        _check("zero_layernorm", status)


def zero_layernorm_backward(x, weight, mean, rstd, dy, dx, dweight, dbias, workspace, accumulate: bool = False,
                            stream=None) -> None:
    """The gradients of zero_layernorm.  dy, dx: x's type; dweight, dbias: x's type or fp32, either
    may be None; accumulate: they are added to.  workspace: of
    zero_layernorm_workspace_bytes(rows, dim) bytes."""
    device, dim, fn = _current(), weight.numel(), "zero_layernorm_backward"
    code, n, xs = _rows("x", x, dim, device, _FLOATS)
    param = _whole("weight", weight, (dim,), device, (code, ZERO_F32))
    _, nd, ds = _rows("dy", dy, dim, device, (code,))
    _, ng, gs = _rows("dx", dx, dim, device, (code,))
    if nd != n or ng != n:
        raise ValueError(f"x has {n} rows, dy {nd}, dx {ng}")
    grad = code
    if dweight is not None:
        grad = _whole("dweight", dweight, (dim,), device, (code, ZERO_F32))
    if dbias is not None:
        grad = _whole("dbias", dbias, (dim,), device, (code, ZERO_F32) if dweight is None else (grad,))
    f = _lib().zero_layernorm_backward
    status = f(code, n, dim, x.data_ptr(), xs, weight.data_ptr(), param, _per_row("mean", mean, n, device),
               _per_row("rstd", rstd, n, device), dy.data_ptr(), ds, dx.data_ptr(), gs, _ptr(dweight), _ptr(dbias), grad,
               bool(accumulate), _space(fn, workspace, zero_layernorm_workspace_bytes(n, dim), device),
               _here(stream, device))
    if status:
        _check(fn, status)


def zero_embedding_workspace_bytes(n_tokens: int, dim: int, vocab: int) -> int:
    return _lib().zero_embedding_workspace_bytes(n_tokens, dim, vocab)


def _table(name: str, t) -> tuple:
    """(vocab, dim)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} has shape {tuple(shape)}")
    return shape


def zero_embedding(tokens, table, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[tokens[t]], zeros for ids outside the table.  tokens: int32 or int64;
    table [vocab, dim] and out [..., dim]: fp16, bf16 or fp32, alike."""
    device, (vocab, dim) = _current(), _table("table", table)
    n, size = _ids("tokens", tokens, device)
    code = _whole("table", table, (vocab, dim), device, _FLOATS)
    _, no, stride = _rows("out", out, dim, device, (code,))
    if no != n:
        raise ValueError(f"{n} tokens, out has {no} rows")
    status = _lib().zero_embedding(code, n, dim, vocab, tokens.data_ptr(), size, table.data_ptr(), scale, out.data_ptr(),
                                   stride, _here(stream, device))
    if status:
        _check("zero_embedding", status)


def zero_embedding_backward(tokens, dout, dtable, workspace, scale: float = 1.0, accumulate: bool = False,
                            stream=None) -> None:
    """The table's gradient: each row the sum of dout over its tokens' places, times scale.
    dtable: dout's type or fp32; accumulate: it is added to (rows without a token are not
    touched), else all of it is written.  workspace: of
    zero_embedding_workspace_bytes(n_tokens, dim, vocab) bytes."""
    device, (vocab, dim), fn = _current(), _table("dtable", dtable), "zero_embedding_backward"
    n, size = _ids("tokens", tokens, device)
    code, nd, stride = _rows("dout", dout, dim, device, _FLOATS)
    if nd != n:
        raise ValueError(f"{n} tokens, dout has {nd} rows")
    grad = _whole("dtable", dtable, (vocab, dim), device, (code, ZERO_F32))
    f = _lib().zero_embedding_backward
    status = f(code, n, dim, vocab, tokens.data_ptr(), size, dout.data_ptr(), stride, scale, dtable.data_ptr(), grad,
               bool(accumulate), _space(fn, workspace, zero_embedding_workspace_bytes(n, dim, vocab), device),
               _here(stream, device))
    if status:
        _check(fn, status)


def zero_head_workspace_bytes(rows: int, dim: int, vocab: int) -> int:
    return _lib().zero_head_workspace_bytes(rows, dim, vocab)


def _head(hidden, weight, targets, device: int) -> tuple:
    """What both of the head's calls check: (type code, rows, dim, vocab), row stride, bytes per
    target."""
    vocab, dim = _table("weight", weight)
    code, n, stride = _rows("hidden", hidden, dim, device, (ZERO_F16, ZERO_BF16))
    _whole("weight", weight, (vocab, dim), device, (code,))
    return (code, n, dim, vocab), stride, _ids("targets", targets, device, n)[1]


def zero_head_loss(hidden, weight, targets, loss, lse, workspace, stream=None) -> None:
    """The cross entropy of every token and its logits' log-sum-exp, from hidden [..., dim] and
    weight [vocab, dim] (fp16 or bf16); the logits are never kept.  Tokens whose target lies outside
    [0, vocab) get 0.  workspace: of zero_head_workspace_bytes(rows, dim, vocab) bytes.  Should a bounded
    wait inside give up, the losses are NaN."""
    device, fn = _current(), "zero_head_loss"
    sizes, stride, width = _head(hidden, weight, targets, device)
    n = sizes[1]
    status = _lib().zero_head_loss(*sizes, hidden.data_ptr(), stride, weight.data_ptr(), targets.data_ptr(), width,
                                   _per_row("loss", loss, n, device), _per_row("lse", lse, n, device),
                                   _space(fn, workspace, zero_head_workspace_bytes(*sizes[1:]), device),
                                   _here(stream, device))
    if status:
        _check(fn, status)


def zero_head_loss_backward(hidden, weight, targets, lse, dhidden, dweight, workspace, scale: float = 1.0,
                            row_scale=None, st=None, accumulate: bool = False, stream=None) -> None:
    """The gradients of sum over tokens of scale * row_scale * loss, times the loss scale that the
    step state st holds (None: 1).  dhidden: hidden's type, or None; dweight: that or fp32, or
    None; accumulate: dweight is added to.  Should a bounded wait inside give up, dhidden and what was
    not formed of dweight are NaN, and st's error word is 1."""
    device, fn = _current(), "zero_head_loss_backward"
    sizes, stride, width = _head(hidden, weight, targets, device)
    code, n, dim, vocab = sizes
    row = None if row_scale is None else _per_row("row_scale", row_scale, n, device)
    hs, grad = dim, code
    if dhidden is not None:
        _, nh, hs = _rows("dhidden", dhidden, dim, device, (code,))
        if nh != n:
            raise ValueError(f"hidden has {n} rows, dhidden {nh}")
    if dweight is not None:
        grad = _whole("dweight", dweight, (vocab, dim), device, (code, ZERO_F32))
    if st is not None and not isinstance(st, int):
        _type_of("st", st, device)
        if st.nbytes < STATE_BYTES:
            raise ValueError(f"st has {st.nbytes} bytes, not {STATE_BYTES}")
    f = _lib().zero_head_loss_backward
    status = f(*sizes, hidden.data_ptr(), stride, weight.data_ptr(), targets.data_ptr(), width,
               _per_row("lse", lse, n, device), scale, row, _ptr(st), _ptr(dhidden), hs, _ptr(dweight), grad,
               bool(accumulate), _space(fn, workspace, zero_head_workspace_bytes(*sizes[1:]), device),
               _here(stream, device))
    if status:
        _check(fn, status)


__all__ = [
    "Layout", "HParams", "StepState", "ZeroError", "hparams", "lib", "STATE_BYTES",
    "ZERO_F16", "ZERO_BF16", "Segment", "zero_partition", "zero_segment_map", "zero_workspace_bytes", "zero_step_state_init",
    "zero_step_state_read", "zero_step_state_write", "zero_reduce_shard_unscale",
    "zero_grad_norm", "zero_adamw_cast_gather", "zero_adamw_cast_gather_host_state", "zero_step",
    "zero_step_host", "zero_step_launches", "zero_reduce_shard_unscale_local",
    "zero_adamw_cast_gather_local", "zero_step_static_workspace",
    "ZERO_F32", "ZERO_U8", "ZERO_STATE8_BLOCK", "Tensor", "TensorList", "zero_tensors_workspace_bytes",
    "zero_tensors_state_init", "zero_tensors_grad_norm", "zero_tensors_adamw", "zero_tensors_adamw8",
    "zero_tensors_state8_read", "zero_tensors_state8_write",
    "zero_layernorm", "zero_layernorm_backward", "zero_layernorm_workspace_bytes", "zero_embedding",
    "zero_embedding_backward", "zero_embedding_workspace_bytes", "zero_head_loss", "zero_head_loss_backward",
    "zero_head_workspace_bytes",
]
