"""Python binding of libzeroshard.so (include/zero_shard.h), via ctypes.

Argument marshalling only: tensors are checked for dtype, device and
contiguity and passed as raw device pointers together with torch's current
HIP stream; every step of the shard update runs in the library's kernels.
Importing this module loads the library and fails loudly if it is missing or
was not built for this tree; there is no fallback path.

torch is imported first so that the library binds to the HIP runtime torch
already loaded (both name the same soname, libamdhip64.so.7).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple, Optional, Sequence, Tuple

import torch  # noqa: F401  (loads the HIP runtime the library binds to)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzeroshard.so")

ZERO_OK = 0
ZERO_EINVAL = -1
ZERO_EOVERFLOW = -2
ZERO_EHIP = -3
ZERO_ENOMEM = -4
ZERO_ENOTSUP = -5
ZERO_ERANGE = -6
ZERO_NOALLOC_SCRATCH_BYTES = 8 << 20
ZERO_NOALLOC_MAX_TENSORS = 1024
ZERO_MAX_SLICES = 256
ZERO_FUSED_SPLIT_SLICES = 16
ZERO_LOG2_SCALE_MAX = 100
ZERO_F16 = 0
ZERO_BF16 = 1
ZERO_F32 = 2
ZERO_DISTILL_MAX_TOP = 1024


class ZeroError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({zero_status_str(status)})")
        self.status = status


class _Layout(ctypes.Structure):
    _fields_ = [("padded_total", ctypes.c_uint64), ("shard_len", ctypes.c_uint64),
                ("offset", ctypes.c_uint64), ("real_len", ctypes.c_uint64)]


class _Comm(ctypes.Structure):
    _fields_ = [("passes", ctypes.c_uint64), ("volume_elems", ctypes.c_uint64),
                ("ring_send_elems", ctypes.c_uint64)]


class _Tensor(ctypes.Structure):
    _fields_ = [("param_f16", ctypes.c_void_p), ("grad_f16", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("n", ctypes.c_uint64)]


class _HParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double)]


class _OffloadInfo(ctypes.Structure):
    _fields_ = [("threads", ctypes.c_uint32), ("numa_node", ctypes.c_int32),
                ("pinned_cpus", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("chunk_elems", ctypes.c_uint64)]


class _Stats(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in (
        "n_tensors", "n_params", "n_chunks", "chunk_elems", "vector_elems",
        "scalar_elems", "table_bytes", "tile_elems", "wg_per_cu")]


class _MXFP4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64),
                ("ld_codes", ctypes.c_uint64), ("ld_scales", ctypes.c_uint64)]


class _Distill(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64),
                ("logits", ctypes.c_void_p), ("ld_logits", ctypes.c_uint64),
                ("grad", ctypes.c_void_p), ("ld_grad", ctypes.c_uint64),
                ("loss", ctypes.c_void_p), ("top_idx", ctypes.c_void_p),
                ("top_logits", ctypes.c_void_p), ("ld_idx", ctypes.c_uint64),
                ("ld_top", ctypes.c_uint64), ("teacher_lse", ctypes.c_void_p),
                ("labels", ctypes.c_void_p), ("row_weight", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("nonfinite_flag", ctypes.c_void_p),
                ("temperature", ctypes.c_double), ("soft_weight", ctypes.c_double),
                ("hard_weight", ctypes.c_double), ("top", ctypes.c_uint32),
                ("logits_type", ctypes.c_int32), ("top_type", ctypes.c_int32),
                ("idx_bytes", ctypes.c_int32), ("label_bytes", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    i32, u32, u64, vp = ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p
    sig = {
        "zero_shard_layout": [u64, u32, u32, u32, ctypes.POINTER(_Layout)],
        "zero_state_bytes": [u32, u64, u32, u32, ctypes.POINTER(ctypes.c_uint64)],
        "zero_comm_volume": [u32, u64, u32, u32, ctypes.POINTER(_Comm)],
        "zero_gather_shards": [ctypes.POINTER(vp), u32, u64, vp, vp],
        "zero_plan_create": [ctypes.POINTER(_Tensor), u32, u32, ctypes.POINTER(vp)],
        "zero_plan_create_bf16": [ctypes.POINTER(_Tensor), u32, u32, ctypes.POINTER(vp)],
        "zero_reduce_grad_shard_bf16": [ctypes.POINTER(vp), u32, u64, vp, vp, vp],
        "zero_plan_stats_of": [vp, ctypes.POINTER(_Stats)],
        "zero_plan_describe": [ctypes.POINTER(_Tensor), u32, u32, ctypes.POINTER(_Stats)],
        "zero_plan_destroy": [vp],
        "zero_adam_scalars": [ctypes.POINTER(_HParams), u64, ctypes.POINTER(ctypes.c_float)],
        "zero_adam_step": [vp, ctypes.POINTER(_HParams), u64, vp, vp, vp],
        "zero_adam_step_scaled": [vp, ctypes.POINTER(_HParams), u64, vp, vp, vp, vp],
        "zero_adam_step_noalloc": [ctypes.POINTER(_Tensor), u32, ctypes.POINTER(_HParams), u64,
                                   vp, vp, vp],
        "zero_loss_scale_update": [vp, vp, u32, ctypes.c_int32, ctypes.c_int32, vp],
        "zero_reduce_grad_shard": [ctypes.POINTER(vp), u32, u64, vp, vp, vp],
        "zero_reduce_adam_step": [ctypes.POINTER(vp), u32, u64, vp, vp, vp, vp, vp,
                                  ctypes.POINTER(_HParams), u64, vp, vp],
        "zero_reduce_adam_step_bf16": [ctypes.POINTER(vp), u32, u64, vp, vp, vp, vp, vp,
                                       ctypes.POINTER(_HParams), u64, vp, vp],
        "zero_adam_step_host": [vp, vp, vp, vp, vp, u64, ctypes.POINTER(_HParams), u64, u32, vp],
        "zero_adam_step_host_bf16": [vp, vp, vp, vp, vp, u64, ctypes.POINTER(_HParams), u64, u32,
                                     vp],
        "zero_offload_create": [u64, u32, ctypes.POINTER(vp)],
        "zero_offload_destroy": [vp],
        "zero_offload_describe": [vp, ctypes.POINTER(_OffloadInfo)],
        "zero_offload_step": [vp, vp, vp, vp, vp, vp, u64, ctypes.POINTER(_HParams), u64, vp, vp],
        "zero_offload_step_bf16": [vp, vp, vp, vp, vp, vp, u64, ctypes.POINTER(_HParams), u64, vp,
                                   vp],
        "zero_mxfp4_layout": [u64, u64, ctypes.POINTER(_MXFP4)],
        "zero_mxfp4_quantize": [vp, i32, u64, ctypes.POINTER(_MXFP4), vp, vp],
        "zero_mxfp4_dequantize": [ctypes.POINTER(_MXFP4), vp, i32, u64, vp],
        "zero_gather_shards_mxfp4": [ctypes.POINTER(vp), ctypes.POINTER(vp), u32, u64, vp, i32,
                                     vp],
        "zero_mxfp4_matmul": [ctypes.POINTER(_MXFP4), ctypes.POINTER(_MXFP4), vp, i32, u64, vp],
        "zero_mxfp4_linear": [vp, i32, u64, u64, ctypes.POINTER(_MXFP4), vp, i32, u64, vp],
        "zero_mxfp4_linear_grad_input": [vp, i32, u64, u64, ctypes.POINTER(_MXFP4), vp, i32, u64,
                                         vp, u64, vp],
        "zero_mxfp4_grad_workspace": [u64, ctypes.POINTER(_MXFP4), ctypes.POINTER(u64)],
        "zero_distill_loss": [ctypes.POINTER(_Distill), vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = i32
    L.zero_status_str.argtypes = [i32]
    L.zero_status_str.restype = ctypes.c_char_p
    return L


_lib = _load()

# Every symbol include/zero_shard.h declares.
EXPORTS = ("zero_shard_layout", "zero_state_bytes", "zero_comm_volume",
           "zero_gather_shards", "zero_plan_create", "zero_plan_create_bf16",
           "zero_reduce_grad_shard_bf16",
           "zero_plan_stats_of", "zero_plan_describe", "zero_plan_destroy",
           "zero_adam_scalars", "zero_adam_step", "zero_reduce_grad_shard",
           "zero_reduce_adam_step", "zero_reduce_adam_step_bf16", "zero_adam_step_host",
           "zero_adam_step_host_bf16", "zero_offload_create", "zero_offload_step_bf16",
           "zero_offload_destroy", "zero_offload_describe", "zero_offload_step", "zero_status_str",
           "zero_adam_step_scaled", "zero_loss_scale_update", "zero_adam_step_noalloc",
           "zero_mxfp4_layout", "zero_mxfp4_quantize", "zero_mxfp4_dequantize",
           "zero_gather_shards_mxfp4", "zero_mxfp4_matmul", "zero_mxfp4_linear",
           "zero_mxfp4_linear_grad_input", "zero_mxfp4_grad_workspace", "zero_distill_loss")


def lib() -> ctypes.CDLL:
    return _lib


def zero_status_str(status: int) -> str:
    return _lib.zero_status_str(int(status)).decode()


def _check(fn: str, rc: int) -> None:
    if rc != ZERO_OK:
        raise ZeroError(fn, rc)


class Layout(NamedTuple):
    padded_total: int
    shard_len: int
    offset: int
    real_len: int


def zero_shard_layout(psi: int, nd: int, rank: int, align: int = 1) -> Layout:
    out = _Layout()
    _check("zero_shard_layout", _lib.zero_shard_layout(psi, nd, rank, align, ctypes.byref(out)))
    return Layout(out.padded_total, out.shard_len, out.offset, out.real_len)


def zero_state_bytes(stage: int, psi: int, nd: int, align: int = 1) -> int:
    out = ctypes.c_uint64()
    _check("zero_state_bytes", _lib.zero_state_bytes(stage, psi, nd, align, ctypes.byref(out)))
    return out.value


def zero_comm_volume(stage: int, psi: int, nd: int, align: int = 1) -> dict:
    """Elements one rank moves per step: {passes, volume_elems, ring_send_elems}."""
    out = _Comm()
    _check("zero_comm_volume", _lib.zero_comm_volume(stage, psi, nd, align, ctypes.byref(out)))
    return {k: getattr(out, k) for k, _ in _Comm._fields_}


@dataclass(frozen=True)
class AdamHParams:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.0

    def _c(self) -> _HParams:
        return _HParams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay)


def _hp(hp) -> _HParams:
    if isinstance(hp, dict):
        hp = AdamHParams(**hp)
    return hp._c()


def zero_adam_scalars(hp, t: int) -> Tuple[float, ...]:
    """{lr, b1, 1-b1, b2, 1-b2, 1-b1^t, 1-b2^t, eps} as the kernel uses them."""
    out = (ctypes.c_float * 8)()
    h = _hp(hp)
    _check("zero_adam_scalars", _lib.zero_adam_scalars(ctypes.byref(h), t, out))
    return tuple(out)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, what: str, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: expected a device (cuda/HIP) tensor, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _flag_ptr(flag: Optional[torch.Tensor], what: str, device) -> Optional[int]:
    if flag is None:
        return None
    _need(flag, torch.int32, what, device)
    if flag.numel() < 1:
        raise ValueError(f"{what}: needs one int32")
    return flag.data_ptr()


def _tensor_entries(tensors: Sequence[Sequence[torch.Tensor]], half=torch.float16):
    """half: the 16-bit dtype of every parameter and gradient (float16 or
    bfloat16)."""
    arr = (_Tensor * max(1, len(tensors)))()
    device = None
    for k, group in enumerate(tensors):
        if len(group) != 5:
            raise ValueError("each tensor is (param, grad, master, m, v)")
        p, g, w, m, v = group
        device = device or w.device
        for x, dt, nm in ((p, half, "param"), (g, half, "grad"),
                          (w, torch.float32, "master"), (m, torch.float32, "m"),
                          (v, torch.float32, "v")):
            _need(x, dt, f"tensor {k} {nm}", device)
        n = w.numel()
        if not (p.numel() == g.numel() == m.numel() == v.numel() == n):
            raise ValueError(f"tensor {k}: the five arrays differ in size")
        arr[k] = _Tensor(p.data_ptr(), g.data_ptr(), w.data_ptr(), m.data_ptr(),
                         v.data_ptr(), n)
    return arr, device


class Plan:
    """A zero_plan: the device chunk table over a list of tensors.  Holds
    references to the tensors so their memory outlives the plan."""

    def __init__(self, handle: int, tensors, device):
        self._h = handle
        self._keep = [tuple(g) for g in tensors]
        self.device = device

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("plan was destroyed")
        return self._h

    def stats(self) -> dict:
        s = _Stats()
        _check("zero_plan_stats_of", _lib.zero_plan_stats_of(self.handle, ctypes.byref(s)))
        return {k: getattr(s, k) for k, _ in _Stats._fields_}

    def destroy(self) -> None:
        if self._h:
            h, self._h = self._h, None
            _check("zero_plan_destroy", _lib.zero_plan_destroy(h))
            self._keep = []

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def zero_plan_create(tensors: Sequence[Sequence[torch.Tensor]], chunk_elems: int = 0) -> Plan:
    """tensors: sequence of (param, grad, master_f32, m_f32, v_f32) where
    every param and grad is float16 (the pages' ledger) or every one is
    bfloat16 (the bfloat16 variant).  chunk_elems: 0 for the library
    default, else a multiple of 512."""
    half = tensors[0][0].dtype if len(tensors) else torch.float16
    if half not in (torch.float16, torch.bfloat16):
        raise TypeError(f"param: expected torch.float16 or torch.bfloat16, got {half}")
    arr, device = _tensor_entries(tensors, half)
    fn = "zero_plan_create_bf16" if half == torch.bfloat16 else "zero_plan_create"
    h = ctypes.c_void_p()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(fn, getattr(_lib, fn)(arr, len(tensors), int(chunk_elems), ctypes.byref(h)))
    return Plan(h.value, tensors, device)


def zero_plan_describe(tensors, chunk_elems: int = 0) -> dict:
    """Classification of a would-be plan, computed on the host only.
    tensors: sequence of (param, grad, master, m, v, n) with integer
    addresses, or of torch tensors as for zero_plan_create."""
    arr = (_Tensor * max(1, len(tensors)))()
    for k, e in enumerate(tensors):
        if len(e) == 6:
            arr[k] = _Tensor(*e)
        else:
            a, _ = _tensor_entries([e])
            arr[k] = a[0]
    s = _Stats()
    _check("zero_plan_describe", _lib.zero_plan_describe(arr, len(tensors), int(chunk_elems),
                                                         ctypes.byref(s)))
    return {k: getattr(s, k) for k, _ in _Stats._fields_}


def zero_plan_destroy(plan: Plan) -> None:
    plan.destroy()


def zero_adam_step(plan: Plan, hp, t: int, nonfinite_flag: Optional[torch.Tensor] = None,
                   skip_if_nonzero: Optional[torch.Tensor] = None, stream=None,
                   loss_scale: Optional["LossScale"] = None) -> None:
    """Enqueue one Adam step over the plan on `stream` (torch's current stream
    by default).  With `loss_scale`, the gradients carry its factor 2^k and
    are multiplied by 2^-k first (zero_adam_step_scaled)."""
    h = _hp(hp)
    f = _flag_ptr(nonfinite_flag, "nonfinite_flag", plan.device)
    s = _flag_ptr(skip_if_nonzero, "skip_if_nonzero", plan.device)
    if loss_scale is None:
        _check("zero_adam_step", _lib.zero_adam_step(plan.handle, ctypes.byref(h), int(t), f, s,
                                                     _stream_handle(stream)))
        return
    if loss_scale.state.device != plan.device:
        raise ValueError(f"loss_scale: on {loss_scale.state.device}, expected {plan.device}")
    _check("zero_adam_step_scaled",
           _lib.zero_adam_step_scaled(plan.handle, ctypes.byref(h), int(t),
                                      loss_scale.state.data_ptr(), f, s, _stream_handle(stream)))


def zero_adam_step_noalloc(tensors: Sequence[Sequence[torch.Tensor]], hp, t: int,
                           nonfinite_flag: Optional[torch.Tensor] = None,
                           skip_if_nonzero: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue one Adam step over float16 tensors (param, grad, master, m, v)
    without a plan: the library rebuilds the chunk table in its fixed
    per-device array and allocates nothing.  Calls that may overlap on one
    device race for that array."""
    arr, device = _tensor_entries(tensors, torch.float16)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    h = _hp(hp)
    f = _flag_ptr(nonfinite_flag, "nonfinite_flag", device)
    s = _flag_ptr(skip_if_nonzero, "skip_if_nonzero", device)
    with torch.cuda.device(device):
        _check("zero_adam_step_noalloc",
               _lib.zero_adam_step_noalloc(arr, len(tensors), ctypes.byref(h), int(t), f, s,
                                           _stream_handle(stream)))


class LossScale:
    """A dynamic loss scale 2^k held on the device as the four int32 of
    zero_loss_scale: (log2_scale, good_steps, skipped_steps, applied_steps).

    One step: zero_reduce_grad_shard(..., flag); zero_adam_step(plan, hp, t,
    skip_if_nonzero=flag, loss_scale=ls); ls.update(flag) -- which halves the
    scale after a non-finite gradient, doubles it after `interval` finite
    steps in a row, and clears the flag."""

    def __init__(self, log2_scale: int = 16, interval: int = 2000, min_log2: int = 0,
                 max_log2: int = 24, device=None):
        if not -ZERO_LOG2_SCALE_MAX <= min_log2 <= max_log2 <= ZERO_LOG2_SCALE_MAX:
            raise ValueError("need -100 <= min_log2 <= max_log2 <= 100")
        if interval < 1:
            raise ValueError("interval must be >= 1")
        self.interval, self.min_log2, self.max_log2 = int(interval), int(min_log2), int(max_log2)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.state = torch.tensor([int(log2_scale), 0, 0, 0], dtype=torch.int32, device=device)

    def update(self, nonfinite_flag: torch.Tensor, stream=None) -> None:
        """Enqueue the scale's update from the step's flag (then set to 0)."""
        f = _flag_ptr(nonfinite_flag, "nonfinite_flag", self.state.device)
        _check("zero_loss_scale_update",
               _lib.zero_loss_scale_update(self.state.data_ptr(), f, self.interval,
                                           self.min_log2, self.max_log2, _stream_handle(stream)))

    def read(self) -> tuple:
        """(log2_scale, good_steps, skipped_steps, applied_steps); waits for
        the device."""
        v = self.state.cpu().tolist()
        return (v[0], v[1] & 0xFFFFFFFF, v[2] & 0xFFFFFFFF, v[3] & 0xFFFFFFFF)


def zero_reduce_grad_shard(slices: Sequence[torch.Tensor], out: torch.Tensor,
                           nonfinite_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = mean over ranks of the slices, fp32 sum in rank order, rounded
    to out's format: float16, or bfloat16 (the bfloat16 variant)."""
    half = out.dtype if out.dtype in (torch.float16, torch.bfloat16) else torch.float16
    _need(out, half, "out")
    n = out.numel()
    nd = len(slices)
    if nd == 0 or nd > ZERO_MAX_SLICES:
        raise ValueError(f"need 1..{ZERO_MAX_SLICES} slices, got {nd}")
    ptrs = (ctypes.c_void_p * nd)()
    for r, s in enumerate(slices):
        _need(s, half, f"slice {r}", out.device)
        if s.numel() != n:
            raise ValueError(f"slice {r} has {s.numel()} elements, out has {n}")
        ptrs[r] = s.data_ptr()
    f = _flag_ptr(nonfinite_flag, "nonfinite_flag", out.device)
    fn = "zero_reduce_grad_shard_bf16" if half == torch.bfloat16 else "zero_reduce_grad_shard"
    _check(fn, getattr(_lib, fn)(ptrs, nd, n, out.data_ptr(), f, _stream_handle(stream)))


def zero_reduce_adam_step(slices: Sequence[torch.Tensor], param: torch.Tensor,
                          master: torch.Tensor, m: torch.Tensor, v: torch.Tensor, hp, t: int,
                          grad_out: Optional[torch.Tensor] = None,
                          nonfinite_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Reduce the 16-bit slices and apply the Adam step in one pass over a
    flat shard (bit-identical to zero_reduce_grad_shard then
    zero_adam_step).  param, the slices and grad_out are all float16 or all
    bfloat16 (the bfloat16 variant)."""
    _need(master, torch.float32, "master")
    dev = master.device
    n = master.numel()
    half = param.dtype if param.dtype in (torch.float16, torch.bfloat16) else torch.float16
    for x, dt, nm in ((param, half, "param"), (m, torch.float32, "m"),
                      (v, torch.float32, "v")):
        _need(x, dt, nm, dev)
        if x.numel() != n:
            raise ValueError(f"{nm} has {x.numel()} elements, master has {n}")
    nd = len(slices)
    if nd == 0 or nd > ZERO_MAX_SLICES:
        raise ValueError(f"need 1..{ZERO_MAX_SLICES} slices, got {nd}")
    ptrs = (ctypes.c_void_p * nd)()
    for r, s in enumerate(slices):
        _need(s, half, f"slice {r}", dev)
        if s.numel() != n:
            raise ValueError(f"slice {r} has {s.numel()} elements, master has {n}")
        ptrs[r] = s.data_ptr()
    go = None
    if grad_out is not None:
        _need(grad_out, half, "grad_out", dev)
        if grad_out.numel() != n:
            raise ValueError(f"grad_out has {grad_out.numel()} elements, master has {n}")
        go = grad_out.data_ptr()
    h = _hp(hp)
    f = _flag_ptr(nonfinite_flag, "nonfinite_flag", dev)
    name = "zero_reduce_adam_step_bf16" if half == torch.bfloat16 else "zero_reduce_adam_step"
    _check(name, getattr(_lib, name)(ptrs, nd, n, param.data_ptr(), master.data_ptr(),
                                     m.data_ptr(), v.data_ptr(), go, ctypes.byref(h), int(t), f,
                                     _stream_handle(stream)))


def zero_gather_shards(shards: Sequence[torch.Tensor], full: torch.Tensor, stream=None) -> None:
    """full[r * S:(r + 1) * S] = shards[r] for every rank r (fp16); shards
    that are already views at their place in full are left alone."""
    _need(full, torch.float16, "full")
    nd = len(shards)
    if nd == 0 or nd > ZERO_MAX_SLICES:
        raise ValueError(f"need 1..{ZERO_MAX_SLICES} shards, got {nd}")
    S = shards[0].numel()
    if full.numel() != nd * S:
        raise ValueError(f"full has {full.numel()} elements, {nd} shards of {S} need {nd * S}")
    ptrs = (ctypes.c_void_p * nd)()
    for r, s in enumerate(shards):
        _need(s, torch.float16, f"shard {r}", full.device)
        if s.numel() != S:
            raise ValueError(f"shard {r} has {s.numel()} elements, shard 0 has {S}")
        ptrs[r] = s.data_ptr()
    _check("zero_gather_shards",
           _lib.zero_gather_shards(ptrs, nd, S, full.data_ptr(), _stream_handle(stream)))


def _host(a, dtype, what: str, n: Optional[int] = None) -> int:
    """Address of a contiguous host numpy array of the given element type."""
    import numpy as np
    if not isinstance(a, np.ndarray):
        raise TypeError(f"{what}: expected a numpy array")
    if a.dtype.itemsize != np.dtype(dtype).itemsize or a.dtype.kind != np.dtype(dtype).kind:
        if not (np.dtype(dtype) == np.uint16 and a.dtype == np.float16):
            raise TypeError(f"{what}: expected {np.dtype(dtype)}, got {a.dtype}")
    if not a.flags["C_CONTIGUOUS"]:
        raise ValueError(f"{what}: must be contiguous")
    if n is not None and a.size != n:
        raise ValueError(f"{what}: has {a.size} elements, expected {n}")
    return a.ctypes.data


def zero_adam_step_host(grad16, param16, master, m, v, hp, t: int, threads: int = 0,
                        nonfinite_flag=None, fmt: str = "f16") -> None:
    """The Adam step on the host CPU over numpy arrays (16-bit values as
    uint16, or float16 for fmt "f16"; fp32 state updated in place);
    bit-identical to zero_adam_step.  fmt: "f16", or "bf16" for the
    bfloat16 variant (gradient and parameter as bfloat16 bit patterns)."""
    if fmt not in ("f16", "bf16"):
        raise ValueError('fmt must be "f16" or "bf16"')
    import numpy as np
    n = master.size
    ptrs = [_host(grad16, np.uint16, "grad", n), _host(param16, np.uint16, "param", n),
            _host(master, np.float32, "master", n), _host(m, np.float32, "m", n),
            _host(v, np.float32, "v", n)]
    f = None if nonfinite_flag is None else _host(nonfinite_flag, np.int32, "nonfinite_flag", 1)
    h = _hp(hp)
    name = "zero_adam_step_host_bf16" if fmt == "bf16" else "zero_adam_step_host"
    _check(name, getattr(_lib, name)(*ptrs, n, ctypes.byref(h), int(t), int(threads), f))


class Offload:
    """A zero_offload pipeline (pinned staging, copy streams, host threads)."""

    def __init__(self, handle: int, device):
        self._h = handle
        self.device = device

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("offload was destroyed")
        return self._h

    def step(self, grad: torch.Tensor, param: torch.Tensor, master, m, v, hp, t: int,
             nonfinite_flag=None, stream=None) -> None:
        """grad, param: device tensors, both float16 or both bfloat16 (the
        bfloat16 variant); master, m, v: host numpy fp32 arrays updated in
        place; nonfinite_flag: None or a numpy int32[1]."""
        import numpy as np
        n = master.size
        half = grad.dtype if grad.dtype in (torch.float16, torch.bfloat16) else torch.float16
        _need(grad, half, "grad", self.device)
        _need(param, half, "param", self.device)
        if grad.numel() != n or param.numel() != n:
            raise ValueError("grad, param and the host state differ in size")
        hs = [_host(master, np.float32, "master", n), _host(m, np.float32, "m", n),
              _host(v, np.float32, "v", n)]
        f = None if nonfinite_flag is None else _host(nonfinite_flag, np.int32, "nonfinite_flag", 1)
        h = _hp(hp)
        name = "zero_offload_step_bf16" if half == torch.bfloat16 else "zero_offload_step"
        _check(name, getattr(_lib, name)(self.handle, grad.data_ptr(), param.data_ptr(), *hs, n,
                                         ctypes.byref(h), int(t), f, _stream_handle(stream)))

    def info(self) -> dict:
        """threads, numa_node (-1: unknown), pinned_cpus (0: not pinned),
        chunk_elems."""
        i = _OffloadInfo()
        _check("zero_offload_describe", _lib.zero_offload_describe(self.handle, ctypes.byref(i)))
        return {k: getattr(i, k) for k, _ in _OffloadInfo._fields_ if k != "reserved"}

    def destroy(self) -> None:
        if self._h:
            h, self._h = self._h, None
            _check("zero_offload_destroy", _lib.zero_offload_destroy(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def zero_offload_create(chunk_elems: int = 0, threads: int = 0) -> Offload:
    h = ctypes.c_void_p()
    _check("zero_offload_create", _lib.zero_offload_create(int(chunk_elems), int(threads),
                                                           ctypes.byref(h)))
    return Offload(h.value, torch.device("cuda", torch.cuda.current_device()))


# ---------------------------------------------------------------------------
# 4-bit parameters (MXFP4) and the distillation loss.
# ---------------------------------------------------------------------------
_TYPES = {torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32}
_HALF = {torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16}
_BYTES = {torch.uint8: 1}
_INTS = {torch.int32: 4, torch.int64: 8}

_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _launch(fn: str, index: int, stream, *args) -> None:
    """Call `fn` with device `index` current and the stream (torch's current
    stream of that device by default) as its last argument."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _launch(fn, index, stream, *args)
    rc = getattr(_lib, fn)(*args, _current_stream(index) if stream is None
                           else _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(fn, rc)


def _torch_stream(handle: int, device):
    """torch's stream of a handle.  Handle 0 is the default stream; torch takes
    an external 0 for none given and makes a stream of its own pool."""
    return torch.cuda.ExternalStream(handle, device) if handle else \
        torch.cuda.default_stream(device)


def _rows(t: torch.Tensor, what: str, types: dict, index: Optional[int] = None):
    """(pointer, types' entry, rows, cols, pitch) of a device tensor of one or
    two dimensions whose rows are contiguous; one dimension is a single row."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    ty = types.get(t.dtype)
    if ty is None:
        raise TypeError(f"{what}: expected one of {[str(d) for d in types]}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a device (cuda/HIP) tensor, got {t.device}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{what}: on {t.device}, expected device {index}")
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        rows, cols = shape
        ld, step = strides
    elif len(shape) == 1:
        rows, cols, ld, step = 1, shape[0], 0, strides[0]
    else:
        raise ValueError(f"{what}: expected one or two dimensions, got {len(shape)}")
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{what}: rows overlap (row stride {ld}, {cols} columns)")
    return t.data_ptr(), ty, rows, cols, ld


def _flat(t: torch.Tensor, what: str, types: dict, n: int, index: int):
    """(pointer, types' entry) of a contiguous device tensor of n elements."""
    if not isinstance(t, torch.Tensor) or t.dtype not in types:
        raise TypeError(f"{what}: expected a torch.Tensor of one of {[str(d) for d in types]}")
    if t.get_device() != index:
        raise ValueError(f"{what}: on {t.device}, expected device {index}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements, got {tuple(t.shape)}")
    return t.data_ptr(), types[t.dtype]


def _flag(flag: Optional[torch.Tensor], index: int) -> Optional[int]:
    if flag is None:
        return None
    if isinstance(flag, torch.Tensor) and flag.get_device() != index:
        raise ValueError(f"nonfinite_flag: on {flag.device}, expected device {index}")
    return _flag_ptr(flag, "nonfinite_flag", None)


class MXFP4:
    """A rows x cols matrix in 4 bits per value with one scale byte per 32
    columns (zero_mxfp4): `codes` uint8 [rows, >= 16 * blocks] and `scales`
    uint8 [rows, >= blocks], blocks = ceil(cols / 32), rows contiguous.  Code
    rows start at 16-byte boundaries; codes past cols are 0."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        cp, _, rows, cb, ldc = _rows(codes, "codes", _BYTES)
        self.index = codes.get_device()
        sp, _, srows, sb, lds = _rows(scales, "scales", _BYTES, self.index)
        blocks = (int(cols) + 31) // 32
        if cols < 0 or srows != rows or cb < 16 * blocks or sb < blocks:
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                             f"hold rows of {cols} columns ({blocks} blocks)")
        if rows <= 1 or blocks == 0:  # the pitch is not used
            ldc, lds = 16 * blocks, blocks
        if ldc % 16 or cp % 16:
            raise ValueError("codes: rows must start at 16-byte boundaries")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, int(cols)
        self._c = _MXFP4(cp, sp, rows, self.cols, ldc, lds)
        self._ref = ctypes.byref(self._c)

    @property
    def device(self):
        return self.codes.device

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "MXFP4":
        """A dense matrix of uninitialised storage."""
        lay = _MXFP4()
        _check("zero_mxfp4_layout", _lib.zero_mxfp4_layout(int(rows), int(cols),
                                                           ctypes.byref(lay)))
        return MXFP4(torch.empty(rows, lay.ld_codes, dtype=torch.uint8, device=device),
                     torch.empty(rows, lay.ld_scales, dtype=torch.uint8, device=device), cols)


def _mx(q: MXFP4, what: str, index: Optional[int] = None) -> MXFP4:
    if not isinstance(q, MXFP4):
        raise TypeError(f"{what}: expected an MXFP4")
    if index is not None and q.index != index:
        raise ValueError(f"{what}: on {q.device}, expected device {index}")
    return q


def _size(what: str, rows: int, cols: int, want_rows: int, want_cols: int) -> None:
    if rows != want_rows or cols != want_cols:
        raise ValueError(f"{what}: is {rows} x {cols}, expected {want_rows} x {want_cols}")


def zero_mxfp4_quantize(src: torch.Tensor, out: MXFP4,
                        nonfinite_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = src (float32, float16 or bfloat16; two dimensions, or one as a
    single row) in 4 bits with a power-of-two scale per 32 columns."""
    i = _mx(out, "out").index
    p, ty, rows, cols, ld = _rows(src, "src", _TYPES, i)
    _size("src", rows, cols, out.rows, out.cols)
    _launch("zero_mxfp4_quantize", i, stream, p, ty, ld, out._ref, _flag(nonfinite_flag, i))


def zero_mxfp4_dequantize(src: MXFP4, out: torch.Tensor, stream=None) -> None:
    """out (float32, float16 or bfloat16) = the values of src."""
    i = _mx(src, "src").index
    p, ty, rows, cols, ld = _rows(out, "out", _TYPES, i)
    _size("out", rows, cols, src.rows, src.cols)
    _launch("zero_mxfp4_dequantize", i, stream, src._ref, p, ty, ld)


def zero_gather_shards_mxfp4(shards: Sequence[MXFP4], full: torch.Tensor, stream=None) -> None:
    """full[r * S:(r + 1) * S] = the values of shards[r], each a single row
    of S elements (a multiple of 32), for every rank r."""
    nd = len(shards)
    if nd == 0 or nd > ZERO_MAX_SLICES:
        raise ValueError(f"need 1..{ZERO_MAX_SLICES} shards, got {nd}")
    i, S = _mx(shards[0], "shard 0").index, shards[0].cols
    for r, q in enumerate(shards):
        _mx(q, f"shard {r}", i)
        if q.rows != 1 or q.cols != S:
            _size(f"shard {r}", q.rows, q.cols, 1, S)
    p, ty = _flat(full, "full", _TYPES, nd * S, i)
    codes = (ctypes.c_void_p * nd)(*[q._c.codes for q in shards])
    scales = (ctypes.c_void_p * nd)(*[q._c.scales for q in shards])
    _launch("zero_gather_shards_mxfp4", i, stream, codes, scales, nd, S, p, ty)


def zero_mxfp4_matmul(a: MXFP4, w: MXFP4, out: torch.Tensor, stream=None) -> None:
    """out[m, n] = sum over k of a[m, k] w[n, k], both in 4 bits."""
    i = _mx(w, "w").index
    _mx(a, "a", i)
    if a.cols != w.cols:
        raise ValueError(f"a has {a.cols} columns, w has {w.cols}")
    p, ty, rows, cols, ld = _rows(out, "out", _TYPES, i)
    _size("out", rows, cols, a.rows, w.rows)
    _launch("zero_mxfp4_matmul", i, stream, a._ref, w._ref, p, ty, ld)


def zero_mxfp4_linear(x: torch.Tensor, w: MXFP4, out: torch.Tensor, stream=None) -> None:
    """out[m, n] = sum over k of x[m, k] w[n, k], x float16 or bfloat16."""
    i = _mx(w, "w").index
    xp, xt, m, k, ldx = _rows(x, "x", _HALF, i)
    _size("x", m, k, m, w.cols)
    p, ty, rows, cols, ld = _rows(out, "out", _TYPES, i)
    _size("out", rows, cols, m, w.rows)
    _launch("zero_mxfp4_linear", i, stream, xp, xt, m, ldx, w._ref, p, ty, ld)


def zero_mxfp4_linear_grad_input(dy: torch.Tensor, w: MXFP4, out: torch.Tensor,
                                 stream=None) -> None:
    """out[m, k] = sum over n of dy[m, n] w[n, k], dy float16 or bfloat16:
    the gradient of zero_mxfp4_linear's x (and of zero_mxfp4_matmul's a) from
    that of its output.  The workspace of a sum taken in parts comes from
    torch's allocator, on the call's stream."""
    i = _mx(w, "w").index
    dp, dt, m, n, ldd = _rows(dy, "dy", _HALF, i)
    _size("dy", m, n, m, w.rows)
    p, ty, rows, cols, ld = _rows(out, "out", _TYPES, i)
    _size("out", rows, cols, m, w.cols)
    need = ctypes.c_uint64()
    _check("zero_mxfp4_grad_workspace",
           _lib.zero_mxfp4_grad_workspace(m, w._ref, ctypes.byref(need)))
    if not need.value:
        return _launch("zero_mxfp4_linear_grad_input", i, stream, dp, dt, m, ldd, w._ref, p, ty,
                       ld, None, 0)
    if stream is None:
        ws = torch.empty(need.value, dtype=torch.uint8, device=w.device)
    else:  # the allocator orders the memory's next use after this stream's work
        with torch.cuda.stream(_torch_stream(_stream_handle(stream), w.device)):
            ws = torch.empty(need.value, dtype=torch.uint8, device=w.device)
    _launch("zero_mxfp4_linear_grad_input", i, stream, dp, dt, m, ldd, w._ref, p, ty, ld,
            ws.data_ptr(), need.value)


_ONE_F32 = {torch.float32: ZERO_F32}


def zero_distill_loss(logits: torch.Tensor, top_idx: Optional[torch.Tensor],
                      top_logits: Optional[torch.Tensor], loss: torch.Tensor, grad: torch.Tensor,
                      temperature: float = 1.0, soft_weight: float = 1.0,
                      hard_weight: float = 0.0, labels: Optional[torch.Tensor] = None,
                      row_weight: Optional[torch.Tensor] = None,
                      teacher_lse: Optional[torch.Tensor] = None,
                      loss_scale: Optional[LossScale] = None,
                      nonfinite_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Distillation from a teacher's top logits: loss[r] of every row of the
    student's logits [rows, vocab] and grad (of their type, or logits itself)
    of the weighted sum of the rows, times the loss scale's 2^k.

    top_idx [rows, k] (int32 or int64; negative: absent) and top_logits
    [rows, k] are the teacher's entries, renormalised among themselves unless
    teacher_lse [rows] (float32) gives its log sum exp(logits / temperature);
    labels [rows] (int32 or int64; negative: none) add hard_weight times the
    cross entropy; row_weight [rows] (float32; 0: the row is left out)."""
    lp, lt, rows, vocab, ldl = _rows(logits, "logits", _TYPES)
    i = logits.get_device()
    gp, gt, grows, gcols, ldg = _rows(grad, "grad", _TYPES, i)
    if gt != lt:
        raise TypeError(f"grad: expected {logits.dtype}, got {grad.dtype}")
    _size("grad", grows, gcols, rows, vocab)
    op, _ = _flat(loss, "loss", _ONE_F32, rows, i)
    ip = tp = lab = wp = ep = sp = None
    ib = lb = 4
    tt = top = ldi = ldt = 0
    if top_idx is not None or top_logits is not None:
        ip, ib, r, top, ldi = _rows(top_idx, "top_idx", _INTS, i)
        _size("top_idx", r, top, rows, top)
        tp, tt, r, k, ldt = _rows(top_logits, "top_logits", _TYPES, i)
        _size("top_logits", r, k, rows, top)
    elif soft_weight:
        raise ValueError("soft_weight without the teacher's entries")
    if labels is not None:
        lab, lb = _flat(labels, "labels", _INTS, rows, i)
    elif hard_weight:
        raise ValueError("hard_weight without labels")
    if row_weight is not None:
        wp, _ = _flat(row_weight, "row_weight", _ONE_F32, rows, i)
    if teacher_lse is not None:
        ep, _ = _flat(teacher_lse, "teacher_lse", _ONE_F32, rows, i)
    if loss_scale is not None:
        if loss_scale.state.get_device() != i:
            raise ValueError(f"loss_scale: on {loss_scale.state.device}, expected device {i}")
        sp = loss_scale.state.data_ptr()
    d = _Distill(rows, vocab, lp, ldl, gp, ldg, op, ip, tp, ldi, ldt, ep, lab, wp, sp,
                 _flag(nonfinite_flag, i), temperature, soft_weight, hard_weight, top, lt, tt, ib,
                 lb)
    _launch("zero_distill_loss", i, stream, ctypes.byref(d))
