"""Python binding of libwoq.so: the weight-only-quantised skinny linears for GB300, the draft-tree
planner, the 8-bit key/value cache with its attention, and a block's norms, routing and experts.

Argument marshalling only: every function forwards to the C ABI of the same
name declared in include/woq.h, woq_tree.h, woq_kv8.h and woq_block.h, passing raw pointers (torch tensors'
``data_ptr()`` for device buffers, numpy arrays for host buffers), sizes and the
current CUDA stream.  Every step of the computation runs in the library's CUDA
kernels; there is no Python or CPU fallback.  Importing this package loads the
in-tree ``libwoq.so`` and raises if it has not been built
(``python weight_only_quantised_gb300/_build.py`` or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# WOQ_LIB selects another build of the same ABI (e.g. the trace build libwoq_trace.so)
LIB_PATH = os.environ.get("WOQ_LIB") or os.path.join(_PKG, "libwoq.so")

WOQ_OK = 0
WOQ_ERR_NULL = 1
WOQ_ERR_ALIGN = 2
WOQ_ERR_SHAPE = 3
WOQ_ERR_WORKSPACE = 4
WOQ_ERR_LAYOUT = 5
WOQ_ERR_CUDA = 6
WOQ_ERR_DEVICE = 7
WOQ_DEVERR_HEADER = 0x1
WOQ_DEVERR_TIMEOUT = 0x2
GROUP = 128
TILE_ROWS = 128

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it first (python weight_only_quantised_gb300/_build.py)")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_SIGS = {
    "woq_version": ([], _I),
    "woq_status_string": ([_I], ctypes.c_char_p),
    "woq_max_m": ([], _I),
    "woq_max_k": ([_I, _I, _I], _I),
    "woq_packed_bytes": ([_I, _I, _I], _Z),
    "woq_pack_w4": ([_P, _P, _I, _I, _P, _Z], _I),
    "woq_pack_w6": ([_P, _P, _I, _I, _P, _Z], _I),
    "woq_unpack": ([_I, _P, _Z, _I, _I, _P, _P], _I),
    "woq_pack_device": ([_I, _P, _P, _I, _I, _P, _Z, _P], _I),
    "woq_relayout_inplace": ([_I, _P, _Z, _I, _I, _P], _I),
    "woq_workspace_bytes": ([_I, _I, _I, _I], _Z),
    "woq_workspace_init": ([_P, _Z, _P], _I),
    "woq_read_status": ([_P, _Z, _I, ctypes.POINTER(ctypes.c_uint32), _P], _I),
    "woq_act_quant_int8": ([_P, _I, _I, _P, _P, _P], _I),
    "woq_w4a8_gemv": ([_P, _Z, _P, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w6a8_gemv": ([_P, _Z, _P, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w4a8_linear_bf16": ([_P, _Z, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w6a8_linear_bf16": ([_P, _Z, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_debug_group_dots": ([_I, _P, _Z, _P, _I, _I, _I, _P, _P], _I),
    "woq_w4a8_linear_bf16_noalloc": ([_P, _Z, _P, _I, _I, _I, _P, _P], _I),
    "woq_noalloc_read_status": ([_I, ctypes.POINTER(ctypes.c_uint32), _P], _I),
    "woq_tune_override": ([_I, _I, _I], _I),
    "woq_tune_path": ([_I], _I),
    "woq_tune_fault": ([_I, _I, _I], _I),
    "woq_prefetch_next": ([_P, _Z, _I, _I, _I, _I], _I),
    "woq_last_cuda_error": ([], _I),
    "woq_cuda_error_name": ([_I], ctypes.c_char_p),
    "woq_w4a8_linear_rmsnorm_bf16": ([_P, _Z, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w6a8_linear_rmsnorm_bf16": ([_P, _Z, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w4a8_linear_swiglu_f32": ([_P, _Z, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_w6a8_linear_swiglu_f32": ([_P, _Z, _P, _I, _I, _I, _P, _P, _Z, _P], _I),
    "woq_rmsnorm_act_quant_int8": ([_P, _P, ctypes.c_float, _I, _I, _P, _P, _P], _I),
    "woq_swiglu_act_quant_int8": ([_P, _I, _I, _P, _P, _P], _I),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class WoqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {lib.woq_status_string(status).decode()} (status {status})"
        if status == WOQ_ERR_CUDA:
            code = lib.woq_last_cuda_error()
            msg += f" [{lib.woq_cuda_error_name(code).decode()}]"
        super().__init__(msg)


def _check(status: int, what: str) -> None:
    if status != WOQ_OK:
        raise WoqError(status, what)


def _dptr(t, name: str = "tensor", itemsize: int = 0, numel: int = -1):
    """Device pointer of a tensor (None -> NULL).  The C entries take bare pointers (most with
    no size), so the tensor is checked here: a contiguous CUDA tensor on the current device,
    elements of itemsize bytes (when given) and at least numel of them (when given)."""
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != _current_device():
        raise ValueError(f"{name}: tensor is on {t.device}, the current device is cuda:{_current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if itemsize and t.element_size() != itemsize:
        raise ValueError(f"{name}: expected {itemsize}-byte elements, got {t.dtype}")
    if numel >= 0 and t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")
    return t.data_ptr()


def _current_device() -> int:
    # bound on first use (importing this package does not import torch): the runtime's own query,
    # without the lazy-initialisation check that torch.cuda.current_device makes on every call (a CUDA
    # tensor is at hand wherever this is asked)
    global _current_device
    import torch
    _current_device = torch._C._cuda_getDevice
    return _current_device()


# Sizes and strides go to the C ABI as int, and ctypes would cut off what does not fit.
_MOST = 2**31 - 1


def _rows(t, name: str) -> int:
    """Row count M of a 2-D activation tensor."""
    if t is None or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D [M, K] tensor")
    rows, width = t.shape
    if rows > _MOST or width > _MOST:
        raise ValueError(f"{name}: sizes up to {_MOST}, got {list(t.shape)}")
    return rows


def _nbytes(t) -> int:
    return 0 if t is None else t.nbytes


def _stream(stream):
    if stream is None:
        return _current_raw_stream(_current_device())
    return stream.cuda_stream


def _current_raw_stream(device: int) -> int:
    # the current stream's handle without a Stream object, bound like _current_device
    global _current_raw_stream
    import torch
    torch.cuda.current_stream()  # initialises CUDA (or says why it cannot)
    _current_raw_stream = torch._C._cuda_getCurrentRawStream
    return _current_raw_stream(device)


def _hptr(a: np.ndarray):
    return ctypes.c_void_p(a.ctypes.data)


# ----------------------------------------------------------------------------- info

def woq_version() -> int:
    return lib.woq_version()


def woq_max_m() -> int:
    return lib.woq_max_m()


def woq_max_k(bits: int, M: int, fused: bool) -> int:
    return lib.woq_max_k(bits, M, int(fused))


def woq_packed_bytes(bits: int, N: int, K: int) -> int:
    return lib.woq_packed_bytes(bits, N, K)


def woq_workspace_bytes(bits: int, M: int, N: int, K: int) -> int:
    return lib.woq_workspace_bytes(bits, M, N, K)


# ----------------------------------------------------------------------------- packing

def _pack_host(fn, bits: int, q: np.ndarray, scales_f16: np.ndarray, N: int, K: int) -> np.ndarray:
    q = np.ascontiguousarray(q, dtype=np.uint8)
    s = np.ascontiguousarray(scales_f16).view(np.uint16)
    out = np.empty(max(lib.woq_packed_bytes(bits, N, K), 1), dtype=np.uint8)
    _check(fn(_hptr(q), _hptr(s), N, K, _hptr(out), out.nbytes), fn.__name__)
    return out[: lib.woq_packed_bytes(bits, N, K)]


def woq_pack_w4(q4: np.ndarray, scales_f16: np.ndarray, N: int, K: int) -> np.ndarray:
    """Host pack: canonical int4 bytes [N, K/2] + fp16 scale bits [N, K/128] -> packed bytes."""
    return _pack_host(lib.woq_pack_w4, 4, q4, scales_f16, N, K)


def woq_pack_w6(q6: np.ndarray, scales_f16: np.ndarray, N: int, K: int) -> np.ndarray:
    """Host pack: canonical int6 bytes [N, 3K/4] + fp16 scale bits [N, K/128] -> packed bytes."""
    return _pack_host(lib.woq_pack_w6, 6, q6, scales_f16, N, K)


def woq_unpack(bits: int, packed: np.ndarray, N: int, K: int):
    """Host unpack: packed bytes -> (canonical bytes [N, row bytes], fp16 scale bits [N, K/128])."""
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    row = K // 2 if bits == 4 else K // 4 * 3
    q = np.zeros((N, row), dtype=np.uint8)
    s = np.zeros((N, K // GROUP), dtype=np.uint16)
    _check(lib.woq_unpack(bits, _hptr(packed), packed.nbytes, N, K, _hptr(q), _hptr(s)), "woq_unpack")
    return q, s


def woq_pack_device(bits: int, q_dev, scales_dev, N: int, K: int, dst_dev, stream=None) -> None:
    """Device pack into dst_dev (uint8 tensor of woq_packed_bytes(bits, N, K) bytes)."""
    row = K // 2 if bits == 4 else K // 4 * 3
    _check(lib.woq_pack_device(bits, _dptr(q_dev, "q_dev", 1, N * row), _dptr(scales_dev, "scales_dev", 2, N * (K // GROUP)),
                               N, K, _dptr(dst_dev, "dst_dev", 1), _nbytes(dst_dev), _stream(stream)), "woq_pack_device")


def woq_relayout_inplace(bits: int, buf, N: int, K: int, stream=None) -> None:
    """In-place relayout of buf (uint8 device tensor of woq_packed_bytes(bits, N, K)
    bytes): canonical weights from byte 256 on, then the fp16 scales; packed on return."""
    _check(lib.woq_relayout_inplace(bits, _dptr(buf, "buf", 1), _nbytes(buf), N, K, _stream(stream)),
           "woq_relayout_inplace")


def canonical_into_buffer(bits: int, q_dev, scales_dev, buf) -> None:
    """Place canonical weights and scales (device tensors) where woq_relayout_inplace expects them."""
    import torch

    qb = q_dev.reshape(-1).view(torch.uint8)
    sb = scales_dev.reshape(-1).view(torch.uint8)
    buf[256:256 + qb.numel()].copy_(qb)
    buf[256 + qb.numel():256 + qb.numel() + sb.numel()].copy_(sb)


# ----------------------------------------------------------------------------- workspace

def woq_workspace_init(ws, stream=None) -> None:
    _check(lib.woq_workspace_init(_dptr(ws, "ws", 1), _nbytes(ws), _stream(stream)), "woq_workspace_init")


def woq_read_status(ws, clear: bool = False, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(lib.woq_read_status(_dptr(ws, "ws", 1), _nbytes(ws), int(clear), ctypes.byref(v), _stream(stream)),
           "woq_read_status")
    return int(v.value)


# ----------------------------------------------------------------------------- compute

def woq_act_quant_int8(x_bf16, q, ascale, stream=None) -> None:
    """x_bf16 [M, K] bf16 -> q [M, K] int8, ascale [M] fp32 (device tensors)."""
    M = _rows(x_bf16, "x_bf16")
    K = x_bf16.shape[1]
    _check(lib.woq_act_quant_int8(_dptr(x_bf16, "x_bf16", 2), M, K, _dptr(q, "q", 1, M * K),
                                  _dptr(ascale, "ascale", 4, M), _stream(stream)), "woq_act_quant_int8")


def _gemv(fn, name, wpacked, q, ascale, N, K, y, ws, stream):
    M = _rows(q, "q")
    _check(fn(_dptr(wpacked, "wpacked", 1), _nbytes(wpacked), _dptr(q, "q", 1, M * K), _dptr(ascale, "ascale", 4, M),
              M, N, K, _dptr(y, "y", 4, M * N), _dptr(ws, "ws", 1), _nbytes(ws), _stream(stream)), name)


def woq_w4a8_gemv(wpacked, q, ascale, N: int, K: int, y, ws, stream=None) -> None:
    _gemv(lib.woq_w4a8_gemv, "woq_w4a8_gemv", wpacked, q, ascale, N, K, y, ws, stream)


def woq_w6a8_gemv(wpacked, q, ascale, N: int, K: int, y, ws, stream=None) -> None:
    _gemv(lib.woq_w6a8_gemv, "woq_w6a8_gemv", wpacked, q, ascale, N, K, y, ws, stream)


def _linear(fn, name, wpacked, x_bf16, N, K, y, ws, stream):
    M = _rows(x_bf16, "x_bf16")
    _check(fn(_dptr(wpacked, "wpacked", 1), _nbytes(wpacked), _dptr(x_bf16, "x_bf16", 2, M * K), M, N, K,
              _dptr(y, "y", 4, M * N), _dptr(ws, "ws", 1), _nbytes(ws), _stream(stream)), name)


def woq_w4a8_linear_bf16(wpacked, x_bf16, N: int, K: int, y, ws, stream=None) -> None:
    _linear(lib.woq_w4a8_linear_bf16, "woq_w4a8_linear_bf16", wpacked, x_bf16, N, K, y, ws, stream)


def woq_w6a8_linear_bf16(wpacked, x_bf16, N: int, K: int, y, ws, stream=None) -> None:
    _linear(lib.woq_w6a8_linear_bf16, "woq_w6a8_linear_bf16", wpacked, x_bf16, N, K, y, ws, stream)


def _linear_rmsnorm(fn, name, wpacked, x_bf16, gamma_bf16, eps, N, K, y, ws, stream):
    M = _rows(x_bf16, "x_bf16")
    _check(fn(_dptr(wpacked, "wpacked", 1), _nbytes(wpacked), _dptr(x_bf16, "x_bf16", 2, M * K),
              _dptr(gamma_bf16, "gamma_bf16", 2, K), float(eps), M, N, K, _dptr(y, "y", 4, M * N),
              _dptr(ws, "ws", 1), _nbytes(ws), _stream(stream)), name)


def woq_w4a8_linear_rmsnorm_bf16(wpacked, x_bf16, gamma_bf16, eps: float, N: int, K: int, y, ws, stream=None) -> None:
    """RMSNorm(x) with gamma, quantised and run through the int4 linear, in one launch."""
    _linear_rmsnorm(lib.woq_w4a8_linear_rmsnorm_bf16, "woq_w4a8_linear_rmsnorm_bf16", wpacked, x_bf16, gamma_bf16, eps,
                    N, K, y, ws, stream)


def woq_w6a8_linear_rmsnorm_bf16(wpacked, x_bf16, gamma_bf16, eps: float, N: int, K: int, y, ws, stream=None) -> None:
    _linear_rmsnorm(lib.woq_w6a8_linear_rmsnorm_bf16, "woq_w6a8_linear_rmsnorm_bf16", wpacked, x_bf16, gamma_bf16, eps,
                    N, K, y, ws, stream)


def _linear_swiglu(fn, name, wpacked, gate_up, N, K, y, ws, stream):
    M = _rows(gate_up, "gate_up")
    _check(fn(_dptr(wpacked, "wpacked", 1), _nbytes(wpacked), _dptr(gate_up, "gate_up", 4, M * 2 * K), M, N, K,
              _dptr(y, "y", 4, M * N), _dptr(ws, "ws", 1), _nbytes(ws), _stream(stream)), name)


def woq_w4a8_linear_swiglu_f32(wpacked, gate_up, N: int, K: int, y, ws, stream=None) -> None:
    """SwiGLU of an fp32 gate+up output [M, 2K], quantised and run through the int4 linear, in one launch."""
    _linear_swiglu(lib.woq_w4a8_linear_swiglu_f32, "woq_w4a8_linear_swiglu_f32", wpacked, gate_up, N, K, y, ws, stream)


def woq_w6a8_linear_swiglu_f32(wpacked, gate_up, N: int, K: int, y, ws, stream=None) -> None:
    _linear_swiglu(lib.woq_w6a8_linear_swiglu_f32, "woq_w6a8_linear_swiglu_f32", wpacked, gate_up, N, K, y, ws, stream)


def woq_rmsnorm_act_quant_int8(x_bf16, gamma_bf16, eps: float, q, ascale, stream=None) -> None:
    M = _rows(x_bf16, "x_bf16")
    K = x_bf16.shape[1]
    _check(lib.woq_rmsnorm_act_quant_int8(_dptr(x_bf16, "x_bf16", 2), _dptr(gamma_bf16, "gamma_bf16", 2, K), float(eps),
                                          M, K, _dptr(q, "q", 1, M * K), _dptr(ascale, "ascale", 4, M),
                                          _stream(stream)), "woq_rmsnorm_act_quant_int8")


def woq_swiglu_act_quant_int8(gate_up, q, ascale, stream=None) -> None:
    M = _rows(gate_up, "gate_up")
    K = gate_up.shape[1] // 2
    _check(lib.woq_swiglu_act_quant_int8(_dptr(gate_up, "gate_up", 4), M, K, _dptr(q, "q", 1, M * K),
                                         _dptr(ascale, "ascale", 4, M), _stream(stream)), "woq_swiglu_act_quant_int8")


def woq_w4a8_linear_bf16_noalloc(wpacked, x_bf16, N: int, K: int, y, stream=None) -> None:
    """woq_w4a8_linear_bf16 for callers that cannot allocate a workspace (the library's own
    2 MiB scratch is used; calls that overlap on the GPU race)."""
    M = _rows(x_bf16, "x_bf16")
    _check(lib.woq_w4a8_linear_bf16_noalloc(_dptr(wpacked, "wpacked", 1), _nbytes(wpacked),
                                            _dptr(x_bf16, "x_bf16", 2, M * K), M, N, K, _dptr(y, "y", 4, M * N),
                                            _stream(stream)), "woq_w4a8_linear_bf16_noalloc")


def woq_noalloc_read_status(clear: bool = False, stream=None) -> int:
    """Status word (WOQ_DEVERR_* bits) of the allocation-free linear's built-in scratch."""
    v = ctypes.c_uint32(0)
    _check(lib.woq_noalloc_read_status(int(clear), ctypes.byref(v), _stream(stream)), "woq_noalloc_read_status")
    return int(v.value)


def woq_debug_group_dots(bits: int, wpacked, q, N: int, K: int, dots, stream=None) -> None:
    M = _rows(q, "q")
    _check(lib.woq_debug_group_dots(bits, _dptr(wpacked, "wpacked", 1), _nbytes(wpacked), _dptr(q, "q", 1, M * K), M, N,
                                    K, _dptr(dots, "dots", 4, M * N * (K // GROUP)), _stream(stream)),
           "woq_debug_group_dots")


class LaunchPlan(ctypes.Structure):
    """woq_launch_plan of include/woq.h."""
    _fields_ = [("ctas", ctypes.c_int), ("stages", ctypes.c_int), ("prefetch_stages", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("consumer", ctypes.c_int)]


lib.woq_plan_launch.argtypes = [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(LaunchPlan)]
lib.woq_plan_launch.restype = _I

PLAN_INT8, PLAN_BF16, PLAN_SWIGLU = 0, 1, 2  # entry kinds of woq_plan_launch


def woq_plan_launch(bits: int, M: int, N: int, K: int, entry: int = PLAN_BF16, sms: int = 0,
                    smem_max: int = 0) -> dict:
    """The launch table's choice (grid, ring stages, L2 prefetch stages, shared memory, consumer)
    for one launch, on the current device or on one with sms SMs and smem_max bytes of opt-in
    shared memory per block; nothing is launched."""
    plan = LaunchPlan()
    _check(lib.woq_plan_launch(bits, M, N, K, entry, sms, smem_max, ctypes.byref(plan)), "woq_plan_launch")
    return {name: getattr(plan, name) for name, _ in LaunchPlan._fields_}


def woq_prefetch_next(next_wpacked, bits: int, N: int, K: int, budget_kb: int = 0) -> None:
    """Hint for the next GEMV / linear call of this thread: the linear that runs after it
    (packed weights next_wpacked of (bits, N, K)); None clears the hint."""
    if next_wpacked is None:
        _check(lib.woq_prefetch_next(None, 0, bits, N, K, 0), "woq_prefetch_next")
        return
    _check(lib.woq_prefetch_next(_dptr(next_wpacked, "next_wpacked", 1), _nbytes(next_wpacked), bits, N, K, budget_kb),
           "woq_prefetch_next")


def woq_tune_override(ctas_per_sm: int = 0, stages: int = 0, prefetch_kb: int = -1) -> None:
    _check(lib.woq_tune_override(ctas_per_sm, stages, prefetch_kb), "woq_tune_override")


def woq_tune_fault(kind: int = 0, cta: int = 0, wait_limit_us: int = 0) -> None:
    """Tests of the bounded waits: inject one CTA's missing arrival (include/woq.h)."""
    _check(lib.woq_tune_fault(kind, cta, wait_limit_us), "woq_tune_fault")


def woq_tune_path(path: int = 0) -> None:
    """int4 consumer of later launches: 0 launch table, 1 dp4a, 2 tensor-core MMA."""
    _check(lib.woq_tune_path(path), "woq_tune_path")


# ----------------------------------------------------------------------------- draft-tree planner
# (include/woq_tree.h; host code in the same library)

_TREE_ROWS, _TREE_BINS, TREE_SHAPES = 7, 8, 64


class TreePlannerState(ctypes.Structure):
    _fields_ = [("counts", (ctypes.c_double * _TREE_BINS) * _TREE_ROWS),
                ("draft_ms", ctypes.c_double), ("verify_ms", ctypes.c_double),
                ("decay", ctypes.c_double), ("hysteresis", ctypes.c_double),
                ("replan_every", ctypes.c_int), ("steps", ctypes.c_int), ("times_seen", ctypes.c_int),
                ("widths", ctypes.c_int * _TREE_ROWS), ("depth", ctypes.c_int)]


_TP = ctypes.POINTER(TreePlannerState)
_IP = ctypes.POINTER(ctypes.c_int)
_DP = ctypes.POINTER(ctypes.c_double)
for _name, (_args, _res) in {
    "woq_tree_init": ([_TP, ctypes.c_double, ctypes.c_double, _I], _I),
    "woq_tree_shape": ([_I, _IP, _IP], _I),
    "woq_tree_score": ([_TP, _IP, _I, _DP, _DP], _I),
    "woq_tree_observe": ([_TP, _I, _IP, ctypes.c_double, ctypes.c_double, _IP], _I),
    "woq_tree_replan": ([_TP, _IP, _DP, _IP], _I),
}.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


def woq_tree_shape(index: int) -> tuple:
    w = (ctypes.c_int * _TREE_ROWS)()
    d = ctypes.c_int()
    _check(lib.woq_tree_shape(index, w, ctypes.byref(d)), "woq_tree_shape")
    return tuple(w[: d.value])


class TreePlanner:
    """The draft-tree planner of include/woq_tree.h (argument marshalling only)."""

    def __init__(self, decay: float = 0.0, hysteresis: float = -1.0, replan_every: int = 0):
        self.state = TreePlannerState()
        _check(lib.woq_tree_init(ctypes.byref(self.state), decay, hysteresis, replan_every), "woq_tree_init")

    @property
    def shape(self) -> tuple:
        return tuple(self.state.widths[: self.state.depth])

    def score(self, widths) -> tuple:
        w = (ctypes.c_int * _TREE_ROWS)(*widths)
        e, s = ctypes.c_double(), ctypes.c_double()
        _check(lib.woq_tree_score(ctypes.byref(self.state), w, len(widths), ctypes.byref(e), ctypes.byref(s)),
               "woq_tree_score")
        return e.value, s.value

    def observe(self, ranks, draft_ms: float = -1.0, verify_ms: float = -1.0) -> bool:
        r = (ctypes.c_int * _TREE_ROWS)(*ranks)
        sw = ctypes.c_int()
        _check(lib.woq_tree_observe(ctypes.byref(self.state), len(ranks), r, draft_ms, verify_ms, ctypes.byref(sw)),
               "woq_tree_observe")
        return bool(sw.value)

    def replan(self) -> tuple:
        i, s, sw = ctypes.c_int(), ctypes.c_double(), ctypes.c_int()
        _check(lib.woq_tree_replan(ctypes.byref(self.state), ctypes.byref(i), ctypes.byref(s), ctypes.byref(sw)),
               "woq_tree_replan")
        return i.value, s.value, bool(sw.value)

    def counts(self) -> np.ndarray:
        return np.array([[self.state.counts[d][b] for b in range(_TREE_BINS)] for d in range(_TREE_ROWS)])


# ----------------------------------------------------------------------------- 8-bit key/value cache
# (include/woq_kv8.h)

KV8_INT8, KV8_E4M3 = 0, 1
KV8_BLOCK, KV8_ROWS, KV8_MAX_SEQS = 64, 8, 1024
WOQ_DEVERR_PAGES = 0x4
WOQ_DEVERR_STATE = 0x8
WOQ_DEVERR_POSITION = 0x10


class KV8Config(ctypes.Structure):
    """woq_kv8_config of include/woq_kv8.h."""
    _fields_ = [("format", ctypes.c_int), ("layers", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("seqs", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("pages", ctypes.c_int)]


class _Rope(ctypes.Structure):
    _fields_ = [("table", _P), ("positions", _I), ("rot_dim", _I), ("interleaved", _I), ("axes", _I), ("pos", _P),
                ("axis_of", _P)]


class Rope:
    """Rotary arguments of appends (woq_rope), checked once: table fp32 [positions, rot_dim / 2, 2] from
    woq_rope_table; pos int32 [axes, rows] (device; its contents may change from call to call); axis_of: the axis
    of each frequency (host integers; None: all 0)."""

    def __init__(self, table, pos, axis_of=None, interleaved: bool = False):
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError("rope table: expected [positions, rot_dim / 2, 2]")
        if pos.dim() != 2:
            raise ValueError(f"rope positions: expected [axes, rows], got {tuple(pos.shape)}")
        axis_of = None if axis_of is None else np.array(axis_of, dtype=np.uint8)
        if axis_of is not None and axis_of.size != table.shape[1]:
            raise ValueError(f"rope axis_of: expected {table.shape[1]} entries, got {axis_of.size}")
        self._args = _Rope(_typed(table, "rope table", _F32, -1), table.shape[0], 2 * table.shape[1], int(bool(interleaved)),
                           pos.shape[0], _typed(pos, "rope positions", _INT32, -1),
                           None if axis_of is None else axis_of.ctypes.data)
        self._held = table, pos, axis_of
        self._rows, self._device = pos.shape[1], pos.get_device()

    def _ref(self, rows: int):
        if rows != self._rows:
            raise ValueError(f"rope positions: expected [axes, {rows}], got {tuple(self._held[1].shape)}")
        if self._device != _current_device():
            raise ValueError(f"rope: tensors are on cuda:{self._device}, the current device is cuda:{_current_device()}")
        return ctypes.byref(self._args)


class KV8Plan(ctypes.Structure):
    """woq_kv8_plan of include/woq_kv8.h."""
    _fields_ = [("ctas", ctypes.c_int), ("warps", ctypes.c_int), ("query_groups", ctypes.c_int), ("stages", ctypes.c_int),
                ("least_units", ctypes.c_int), ("smem_bytes", ctypes.c_int)]


_CP = ctypes.POINTER(KV8Config)
_RP = ctypes.POINTER(_Rope)
for _name, (_args, _res) in {
    "woq_kv8_bytes": ([_CP], _Z),
    "woq_kv8_page_offset": ([_CP, _I], _Z),
    "woq_kv8_init": ([_CP, _P, _Z, _P], _I),
    "woq_rope_table": ([ctypes.c_double, _I, _I, _P, _P], _I),
    "woq_kv8_append_rows": ([_CP, _P, _Z, _I, _P, _I, _I, _P, _I, _I, _I, _RP, _P, _P], _I),
    "woq_kv8_append_prompt": ([_CP, _P, _Z, _I, _I, _I, _P, _I, _I, _I, _RP, _P, _P], _I),
    "woq_kv8_accept": ([_CP, _P, _Z, _P, _I, _P, _P], _I),
    "woq_kv8_extend": ([_CP, _P, _Z, _I, _I, _P], _I),
    "woq_kv8_attention_workspace": ([_CP, _I, _I, _I], _Z),
    "woq_kv8_attention": ([_CP, _P, _Z, _I, _P, _I, _I, _P, _I, _P, ctypes.c_float, _I, _I, _P, _P, _Z, _P], _I),
    "woq_kv8_plan_attention": ([_CP, _I, _I, _I, _I, _I, ctypes.POINTER(KV8Plan)], _I),
    "woq_kv8_fork": ([_CP, _P, _Z, _P, _P, _I, _P], _I),
    "woq_kv8_free": ([_CP, _P, _Z, _P, _I, _P], _I),
    "woq_kv8_copy": ([_CP, _P, _Z, _CP, _P, _Z, _P, _P, _I, _P], _I),
    "woq_kv8_compact": ([_CP, _P, _Z, _I, _P], _I),
    "woq_kv8_read": ([_CP, _P, _Z, _I, _I, _I, _I, _P, _P, _P], _I),
    "woq_kv8_state": ([_CP, _P, _Z, _P, _P, _P, _P], _I),
}.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


def woq_kv8_bytes(cfg: KV8Config) -> int:
    return lib.woq_kv8_bytes(ctypes.byref(cfg))


def woq_kv8_page_offset(cfg: KV8Config, page: int) -> int:
    return lib.woq_kv8_page_offset(ctypes.byref(cfg), page)


def woq_kv8_attention_workspace(cfg: KV8Config, n: int, rows: int, q_heads: int) -> int:
    return lib.woq_kv8_attention_workspace(ctypes.byref(cfg), n, rows, q_heads)


def woq_kv8_plan_attention(cfg: KV8Config, n: int, rows: int, q_heads: int, sms: int = 0, smem_max: int = 0) -> dict:
    """The attention's launch shape on the current device, or on one with sms SMs and smem_max bytes of
    opt-in shared memory per block; nothing is launched."""
    plan = KV8Plan()
    _check(lib.woq_kv8_plan_attention(ctypes.byref(cfg), n, rows, q_heads, sms, smem_max, ctypes.byref(plan)),
           "woq_kv8_plan_attention")
    return {name: getattr(plan, name) for name, _ in KV8Plan._fields_}


# The cache's calls come many to a step, so their checks are written to cost little (about half a microsecond a
# tensor): one pass over what has to hold, and _dptr's messages where something does not.
_INT32, _BF16, _F32 = "int32", "bfloat16", "float32"
_DTYPES = {}  # element type -> the torch dtypes that hold it (bound on first use)
_bf16 = _i32 = None  # torch.bfloat16, torch.int32 (bound with them)


def _dtypes(kind: str):
    global _bf16, _i32
    import torch
    _bf16, _i32 = torch.bfloat16, torch.int32
    _DTYPES.update({_INT32: (torch.int32, getattr(torch, "uint32", torch.int32)), _BF16: (torch.bfloat16,),
                    _F32: (torch.float32,), "qkv": {torch.bfloat16: 0, torch.float32: 1}})
    return _DTYPES[kind]


def _typed(t, name: str, kind: str, numel: int):
    """Device pointer of a contiguous tensor of the kind with at least numel elements (None -> NULL)."""
    if t is None:
        return None
    if t.dtype not in (_DTYPES.get(kind) or _dtypes(kind)):
        raise ValueError(f"{name}: expected {kind}, got {t.dtype}")
    device = t.get_device()  # -1 on the host
    if device < 0 or device != _current_device() or not t.is_contiguous() or t.numel() < numel:
        return _dptr(t, name, 0, numel)  # says what is wrong
    return t.data_ptr()


def _bytes(t, name: str):
    """Device pointer of a contiguous tensor of bytes (None -> NULL)."""
    device = -1 if t is None else t.get_device()
    if device < 0 or device != _current_device() or not t.is_contiguous() or t.element_size() != 1:
        return _dptr(t, name, 1)
    return t.data_ptr()


# The calls of a step are short, so theirs try each tensor in one expression and leave what fails it to _typed and
# _bytes, which say what is wrong.

def _shared_device(t) -> int:
    """The current device if t is there, else one that no tensor is on."""
    device = t.get_device()
    return device if device >= 0 and device == _current_device() else -2


def _is_bytes(t, on: int) -> bool:
    return t is not None and t.get_device() == on and t.element_size() == 1 and t.is_contiguous()


def _cache_args(cfg: KV8Config, cache):
    return ctypes.byref(cfg), _bytes(cache, "cache"), _nbytes(cache)


def _raise(status: int, what: str):
    raise WoqError(status, what)


def woq_kv8_init(cfg: KV8Config, cache, stream=None) -> None:
    """Make an empty cache of a uint8 tensor of woq_kv8_bytes(cfg) bytes."""
    _check(lib.woq_kv8_init(*_cache_args(cfg, cache), _stream(stream)), "woq_kv8_init")


def woq_rope_table(theta: float, rot_dim: int, table, stream=None) -> None:
    """Fill table (fp32 [positions, rot_dim / 2, 2]) with cos and sin of each position and frequency."""
    if table.dim() != 3 or 2 * table.shape[1] != rot_dim or table.shape[2] != 2:
        raise ValueError(f"table: expected [positions, {rot_dim} / 2, 2], got {tuple(table.shape)}")
    _check(lib.woq_rope_table(theta, rot_dim, table.shape[0], _typed(table, "table", _F32, -1), _stream(stream)),
           "woq_rope_table")


def _qkv(cfg, qkv, q_heads, q_out, rope):
    """Arguments of an append from qkv [rows, >= (q_heads + 2 kv_heads) head_dim] (rows may be strided)."""
    rows = _rows(qkv, "qkv")
    need = (q_heads + 2 * cfg.kv_heads) * cfg.head_dim
    kind = (_DTYPES.get("qkv") or _dtypes("qkv")).get(qkv.dtype)
    if kind is None:
        raise ValueError(f"qkv: expected bfloat16 or float32, got {qkv.dtype}")
    width, (stride, inner) = qkv.shape[1], qkv.stride()
    if width < need or (rows > 0 and inner != 1):
        raise ValueError(f"qkv: rows of at least {need} neighbouring elements are needed, got {tuple(qkv.shape)}")
    if rows <= 1:
        stride = -(-width // 8) * 8  # one row: its stride says nothing
    if stride < need:
        raise ValueError(f"qkv: rows overlap (row stride {stride}, {need} elements a row)")
    if stride > _MOST:
        raise ValueError(f"qkv: row strides up to {_MOST}, got {stride}")
    on = _shared_device(qkv)
    ptr = qkv.data_ptr() if on >= 0 else _dptr(qkv[:1], "qkv")  # the rows may be strided
    count = rows * q_heads * cfg.head_dim
    q = (q_out.data_ptr() if q_out is not None and q_out.dtype is _bf16 and q_out.get_device() == on and q_out.is_contiguous()
         and q_out.numel() >= count else _typed(q_out, "q_out", _BF16, count))
    return ptr, kind, stride, q_heads, None if rope is None else rope._ref(rows), q


def woq_kv8_append_rows(cfg: KV8Config, cache, layer: int, seqs, rows: int, qkv, q_heads: int, q_out, rope=None,
                        stream=None) -> None:
    """`rows` draft rows behind each sequence of seqs (int32 [n]; None: as many as qkv has, from 0 on):
    qkv [n * rows, ...] rotated, queries to q_out, keys and values into the cache."""
    total = _rows(qkv, "qkv")
    n = total // max(rows, 1) if seqs is None else seqs.numel()
    if n * rows != total:
        raise ValueError(f"qkv: {total} rows, the call needs {n} x {rows}")
    args = _qkv(cfg, qkv, q_heads, q_out, rope)
    on = _shared_device(qkv)
    c = cache.data_ptr() if _is_bytes(cache, on) else _bytes(cache, "cache")
    e = (seqs.data_ptr() if seqs is not None and seqs.dtype is _i32 and seqs.get_device() == on and seqs.is_contiguous()
         else _typed(seqs, "seqs", _INT32, n))
    status = lib.woq_kv8_append_rows(ctypes.byref(cfg), c, _nbytes(cache), layer, e, n, rows, *args,
                                     _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_kv8_append_rows")


def woq_kv8_append_prompt(cfg: KV8Config, cache, layer: int, seq: int, qkv, q_heads: int, q_out, rope=None,
                          stream=None) -> None:
    """Fill the last tokens of a sequence (those of its last woq_kv8_extend) in one layer."""
    args = _qkv(cfg, qkv, q_heads, q_out, rope)
    _check(lib.woq_kv8_append_prompt(*_cache_args(cfg, cache), layer, seq, _rows(qkv, "qkv"), *args,
                                     _stream(stream)), "woq_kv8_append_prompt")


def woq_kv8_extend(cfg: KV8Config, cache, seq: int, tokens: int, stream=None) -> None:
    _check(lib.woq_kv8_extend(*_cache_args(cfg, cache), seq, tokens, _stream(stream)), "woq_kv8_extend")


def woq_kv8_accept(cfg: KV8Config, cache, seqs, keep, stream=None) -> None:
    """Take the draft rows of each mask of keep (int32 [n], bit j: row j) into the sequences."""
    n = keep.numel()
    if seqs is not None and seqs.numel() != n:
        raise ValueError(f"keep: {n} entries for {seqs.numel()} sequences")
    _check(lib.woq_kv8_accept(*_cache_args(cfg, cache), _typed(seqs, "seqs", _INT32, n), n, _typed(keep, "keep", _INT32, n),
                              _stream(stream)), "woq_kv8_accept")


def woq_kv8_attention(cfg: KV8Config, cache, layer: int, seqs, rows: int, q, q_heads: int, out, ws, scale: float,
                      window: int = 0, sinks: int = 0, vis=None, stream=None) -> None:
    """Attention of `rows` rows of each sequence of seqs (int32 [n]; None: as many as q has, from 0 on):
    q, out bf16 [n * rows, q_heads, head_dim]; vis int32 [n, rows], the draft rows each row sees (None: a chain)."""
    per = rows * q_heads * cfg.head_dim
    if per < 1:
        per = 1
    total = q.numel()
    n = total // per if seqs is None else seqs.numel()
    if n * per != total:
        raise ValueError(f"q: {total} elements, the call needs {n} x {per}")
    on = _shared_device(q)
    c = cache.data_ptr() if _is_bytes(cache, on) else _bytes(cache, "cache")
    w = ws.data_ptr() if _is_bytes(ws, on) else _bytes(ws, "ws")
    a = q.data_ptr() if q.dtype is _bf16 and on >= 0 and q.is_contiguous() else _typed(q, "q", _BF16, total)
    b = (out.data_ptr() if out is not None and out.dtype is _bf16 and out.get_device() == on and out.is_contiguous()
         and out.numel() >= total else _typed(out, "out", _BF16, total))
    e = (seqs.data_ptr() if seqs is not None and seqs.dtype is _i32 and seqs.get_device() == on and seqs.is_contiguous()
         else _typed(seqs, "seqs", _INT32, n))
    status = lib.woq_kv8_attention(
        ctypes.byref(cfg), c, _nbytes(cache), layer, e, n, rows, a, q_heads,
        None if vis is None else _typed(vis, "vis", _INT32, n * rows), scale, window, sinks, b, w, _nbytes(ws),
        _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_kv8_attention")


def woq_kv8_fork(cfg: KV8Config, cache, src, dst, stream=None) -> None:
    n = dst.numel()
    if src.numel() != n:
        raise ValueError(f"src: {src.numel()} entries for {n} in dst")
    _check(lib.woq_kv8_fork(*_cache_args(cfg, cache), _typed(src, "src", _INT32, n), _typed(dst, "dst", _INT32, n), n,
                            _stream(stream)), "woq_kv8_fork")


def woq_kv8_free(cfg: KV8Config, cache, seqs, stream=None) -> None:
    _check(lib.woq_kv8_free(*_cache_args(cfg, cache), _typed(seqs, "seqs", _INT32, seqs.numel()), seqs.numel(),
                            _stream(stream)), "woq_kv8_free")


def woq_kv8_copy(src_cfg: KV8Config, src, dst_cfg: KV8Config, dst, src_seqs, dst_seqs, stream=None) -> None:
    """Copies of sequences, with pages of their own, in the same cache or another."""
    n = dst_seqs.numel()
    if src_seqs.numel() != n:
        raise ValueError(f"src_seqs: {src_seqs.numel()} entries for {n} in dst_seqs")
    _check(lib.woq_kv8_copy(*_cache_args(src_cfg, src), *_cache_args(dst_cfg, dst), _typed(src_seqs, "src_seqs", _INT32, n),
                            _typed(dst_seqs, "dst_seqs", _INT32, n), n, _stream(stream)), "woq_kv8_copy")


def woq_kv8_compact(cfg: KV8Config, cache, limit: int, stream=None) -> None:
    _check(lib.woq_kv8_compact(*_cache_args(cfg, cache), limit, _stream(stream)), "woq_kv8_compact")


def woq_kv8_read(cfg: KV8Config, cache, layer: int, seq: int, first: int, k, v, stream=None) -> None:
    """Tokens first .. of a sequence back in bf16: k, v [count, kv_heads, head_dim], or with layer = -1
    [layers, count, kv_heads, head_dim]."""
    per = (cfg.layers if layer < 0 else 1) * cfg.kv_heads * cfg.head_dim
    total = k.numel()
    count = total // per if per > 0 else 0
    if count * per != total or v.numel() != total:
        raise ValueError(f"k, v: {total} and {v.numel()} elements, expected the same multiple of {per}")
    on = _shared_device(k)
    c = cache.data_ptr() if _is_bytes(cache, on) else _bytes(cache, "cache")
    a = k.data_ptr() if k.dtype is _bf16 and on >= 0 and k.is_contiguous() else _typed(k, "k", _BF16, -1)
    b = (v.data_ptr() if v.dtype is _bf16 and v.get_device() == on and v.is_contiguous() else _typed(v, "v", _BF16, -1))
    status = lib.woq_kv8_read(ctypes.byref(cfg), c, _nbytes(cache), layer, seq, first, count, a, b,
                              _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_kv8_read")


def woq_kv8_state(cfg: KV8Config, cache, lens=None, refs=None, table=None, stream=None) -> None:
    """Copies of the lengths [seqs], page reference counts [pages] and page tables [seqs, ceil(max_tokens / 64)]."""
    blocks = -(-cfg.max_tokens // KV8_BLOCK)
    _check(lib.woq_kv8_state(*_cache_args(cfg, cache), _typed(lens, "lens", _INT32, cfg.seqs), _typed(refs, "refs", _INT32, cfg.pages),
                             _typed(table, "table", _INT32, cfg.seqs * blocks), _stream(stream)), "woq_kv8_state")


# ----------------------------------------------------------------------------- a block around its linears
# (include/woq_block.h)

ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1


class _Router(ctypes.Structure):
    _fields_ = [("score", _I), ("experts", _I), ("k", _I), ("groups", _I), ("top_groups", _I), ("group_best", _I),
                ("renormalise", _I), ("scale", ctypes.c_float)]


_FL = ctypes.c_float
for _name, (_args, _res) in {
    "woq_block_norm": ([_P, _I, _P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _FL, _FL, _FL, _FL, _P], _I),
    "woq_route": ([ctypes.POINTER(_Router), _P, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "woq_experts_bytes": ([_I, _I, _I, _I], _Z),
    "woq_experts_workspace": ([_I, _I, _I, _I, _I], _Z),
    "woq_experts_swiglu": ([_I, _I, _P, _Z, _P, _Z, _P, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P], _I),
}.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


def _kind(t, name: str) -> int:
    """WOQ_KV8_BF16 or WOQ_KV8_F32 of a tensor."""
    kind = (_DTYPES.get("qkv") or _dtypes("qkv")).get(t.dtype)
    if kind is None:
        raise ValueError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return kind


def _shaped(t, name: str, kind: str, shape: tuple, on: int):
    """Device pointer of a contiguous tensor of the kind and shape on device `on` (None -> NULL)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")
    if t.get_device() == on and t.is_contiguous() and t.dtype in (_DTYPES.get(kind) or _dtypes(kind)):
        return t.data_ptr()
    return _typed(t, name, kind, -1)


def woq_block_norm(u, r, r_out, out, post=None, gate=None, pre=None, alpha: float = 1.0, beta: float = 1.0,
                   offset: float = 0.0, eps: float = 1e-6, stream=None) -> None:
    """r_out = alpha r + beta gate RMSNorm(u; post + offset), out = RMSNorm(r_out; pre + offset), in one pass:
    u, r, r_out [T, D] bf16 or fp32 (r_out may be r), out [T, D] bf16 (None: not formed); post, pre [D] and gate
    [gate_rows, D] bf16, row t of u taking gate row t // (T // gate_rows)."""
    T = _rows(u, "u")
    D = u.shape[1]
    ukind, rkind = _kind(u, "u"), _kind(r, "r")
    on = _shared_device(u)
    if getattr(r_out, "dtype", None) is not r.dtype:
        raise ValueError(f"r_out: expected {r.dtype}, got {getattr(r_out, 'dtype', r_out)}")
    shape, rname = (T, D), _F32 if rkind else _BF16
    if gate is not None and (gate.dim() != 2 or gate.shape[1] != D or (T > 0 and (gate.shape[0] < 1 or T % gate.shape[0]))):
        raise ValueError(f"gate: expected [rows, {D}] with rows a divisor of {T}, got {list(gate.shape)}")
    status = lib.woq_block_norm(
        _shaped(u, "u", _F32 if ukind else _BF16, shape, on), ukind, _shaped(r, "r", rname, shape, on),
        _shaped(r_out, "r_out", rname, shape, on), rkind, _shaped(out, "out", _BF16, shape, on), T, D,
        _shaped(post, "post", _BF16, (D,), on), None if gate is None else _shaped(gate, "gate", _BF16, tuple(gate.shape), on),
        1 if gate is None else gate.shape[0], _shaped(pre, "pre", _BF16, (D,), on), alpha, beta, offset, eps,
        _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_block_norm")


def woq_route(logits, k: int, ids, weights, score: int = ROUTE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
              group_best: int = 1, renormalise: bool = True, scale: float = 1.0, live=None, stream=None) -> None:
    """Each row's k experts of largest score (+ bias [E] fp32) and their weights: logits [T, E] bf16 or fp32 (rows may be
    strided) -> ids [T, k] int32, weights [T, k] fp32; live: int32 [1], rows from it on get id -1 and weight 0."""
    T = _rows(logits, "logits")
    E = logits.shape[1]
    kind = _kind(logits, "logits")
    on = _shared_device(logits)
    stride, inner = logits.stride()
    if T <= 1:
        stride = E  # one row: its stride says nothing
    if E > 1 and inner != 1 or stride < E:
        raise ValueError(f"logits: expected rows of neighbouring elements, got strides {logits.stride()}")
    if stride > _MOST:
        raise ValueError(f"logits: row strides up to {_MOST}, got {stride}")
    ptr = logits.data_ptr() if on >= 0 else _dptr(logits[:1], "logits")
    cfg = _Router(score, E, k, groups, top_groups, group_best, 1 if renormalise else 0, scale)
    status = lib.woq_route(ctypes.byref(cfg), ptr, kind, stride, T, _shaped(bias, "bias", _F32, (E,), on),
                           _shaped(live, "live", _INT32, (1,), on), _shaped(ids, "ids", _INT32, (T, k), on),
                           _shaped(weights, "weights", _F32, (T, k), on),
                           _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_route")


def woq_experts_bytes(bits: int, E: int, N: int, K: int) -> int:
    """Bytes of E packed matrices one behind the other; matrix e (woq_pack_device) starts at e / E of them."""
    return lib.woq_experts_bytes(bits, E, N, K)


def woq_experts_workspace(E: int, T: int, k: int, H: int, I: int) -> int:
    return lib.woq_experts_workspace(E, T, k, H, I)


def woq_experts_swiglu(bits: int, E: int, gate_up, down, x_bf16, ids, weights, I: int, y_bf16, ws, stream=None) -> None:
    """y = sum of each row's experts: x_bf16 [T, H], ids int32 [T, k] (-1: none), weights fp32 [T, k], y_bf16 [T, H];
    gate_up: E packed matrices of (2 I, H), down: of (H, I), one behind the other (uint8)."""
    T = _rows(x_bf16, "x_bf16")
    H = x_bf16.shape[1]
    k = ids.shape[1] if ids.dim() == 2 else -1
    if k > _MOST or abs(I) > _MOST:
        raise ValueError(f"ids, I: sizes up to {_MOST}, got {k} places and I {I}")
    on = _shared_device(x_bf16)
    status = lib.woq_experts_swiglu(
        bits, E, gate_up.data_ptr() if _is_bytes(gate_up, on) else _bytes(gate_up, "gate_up"), _nbytes(gate_up),
        down.data_ptr() if _is_bytes(down, on) else _bytes(down, "down"), _nbytes(down),
        _shaped(x_bf16, "x_bf16", _BF16, (T, H), on), _shaped(ids, "ids", _INT32, (T, k), on),
        _shaped(weights, "weights", _F32, (T, k), on), T, k, H, I, _shaped(y_bf16, "y_bf16", _BF16, (T, H), on),
        ws.data_ptr() if _is_bytes(ws, on) else _bytes(ws, "ws"), _nbytes(ws),
        _current_raw_stream(on) if stream is None and on >= 0 else _stream(stream))
    if status:
        _raise(status, "woq_experts_swiglu")
