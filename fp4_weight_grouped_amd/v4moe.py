"""ctypes binding of libv4moe (``include/v4moe.h``).

Argument marshalling only: every function forwards torch device tensors'
pointers and the current HIP stream to the C entry point of the same name and
raises :class:`V4MoeError` on a non-zero return code.  PyTorch provides device
memory and streams; every step of the layer runs in the library's kernels.
The library must have been built (``fp4_weight_grouped_amd.build``); there is
no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import dataclasses
import functools
import operator
import os
import re
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(HERE, "libv4moe.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "v4moe.h")

ROUTE_LEARNED = 0
ROUTE_HASH = 1

ACT_SWIGLU = 0
ACT_RELU2 = 1
ACT_RELU = 2

TYPE_F32 = 0
TYPE_BF16 = 1

SCORE_SIGMOID = 0
SCORE_SOFTMAX = 1
SCORE_SQRTSOFTPLUS = 2

SCALE_BLOCK = 0
SCALE_ROW = 1


class V4MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libv4moe error {code}: {msg}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("act", ctypes.c_int32)]


class Mat(ctypes.Structure):
    _fields_ = [("fp4", ctypes.c_void_p), ("e8m0", ctypes.c_void_p), ("blk", ctypes.c_void_p)]


class ExpertsC(ctypes.Structure):
    _fields_ = [("gate", Mat), ("up", Mat), ("down", Mat)]


class GateC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class GemmC(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("b_scale", ctypes.c_int32),
                ("c_type", ctypes.c_int32), ("accumulate", ctypes.c_int32), ("lda", ctypes.c_int64),
                ("ldb", ctypes.c_int64), ("ldc", ctypes.c_int64), ("bs_n", ctypes.c_int64), ("bs_k", ctypes.c_int64)]


class FP8MatC(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("q", ctypes.c_void_p), ("qt", ctypes.c_void_p),
                ("blk", ctypes.c_void_p)]


class TensorC(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int32)]


_lib = None
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_sz = ctypes.c_size_t
_DP = ctypes.POINTER(Dims)


def lib():
    """Load libv4moe.so; raise if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(SO):
            raise RuntimeError(f"{SO} is missing: build it with fp4_weight_grouped_amd.build.build()")
        L = ctypes.CDLL(SO)
        L.moe_workspace_bytes.argtypes = [_DP]
        L.moe_workspace_bytes.restype = _sz
        L.moe_strerror.argtypes = [ctypes.c_int]
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_route.argtypes = [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp]
        L.moe_permute.argtypes = [_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.moe_expert_ffn.argtypes = [_DP, _vp, _vp, _vp, _vp, ctypes.POINTER(ExpertsC), _vp, _vp, _sz, _vp]
        L.moe_combine.argtypes = [_DP, _vp, _vp, _vp, _vp]
        L.moe_layer_forward.argtypes = [_DP, _vp, _vp, _vp, _i32, _vp, ctypes.POINTER(ExpertsC),
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.moe_prepack_weights.argtypes = [_DP, ctypes.POINTER(ExpertsC), ctypes.POINTER(ExpertsC),
                                          _vp, _sz, _vp]
        L.moe_dequant_fp8.argtypes = [ctypes.POINTER(Mat), _i32, _i32, _i32, _vp, _vp]
        L.moe_quantize_weights.argtypes = [_i32, _i32, _i32, _vp, _i32, ctypes.POINTER(Mat), _vp, _vp]
        L.moe_backward_workspace_bytes.argtypes = [_DP]
        L.moe_backward_workspace_bytes.restype = _sz
        L.moe_transpose_weights.argtypes = [_DP, ctypes.POINTER(ExpertsC), _vp, _vp, _vp]
        L.moe_layer_backward.argtypes = [_DP, _vp, _vp, _vp, _i32, _vp, ctypes.POINTER(ExpertsC), _vp, _vp,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.moe_layer_forward_noalloc.argtypes = [_DP, _vp, _vp, _vp, _i32, _vp, ctypes.POINTER(ExpertsC),
                                                _vp, _vp, _vp, _vp, _vp]
        L.moe_noalloc_max_workspace_bytes.argtypes = []
        L.moe_noalloc_max_workspace_bytes.restype = _sz
        GP, MP = ctypes.POINTER(GateC), ctypes.POINTER(FP8MatC)
        L.moe_gate.argtypes = [GP, _vp, _i32, _i64, _vp, _vp, _vp, _vp]
        L.moe_gate_backward.argtypes = [GP, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _i64, _vp]
        L.moe_fp8_quantize.argtypes = [_i32, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp]
        L.moe_fp8_quantize_weights.argtypes = [_i32, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp]
        L.moe_fp8_gemm.argtypes = [ctypes.POINTER(GemmC), _vp, _vp, _vp, _vp, _vp, _vp]
        L.moe_fp8_linear_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32]
        L.moe_fp8_linear_workspace_bytes.restype = _sz
        L.moe_fp8_linear.argtypes = [_i32, _vp, _i32, _i64, MP, _vp, _i32, _i64, _vp, _sz, _vp]
        L.moe_fp8_linear_backward.argtypes = [_i32, _vp, _i32, _i64, _vp, _i32, _i64, MP, _vp, _i32, _i64, _vp, _i32,
                                              _i64, _i32, _vp, _sz, _vp]
        L.moe_clip_workspace_bytes.argtypes = [_i32]
        L.moe_clip_workspace_bytes.restype = _sz
        L.moe_clip_grads.argtypes = [_i32, _vp, _f32, _vp, _vp, _sz, _vp]
        EP = ctypes.POINTER(ExpertsC)
        L.moe_routed_forward.argtypes = [_DP, _vp, _vp, _vp, EP, _vp, _vp, _vp, _sz, _vp]
        L.moe_routed_backward.argtypes = [_DP, _vp, _vp, _vp, EP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.moe_time_next_ffn.argtypes = [_vp, _vp]
        L.moe_time_next_ffn.restype = None
        for f in ("moe_route", "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward",
                  "moe_layer_forward_noalloc",
                  "moe_prepack_weights", "moe_dequant_fp8", "moe_quantize_weights", "moe_transpose_weights",
                  "moe_layer_backward", "moe_routed_forward", "moe_routed_backward", "moe_gate", "moe_gate_backward", "moe_fp8_quantize",
                  "moe_fp8_quantize_weights", "moe_fp8_gemm", "moe_fp8_linear", "moe_fp8_linear_backward",
                  "moe_clip_grads"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def declared_functions() -> list:
    """Names of the functions declared in include/v4moe.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src)))


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def _check(rc: int):
    if rc != 0:
        raise V4MoeError(rc, strerror(rc))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def dims(T: int, H: int, I: int, E: int, topk: int, act: int = ACT_SWIGLU) -> Dims:
    return Dims(T, H, I, E, topk, act)


@dataclasses.dataclass
class DeviceMatrix:
    fp4: torch.Tensor   # uint8
    e8m0: torch.Tensor  # uint8
    blk: torch.Tensor   # float32

    def c(self) -> Mat:
        return Mat(self.fp4.data_ptr(), self.e8m0.data_ptr(), self.blk.data_ptr())


@dataclasses.dataclass
class DeviceExperts:
    gate: Optional[DeviceMatrix]   # None for the gate-less activations
    up: DeviceMatrix
    down: DeviceMatrix

    def c(self) -> ExpertsC:
        return ExpertsC(Mat() if self.gate is None else self.gate.c(), self.up.c(), self.down.c())


# ---- the C entry points ------------------------------------------------------------------
def moe_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(d)))


def moe_route(d: Dims, x, w_router, bias, mode, token_ids, topk_ids, topk_w, workspace):
    _check(lib().moe_route(ctypes.byref(d), _p(x), _p(w_router), _p(bias), mode, _p(token_ids),
                           _p(topk_ids), _p(topk_w), _p(workspace),
                           0 if workspace is None else workspace.numel(), _stream()))


def moe_permute(d: Dims, x, topk_ids, expert_offsets, sorted_pair, pair_pos, xq, xs, workspace):
    _check(lib().moe_permute(ctypes.byref(d), _p(x), _p(topk_ids), _p(expert_offsets), _p(sorted_pair),
                             _p(pair_pos), _p(xq), _p(xs), _p(workspace), workspace.numel(), _stream()))


def moe_expert_ffn(d: Dims, xq, xs, expert_offsets, sorted_pair, experts: DeviceExperts, y, workspace):
    ex = experts.c()
    _check(lib().moe_expert_ffn(ctypes.byref(d), _p(xq), _p(xs), _p(expert_offsets), _p(sorted_pair),
                                ctypes.byref(ex), _p(y), _p(workspace), workspace.numel(), _stream()))


def moe_combine(d: Dims, y, topk_w, out):
    _check(lib().moe_combine(ctypes.byref(d), _p(y), _p(topk_w), _p(out), _stream()))


def moe_layer_forward(d: Dims, x, w_router, bias, mode, token_ids, experts: DeviceExperts,
                      topk_ids, topk_w, expert_offsets, out, workspace):
    ex = experts.c()
    _check(lib().moe_layer_forward(ctypes.byref(d), _p(x), _p(w_router), _p(bias), mode, _p(token_ids),
                                   ctypes.byref(ex), _p(topk_ids), _p(topk_w), _p(expert_offsets),
                                   _p(out), _p(workspace), workspace.numel(), _stream()))


def moe_layer_forward_noalloc(d: Dims, x, w_router, bias, mode, token_ids, experts: DeviceExperts,
                              topk_ids, topk_w, expert_offsets, out):
    ex = experts.c()
    _check(lib().moe_layer_forward_noalloc(ctypes.byref(d), _p(x), _p(w_router), _p(bias), mode, _p(token_ids),
                                           ctypes.byref(ex), _p(topk_ids), _p(topk_w), _p(expert_offsets),
                                           _p(out), _stream()))


def moe_noalloc_max_workspace_bytes() -> int:
    return lib().moe_noalloc_max_workspace_bytes()


def moe_prepack_weights(d: Dims, canonical: DeviceExperts, packed: DeviceExperts, workspace):
    a, b = canonical.c(), packed.c()
    _check(lib().moe_prepack_weights(ctypes.byref(d), ctypes.byref(a), ctypes.byref(b), _p(workspace),
                                     workspace.numel(), _stream()))


def moe_dequant_fp8(m: DeviceMatrix, N: int, K: int, expert: int, out):
    mc = m.c()
    _check(lib().moe_dequant_fp8(ctypes.byref(mc), N, K, expert, _p(out), _stream()))


def moe_quantize_weights(w, out: DeviceMatrix, clamped=None, packed: bool = False):
    """w: fp32 [E][N][K] on the device -> out (fp4 and e8m0 in the canonical
    or the packed layout, blk [E][N/128][K/128]); clamped: int64 [1] device
    tensor the number of clamped sub-blocks is added to, or None."""
    E, N, K = w.shape
    oc = out.c()
    _check(lib().moe_quantize_weights(E, N, K, _p(w), 1 if packed else 0, ctypes.byref(oc), _p(clamped),
                                      _stream()))


def quantize_weights(w, clamped=None, packed: bool = False) -> DeviceMatrix:
    """Allocating convenience around moe_quantize_weights (the packed layout
    has the same byte counts as the canonical one)."""
    E, N, K = w.shape
    dev = w.device
    out = DeviceMatrix(fp4=torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev),
                       e8m0=torch.empty((E, N, K // 32), dtype=torch.uint8, device=dev),
                       blk=torch.empty((E, N // 128, K // 128), dtype=torch.float32, device=dev))
    moe_quantize_weights(w, out, clamped, packed)
    return out


def moe_backward_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_backward_workspace_bytes(ctypes.byref(d)))


def moe_transpose_weights(d: Dims, experts: DeviceExperts, wt_gu, wt_d):
    ex = experts.c()
    _check(lib().moe_transpose_weights(ctypes.byref(d), ctypes.byref(ex), _p(wt_gu), _p(wt_d), _stream()))


def moe_layer_backward(d: Dims, x, w_router, bias, mode, token_ids, experts: DeviceExperts, wt_gu, wt_d, dout,
                       dx, dw, dWg, dWu, dWd, workspace):
    ex = experts.c()
    _check(lib().moe_layer_backward(ctypes.byref(d), _p(x), _p(w_router), _p(bias), mode, _p(token_ids),
                                    ctypes.byref(ex), _p(wt_gu), _p(wt_d), _p(dout), _p(dx), _p(dw), _p(dWg),
                                    _p(dWu), _p(dWd), _p(workspace), workspace.numel(), _stream()))


def _routing(d: Dims, x, topk_ids, topk_w, dev: int):
    """Addresses of the layer's input and of a routing the caller made, checked: the ids become indices."""
    return (_given(x, (d.T, d.H), _BF16_BITS, "x", dev), _given(topk_ids, (d.T, d.topk), _INT32, "topk_ids", dev),
            _given(topk_w, (d.T, d.topk), _FLOAT32, "topk_w", dev))


def moe_routed_forward(d: Dims, x, topk_ids, topk_w, experts: DeviceExperts, expert_offsets, out, workspace):
    ex = experts.c()
    dev = _device_of(workspace, "workspace")
    _check(lib().moe_routed_forward(ctypes.byref(d), *_routing(d, x, topk_ids, topk_w, dev), ctypes.byref(ex),
                                    _given(expert_offsets, (d.E + 1,), _INT32, "expert_offsets", dev),
                                    _given(out, (d.T, d.H), _BF16_BITS, "out", dev), _p(workspace), workspace.numel(),
                                    _stream()))


def moe_routed_backward(d: Dims, x, topk_ids, topk_w, experts: DeviceExperts, wt_gu, wt_d, dout, dx, dw, dWg, dWu, dWd,
                        workspace):
    ex = experts.c()
    dev = _device_of(workspace, "workspace")
    T, H, I, E = d.T, d.H, d.I, d.E
    _check(lib().moe_routed_backward(
        ctypes.byref(d), *_routing(d, x, topk_ids, topk_w, dev), ctypes.byref(ex),
        _given(wt_gu, (E, H, 2 * I if d.act == ACT_SWIGLU else I), _UINT8, "wt_gu", dev),
        _given(wt_d, (E, I, H), _UINT8, "wt_d", dev), _given(dout, (T, H), _BF16_BITS, "dout", dev),
        _given(dx, (T, H), _FLOAT32, "dx", dev), _given(dw, (T, d.topk), _FLOAT32, "dw", dev),
        _given(dWg, (E, I, H), _FLOAT32, "dWg", dev), _given(dWu, (E, I, H), _FLOAT32, "dWu", dev),
        _given(dWd, (E, H, I), _FLOAT32, "dWd", dev), _p(workspace), workspace.numel(), _stream()))


def moe_time_next_ffn(start_event, stop_event):
    """start/stop: torch.cuda.Event(enable_timing=True) objects, or None."""
    a = None if start_event is None else ctypes.c_void_p(start_event.cuda_event)
    b = None if stop_event is None else ctypes.c_void_p(stop_event.cuda_event)
    lib().moe_time_next_ffn(a, b)


# ---- operators next to the layer ---------------------------------------------------------------
# These wrap launches of a few microseconds, so the checks are plain attribute reads, the stream
# comes from the runtime without a Stream object, and pointers travel as integers.
_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _require(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


_dtype_of = operator.attrgetter("dtype")


def _type(t: torch.Tensor) -> int:
    ty = _TYPES.get(t.dtype)
    if ty is None:
        raise TypeError(f"float32 or bfloat16 expected, got {t.dtype}")
    return ty


def _device_of(t: torch.Tensor, what: str) -> int:
    """The current GPU, after checking that t is on it; the other tensors of a call are then compared with it, as
    every address a kernel gets is that device's."""
    i = t.get_device()
    if i < 0 or i != _current_device():
        _elsewhere(t, what)
    return i


def _elsewhere(t: torch.Tensor, what: str):
    raise ValueError(f"{what} must be on a GPU" if t.get_device() < 0 else
                     f"{what} is on GPU {t.get_device()}, which is not the current device")


def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A new [rows][cols] tensor (strides spelled out: a call's time is the host's where the work is small)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty_strided((n,), (1,), dtype=torch.uint8, device=device)


def _matrix(t: torch.Tensor, rows: int, cols: int, what: str, dev: int, dtype=None) -> int:
    """t's leading dimension, after checking that it is [rows][cols] with contiguous columns on GPU dev."""
    if t.get_device() != dev:
        _elsewhere(t, what)
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must be [{rows}][{cols}], got {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    ld, st = t.stride()
    if st != 1 and cols > 1:
        raise ValueError(f"{what} must have contiguous rows")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{what} must not have overlapping rows")
    return ld


def _dense(t: torch.Tensor, shape: tuple, dtype, what: str, dev: int) -> int:
    """t's address, after checking that it is contiguous, of this shape and type, on GPU dev."""
    if t.get_device() != dev:
        _elsewhere(t, what)
    if not (t.shape == shape and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{what} must be contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)
_INT32, _FLOAT32, _UINT8 = (torch.int32,), (torch.float32,), (torch.uint8,)


def _given(t: Optional[torch.Tensor], shape: tuple, dtypes: tuple, what: str, dev: int):
    """t's address as _dense, of one of several types; None stays None (the library says where it may)."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    return _dense(t, shape, t.dtype, what, dev)


def gate(logits: torch.Tensor, topk: int, score: int = SCORE_SIGMOID, bias: Optional[torch.Tensor] = None,
         groups: int = 1, topk_groups: int = 1, renorm: bool = True, scale: float = 1.0):
    """Routing from logits [T][E] (fp32 or bf16, rows may be strided); bias: fp32 [E], selection only.
    Returns (topk_ids int32 [T][topk], topk_w fp32 [T][topk]).  See moe_gate in include/v4moe.h."""
    T, E = logits.shape
    gpu = _device_of(logits, "logits")
    ld = _matrix(logits, T, E, "logits", gpu)
    stream = _raw_stream(gpu)
    b = None if bias is None else _dense(bias, (E,), torch.float32, "bias", gpu)
    g = GateC(T, E, topk, score, groups, topk_groups, 1 if renorm else 0, scale)
    dev = logits.device
    ids = _empty(T, topk, torch.int32, dev)
    w = _empty(T, topk, torch.float32, dev)
    _check(lib().moe_gate(ctypes.byref(g), logits.data_ptr(), _type(logits), ld, b, ids.data_ptr(), w.data_ptr(), stream))
    return ids, w


def gate_backward(logits: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, dw: torch.Tensor,
                  score: int = SCORE_SIGMOID, renorm: bool = True, scale: float = 1.0) -> torch.Tensor:
    """dL/dlogits [T][E] (the logits' type) from dw = dL/dtopk_w and gate()'s outputs."""
    T, E = logits.shape
    gpu = _device_of(logits, "logits")
    ld = _matrix(logits, T, E, "logits", gpu)
    stream = _raw_stream(gpu)
    k = topk_ids.shape[1]
    ids = _dense(topk_ids, (T, k), torch.int32, "topk_ids", gpu)
    w = _dense(topk_w, (T, k), torch.float32, "topk_w", gpu)
    d = _dense(dw, (T, k), torch.float32, "dw", gpu)
    g = GateC(T, E, k, score, 1, 1, 1 if renorm else 0, scale)
    dl = _empty(T, E, logits.dtype, logits.device)
    _check(lib().moe_gate_backward(ctypes.byref(g), logits.data_ptr(), _type(logits), ld, ids, w, d, dl.data_ptr(), E,
                                   stream))
    return dl


def _up16(n: int) -> int:
    return (n + 15) // 16 * 16


def _chunks(n: int) -> int:
    return (n + 127) // 128


@dataclasses.dataclass
class FP8Matrix:
    """A dense weight [N][K] in E4M3 (v4moe_fp8mat)."""
    N: int
    K: int
    q: torch.Tensor     # uint8 [N][K rounded up to 16]
    qt: torch.Tensor    # uint8 [K][N rounded up to 16]
    blk: torch.Tensor   # float32 [ceil(N/128)][ceil(K/128)]

    def c(self, dev: Optional[int] = None) -> FP8MatC:
        """For a call on GPU dev (by default the current one)."""
        N, K = self.N, self.K
        q, qt, blk = _fp8_shapes(N, K)
        if dev is None:
            dev = _device_of(self.q, "q")
        return FP8MatC(N, K, _dense(self.q, q, torch.uint8, "q", dev), _dense(self.qt, qt, torch.uint8, "qt", dev),
                       _dense(self.blk, blk, torch.float32, "blk", dev))


@functools.lru_cache(maxsize=4096)
def _fp8_shapes(N: int, K: int):
    return (N, _up16(K)), (K, _up16(N)), (_chunks(N), _chunks(K))


def fp8_quantize(x: torch.Tensor, rows: bool = True, cols: bool = False):
    """E4M3 codes of x [M][K] and their scales: (q, s) by rows and / or (qt, st) by columns, None where not asked."""
    M, K = x.shape
    gpu = _device_of(x, "x")
    ld = _matrix(x, M, K, "x", gpu)
    stream = _raw_stream(gpu)
    dev = x.device
    q = _empty(M, _up16(K), torch.uint8, dev) if rows else None
    s = _empty(_chunks(K), M, torch.float32, dev) if rows else None
    qt = _empty(K, _up16(M), torch.uint8, dev) if cols else None
    st = _empty(_chunks(M), K, torch.float32, dev) if cols else None
    _check(lib().moe_fp8_quantize(M, K, x.data_ptr(), _type(x), ld, _p(q), _p(s), _p(qt), _p(st), stream))
    return q, s, qt, st


def fp8_weights(w: torch.Tensor) -> FP8Matrix:
    """E4M3 codes of a weight [N][K] (fp32 or bf16) in both orders, a scale for each 128x128 block."""
    N, K = w.shape
    gpu = _device_of(w, "w")
    ld = _matrix(w, N, K, "w", gpu)
    stream = _raw_stream(gpu)
    dev = w.device
    m = FP8Matrix(N, K, _empty(N, _up16(K), torch.uint8, dev),
                  _empty(K, _up16(N), torch.uint8, dev),
                  _empty(_chunks(N), _chunks(K), torch.float32, dev))
    _check(lib().moe_fp8_quantize_weights(N, K, w.data_ptr(), _type(w), ld, m.q.data_ptr(), m.qt.data_ptr(),
                                          m.blk.data_ptr(), stream))
    return m


def fp8_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, rows: bool = False,
             out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """a [M][K] times b [N][K] transposed, E4M3 codes (K a multiple of 16) with scales a_scale [ceil(K/128)][M] and
    b_scale: [ceil(N/128)][ceil(K/128)] (any strides), or with ``rows`` [ceil(K/128)][N].  out: [M][N], bf16 by default."""
    (M, K), N = a.shape, b.shape[0]
    gpu = _device_of(a, "a")
    lda, ldb = _matrix(a, M, K, "a", gpu, torch.uint8), _matrix(b, N, K, "b", gpu, torch.uint8)
    stream = _raw_stream(gpu)
    n = _chunks(K)
    sa = _dense(a_scale, (n, M), torch.float32, "a_scale", gpu)
    if rows:
        sb, bs = _dense(b_scale, (n, N), torch.float32, "b_scale", gpu), (0, 0)
    else:
        _device_of(b_scale, "b_scale")
        _require(b_scale.shape == (_chunks(N), n) and b_scale.dtype == torch.float32,
                 f"b_scale must be float32 [{_chunks(N)}][{n}]")
        sb, bs = b_scale.data_ptr(), b_scale.stride()
    if out is None:
        _require(not accumulate, "accumulate needs out")
        out = _empty(M, N, torch.bfloat16, a.device)
    ldc = _matrix(out, M, N, "out", gpu)
    g = GemmC(M, N, K, SCALE_ROW if rows else SCALE_BLOCK, _type(out), 1 if accumulate else 0, lda, ldb, ldc, bs[0], bs[1])
    _check(lib().moe_fp8_gemm(ctypes.byref(g), a.data_ptr(), sa, b.data_ptr(), sb, out.data_ptr(), stream))
    return out


@functools.lru_cache(maxsize=4096)
def moe_fp8_linear_workspace_bytes(M: int, N: int, K: int, backward: int) -> int:
    return int(lib().moe_fp8_linear_workspace_bytes(M, N, K, backward))


def fp8_linear(x: torch.Tensor, w: FP8Matrix, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W^T: x [M][K] bf16 or fp32, quantised by rows; y [M][N] (bf16 unless ``out`` says otherwise)."""
    M, N, K = x.shape[0], w.N, w.K
    gpu = _device_of(x, "x")
    ldx = _matrix(x, M, K, "x", gpu)
    stream = _raw_stream(gpu)
    dev = x.device
    if out is None:
        out, ldy, ty = _empty(M, N, torch.bfloat16, dev), N, TYPE_BF16
    else:
        ldy, ty = _matrix(out, M, N, "out", gpu), _type(out)
    c = w.c(gpu)
    n = moe_fp8_linear_workspace_bytes(M, N, K, 0)
    ws = _bytes(n, dev)
    _check(lib().moe_fp8_linear(M, x.data_ptr(), _type(x), ldx, ctypes.byref(c), out.data_ptr(), ty, ldy, ws.data_ptr(), n,
                                stream))
    return out


def fp8_linear_backward(x: torch.Tensor, dy: torch.Tensor, w: FP8Matrix, dx: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, accumulate: bool = False):
    """Gradients of fp8_linear: (dx [M][K], dw [N][K]), bf16 unless given; accumulate adds to the given dw."""
    M, N, K = x.shape[0], w.N, w.K
    gpu = _device_of(x, "x")
    ldx, lddy = _matrix(x, M, K, "x", gpu), _matrix(dy, M, N, "dy", gpu)
    stream = _raw_stream(gpu)
    dev = x.device
    _require(dw is not None or not accumulate, "accumulate needs dw")
    if dx is None:
        dx = _empty(M, K, torch.bfloat16, dev)
    if dw is None:
        dw = _empty(N, K, torch.bfloat16, dev)
    lddx, lddw = _matrix(dx, M, K, "dx", gpu), _matrix(dw, N, K, "dw", gpu)
    c = w.c(gpu)
    n = moe_fp8_linear_workspace_bytes(M, N, K, 1)
    ws = _bytes(n, dev)
    _check(lib().moe_fp8_linear_backward(M, x.data_ptr(), _type(x), ldx, dy.data_ptr(), _type(dy), lddy, ctypes.byref(c),
                                         dx.data_ptr(), _type(dx), lddx, dw.data_ptr(), _type(dw), lddw,
                                         1 if accumulate else 0, ws.data_ptr(), n, stream))
    return dx, dw


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Scales contiguous fp32 / bf16 gradients so that their joint norm is at most max_norm: in place, or into the
    tensors of ``out`` (same shapes and types).  Returns the norm before (fp32, on the GPU, no synchronisation)."""
    grads = list(grads)
    n = len(grads)
    _require(n > 0, "no gradients")
    stream = _raw_stream(_device_of(grads[0], "gradients"))
    dev = grads[0].device

    def words(tensors):     # addresses, sizes and types, by maps over the list: a small step's time is the host's
        if not all(map(torch.Tensor.is_contiguous, tensors)) or set(map(torch.Tensor.get_device, tensors)) != {dev.index}:
            raise ValueError("gradients must be contiguous on one GPU")
        return (array.array("q", map(torch.Tensor.data_ptr, tensors)), array.array("q", map(torch.Tensor.numel, tensors)),
                list(map(_dtype_of, tensors)))

    g, sizes, dtypes = words(grads)
    o = g
    if out is not None:
        out = list(out)
        _require(len(out) == n, "out must match grads")
        o, *same = words(out)
        _require(same == [sizes, dtypes], "out must match grads")
    table = array.array("q", bytes(32 * n))     # v4moe_tensor is four 64-bit words: g, out, n, type
    try:
        table[0::4], table[1::4], table[2::4], table[3::4] = g, o, sizes, array.array("q", map(_TYPES.__getitem__, dtypes))
    except KeyError as e:
        raise TypeError(f"float32 or bfloat16 expected, got {e.args[0]}") from None
    norm = torch.empty((), dtype=torch.float32, device=dev)
    size = _clip_workspace_bytes(n)
    ws = _bytes(size, dev)
    _check(lib().moe_clip_grads(n, table.buffer_info()[0], max_norm, norm.data_ptr(), ws.data_ptr(), size, stream))
    return norm


@functools.lru_cache(maxsize=1024)
def _clip_workspace_bytes(count: int) -> int:
    return int(lib().moe_clip_workspace_bytes(count))


# ---- conveniences for callers holding host (numpy) weights ----------------------------------
def upload_matrix(m, device="cuda") -> DeviceMatrix:
    return DeviceMatrix(fp4=torch.from_numpy(m.fp4).to(device),
                        e8m0=torch.from_numpy(m.e8m0).to(device),
                        blk=torch.from_numpy(m.blk).to(device))


def prepack(d: Dims, canonical: DeviceExperts) -> DeviceExperts:
    """Canonical -> packed device weights (blk tensors are shared)."""
    def like(m: Optional[DeviceMatrix]) -> Optional[DeviceMatrix]:
        if m is None:
            return None
        return DeviceMatrix(torch.empty_like(m.fp4), torch.empty_like(m.e8m0), m.blk)
    packed = DeviceExperts(like(canonical.gate), like(canonical.up), like(canonical.down))
    ws = torch.empty(256, dtype=torch.uint8, device=canonical.up.fp4.device)
    moe_prepack_weights(d, canonical, packed, ws)
    return packed


def upload_experts(ex, d: Dims, device="cuda") -> DeviceExperts:
    """Host canonical weights (objects with gate/up/down, each fp4/e8m0/blk numpy
    arrays) -> packed device weights."""
    canon = DeviceExperts(None if ex.gate is None else upload_matrix(ex.gate, device), upload_matrix(ex.up, device),
                          upload_matrix(ex.down, device))
    packed = prepack(d, canon)
    del canon
    return packed


class MoELayer:
    """Device-resident layer: packed expert weights, router and a workspace."""

    def __init__(self, H: int, I: int, E: int, topk: int, experts: DeviceExperts,
                 w_router: torch.Tensor, device="cuda", act: int = ACT_SWIGLU):
        self.H, self.I, self.E, self.topk, self.act = H, I, E, topk, act
        self.experts = experts
        self.w_router = w_router
        self.device = device
        self._ws = None

    def dims(self, T: int) -> Dims:
        return Dims(T, self.H, self.I, self.E, self.topk, self.act)

    def workspace(self, T: int) -> torch.Tensor:
        n = moe_workspace_bytes(self.dims(T))
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        return self._ws

    def forward(self, x: torch.Tensor, bias=None, mode=ROUTE_LEARNED, token_ids=None, out=None):
        """x: uint16 (bf16 bits) or bfloat16 [T][H] on the device.
        Returns (out bf16 bits [T][H], topk_ids, topk_w, expert_offsets)."""
        T = x.shape[0]
        d = self.dims(T)
        dev = self.device
        ids = torch.empty((T, self.topk), dtype=torch.int32, device=dev)
        w = torch.empty((T, self.topk), dtype=torch.float32, device=dev)
        off = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.int16, device=dev)
        moe_layer_forward(d, x, self.w_router, bias, mode, token_ids, self.experts, ids, w, off, out,
                          self.workspace(T))
        return out, ids, w, off

    def set_experts(self, experts: DeviceExperts):
        """Another version of the (packed) expert weights, e.g. after an optimizer step."""
        self.experts = experts
        self._wt = None

    def transposed_weights(self):
        """The transposed FP8 weight values (E4M3 bytes) the backward reads (made once)."""
        if getattr(self, "_wt", None) is None:
            d = self.dims(1)
            gI = 2 * self.I if self.act == ACT_SWIGLU else self.I
            wt_gu = torch.empty((self.E, self.H, gI), dtype=torch.uint8, device=self.device)
            wt_d = torch.empty((self.E, self.I, self.H), dtype=torch.uint8, device=self.device)
            moe_transpose_weights(d, self.experts, wt_gu, wt_d)
            self._wt = (wt_gu, wt_d)
        return self._wt

    def backward(self, x: torch.Tensor, dout: torch.Tensor, bias=None, mode=ROUTE_LEARNED, token_ids=None,
                 grads=None):
        """Gradients of sum(dout * out): dict(dx [T][H], dw [T][k], dWg / dWu [E][I][H], dWd [E][H][I])
        (fp32; dWg absent gate-less).  ``grads`` may hold preallocated outputs."""
        T = x.shape[0]
        d, g = self.dims(T), grads or self._gradients(T)
        wt_gu, wt_d = self.transposed_weights()
        moe_layer_backward(d, x, self.w_router, bias, mode, token_ids, self.experts, wt_gu, wt_d, dout,
                           g["dx"], g["dw"], g.get("dWg"), g["dWu"], g["dWd"], self._backward_workspace(d))
        return g

    def _gradients(self, T: int):
        dev = self.device
        gated = self.act == ACT_SWIGLU
        return dict(
            dx=torch.empty((T, self.H), dtype=torch.float32, device=dev),
            dw=torch.empty((T, self.topk), dtype=torch.float32, device=dev),
            dWu=torch.empty((self.E, self.I, self.H), dtype=torch.float32, device=dev),
            dWd=torch.empty((self.E, self.H, self.I), dtype=torch.float32, device=dev),
            **({"dWg": torch.empty((self.E, self.I, self.H), dtype=torch.float32, device=dev)} if gated else {}))

    def _backward_workspace(self, d: Dims):
        n = moe_backward_workspace_bytes(d)
        if getattr(self, "_bws", None) is None or self._bws.numel() < n:
            self._bws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        return self._bws

    def forward_routed(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, out=None):
        """The layer with the routing given (gate()'s outputs).  Returns (out bf16 bits [T][H], expert_offsets)."""
        T = x.shape[0]
        off = torch.empty(self.E + 1, dtype=torch.int32, device=self.device)
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.int16, device=self.device)
        moe_routed_forward(self.dims(T), x, topk_ids, topk_w, self.experts, off, out, self.workspace(T))
        return out, off

    def backward_routed(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, dout: torch.Tensor,
                        grads=None):
        """backward() with the routing given; its dw is what gate_backward() takes."""
        T = x.shape[0]
        d, g = self.dims(T), grads or self._gradients(T)
        wt_gu, wt_d = self.transposed_weights()
        moe_routed_backward(d, x, topk_ids, topk_w, self.experts, wt_gu, wt_d, dout, g["dx"], g["dw"], g.get("dWg"),
                            g["dWu"], g["dWd"], self._backward_workspace(d))
        return g

    def forward_unfused(self, x: torch.Tensor, bias=None, mode=ROUTE_LEARNED, token_ids=None):
        """The same layer through the four separate entry points."""
        T = x.shape[0]
        d = self.dims(T)
        dev = self.device
        P = T * self.topk
        ids = torch.empty((T, self.topk), dtype=torch.int32, device=dev)
        w = torch.empty((T, self.topk), dtype=torch.float32, device=dev)
        off = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        sp = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
        pp = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
        xq = torch.empty((max(T, 1), self.H), dtype=torch.uint8, device=dev)
        xs = torch.empty((max(T, 1), self.H // 128), dtype=torch.float32, device=dev)
        y = torch.empty((max(P, 1), self.H), dtype=torch.int16, device=dev)
        out = torch.empty((T, self.H), dtype=torch.int16, device=dev)
        ws = self.workspace(T)
        moe_route(d, x, self.w_router, bias, mode, token_ids, ids, w, ws)
        moe_permute(d, x, ids, off, sp, pp, xq, xs, ws)
        moe_expert_ffn(d, xq, xs, off, sp, self.experts, y, ws)
        moe_combine(d, y, w, out)
        return dict(out=out, ids=ids, w=w, offsets=off, sorted_pair=sp[:P], pair_pos=pp[:P],
                    xq=xq[:T], xs=xs[:T], y=y[:P])
