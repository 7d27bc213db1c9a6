"""ctypes binding of libq4.so (include/q4.h).

Argument marshalling only: every step of quantization, dequantization and the
fused matmuls runs in the library's sm_100a kernels.  torch supplies device
memory (the state buffers, outputs and workspaces are torch tensors) and the
current CUDA stream.  There is no CPU fallback: without the built library or
without a B200 every op raises Q4Error.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4.so")

NF4, INT4_SYM, INT4_ASYM = 0, 1, 2
SCALE_F16 = 0x100  # OR into an INT4 qtype: binary16 group scales
F16, BF16, F32 = 0, 1, 2
QTYPES = {"nf4": NF4, "int4_sym": INT4_SYM, "int4_asym": INT4_ASYM}
_DT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_DT_INV = {v: k for k, v in _DT.items()}
_DT16 = (torch.float16, torch.bfloat16)
DQ_GROUP = 256
INT8_MAX_K = 131071  # Q4_INT8_MAX_K


class Q4Error(RuntimeError):
    pass


class _CState(ctypes.Structure):
    _fields_ = [("qtype", ctypes.c_int32), ("src_dtype", ctypes.c_int32), ("n", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("blocksize", ctypes.c_int32), ("double_quant", ctypes.c_int32),
                ("dq_group", ctypes.c_int32), ("scale_f16", ctypes.c_int32),
                ("packed", ctypes.c_void_p), ("absmax", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("absmax_q", ctypes.c_void_p), ("absmax_scale", ctypes.c_void_p),
                ("absmax_mean", ctypes.c_void_p)]


class _CKVCache(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("blocksize", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages", ctypes.c_int64), ("k_codes", ctypes.c_void_p),
                ("k_state", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("v_state", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()


def library():
    """Load libq4.so (built in-tree by ``bit_blockwise_weight_absmax_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise Q4Error(f"{LIB_PATH} is not built: run `python -m "
                          "bit_blockwise_weight_absmax_b200.build` (needs nvcc)")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        SP = ctypes.POINTER(_CState)
        sig = {
            "q4_state_sizes": ([i32, i64, i32, i32, ctypes.POINTER(sz)], i32),
            "q4_quantize_workspace_size": ([i32, i64, i32, i32, ctypes.POINTER(sz)], i32),
            "q4_quantize": ([P, i32, i64, i64, i32, i32, i32, SP, P, sz, P], i32),
            "q4_quantize_grouped_workspace_size": ([i32, ctypes.POINTER(i64), ctypes.POINTER(i64), i32, i32, i32,
                                                    ctypes.POINTER(sz)], i32),
            "q4_quantize_grouped": ([i32, ctypes.POINTER(P), i32, ctypes.POINTER(i64), ctypes.POINTER(i64), i32, i32,
                                     i32, ctypes.POINTER(SP), P, sz, P], i32),
            "q4_dequantize": ([SP, P, i32, P], i32),
            "q4_dequantize_grouped": ([i32, ctypes.POINTER(SP), ctypes.POINTER(P), i32, P], i32),
            "q4_gemv_workspace_size": ([i32, ctypes.POINTER(SP), i64, ctypes.POINTER(sz)], i32),
            "q4_gemv": ([P, i32, i64, SP, P, i32, P, sz, P], i32),
            "q4_gemv_grouped": ([i32, ctypes.POINTER(P), ctypes.POINTER(SP), ctypes.POINTER(P), i64,
                                 i32, i32, P, sz, P], i32),
            "q4_gemm_workspace_size": ([i32, ctypes.POINTER(SP), i64, ctypes.POINTER(ctypes.c_size_t)], i32),
            "q4_gemm_plan_info": ([i32, ctypes.POINTER(SP), i64, i32, ctypes.c_size_t, ctypes.POINTER(i32),
                                   ctypes.POINTER(i32), ctypes.POINTER(i64)], i32),
            "q4_gemm": ([P, i32, i64, SP, P, i32, P, ctypes.c_size_t, P], i32),
            "q4_gemm_grouped": ([i32, ctypes.POINTER(P), ctypes.POINTER(SP), ctypes.POINTER(P), i64,
                                 i32, i32, P, ctypes.c_size_t, P], i32),
            "q4_int8_quantize_rows": ([P, i32, i64, i64, i64, P, i64, P, P], i32),
            "q4_int8_quantize_rows_f32": ([P, i64, i64, i64, P, i64, P, P], i32),
            "q4_int8_gemm_workspace_size": ([i64, i64, i64, ctypes.POINTER(sz)], i32),
            "q4_int8_gemm": ([P, i64, P, i64, P, i64, P, i64, i64, P, i32, P, i64, i32, P, sz, P], i32),
            "q4_int8_linear_scratch_size": ([i64, i64, ctypes.POINTER(sz)], i32),
            "q4_int8_linear": ([P, i32, i64, i64, P, i64, P, i64, i64, P, i32, P, i64, i32, P, sz, P, sz, P], i32),
            "q4_kv_append": ([ctypes.POINTER(_CKVCache), P, P, i32, i64, i64, i64, i64, i64, P, P], i32),
            "q4_kv_dequantize": ([ctypes.POINTER(_CKVCache), P, i64, P, P, i32, P], i32),
            "q4_kv_attention_workspace_size": ([ctypes.POINTER(_CKVCache), i64, i64, i32, ctypes.POINTER(sz)], i32),
            "q4_kv_attention": ([ctypes.POINTER(_CKVCache), P, i32, i64, i32, i64, i64, P, P, P, i64, i64, i64, i64,
                                 ctypes.c_float, i32, i64, P, P, P, sz, P], i32),
            "q4_device_status": ([ctypes.POINTER(i32)], i32),
            "q4_clear_device_status": ([], i32),
            "q4_set_wait_limit_ns": ([ctypes.c_uint64], i32),
            "q4_set_copy_stall": ([i32], i32),
            "q4_check_device": ([], i32),
            "q4_nf4_levels": ([ctypes.POINTER(ctypes.c_float)], i32),
            "q4_nf4_thresholds": ([ctypes.POINTER(ctypes.c_float)], i32),
            "q4_strerror": ([i32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = library().q4_strerror(rc).decode()
        raise Q4Error(f"{what}: {msg} (code {rc})")


def _require_gpu(t: torch.Tensor | None = None):
    if not torch.cuda.is_available():
        raise Q4Error("no CUDA device: libq4 has no CPU fallback")
    if t is not None and not t.is_cuda:
        raise Q4Error("tensor must be on a CUDA device")
    _check(library().q4_check_device(), "q4_check_device")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ state ----

@dataclass
class Q4State:
    """A quantized weight [rows, cols] and its device buffers (torch tensors)."""
    qtype: int
    src_dtype: torch.dtype
    rows: int
    cols: int
    blocksize: int
    double_quant: bool
    packed: torch.Tensor
    absmax: torch.Tensor | None  # with double quantization no consumer reads it
    zero: torch.Tensor | None = None
    absmax_q: torch.Tensor | None = None
    absmax_scale: torch.Tensor | None = None
    absmax_mean: torch.Tensor | None = None
    scale_f16: bool = False  # INT4: absmax holds binary16 scales

    @property
    def n(self) -> int:
        return self.rows * self.cols

    @property
    def device(self):
        return self.packed.device

    def c_struct(self) -> _CState:
        """The C view of the state, built once and rebuilt only when a buffer
        or a field has changed."""
        key = (self.qtype, self.src_dtype, self.rows, self.cols, self.blocksize, self.double_quant, self.scale_f16,
               self.packed.data_ptr(), None if self.absmax is None else self.absmax.data_ptr(),
               None if self.zero is None else self.zero.data_ptr(),
               None if self.absmax_q is None else self.absmax_q.data_ptr(),
               None if self.absmax_scale is None else self.absmax_scale.data_ptr(),
               None if self.absmax_mean is None else self.absmax_mean.data_ptr())
        cached = self.__dict__.get("_cs")
        if cached is not None and cached[0] == key:
            return cached[1]
        s = self._build_c_struct()
        self.__dict__["_cs"] = (key, s)
        return s

    def _build_c_struct(self) -> _CState:
        s = _CState()
        s.qtype = self.qtype
        s.src_dtype = _DT[self.src_dtype]
        s.n = self.n
        s.rows = self.rows
        s.cols = self.cols
        s.blocksize = self.blocksize
        s.double_quant = int(self.double_quant)
        s.dq_group = DQ_GROUP
        s.scale_f16 = int(self.scale_f16)
        s.packed = self.packed.data_ptr()
        s.absmax = None if self.absmax is None else self.absmax.data_ptr()
        s.zero = None if self.zero is None else self.zero.data_ptr()
        s.absmax_q = None if self.absmax_q is None else self.absmax_q.data_ptr()
        s.absmax_scale = None if self.absmax_scale is None else self.absmax_scale.data_ptr()
        s.absmax_mean = None if self.absmax_mean is None else self.absmax_mean.data_ptr()
        return s

    def release_absmax(self):
        """Drop the fp32 block absmax of a double-quantized state: the
        consumers read the 8-bit codes, their scales and the mean instead, so
        the fp32 copy (0.5 bit per weight at blocksize 64) is only needed to
        inspect the state."""
        if not self.double_quant:
            raise Q4Error("the fp32 absmax is the block scale of a state without double quantization")
        self.absmax = None

    def held_bytes(self) -> int:
        """Device bytes of every buffer the state still holds."""
        return sum(t.numel() * t.element_size() for t in (self.packed, self.absmax, self.zero, self.absmax_q,
                                                         self.absmax_scale, self.absmax_mean) if t is not None)

    def resident_bytes(self) -> int:
        """Bytes of the format a consumer reads (codes + block state); with
        double quantization the fp32 absmax kept for inspection is excluded."""
        b = self.packed.numel()
        if self.double_quant:
            b += self.absmax_q.numel() + 4 * self.absmax_scale.numel() + 4
        else:
            b += self.absmax.numel() * self.absmax.element_size()
            if self.zero is not None:
                b += self.zero.numel()
        return b


def state_sizes(qtype, n: int, blocksize: int, double_quant: bool) -> tuple:
    qt = QTYPES[qtype] if isinstance(qtype, str) else int(qtype)
    out = (ctypes.c_size_t * 6)()
    _check(library().q4_state_sizes(qt, n, blocksize, int(double_quant), out), "q4_state_sizes")
    return tuple(out)


def nf4_levels() -> list:
    out = (ctypes.c_float * 16)()
    _check(library().q4_nf4_levels(out), "q4_nf4_levels")
    return list(out)


def nf4_thresholds() -> list:
    out = (ctypes.c_float * 15)()
    _check(library().q4_nf4_thresholds(out), "q4_nf4_thresholds")
    return list(out)


def last_device_status() -> int:
    v = ctypes.c_int32(0)
    _check(library().q4_device_status(ctypes.byref(v)), "q4_device_status")
    return v.value


def clear_device_status():
    _check(library().q4_clear_device_status(), "q4_clear_device_status")


def set_wait_limit_ns(ns: int):
    """Bound (ns) of every device-side wait of later launches; 0 = default 2 s."""
    _check(library().q4_set_wait_limit_ns(int(ns)), "q4_set_wait_limit_ns")


def set_copy_stall(on: bool):
    """Test hook: while on, the kernels with copy pipelines (GEMV, GEMM, grouped
    quantize, int8 GEMM, cache attention) bring in no operands, so their stage
    waits run out after the wait limit (Q4_STATUS_TIMEOUT)."""
    _check(library().q4_set_copy_stall(int(bool(on))), "q4_set_copy_stall")


def reset_workspaces():
    """Zero-fill every cached workspace again (needed after a call ended with
    Q4_STATUS_TIMEOUT, which leaves its workspace undefined)."""
    for t in _ws.values():
        t.zero_()


# -------------------------------------------------------------- workspaces --
# Workspaces must start zero-filled; every call leaves them zeroed again, so
# one buffer per (device, kind) is reused.  Calls on different streams that
# overlap in time must not share a workspace.
_ws: dict = {}


def _workspace(device, kind: str, nbytes: int) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    key = (device.index if device.index is not None else torch.cuda.current_device(), kind)
    t = _ws.get(key)
    if t is None or t.numel() < nbytes:
        t = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws[key] = t
    return t


# ------------------------------------------------------------------- ops ----

def quantize(W: torch.Tensor, blocksize: int = 64, qtype="nf4", double_quant: bool = False,
             stream=None, out: Q4State | None = None, scale_f16: bool = False) -> Q4State:
    """Blockwise 4-bit quantization of a 2-D fp16/bf16 CUDA tensor.

    `out` reuses the buffers of an earlier state of the same shape and format
    (no allocation: the call can be captured in a CUDA graph).  scale_f16
    (INT4 only): binary16 group scales, the codes taken against them."""
    _require_gpu(W)
    if W.dtype not in (torch.float16, torch.bfloat16) or W.dim() != 2:
        raise Q4Error("W must be a 2-D float16/bfloat16 tensor")
    W = W.contiguous()
    qt = QTYPES[qtype] if isinstance(qtype, str) else int(qtype)
    qt_arg = qt | (SCALE_F16 if scale_f16 else 0)
    rows, cols = W.shape
    n = rows * cols
    dev = W.device
    if out is not None:
        if (out.qtype, out.rows, out.cols, out.blocksize, out.double_quant, out.scale_f16) != \
                (qt, rows, cols, blocksize, bool(double_quant), bool(scale_f16)):
            raise Q4Error("out= state has a different shape or format")
        if out.absmax is None:
            raise Q4Error("out= state has released its absmax buffer, which quantize writes")
        out.src_dtype = W.dtype
    st = out if out is not None else _new_state(qt, W.dtype, rows, cols, blocksize, double_quant, dev, scale_f16)
    wsz = ctypes.c_size_t(0)
    _check(library().q4_quantize_workspace_size(qt_arg, n, blocksize, int(double_quant), ctypes.byref(wsz)),
           "q4_quantize_workspace_size")
    ws = _workspace(dev, "quantize", wsz.value)
    cs = st.c_struct()
    _check(library().q4_quantize(_ptr(W), _DT[W.dtype], rows, cols, blocksize, qt_arg, int(double_quant),
                                 ctypes.byref(cs), _ptr(ws), 0 if ws is None else ws.numel(),
                                 _stream(stream)), "q4_quantize")
    return st


def _new_state(qt, dtype, rows, cols, blocksize, double_quant, dev, scale_f16=False) -> Q4State:
    sz = state_sizes(qt | (SCALE_F16 if scale_f16 else 0), rows * cols, blocksize, double_quant)
    return Q4State(qt, dtype, rows, cols, blocksize, bool(double_quant),
                   packed=torch.empty(sz[0], dtype=torch.uint8, device=dev),
                   absmax=(torch.empty(sz[1] // 2, dtype=torch.float16, device=dev) if scale_f16 else
                           torch.empty(sz[1] // 4, dtype=torch.float32, device=dev)),
                   zero=torch.empty(sz[2], dtype=torch.uint8, device=dev) if sz[2] else None,
                   absmax_q=torch.empty(sz[3], dtype=torch.int8, device=dev) if sz[3] else None,
                   absmax_scale=torch.empty(sz[4] // 4, dtype=torch.float32, device=dev) if sz[4] else None,
                   absmax_mean=torch.empty(1, dtype=torch.float32, device=dev) if sz[5] else None,
                   scale_f16=bool(scale_f16))


def quantize_grouped(Ws, blocksize: int = 64, qtype="nf4", double_quant: bool = False, stream=None,
                     outs=None, scale_f16: bool = False) -> list:
    """Quantize several 2-D weights of one dtype and one format in one launch
    (plus one second-level launch with double quantization); the states are
    bit for bit those of quantize() on each weight.  `outs` reuses earlier
    states of the same shapes and format (no allocation)."""
    _require_gpu(Ws[0])
    qt = QTYPES[qtype] if isinstance(qtype, str) else int(qtype)
    qt_arg = qt | (SCALE_F16 if scale_f16 else 0)
    dtype = Ws[0].dtype
    for W in Ws:
        if W.dtype != dtype or W.dim() != 2 or W.dtype not in (torch.float16, torch.bfloat16):
            raise Q4Error("weights must be 2-D float16/bfloat16 tensors of one dtype")
    Ws = [W.contiguous() for W in Ws]
    dev = Ws[0].device
    if outs is None:
        outs = [_new_state(qt, dtype, W.shape[0], W.shape[1], blocksize, double_quant, dev, scale_f16)
                for W in Ws]
    else:
        for st, W in zip(outs, Ws):
            if (st.qtype, st.rows, st.cols, st.blocksize, st.double_quant, st.scale_f16) != \
                    (qt, W.shape[0], W.shape[1], blocksize, bool(double_quant), bool(scale_f16)) \
                    or st.absmax is None:
                raise Q4Error("outs= states have a different shape or format")
            st.src_dtype = dtype
    n = len(Ws)
    rows = (ctypes.c_int64 * n)(*[W.shape[0] for W in Ws])
    cols = (ctypes.c_int64 * n)(*[W.shape[1] for W in Ws])
    wsz = ctypes.c_size_t(0)
    _check(library().q4_quantize_grouped_workspace_size(n, rows, cols, blocksize, qt_arg, int(double_quant),
                                                         ctypes.byref(wsz)), "q4_quantize_grouped_workspace_size")
    ws = _workspace(dev, "quantize", wsz.value)
    structs = [st.c_struct() for st in outs]
    arr = _struct_array(structs)
    wp = (ctypes.c_void_p * n)(*[W.data_ptr() for W in Ws])
    _check(library().q4_quantize_grouped(n, wp, _DT[dtype], rows, cols, blocksize, qt_arg, int(double_quant), arr,
                                         _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "q4_quantize_grouped")
    return outs


def dequantize(st: Q4State, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    _require_gpu(st.packed)
    dtype = dtype or st.src_dtype
    if out is None:
        out = torch.empty(st.rows, st.cols, dtype=dtype, device=st.device)
    cs = st.c_struct()
    _check(library().q4_dequantize(ctypes.byref(cs), _ptr(out), _DT[dtype], _stream(stream)),
           "q4_dequantize")
    return out


def dequantize_grouped(states, dtype: torch.dtype | None = None, outs=None, stream=None) -> list:
    """q4.dequantize of several states of one format in one launch."""
    _require_gpu(states[0].packed)
    dtype = dtype or states[0].src_dtype
    if outs is None:
        outs = [torch.empty(st.rows, st.cols, dtype=dtype, device=st.device) for st in states]
    structs = [st.c_struct() for st in states]
    n = len(states)
    arr = _struct_array(structs)
    op = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    _check(library().q4_dequantize_grouped(n, arr, op, _DT[dtype], _stream(stream)), "q4_dequantize_grouped")
    return outs


_gemv_ws_need = {}  # (shapes and formats of the group, M) -> workspace bytes


_struct_arrays = {}


def _struct_array(structs):
    """The C array of pointers to these state structs, built once per tuple
    of structs (c_struct() returns the same object while a state is
    unchanged; the cache holds the structs, so their ids stay theirs)."""
    key = tuple(id(s) for s in structs)
    hit = _struct_arrays.get(key)
    if hit is not None:
        return hit[1]
    arr = (ctypes.POINTER(_CState) * len(structs))(*[ctypes.pointer(s) for s in structs])
    if len(_struct_arrays) >= 256:
        _struct_arrays.clear()
    _struct_arrays[key] = (tuple(structs), arr)
    return arr


def _gemv_workspace(states, structs, M, device):
    arr = _struct_array(structs)
    key = (tuple((s.rows, s.cols, s.blocksize, s.qtype, s.double_quant) for s in states), M)
    need = _gemv_ws_need.get(key)
    if need is None:
        n = ctypes.c_size_t(0)
        _check(library().q4_gemv_workspace_size(len(structs), arr, M, ctypes.byref(n)),
               "q4_gemv_workspace_size")
        need = _gemv_ws_need[key] = n.value
    return arr, _workspace(device, "gemv", need)


def gemv_grouped(As, states, out_dtype: torch.dtype | None = None, outs=None, stream=None):
    """Y_i = A_i . W^_i^T for each i in one launch; A_i [M, K_i], 1 <= M <= 32."""
    _require_gpu(As[0])
    M = As[0].shape[0]
    a_dtype = As[0].dtype
    out_dtype = out_dtype or a_dtype
    structs = [s.c_struct() for s in states]
    arr, ws = _gemv_workspace(states, structs, M, As[0].device)
    if outs is None:
        outs = [torch.empty(M, s.rows, dtype=out_dtype, device=As[0].device) for s in states]
    a_ptrs = (ctypes.c_void_p * len(As))(*[a.data_ptr() for a in As])
    y_ptrs = (ctypes.c_void_p * len(As))(*[y.data_ptr() for y in outs])
    for a, s in zip(As, states):
        if a.dtype != a_dtype or a.shape != (M, s.cols) or not a.is_contiguous():
            raise Q4Error("activations must be contiguous [M, K] of one dtype")
    _check(library().q4_gemv_grouped(len(As), a_ptrs, arr, y_ptrs, M, _DT[a_dtype], _DT[out_dtype],
                                     _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "q4_gemv_grouped")
    return outs


def gemv(A: torch.Tensor, st: Q4State, out_dtype: torch.dtype | None = None, out=None,
         stream=None) -> torch.Tensor:
    return gemv_grouped([A], [st], out_dtype, None if out is None else [out], stream)[0]


def gemm_grouped(As, states, out_dtype: torch.dtype | None = None, outs=None, stream=None):
    """Y_i = A_i . W^_i^T for each i, tcgen05 W4A16 GEMM, one persistent launch."""
    _require_gpu(As[0])
    M = As[0].shape[0]
    a_dtype = As[0].dtype
    out_dtype = out_dtype or a_dtype
    structs = [s.c_struct() for s in states]
    arr = _struct_array(structs)
    if outs is None:
        outs = [torch.empty(M, s.rows, dtype=out_dtype, device=As[0].device) for s in states]
    for a, s in zip(As, states):
        if a.dtype != a_dtype or a.shape != (M, s.cols) or not a.is_contiguous():
            raise Q4Error("activations must be contiguous [M, K] of one dtype")
    a_ptrs = (ctypes.c_void_p * len(As))(*[a.data_ptr() for a in As])
    y_ptrs = (ctypes.c_void_p * len(As))(*[y.data_ptr() for y in outs])
    # the workspace that lets the launch cut tiles in k where that evens out
    # the CTAs' work (cached per device; zero-filled, left zeroed)
    wsz = ctypes.c_size_t(0)
    _check(library().q4_gemm_workspace_size(len(As), arr, M, ctypes.byref(wsz)), "q4_gemm_workspace_size")
    ws = _workspace(As[0].device, "gemm", wsz.value)
    _check(library().q4_gemm_grouped(len(As), a_ptrs, arr, y_ptrs, M, _DT[a_dtype], _DT[out_dtype],
                                     _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "q4_gemm_grouped")
    return outs


def gemm(A: torch.Tensor, st: Q4State, out_dtype: torch.dtype | None = None, out=None,
         stream=None) -> torch.Tensor:
    return gemm_grouped([A], [st], out_dtype, None if out is None else [out], stream)[0]


# ------------------------------------------- 8-bit integers and the KV cache --
# These calls run on the device and the current stream of their tensors'
# device (or on `stream`); what they allocate belongs to that stream.  Their
# workspaces are one per device, kind and stream; a call that is captured into
# a CUDA graph takes a workspace of its own, so graphs share none.

def _elsewhere(t: torch.Tensor, stream):
    """None when t's device is current and no stream is given; otherwise the
    context that makes them current, under which the caller calls itself."""
    if stream is None and t.is_cuda and t.get_device() == torch._C._cuda_getDevice():
        return None
    if not t.is_cuda:
        raise Q4Error("no CUDA device: libq4 has no CPU fallback" if not torch.cuda.is_available()
                      else "tensor must be on a CUDA device")
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise Q4Error(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _current_stream(t: torch.Tensor) -> int:
    """The handle of the current stream of t's device (torch.cuda.current_stream
    builds an object for it, at 3 us a call)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


WORKSPACE_HEAD = 16384  # Q4_WORKSPACE_HEAD: the part of a workspace that starts zero-filled


def _stream_workspace(device, stream: int, nbytes: int):
    """(pointer, bytes, owner) of the current stream's workspace."""
    if nbytes == 0:
        return None, 0, None
    if torch._C._cuda_isCurrentStreamCapturing():
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
        t[:WORKSPACE_HEAD].zero_()
        return t.data_ptr(), nbytes, t
    key = (device.index, "stream", stream)
    t = _ws.get(key)
    if t is None or t.numel() < nbytes:
        t = _ws[key] = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    return t.data_ptr(), t.numel(), t


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise Q4Error(f"{name} is on {t.device}, expected {dev}")


def _rows16(x: torch.Tensor, name: str) -> torch.Tensor:
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise Q4Error(f"{name} must be float16 or bfloat16, got {x.dtype}")
    return x


def int8_quantize_rows(X: torch.Tensor, stream=None) -> tuple:
    """(codes, scale) of a 2-D fp16/bf16/fp32 tensor: symmetric 8-bit codes with
    one scale per row, X ~ codes * scale[:, None].  For a weight [N, K] (a
    scale per output channel, once at load time) or for activations [M, K] (a
    scale per token).  The code rows are padded to a multiple of 16 bytes:
    codes is a [rows, K] view of that buffer."""
    if X.dtype not in _DT:
        raise Q4Error(f"X must be float16, bfloat16 or float32, got {X.dtype}")
    if X.dim() != 2:
        raise Q4Error("X must be 2-D")
    rows, K = X.shape
    if K < 1:
        raise Q4Error("X has no columns")
    ctx = _elsewhere(X, stream)
    if ctx is not None:
        with ctx:
            return int8_quantize_rows(X)
    if X.stride(1) != 1 and K > 1 or rows > 1 and X.stride(0) < K:
        X = X.contiguous()
    ldc = (K + 15) // 16 * 16
    codes = torch.empty(rows, ldc, dtype=torch.int8, device=X.device)[:, :K]
    scale = torch.empty(rows, dtype=torch.float32, device=X.device)
    if rows:
        ldx, s = max(X.stride(0), K), _current_stream(X)
        if X.dtype == torch.float32:
            _check(library().q4_int8_quantize_rows_f32(X.data_ptr(), rows, K, ldx, codes.data_ptr(), ldc,
                                                       scale.data_ptr(), s), "q4_int8_quantize_rows_f32")
        else:
            _check(library().q4_int8_quantize_rows(X.data_ptr(), _DT[X.dtype], rows, K, ldx, codes.data_ptr(), ldc,
                                                   scale.data_ptr(), s), "q4_int8_quantize_rows")
    return codes, scale


def _check_codes(name, codes, scale):
    """The row stride of int8 [rows, K] codes with float32 [rows] scales."""
    cs, ss = codes.shape, scale.shape
    if codes.dtype != torch.int8 or len(cs) != 2 or scale.dtype != torch.float32 or len(ss) != 1:
        raise Q4Error(f"{name} must be int8 [rows, K] codes with float32 [rows] scales")
    if ss[0] != cs[0] or not scale.is_contiguous():
        raise Q4Error(f"{name}: one contiguous scale per row is needed")
    ld, one = codes.stride()
    if one != 1 or ld & 15 or ld < cs[1] or codes.data_ptr() & 15:
        raise Q4Error(f"{name}: code rows must be adjacent bytes that begin at multiples of 16 bytes "
                      "(as int8_quantize_rows gives them)")
    return ld


def _check_bias_out(bias, out, M, N, out_dtype, dev):
    if bias is not None and (bias.shape != (N,) or bias.dtype not in _DT or not bias.is_contiguous()):
        raise Q4Error(f"bias must be a contiguous float tensor of {N} elements")
    if out is None:
        return torch.empty(M, N, dtype=out_dtype, device=dev)
    if out.shape != (M, N) or out.dtype != out_dtype or out.stride(1) != 1 or out.stride(0) < N:
        raise Q4Error(f"out must be {out_dtype} [{M}, {N}] with adjacent elements")
    return out


_int8_ws_need = {}  # (M, N, K, device) -> workspace bytes of the product, scratch bytes of the linear layer


def _int8_ws_sizes(M, N, K, device):
    key = (M, N, K, device.index)
    need = _int8_ws_need.get(key)
    if need is None:
        a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
        _check(library().q4_int8_gemm_workspace_size(M, N, K, ctypes.byref(a)), "q4_int8_gemm_workspace_size")
        _check(library().q4_int8_linear_scratch_size(M, K, ctypes.byref(b)), "q4_int8_linear_scratch_size")
        if len(_int8_ws_need) >= 4096:
            _int8_ws_need.clear()
        need = _int8_ws_need[key] = (a.value, b.value)
    return need


def int8_gemm(A: torch.Tensor, a_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
              bias: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float16, out=None,
              stream=None) -> torch.Tensor:
    """Y = (A . W^T) * a_scale[:, None] * w_scale[None, :] + bias from 8-bit
    codes A [M, K] and W [N, K] (see int8_quantize_rows): exact 32-bit integer
    sums, one rounding to out_dtype (fp16, bf16 or fp32)."""
    _check_codes("A", A, a_scale)
    _check_codes("W", W, w_scale)
    (M, K), N = A.shape, W.shape[0]
    if W.shape[1] != K:
        raise Q4Error(f"A has {K} columns, W {W.shape[1]}")
    if out_dtype not in _DT:
        raise Q4Error(f"out_dtype {out_dtype} is not float16, bfloat16 or float32")
    _same_device(A.device, a_scale=a_scale, W=W, w_scale=w_scale, bias=bias, out=out)
    ctx = _elsewhere(A, stream)
    if ctx is not None:
        with ctx:
            return int8_gemm(A, a_scale, W, w_scale, bias, out_dtype, out)
    y = _check_bias_out(bias, out, M, N, out_dtype, A.device)
    if M and N:
        s = _current_stream(A)
        ws, ws_bytes, _ = _stream_workspace(A.device, s, _int8_ws_sizes(M, N, K, A.device)[0])
        _check(library().q4_int8_gemm(
            A.data_ptr(), A.stride(0), a_scale.data_ptr(), M, W.data_ptr(), W.stride(0), w_scale.data_ptr(), N, K,
            None if bias is None else bias.data_ptr(), 0 if bias is None else _DT[bias.dtype], y.data_ptr(),
            max(y.stride(0), N), _DT[out_dtype], ws, ws_bytes, s), "q4_int8_gemm")
    return y


def int8_linear(X: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
                out_dtype: torch.dtype | None = None, out=None, stream=None) -> torch.Tensor:
    """Y = X . W^T + bias with 16-bit activations X [M, K], quantized per token
    on the way, and 8-bit weights (see int8_quantize_rows): int8_gemm of
    int8_quantize_rows(X), in one call."""
    _rows16(X, "X")
    _check_codes("W", W, w_scale)
    if X.dim() != 2 or X.shape[1] != W.shape[1]:
        raise Q4Error(f"X must be [M, {W.shape[1]}], got {tuple(X.shape)}")
    (M, K), N = X.shape, W.shape[0]
    out_dtype = out_dtype or X.dtype
    if out_dtype not in _DT:
        raise Q4Error(f"out_dtype {out_dtype} is not float16, bfloat16 or float32")
    _same_device(X.device, W=W, w_scale=w_scale, bias=bias, out=out)
    ctx = _elsewhere(X, stream)
    if ctx is not None:
        with ctx:
            return int8_linear(X, W, w_scale, bias, out_dtype, out)
    if X.stride(1) != 1 and K > 1 or M > 1 and X.stride(0) < K:
        X = X.contiguous()
    y = _check_bias_out(bias, out, M, N, out_dtype, X.device)
    if M and N:
        s = _current_stream(X)
        need, scratch_need = _int8_ws_sizes(M, N, K, X.device)
        ws, ws_bytes, _ = _stream_workspace(X.device, s, need)
        scratch = torch.empty(scratch_need, dtype=torch.uint8, device=X.device) if scratch_need else None
        _check(library().q4_int8_linear(
            X.data_ptr(), _DT[X.dtype], max(X.stride(0), K), M, W.data_ptr(), W.stride(0), w_scale.data_ptr(), N, K,
            None if bias is None else bias.data_ptr(), 0 if bias is None else _DT[bias.dtype], y.data_ptr(),
            max(y.stride(0), N), _DT[out_dtype], None if scratch is None else scratch.data_ptr(), scratch_need, ws,
            ws_bytes, s), "q4_int8_linear")
    return y


@dataclass
class KVCache:
    """A paged key/value cache in 4 bits (its four device buffers; the format
    is that of q4_kv_cache in include/q4.h).  codes: uint8 [pages, kv_heads,
    page_size, head_dim / 2]; state: float16 [pages, kv_heads, page_size,
    head_dim / blocksize, 2], the pairs (scale, zero-point)."""
    k_codes: torch.Tensor
    k_state: torch.Tensor
    v_codes: torch.Tensor
    v_state: torch.Tensor

    def __post_init__(self):
        c, st = self.k_codes, self.k_state
        if c.dim() != 4 or st.dim() != 5 or st.shape[-1] != 2 or st.shape[:3] != c.shape[:3] or not st.shape[3] \
                or 2 * c.shape[3] % st.shape[3]:
            raise Q4Error("codes must be [pages, heads, page_size, head_dim / 2], states [pages, heads, page_size, "
                          "head_dim / blocksize, 2]")
        for name, t, want in (("k_codes", c, torch.uint8), ("v_codes", self.v_codes, torch.uint8),
                              ("k_state", st, torch.float16), ("v_state", self.v_state, torch.float16)):
            if t.dtype != want or not t.is_contiguous() or t.device != c.device or \
                    t.shape != (c if want == torch.uint8 else st).shape:
                raise Q4Error(f"{name} must be a contiguous {want} tensor like its partners")
        # asked for on every call, so plain attributes
        put = lambda name, value: object.__setattr__(self, name, value)
        put("device", c.device)
        put("pages", c.shape[0])
        put("kv_heads", c.shape[1])
        put("page_size", c.shape[2])
        put("head_dim", 2 * c.shape[3])
        put("blocksize", self.head_dim // st.shape[3])
        s = _CKVCache(self.head_dim, self.blocksize, self.kv_heads, self.page_size, self.pages, c.data_ptr(),
                      st.data_ptr(), self.v_codes.data_ptr(), self.v_state.data_ptr())
        put("_c", s)
        put("_ref", ctypes.byref(s))
        put("_ws_need", {})  # (batch, rows, query heads) -> workspace bytes of attention
        put("_fixed", True)

    def __setattr__(self, name, value):
        if "_fixed" in self.__dict__:
            raise Q4Error("the buffers of a KVCache are fixed: make a new one")
        object.__setattr__(self, name, value)

    def held_bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.k_state, self.v_codes, self.v_state))


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, blocksize: int = 64,
             device="cuda") -> KVCache:
    """Allocate a cache of pages * page_size tokens (head_dim 64 or 128;
    blocksize 64 or 128, a divisor of it; page_size 16, 32, 64, 128 or 256)."""
    if head_dim not in (64, 128) or blocksize not in (64, 128) or head_dim % blocksize:
        raise Q4Error(f"head_dim {head_dim} with blocksize {blocksize}: head_dim must be 64 or 128, blocksize 64 or 128 "
                      "and a divisor of it")
    if page_size not in (16, 32, 64, 128, 256):
        raise Q4Error(f"page_size {page_size} is not 16, 32, 64, 128 or 256")
    if pages < 1 or kv_heads < 1:
        raise Q4Error("a cache needs at least one page and one head")
    c = torch.empty(2, pages, kv_heads, page_size, head_dim // 2, dtype=torch.uint8, device=device)
    s = torch.empty(2, pages, kv_heads, page_size, head_dim // blocksize, 2, dtype=torch.float16, device=device)
    return KVCache(c[0], s[0], c[1], s[1])


def _head_rows(x: torch.Tensor, heads, dim: int, name: str):
    """x as [rows, heads, dim] with strides the kernels read (a copy if its own
    are not), its shape, its token and head strides."""
    shape, st = x.shape, x.stride()
    if x.dtype not in _DT16 or len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise Q4Error(f"{name} must be float16 or bfloat16 [rows, {heads or 'heads'}, {dim}], got {x.dtype} "
                      f"{tuple(shape)}")
    if st[2] != 1 or st[0] & 7 or st[1] & 7 or st[0] < 0 or x.data_ptr() & 15:
        x = x.contiguous()
        if x.data_ptr() & 15:
            x = x.clone()
        st = x.stride()
    return x, shape, st[0], st[1]


def _index(t: torch.Tensor, dtype, n: int | None, name: str) -> torch.Tensor:
    """t as a contiguous 1-D tensor of n integers of dtype."""
    if t.dtype != dtype or t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise Q4Error(f"{name} must be {dtype} of {'' if n is None else n} elements, got {t.dtype} {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize keys and values [tokens, kv_heads, head_dim] (fp16 or bf16) into
    the cache at slots (int64 [tokens], page * page_size + offset; a negative
    one passes its token over).  The slots of a call are distinct."""
    ctx = _elsewhere(k, stream)
    if ctx is not None:
        with ctx:
            return kv_append(cache, k, v, slots)
    k, shape, kt, kh = _head_rows(k, cache.kv_heads, cache.head_dim, "k")
    v, v_shape, vt, vh = _head_rows(v, cache.kv_heads, cache.head_dim, "v")
    if shape != v_shape or k.dtype != v.dtype:
        raise Q4Error("k and v must have one shape and dtype")
    n = shape[0]
    slots = _index(slots, torch.int64, n, "slots")
    dev = k.device
    if v.device != dev or slots.device != dev or cache.device != dev:
        _same_device(dev, v=v, slots=slots, cache=cache)
    if n:
        _check(library().q4_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), _DT[k.dtype], n, kt, kh, vt, vh,
                                      slots.data_ptr(), _current_stream(k)), "q4_kv_append")


def kv_dequantize(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.float16, stream=None) -> tuple:
    """(k, v) [n, kv_heads, head_dim] of the given slots as 16-bit floats;
    zeros for a negative slot."""
    if dtype not in (torch.float16, torch.bfloat16):
        raise Q4Error("dtype must be float16 or bfloat16")
    ctx = _elsewhere(slots, stream)
    if ctx is not None:
        with ctx:
            return kv_dequantize(cache, slots, dtype)
    slots = _index(slots, torch.int64, None, "slots")
    _same_device(slots.device, cache=cache)
    n = slots.shape[0]
    k, v = torch.empty(2, n, cache.kv_heads, cache.head_dim, dtype=dtype, device=slots.device).unbind()
    if n:
        _check(library().q4_kv_dequantize(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _DT[dtype],
                                          _current_stream(slots)), "q4_kv_dequantize")
    return k, v


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 cu_seqlens_q: torch.Tensor | None = None, max_q: int | None = None, scale: float | None = None,
                 causal: bool = True, window: int = 0, out: torch.Tensor | None = None, return_lse: bool = False,
                 stream=None):
    """softmax(scale q k^T) v over the cached keys and values.

    q [rows, q_heads, head_dim] (fp16 or bf16; q_heads a multiple of the
    cache's heads); block_table int32 [batch, n], the page of each page_size
    keys; seq_lens int32 [batch], keys of each sequence, those of its query
    rows included.  cu_seqlens_q int32 [batch + 1]: sequence b has the rows
    cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1, its last ones; None: one row
    each (rows = batch).  max_q: the most rows of a sequence, a hint that
    chooses the kernel (default: 1 where there are as many rows as sequences,
    else the rows of the whole call).  scale: 1 /
    sqrt(head_dim) unless given.  causal: a row attends to the keys up to its
    own position; window > 0: only to the last `window` of them.  Rows that
    attend to nothing are zero, with log sum exp -inf; rows outside
    cu_seqlens_q are left as they were (pass `out` to have them defined).
    At most 65535 sequences a call.
    Returns out [rows, q_heads, head_dim], with return_lse also float32 [rows,
    q_heads], the log sum exp of the scaled scores (over long prompts it takes
    a quarter more time)."""
    ctx = _elsewhere(q, stream)
    if ctx is not None:
        with ctx:
            return kv_attention(q, cache, block_table, seq_lens, cu_seqlens_q, max_q, scale, causal, window, out, return_lse)
    dim = cache.head_dim
    q, shape, qt, qh = _head_rows(q, None, dim, "q")
    rows, heads, _ = shape
    if heads == 0 or heads % cache.kv_heads:
        raise Q4Error(f"{heads} query heads are no multiple of {cache.kv_heads} key/value heads")
    if window < 0:
        raise Q4Error("window must be 0 (none) or positive")
    seq_lens = _index(seq_lens, torch.int32, None, "seq_lens")
    batch = seq_lens.shape[0]
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != batch or \
            block_table.shape[1] < 1:
        raise Q4Error(f"block_table must be int32 [{batch}, pages], got {block_table.dtype} "
                      f"{tuple(block_table.shape)}")
    bt, one = block_table.stride()
    pages = block_table.shape[1]
    if one != 1 or bt < pages:
        block_table = block_table.contiguous()
        bt = pages
    if cu_seqlens_q is not None:
        cu_seqlens_q = _index(cu_seqlens_q, torch.int32, batch + 1, "cu_seqlens_q")
    elif rows != batch:
        raise Q4Error(f"{rows} query rows for {batch} sequences: pass cu_seqlens_q")
    dev = q.device
    if cache.device != dev or block_table.device != dev or seq_lens.device != dev or \
            (cu_seqlens_q is not None and cu_seqlens_q.device != dev) or (out is not None and out.device != dev):
        _same_device(dev, cache=cache, block_table=block_table, seq_lens=seq_lens, cu_seqlens_q=cu_seqlens_q, out=out)
    if out is None:
        out = torch.empty(rows, heads, dim, dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise Q4Error("out must be a contiguous tensor of q's shape and dtype")
    lse = torch.empty(rows, heads, dtype=torch.float32, device=dev) if return_lse else None
    if rows and batch:
        key = (batch, rows, heads)
        need = cache._ws_need.get(key)
        if need is None:
            n = ctypes.c_size_t(0)
            _check(library().q4_kv_attention_workspace_size(cache._ref, batch, rows, heads, ctypes.byref(n)),
                   "q4_kv_attention_workspace_size")
            if len(cache._ws_need) >= 4096:
                cache._ws_need.clear()
            need = cache._ws_need[key] = n.value
        s = _current_stream(q)
        ws, ws_bytes, _ = _stream_workspace(dev, s, need)
        if max_q is None:
            max_q = 1 if cu_seqlens_q is None or rows == batch else rows
        _check(library().q4_kv_attention(
            cache._ref, q.data_ptr(), _DT[q.dtype], rows, heads, qt, qh,
            None if cu_seqlens_q is None else cu_seqlens_q.data_ptr(), seq_lens.data_ptr(),
            block_table.data_ptr(), bt, pages, batch,
            max(1, max_q), 1.0 / math.sqrt(dim) if scale is None else scale, int(causal), window, out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws, ws_bytes, s), "q4_kv_attention")
    return (out, lse) if return_lse else out
