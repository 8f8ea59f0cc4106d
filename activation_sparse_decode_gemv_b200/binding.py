"""Thin ctypes binding of libpi_ffn.so (argument marshalling only).

Every step of the decode path runs in the CUDA library; this module only
passes device pointers, sizes and the current torch stream across the C ABI.
The functions keep the C names (pi_predict, pi_sparse_ffn, ...) and take
torch CUDA tensors.  If the library is missing or fails to load, every entry
point raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import List, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# PI_FFN_LIB: another build of this library (the sanitizer test's host-
# instrumented one); there is no non-CUDA implementation to fall back to
LIB_PATH = os.environ.get("PI_FFN_LIB") or os.path.join(HERE, "libpi_ffn.so")

PI_OK, PI_ERR_INVALID_ARG, PI_ERR_UNSUPPORTED, PI_ERR_MISALIGNED = 0, 1, 2, 3
PI_ERR_CUDA, PI_ERR_TIMEOUT, PI_ERR_DEVICE_STATUS, PI_ERR_WORKSPACE = 4, 5, 6, 7
PI_ACT_RELU, PI_ACT_SWIGLU = 0, 1
PI_W_F32, PI_W_F16, PI_W_INT4G32 = 0, 1, 2
PI_FFN_ACCUMULATE, PI_FFN_HOT_DENSE, PI_FFN_HOT_INDEX = 1, 2, 4
PI_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # device scratch of pi_decode_ffn_static

PI_DT_F32, PI_DT_F16, PI_DT_BF16 = 0, 1, 2
PI_GATE_SILU, PI_GATE_RELU, PI_GATE_GELU = 0, 1, 2
PI_GRAD_ACCUMULATE = 1

WTYPE = {"f32": PI_W_F32, "f16": PI_W_F16, "int4g32": PI_W_INT4G32}
ACT = {"relu": PI_ACT_RELU, "swiglu": PI_ACT_SWIGLU}
DTYPE = {torch.float32: PI_DT_F32, torch.float16: PI_DT_F16, torch.bfloat16: PI_DT_BF16}
GATE_ACT = {"silu": PI_GATE_SILU, "relu": PI_GATE_RELU, "gelu": PI_GATE_GELU}

# every symbol the header declares
EXPORTS = ("pi_ffn_create", "pi_ffn_destroy", "pi_workspace_size", "pi_workspace_init", "pi_predict",
           "pi_sparse_ffn", "pi_decode_ffn", "pi_decode_ffn_stack", "pi_decode_ffn_static", "pi_debug_wait_fault",
           "pi_get_device_status", "pi_status_string",
           "pi_gated_ffn_create", "pi_gated_ffn_destroy", "pi_gated_ffn_workspace_size", "pi_gated_ffn_forward",
           "pi_gated_ffn_backward", "pi_block_norm_forward", "pi_block_norm_workspace_size",
           "pi_block_norm_backward", "pi_quantize_i8", "pi_matmul_i8_workspace_size", "pi_matmul_i8",
           "pi_debug_dense_plan")


class PiError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class pi_ffn_desc(C.Structure):
    _fields_ = [("d_model", C.c_int), ("d_ffn", C.c_int), ("rank", C.c_int), ("act", C.c_int),
                ("wtype", C.c_int), ("ptype", C.c_int), ("hot_prefix", C.c_int), ("hot_p_mean", C.c_float),
                ("w_up", C.c_void_p), ("w_gate", C.c_void_p), ("w_down_t", C.c_void_p),
                ("s_up", C.c_void_p), ("s_gate", C.c_void_p), ("s_down_t", C.c_void_p),
                ("b_up", C.c_void_p), ("p1", C.c_void_p), ("p2", C.c_void_p), ("p_bias", C.c_void_p)]


class pi_gated_ffn_desc(C.Structure):
    _fields_ = [("d_model", C.c_int), ("d_ffn", C.c_int), ("act", C.c_int), ("dtype", C.c_int),
                ("w_gate", C.c_void_p), ("w_up", C.c_void_p), ("w_down_t", C.c_void_p)]


class pi_block_norm_desc(C.Structure):
    _fields_ = [("d_model", C.c_int), ("y_dtype", C.c_int), ("u_dtype", C.c_int), ("post_norm", C.c_int),
                ("eps", C.c_float), ("residual_scale", C.c_float), ("branch_scale", C.c_float),
                ("w_post", C.c_void_p), ("w_pre", C.c_void_p), ("gate", C.c_void_p), ("tokens_per_gate", C.c_int)]


_lib = None


def lib() -> C.CDLL:
    """Load libpi_ffn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run activation_sparse_decode_gemv_b200/build.py "
                               "(there is no non-CUDA implementation)")
        L = C.CDLL(LIB_PATH)
        vp, i, sz = C.c_void_p, C.c_int, C.c_size_t
        L.pi_ffn_create.argtypes = [C.POINTER(pi_ffn_desc), C.POINTER(vp)]
        L.pi_ffn_destroy.argtypes = [vp]
        L.pi_ffn_destroy.restype = None
        L.pi_workspace_size.argtypes = [C.POINTER(vp), i, i, C.POINTER(sz)]
        L.pi_workspace_init.argtypes = [vp, sz, vp]
        L.pi_predict.argtypes = [vp, vp, i, vp, vp, vp, sz, vp]
        L.pi_sparse_ffn.argtypes = [vp, vp, i, vp, vp, vp, C.c_uint, vp, sz, vp]
        L.pi_decode_ffn.argtypes = [vp, vp, i, vp, vp, vp, C.c_uint, vp, sz, vp]
        L.pi_decode_ffn_stack.argtypes = [C.POINTER(vp), i, vp, i, vp, vp, C.c_uint, vp, sz, vp]
        L.pi_decode_ffn_static.argtypes = [vp, vp, vp, vp, vp, C.c_uint, vp, vp]
        L.pi_debug_wait_fault.argtypes = [i, C.c_uint]
        L.pi_get_device_status.argtypes = [vp, vp, C.POINTER(i)]
        L.pi_status_string.argtypes = [i]
        L.pi_status_string.restype = C.c_char_p
        L.pi_gated_ffn_create.argtypes = [C.POINTER(pi_gated_ffn_desc), C.POINTER(vp)]
        L.pi_gated_ffn_destroy.argtypes = [vp]
        L.pi_gated_ffn_destroy.restype = None
        L.pi_gated_ffn_workspace_size.argtypes = [vp, i, i, C.POINTER(sz)]
        L.pi_gated_ffn_forward.argtypes = [vp, vp, i, vp, vp, vp, vp, sz, vp]
        L.pi_gated_ffn_backward.argtypes = [vp, vp, vp, vp, vp, i, vp, vp, vp, vp, i, C.c_uint, vp, sz, vp]
        nd = C.POINTER(pi_block_norm_desc)
        L.pi_block_norm_forward.argtypes = [nd, vp, vp, i, vp, vp, vp, vp, vp]
        L.pi_block_norm_workspace_size.argtypes = [nd, i, C.POINTER(sz)]
        L.pi_block_norm_backward.argtypes = [nd] + [vp] * 6 + [i] + [vp] * 5 + [C.c_uint, vp, sz, vp]
        L.pi_quantize_i8.argtypes = [vp, i, i, i, vp, vp, vp]
        L.pi_matmul_i8_workspace_size.argtypes = [i, i, i, C.POINTER(sz)]
        L.pi_matmul_i8.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, i, vp, sz, vp]
        L.pi_debug_dense_plan.argtypes = [i, i, i, i]
        for n in ("pi_gated_ffn_create", "pi_gated_ffn_workspace_size", "pi_gated_ffn_forward",
                  "pi_gated_ffn_backward", "pi_block_norm_forward", "pi_block_norm_workspace_size",
                  "pi_block_norm_backward", "pi_quantize_i8", "pi_matmul_i8_workspace_size", "pi_matmul_i8",
                  "pi_debug_dense_plan"):
            getattr(L, n).restype = C.c_int
        for n in ("pi_ffn_create", "pi_workspace_size", "pi_workspace_init", "pi_predict", "pi_sparse_ffn",
                  "pi_decode_ffn", "pi_decode_ffn_stack", "pi_decode_ffn_static", "pi_debug_wait_fault",
                  "pi_get_device_status"):
            getattr(L, n).restype = C.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pi_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != PI_OK:
        raise PiError(rc, what)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


# The C ABI sees only pointers, so the binding checks what it cannot: each
# tensor's dtype, size (at least the extent the header states) and
# contiguity, then that all of them are CUDA tensors.  Null pointers and
# everything the header validates are left to the library.
def _need(t: Optional[torch.Tensor], what: str, dtype: torch.dtype, min_numel: int):
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.numel() < min_numel:
        raise ValueError(f"{what}: {t.numel()} elements, the call needs at least {min_numel}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _on_device(**tensors: Optional[torch.Tensor]):
    for what, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{what}: must be a CUDA tensor")


def _c_int(n, what: str) -> int:
    """n as a C int, which ctypes would take modulo 2^32."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{what}: {n}, over 2147483647 in size")
    return n


def _tokens(u: torch.Tensor, d: int, what: str) -> int:
    """Batch size of a [B, d] token tensor."""
    shape = u.shape
    if len(shape) != 2 or shape[1] != d:
        raise ValueError(f"{what}: shape {tuple(shape)}, expected [B, {d}]")
    n = shape[0]
    return n if n < 2 ** 31 else _c_int(n, f"{what}: rows")


def _need_ws(ws: torch.Tensor):
    if not ws.is_contiguous():
        raise ValueError("workspace: must be contiguous")


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


class FfnLayer:
    """A created pi_ffn handle plus references to the tensors it borrows."""

    def __init__(self, w_up, w_down_t, p1, p2, p_bias, *, act: str, wtype: str, d: int, f: int, r: int,
                 b_up=None, w_gate=None, s_up=None, s_gate=None, s_down_t=None, hot_prefix: int = 0,
                 hot_p_mean: float = 0.0):
        self._keep = [w_up, w_down_t, p1, p2, p_bias, b_up, w_gate, s_up, s_gate, s_down_t]
        ptype = PI_W_F32 if p1.dtype == torch.float32 else PI_W_F16
        self.desc = pi_ffn_desc(d, f, r, ACT[act], WTYPE[wtype], ptype, int(hot_prefix), float(hot_p_mean),
                                _p(w_up), _p(w_gate), _p(w_down_t), _p(s_up), _p(s_gate), _p(s_down_t),
                                _p(b_up), _p(p1), _p(p2), _p(p_bias))
        self.d, self.f, self.r, self.act, self.wtype = d, f, r, act, wtype
        self.u_dtype = torch.float32 if wtype == "f32" else torch.float16  # FFN input u
        h = C.c_void_p()
        _check(lib().pi_ffn_create(C.byref(self.desc), C.byref(h)), "pi_ffn_create")
        self.handle = h

    @classmethod
    def from_tensors(cls, lt) -> "FfnLayer":
        """From an ``inputs.LayerTensors`` already on the device."""
        return cls(lt.w_up, lt.w_down_t, lt.p1, lt.p2, lt.p_bias, act=lt.cfg.act, wtype=lt.cfg.wtype, d=lt.d, f=lt.f,
                   r=lt.r, b_up=lt.b_up, w_gate=lt.w_gate, s_up=lt.s_up, s_gate=lt.s_gate, s_down_t=lt.s_down_t,
                   hot_prefix=lt.hot_prefix, hot_p_mean=lt.hot_p_mean)

    def close(self):
        if getattr(self, "handle", None):
            lib().pi_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pi_workspace_size(layers: Sequence[FfnLayer], max_batch: int) -> int:
    arr = (C.c_void_p * len(layers))(*[l.handle for l in layers])
    n = C.c_size_t()
    _check(lib().pi_workspace_size(arr, len(layers), int(max_batch), C.byref(n)), "pi_workspace_size")
    return n.value


def pi_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().pi_workspace_init(_p(ws), ws.numel() * ws.element_size(), _stream(stream)), "pi_workspace_init")


def make_workspace(layers: Sequence[FfnLayer], max_batch: int, device=None) -> torch.Tensor:
    """Allocate (with torch) and zero a workspace for these layers."""
    n = pi_workspace_size(layers, max_batch)
    ws = torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))
    pi_workspace_init(ws)
    return ws


def _wsargs(ws: torch.Tensor):
    return _p(ws), ws.numel() * ws.element_size()


def pi_predict(layer: FfnLayer, u: torch.Tensor, idx: torch.Tensor, count: torch.Tensor, ws: torch.Tensor,
               stream=None):
    """u [B, d]; idx int32 [B, f] (ascending ids, row b at b*f); count int32 [B]."""
    B = _tokens(u, layer.d, "u")
    _need(u, "u", layer.u_dtype, B * layer.d)
    _need(idx, "idx", torch.int32, B * layer.f)
    _need(count, "count", torch.int32, B)
    _need_ws(ws)
    _on_device(u=u, idx=idx, count=count, workspace=ws)
    _check(lib().pi_predict(layer.handle, _p(u), B, _p(idx), _p(count), *_wsargs(ws), _stream(stream)), "pi_predict")


def pi_sparse_ffn(layer: FfnLayer, u: torch.Tensor, idx: torch.Tensor, count: torch.Tensor, y: torch.Tensor,
                  ws: torch.Tensor, flags: int = 0, stream=None):
    """u [B, d]; idx int32 [B, f] and count int32 [B] (the sets); y fp32 [B, d]."""
    B = _tokens(u, layer.d, "u")
    _need(u, "u", layer.u_dtype, B * layer.d)
    _need(idx, "idx", torch.int32, B * layer.f)
    _need(count, "count", torch.int32, B)
    _need(y, "y", torch.float32, B * layer.d)
    _need_ws(ws)
    _on_device(u=u, idx=idx, count=count, y=y, workspace=ws)
    _check(lib().pi_sparse_ffn(layer.handle, _p(u), B, _p(idx), _p(count), _p(y), int(flags), *_wsargs(ws),
                               _stream(stream)), "pi_sparse_ffn")


def pi_decode_ffn(layer: FfnLayer, u: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                  idx: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None, flags: int = 0,
                  stream=None):
    """u [B, d]; y fp32 [B, d]; optional idx int32 [B, f] and count int32 [B]."""
    B = _tokens(u, layer.d, "u")
    _need(u, "u", layer.u_dtype, B * layer.d)
    _need(y, "y", torch.float32, B * layer.d)
    _need(idx, "idx", torch.int32, B * layer.f)
    _need(count, "count", torch.int32, B)
    _need_ws(ws)
    _on_device(u=u, y=y, idx=idx, count=count, workspace=ws)
    _check(lib().pi_decode_ffn(layer.handle, _p(u), B, _p(y), _p(idx), _p(count), int(flags), *_wsargs(ws),
                               _stream(stream)), "pi_decode_ffn")


def pi_decode_ffn_static(layer: FfnLayer, u: torch.Tensor, y: torch.Tensor, idx: Optional[torch.Tensor] = None,
                         count: Optional[torch.Tensor] = None, flags: int = 0,
                         dev_status: Optional[torch.Tensor] = None, stream=None):
    """Batch-1 decode step on the library's static device scratch (no workspace)."""
    if u.numel() != layer.d or y.numel() != layer.d:
        raise ValueError("pi_decode_ffn_static is batch 1: u and y hold d elements")
    _need(u, "u", layer.u_dtype, layer.d)
    _need(y, "y", torch.float32, layer.d)
    _need(idx, "idx", torch.int32, layer.f)
    _need(count, "count", torch.int32, 1)
    _need(dev_status, "dev_status", torch.int32, 1)
    _on_device(u=u, y=y, idx=idx, count=count, dev_status=dev_status)
    _check(lib().pi_decode_ffn_static(layer.handle, _p(u), _p(y), _p(idx), _p(count), int(flags), _p(dev_status),
                                      _stream(stream)), "pi_decode_ffn_static")


def pi_decode_ffn_stack(layers: Sequence[FfnLayer], x: torch.Tensor, ws: torch.Tensor,
                        idx_trace: Optional[torch.Tensor] = None, count_trace: Optional[torch.Tensor] = None,
                        flags: int = 0, stream=None):
    """x fp32 [B, d] (the residual, updated in place); optional idx_trace int32
    [L, B, f_max] and count_trace int32 [L, B]."""
    if not layers:
        raise ValueError("pi_decode_ffn_stack needs at least one layer")
    B = _tokens(x, layers[0].d, "x")
    L, fmax = len(layers), max(l.f for l in layers)
    _need(x, "x", torch.float32, B * layers[0].d)
    _need(idx_trace, "idx_trace", torch.int32, L * B * fmax)
    _need(count_trace, "count_trace", torch.int32, L * B)
    _need_ws(ws)
    _on_device(x=x, idx_trace=idx_trace, count_trace=count_trace, workspace=ws)
    arr = (C.c_void_p * len(layers))(*[l.handle for l in layers])
    _check(lib().pi_decode_ffn_stack(arr, len(layers), _p(x), B, _p(idx_trace), _p(count_trace), int(flags),
                                     *_wsargs(ws), _stream(stream)), "pi_decode_ffn_stack")


def pi_debug_wait_fault(withhold_row: int = -1, limit_us: int = 0):
    """Test support: batch-1 fused launches never publish entry ``withhold_row``
    of h and wait at most ``limit_us`` (see the header); (-1, 0) restores
    normal runs."""
    _check(lib().pi_debug_wait_fault(int(withhold_row), int(limit_us)), "pi_debug_wait_fault")


def pi_get_device_status(ws: torch.Tensor, stream=None) -> int:
    code = C.c_int()
    _check(lib().pi_get_device_status(_p(ws), _stream(stream), C.byref(code)), "pi_get_device_status")
    return code.value


# ---------------------------------------------------------------- dense block operators
# These calls serve single tokens too, where a call's host time is what the
# user waits for, so the checks make one pass over the tensors.
def _check_out(t: Optional[torch.Tensor], what: str, dtype, shape):
    """An exactly shaped contiguous tensor (None passes)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _check_in(t: torch.Tensor, what: str, dtype):
    """A contiguous tensor whose shape _tokens has checked."""
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _ptrs(names: str, *tensors: Optional[torch.Tensor]):
    """The tensors' addresses (None stays None).  All of them on the current
    CUDA device: kernels launch there, on its current stream."""
    dev = None
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        d = t.get_device()
        if d != dev:
            dev = _check_device(names, tensors, d)
        out.append(t.data_ptr())
    return out


def _check_moved(kept):
    """The tensors whose addresses a handle or a description holds, as (name, tensor, address), still lie there: their
    values may change in place, but one that was given other memory (w.data = ...) would be read where it was."""
    for what, t, p in kept:
        if t.data_ptr() != p:
            raise ValueError(f"{what}: its memory has moved since the layer or norm was made; make a new one")


def _check_device(names: str, tensors, d: int) -> int:
    """Device d of one of the tensors, if it is the current one."""
    if d < 0 or d != torch.cuda.current_device():
        what, t = next((w, t) for w, t in zip(names.split(), tensors) if t is not None and t.get_device() == d)
        if d < 0:
            raise ValueError(f"{what}: must be a CUDA tensor")
        raise ValueError(f"{what}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return d


# the current stream's handle without building a Stream object (3 us a call), where torch has it
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ws_bytes(ws: torch.Tensor) -> int:
    _need_ws(ws)
    return ws.numel() * ws.element_size()


def _zeroed_workspace(n: int, device=None) -> torch.Tensor:
    ws = torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))
    ws[:256].zero_()
    return ws


class GatedFfnLayer:
    """A created pi_gated_ffn handle plus references to the weights it borrows
    (each [f, d], fp16 or bf16, contiguous)."""

    def __init__(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down_t: torch.Tensor, *, act: str = "silu"):
        if w_gate.dim() != 2 or w_gate.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"w_gate: {w_gate.dtype} of shape {tuple(w_gate.shape)}, expected fp16 or bf16 [f, d]")
        if act not in GATE_ACT:
            raise ValueError(f"act: {act!r}, expected one of {sorted(GATE_ACT)}")
        self.f, self.d = w_gate.shape
        self.dtype, self.act = w_gate.dtype, act
        for what, t in (("w_gate", w_gate), ("w_up", w_up), ("w_down_t", w_down_t)):
            _check_out(t, what, self.dtype, (self.f, self.d))
            if t.device != w_gate.device:
                raise ValueError(f"{what}: on {t.device}, w_gate is on {w_gate.device}")
        self._keep = (w_gate, w_up, w_down_t)
        self._kept = tuple((n, t, t.data_ptr()) for n, t in zip(("w_gate", "w_up", "w_down_t"), self._keep))
        self.desc = pi_gated_ffn_desc(self.d, self.f, GATE_ACT[act], DTYPE[self.dtype], _p(w_gate), _p(w_up),
                                      _p(w_down_t))
        h = C.c_void_p()
        _check(lib().pi_gated_ffn_create(C.byref(self.desc), C.byref(h)), "pi_gated_ffn_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            lib().pi_gated_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pi_gated_ffn_workspace_size(layer: GatedFfnLayer, max_tokens: int, backward: bool = False) -> int:
    n = C.c_size_t()
    _check(lib().pi_gated_ffn_workspace_size(layer.handle, _c_int(max_tokens, "max_tokens"), int(bool(backward)),
                                             C.byref(n)), "pi_gated_ffn_workspace_size")
    return n.value


def make_gated_ffn_workspace(layer: GatedFfnLayer, max_tokens: int, backward: bool = False, device=None):
    """Allocate (with torch) a workspace for calls of up to max_tokens tokens."""
    return _zeroed_workspace(pi_gated_ffn_workspace_size(layer, max_tokens, backward), device)


def pi_gated_ffn_forward(layer: GatedFfnLayer, u: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                         gate: Optional[torch.Tensor] = None, up: Optional[torch.Tensor] = None, stream=None):
    """u [T, d] -> y [T, d]; gate, up: optional outputs [T, f] (the pre-activations)."""
    T = _tokens(u, layer.d, "u")
    _check_moved(layer._kept)
    _check_in(u, "u", layer.dtype)
    _check_out(y, "y", layer.dtype, (T, layer.d))
    _check_out(gate, "gate", layer.dtype, (T, layer.f))
    _check_out(up, "up", layer.dtype, (T, layer.f))
    n = _ws_bytes(ws)
    pu, py, pg, pp, pw, _ = _ptrs("u y gate up workspace weights", u, y, gate, up, ws, layer._keep[0])
    _check(lib().pi_gated_ffn_forward(layer.handle, pu, T, py, pg, pp, pw, n, _raw_stream(stream)),
           "pi_gated_ffn_forward")


def pi_gated_ffn_backward(layer: GatedFfnLayer, u: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                          dy: torch.Tensor, ws: torch.Tensor, du: Optional[torch.Tensor] = None,
                          dw_gate: Optional[torch.Tensor] = None, dw_up: Optional[torch.Tensor] = None,
                          dw_down_t: Optional[torch.Tensor] = None, flags: int = 0, stream=None):
    """Gradients at a forward call's u, gate and up, for dy [T, d].  du [T, d];
    dw_* [f, d], all fp32 or all of the layer's type; each may be left out."""
    T = _tokens(u, layer.d, "u")
    _check_moved(layer._kept)
    for what, t in (("u", u), ("dy", dy), ("du", du)):
        _check_out(t, what, layer.dtype, (T, layer.d))
    for what, t in (("gate", gate), ("up", up)):
        _check_out(t, what, layer.dtype, (T, layer.f))
    gtype = next((t.dtype for t in (dw_gate, dw_up, dw_down_t) if t is not None), layer.dtype)
    if gtype not in (torch.float32, layer.dtype):
        raise ValueError(f"dw_*: dtype {gtype}, expected torch.float32 or {layer.dtype}")
    for what, t in (("dw_gate", dw_gate), ("dw_up", dw_up), ("dw_down_t", dw_down_t)):
        _check_out(t, what, gtype, (layer.f, layer.d))
    n = _ws_bytes(ws)
    pu, pg, pp, pdy, pdu, p0, p1, p2, pw, _ = _ptrs("u gate up dy du dw_gate dw_up dw_down_t workspace weights", u,
                                                    gate, up, dy, du, dw_gate, dw_up, dw_down_t, ws, layer._keep[0])
    _check(lib().pi_gated_ffn_backward(layer.handle, pu, pg, pp, pdy, T, pdu, p0, p1, p2, DTYPE[gtype], int(flags),
                                       pw, n, _raw_stream(stream)), "pi_gated_ffn_backward")


class BlockNorm:
    """The parameters of the norms around a block (see pi_block_norm_desc) and
    references to the tensors they borrow.  w_post, w_pre: fp32 [d] or None;
    gate: fp32 [rows, d] or None, row t // tokens_per_gate for token t."""

    def __init__(self, d: int, *, y_dtype=torch.float16, u_dtype=torch.float16, eps: float = 1e-6,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, post_norm: bool = False,
                 w_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None, tokens_per_gate: int = 0):
        d, tokens_per_gate = _c_int(d, "d"), _c_int(tokens_per_gate, "tokens_per_gate")
        for what, t in (("y_dtype", y_dtype), ("u_dtype", u_dtype)):
            if t not in DTYPE:
                raise ValueError(f"{what}: {t}, expected one of {list(DTYPE)}")
        _check_out(w_post, "w_post", torch.float32, (d,))
        _check_out(w_pre, "w_pre", torch.float32, (d,))
        if gate is not None:
            if gate.dim() != 2 or tokens_per_gate <= 0:
                raise ValueError("gate: expected [rows, d] and tokens_per_gate > 0")
            _check_out(gate, "gate", torch.float32, (gate.shape[0], d))
        self.d, self.y_dtype, self.u_dtype, self.post_norm = d, y_dtype, u_dtype, bool(post_norm)
        self.gate, self.tokens_per_gate = gate, tokens_per_gate
        self.w_post, self.w_pre = w_post, w_pre
        self._kept = tuple((n, t, t.data_ptr()) for n, t in (("w_post", w_post), ("w_pre", w_pre), ("gate", gate))
                           if t is not None)
        # one of them per device, for the check of devices (what has not moved is on the device where it was)
        lead = {t.device: (n, t) for n, t, _ in self._kept}.values()
        self._lead_names, self._lead = " ".join(n for n, _ in lead), tuple(t for _, t in lead)
        self.desc = pi_block_norm_desc(d, DTYPE[y_dtype], DTYPE[u_dtype], int(post_norm), eps, residual_scale,
                                       branch_scale, _p(w_post), _p(w_pre), _p(gate), tokens_per_gate)
        self.ref = C.byref(self.desc)

    def _check_tokens(self, T: int):
        """The gate has a row for each of T tokens, and the parameters lie where they did."""
        _check_moved(self._kept)
        if self.gate is not None and self.gate.shape[0] * self.tokens_per_gate < T:
            raise ValueError(f"gate: {self.gate.shape[0]} rows of {self.tokens_per_gate} tokens for {T} tokens")


def pi_block_norm_forward(norm: BlockNorm, x: torch.Tensor, y: Optional[torch.Tensor],
                          x_out: Optional[torch.Tensor], u: Optional[torch.Tensor],
                          rstd_post: Optional[torch.Tensor] = None, rstd_pre: Optional[torch.Tensor] = None,
                          stream=None):
    """x fp32 [T, d] and y [T, d] -> the new stream x_out fp32 [T, d] (may be x)
    and the next block's input u [T, d]; rstd_post, rstd_pre: optional fp32 [T]."""
    T = _tokens(x, norm.d, "x")
    norm._check_tokens(T)
    _check_in(x, "x", torch.float32)
    _check_out(y, "y", norm.y_dtype, (T, norm.d))
    _check_out(x_out, "x_out", torch.float32, (T, norm.d))
    _check_out(u, "u", norm.u_dtype, (T, norm.d))
    _check_out(rstd_post, "rstd_post", torch.float32, (T,))
    _check_out(rstd_pre, "rstd_pre", torch.float32, (T,))
    px, py, po, pu, pk, pr, *_ = _ptrs("x y x_out u rstd_post rstd_pre " + norm._lead_names, x, y, x_out, u, rstd_post,
                                       rstd_pre, *norm._lead)
    _check(lib().pi_block_norm_forward(norm.ref, px, py, T, po, pu, pk, pr, _raw_stream(stream)),
           "pi_block_norm_forward")


def pi_block_norm_workspace_size(norm: BlockNorm, max_tokens: int) -> int:
    n = C.c_size_t()
    _check(lib().pi_block_norm_workspace_size(norm.ref, _c_int(max_tokens, "max_tokens"), C.byref(n)),
           "pi_block_norm_workspace_size")
    return n.value


def make_block_norm_workspace(norm: BlockNorm, max_tokens: int, device=None):
    """Allocate (with torch) a workspace for backward calls of up to max_tokens tokens."""
    return _zeroed_workspace(pi_block_norm_workspace_size(norm, max_tokens), device)


def pi_block_norm_backward(norm: BlockNorm, x_out: Optional[torch.Tensor], y: Optional[torch.Tensor],
                           rstd_post: Optional[torch.Tensor], rstd_pre: Optional[torch.Tensor],
                           du: Optional[torch.Tensor], dx_out: Optional[torch.Tensor], dx: Optional[torch.Tensor],
                           dy: Optional[torch.Tensor], ws: torch.Tensor, dw_post: Optional[torch.Tensor] = None,
                           dw_pre: Optional[torch.Tensor] = None, dgate: Optional[torch.Tensor] = None,
                           flags: int = 0, stream=None):
    """Gradients for du [T, d] and dx_out fp32 [T, d] (either may be None): dx
    fp32 [T, d] (may be dx_out), dy [T, d] (may be y), dw_post, dw_pre fp32 [d] and
    dgate of the gate's shape (gate rows behind the last token's keep what dgate
    holds); each may be left out."""
    lead = du if du is not None else dx_out
    if lead is None:
        raise ValueError("pi_block_norm_backward needs du or dx_out")
    T = _tokens(lead, norm.d, "du" if du is not None else "dx_out")
    norm._check_tokens(T)
    for what, t, dt in (("x_out", x_out, torch.float32), ("y", y, norm.y_dtype), ("du", du, norm.u_dtype),
                        ("dx_out", dx_out, torch.float32), ("dx", dx, torch.float32), ("dy", dy, norm.y_dtype)):
        _check_out(t, what, dt, (T, norm.d))
    _check_out(rstd_post, "rstd_post", torch.float32, (T,))
    _check_out(rstd_pre, "rstd_pre", torch.float32, (T,))
    _check_out(dw_post, "dw_post", torch.float32, (norm.d,))
    _check_out(dw_pre, "dw_pre", torch.float32, (norm.d,))
    if dgate is not None:
        if norm.gate is None:
            raise ValueError("dgate: there is no gate")
        _check_out(dgate, "dgate", torch.float32, norm.gate.shape)
    n = _ws_bytes(ws)
    (pr, py, pkp, pkr, pdu, pg, pdx, pdy, pw, p0, p1, p2, *_) = _ptrs(
        "x_out y rstd_post rstd_pre du dx_out dx dy workspace dw_post dw_pre dgate " + norm._lead_names, x_out, y,
        rstd_post, rstd_pre, du, dx_out, dx, dy, ws, dw_post, dw_pre, dgate, *norm._lead)
    _check(lib().pi_block_norm_backward(norm.ref, pr, py, pkp, pkr, pdu, pg, T, pdx, pdy, p0, p1, p2, int(flags), pw,
                                        n, _raw_stream(stream)), "pi_block_norm_backward")


def pi_quantize_i8(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None):
    """Rows of x [rows, k] (fp32, fp16 or bf16) -> int8 codes q [rows, k] and fp32 scales [rows]."""
    if x.dim() != 2 or x.dtype not in DTYPE:
        raise ValueError(f"x: {x.dtype} of shape {tuple(x.shape)}, expected fp32, fp16 or bf16 [rows, k]")
    rows, k = _c_int(x.shape[0], "x: rows"), _c_int(x.shape[1], "x: columns")
    _check_out(x, "x", x.dtype, (rows, k))
    _check_out(q, "q", torch.int8, (rows, k))
    _check_out(scales, "scales", torch.float32, (rows,))
    px, pq, ps = _ptrs("x q scales", x, q, scales)
    _check(lib().pi_quantize_i8(px, DTYPE[x.dtype], rows, k, pq, ps, _raw_stream(stream)), "pi_quantize_i8")


def pi_matmul_i8_workspace_size(tokens: int, n: int, k: int) -> int:
    size = C.c_size_t()
    _check(lib().pi_matmul_i8_workspace_size(_c_int(tokens, "tokens"), _c_int(n, "n"), _c_int(k, "k"), C.byref(size)),
           "pi_matmul_i8_workspace_size")
    return size.value


def make_matmul_i8_workspace(max_tokens: int, n: int, k: int, device=None):
    """Allocate (with torch) a workspace for products of up to max_tokens tokens."""
    return _zeroed_workspace(pi_matmul_i8_workspace_size(max_tokens, n, k), device)


def pi_matmul_i8(xq: torch.Tensor, x_scales: torch.Tensor, wq: torch.Tensor, w_scales: torch.Tensor,
                 y: torch.Tensor, ws: torch.Tensor, bias: Optional[torch.Tensor] = None, stream=None):
    """xq int8 [T, k] with x_scales fp32 [T], wq int8 [n, k] with w_scales fp32
    [n], bias fp32 [n] or None -> y [T, n] (fp32, fp16 or bf16)."""
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError(f"xq {tuple(xq.shape)} and wq {tuple(wq.shape)}: expected [T, k] and [n, k]")
    if y.dtype not in DTYPE:
        raise ValueError(f"y: dtype {y.dtype}, expected one of {list(DTYPE)}")
    T, k, n = _c_int(xq.shape[0], "xq: rows"), _c_int(xq.shape[1], "xq: columns"), _c_int(wq.shape[0], "wq: rows")
    _check_out(xq, "xq", torch.int8, (T, k))
    _check_out(wq, "wq", torch.int8, (n, k))
    _check_out(x_scales, "x_scales", torch.float32, (T,))
    _check_out(w_scales, "w_scales", torch.float32, (n,))
    _check_out(bias, "bias", torch.float32, (n,))
    _check_out(y, "y", y.dtype, (T, n))
    size = _ws_bytes(ws)
    pq, ps, pwq, pws, pb_, py, pw = _ptrs("xq x_scales wq w_scales bias y workspace", xq, x_scales, wq, w_scales, bias,
                                          y, ws)
    _check(lib().pi_matmul_i8(pq, ps, pwq, pws, pb_, T, n, k, py, DTYPE[y.dtype], pw, size, _raw_stream(stream)),
           "pi_matmul_i8")


def pi_debug_dense_plan(product: int, mb: int = 0, nt: int = 0, split: int = 0):
    """Test support: a dense product's following calls use this tiling (see
    the header); product -1 alone restores the rule for all."""
    _check(lib().pi_debug_dense_plan(int(product), int(mb), int(nt), int(split)), "pi_debug_dense_plan")
