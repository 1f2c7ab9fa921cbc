"""ctypes binding of libfnl.so (include/fnl.h), same names as the C entry points.

Argument marshalling only: the functions take torch CUDA tensors, check their
dtype/device/contiguity, allocate missing outputs with torch, and pass raw
pointers plus the current CUDA stream to the C library. Every step of the fused
op runs in the library's kernels. There is no fallback: if the library is
missing or the device is not sm_100, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

# FNL_LIBRARY=debug selects the debug build (output stores checked against their buffers)
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libfnl_debug.so" if os.environ.get("FNL_LIBRARY") == "debug" else "libfnl.so")
_lib = None

FNL_OK = 0
STATUS_NAMES = {0: "FNL_OK", 1: "FNL_ERR_INVALID_ARG", 2: "FNL_ERR_ALIGNMENT", 3: "FNL_ERR_ALIAS",
                4: "FNL_ERR_UNSUPPORTED", 5: "FNL_ERR_CUDA", 6: "FNL_ERR_DEVICE_STATUS"}
NORMS = {"layernorm": 0, "rmsnorm": 1}
PATHS = {"auto": 0, "tile": 1, "splitk": 2, "wide": 3, "cluster": 4, "pair": 5, "pair_sk": 6}
PRECISIONS = {"default": 0, "split": 1, "single": 2}
KV_FORMATS = {"bf16": 0, "int4": 1}

EXPORTED = ("fnl_create", "fnl_destroy", "fnl_status_string", "fnl_last_error", "fnl_last_plan", "fnl_check",
            "fnl_add_norm_qkv", "fnl_add_norm_swiglu", "fnl_add_bias_norm_gelu", "fnl_linear_add_residual",
            "fnl_add_norm_qkv_fp8", "fnl_add_norm_swiglu_fp8", "fnl_add_bias_norm_gelu_fp8",
            "fnl_quantize_weight_fp8", "fnl_tp_allreduce",
            "fnl_add_norm_qkv_static", "fnl_check_static",
            "fnl_rope_append_kv", "fnl_kv_gather", "fnl_paged_attention")


class FnlError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class _Options(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int), ("max_n", ctypes.c_int), ("path", ctypes.c_int),
                ("max_ctas", ctypes.c_int), ("precision", ctypes.c_int), ("wait_ns", ctypes.c_longlong),
                ("debug_stall_calls", ctypes.c_int), ("tune", ctypes.c_int)]


class _KvCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("scale_page_stride", ctypes.c_longlong)]


class _KvBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("max_q", ctypes.c_int), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int)]


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libfnl.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                           "`python -m transformer_layer_residual_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.fnl_create.argtypes = [ctypes.POINTER(P), I, ctypes.POINTER(_Options)]
    L.fnl_destroy.argtypes = [P]
    L.fnl_status_string.argtypes = [I]
    L.fnl_status_string.restype = ctypes.c_char_p
    L.fnl_last_error.argtypes = [P]
    L.fnl_last_error.restype = ctypes.c_char_p
    L.fnl_last_plan.argtypes = [P]
    L.fnl_last_plan.restype = ctypes.c_char_p
    L.fnl_check.argtypes = [P, P]
    L.fnl_add_norm_qkv.argtypes = [P, P, P, P, P, P, P, I, F, P, P, I, I, I, I, I, P, P, P, P, P]
    L.fnl_add_norm_swiglu.argtypes = [P, P, P, P, P, P, P, I, F, P, P, I, I, I, P, P, P]
    L.fnl_add_bias_norm_gelu.argtypes = [P, P, P, P, P, P, P, P, I, F, P, P, I, I, I, P, P, P]
    L.fnl_linear_add_residual.argtypes = [P, P, P, P, P, P, P, I, I, I]
    L.fnl_add_norm_qkv_fp8.argtypes = [P, P, P, P, P, P, P, I, F, P, P, P, I, I, I, I, I, P, P, P, P, P]
    L.fnl_quantize_weight_fp8.argtypes = [P, P, P, I, I, P, P]
    L.fnl_tp_allreduce.argtypes = [P, P, ctypes.POINTER(P), I, P, ctypes.c_longlong]
    L.fnl_add_norm_swiglu_fp8.argtypes = [P, P, P, P, P, P, P, I, F, P, P, P, I, I, I, P, P, P]
    L.fnl_add_bias_norm_gelu_fp8.argtypes = [P, P, P, P, P, P, P, P, I, F, P, P, P, I, I, I, P, P, P]
    L.fnl_add_norm_qkv_static.argtypes = [P, P, P, P, P, P, I, F, P, P, I, I, I, I, I, P, P, P, P, P]
    L.fnl_check_static.argtypes = [P]
    # the cache and the batch go as the addresses of their structures
    L.fnl_rope_append_kv.argtypes = [P, P, P, P, I, I, P, P, P, P, P, I, I, I, P]
    L.fnl_kv_gather.argtypes = [P, P, P, P, I, P, P]
    L.fnl_paged_attention.argtypes = [P, P, P, P, I, I, P, F, I, I, P, P]
    for name in EXPORTED:
        if getattr(L, name).restype is None and name not in ("fnl_status_string", "fnl_last_error", "fnl_last_plan"):
            getattr(L, name).restype = I
    _lib = L
    return L


class Handle:
    """Owns an fnl_handle (device workspace). One stream / thread at a time.

    max_tokens / max_n reserve the workspace up front (no reallocation, and so
    no stream synchronisation, on later calls up to that size). path forces a
    kernel: "auto" (by M), "splitk" (small-M kernel, stream-K form), "cluster"
    (small-M kernel, cluster form), "tile" (128x256 tiles), "wide" (128x512
    tiles), "pair" (256x512 tiles on CTA pairs), "pair_sk" (the pair kernel's
    stream-K form, its split tiles finished by the fix-up kernel). max_ctas
    caps the persistent grids (0 = all SMs). precision: "default" (split
    hi + lo operand for SwiGLU only), "split", "single". wait_ns: limit of the
    kernels' main-loop waits (0 = 4 s). debug_stall_calls: fault injection for
    tests of the status path (the next that-many calls withhold one weight copy,
    or their first key copies, so a wait runs out and check() raises; calls without
    a bounded wait are not counted, see fnl.h). tune: shape auto-tuning (the first
    call of each shape times the candidate plans and keeps the fastest)."""

    def __init__(self, device: int = 0, max_tokens: int = 0, max_n: int = 0, path: str = "auto",
                 max_ctas: int = 0, precision: str = "default", wait_ns: int = 0, debug_stall_calls: int = 0,
                 tune: bool = False):
        L = lib()
        self._h = ctypes.c_void_p()
        opt = _Options(max_tokens, max_n, PATHS[path], max_ctas, PRECISIONS[precision], wait_ns,
                       debug_stall_calls, int(bool(tune)))
        st = L.fnl_create(ctypes.byref(self._h), device, ctypes.byref(opt))
        if st != FNL_OK:
            raise FnlError(st, f"fnl_create(device={device}) failed")
        self.device = device

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            lib().fnl_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def ptr(self):
        return self._h

    def _raise(self, st: int, what: str):
        msg = lib().fnl_last_error(self._h)
        raise FnlError(st, f"{what}: {msg.decode() if msg else ''}")

    def last_plan(self) -> str:
        """fnl_last_plan: the kernel, form and grid of the last call."""
        t = lib().fnl_last_plan(self._h)
        return t.decode() if t else ""

    def check(self, stream: Optional[torch.cuda.Stream] = None):
        """Synchronise the stream and raise if a kernel gave up a bounded wait."""
        st = lib().fnl_check(self._h, _stream_ptr(stream))
        if st != FNL_OK:
            self._raise(st, "fnl_check")


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape=None, dtype=torch.bfloat16):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _common(x, residual, gamma, beta, norm, residual_out, mean_out, rstd_out, W, bias):
    M, K = x.shape
    _need(x, "x", (M, K))
    _need(residual, "residual", (M, K))
    _need(gamma, "gamma", (K,))
    _need(beta, "beta", (K,))
    _need(W, "W")
    if W.dim() != 2 or W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    _need(bias, "bias", (W.shape[0],))
    if residual_out is None:
        residual_out = torch.empty_like(x)
    _need(residual_out, "residual_out", (M, K))
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {list(NORMS)}")
    if rstd_out is not None:
        _need(rstd_out, "rstd_out", (M,), torch.float32)
    if mean_out is not None:
        _need(mean_out, "mean_out", (M,), torch.float32)
    return M, K, residual_out


def add_norm_qkv(h: Handle, x, residual, gamma, beta, W, Hq, Hkv, D, norm="rmsnorm", eps=1e-5, bias=None,
                 residual_out=None, q=None, k=None, v=None, mean_out=None, rstd_out=None, stream=None):
    """fnl_add_norm_qkv. Returns dict(residual_out, q [Hq,M,D], k, v, mean, rstd)."""
    M, K, residual_out = _common(x, residual, gamma, beta, norm, residual_out, mean_out, rstd_out, W, bias)
    q = torch.empty(Hq, M, D, dtype=torch.bfloat16, device=x.device) if q is None else q
    k = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if k is None else k
    v = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if v is None else v
    _need(q, "q", (Hq, M, D)); _need(k, "k", (Hkv, M, D)); _need(v, "v", (Hkv, M, D))
    st = lib().fnl_add_norm_qkv(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(residual_out), _p(gamma),
                                _p(beta), NORMS[norm], float(eps), _p(W), _p(bias), M, K, Hq, Hkv, D,
                                _p(q), _p(k), _p(v), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_norm_qkv")
    return {"residual_out": residual_out, "q": q, "k": k, "v": v, "mean": mean_out, "rstd": rstd_out}


def add_norm_swiglu(h: Handle, x, residual, gamma, beta, W, I, norm="rmsnorm", eps=1e-5, bias=None,
                    residual_out=None, out=None, mean_out=None, rstd_out=None, stream=None):
    """fnl_add_norm_swiglu. W is [2I, K] (gate rows then up rows). Returns dict."""
    M, K, residual_out = _common(x, residual, gamma, beta, norm, residual_out, mean_out, rstd_out, W, bias)
    out = torch.empty(M, I, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, "out", (M, I))
    st = lib().fnl_add_norm_swiglu(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(residual_out),
                                   _p(gamma), _p(beta), NORMS[norm], float(eps), _p(W), _p(bias), M, K, I,
                                   _p(out), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_norm_swiglu")
    return {"residual_out": residual_out, "out": out, "mean": mean_out, "rstd": rstd_out}


def add_bias_norm_gelu(h: Handle, x, residual, gamma, beta, W, bias_in=None, bias_out=None, norm="layernorm",
                       eps=1e-5, residual_out=None, out=None, mean_out=None, rstd_out=None, stream=None):
    """fnl_add_bias_norm_gelu. Returns dict(residual_out, out [M,N], mean, rstd)."""
    M, K, residual_out = _common(x, residual, gamma, beta, norm, residual_out, mean_out, rstd_out, W,
                                 bias_out)
    _need(bias_in, "bias_in", (K,))
    N = W.shape[0]
    out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, "out", (M, N))
    st = lib().fnl_add_bias_norm_gelu(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(bias_in),
                                      _p(residual_out), _p(gamma), _p(beta), NORMS[norm], float(eps), _p(W),
                                      _p(bias_out), M, K, N, _p(out), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_bias_norm_gelu")
    return {"residual_out": residual_out, "out": out, "mean": mean_out, "rstd": rstd_out}


def tp_allreduce(h: Handle, parts, out=None, stream=None):
    """fnl_tp_allreduce: out = bf16(sum of the P same-shape bf16 tensors in
    `parts`, in list order). On a node the parts are the ranks' partial outputs
    (the peers' as tensors over their mapped memory); here any device tensors.
    Returns out."""
    parts = list(parts)
    if not parts:
        raise ValueError("tp_allreduce needs at least one part")
    shape = tuple(parts[0].shape)
    for t in parts:
        _need(t, "part", shape)
    out = torch.empty(shape, dtype=torch.bfloat16, device=parts[0].device) if out is None else out
    _need(out, "out", shape)
    arr = (ctypes.c_void_p * len(parts))(*[t.data_ptr() for t in parts])
    st = lib().fnl_tp_allreduce(h.ptr, _stream_ptr(stream), arr, len(parts), _p(out), out.numel())
    if st != FNL_OK:
        h._raise(st, "fnl_tp_allreduce")
    return out


def add_norm_qkv_tp(h: Handle, parts, residual, gamma, beta, W, Hq, Hkv, D, norm="rmsnorm", eps=1e-5, bias=None,
                    x_buf=None, stream=None, **outs):
    """The QKV op fed by the tensor-parallel all-reduce: x = tp_allreduce(parts)
    (into x_buf if given), then add_norm_qkv(x, residual, ...). Two launches on
    the stream; the fused op is a programmatic dependent of the all-reduce."""
    x = tp_allreduce(h, parts, out=x_buf, stream=stream)
    return add_norm_qkv(h, x, residual, gamma, beta, W, Hq, Hkv, D, norm=norm, eps=eps, bias=bias, stream=stream,
                        **outs)


def linear_add_residual(h: Handle, a, W, residual, bias=None, out=None, stream=None):
    """fnl_linear_add_residual: out = residual + a W^T (+ bias), bf16. a [M, K],
    W [N, K], residual [M, N]; out may be `residual` itself (in-place update of
    the residual stream). Returns dict(out)."""
    M, K = a.shape
    _need(a, "a", (M, K))
    _need(W, "W")
    if W.dim() != 2 or W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    N = W.shape[0]
    _need(bias, "bias", (N,))
    _need(residual, "residual", (M, N))
    out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device) if out is None else out
    _need(out, "out", (M, N))
    st = lib().fnl_linear_add_residual(h.ptr, _stream_ptr(stream), _p(a), _p(W), _p(bias), _p(residual), _p(out),
                                       M, K, N)
    if st != FNL_OK:
        h._raise(st, "fnl_linear_add_residual")
    return {"out": out}


def quantize_weight_fp8(h: Handle, W, stream=None):
    """fnl_quantize_weight_fp8: (Wq uint8 [N, K] e4m3 codes, w_scale fp32 [N])."""
    _need(W, "W")
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    Wq = torch.empty(N, K, dtype=torch.uint8, device=W.device)
    w_scale = torch.empty(N, dtype=torch.float32, device=W.device)
    st = lib().fnl_quantize_weight_fp8(h.ptr, _stream_ptr(stream), _p(W), N, K, _p(Wq), _p(w_scale))
    if st != FNL_OK:
        h._raise(st, "fnl_quantize_weight_fp8")
    return Wq, w_scale


def add_norm_qkv_fp8(h: Handle, x, residual, gamma, beta, Wq, w_scale, Hq, Hkv, D, norm="rmsnorm", eps=1e-5,
                     bias=None, residual_out=None, q=None, k=None, v=None, mean_out=None, rstd_out=None,
                     stream=None):
    """fnl_add_norm_qkv_fp8: Wq uint8 [N, K] e4m3 codes, w_scale fp32 [N].
    Returns dict(residual_out, q, k, v, mean, rstd)."""
    M, K = x.shape
    _need(x, "x", (M, K))
    _need(residual, "residual", (M, K))
    _need(gamma, "gamma", (K,))
    _need(beta, "beta", (K,))
    N = (Hq + 2 * Hkv) * D
    _need(Wq, "Wq", (N, K), torch.uint8)
    _need(w_scale, "w_scale", (N,), torch.float32)
    _need(bias, "bias", (N,))
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {list(NORMS)}")
    residual_out = torch.empty_like(x) if residual_out is None else residual_out
    q = torch.empty(Hq, M, D, dtype=torch.bfloat16, device=x.device) if q is None else q
    k = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if k is None else k
    v = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if v is None else v
    _need(residual_out, "residual_out", (M, K))
    _need(q, "q", (Hq, M, D)); _need(k, "k", (Hkv, M, D)); _need(v, "v", (Hkv, M, D))
    if rstd_out is not None:
        _need(rstd_out, "rstd_out", (M,), torch.float32)
    if mean_out is not None:
        _need(mean_out, "mean_out", (M,), torch.float32)
    st = lib().fnl_add_norm_qkv_fp8(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(residual_out), _p(gamma),
                                    _p(beta), NORMS[norm], float(eps), _p(Wq), _p(w_scale), _p(bias), M, K, Hq,
                                    Hkv, D, _p(q), _p(k), _p(v), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_norm_qkv_fp8")
    return {"residual_out": residual_out, "q": q, "k": k, "v": v, "mean": mean_out, "rstd": rstd_out}


def _fp8_common(x, residual, gamma, beta, Wq, w_scale, n_rows, norm, residual_out, mean_out, rstd_out):
    M, K = x.shape
    _need(x, "x", (M, K))
    _need(residual, "residual", (M, K))
    _need(gamma, "gamma", (K,))
    _need(beta, "beta", (K,))
    _need(Wq, "Wq", (n_rows, K), torch.uint8)
    _need(w_scale, "w_scale", (n_rows,), torch.float32)
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {list(NORMS)}")
    residual_out = torch.empty_like(x) if residual_out is None else residual_out
    _need(residual_out, "residual_out", (M, K))
    if rstd_out is not None:
        _need(rstd_out, "rstd_out", (M,), torch.float32)
    if mean_out is not None:
        _need(mean_out, "mean_out", (M,), torch.float32)
    return M, K, residual_out


def add_norm_swiglu_fp8(h: Handle, x, residual, gamma, beta, Wq, w_scale, I, norm="rmsnorm", eps=1e-5, bias=None,
                        residual_out=None, out=None, mean_out=None, rstd_out=None, stream=None):
    """fnl_add_norm_swiglu_fp8: Wq uint8 [2I, K] e4m3 codes (gate rows, then up
    rows), w_scale fp32 [2I]. Returns dict(residual_out, out [M, I], mean, rstd)."""
    M, K, residual_out = _fp8_common(x, residual, gamma, beta, Wq, w_scale, 2 * I, norm, residual_out, mean_out,
                                     rstd_out)
    _need(bias, "bias", (2 * I,))
    out = torch.empty(M, I, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, "out", (M, I))
    st = lib().fnl_add_norm_swiglu_fp8(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(residual_out),
                                       _p(gamma), _p(beta), NORMS[norm], float(eps), _p(Wq), _p(w_scale), _p(bias),
                                       M, K, I, _p(out), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_norm_swiglu_fp8")
    return {"residual_out": residual_out, "out": out, "mean": mean_out, "rstd": rstd_out}


def add_bias_norm_gelu_fp8(h: Handle, x, residual, gamma, beta, Wq, w_scale, bias_in=None, bias_out=None,
                           norm="layernorm", eps=1e-5, residual_out=None, out=None, mean_out=None, rstd_out=None,
                           stream=None):
    """fnl_add_bias_norm_gelu_fp8: Wq uint8 [N, K] e4m3 codes, w_scale fp32 [N].
    Returns dict(residual_out, out [M, N], mean, rstd)."""
    N = Wq.shape[0]
    M, K, residual_out = _fp8_common(x, residual, gamma, beta, Wq, w_scale, N, norm, residual_out, mean_out,
                                     rstd_out)
    _need(bias_in, "bias_in", (K,))
    _need(bias_out, "bias_out", (N,))
    out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device) if out is None else out
    _need(out, "out", (M, N))
    st = lib().fnl_add_bias_norm_gelu_fp8(h.ptr, _stream_ptr(stream), _p(x), _p(residual), _p(bias_in),
                                          _p(residual_out), _p(gamma), _p(beta), NORMS[norm], float(eps), _p(Wq),
                                          _p(w_scale), _p(bias_out), M, K, N, _p(out), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        h._raise(st, "fnl_add_bias_norm_gelu_fp8")
    return {"residual_out": residual_out, "out": out, "mean": mean_out, "rstd": rstd_out}


class KVCache:
    """A paged key/value cache (fnl_kv_cache) over the caller's tensors.

    bf16: k, v [num_pages, Hkv, page_size, D] bfloat16. int4: k, v uint8
    [num_pages, Hkv, page_size, D / 2] (the even d in the low nibble) with k_scale,
    v_scale bfloat16 [num_pages, Hkv, page_size, 2] (scale, minimum). The page
    dimension may be strided (k and v as halves of one allocation); the others are
    contiguous. The object holds the tensors; it may be kept for the cache's life."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in (torch.bfloat16, torch.uint8):
            raise ValueError(f"k must be torch.bfloat16 or torch.uint8, got {k.dtype}")
        self.format = "bf16" if k.dtype == torch.bfloat16 else "int4"
        if k.dim() != 4:
            raise ValueError("k must be [num_pages, Hkv, page_size, D] (D / 2 bytes for int4)")
        n, self.Hkv, self.page_size, last = k.shape
        self.D = last if self.format == "bf16" else 2 * last
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        stride = self._pages(k, "k", k.shape, k.dtype)
        if self._pages(v, "v", k.shape, k.dtype) != stride:
            raise ValueError("k and v must have the same page stride")
        scale_stride = 0
        if self.format == "int4":
            shape = (n, self.Hkv, self.page_size, 2)
            scale_stride = self._pages(k_scale, "k_scale", shape, torch.bfloat16)
            if self._pages(v_scale, "v_scale", shape, torch.bfloat16) != scale_stride:
                raise ValueError("k_scale and v_scale must have the same page stride")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no k_scale and v_scale")
        self.device, self.index = k.device, k.get_device()
        if any(t is not None and t.get_device() != self.index for t in (v, k_scale, v_scale)):
            raise ValueError("the cache's tensors must be on one device")
        self.c = _KvCache(KV_FORMATS[self.format], n, self.page_size, self.Hkv, self.D, _p(k), _p(v), _p(k_scale),
                          _p(v_scale), stride, scale_stride)
        self.ptr = ctypes.addressof(self.c)

    @staticmethod
    def _pages(t, name, shape, dtype):
        if t is None:
            raise ValueError(f"{name} is required")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        inner = (shape[2] * shape[3], shape[3], 1)
        if any(st != want for st, want, n in zip(t.stride()[1:], inner, shape[1:]) if n > 1):
            raise ValueError(f"{name} must be contiguous within a page")
        if shape[0] > 1 and t.stride(0) < shape[1] * shape[2] * shape[3]:
            raise ValueError(f"the pages of {name} overlap (page stride {t.stride(0)})")
        return t.stride(0) * t.element_size() if shape[0] > 1 else 0

    @classmethod
    def empty(cls, num_pages, page_size, Hkv, D, format="bf16", device="cuda"):
        """A new, uninitialised cache."""
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {list(KV_FORMATS)}")
        if format == "bf16":
            return cls(*(torch.empty(num_pages, Hkv, page_size, D, dtype=torch.bfloat16, device=device)
                         for _ in range(2)))
        return cls(*(torch.empty(num_pages, Hkv, page_size, D // 2, dtype=torch.uint8, device=device)
                     for _ in range(2)),
                   *(torch.empty(num_pages, Hkv, page_size, 2, dtype=torch.bfloat16, device=device)
                     for _ in range(2)))


class KVBatch:
    """A packed batch over a paged cache (fnl_kv_batch): cu_q int32 [B + 1], kv_len
    int32 [B], block_table int32 [B, max_pages], all on the GPU, and max_q, the
    caller's bound on any sequence's new tokens. The kernels read the arrays when
    they run, so the object may be kept and its tensors updated in place."""

    def __init__(self, cu_q, kv_len, block_table, max_q):
        B = kv_len.shape[0]
        _need(kv_len, "kv_len", (B,), torch.int32)
        _need(cu_q, "cu_q", (B + 1,), torch.int32)
        _need(block_table, "block_table", None, torch.int32)
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"block_table must be [{B}, max_pages], got {tuple(block_table.shape)}")
        self.cu_q, self.kv_len, self.block_table, self.max_q = cu_q, kv_len, block_table, int(max_q)
        self.device, self.index = kv_len.device, kv_len.get_device()
        if cu_q.device != self.device or block_table.device != self.device:
            raise ValueError("cu_q, kv_len and block_table must be on one device")
        self.c = _KvBatch(B, self.max_q, _p(cu_q), _p(kv_len), _p(block_table), block_table.shape[1])
        self.ptr = ctypes.addressof(self.c)


def _kv_stream(h, cache, batch, stream):
    """The call's stream: `stream`, or the current one of the handle's device."""
    if cache.index != h.device or batch.index != h.device:
        raise ValueError(f"the cache and the batch must be on the handle's device, cuda:{h.device}")
    return torch._C._cuda_getCurrentRawStream(h.device) if stream is None else stream.cuda_stream


def _kv_need(h, t, name, shape, dtype=torch.bfloat16):
    """The data pointer of t after its checks (a decode step makes these calls once a layer: the one test first)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == h.device and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, shape, dtype)
    raise ValueError(f"{name} must be on the handle's device, cuda:{h.device}")


def rope_append_kv(h: Handle, cache: KVCache, batch: KVBatch, q, k, v, cos=None, sin=None, interleaved=False,
                   q_out=None, stream=None):
    """fnl_rope_append_kv. q [Hq, M, D], k and v [Hkv, M, D] (as add_norm_qkv returns
    them), cos and sin fp32 [max_pos, rot_dim / 2]. k (rotated) and v go to their
    pages; q_out (allocated when not given; may be q) gets the rotated q. Without
    cos and sin nothing is rotated and q is returned as it is. Returns dict(q)."""
    if k.dim() != 3:
        raise ValueError("k must be [Hkv, M, D]")
    Hkv, M, D = cache.Hkv, k.shape[1], cache.D
    kp = _kv_need(h, k, "k", (Hkv, M, D))
    vp = _kv_need(h, v, "v", (Hkv, M, D))
    s = _kv_stream(h, cache, batch, stream)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin are given together")
    if cos is None:
        if q_out is not None:
            raise ValueError("q_out is written by the rotation only: give cos and sin")
        st = lib().fnl_rope_append_kv(h.ptr, s, cache.ptr, batch.ptr, M, 0, None, kp, vp, None, None, 0, 0, 0, None)
    else:
        if q.dim() != 3 or cos.dim() != 2:
            raise ValueError("q must be [Hq, M, D], cos and sin [max_pos, rot_dim / 2]")
        shape, table = (q.shape[0], M, D), cos.shape
        qp = _kv_need(h, q, "q", shape)
        cp = _kv_need(h, cos, "cos", table, torch.float32)
        sp = _kv_need(h, sin, "sin", table, torch.float32)
        if q_out is None:
            q_out = torch.empty_like(q)
            op = q_out.data_ptr()
        else:
            op = _kv_need(h, q_out, "q_out", shape)
        st = lib().fnl_rope_append_kv(h.ptr, s, cache.ptr, batch.ptr, M, shape[0], qp, kp, vp, cp, sp, 2 * table[1],
                                      table[0], 1 if interleaved else 0, op)
    if st != FNL_OK:
        h._raise(st, "fnl_rope_append_kv")
    return {"q": q if cos is None else q_out}


def kv_gather(h: Handle, cache: KVCache, batch: KVBatch, M=None, k=None, v=None, stream=None):
    """fnl_kv_gather: the batch's new tokens read back from their pages, k and v
    bf16 [Hkv, M, D]. M (the packed rows) comes from k or v, or is given, or, when
    none is, read from cu_q, which waits for the device. Returns dict(k, v)."""
    if k is not None or v is not None:
        M = (v if k is None else k).shape[1]
    elif M is None:
        M = int(batch.cu_q[-1])
    shape = (cache.Hkv, M, cache.D)
    s = _kv_stream(h, cache, batch, stream)
    k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if v is None else v
    st = lib().fnl_kv_gather(h.ptr, s, cache.ptr, batch.ptr, M, _kv_need(h, k, "k", shape), _kv_need(h, v, "v", shape))
    if st != FNL_OK:
        h._raise(st, "fnl_kv_gather")
    return {"k": k, "v": v}


def paged_attention(h: Handle, cache: KVCache, batch: KVBatch, q, scale=None, window=0, sinks=0, out=None, lse=None,
                    stream=None):
    """fnl_paged_attention: q [Hq, M, D] -> out [M, Hq * D], causal, with a sliding
    window and `sinks` first tokens that stay visible when window > 0. scale
    defaults to D ** -0.5; lse (fp32 [Hq, M]) is filled when given. Returns
    dict(out, lse)."""
    if q.dim() != 3:
        raise ValueError("q must be [Hq, M, D]")
    Hq, M, D = q.shape
    qp = _kv_need(h, q, "q", (Hq, M, cache.D))
    s = _kv_stream(h, cache, batch, stream)
    if out is None:
        out = torch.empty((M, Hq * D), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _kv_need(h, out, "out", (M, Hq * D))
    lp = None if lse is None else _kv_need(h, lse, "lse", (Hq, M), torch.float32)
    st = lib().fnl_paged_attention(h.ptr, s, cache.ptr, batch.ptr, M, Hq, qp, D ** -0.5 if scale is None else scale, window,
                                   sinks, op, lp)
    if st != FNL_OK:
        h._raise(st, "fnl_paged_attention")
    return {"out": out, "lse": lse}


def run_workload(h: Handle, w, dev: dict, stats: bool = True, stream=None) -> dict:
    """Run a synthetic.Workload on device tensors `dev` (same keys as
    synthetic.make_inputs). Allocates the outputs and statistics buffers."""
    if w.op == "residual":
        return linear_add_residual(h, dev["x"], dev["W"], dev["residual"], bias=dev.get("bias_out"), stream=stream)
    M = dev["x"].shape[0]
    if w.op.endswith("_fp8"):   # dev["W_fp8"]: e4m3 codes (float8_e4m3fn or uint8), dev["w_scale"]: fp32 [N]
        rstd = torch.empty(M, dtype=torch.float32, device=dev["x"].device) if stats else None
        mean = (torch.empty(M, dtype=torch.float32, device=dev["x"].device)
                if stats and w.norm == "layernorm" else None)
        Wq = dev["W_fp8"]
        Wq = Wq.view(torch.uint8) if Wq.dtype != torch.uint8 else Wq
        if w.op == "swiglu_fp8":
            return add_norm_swiglu_fp8(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), Wq,
                                       dev["w_scale"], w.I, norm=w.norm, eps=w.eps, bias=dev.get("bias_out"),
                                       mean_out=mean, rstd_out=rstd, stream=stream)
        if w.op == "gelu_fp8":
            return add_bias_norm_gelu_fp8(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), Wq,
                                          dev["w_scale"], bias_in=dev.get("bias_in"), bias_out=dev.get("bias_out"),
                                          norm=w.norm, eps=w.eps, mean_out=mean, rstd_out=rstd, stream=stream)
        return add_norm_qkv_fp8(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), Wq, dev["w_scale"],
                                w.Hq, w.Hkv, w.D, norm=w.norm, eps=w.eps, bias=dev.get("bias_out"), mean_out=mean,
                                rstd_out=rstd, stream=stream)
    rstd = torch.empty(M, dtype=torch.float32, device=dev["x"].device) if stats else None
    mean = (torch.empty(M, dtype=torch.float32, device=dev["x"].device)
            if stats and w.norm == "layernorm" else None)
    if w.op == "qkv":
        return add_norm_qkv(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), dev["W"], w.Hq, w.Hkv,
                            w.D, norm=w.norm, eps=w.eps, bias=dev.get("bias_out"), mean_out=mean,
                            rstd_out=rstd, stream=stream)
    if w.op == "swiglu":
        return add_norm_swiglu(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), dev["W"], w.I,
                               norm=w.norm, eps=w.eps, bias=dev.get("bias_out"), mean_out=mean, rstd_out=rstd,
                               stream=stream)
    return add_bias_norm_gelu(h, dev["x"], dev["residual"], dev["gamma"], dev.get("beta"), dev["W"],
                              bias_in=dev.get("bias_in"), bias_out=dev.get("bias_out"), norm=w.norm, eps=w.eps,
                              mean_out=mean, rstd_out=rstd, stream=stream)


def add_norm_qkv_static(x, residual, gamma, beta, W, Hq, Hkv, D, norm="rmsnorm", eps=1e-5, bias=None,
                        residual_out=None, q=None, k=None, v=None, mean_out=None, rstd_out=None, stream=None):
    """fnl_add_norm_qkv_static: fnl_add_norm_qkv without a handle and without
    any device allocation inside the library (its scratch is a static device
    array of the library; M <= 128). Output tensors not given are allocated
    here by torch, before the call. Returns the same dict as add_norm_qkv."""
    M, K, residual_out = _common(x, residual, gamma, beta, norm, residual_out, mean_out, rstd_out, W, bias)
    q = torch.empty(Hq, M, D, dtype=torch.bfloat16, device=x.device) if q is None else q
    k = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if k is None else k
    v = torch.empty(Hkv, M, D, dtype=torch.bfloat16, device=x.device) if v is None else v
    _need(q, "q", (Hq, M, D)); _need(k, "k", (Hkv, M, D)); _need(v, "v", (Hkv, M, D))
    st = lib().fnl_add_norm_qkv_static(_stream_ptr(stream), _p(x), _p(residual), _p(residual_out), _p(gamma),
                                       _p(beta), NORMS[norm], float(eps), _p(W), _p(bias), M, K, Hq, Hkv, D,
                                       _p(q), _p(k), _p(v), _p(mean_out), _p(rstd_out))
    if st != FNL_OK:
        raise FnlError(st, "fnl_add_norm_qkv_static")
    return {"residual_out": residual_out, "q": q, "k": k, "v": v, "mean": mean_out, "rstd": rstd_out}


def check_static(stream=None):
    """fnl_check_static: synchronise the stream and raise if a call of the
    allocation-free entry point gave up a bounded wait since the last check."""
    st = lib().fnl_check_static(_stream_ptr(stream))
    if st != FNL_OK:
        raise FnlError(st, "fnl_check_static")
