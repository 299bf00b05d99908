"""Thin ctypes binding of libsage (C ABI in include/sage.h).

Argument marshalling only: torch supplies device memory and the current
stream; every step of the attention path runs in the CUDA library.  If the
library is missing or fails to load, every entry point raises -- there is no
fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Dict, Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libsage.so")

SAGE_OK = 0
STATUS_NAMES = {
    0: "SAGE_OK", 1: "SAGE_ERR_INVALID_ARG", 2: "SAGE_ERR_UNSUPPORTED_HEADDIM",
    3: "SAGE_ERR_UNSUPPORTED_DTYPE", 4: "SAGE_ERR_UNSUPPORTED_ARCH", 5: "SAGE_ERR_WORKSPACE_TOO_SMALL",
    6: "SAGE_ERR_CUDA", 7: "SAGE_ERR_TIMEOUT", 8: "SAGE_ERR_MISALIGNED", 9: "SAGE_ERR_BAD_PAGE",
}
EXPORTED = ("sage_workspace_bytes", "sage_quant_qkv", "sage_attn_fwd_quantized", "sage_attn_fwd",
            "sage_debug_qk_int32", "sage_last_device_error", "sage_debug_bounded_wait",
            "sage_status_string", "sage_attn_fwd_noalloc", "sage_debug_f8_accum_probe",
            "sage_nvfp4_workspace_bytes", "sage_quant_nvfp4", "sage_attn_fwd_nvfp4_quantized",
            "sage_attn_fwd_nvfp4", "sage_debug_qk_nvfp4", "sage_debug_exp2_poly",
            "sage_debug_kv_quant_two_pass", "sage_quant_kernel_count", "sage_quant_nvfp4_kernel_count",
            "sage_attn_fwd_quantized_lse", "sage_attn_fwd_lse", "sage_debug_mma_rate",
            "sage_debug_wait_limit", "sage_kv_append", "sage_decode_workspace_bytes", "sage_attn_decode",
            "sage_kv_evict", "sage_attn_window_fwd")


class SageError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class SageParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("smooth_k", ctypes.c_int32),
                ("smooth_q", ctypes.c_int32), ("bq", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("pv_accum", ctypes.c_int32), ("return_lse", ctypes.c_int32), ("layout", ctypes.c_int32)]


PV_TWO_LEVEL, PV_TMEM_FP32 = 0, 1
LAYOUTS = {"HND": 0, "NHD": 1}


class SageQuantView(ctypes.Structure):
    _fields_ = [("q8", ctypes.c_void_p), ("k8", ctypes.c_void_p), ("v8t", ctypes.c_void_p),
                ("s_q", ctypes.c_void_p), ("s_k", ctypes.c_void_p), ("s_v", ctypes.c_void_p),
                ("km", ctypes.c_void_p), ("qbar", ctypes.c_void_p), ("dS", ctypes.c_void_p),
                ("Np", ctypes.c_int64), ("qkm", ctypes.c_void_p)]


class SageNvfp4View(ctypes.Structure):
    _fields_ = [("q4", ctypes.c_void_p), ("k4", ctypes.c_void_p), ("v4t", ctypes.c_void_p),
                ("sfq", ctypes.c_void_p), ("sfk", ctypes.c_void_p), ("sfv", ctypes.c_void_p),
                ("km", ctypes.c_void_p), ("qbar", ctypes.c_void_p), ("dS", ctypes.c_void_p),
                ("Np", ctypes.c_int64)]


class SageKvCache(ctypes.Structure):
    _fields_ = [("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("quantized", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("weight", ctypes.c_void_p)]


class SageKvSeqs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p)]


class SageDecodeParams(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("sm_scale", ctypes.c_float)]


class SageWindowParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("zero_tail", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsage.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libsage.so not built ({LIB_PATH}); run python -m quantized_attention_block_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        P, V = ctypes.POINTER(SageParams), ctypes.POINTER(SageQuantView)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        L.sage_workspace_bytes.argtypes, L.sage_workspace_bytes.restype = [P], ctypes.c_size_t
        L.sage_quant_qkv.argtypes = [vp, vp, vp, P, vp, ctypes.c_size_t, V, vp]
        L.sage_attn_fwd_quantized.argtypes = [V, vp, P, vp]
        L.sage_attn_fwd.argtypes = [vp, vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        L.sage_attn_fwd_quantized_lse.argtypes = [V, vp, vp, P, vp]
        L.sage_attn_fwd_quantized_lse.restype = ctypes.c_int
        L.sage_attn_fwd_lse.argtypes = [vp, vp, vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        L.sage_attn_fwd_lse.restype = ctypes.c_int
        L.sage_debug_qk_int32.argtypes = [V, P, i32, i32, i32, i32, vp, vp]
        L.sage_last_device_error.argtypes = [vp]
        L.sage_debug_bounded_wait.argtypes = [ctypes.c_uint32, vp]
        L.sage_status_string.argtypes, L.sage_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        L.sage_attn_fwd_noalloc.argtypes, L.sage_attn_fwd_noalloc.restype = [vp, vp, vp, vp, P, vp], ctypes.c_int
        L.sage_debug_f8_accum_probe.argtypes, L.sage_debug_f8_accum_probe.restype = [vp, vp], ctypes.c_int
        F = ctypes.POINTER(SageNvfp4View)
        L.sage_nvfp4_workspace_bytes.argtypes, L.sage_nvfp4_workspace_bytes.restype = [P], ctypes.c_size_t
        L.sage_quant_nvfp4.argtypes = [vp, vp, vp, P, vp, ctypes.c_size_t, F, vp]
        L.sage_attn_fwd_nvfp4_quantized.argtypes = [F, vp, P, vp]
        L.sage_attn_fwd_nvfp4.argtypes = [vp, vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        L.sage_debug_qk_nvfp4.argtypes = [F, P, i32, i32, i32, i32, vp, vp]
        L.sage_debug_exp2_poly.argtypes, L.sage_debug_exp2_poly.restype = [vp, vp, i32, vp], ctypes.c_int
        L.sage_debug_kv_quant_two_pass.argtypes, L.sage_debug_kv_quant_two_pass.restype = [i32], ctypes.c_int
        L.sage_debug_mma_rate.argtypes = [i32, i32, i32, i32, ctypes.POINTER(ctypes.c_double), vp]
        L.sage_debug_mma_rate.restype = ctypes.c_int
        L.sage_debug_wait_limit.argtypes, L.sage_debug_wait_limit.restype = [ctypes.c_uint32, vp], ctypes.c_int
        L.sage_quant_kernel_count.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        L.sage_quant_kernel_count.restype = ctypes.c_int
        L.sage_quant_nvfp4_kernel_count.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        L.sage_quant_nvfp4_kernel_count.restype = ctypes.c_int
        C, S = ctypes.POINTER(SageKvCache), ctypes.POINTER(SageKvSeqs)
        D, W = ctypes.POINTER(SageDecodeParams), ctypes.POINTER(SageWindowParams)
        L.sage_kv_append.argtypes, L.sage_kv_append.restype = [vp, vp, vp, vp, i32, i32, C, S, vp], ctypes.c_int
        L.sage_decode_workspace_bytes.argtypes = [C, S, D]
        L.sage_decode_workspace_bytes.restype = ctypes.c_size_t
        L.sage_attn_decode.argtypes = [vp, vp, vp, vp, C, S, D, vp, ctypes.c_size_t, vp]
        L.sage_attn_decode.restype = ctypes.c_int
        L.sage_kv_evict.argtypes = [C, S, vp, i32, i32, i32, i32, vp, vp, vp]
        L.sage_kv_evict.restype = ctypes.c_int
        L.sage_attn_window_fwd.argtypes, L.sage_attn_window_fwd.restype = [vp, vp, vp, vp, vp, vp, W, vp], ctypes.c_int
        for n in ("sage_quant_qkv", "sage_attn_fwd_quantized", "sage_attn_fwd", "sage_debug_qk_int32",
                  "sage_last_device_error", "sage_debug_bounded_wait", "sage_quant_nvfp4",
                  "sage_attn_fwd_nvfp4_quantized", "sage_attn_fwd_nvfp4", "sage_debug_qk_nvfp4"):
            getattr(L, n).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != SAGE_OK:
        raise SageError(status, what)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def make_params(q: torch.Tensor, k: torch.Tensor, *, causal: bool = False, sm_scale: Optional[float] = None,
                smooth_k: bool = True, smooth_q: bool = False, bq: int = 128, bk: int = 64,
                pv_accum: int = PV_TWO_LEVEL, return_lse: bool = False, tensor_layout: str = "HND") -> SageParams:
    """Parameters for q [B, Hq, N, d], k [B, Hkv, N, d] (tensor_layout "HND") or
    q [B, N, Hq, d], k [B, N, Hkv, d] ("NHD")."""
    if tensor_layout not in LAYOUTS:
        raise ValueError(f"tensor_layout must be one of {sorted(LAYOUTS)}")
    if tensor_layout == "HND":
        B, Hq, N, d = q.shape
        Hkv = k.shape[1]
    else:
        B, N, Hq, d = q.shape
        Hkv = k.shape[2]
    dt = {torch.bfloat16: 0, torch.float16: 1}.get(q.dtype, -1)
    return SageParams(B, Hq, Hkv, N, d, dt, int(causal), float(sm_scale if sm_scale else 0.0),
                      int(smooth_k), int(smooth_q), bq, bk, int(pv_accum), int(return_lse), LAYOUTS[tensor_layout])


def workspace_bytes(p: SageParams) -> int:
    return int(lib().sage_workspace_bytes(ctypes.byref(p)))


def alloc_workspace(p: SageParams, device=None) -> torch.Tensor:
    n = workspace_bytes(p)
    if n == 0:
        raise SageError(1, "sage_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def sage_quant_qkv(q, k, v, p: SageParams, workspace: torch.Tensor, stream=None) -> SageQuantView:
    view = SageQuantView()
    _check(lib().sage_quant_qkv(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(p), _ptr(workspace),
                                workspace.numel(), ctypes.byref(view), _stream(stream)), "sage_quant_qkv")
    return view


def sage_attn_fwd_quantized(view: SageQuantView, o: torch.Tensor, p: SageParams, stream=None) -> torch.Tensor:
    _check(lib().sage_attn_fwd_quantized(ctypes.byref(view), _ptr(o), ctypes.byref(p), _stream(stream)),
           "sage_attn_fwd_quantized")
    return o


def sage_attn_fwd(q, k, v, *, causal: bool = False, sm_scale: Optional[float] = None, smooth_k: bool = True,
                  smooth_q: bool = False, bq: int = 128, bk: int = 64, pv_accum: int = PV_TWO_LEVEL,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None, tensor_layout: str = "HND") -> torch.Tensor:
    """SageAttention forward: [B,Hq,N,d] x [B,Hkv,N,d] -> [B,Hq,N,d] (input dtype); with
    tensor_layout "NHD" the tensors are [B,N,H,d]."""
    p = make_params(q, k, causal=causal, sm_scale=sm_scale, smooth_k=smooth_k, smooth_q=smooth_q, bq=bq, bk=bk,
                    pv_accum=pv_accum, tensor_layout=tensor_layout)
    if workspace is None:
        workspace = alloc_workspace(p, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(lib().sage_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), ctypes.byref(p), _ptr(workspace),
                               workspace.numel(), _stream(stream)), "sage_attn_fwd")
    return out


def sage_attn_fwd_lse(q, k, v, *, causal: bool = False, sm_scale: Optional[float] = None, smooth_k: bool = True,
                      smooth_q: bool = False, bq: int = 128, bk: int = 64, pv_accum: int = PV_TWO_LEVEL,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None, tensor_layout: str = "HND"):
    """sage_attn_fwd that also returns each row's log-sum-exp of the scores
    (fp32 [B,Hq,N], natural log, for the original keys): (out, lse)."""
    p = make_params(q, k, causal=causal, sm_scale=sm_scale, smooth_k=smooth_k, smooth_q=smooth_q, bq=bq, bk=bk,
                    pv_accum=pv_accum, tensor_layout=tensor_layout)
    if workspace is None:
        workspace = alloc_workspace(p, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((p.B, p.Hq, p.N), dtype=torch.float32, device=q.device)
    _check(lib().sage_attn_fwd_lse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), ctypes.byref(p),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "sage_attn_fwd_lse")
    return out, lse


def sage_attn_fwd_quantized_lse(view: SageQuantView, o: torch.Tensor, lse: torch.Tensor, p: SageParams,
                                stream=None) -> None:
    _check(lib().sage_attn_fwd_quantized_lse(ctypes.byref(view), _ptr(o), _ptr(lse), ctypes.byref(p),
                                             _stream(stream)), "sage_attn_fwd_quantized_lse")


def sage_debug_qk_int32(view: SageQuantView, p: SageParams, b: int, h: int, qtile: int, ktile: int,
                        stream=None) -> torch.Tensor:
    out = torch.empty((128, 128), dtype=torch.int32, device="cuda")
    _check(lib().sage_debug_qk_int32(ctypes.byref(view), ctypes.byref(p), b, h, qtile, ktile, _ptr(out),
                                     _stream(stream)), "sage_debug_qk_int32")
    return out


def sage_last_device_error(stream=None) -> int:
    return int(lib().sage_last_device_error(_stream(stream)))


def sage_debug_bounded_wait(timeout_us: int, stream=None) -> int:
    return int(lib().sage_debug_bounded_wait(int(timeout_us), _stream(stream)))


F8_ACCUM_PROBE_EXACT = (1 + 2.0 ** -18, 1 + 2.0 ** -14, 1 + 2.0 ** -12, 256.0, 32.0, 4096 + 2.0 ** -10,
                        1 + 2.0 ** -18, 1 + 2.0 ** -13)


def sage_debug_f8_accum_probe(stream=None) -> torch.Tensor:
    """The 8 probe sums of the FP8 tensor-core accumulator (exact values in F8_ACCUM_PROBE_EXACT)."""
    out = torch.zeros(8, dtype=torch.float32, device="cuda")
    _check(lib().sage_debug_f8_accum_probe(_ptr(out), _stream(stream)), "sage_debug_f8_accum_probe")
    return out


def view_tensors(view: SageQuantView, p: SageParams, workspace: torch.Tensor) -> Dict[str, torch.Tensor]:
    """torch views of the quantised tensors inside the workspace (for inspection)."""
    B, Hq, Hkv, N, d = p.B, p.Hq, p.Hkv, p.N, p.d
    Np = int(view.Np)
    Tm, Tn = -(-N // p.bq), -(-N // p.bk)
    base = workspace.data_ptr()

    def sl(ptr, nbytes, dtype, shape):
        off = ptr - base
        return workspace[off:off + nbytes].view(dtype).view(*shape)

    out = {
        "q8": sl(view.q8, B * Hq * Np * d, torch.int8, (B, Hq, Np, d)),
        "k8": sl(view.k8, B * Hkv * Np * d, torch.int8, (B, Hkv, Np, d)),
        "v8t": sl(view.v8t, B * Hkv * d * Np, torch.uint8, (B, Hkv, d, Np)),
        "s_q": sl(view.s_q, 4 * B * Hq * Tm, torch.float32, (B, Hq, Tm)),
        "s_k": sl(view.s_k, 4 * B * Hkv * Tn, torch.float32, (B, Hkv, Tn)),
        "s_v": sl(view.s_v, 4 * B * Hkv * d, torch.float32, (B, Hkv, d)),
        "km": sl(view.km, 4 * B * Hkv * d, torch.float32, (B, Hkv, d)),
    }
    if view.qkm:
        out["qkm"] = sl(view.qkm, 4 * B * Hq * Np, torch.float32, (B, Hq, Np))
    if view.qbar:
        out["qbar"] = sl(view.qbar, 4 * B * Hq * Tm * d, torch.float32, (B, Hq, Tm, d))
        out["dS"] = sl(view.dS, 4 * B * Hq * Tm * Np, torch.float32, (B, Hq, Tm, Np))
    return out


# ---------------------------------------------------------------- NVFP4 path
def nvfp4_workspace_bytes(p: SageParams) -> int:
    return int(lib().sage_nvfp4_workspace_bytes(ctypes.byref(p)))


def alloc_nvfp4_workspace(p: SageParams, device=None) -> torch.Tensor:
    n = nvfp4_workspace_bytes(p)
    if n == 0:
        raise SageError(1, "sage_nvfp4_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def sage_quant_nvfp4(q, k, v, p: SageParams, workspace: torch.Tensor, stream=None) -> SageNvfp4View:
    view = SageNvfp4View()
    _check(lib().sage_quant_nvfp4(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(p), _ptr(workspace),
                                  workspace.numel(), ctypes.byref(view), _stream(stream)), "sage_quant_nvfp4")
    return view


def sage_attn_fwd_nvfp4_quantized(view: SageNvfp4View, o: torch.Tensor, p: SageParams,
                                  stream=None) -> torch.Tensor:
    _check(lib().sage_attn_fwd_nvfp4_quantized(ctypes.byref(view), _ptr(o), ctypes.byref(p), _stream(stream)),
           "sage_attn_fwd_nvfp4_quantized")
    return o


def sage_attn_fwd_nvfp4(q, k, v, *, causal: bool = False, sm_scale: Optional[float] = None,
                        smooth_k: bool = True, smooth_q: bool = True, bq: int = 128,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None, tensor_layout: str = "HND") -> torch.Tensor:
    """SageAttention3-style NVFP4 forward: [B,Hq,N,128] x [B,Hkv,N,128] -> [B,Hq,N,128]
    (tensor_layout "NHD": [B,N,H,128])."""
    p = make_params(q, k, causal=causal, sm_scale=sm_scale, smooth_k=smooth_k, smooth_q=smooth_q, bq=bq,
                    tensor_layout=tensor_layout)
    if workspace is None:
        workspace = alloc_nvfp4_workspace(p, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(lib().sage_attn_fwd_nvfp4(_ptr(q), _ptr(k), _ptr(v), _ptr(out), ctypes.byref(p), _ptr(workspace),
                                     workspace.numel(), _stream(stream)), "sage_attn_fwd_nvfp4")
    return out


def sage_debug_qk_nvfp4(view: SageNvfp4View, p: SageParams, b: int, h: int, qtile: int, ktile: int,
                        stream=None) -> torch.Tensor:
    out = torch.empty((128, 128), dtype=torch.float32, device="cuda")
    _check(lib().sage_debug_qk_nvfp4(ctypes.byref(view), ctypes.byref(p), b, h, qtile, ktile, _ptr(out),
                                     _stream(stream)), "sage_debug_qk_nvfp4")
    return out


def sage_debug_exp2_poly(x: torch.Tensor, stream=None) -> torch.Tensor:
    """2^x of a float32 device tensor through the kernel's FMA-pipe exponential."""
    y = torch.empty_like(x)
    _check(lib().sage_debug_exp2_poly(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "sage_debug_exp2_poly")
    return y


MMA_KINDS = {"i8": 0, "f8": 1, "f4": 2}


def sage_debug_mma_rate(kind: str, n: int, iters: int, ctas: int = 0, stream=None) -> float:
    """Enqueue the tensor-core rate probe (one CTA per SM by default) on `stream`
    and return the operation count of that launch; time it with CUDA events."""
    ops = ctypes.c_double(0.0)
    _check(lib().sage_debug_mma_rate(MMA_KINDS[kind], int(n), int(iters), int(ctas), ctypes.byref(ops),
                                     _stream(stream)), "sage_debug_mma_rate")
    return float(ops.value)


def sage_quant_kernel_count(p: SageParams) -> int:
    """Kernels sage_quant_qkv enqueues for p on the current device (memsets not counted)."""
    n = ctypes.c_int32(0)
    _check(lib().sage_quant_kernel_count(ctypes.byref(p), ctypes.byref(n)), "sage_quant_kernel_count")
    return int(n.value)


def sage_quant_nvfp4_kernel_count(p: SageParams) -> int:
    """Kernels sage_quant_nvfp4 enqueues for p on the current device (memsets not counted)."""
    n = ctypes.c_int32(0)
    _check(lib().sage_quant_nvfp4_kernel_count(ctypes.byref(p), ctypes.byref(n)), "sage_quant_nvfp4_kernel_count")
    return int(n.value)


def sage_debug_kv_quant_two_pass(on) -> None:
    """Force (True / 1) or release (False / 0) the two-pass K/V quantisation path in
    this process; 2 forces the one-read path even when a group's tiles may not
    all be resident (a test of its bounded waits)."""
    _check(lib().sage_debug_kv_quant_two_pass(int(on)), "sage_debug_kv_quant_two_pass")


def sage_debug_wait_limit(timeout_us: int, stream=None) -> None:
    """Limit of the in-kernel bounded waits for later launches (0: the default 4 s)."""
    _check(lib().sage_debug_wait_limit(int(timeout_us), _stream(stream)), "sage_debug_wait_limit")


def nvfp4_view_tensors(view: SageNvfp4View, p: SageParams, workspace: torch.Tensor) -> Dict[str, torch.Tensor]:
    """torch views (raw device layouts) of the NVFP4 tensors inside the workspace."""
    B, Hq, Hkv, N, d = p.B, p.Hq, p.Hkv, p.N, p.d
    Np = int(view.Np)
    T, Tm = Np // 128, -(-N // p.bq)
    base = workspace.data_ptr()

    def sl(ptr, nbytes, dtype, shape):
        off = ptr - base
        return workspace[off:off + nbytes].view(dtype).view(*shape)

    out = {
        "q4": sl(view.q4, B * Hq * Np * d // 2, torch.uint8, (B, Hq, Np, d // 2)),
        "k4": sl(view.k4, B * Hkv * Np * d // 2, torch.uint8, (B, Hkv, Np, d // 2)),
        "v4t": sl(view.v4t, B * Hkv * d * Np // 2, torch.uint8, (B, Hkv, d, Np // 2)),
        "sfq": sl(view.sfq, B * Hq * T * 1024, torch.uint8, (B, Hq, T, 1024)),
        "sfk": sl(view.sfk, B * Hkv * T * 1024, torch.uint8, (B, Hkv, T, 1024)),
        "sfv": sl(view.sfv, B * Hkv * T * 1024, torch.uint8, (B, Hkv, T, 1024)),
        "km": sl(view.km, 4 * B * Hkv * d, torch.float32, (B, Hkv, d)),
    }
    if view.qbar:
        out["qbar"] = sl(view.qbar, 4 * B * Hq * Tm * d, torch.float32, (B, Hq, Tm, d))
        out["dS"] = sl(view.dS, 4 * B * Hq * Tm * Np, torch.float32, (B, Hq, Tm, Np))
    return out


# ---------------------------------------------------------------- serving: paged cache, one-token and window attention
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _expect(name: str, t: torch.Tensor, shape, dtype) -> None:
    """A contiguous tensor of this shape (None: any extent) and type, else ValueError."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _one_device(names: str, index: int, *ts) -> int:
    """`index`, the number of the CUDA device that all the tensors (None: absent) must be on."""
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{names} must be on one device, got {[str(x.device) for x in ts if x is not None]} "
                             f"beside device {index}")
    if index < 0:
        raise ValueError(f"{names} must be on a CUDA device")
    return index


def _layout(tensor_layout: str) -> int:
    if tensor_layout not in LAYOUTS:
        raise ValueError(f"tensor_layout must be one of {sorted(LAYOUTS)}")
    return LAYOUTS[tensor_layout]


def _range32(names: str, *ns) -> None:
    for n in ns:
        if not 0 <= n < 2147483648:
            raise ValueError(f"{names} must be in [0, 2^31), got {ns}")


# torch's own number of the current device and handle of a device's current stream, without the objects around
# them (the tensors of the call are on a CUDA device, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index: int, stream: Optional[torch.cuda.Stream], work):
    """work(raw stream) on a device (by number) and a stream (None: the device's current one), which are current
    meanwhile, so that tensors made there belong to both."""
    if stream is None:
        if index == _current_device():
            return work(_raw_stream(index))
        with torch.cuda.device(index):
            return work(_raw_stream(index))
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return work(stream.cuda_stream)


class KVCache:
    """A pool of pages of keys and values (sage_kv_cache), around the caller's tensors.

    k_pages, v_pages: [n_pages, Hkv, page_size, d] (tensor_layout "HND") or
    [n_pages, page_size, Hkv, d] ("NHD"); bf16 or fp16, or int8 keys with
    float8_e4m3fn values, which need k_scale and v_scale, fp32
    [n_pages, Hkv, page_size] in either layout.  weight (same shape, optional):
    the attention weight that each cached token has gathered.  `alloc` makes the
    tensors.  The pages of a sequence are named by the page table of each call.
    """

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None, weight=None, *, tensor_layout: str = "HND"):
        layout = _layout(tensor_layout)
        if k_pages.dim() != 4:
            raise ValueError(f"k_pages must have 4 dimensions, got {tuple(k_pages.shape)}")
        self.quantized = k_pages.dtype == torch.int8
        _expect("k_pages", k_pages, k_pages.shape, k_pages.dtype)
        _expect("v_pages", v_pages, k_pages.shape, torch.float8_e4m3fn if self.quantized else k_pages.dtype)
        if not self.quantized and k_pages.dtype not in _DTYPES:
            raise ValueError(f"pages must be bfloat16, float16 or int8 (keys), got {k_pages.dtype}")
        n_pages, a, b, d = k_pages.shape
        heads, page = (a, b) if layout == 0 else (b, a)
        if page < 16 or page > 1024 or page & (page - 1):
            raise ValueError(f"page_size must be a power of two from 16 to 1024, got {page}")
        if d not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {d}")
        if self.quantized != (k_scale is not None) or self.quantized != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with int8 keys and float8_e4m3fn values")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale), ("weight", weight)):
            if t is not None:
                _expect(name, t, (n_pages, heads, page), torch.float32)
        self.k_pages, self.v_pages, self.k_scale, self.v_scale, self.weight = k_pages, v_pages, k_scale, v_scale, weight
        self.n_pages, self.Hkv, self.page_size, self.d, self.tensor_layout = n_pages, heads, page, d, tensor_layout
        self.device = k_pages.device
        self._index = k_pages.get_device() if k_pages.is_cuda else -1
        self._ws_bytes, self._no_workspace = {}, torch.empty(256, dtype=torch.uint8, device=self.device)
        for t in (v_pages, k_scale, v_scale, weight):
            if t is not None and t.device != self.device:
                raise ValueError(f"the cache's tensors must be on one device, got {self.device} and {t.device}")
        # one struct for each type of the tokens (a 16-bit cache has one)
        self._c = {dt: SageKvCache(heads, d, code, int(self.quantized), page, n_pages, layout, _ptr(k_pages),
                                   _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(weight))
                   for dt, code in _DTYPES.items() if self.quantized or dt == k_pages.dtype}

    @classmethod
    def alloc(cls, n_pages: int, page_size: int, Hkv: int, d: int, dtype=torch.bfloat16, *, quantized: bool = False,
              track_weight: bool = False, tensor_layout: str = "HND", device="cuda") -> "KVCache":
        """An empty pool: 16-bit pages of `dtype`, or INT8 keys and E4M3 values."""
        shape = (n_pages, Hkv, page_size, d) if _layout(tensor_layout) == 0 else (n_pages, page_size, Hkv, d)
        k = torch.zeros(shape, dtype=torch.int8 if quantized else dtype, device=device)
        v = torch.zeros(shape, dtype=torch.int8, device=device).view(torch.float8_e4m3fn) if quantized else k.clone()
        scale = (n_pages, Hkv, page_size)
        s = [torch.zeros(scale, dtype=torch.float32, device=device) if quantized else None for _ in range(2)]
        w = torch.zeros(scale, dtype=torch.float32, device=device) if track_weight else None
        return cls(k, v, *s, w, tensor_layout=tensor_layout)

    def _struct(self, dtype) -> SageKvCache:
        c = self._c.get(dtype)
        if c is None:
            raise ValueError(f"the cache takes tokens of {' or '.join(map(str, self._c))}, got {dtype}")
        return c

    def _workspace(self, q, sizes, args) -> torch.Tensor:
        """A workspace for a decode of these sizes (the number of bytes goes by them alone)."""
        n = self._ws_bytes.get(sizes)
        if n is None:
            n = self._ws_bytes[sizes] = int(lib().sage_decode_workspace_bytes(*args))
        if n <= 256:  # nothing is kept there: any place will do
            return self._no_workspace
        return q.new_empty((n,), dtype=torch.uint8)

    def _seqs(self, page_table, lens) -> SageKvSeqs:
        shape = page_table.shape if isinstance(page_table, torch.Tensor) else ()
        if len(shape) != 2 or page_table.dtype is not torch.int32 or not page_table.is_contiguous():
            _expect("page_table", page_table, (None, None), torch.int32)
        B, max_pages = shape
        _expect("lens", lens, (B,), torch.int32)
        if B < 1 or max_pages < 1:
            raise ValueError(f"page_table must not be empty, got {tuple(shape)}")
        return SageKvSeqs(B, max_pages, page_table.data_ptr(), lens.data_ptr())


def sage_kv_append(k, v, cache: KVCache, page_table, lens, *, n_new=None, km=None, tensor_layout: str = "HND",
                   stream=None) -> None:
    """Write new tokens k, v [B,Hkv,T,d] ("NHD": [B,T,Hkv,d]) behind the lens[b] tokens that sequence
    b holds in the pages page_table[b] (int32 [B, max_pages]); of sequence b the first n_new[b]
    (default: T).  lens is not changed.  Quantised caches store INT8 codes of k - km (km: fp32
    [B,Hkv,d], optional) and E4M3 codes of v, with one scale per token and head."""
    layout = _layout(tensor_layout)
    c, s = cache._struct(k.dtype), cache._seqs(page_table, lens)
    T = k.shape[2 - layout] if k.dim() == 4 else 0
    shape = (s.B, cache.Hkv, T, cache.d) if layout == 0 else (s.B, T, cache.Hkv, cache.d)
    _expect("k", k, shape, k.dtype)
    _expect("v", v, shape, k.dtype)
    if n_new is not None:
        _expect("n_new", n_new, (s.B,), torch.int32)
    if km is not None:
        if not cache.quantized:
            raise ValueError("km goes with a quantized cache")
        _expect("km", km, (s.B, cache.Hkv, cache.d), torch.float32)
    index = _one_device("cache, k, v, page_table, lens, n_new, km", cache._index, k, v, page_table, lens, n_new, km)
    _on(index, stream, lambda raw: _check(
        lib().sage_kv_append(k.data_ptr(), v.data_ptr(), _ptr(n_new), _ptr(km), T, layout, ctypes.byref(c),
                             ctypes.byref(s), raw), "sage_kv_append"))


def decode_workspace_bytes(cache: KVCache, page_table, lens, Hq: int, *, window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace of sage_attn_decode for these sizes (0: invalid)."""
    _range32("window, sinks", window, sinks)
    p = SageDecodeParams(Hq, window, sinks, 0.0)
    c = next(iter(cache._c.values()))
    return int(lib().sage_decode_workspace_bytes(ctypes.byref(c), ctypes.byref(cache._seqs(page_table, lens)),
                                                 ctypes.byref(p)))


def _decode(q, cache, page_table, lens, window, sinks, sm_scale, km, out, lse, want_lse, workspace, stream):
    _range32("window, sinks", window, sinks)
    c, s = cache._struct(q.dtype), cache._seqs(page_table, lens)
    B, max_pages = page_table.shape
    Hq = q.shape[1] if q.dim() == 3 else 0
    _expect("q", q, (B, Hq, cache.d), q.dtype)
    if Hq < 1 or Hq % cache.Hkv:
        raise ValueError(f"query heads must be a multiple of {cache.Hkv}, got {Hq}")
    index = _one_device("cache, q, page_table, lens", cache._index, q, page_table, lens)
    if out is not None:
        _expect("out", out, q.shape, q.dtype)
    if lse is not None:
        _expect("lse", lse, (B, Hq), torch.float32)
    if km is not None:
        if not cache.quantized:
            raise ValueError("km goes with a quantized cache")
        _expect("km", km, (B, cache.Hkv, cache.d), torch.float32)
    if workspace is not None:
        _expect("workspace", workspace, (workspace.numel(),), torch.uint8)
    if not (out is lse is km is workspace is None):
        _one_device("cache, km, out, lse, workspace", index, km, out, lse, workspace)
    p = SageDecodeParams(Hq, window, sinks, float(sm_scale if sm_scale else 0.0))
    args = ctypes.byref(c), ctypes.byref(s), ctypes.byref(p)

    def work(raw):
        o = torch.empty_like(q) if out is None else out
        z = q.new_empty((B, Hq), dtype=torch.float32) if lse is None and want_lse else lse
        ws = cache._workspace(q, (B, max_pages, Hq, window, sinks), args) if workspace is None else workspace
        _check(lib().sage_attn_decode(q.data_ptr(), o.data_ptr(), _ptr(z), _ptr(km), *args, ws.data_ptr(), ws.numel(),
                                      raw), "sage_attn_decode")
        return o, z

    return _on(index, stream, work)


def sage_attn_decode(q, cache: KVCache, page_table, lens, *, window: int = 0, sinks: int = 0,
                     sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token a sequence: q [B,Hq,d] at position lens[b] - 1 over the lens[b] tokens
    of sequence b in the cache -> [B,Hq,d].  window > 0: the last `window` keys and the first `sinks`
    tokens alone.  If the cache tracks weights, they grow by this token's attention."""
    return _decode(q, cache, page_table, lens, window, sinks, sm_scale, None, out, None, False, workspace, stream)[0]


def sage_attn_decode_lse(q, cache: KVCache, page_table, lens, *, window: int = 0, sinks: int = 0,
                         sm_scale: Optional[float] = None, km=None, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """sage_attn_decode that also returns each head's log-sum-exp of the scores (fp32 [B,Hq], natural log;
    with km, the mean that a quantized cache's keys are stored without, for the keys as they were):
    (out, lse)."""
    return _decode(q, cache, page_table, lens, window, sinks, sm_scale, km, out, lse, True, workspace, stream)


def sage_kv_evict(cache: KVCache, page_table, lens, dst_table, keep: int, *, sinks: int = 0, recent: int = 0,
                  new_lens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None, stream=None):
    """Hold every sequence to `keep` tokens: the first `sinks`, the last `recent`, and those of the others
    with the largest gathered weight, per head.  They move, in order, to the pages dst_table [B, n] (int32),
    which no sequence may be using.  Returns (new_lens [B], kept [B,Hkv,keep]: old positions, -1 behind)."""
    if cache.weight is None:
        raise ValueError("the cache does not track weights")
    _range32("keep, sinks, recent", keep, sinks, recent)
    if keep < 1 or sinks + recent > keep:
        raise ValueError(f"keep must be at least 1 and hold sinks and recent, got {keep}, {sinks}, {recent}")
    c, s = next(iter(cache._c.values())), cache._seqs(page_table, lens)
    n = dst_table.shape[1] if dst_table.dim() == 2 else 0
    _expect("dst_table", dst_table, (s.B, n), torch.int32)
    if dst_table.shape[1] * cache.page_size < keep:
        raise ValueError(f"dst_table holds {dst_table.shape[1]} pages of {cache.page_size}: too few for {keep} tokens")
    if new_lens is not None:
        _expect("new_lens", new_lens, (s.B,), torch.int32)
    if kept is not None:
        _expect("kept", kept, (s.B, cache.Hkv, keep), torch.int32)
    index = _one_device("cache, page_table, lens, dst_table, new_lens, kept", cache._index, page_table, lens,
                        dst_table, new_lens, kept)

    def work(raw):
        n = torch.empty_like(lens) if new_lens is None else new_lens
        at = lens.new_empty((s.B, cache.Hkv, keep)) if kept is None else kept
        _check(lib().sage_kv_evict(ctypes.byref(c), ctypes.byref(s), dst_table.data_ptr(), dst_table.shape[1], keep,
                                   sinks, recent, n.data_ptr(), at.data_ptr(), raw), "sage_kv_evict")
        return n, at

    return _on(index, stream, work)


def _window_fwd(q, k, v, window, sinks, lens, sm_scale, out, lse, want_lse, stream, tensor_layout):
    layout = _layout(tensor_layout)
    _range32("window, sinks", window, sinks)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must have 4 dimensions, got {tuple(q.shape)} and {tuple(k.shape)}")
    if q.dtype not in _DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    B, Hq, N, d = q.shape if layout == 0 else (q.shape[0], q.shape[2], q.shape[1], q.shape[3])
    Hkv = k.shape[1 + layout]
    kv_shape = (B, Hkv, N, d) if layout == 0 else (B, N, Hkv, d)
    _expect("q", q, q.shape, q.dtype)
    _expect("k", k, kv_shape, q.dtype)
    _expect("v", v, kv_shape, q.dtype)
    if lens is not None:
        _expect("lens", lens, (B,), torch.int32)
    if out is not None:
        _expect("out", out, q.shape, q.dtype)
    if lse is not None:
        _expect("lse", lse, (B, Hq, N), torch.float32)
    index = _one_device("q, k, v, lens, out, lse", q.get_device(), k, v, lens, out, lse)
    # rows behind a sequence's end are not written: zeros in tensors made here
    zero = 0 if lens is None else (1 if out is None else 0) | (2 if lse is None else 0)
    p = SageWindowParams(B, Hq, Hkv, N, d, _DTYPES[q.dtype], layout, window, sinks, float(sm_scale if sm_scale else 0.0),
                         zero)

    def work(raw):
        o = torch.empty_like(q) if out is None else out
        z = q.new_empty((B, Hq, N), dtype=torch.float32) if lse is None and want_lse else lse
        _check(lib().sage_attn_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(z), _ptr(lens),
                                          ctypes.byref(p), raw), "sage_attn_window_fwd")
        return o, z

    return _on(index, stream, work)


def sage_attn_window_fwd(q, k, v, *, window: int, sinks: int = 0, lens=None, sm_scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, stream=None, tensor_layout: str = "HND") -> torch.Tensor:
    """Sliding-window causal attention in the inputs' 16-bit type: row i sees the last `window` keys up to
    its own (0: all of them) and the first `sinks`.  [B,Hq,N,d] x [B,Hkv,N,d] -> [B,Hq,N,d] ("NHD":
    [B,N,H,d]).  lens (int32 [B], optional): rows behind a sequence's length are not written (zeros in an
    output made here) and not read."""
    return _window_fwd(q, k, v, window, sinks, lens, sm_scale, out, None, False, stream, tensor_layout)[0]


def sage_attn_window_fwd_lse(q, k, v, *, window: int, sinks: int = 0, lens=None, sm_scale: Optional[float] = None,
                             out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None,
                             tensor_layout: str = "HND"):
    """sage_attn_window_fwd that also returns each row's log-sum-exp (fp32 [B,Hq,N], natural log): (out, lse)."""
    return _window_fwd(q, k, v, window, sinks, lens, sm_scale, out, lse, True, stream, tensor_layout)


def attention_ops(B: int, Hq: int, N: int, d: int, causal: bool) -> float:
    """4 N^2 d per head (two matmuls), halved when causal (the TOPS numerator)."""
    full = 4.0 * B * Hq * N * N * d
    return full / 2 if causal else full
