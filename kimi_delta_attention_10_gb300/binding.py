"""Binding of libkda_gb300.so (include/kda.h): argument marshalling only, by ctypes and,
for the paged-attention calls, by the C++ module _marshal.

Every computation runs in the library's CUDA kernels; PyTorch provides the
device memory and the stream.  There is no fallback: if the library is
missing, or a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sys
import threading
from typing import Optional, Sequence, Tuple

import torch

from . import _build

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_ALIGNMENT = 3
KDA_ERR_CUDA = 4
KDA_ERR_TIMEOUT = 5
KDA_ERR_DEVICE_ARG = 6
KDA_ERR_TOO_LARGE = 7
KDA_ERR_RANGE = 8
KDA_ERR_NO_PAGES = 9

# kda_test_set_fault values (test hook)
KDA_TEST_FAULT_NONE = 0
KDA_TEST_FAULT_SCAN = 1
KDA_TEST_FAULT_PREP = 2
KDA_TEST_FAULT_SINGLE_PASS = 3

KDA_F32 = 0
KDA_BF16 = 1

KDA_MODE_BF16_TC = 0
KDA_MODE_FP32_EXACT = 1

MODES = {"bf16_tc": KDA_MODE_BF16_TC, "fp32_exact": KDA_MODE_FP32_EXACT}

# Every symbol include/kda.h declares.
EXPORTS = ("kda_gate", "kda_chunk_workspace_size", "kda_chunk_fwd", "kda_chunk_fwd_gated",
           "kda_chunk_fwd_gated_norm",
           "kda_chunk_fwd_static", "kda_recurrent_step", "kda_gated_rmsnorm",
           "kda_chunk_bwd_workspace_size", "kda_chunk_bwd", "kda_page_plan",
           "kda_rope_inv_freq", "kda_qk_norm_rope", "kda_qk_norm_rope_append",
           "kda_qk_norm_rope_bwd_workspace_size", "kda_qk_norm_rope_bwd",
           "kda_paged_decode_workspace_size", "kda_paged_decode", "kda_test_set_fault",
           "kda_status_string", "kda_abi_version")

_lock = threading.Lock()
_lib = None


class KDAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libkda_gb300.so (optionally building it first)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(
                    f"{path} is missing: build it with kimi_delta_attention_10_gb300._build.build()")
            _build.build()
        lib = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        lib.kda_gate.argtypes = [vp, i32, vp, vp, vp, i32, i64, i32, i32, vp, vp, vp]
        lib.kda_gate.restype = i32
        lib.kda_chunk_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32,
                                                 ctypes.POINTER(i64)]
        lib.kda_chunk_workspace_size.restype = i32
        lib.kda_chunk_fwd.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                      ctypes.c_float, i32, i32, vp, i32, vp, vp, vp, i64, vp, vp]
        lib.kda_chunk_fwd.restype = i32
        lib.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp,
                                            i32, i64, i32, i32, i32, ctypes.c_float, i32, i32,
                                            vp, i32, vp, vp, vp, i64, vp, vp]
        lib.kda_chunk_fwd_gated.restype = i32
        lib.kda_chunk_fwd_gated_norm.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, vp,
                                                 vp, i32, i64, i32, i32, i32, ctypes.c_float, i32,
                                                 i32, vp, i32, vp, ctypes.c_float, vp, i32, vp, vp,
                                                 vp, i64, vp, vp]
        lib.kda_chunk_fwd_gated_norm.restype = i32
        lib.kda_chunk_fwd_static.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i64, i32, i32,
                                             i32, ctypes.c_float, i32, vp, i32, vp, vp, vp, vp]
        lib.kda_chunk_fwd_static.restype = i32
        lib.kda_recurrent_step.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32,
                                           ctypes.c_float, i32, vp, vp, i32, vp]
        lib.kda_recurrent_step.restype = i32
        lib.kda_gated_rmsnorm.argtypes = [vp, i32, vp, i32, vp, i64, i32, ctypes.c_float, vp, i32,
                                          vp]
        lib.kda_gated_rmsnorm.restype = i32
        lib.kda_chunk_bwd_workspace_size.argtypes = [i32, i64, i32, i32, i32, ctypes.POINTER(i64)]
        lib.kda_chunk_bwd_workspace_size.restype = i32
        lib.kda_chunk_bwd.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                      ctypes.c_float, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                      vp, vp, i64, vp, vp]
        lib.kda_chunk_bwd.restype = i32
        f32, f64 = ctypes.c_float, ctypes.c_double
        lib.kda_page_plan.argtypes = [vp, vp, i32, i64, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp,
                                      vp, vp]
        lib.kda_page_plan.restype = i32
        lib.kda_rope_inv_freq.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
        lib.kda_rope_inv_freq.restype = i32
        rope = [vp, vp, i32, i32, f32, vp, vp, f32, i32, i64, i32, i32, i32]
        lib.kda_qk_norm_rope.argtypes = [vp, i64, vp, i64, i32, *rope, vp, vp, i32, vp]
        lib.kda_qk_norm_rope.restype = i32
        lib.kda_qk_norm_rope_append.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, *rope, vp, vp,
                                                vp, i32, i32, i32, vp, vp]
        lib.kda_qk_norm_rope_append.restype = i32
        lib.kda_qk_norm_rope_bwd_workspace_size.argtypes = [i64, i32, i32, i32,
                                                            ctypes.POINTER(i64)]
        lib.kda_qk_norm_rope_bwd_workspace_size.restype = i32
        lib.kda_qk_norm_rope_bwd.argtypes = [vp, i64, vp, i64, i32, vp, vp, i32, *rope, vp, vp,
                                             i32, vp, vp, vp, i64, vp]
        lib.kda_qk_norm_rope_bwd.restype = i32
        lib.kda_paged_decode_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i64)]
        lib.kda_paged_decode_workspace_size.restype = i32
        lib.kda_paged_decode.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                         i32, f32, vp, i32, vp, vp, i64, vp, vp]
        lib.kda_paged_decode.restype = i32
        lib.kda_test_set_fault.argtypes = [i32]
        lib.kda_test_set_fault.restype = i32
        lib.kda_status_string.argtypes = [i32]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_abi_version.argtypes = []
        lib.kda_abi_version.restype = i32
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def set_test_fault(where: int) -> None:
    """Test hook: make CTA 0 of the named kernel lose one arrival so that its
    bounded wait gives up (KDA_TEST_FAULT_*; KDA_TEST_FAULT_NONE turns it off)."""
    st = load_library().kda_test_set_fault(int(where))
    if st != KDA_OK:
        raise KDAError(st, "kda_test_set_fault")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev_ptr(t: Optional[torch.Tensor], name: str) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream_handle(stream: Optional[torch.cuda.Stream], device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def kda_gate(f: torch.Tensor, A_log: torch.Tensor, dt_bias: torch.Tensor, b: torch.Tensor,
             g_out: Optional[torch.Tensor] = None, beta_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """g = -exp(A_log[h]) * softplus(f + dt_bias), beta = sigmoid(b) (FP32 outputs)."""
    lib = load_library()
    T, H, K = f.shape
    if g_out is None:
        g_out = torch.empty((T, H, K), dtype=torch.float32, device=f.device)
    if beta_out is None:
        beta_out = torch.empty((T, H), dtype=torch.float32, device=f.device)
    st = lib.kda_gate(_dev_ptr(f, "f"), _dtype_code(f), _dev_ptr(A_log, "A_log"),
                      _dev_ptr(dt_bias, "dt_bias"), _dev_ptr(b, "b"), _dtype_code(b), T, H, K,
                      _dev_ptr(g_out, "g_out"), _dev_ptr(beta_out, "beta_out"),
                      _stream_handle(stream, f.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_gate")
    return g_out, beta_out


def _chunk_outputs(q, v, cu_seqlens, out, out_dtype, output_final_state, final_state):
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((T, H, V), dtype=out_dtype or v.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    return out, final_state


def chunk_workspace_size(N: int, T: int, H: int, K: int = 128, V: int = 128,
                         mode: str = "bf16_tc") -> int:
    """Bytes of workspace the mode's two-phase chunk path needs."""
    out = ctypes.c_int64(0)
    st = load_library().kda_chunk_workspace_size(N, T, H, K, V, MODES[mode], ctypes.byref(out))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_workspace_size")
    return out.value


def _workspace(workspace, mode, N, T, H, K, V, device):
    """(pointer, bytes) for the call: None -> no workspace (single-pass
    kernel); "auto" -> a fresh buffer of the size the mode's two-phase path
    needs; a tensor -> its storage."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be None, 'auto' or a CUDA tensor")
        workspace = torch.empty(chunk_workspace_size(N, T, H, K, V, mode), dtype=torch.uint8,
                                device=device)
    ptr = _dev_ptr(workspace, "workspace")
    return ptr, workspace.numel() * workspace.element_size(), workspace


def _host_offsets(cu_seqlens_host):
    if cu_seqlens_host is None:
        return None, None
    arr = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def kda_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, cu_seqlens: torch.Tensor, scale: Optional[float] = None,
                  mode: str = "bf16_tc", out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, output_final_state: bool = True,
                  final_state: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  cu_seqlens_host: Optional[Sequence[int]] = None, qk_l2norm: bool = True,
                  status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, workspace="auto"):
    """Chunked KDA forward.  Returns (out [T,H,V], final_state [N,H,K,V] or None).

    workspace: "auto" (bf16_tc allocates the two-phase path's scratch), a CUDA
    tensor of at least chunk_workspace_size(...) bytes, or None (single-pass
    kernel, no scratch)."""
    lib = load_library()
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    out, final_state = _chunk_outputs(q, v, cu_seqlens, out, out_dtype, output_final_state,
                                      final_state)
    keep, host = _host_offsets(cu_seqlens_host)
    ws, ws_bytes, ws_keep = _workspace(workspace, mode, N, T, H, K, V, q.device)
    st = lib.kda_chunk_fwd(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(g, "g"), _dev_ptr(beta, "beta"), _dev_ptr(cu_seqlens, "cu_seqlens"), host,
        N, T, H, K, V, float(scale), 1 if qk_l2norm else 0, MODES[mode],
        _dev_ptr(out, "out"), _dtype_code(out), _dev_ptr(initial_state, "initial_state"),
        _dev_ptr(final_state, "final_state"), ws, ws_bytes, _dev_ptr(status, "status"),
        _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd")
    return out, final_state


def kda_chunk_fwd_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, f: torch.Tensor,
                        A_log: torch.Tensor, dt_bias: torch.Tensor, b: torch.Tensor,
                        cu_seqlens: torch.Tensor, scale: Optional[float] = None,
                        mode: str = "bf16_tc", out: Optional[torch.Tensor] = None,
                        out_dtype: Optional[torch.dtype] = None, output_final_state: bool = True,
                        final_state: Optional[torch.Tensor] = None,
                        initial_state: Optional[torch.Tensor] = None,
                        cu_seqlens_host: Optional[Sequence[int]] = None, qk_l2norm: bool = True,
                        status: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None, workspace="auto"):
    """Chunked KDA forward with the gate (g, beta from f, A_log, dt_bias, b) fused in;
    workspace as kda_chunk_fwd."""
    lib = load_library()
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    out, final_state = _chunk_outputs(q, v, cu_seqlens, out, out_dtype, output_final_state,
                                      final_state)
    keep, host = _host_offsets(cu_seqlens_host)
    ws, ws_bytes, ws_keep = _workspace(workspace, mode, N, T, H, K, V, q.device)
    st = lib.kda_chunk_fwd_gated(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(f, "f"), _dtype_code(f), _dev_ptr(A_log, "A_log"), _dev_ptr(dt_bias, "dt_bias"),
        _dev_ptr(b, "b"), _dtype_code(b), _dev_ptr(cu_seqlens, "cu_seqlens"), host,
        N, T, H, K, V, float(scale), 1 if qk_l2norm else 0, MODES[mode],
        _dev_ptr(out, "out"), _dtype_code(out), _dev_ptr(initial_state, "initial_state"),
        _dev_ptr(final_state, "final_state"), ws, ws_bytes, _dev_ptr(status, "status"),
        _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd_gated")
    return out, final_state


def kda_chunk_fwd_gated_norm(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, f: torch.Tensor,
                             A_log: torch.Tensor, dt_bias: torch.Tensor, b: torch.Tensor,
                             cu_seqlens: torch.Tensor, z: torch.Tensor, weight: torch.Tensor,
                             scale: Optional[float] = None, eps: float = 1e-6,
                             mode: str = "bf16_tc", out: Optional[torch.Tensor] = None,
                             out_dtype: Optional[torch.dtype] = None,
                             output_final_state: bool = True,
                             final_state: Optional[torch.Tensor] = None,
                             initial_state: Optional[torch.Tensor] = None,
                             cu_seqlens_host: Optional[Sequence[int]] = None,
                             qk_l2norm: bool = True, status: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None, workspace="auto"):
    """kda_chunk_fwd_gated with the output gate and gated RMSNorm applied to its
    output (z [T,H,V] gate pre-activation, weight [V]); returns (y, final_state)."""
    lib = load_library()
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    out, final_state = _chunk_outputs(q, v, cu_seqlens, out, out_dtype, output_final_state,
                                      final_state)
    keep, host = _host_offsets(cu_seqlens_host)
    ws, ws_bytes, ws_keep = _workspace(workspace, mode, N, T, H, K, V, q.device)
    st = lib.kda_chunk_fwd_gated_norm(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(f, "f"), _dtype_code(f), _dev_ptr(A_log, "A_log"), _dev_ptr(dt_bias, "dt_bias"),
        _dev_ptr(b, "b"), _dtype_code(b), _dev_ptr(cu_seqlens, "cu_seqlens"), host,
        N, T, H, K, V, float(scale), 1 if qk_l2norm else 0, MODES[mode],
        _dev_ptr(z, "z"), _dtype_code(z), _dev_ptr(weight, "weight"), float(eps),
        _dev_ptr(out, "out"), _dtype_code(out), _dev_ptr(initial_state, "initial_state"),
        _dev_ptr(final_state, "final_state"), ws, ws_bytes, _dev_ptr(status, "status"),
        _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd_gated_norm")
    return out, final_state


def kda_chunk_fwd_static(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                         beta: torch.Tensor, cu_seqlens: torch.Tensor, out: torch.Tensor,
                         scale: Optional[float] = None,
                         final_state: Optional[torch.Tensor] = None,
                         initial_state: Optional[torch.Tensor] = None,
                         cu_seqlens_host: Optional[Sequence[int]] = None, qk_l2norm: bool = True,
                         status: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """kda_chunk_fwd (bf16_tc, two-phase) on the library's static scratch: allocates
    nothing, so `out` (and `final_state`, if wanted) are the caller's.  Problems
    beyond the 64 MiB scratch raise KDAError(KDA_ERR_TOO_LARGE)."""
    lib = load_library()
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    keep, host = _host_offsets(cu_seqlens_host)
    st = lib.kda_chunk_fwd_static(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(g, "g"), _dev_ptr(beta, "beta"), _dev_ptr(cu_seqlens, "cu_seqlens"), host,
        N, T, H, K, V, float(scale), 1 if qk_l2norm else 0,
        _dev_ptr(out, "out"), _dtype_code(out), _dev_ptr(initial_state, "initial_state"),
        _dev_ptr(final_state, "final_state"), _dev_ptr(status, "status"),
        _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd_static")


def kda_recurrent_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                       beta: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                       qk_l2norm: bool = True, stream: Optional[torch.cuda.Stream] = None):
    """One decode token per sequence: q, k [N,H,K], v [N,H,V], g [N,H,K], beta [N,H];
    state [N,H,K,V] FP32 is updated in place.  Returns out [N,H,V]."""
    lib = load_library()
    N, H, K = q.shape
    V = v.shape[2]
    if scale is None:
        scale = K ** -0.5
    if out is None:
        out = torch.empty((N, H, V), dtype=out_dtype or v.dtype, device=q.device)
    st = lib.kda_recurrent_step(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(g, "g"), _dev_ptr(beta, "beta"), N, H, K, V, float(scale),
        1 if qk_l2norm else 0, _dev_ptr(state, "state"), _dev_ptr(out, "out"),
        _dtype_code(out), _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_recurrent_step")
    return out


def kda_gated_rmsnorm(o: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = o / sqrt(mean(o^2) + eps) * weight * sigmoid(z) over the last dim (V = 128);
    o and z of shape [..., V], weight [V] FP32.  Returns y (out if given)."""
    lib = load_library()
    V = o.shape[-1]
    rows = o.numel() // V if V else 0
    if out is None:
        out = torch.empty(o.shape, dtype=out_dtype or o.dtype, device=o.device)
    st = lib.kda_gated_rmsnorm(_dev_ptr(o, "o"), _dtype_code(o), _dev_ptr(z, "z"), _dtype_code(z),
                               _dev_ptr(weight, "weight"), rows, V, float(eps),
                               _dev_ptr(out, "out"), _dtype_code(out),
                               _stream_handle(stream, o.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_gated_rmsnorm")
    return out


def chunk_bwd_workspace_size(N: int, T: int, H: int, K: int = 128, V: int = 128) -> int:
    """Bytes of workspace kda_chunk_bwd needs."""
    out = ctypes.c_int64(0)
    st = load_library().kda_chunk_bwd_workspace_size(N, T, H, K, V, ctypes.byref(out))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_bwd_workspace_size")
    return out.value


def kda_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, cu_seqlens: torch.Tensor, dout: torch.Tensor,
                  scale: Optional[float] = None, dfinal_state: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None, want_dinitial: bool = True,
                  cu_seqlens_host: Optional[Sequence[int]] = None, qk_l2norm: bool = True,
                  status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, workspace=None):
    """Backward of kda_chunk_fwd.  Returns FP32 (dq, dk, dv, dg, dbeta, dinitial_state
    or None).  workspace: None (a fresh buffer) or a CUDA tensor of at least
    chunk_bwd_workspace_size(...) bytes."""
    lib = load_library()
    T, H, K = q.shape
    V = v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk, dg = (torch.empty((T, H, K), **f32) for _ in range(3))
    dv = torch.empty((T, H, V), **f32)
    dbeta = torch.empty((T, H), **f32)
    dinit = torch.empty((N, H, K, V), **f32) if want_dinitial else None
    if workspace is None:
        workspace = torch.empty(chunk_bwd_workspace_size(N, T, H, K, V), dtype=torch.uint8,
                                device=dev)
    keep, host = _host_offsets(cu_seqlens_host)
    st = lib.kda_chunk_bwd(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dtype_code(q),
        _dev_ptr(g, "g"), _dev_ptr(beta, "beta"), _dev_ptr(cu_seqlens, "cu_seqlens"), host,
        N, T, H, K, V, float(scale), 1 if qk_l2norm else 0,
        _dev_ptr(dout, "dout"), _dtype_code(dout), _dev_ptr(initial_state, "initial_state"),
        _dev_ptr(dfinal_state, "dfinal_state"), _dev_ptr(dq, "dq"), _dev_ptr(dk, "dk"),
        _dev_ptr(dv, "dv"), _dev_ptr(dg, "dg"), _dev_ptr(dbeta, "dbeta"),
        _dev_ptr(dinit, "dinitial_state"), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _dev_ptr(status, "status"),
        _stream_handle(stream, dev))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_bwd")
    return dq, dk, dv, dg, dbeta, dinit


# ---------------------------------------------------------------- paged attention
# These calls are short on the GPU, so their tensors are looked at in C++ (marshal.cpp):
# a call costs the host the launch and little else.  All tensors of a call are on one device.
# stream: None (the current one) or the call's; what the call allocates belongs to it.
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
_fast = None


def _load_marshal():
    """The _marshal module of this interpreter and PyTorch, bound to the loaded library's
    functions."""
    global _fast
    lib = load_library()
    if _fast is None:
        path, name = _build.marshal_path(), __package__ + "._marshal"
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with {_build.__name__}.build()")
        if name not in sys.modules:
            spec = importlib.util.spec_from_file_location(name, path)
            sys.modules[name] = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(sys.modules[name])
        _marshal = sys.modules[name]
        _marshal.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                       for name in EXPORTS})
        _fast = _marshal
    return _fast


def kda_page_plan(cached_lens: torch.Tensor, cu_seqlens: torch.Tensor, block_table: torch.Tensor,
                  free_pages: torch.Tensor, page_size: int, num_tokens: int,
                  free_start: Optional[torch.Tensor] = None,
                  seq_lens: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                  free_end: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None):
    """Pages, slots and positions of the new tokens of N requests, from lengths on the
    device: cached_lens [N], cu_seqlens [N+1] packing num_tokens new tokens, block_table
    [N, max_pages] (new entries written in place), free_pages (taken in order from
    free_start).  Returns (seq_lens [N], positions [T], slots [T] int64, free_end [1])."""
    r = (_fast or _load_marshal()).page_plan(cached_lens, cu_seqlens, block_table, free_pages,
                                             page_size, num_tokens, free_start, seq_lens,
                                             positions, slots, free_end, status, stream)
    if r.__class__ is int:
        raise KDAError(r, "kda_page_plan")
    return r


def rope_inv_freq(rot_dim: int, theta: float = 10000.0, scaling: str = "plain",
                  factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0,
                  beta_slow: float = 1.0, device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq [rot_dim / 2] FP32 on `device`, rope_scale) of a rotation, scaled for long
    contexts by "linear", "ntk" or "yarn" (the last reads original_len and the betas)."""
    f = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float32)
    m = ctypes.c_float(1.0)
    st = load_library().kda_rope_inv_freq(rot_dim, theta, ROPE_SCALINGS[scaling], factor,
                                          original_len, beta_fast, beta_slow, f.data_ptr(),
                                          ctypes.addressof(m))
    if st != KDA_OK:
        raise KDAError(st, "kda_rope_inv_freq")
    return f.to(device) if device is not None else f, m.value


def kda_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                     inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     qk_norm: bool = True, interleaved: bool = False, rope_scale: float = 1.0,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """Per-head RMS norm of q [T,Hq,D] and k [T,Hk,D] (weights [D] or None) and rotation of
    the first 2 * len(inv_freq) channels by position, in one pass (None: no rotation).  q and
    k may be slices of one projection.  Returns (q_out, k_out)."""
    r = (_fast or _load_marshal()).norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps,
                                             qk_norm, interleaved, rope_scale, q_out, k_out,
                                             out_dtype, stream)
    if r.__class__ is int:
        raise KDAError(r, "kda_qk_norm_rope")
    return r


def kda_qk_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            positions: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, inv_freq: Optional[torch.Tensor],
                            q_weight: Optional[torch.Tensor] = None,
                            k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                            qk_norm: bool = True, interleaved: bool = False,
                            rope_scale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """kda_qk_norm_rope with the keys, and the values v [T,Hk,D], written to the slots
    (int64 [T], negative: skipped) of k_cache and v_cache [num_pages,Hk,page_size,D] in
    place.  Returns q_out in the cache's dtype."""
    r = (_fast or _load_marshal()).append(q, k, v, slots, k_cache, v_cache, positions, inv_freq,
                                          q_weight, k_weight, eps, qk_norm, interleaved,
                                          rope_scale, q_out, status, stream)
    if r.__class__ is int:
        raise KDAError(r, "kda_qk_norm_rope_append")
    return r


def qk_norm_rope_bwd_workspace_size(T: int, Hq: int, Hk: int, D: int = 128) -> int:
    """Bytes of workspace kda_qk_norm_rope_bwd needs."""
    out = ctypes.c_int64(0)
    st = load_library().kda_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D, ctypes.byref(out))
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_norm_rope_bwd_workspace_size")
    return out.value


def kda_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, dq_out: torch.Tensor,
                         dk_out: torch.Tensor, positions: torch.Tensor,
                         inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                         k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                         qk_norm: bool = True, interleaved: bool = False, rope_scale: float = 1.0,
                         q_grad: Optional[torch.Tensor] = None,
                         k_grad: Optional[torch.Tensor] = None,
                         grad_dtype: Optional[torch.dtype] = None,
                         stream: Optional[torch.cuda.Stream] = None, workspace=None):
    """Backward of kda_qk_norm_rope.  Returns (q_grad, k_grad, q_weight_grad, k_weight_grad):
    the first two FP32 unless grad_dtype or given tensors say otherwise, the weights' FP32
    (None where the weight is None or qk_norm is off).  workspace: None (one kept per
    stream) or a CUDA tensor of at least qk_norm_rope_bwd_workspace_size(...) bytes."""
    r = (_fast or _load_marshal()).norm_rope_bwd(q, k, dq_out, dk_out, positions, inv_freq,
                                                 q_weight, k_weight, eps, qk_norm, interleaved,
                                                 rope_scale, q_grad, k_grad, grad_dtype, workspace,
                                                 stream)
    if r.__class__ is int:
        raise KDAError(r, "kda_qk_norm_rope_bwd")
    return r


def paged_decode_workspace_size(N: int, Hq: int, Hk: int, D: int = 128) -> int:
    """Bytes of workspace kda_paged_decode needs, whatever the lengths."""
    out = ctypes.c_int64(0)
    st = load_library().kda_paged_decode_workspace_size(N, Hq, Hk, D, ctypes.byref(out))
    if st != KDA_OK:
        raise KDAError(st, "kda_paged_decode_workspace_size")
    return out.value


def kda_paged_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_table: torch.Tensor, seq_lens: torch.Tensor,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None, lse: Optional[torch.Tensor] = None,
                     want_lse: bool = False, status: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None, workspace=None):
    """Attention of one new token per request, q [N,Hq,D], over the pages of k_cache and
    v_cache [num_pages,Hk,page_size,D] named by block_table [N,max_pages], seq_lens [N] tokens
    each.  Returns (out [N,Hq,D], lse [N,Hq] or None).  workspace: None (one kept per stream)
    or a CUDA tensor of at least paged_decode_workspace_size(...) bytes."""
    r = (_fast or _load_marshal()).paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale,
                                                out, out_dtype, lse, want_lse, status, workspace,
                                                stream)
    if r.__class__ is int:
        raise KDAError(r, "kda_paged_decode")
    return r
