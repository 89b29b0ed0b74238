"""ctypes binding of libkda_gb300.so (include/kda.h): argument marshalling only.

Every computation runs in the library's CUDA kernels; PyTorch provides the
device memory and the stream.  There is no fallback: if the library is
missing, or a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from functools import lru_cache
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


# The current stream's handle without building a Stream object (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream: Optional[torch.cuda.Stream], device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


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
# These calls are short on the GPU, so their marshalling is kept to one look at each
# tensor: a launch every few microseconds is bound by this file, not by the kernels.
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
_CODE = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_I32, _I64, _FP32 = torch.int32, torch.int64, torch.float32


def _refuse(t, name: str, dtype: torch.dtype, n: int = -1):
    """Raises for the first thing that is wrong with `t`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if n >= 0 and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, not {t.numel()}")
    _dev_ptr(t, name)
    raise ValueError(f"{name}: unsupported tensor")


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype) -> int:
    """Device pointer of a contiguous tensor of `dtype`."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, dtype)
    return t.data_ptr()


def _ptr_n(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, n: int) -> Optional[int]:
    """_ptr of `n` elements; None passes."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, dtype, n)
    return t.data_ptr()


def _rows_ptr(t: torch.Tensor, name: str, dtype: torch.dtype, T: int, H: int, D: int):
    """(pointer, token stride) of [T, H, D] whose heads are dense within a token."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != (T, H, D):
        raise ValueError(f"{name} must have shape {(T, H, D)}, not {tuple(t.shape)}")
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    st, sh, sc = t.stride()
    if (sc != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be dense (strides {t.stride()})")
    return t.data_ptr(), st if T > 1 else H * D


def _dense_ptr(t: torch.Tensor, name: str, shape, dtype: torch.dtype) -> int:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return _ptr(t, name, dtype)


_scratch = {}


def _own_scratch(nbytes: int, dev, stream: Optional[torch.cuda.Stream], handle: int) -> int:
    """Pointer to the workspace of a call that was given none: one buffer per stream, kept
    and grown, since calls on one stream are ordered.  (An allocation between two launches
    costs as much host time as a launch.)  A captured call gets a buffer of its graph's own."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev).data_ptr()
    key = (dev.index, handle)
    buf = _scratch.get(key)
    if buf is None or buf.nbytes < nbytes:
        if stream is None:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _scratch[key] = buf
    return buf.data_ptr()


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
    lib = _lib or load_library()
    N, T = cached_lens.numel(), int(num_tokens)
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError(f"block_table must have shape [{N}, max_pages]")
    dev = cached_lens.device
    if seq_lens is None:
        seq_lens = torch.empty(N, dtype=_I32, device=dev)
    if positions is None:
        positions = torch.empty(T, dtype=_I32, device=dev)
    if slots is None:
        slots = torch.empty(T, dtype=_I64, device=dev)
    if free_end is None:
        free_end = torch.empty(1, dtype=_I32, device=dev)
    st = lib.kda_page_plan(
        _ptr(cached_lens, "cached_lens", _I32), _ptr_n(cu_seqlens, "cu_seqlens", _I32, N + 1), N, T,
        int(page_size), _ptr(block_table, "block_table", _I32), block_table.shape[1],
        _ptr(free_pages, "free_pages", _I32), free_pages.numel(),
        _ptr_n(free_start, "free_start", _I32, 1), _ptr_n(seq_lens, "seq_lens", _I32, N),
        _ptr_n(positions, "positions", _I32, T), _ptr_n(slots, "slots", _I64, T),
        _ptr_n(free_end, "free_end", _I32, 1), _dev_ptr(status, "status"),
        _stream_handle(stream, dev))
    if st != KDA_OK:
        raise KDAError(st, "kda_page_plan")
    return seq_lens, positions, slots, free_end


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


def _code(dtype: torch.dtype) -> int:
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


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
    lib = _lib or load_library()
    T, Hq, D = q.shape
    Hk, dev, dt = k.shape[1], q.device, q.dtype
    if k.dtype is not dt:
        raise TypeError(f"k must be {dt}, not {k.dtype}")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=out_dtype or dt, device=dev)
    odt = q_out.dtype
    if k_out is None:
        k_out = torch.empty((T, Hk, D), dtype=odt, device=dev)
    pairs = 0 if inv_freq is None else inv_freq.numel()
    qp, qs = _rows_ptr(q, "q", dt, T, Hq, D)
    kp, ks = _rows_ptr(k, "k", dt, T, Hk, D)
    st = lib.kda_qk_norm_rope(
        qp, qs, kp, ks, _code(dt), _ptr_n(positions, "positions", _I32, T),
        _ptr_n(inv_freq, "inv_freq", _FP32, pairs), 2 * pairs, 1 if interleaved else 0, rope_scale,
        _ptr_n(q_weight, "q_weight", _FP32, D), _ptr_n(k_weight, "k_weight", _FP32, D), eps,
        1 if qk_norm else 0, T, Hq, Hk, D, _dense_ptr(q_out, "q_out", (T, Hq, D), odt),
        _dense_ptr(k_out, "k_out", (T, Hk, D), odt), _code(odt), _stream_handle(stream, dev))
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_norm_rope")
    return q_out, k_out


def _cache_shape(k_cache, v_cache, Hk, D):
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] != Hk or shape[3] != D:
        raise ValueError(f"k_cache must have shape [num_pages, {Hk}, page_size, {D}], not "
                         f"{tuple(shape)}")
    if v_cache.shape != shape or v_cache.dtype is not k_cache.dtype:
        raise ValueError("v_cache must have the shape and dtype of k_cache")
    return shape


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
    lib = _lib or load_library()
    T, Hq, D = q.shape
    Hk, dev, dt, cdt = k.shape[1], q.device, q.dtype, k_cache.dtype
    if k.dtype is not dt or v.dtype is not dt:
        raise TypeError(f"k must be {dt} and v as well, not {k.dtype} and {v.dtype}")
    num_pages, _, page_size, _ = _cache_shape(k_cache, v_cache, Hk, D)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=cdt, device=dev)
    pairs = 0 if inv_freq is None else inv_freq.numel()
    qp, qs = _rows_ptr(q, "q", dt, T, Hq, D)
    kp, ks = _rows_ptr(k, "k", dt, T, Hk, D)
    vp, vs = _rows_ptr(v, "v", dt, T, Hk, D)
    st = lib.kda_qk_norm_rope_append(
        qp, qs, kp, ks, vp, vs, _code(dt), _ptr_n(positions, "positions", _I32, T),
        _ptr_n(slots, "slots", _I64, T), _ptr_n(inv_freq, "inv_freq", _FP32, pairs), 2 * pairs,
        1 if interleaved else 0, rope_scale, _ptr_n(q_weight, "q_weight", _FP32, D),
        _ptr_n(k_weight, "k_weight", _FP32, D), eps, 1 if qk_norm else 0, T, Hq, Hk, D,
        _dense_ptr(q_out, "q_out", (T, Hq, D), cdt), _ptr(k_cache, "k_cache", cdt),
        _ptr(v_cache, "v_cache", cdt), _code(cdt), num_pages, page_size,
        _dev_ptr(status, "status"), _stream_handle(stream, dev))
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_norm_rope_append")
    return q_out


@lru_cache(maxsize=256)
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
    lib = _lib or load_library()
    T, Hq, D = q.shape
    Hk, dev, dt, ydt = k.shape[1], q.device, q.dtype, dq_out.dtype
    if k.dtype is not dt:
        raise TypeError(f"k must be {dt}, not {k.dtype}")
    if q_grad is None:
        q_grad = torch.empty((T, Hq, D), dtype=grad_dtype or _FP32, device=dev)
    gdt = q_grad.dtype
    if k_grad is None:
        k_grad = torch.empty((T, Hk, D), dtype=gdt, device=dev)
    qp, qs = _rows_ptr(q, "q", dt, T, Hq, D)
    kp, ks = _rows_ptr(k, "k", dt, T, Hk, D)
    wq = wk = None
    handle = _stream_handle(stream, dev)
    ws, ws_bytes = None, 0
    if qk_norm and (q_weight is not None or k_weight is not None):
        if q_weight is not None:
            wq = torch.empty(D, dtype=_FP32, device=dev)
        if k_weight is not None:
            wk = torch.empty(D, dtype=_FP32, device=dev)
        if workspace is None:
            ws_bytes = qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D)
            ws = _own_scratch(ws_bytes, dev, stream, handle)
    if workspace is not None:
        ws, ws_bytes = _dev_ptr(workspace, "workspace"), workspace.nbytes
    pairs = 0 if inv_freq is None else inv_freq.numel()
    st = lib.kda_qk_norm_rope_bwd(
        qp, qs, kp, ks, _code(dt), _dense_ptr(dq_out, "dq_out", (T, Hq, D), ydt),
        _dense_ptr(dk_out, "dk_out", (T, Hk, D), ydt), _code(ydt),
        _ptr_n(positions, "positions", _I32, T), _ptr_n(inv_freq, "inv_freq", _FP32, pairs),
        2 * pairs, 1 if interleaved else 0, rope_scale, _ptr_n(q_weight, "q_weight", _FP32, D),
        _ptr_n(k_weight, "k_weight", _FP32, D), eps, 1 if qk_norm else 0, T, Hq, Hk, D,
        _dense_ptr(q_grad, "q_grad", (T, Hq, D), gdt),
        _dense_ptr(k_grad, "k_grad", (T, Hk, D), gdt), _code(gdt),
        None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(), ws, ws_bytes,
        handle)
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_norm_rope_bwd")
    return q_grad, k_grad, wq, wk


@lru_cache(maxsize=256)
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
    each.  Returns (out [N,Hq,D], lse [N,Hq] or None).  workspace: None (one kept per stream) or a
    CUDA tensor of at least paged_decode_workspace_size(...) bytes."""
    lib = _lib or load_library()
    N, Hq, D = q.shape
    dev, dt = q.device, k_cache.dtype
    num_pages, Hk, page_size, _ = _cache_shape(k_cache, v_cache, k_cache.shape[1], D)
    rows, max_pages = block_table.shape
    if rows != N:
        raise ValueError(f"block_table must have shape [{N}, max_pages]")
    if out is None:
        out = torch.empty((N, Hq, D), dtype=out_dtype or q.dtype, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((N, Hq), dtype=_FP32, device=dev)
    qp = _ptr(q, "q", dt)
    handle = _stream_handle(stream, dev)
    if workspace is None:
        ws_bytes = paged_decode_workspace_size(N, Hq, Hk, D)
        ws = _own_scratch(ws_bytes, dev, stream, handle)
    else:
        ws, ws_bytes = _dev_ptr(workspace, "workspace"), workspace.nbytes
    odt = out.dtype
    st = lib.kda_paged_decode(
        qp, _ptr(k_cache, "k_cache", dt), _ptr(v_cache, "v_cache", dt), _code(dt),
        _ptr(block_table, "block_table", _I32), _ptr_n(seq_lens, "seq_lens", _I32, N), N, Hq, Hk, D,
        num_pages, page_size, max_pages, D ** -0.5 if scale is None else scale,
        _dense_ptr(out, "out", (N, Hq, D), odt), _code(odt), _ptr_n(lse, "lse", _FP32, N * Hq),
        ws, ws_bytes, _dev_ptr(status, "status"), handle)
    if st != KDA_OK:
        raise KDAError(st, "kda_paged_decode")
    return out, lse
