"""ctypes binding of libfp8bs.so (argument marshalling only).

Every function here checks torch dtypes, shapes, contiguity and devices, then
passes raw device pointers and the current HIP stream to the C ABI declared in
include/fp8bs.h, include/fp8bs_g128.h and include/fp8bs_layer.h.  No arithmetic of the method happens in Python; if
the library is missing the call raises ``Fp8bsError`` - there is no fallback path.
"""

from __future__ import annotations

import array
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libfp8bs.so"
_lock = threading.Lock()
_lib = None

BLOCK = 32
E4M3_DTYPES = (torch.uint8, torch.float8_e4m3fn)
STATUS = {0: "FP8BS_OK", 1: "FP8BS_EINVAL", 2: "FP8BS_ESHAPE", 3: "FP8BS_EALIGN", 4: "FP8BS_EHIP",
          5: "FP8BS_ENOSYS"}


class Fp8bsError(RuntimeError):
    """Raised for a non-OK status from the library or a missing library."""


def library_path() -> str:
    return os.environ.get("FP8BS_LIBRARY", os.path.join(_PKG, _LIB_NAME))


def load_library() -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise Fp8bsError(f"{path} not found: build it first (python -m fp8_block_scaled_03_amd.build)")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.fp8bs_quantize.argtypes = [vp, i64, i64, vp, vp, vp]
        lib.fp8bs_quantize.restype = ctypes.c_int
        lib.fp8bs_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm.restype = ctypes.c_int
        lib.fp8bs_grouped_gemm.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, vp]
        lib.fp8bs_grouped_gemm.restype = ctypes.c_int
        lib.fp8bs_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_nt.restype = ctypes.c_int
        lib.fp8bs_quantize_tg.argtypes = [vp, i64, i64, vp, vp, vp]
        lib.fp8bs_quantize_tg.restype = ctypes.c_int
        lib.fp8bs_gemm_tg.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_tg.restype = ctypes.c_int
        lib.fp8bs_gemm_tg_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_tg_nt.restype = ctypes.c_int
        lib.fp8bs_grouped_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, vp]
        lib.fp8bs_grouped_gemm_nt.restype = ctypes.c_int
        lib.fp8bs_rmsnorm_quantize_tg.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, vp, vp, vp, vp]
        lib.fp8bs_rmsnorm_quantize_tg.restype = ctypes.c_int
        lib.fp8bs_quantize_e8m0.argtypes = [vp, i64, i64, vp, vp, vp]
        lib.fp8bs_quantize_e8m0.restype = ctypes.c_int
        lib.fp8bs_gemm_e8m0_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_e8m0_nt.restype = ctypes.c_int
        lib.fp8bs_quantize_tg128.argtypes = [vp, i64, i64, vp, vp, vp]
        lib.fp8bs_quantize_tg128.restype = ctypes.c_int
        lib.fp8bs_quantize_b128.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
        lib.fp8bs_quantize_b128.restype = ctypes.c_int
        lib.fp8bs_gemm_tg128_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_tg128_nt.restype = ctypes.c_int
        lib.fp8bs_grouped_gemm_tg128_nt.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, vp]
        lib.fp8bs_grouped_gemm_tg128_nt.restype = ctypes.c_int
        lib.fp8bs_grouped_wgrad.argtypes = [vp, vp, vp, i32, vp, i32, i64, i64, i64, vp]
        lib.fp8bs_grouped_wgrad.restype = ctypes.c_int
        lib.fp8bs_swiglu_quantize_tg128.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        lib.fp8bs_swiglu_quantize_tg128.restype = ctypes.c_int
        lib.fp8bs_swiglu_backward_quantize_tg128.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, vp]
        lib.fp8bs_swiglu_backward_quantize_tg128.restype = ctypes.c_int
        f32, f64 = ctypes.c_float, ctypes.c_double
        lib.fp8bs_layernorm_quantize_tg128.argtypes = [vp, vp, vp, vp, f32, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        lib.fp8bs_layernorm_quantize_tg128.restype = ctypes.c_int
        lib.fp8bs_layernorm.argtypes = [vp, vp, vp, vp, f32, i64, i64, vp, vp, vp, vp, vp]
        lib.fp8bs_layernorm.restype = ctypes.c_int
        lib.fp8bs_layernorm_backward_workspace.argtypes = [i64, i64]
        lib.fp8bs_layernorm_backward_workspace.restype = i64
        lib.fp8bs_layernorm_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, i32, vp, i64, vp]
        lib.fp8bs_layernorm_backward.restype = ctypes.c_int
        lib.fp8bs_gemm_tg128_nt_epilogue.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_gemm_tg128_nt_epilogue.restype = ctypes.c_int
        lib.fp8bs_epilogue_backward_workspace.argtypes = [i64, i64]
        lib.fp8bs_epilogue_backward_workspace.restype = i64
        lib.fp8bs_epilogue_backward_quantize_tg128.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, i32, vp, i64, vp]
        lib.fp8bs_epilogue_backward_quantize_tg128.restype = ctypes.c_int
        lib.fp8bs_moe_decode_b128_workspace.argtypes = [i64, i64, i64, i64, i64]
        lib.fp8bs_moe_decode_b128_workspace.restype = i64
        lib.fp8bs_moe_decode_b128.argtypes = [vp] * 9 + [i64] * 5 + [vp, i64, vp]
        lib.fp8bs_moe_decode_b128.restype = ctypes.c_int
        lib.fp8bs_grad_norm_workspace.argtypes = [i32]
        lib.fp8bs_grad_norm_workspace.restype = i64
        lib.fp8bs_grad_norm.argtypes = [vp, vp, vp, i32, vp, vp, i64, vp]
        lib.fp8bs_grad_norm.restype = ctypes.c_int
        lib.fp8bs_clip_grads.argtypes = [vp, vp, vp, vp, i32, vp, f64, f64, vp]
        lib.fp8bs_clip_grads.restype = ctypes.c_int
        lib.fp8bs_clip_grad_norm.argtypes = [vp, vp, vp, vp, i32, f64, f64, vp, vp, i64, vp]
        lib.fp8bs_clip_grad_norm.restype = ctypes.c_int
        lib.fp8bs_status_str.argtypes = [ctypes.c_int]
        lib.fp8bs_status_str.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != 0:
        msg = load_library().fp8bs_status_str(status).decode()
        raise Fp8bsError(msg)


def _stream_ptr(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtypes, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise TypeError(f"{name}: dtype {t.dtype} not accepted ({dtypes})")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")


def _same_device(*ts: torch.Tensor) -> None:
    dev = ts[0].device
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError("all tensors must be on the same device")


# ---- raw pointer entry points (used by tests of the ABI itself) ------------------------
def quantize_raw(x_ptr, rows, cols, q_ptr, s_ptr, stream=None) -> int:
    return load_library().fp8bs_quantize(x_ptr, rows, cols, q_ptr, s_ptr, stream)


def gemm_raw(a_ptr, sa_ptr, b_ptr, sb_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm(a_ptr, sa_ptr, b_ptr, sb_ptr, c_ptr, M, N, K, stream)


def quantize_tg_raw(x_ptr, rows, cols, q_ptr, s_ptr, stream=None) -> int:
    return load_library().fp8bs_quantize_tg(x_ptr, rows, cols, q_ptr, s_ptr, stream)


def gemm_tg_raw(a_ptr, sa_ptr, b_ptr, sb_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm_tg(a_ptr, sa_ptr, b_ptr, sb_ptr, c_ptr, M, N, K, stream)


def gemm_tg_nt_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm_tg_nt(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream)


def rmsnorm_quantize_tg_raw(x_ptr, res_ptr, gamma_ptr, eps, rows, d, q_ptr, s_ptr, y_ptr, stream=None) -> int:
    return load_library().fp8bs_rmsnorm_quantize_tg(x_ptr, res_ptr, gamma_ptr, eps, rows, d, q_ptr, s_ptr, y_ptr,
                                                    stream)


def quantize_e8m0_raw(x_ptr, rows, cols, q_ptr, e_ptr, stream=None) -> int:
    return load_library().fp8bs_quantize_e8m0(x_ptr, rows, cols, q_ptr, e_ptr, stream)


def gemm_e8m0_nt_raw(a_ptr, ea_ptr, bt_ptr, ebt_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm_e8m0_nt(a_ptr, ea_ptr, bt_ptr, ebt_ptr, c_ptr, M, N, K, stream)


def gemm_nt_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm_nt(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream)


def grouped_gemm_nt_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, off_ptr, G, c_ptr, M_total, N, K, stream=None) -> int:
    return load_library().fp8bs_grouped_gemm_nt(a_ptr, sa_ptr, bt_ptr, sbt_ptr, off_ptr, G, c_ptr, M_total, N, K,
                                                stream)


def grouped_gemm_raw(a_ptr, sa_ptr, b_ptr, sb_ptr, off_ptr, G, c_ptr, M_total, N, K, stream=None) -> int:
    return load_library().fp8bs_grouped_gemm(a_ptr, sa_ptr, b_ptr, sb_ptr, off_ptr, G, c_ptr, M_total, N, K, stream)


def quantize_tg128_raw(x_ptr, rows, cols, q_ptr, s_ptr, stream=None) -> int:
    return load_library().fp8bs_quantize_tg128(x_ptr, rows, cols, q_ptr, s_ptr, stream)


def quantize_b128_raw(x_ptr, G, rows, cols, q_ptr, s_ptr, qt_ptr, st_ptr, stream=None) -> int:
    return load_library().fp8bs_quantize_b128(x_ptr, G, rows, cols, q_ptr, s_ptr, qt_ptr, st_ptr, stream)


def gemm_tg128_nt_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream=None) -> int:
    return load_library().fp8bs_gemm_tg128_nt(a_ptr, sa_ptr, bt_ptr, sbt_ptr, c_ptr, M, N, K, stream)


def grouped_gemm_tg128_nt_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, off_ptr, G, c_ptr, M_total, N, K, stream=None) -> int:
    return load_library().fp8bs_grouped_gemm_tg128_nt(a_ptr, sa_ptr, bt_ptr, sbt_ptr, off_ptr, G, c_ptr, M_total, N,
                                                      K, stream)


def grouped_wgrad_raw(dy_ptr, x_ptr, off_ptr, G, dw_ptr, accumulate, M_total, N, K, stream=None) -> int:
    return load_library().fp8bs_grouped_wgrad(dy_ptr, x_ptr, off_ptr, G, dw_ptr, accumulate, M_total, N, K, stream)


def swiglu_quantize_tg128_raw(gu_ptr, rows, d, q_ptr, s_ptr, y_ptr, stream=None) -> int:
    return load_library().fp8bs_swiglu_quantize_tg128(gu_ptr, rows, d, q_ptr, s_ptr, y_ptr, stream)


def swiglu_backward_quantize_tg128_raw(gu_ptr, dy_ptr, rows, d, dgu_ptr, q_ptr, s_ptr, y_ptr, stream=None) -> int:
    return load_library().fp8bs_swiglu_backward_quantize_tg128(gu_ptr, dy_ptr, rows, d, dgu_ptr, q_ptr, s_ptr, y_ptr,
                                                               stream)


def layernorm_quantize_tg128_raw(x_ptr, res_ptr, gamma_ptr, beta_ptr, eps, rows, d, h_ptr, q_ptr, s_ptr, y_ptr,
                                 mean_ptr, rstd_ptr, stream=None) -> int:
    return load_library().fp8bs_layernorm_quantize_tg128(x_ptr, res_ptr, gamma_ptr, beta_ptr, eps, rows, d, h_ptr,
                                                         q_ptr, s_ptr, y_ptr, mean_ptr, rstd_ptr, stream)


def layernorm_raw(x_ptr, res_ptr, gamma_ptr, beta_ptr, eps, rows, d, h_ptr, y_ptr, mean_ptr, rstd_ptr,
                  stream=None) -> int:
    return load_library().fp8bs_layernorm(x_ptr, res_ptr, gamma_ptr, beta_ptr, eps, rows, d, h_ptr, y_ptr, mean_ptr,
                                          rstd_ptr, stream)


def layernorm_backward_raw(dy_ptr, h_ptr, gamma_ptr, mean_ptr, rstd_ptr, dres_ptr, rows, d, dx_ptr, dgamma_ptr,
                           dbeta_ptr, accumulate, ws_ptr, ws_bytes, stream=None) -> int:
    return load_library().fp8bs_layernorm_backward(dy_ptr, h_ptr, gamma_ptr, mean_ptr, rstd_ptr, dres_ptr, rows, d,
                                                   dx_ptr, dgamma_ptr, dbeta_ptr, accumulate, ws_ptr, ws_bytes, stream)


def gemm_tg128_nt_epilogue_raw(a_ptr, sa_ptr, bt_ptr, sbt_ptr, bias_ptr, activation, res_ptr, c_ptr, pre_ptr, M, N, K,
                               stream=None) -> int:
    return load_library().fp8bs_gemm_tg128_nt_epilogue(a_ptr, sa_ptr, bt_ptr, sbt_ptr, bias_ptr, activation, res_ptr,
                                                       c_ptr, pre_ptr, M, N, K, stream)


def epilogue_backward_quantize_tg128_raw(dout_ptr, pre_ptr, activation, rows, n, dz_ptr, q_ptr, s_ptr, dbias_ptr,
                                         accumulate, ws_ptr, ws_bytes, stream=None) -> int:
    return load_library().fp8bs_epilogue_backward_quantize_tg128(dout_ptr, pre_ptr, activation, rows, n, dz_ptr, q_ptr,
                                                                 s_ptr, dbias_ptr, accumulate, ws_ptr, ws_bytes,
                                                                 stream)


def moe_decode_b128_raw(x_ptr, ids_ptr, weights_ptr, w1_ptr, s1_ptr, w2_ptr, s2_ptr, res_ptr, out_ptr, tokens, top,
                        experts, hidden, inner, ws_ptr, ws_bytes, stream=None) -> int:
    return load_library().fp8bs_moe_decode_b128(x_ptr, ids_ptr, weights_ptr, w1_ptr, s1_ptr, w2_ptr, s2_ptr, res_ptr,
                                                out_ptr, tokens, top, experts, hidden, inner, ws_ptr, ws_bytes, stream)


def grad_norm_raw(grads, counts, types, n, norm_ptr, ws_ptr, ws_bytes, stream=None) -> int:
    return load_library().fp8bs_grad_norm(grads, counts, types, n, norm_ptr, ws_ptr, ws_bytes, stream)


def clip_grads_raw(grads, outs, counts, types, n, norm_ptr, max_norm, eps, stream=None) -> int:
    return load_library().fp8bs_clip_grads(grads, outs, counts, types, n, norm_ptr, max_norm, eps, stream)


def clip_grad_norm_raw(grads, outs, counts, types, n, max_norm, eps, norm_ptr, ws_ptr, ws_bytes, stream=None) -> int:
    return load_library().fp8bs_clip_grad_norm(grads, outs, counts, types, n, max_norm, eps, norm_ptr, ws_ptr,
                                               ws_bytes, stream)


# ---- tensor entry points -----------------------------------------------------------------
def quantize(x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """bf16 [R, C] -> (E4M3 codes uint8 [R, C], fp32 scales [ceil(R/32), C/32])."""
    _need(x, "x", torch.bfloat16, 2)
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(((R + BLOCK - 1) // BLOCK, C // BLOCK), dtype=torch.float32, device=x.device)
    _need(q, "q", E4M3_DTYPES, 2)
    _need(scales, "scales", torch.float32, 2)
    _same_device(x, q, scales)
    if tuple(q.shape) != (R, C) or tuple(scales.shape) != ((R + BLOCK - 1) // BLOCK, C // BLOCK):
        raise ValueError("output shapes do not match the input")
    _check(quantize_raw(_ptr(x), R, C, _ptr(q), _ptr(scales), _stream_ptr(x)))
    return q, scales


def gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, out: torch.Tensor | None = None):
    """E4M3 a [M, K], sa [ceil(M/32), K/32], b [K, N], sb [K/32, N/32] -> bf16 [M, N]."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(b, "b", E4M3_DTYPES, 2)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 2)
    M, K = a.shape
    K2, N = b.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if tuple(sa.shape) != ((M + BLOCK - 1) // BLOCK, K // BLOCK) or tuple(sb.shape) != (K // BLOCK, N // BLOCK):
        raise ValueError("scale grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, sa, b, sb, out)
    _check(gemm_raw(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), M, N, K, _stream_ptr(a)))
    return out


def grouped_gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, offsets: torch.Tensor,
                 out: torch.Tensor | None = None):
    """a [M_total, K], sa [M_total/32, K/32], b [G, K, N], sb [G, K/32, N/32], offsets int32 [G+1] on device."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(b, "b", E4M3_DTYPES, 3)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 3)
    _need(offsets, "offsets", torch.int32, 1)
    M, K = a.shape
    G, K2, N = b.shape
    if K2 != K or offsets.shape[0] != G + 1:
        raise ValueError("shape mismatch between a, b and offsets")
    if tuple(sa.shape) != (M // BLOCK, K // BLOCK) or tuple(sb.shape) != (G, K // BLOCK, N // BLOCK):
        raise ValueError("scale grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, sa, b, sb, offsets, out)
    _check(grouped_gemm_raw(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(offsets), G, _ptr(out), M, N, K,
                            _stream_ptr(a)))
    return out


def gemm_nt(a: torch.Tensor, sa: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor,
            out: torch.Tensor | None = None):
    """K-major weight: E4M3 a [M, K], sa [ceil(M/32), K/32], bt [N, K], sbt [N/32, K/32] -> bf16 [M, N]."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 2)
    _need(sa, "sa", torch.float32, 2)
    _need(sbt, "sbt", torch.float32, 2)
    M, K = a.shape
    N, K2 = bt.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if tuple(sa.shape) != ((M + BLOCK - 1) // BLOCK, K // BLOCK) or tuple(sbt.shape) != (N // BLOCK, K // BLOCK):
        raise ValueError("scale grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, sa, bt, sbt, out)
    _check(gemm_nt_raw(_ptr(a), _ptr(sa), _ptr(bt), _ptr(sbt), _ptr(out), M, N, K, _stream_ptr(a)))
    return out


def grouped_gemm_nt(a: torch.Tensor, sa: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor, offsets: torch.Tensor,
                    out: torch.Tensor | None = None):
    """a [M_total, K], sa [M_total/32, K/32], bt [G, N, K], sbt [G, N/32, K/32], offsets int32 [G+1] on device."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 3)
    _need(sa, "sa", torch.float32, 2)
    _need(sbt, "sbt", torch.float32, 3)
    _need(offsets, "offsets", torch.int32, 1)
    M, K = a.shape
    G, N, K2 = bt.shape
    if K2 != K or offsets.shape[0] != G + 1:
        raise ValueError("shape mismatch between a, bt and offsets")
    if tuple(sa.shape) != (M // BLOCK, K // BLOCK) or tuple(sbt.shape) != (G, N // BLOCK, K // BLOCK):
        raise ValueError("scale grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, sa, bt, sbt, offsets, out)
    _check(grouped_gemm_nt_raw(_ptr(a), _ptr(sa), _ptr(bt), _ptr(sbt), _ptr(offsets), G, _ptr(out), M, N, K,
                               _stream_ptr(a)))
    return out


def quantize_tg(x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """bf16 [R, C] -> (E4M3 codes uint8 [R, C], fp32 per-token-group scales [R, C/32])."""
    _need(x, "x", torch.bfloat16, 2)
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((R, C // BLOCK), dtype=torch.float32, device=x.device)
    _need(q, "q", E4M3_DTYPES, 2)
    _need(scales, "scales", torch.float32, 2)
    _same_device(x, q, scales)
    if tuple(q.shape) != (R, C) or tuple(scales.shape) != (R, C // BLOCK):
        raise ValueError("output shapes do not match the input")
    _check(quantize_tg_raw(_ptr(x), R, C, _ptr(q), _ptr(scales), _stream_ptr(x)))
    return q, scales


def _gemm_tg_checked(raw, a, sa_rows, w, sw, out, k_major):
    _need(a, "a", E4M3_DTYPES, 2)
    _need(w, "b", E4M3_DTYPES, 2)
    _need(sa_rows, "sa_rows", torch.float32, 2)
    _need(sw, "sb", torch.float32, 2)
    M, K = a.shape
    if k_major:
        N, K2 = w.shape
        sw_shape = (N // BLOCK, K // BLOCK)
    else:
        K2, N = w.shape
        sw_shape = (K // BLOCK, N // BLOCK)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if tuple(sa_rows.shape) != (M, K // BLOCK) or tuple(sw.shape) != sw_shape:
        raise ValueError("scale grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, sa_rows, w, sw, out)
    _check(raw(_ptr(a), _ptr(sa_rows), _ptr(w), _ptr(sw), _ptr(out), M, N, K, _stream_ptr(a)))
    return out


def gemm_tg(a: torch.Tensor, sa_rows: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
            out: torch.Tensor | None = None):
    """E4M3 a [M, K] with per-token-group scales sa_rows [M, K/32], b [K, N], sb [K/32, N/32] -> bf16 [M, N]."""
    return _gemm_tg_checked(gemm_tg_raw, a, sa_rows, b, sb, out, False)


def gemm_tg_nt(a: torch.Tensor, sa_rows: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor,
               out: torch.Tensor | None = None):
    """As gemm_tg with the weight K-major: bt [N, K], sbt [N/32, K/32]."""
    return _gemm_tg_checked(gemm_tg_nt_raw, a, sa_rows, bt, sbt, out, True)


def rmsnorm_quantize_tg(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                        q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                        y: torch.Tensor | None = None, want_y: bool = False):
    """Residual add (in place on ``residual`` when given) + RMSNorm + per-token-group
    quantization of bf16 x [R, d] with weight gamma [d].

    Returns (q uint8 [R, d], scales fp32 [R, d/32]), plus the bf16 normalised rows
    [R, d] as a third element when ``want_y`` is true or ``y`` is given."""
    _need(x, "x", torch.bfloat16, 2)
    _need(gamma, "gamma", torch.bfloat16, 1)
    R, d = x.shape
    if gamma.shape[0] != d:
        raise ValueError(f"gamma has {gamma.shape[0]} entries, rows have {d}")
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, 2)
        if tuple(residual.shape) != (R, d):
            raise ValueError("residual has the wrong shape")
    if q is None:
        q = torch.empty((R, d), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((R, d // BLOCK), dtype=torch.float32, device=x.device)
    if y is None and want_y:
        y = torch.empty((R, d), dtype=torch.bfloat16, device=x.device)
    _need(q, "q", E4M3_DTYPES, 2)
    _need(scales, "scales", torch.float32, 2)
    if tuple(q.shape) != (R, d) or tuple(scales.shape) != (R, d // BLOCK):
        raise ValueError("output shapes do not match the input")
    if y is not None:
        _need(y, "y", torch.bfloat16, 2)
        if tuple(y.shape) != (R, d):
            raise ValueError("y has the wrong shape")
    _same_device(*[t for t in (x, gamma, residual, q, scales, y) if t is not None])
    _check(rmsnorm_quantize_tg_raw(_ptr(x), _ptr(residual), _ptr(gamma), float(eps), R, d, _ptr(q), _ptr(scales),
                                   _ptr(y), _stream_ptr(x)))
    return (q, scales) if y is None else (q, scales, y)


def quantize_e8m0(x: torch.Tensor, q: torch.Tensor | None = None, e8m0: torch.Tensor | None = None):
    """bf16 [R, C] -> (E4M3 codes uint8 [R, C], E8M0 exponent bytes uint8 [ceil(R/32), C/32])."""
    _need(x, "x", torch.bfloat16, 2)
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if e8m0 is None:
        e8m0 = torch.empty(((R + BLOCK - 1) // BLOCK, C // BLOCK), dtype=torch.uint8, device=x.device)
    _need(q, "q", E4M3_DTYPES, 2)
    _need(e8m0, "e8m0", torch.uint8, 2)
    _same_device(x, q, e8m0)
    if tuple(q.shape) != (R, C) or tuple(e8m0.shape) != ((R + BLOCK - 1) // BLOCK, C // BLOCK):
        raise ValueError("output shapes do not match the input")
    _check(quantize_e8m0_raw(_ptr(x), R, C, _ptr(q), _ptr(e8m0), _stream_ptr(x)))
    return q, e8m0


def gemm_e8m0_nt(a: torch.Tensor, ea: torch.Tensor, bt: torch.Tensor, ebt: torch.Tensor,
                 out: torch.Tensor | None = None):
    """E4M3 a [M, K] with E8M0 bytes ea [ceil(M/32), K/32], bt [N, K] with ebt [N/32, K/32] -> bf16 [M, N]."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 2)
    _need(ea, "ea", torch.uint8, 2)
    _need(ebt, "ebt", torch.uint8, 2)
    M, K = a.shape
    N, K2 = bt.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if tuple(ea.shape) != ((M + BLOCK - 1) // BLOCK, K // BLOCK) or tuple(ebt.shape) != (N // BLOCK, K // BLOCK):
        raise ValueError("exponent grid shapes do not match the operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _same_device(a, ea, bt, ebt, out)
    _check(gemm_e8m0_nt_raw(_ptr(a), _ptr(ea), _ptr(bt), _ptr(ebt), _ptr(out), M, N, K, _stream_ptr(a)))
    return out


# ---- scales of 128 values (include/fp8bs_g128.h) -------------------------------------------
GROUP = 128
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _blocks128(n: int) -> int:
    return (n + GROUP - 1) // GROUP


def _call_on(device: torch.device, name: str, *args) -> None:
    """One library call on the current stream of ``device``, whichever device is current."""
    fn = getattr(_lib or load_library(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():  # there is a tensor on it: CUDA is initialised
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        _check(status)


def _need_like(t: torch.Tensor, name: str, dtypes, shape: tuple, device: torch.device) -> torch.Tensor:
    """t, which must be contiguous and of the given type, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not accepted ({dtypes})")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError("all tensors must be on the same device")
    return t


def _need_size(t: torch.Tensor, name: str, dim: int, size: int, device: torch.device) -> None:
    """One size and the device of t, which _need has looked at."""
    if t.shape[dim] != size:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {size} in dimension {dim}")
    if t.device != device:
        raise ValueError("all tensors must be on the same device")


def _output(t: torch.Tensor | None, name: str, dtypes, shape: tuple, device: torch.device) -> torch.Tensor:
    """The caller's output, checked, or a new one of the first of ``dtypes``."""
    if t is None:
        return torch.empty(*shape, dtype=dtypes[0], device=device)  # 0.4 us less than with the tuple
    return _need_like(t, name, dtypes, shape, device)


def quantize_tg128(x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """bf16 [R, C] -> (E4M3 codes uint8 [R, C], fp32 scales [R, ceil(C/128)], one per row and 128 columns)."""
    _need(x, "x", _BF16, 2)
    R, C = x.shape
    dev = x.device
    q = _output(q, "q", E4M3_DTYPES, (R, C), dev)
    scales = _output(scales, "scales", _F32, (R, _blocks128(C)), dev)
    _call_on(dev, "fp8bs_quantize_tg128", x.data_ptr(), R, C, q.data_ptr(), scales.data_ptr())
    return q, scales


def quantize_b128(x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                  transposed: bool = False, qt: torch.Tensor | None = None, scales_t: torch.Tensor | None = None):
    """bf16 weight [R, C] or weights [G, R, C] -> (E4M3 codes uint8 of the same shape, fp32 scales
    [(G,) ceil(R/128), ceil(C/128)], one per 128x128 block).

    With ``transposed`` (or when ``qt`` and ``scales_t`` are given) also the transposed codes [(G,) C, R]
    and scales [(G,) ceil(C/128), ceil(R/128)], as third and fourth elements."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be a tensor of 2 or 3 dimensions")
    _need(x, "x", _BF16, x.dim())
    lead = tuple(x.shape[:-2])
    R, C = x.shape[-2:]
    G = lead[0] if lead else 1
    dev = x.device
    if (qt is None) != (scales_t is None):
        raise ValueError("qt and scales_t go together")
    transposed = transposed or qt is not None
    q = _output(q, "q", E4M3_DTYPES, lead + (R, C), dev)
    scales = _output(scales, "scales", _F32, lead + (_blocks128(R), _blocks128(C)), dev)
    if transposed:
        qt = _output(qt, "qt", E4M3_DTYPES, lead + (C, R), dev)
        scales_t = _output(scales_t, "scales_t", _F32, lead + (_blocks128(C), _blocks128(R)), dev)
    _call_on(dev, "fp8bs_quantize_b128", x.data_ptr(), G, R, C, q.data_ptr(), scales.data_ptr(), _ptr(qt),
             _ptr(scales_t))
    return (q, scales, qt, scales_t) if transposed else (q, scales)


def gemm_tg128_nt(a: torch.Tensor, sa: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor,
                  out: torch.Tensor | None = None):
    """E4M3 a [M, K], sa [M, ceil(K/128)], K-major weight bt [N, K], sbt [ceil(N/128), ceil(K/128)] -> bf16 [M, N]."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 2)
    M, K = a.shape
    N, KB, dev = bt.shape[0], _blocks128(K), a.device
    _need_size(bt, "bt", 1, K, dev)
    _need_like(sa, "sa", _F32, (M, KB), dev)
    _need_like(sbt, "sbt", _F32, (_blocks128(N), KB), dev)
    out = _output(out, "out", _BF16, (M, N), dev)
    _call_on(dev, "fp8bs_gemm_tg128_nt", a.data_ptr(), sa.data_ptr(), bt.data_ptr(), sbt.data_ptr(), out.data_ptr(), M,
             N, K)
    return out


def grouped_gemm_tg128_nt(a: torch.Tensor, sa: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor,
                          offsets: torch.Tensor, out: torch.Tensor | None = None):
    """a [M_total, K], sa [M_total, ceil(K/128)], weights bt [G, N, K], sbt [G, ceil(N/128), ceil(K/128)],
    offsets int32 [G+1] on the device (any ascending row numbers) -> bf16 [M_total, N].

    Rows outside every range keep what ``out`` holds (a new ``out`` is not initialised)."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 3)
    M, K = a.shape
    G, N, _ = bt.shape
    KB, dev = _blocks128(K), a.device
    _need_size(bt, "bt", 2, K, dev)
    _need_like(offsets, "offsets", _I32, (G + 1,), dev)
    _need_like(sa, "sa", _F32, (M, KB), dev)
    _need_like(sbt, "sbt", _F32, (G, _blocks128(N), KB), dev)
    out = _output(out, "out", _BF16, (M, N), dev)
    _call_on(dev, "fp8bs_grouped_gemm_tg128_nt", a.data_ptr(), sa.data_ptr(), bt.data_ptr(), sbt.data_ptr(),
             offsets.data_ptr(), G, out.data_ptr(), M, N, K)
    return out


def grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                  accumulate: bool = False):
    """bf16 dy [M_total, N], x [M_total, K], offsets int32 [G+1] on the device -> fp32 [G, N, K], the sums of
    dy[m, n] * x[m, k] over each range's rows; with ``accumulate`` they are added to ``out``."""
    _need(dy, "dy", _BF16, 2)
    _need(x, "x", _BF16, 2)
    _need(offsets, "offsets", _I32, 1)
    M, N = dy.shape
    K, G, dev = x.shape[1], offsets.shape[0] - 1, dy.device
    _need_size(x, "x", 0, M, dev)
    _need_size(offsets, "offsets", 0, G + 1, dev)
    if G < 1:
        raise ValueError("offsets needs at least two entries")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out = _output(out, "out", _F32, (G, N, K), dev)
    _call_on(dev, "fp8bs_grouped_wgrad", dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), G, out.data_ptr(),
             1 if accumulate else 0, M, N, K)
    return out


def swiglu_quantize_tg128(gu: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                          y: torch.Tensor | None = None, want_y: bool = False):
    """bf16 [R, 2d] = [gate | up] -> silu(gate) * up, quantized as by quantize_tg128 from its fp32 values:
    (q uint8 [R, d], scales fp32 [R, ceil(d/128)]), plus the bf16 values [R, d] as a third element when
    ``want_y`` is true or ``y`` is given."""
    _need(gu, "gu", _BF16, 2)
    R, d2 = gu.shape
    if d2 % 2:
        raise ValueError("gu needs an even number of columns")
    d, dev = d2 // 2, gu.device
    q = _output(q, "q", E4M3_DTYPES, (R, d), dev)
    scales = _output(scales, "scales", _F32, (R, _blocks128(d)), dev)
    if y is not None or want_y:
        y = _output(y, "y", _BF16, (R, d), dev)
    _call_on(dev, "fp8bs_swiglu_quantize_tg128", gu.data_ptr(), R, d, q.data_ptr(), scales.data_ptr(), _ptr(y))
    return (q, scales) if y is None else (q, scales, y)


def swiglu_backward_quantize_tg128(gu: torch.Tensor, dy: torch.Tensor, dgu: torch.Tensor | None = None,
                                   q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                                   y: torch.Tensor | None = None, want_y: bool = False):
    """The gradient of silu(gate) * up for bf16 gu [R, 2d] and dy [R, d]: (dgu bf16 [R, 2d], its codes uint8
    [R, 2d] and scales fp32 [R, ceil(2d/128)] as by quantize_tg128 from the fp32 values), plus the forward
    value bf16 [R, d] as a fourth element when ``want_y`` is true or ``y`` is given."""
    _need(gu, "gu", _BF16, 2)
    _need(dy, "dy", _BF16, 2)
    R, d = dy.shape
    dev = dy.device
    _need_like(gu, "gu", _BF16, (R, 2 * d), dev)
    dgu = _output(dgu, "dgu", _BF16, (R, 2 * d), dev)
    q = _output(q, "q", E4M3_DTYPES, (R, 2 * d), dev)
    scales = _output(scales, "scales", _F32, (R, _blocks128(2 * d)), dev)
    if y is not None or want_y:
        y = _output(y, "y", _BF16, (R, d), dev)
    _call_on(dev, "fp8bs_swiglu_backward_quantize_tg128", gu.data_ptr(), dy.data_ptr(), R, d, dgu.data_ptr(),
             q.data_ptr(), scales.data_ptr(), _ptr(y))
    return (dgu, q, scales) if y is None else (dgu, q, scales, y)


# ---- between the products of a block (include/fp8bs_layer.h) ----------------------------------
def _norm_inputs(x, gamma, beta, residual, h, mean, rstd, want_stats):
    """The arguments that both forms of the layer norm have, checked, and the outputs that are not given:
    (rows, columns, device, h, mean, rstd)."""
    _need(x, "x", _BF16, 2)
    R, d = x.shape
    dev = x.device
    _need_like(gamma, "gamma", _BF16, (d,), dev)
    if beta is not None:
        _need_like(beta, "beta", _BF16, (d,), dev)
    if residual is not None:
        _need_like(residual, "residual", _BF16, (R, d), dev)
        h = residual if h is None else _need_like(h, "h", _BF16, (R, d), dev)
    elif h is not None:
        raise ValueError("h needs residual")
    if (mean is None) != (rstd is None):
        raise ValueError("mean and rstd go together")
    if want_stats or mean is not None:
        mean, rstd = _output(mean, "mean", _F32, (R,), dev), _output(rstd, "rstd", _F32, (R,), dev)
    return R, d, dev, h, mean, rstd


def layernorm_quantize_tg128(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor | None, eps: float,
                             residual: torch.Tensor | None = None, h: torch.Tensor | None = None,
                             q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                             y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                             rstd: torch.Tensor | None = None, want_y: bool = False, want_stats: bool = False):
    """Residual add + layer norm of bf16 x [R, d] with weight gamma [d] and bias beta [d] (or None), quantized as
    by quantize_tg128 from its fp32 values: (q uint8 [R, d], scales fp32 [R, ceil(d/128)]).

    With ``residual`` the rows are h = x + residual, written to ``h``, or in place to ``residual`` if ``h`` is not
    given.  When ``want_y`` is true or ``y`` is given the bf16 rows follow, when ``want_stats`` is true or ``mean``
    and ``rstd`` are given the fp32 statistics [R] that layernorm_backward takes: (q, scales[, y][, mean, rstd])."""
    R, d, dev, h, mean, rstd = _norm_inputs(x, gamma, beta, residual, h, mean, rstd, want_stats)
    q = _output(q, "q", E4M3_DTYPES, (R, d), dev)
    scales = _output(scales, "scales", _F32, (R, _blocks128(d)), dev)
    if y is not None or want_y:
        y = _output(y, "y", _BF16, (R, d), dev)
    _call_on(dev, "fp8bs_layernorm_quantize_tg128", x.data_ptr(), _ptr(residual), gamma.data_ptr(), _ptr(beta),
             float(eps), R, d, _ptr(h), q.data_ptr(), scales.data_ptr(), _ptr(y), _ptr(mean), _ptr(rstd))
    return (q, scales) + (() if y is None else (y,)) + (() if mean is None else (mean, rstd))


def layernorm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor | None, eps: float,
              residual: torch.Tensor | None = None, h: torch.Tensor | None = None, y: torch.Tensor | None = None,
              mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None, want_stats: bool = False):
    """As layernorm_quantize_tg128 without codes: y bf16 [R, d], or (y, mean, rstd) when ``want_stats`` is true or
    ``mean`` and ``rstd`` are given."""
    R, d, dev, h, mean, rstd = _norm_inputs(x, gamma, beta, residual, h, mean, rstd, want_stats)
    y = _output(y, "y", _BF16, (R, d), dev)
    _call_on(dev, "fp8bs_layernorm", x.data_ptr(), _ptr(residual), gamma.data_ptr(), _ptr(beta), float(eps), R, d,
             _ptr(h), y.data_ptr(), _ptr(mean), _ptr(rstd))
    return y if mean is None else (y, mean, rstd)


def layernorm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor,
                       rstd: torch.Tensor, dresidual: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                       dgamma: torch.Tensor | None = None, dbeta: torch.Tensor | None = None,
                       accumulate: bool = False):
    """The gradients of the layer norm of the bf16 rows h [R, d] for bf16 dy [R, d], with the statistics that the
    forward call gave: (dx bf16 [R, d], dgamma fp32 [d], dbeta fp32 [d]).

    ``dresidual`` bf16 [R, d], the gradient that reaches h past the norm, is added to dx; with ``accumulate`` the sums
    are added to the given ``dgamma`` and ``dbeta``."""
    _need(dy, "dy", _BF16, 2)
    R, d = dy.shape
    dev = dy.device
    _need_like(h, "h", _BF16, (R, d), dev)
    _need_like(gamma, "gamma", _BF16, (d,), dev)
    _need_like(mean, "mean", _F32, (R,), dev)
    _need_like(rstd, "rstd", _F32, (R,), dev)
    if dresidual is not None:
        _need_like(dresidual, "dresidual", _BF16, (R, d), dev)
    if accumulate and (dgamma is None or dbeta is None):
        raise ValueError("accumulate needs dgamma and dbeta")
    dx = _output(dx, "dx", _BF16, (R, d), dev)
    dgamma, dbeta = _output(dgamma, "dgamma", _F32, (d,), dev), _output(dbeta, "dbeta", _F32, (d,), dev)
    size = (_lib or load_library()).fp8bs_layernorm_backward_workspace(R, d)
    ws = _workspace(size, dev)
    _call_on(dev, "fp8bs_layernorm_backward", dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), mean.data_ptr(),
             rstd.data_ptr(), _ptr(dresidual), R, d, dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(),
             1 if accumulate else 0, ws.data_ptr(), size)
    return dx, dgamma, dbeta


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation {name!r} is none of {tuple(ACTIVATIONS)}")
    return code


def gemm_tg128_nt_epilogue(a: torch.Tensor, sa: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor,
                           bias: torch.Tensor | None = None, activation: str = "none",
                           residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                           pre: torch.Tensor | None = None, want_pre: bool = False):
    """act(a bt' + bias) + residual for operands as gemm_tg128_nt's, bias bf16 [N], residual bf16 [M, N] (``out`` may
    be it) and an activation of ACTIVATIONS, all in fp32 and rounded once to bf16 [M, N]; when ``want_pre`` is true
    or ``pre`` is given, (out, pre) with a bt' + bias in bf16 for epilogue_backward_quantize_tg128."""
    _need(a, "a", E4M3_DTYPES, 2)
    _need(bt, "bt", E4M3_DTYPES, 2)
    code = _activation(activation)
    M, K = a.shape
    N, KB, dev = bt.shape[0], _blocks128(K), a.device
    _need_size(bt, "bt", 1, K, dev)
    _need_like(sa, "sa", _F32, (M, KB), dev)
    _need_like(sbt, "sbt", _F32, (_blocks128(N), KB), dev)
    if bias is not None:
        _need_like(bias, "bias", _BF16, (N,), dev)
    if residual is not None:
        _need_like(residual, "residual", _BF16, (M, N), dev)
    out = _output(out, "out", _BF16, (M, N), dev)
    if pre is not None or want_pre:
        pre = _output(pre, "pre", _BF16, (M, N), dev)
    _call_on(dev, "fp8bs_gemm_tg128_nt_epilogue", a.data_ptr(), sa.data_ptr(), bt.data_ptr(), sbt.data_ptr(),
             _ptr(bias), code, _ptr(residual), out.data_ptr(), _ptr(pre), M, N, K)
    return out if pre is None else (out, pre)


def epilogue_backward_quantize_tg128(dout: torch.Tensor, pre: torch.Tensor | None, activation: str = "none",
                                     dz: torch.Tensor | None = None, q: torch.Tensor | None = None,
                                     scales: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                                     accumulate: bool = False):
    """The gradient of act(z) + residual with respect to z for bf16 dout [R, N] and the forward call's ``pre`` (which
    "none" does not need): (dz bf16 [R, N], its codes uint8 [R, N] and scales fp32 [R, ceil(N/128)] as by
    quantize_tg128 from the fp32 values, dbias fp32 [N], the sums of dz over the rows).  With ``accumulate`` they are
    added to the given ``dbias``."""
    _need(dout, "dout", _BF16, 2)
    code = _activation(activation)
    R, N = dout.shape
    dev = dout.device
    if pre is not None:
        _need_like(pre, "pre", _BF16, (R, N), dev)
    elif code:
        raise ValueError(f"activation {activation!r} needs pre")
    if accumulate and dbias is None:
        raise ValueError("accumulate needs dbias")
    dz = _output(dz, "dz", _BF16, (R, N), dev)
    q = _output(q, "q", E4M3_DTYPES, (R, N), dev)
    scales = _output(scales, "scales", _F32, (R, _blocks128(N)), dev)
    dbias = _output(dbias, "dbias", _F32, (N,), dev)
    size = (_lib or load_library()).fp8bs_epilogue_backward_workspace(R, N)
    ws = _workspace(size, dev)
    _call_on(dev, "fp8bs_epilogue_backward_quantize_tg128", dout.data_ptr(), _ptr(pre), code, R, N, dz.data_ptr(),
             q.data_ptr(), scales.data_ptr(), dbias.data_ptr(), 1 if accumulate else 0, ws.data_ptr(), size)
    return dz, q, scales, dbias


def moe_decode_b128(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w1: torch.Tensor, s1: torch.Tensor,
                    w2: torch.Tensor, s2: torch.Tensor, residual: torch.Tensor | None = None,
                    out: torch.Tensor | None = None):
    """A whole mixture-of-experts layer for a few tokens (tokens * choices <= 512): bf16 x [T, H], int32 ids [T, k],
    fp32 weights [T, k], E4M3 w1 [E, 2I, H] (gates, then ups) and w2 [E, H, I] with the fp32 scales of their 128x128
    blocks (quantize_b128) -> bf16 [T, H], the weighted sum over the choices of w2 (silu(gate) * up), plus
    ``residual`` bf16 [T, H] if given (``out`` may be it).  Choices with an id outside [0, E) add nothing.  From about
    15 choices of each expert on, quantize_tg128, grouped_gemm_tg128_nt and swiglu_quantize_tg128 take less time."""
    _need(x, "x", _BF16, 2)
    _need(w1, "w1", E4M3_DTYPES, 3)
    _need(ids, "ids", _I32, 2)
    T, H = x.shape
    E, I2, _ = w1.shape
    k, dev = ids.shape[1], x.device
    if I2 % 2:
        raise ValueError("w1 needs an even number of rows")
    inner = I2 // 2
    _need_size(w1, "w1", 2, H, dev)
    _need_size(ids, "ids", 0, T, dev)
    _need_like(weights, "weights", _F32, (T, k), dev)
    _need_like(w2, "w2", E4M3_DTYPES, (E, H, inner), dev)
    _need_like(s1, "s1", _F32, (E, _blocks128(I2), _blocks128(H)), dev)
    _need_like(s2, "s2", _F32, (E, _blocks128(H), _blocks128(inner)), dev)
    if residual is not None:
        _need_like(residual, "residual", _BF16, (T, H), dev)
    out = _output(out, "out", _BF16, (T, H), dev)
    size = (_lib or load_library()).fp8bs_moe_decode_b128_workspace(T, k, E, H, inner)
    ws = _workspace(size, dev)
    _call_on(dev, "fp8bs_moe_decode_b128", x.data_ptr(), ids.data_ptr(), weights.data_ptr(), w1.data_ptr(),
             s1.data_ptr(), w2.data_ptr(), s2.data_ptr(), _ptr(residual), out.data_ptr(), T, k, E, H, inner,
             ws.data_ptr(), size)
    return out


_GRAD_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _scalar(t: torch.Tensor | None, name: str, device: torch.device) -> torch.Tensor:
    """The caller's fp32 tensor without dimensions, checked, or a new one."""
    return torch.empty((), dtype=torch.float32, device=device) if t is None else _need_like(t, name, _F32, (), device)


def _workspace(size: int, device: torch.device) -> torch.Tensor:
    return torch.empty(size, dtype=torch.uint8, device=device)


_dtype_of = torch.Tensor.dtype.__get__


def _gradients(grads, name: str):
    """The tensors of a sequence, checked: (their dtypes, arrays of their addresses and counts, device).
    One pass over the list for each property, without a Python frame for each tensor (61 tensors: 54 -> 37 us)."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError(f"{name} is empty")
    try:
        dtypes = list(map(_dtype_of, grads))
    except TypeError:
        raise TypeError(f"{name} must hold tensors") from None
    for dtype in set(dtypes):
        if dtype not in _GRAD_TYPES:
            raise TypeError(f"{name}: dtype {dtype} not accepted ({tuple(_GRAD_TYPES)})")
    indices = set(map(torch.Tensor.get_device, grads))
    if -1 in indices or not grads[0].is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if len(indices) > 1:
        raise ValueError("all tensors must be on the same device")
    if not all(map(torch.Tensor.is_contiguous, grads)):
        raise ValueError(f"{name} must be contiguous")
    return (dtypes, array.array("Q", map(torch.Tensor.data_ptr, grads)),
            array.array("q", map(torch.Tensor.numel, grads)), grads[0].device)


class _Grads:
    """The host arrays of one call; they live until it returns."""

    def __init__(self, grads, out=None, clips=False):
        dtypes, self.src, self.counts, self.device = _gradients(grads, "grads")
        self.n = len(dtypes)
        self.types = array.array("i", map(_GRAD_TYPES.__getitem__, dtypes))
        self.dst = self.src
        if clips and out is not None:
            out_dtypes, self.dst, counts, device = _gradients(out, "out")
            if out_dtypes != dtypes or counts != self.counts or device != self.device:
                raise ValueError("out must match the gradients in number, types, sizes and device")

    def arguments(self, *arrays):
        return [a.buffer_info()[0] for a in arrays] + [self.n]

    def workspace(self):
        size = (_lib or load_library()).fp8bs_grad_norm_workspace(self.n)
        return _workspace(size, self.device), size


def grad_norm(grads, out: torch.Tensor | None = None) -> torch.Tensor:
    """The norm over all values of a sequence of contiguous fp32 and bf16 tensors: sqrt(sum of squares), summed
    in 64 bits, as an fp32 tensor without dimensions (on the device; nothing is copied to the host)."""
    g = _Grads(grads)
    out = _scalar(out, "out", g.device)
    ws, size = g.workspace()
    _call_on(g.device, "fp8bs_grad_norm", *g.arguments(g.src, g.counts, g.types), out.data_ptr(), ws.data_ptr(), size)
    return out


def clip_grads(grads, norm: torch.Tensor, max_norm: float, out=None, eps: float = 1e-6) -> None:
    """Scales the gradients by min(1, max_norm / (norm + eps)) for an fp32 ``norm`` on the device, in place, or into
    the tensors ``out`` (each of its gradient's type and size; a gradient itself, or memory of its own)."""
    g = _Grads(grads, out, clips=True)
    _need_like(norm, "norm", _F32, (), g.device)
    _call_on(g.device, "fp8bs_clip_grads", *g.arguments(g.src, g.dst, g.counts, g.types), norm.data_ptr(),
             float(max_norm), float(eps))


def clip_grad_norm(grads, max_norm: float, out=None, eps: float = 1e-6,
                   norm: torch.Tensor | None = None) -> torch.Tensor:
    """The norm over all gradients (as by grad_norm), which is returned, and their scaling by
    min(1, max_norm / (norm + eps)), in place or into ``out`` (as by clip_grads).  ``max_norm`` is finite: the norm
    without clipping is grad_norm's."""
    g = _Grads(grads, out, clips=True)
    norm = _scalar(norm, "norm", g.device)
    ws, size = g.workspace()
    _call_on(g.device, "fp8bs_clip_grad_norm", *g.arguments(g.src, g.dst, g.counts, g.types), float(max_norm),
             float(eps), norm.data_ptr(), ws.data_ptr(), size)
    return norm
