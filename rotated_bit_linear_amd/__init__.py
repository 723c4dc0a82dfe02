"""Thin Python binding of libconvrot.so (the gfx950 rotated W8A8 NVFP4 linear layer).

Argument marshalling only: torch tensors provide device memory and the current HIP
stream; every step of the computation runs in the library's HIP kernels.  There is no
fallback: if the library is missing it is built, and if it cannot be loaded or the
device is not gfx950 the calls raise.

The C entry points are exposed under their own names (``cr_quant_act`` ...), taking
tensors in place of pointers; ``linear_nvfp4`` allocates the output and the workspace
and runs the whole layer.
"""
from __future__ import annotations

import ctypes as C
import os
import re

import torch

from . import build as _build

CR_ABI_VERSION = 3
CR_BF16, CR_FP16, CR_FP32, CR_I32 = 0, 1, 2, 3
CR_FLAG_NONE, CR_FLAG_FORCE_TWO_PASS, CR_FLAG_BLOCK_TRANSPOSED = 0, 1, 2
CR_FLAG_CAUSAL, CR_FLAG_ROPE_INTERLEAVED = 16, 32
KV8_PAGE = 64
CR_MAX_K_PAD = 133120
NOALLOC_SCRATCH_BYTES = 64 << 20
DEFAULT_MAX_TILE_BYTES = 128 << 20
STATUS = {0: "CR_OK", 1: "CR_ERR_INVALID_ARG", 2: "CR_ERR_UNSUPPORTED_DTYPE", 3: "CR_ERR_MISALIGNED",
          4: "CR_ERR_TOO_LARGE", 5: "CR_ERR_NO_DEVICE", 6: "CR_ERR_LAUNCH"}

_TORCH_TO_CR = {torch.bfloat16: CR_BF16, torch.float16: CR_FP16, torch.float32: CR_FP32,
                torch.int32: CR_I32}
_CR_TO_TORCH = {v: k for k, v in _TORCH_TO_CR.items()}

LIB_PATH = _build.LIB
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "convrot.h")


class _Kv8(C.Structure):
    """cr_kv8_cache"""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("n_pages", C.c_int64), ("page_table", C.c_void_p), ("ld_table", C.c_int64)]


class CrError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def lib() -> C.CDLL:
    """The loaded library (built in-tree first if absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            _build.build()
        L = C.CDLL(LIB_PATH)
        i64, u32, vp, sz = C.c_int64, C.c_uint32, C.c_void_p, C.c_size_t
        sig = {
            "cr_abi_version": (C.c_int, []),
            "cr_status_string": (C.c_char_p, [C.c_int]),
            "cr_padded_k": (i64, [i64]),
            "cr_prep_weight_nvfp4": (C.c_int, [vp, i64, vp, i64, vp, i64, i64, vp, i64, vp, u32, vp]),
            "cr_quant_act": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, i64, vp, u32, vp]),
            "cr_quant_act_swiglu": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, i64, vp, u32, vp]),
            "cr_quant_act_rmsnorm": (C.c_int, [vp, C.c_int, i64, vp, i64, vp, i64, vp, C.c_float, i64, i64, vp, i64,
                                               vp, u32, vp]),
            "cr_swiglu": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, i64, vp]),
            "cr_gemm_s8_rowscale": (C.c_int, [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, C.c_int, i64, vp]),
            "cr_gemm_s8_rowscale_bias": (C.c_int, [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, vp, C.c_int, i64,
                                                   vp]),
            "cr_quant_act_ex": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, vp, i64, vp, u32, vp]),
            "cr_linear_nvfp4_workspace_bytes": (sz, [i64, i64, i64, sz]),
            "cr_linear_nvfp4_plan": (C.c_int, [i64, i64, i64, sz, C.POINTER(i64), C.POINTER(i64)]),
            "cr_linear_nvfp4": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, i64, vp, i64,
                                          vp, C.c_int, i64, vp, sz, sz, u32, vp, vp]),
            "cr_linear_nvfp4_ex": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, vp, i64, vp, i64, vp,
                                             i64, vp, vp, C.c_int, i64, vp, sz, sz, u32, vp, vp]),
            "cr_linear_nvfp4_noalloc": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, vp, i64, vp, i64, vp,
                                                  i64, vp, vp, C.c_int, i64, sz, u32, vp]),
            "cr_weight_amax_nvfp4": (C.c_int, [vp, i64, vp, i64, vp, i64, i64, vp, u32, vp]),
            "cr_quant_weight_w4": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, i64, vp, u32, vp]),
            "cr_gemm_s8s4_rowscale": (C.c_int, [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, vp, C.c_int, i64, vp]),
            "cr_linear_w4a8_workspace_bytes": (sz, [i64, i64]),
            "cr_linear_w4a8": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, i64, vp, vp, C.c_int,
                                         i64, vp, sz, u32, vp]),
            "cr_quant_act_w4": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, u32, vp]),
            "cr_gemm_s4s4_rowscale": (C.c_int, [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, vp, C.c_int, i64, vp]),
            "cr_linear_w4a4_workspace_bytes": (sz, [i64, i64]),
            "cr_linear_w4a4": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, i64, vp, vp, C.c_int,
                                         i64, vp, sz, u32, vp]),
            "cr_quant_weight_w4_e2m3": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, i64, vp, u32, vp]),
            "cr_repack_w4_e2m3": (C.c_int, [vp, i64, i64, i64, vp, i64, vp]),
            "cr_quant_act_w4_e2m3": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, u32, vp]),
            "cr_gemm_e2m3_rowscale": (C.c_int, [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, vp, C.c_int, i64, vp]),
            "cr_linear_w4a4_e2m3_workspace_bytes": (sz, [i64, i64]),
            "cr_linear_w4a4_e2m3": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, i64, vp, i64, vp, i64, vp, vp,
                                              C.c_int, i64, vp, sz, u32, vp]),
            "cr_rope_append_kv8": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, vp, i64, i64, i64, i64, vp, vp, C.c_float,
                                             vp, i64, i64, vp, vp, vp, i64, C.POINTER(_Kv8), u32, vp]),
            "cr_attn_kv8_workspace_bytes": (sz, [i64, i64, i64, i64, i64, i64, i64]),
            "cr_attn_kv8": (C.c_int, [vp, C.c_int, i64, i64, i64, vp, vp, i64, i64, i64, i64, i64, C.POINTER(_Kv8),
                                      C.c_float, vp, i64, vp, sz, u32, vp]),
            "cr_gemm_nvfp4_fused": (C.c_int, [vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, vp,
                                              C.c_int, i64, u32, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        v = L.cr_abi_version()
        if v != CR_ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH}: ABI version {v}, binding expects {CR_ABI_VERSION}")
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/convrot.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(cr_\w+)\s*\(", src)))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without a Stream object: 0.2 us a call against 2.8 of the public way,
# where a short call takes 11.  The names are not public, so a torch without them has the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is None or _raw_device is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_raw_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise CrError(fn, status)


def _rows_ld(t: torch.Tensor):
    st = t.stride()
    assert len(st) == 2 and st[1] == 1, "expected a row-major 2-D tensor (unit column stride)"
    return t.size(0), st[0]


def _ld(t: torch.Tensor) -> int:
    """Row stride of a row-major 2-D tensor."""
    st = t.stride()
    assert len(st) == 2 and st[1] == 1, "expected a row-major 2-D tensor (unit column stride)"
    return st[0]


def _vector(name: str, t, n: int, dtype=torch.float32) -> int | None:
    """Address of an optional contiguous vector argument of at least n elements."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {n} elements")
    return t.data_ptr()


def padded_k(k: int) -> int:
    return int(lib().cr_padded_k(k))


# ------------------------------------------------------------------- entry points ----

def cr_prep_weight_nvfp4(w_fp4, w_sf, global_scale, K, w_s8, w_scale, flags=0, stream=None):
    n, ld_fp4 = _rows_ld(w_fp4)
    _, ld_sf = _rows_ld(w_sf)
    _, ld_s8 = _rows_ld(w_s8)
    _check("cr_prep_weight_nvfp4", lib().cr_prep_weight_nvfp4(
        _ptr(w_fp4), ld_fp4, _ptr(w_sf), ld_sf, _ptr(global_scale), n, K, _ptr(w_s8), ld_s8,
        _ptr(w_scale), flags, _stream(stream)))


def cr_quant_act(x, K, x_s8, x_scale, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    _, ld_s8 = _rows_ld(x_s8)
    _check("cr_quant_act", lib().cr_quant_act(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, M, K, _ptr(x_s8), ld_s8, _ptr(x_scale), flags,
        _stream(stream)))


def cr_quant_act_swiglu(h, F, x_s8, x_scale, flags=0, stream=None):
    M, ld_h = _rows_ld(h)
    _, ld_s8 = _rows_ld(x_s8)
    _check("cr_quant_act_swiglu", lib().cr_quant_act_swiglu(
        _ptr(h), _TORCH_TO_CR[h.dtype], ld_h, M, F, _ptr(x_s8), ld_s8, _ptr(x_scale), flags,
        _stream(stream)))


def cr_quant_act_ex(x, K, swiglu, pre_scale, x_s8, x_scale, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    _, ld_s8 = _rows_ld(x_s8)
    _check("cr_quant_act_ex", lib().cr_quant_act_ex(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(pre_scale), _ptr(x_s8), ld_s8,
        _ptr(x_scale), flags, _stream(stream)))


def cr_quant_act_rmsnorm(x, residual, sum, weight, eps, K, x_s8, x_scale, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    r = h = None
    ld_r = ld_h = 0
    if residual is not None:
        if residual.shape != x.shape or residual.dtype is not x.dtype:
            raise ValueError("residual must have the shape and dtype of x")
        r, ld_r = residual.data_ptr(), _ld(residual)
    if sum is not None:
        if sum.shape != x.shape or sum.dtype is not x.dtype:
            raise ValueError("sum must have the shape and dtype of x")
        h, ld_h = sum.data_ptr(), _ld(sum)
    status = lib().cr_quant_act_rmsnorm(
        x.data_ptr(), _TORCH_TO_CR.get(x.dtype, -1), ld_x, r, ld_r, h, ld_h, _vector("weight", weight, K), eps, M, K,
        x_s8.data_ptr(), _ld(x_s8), x_scale.data_ptr(), flags, _stream(stream))
    if status:
        raise CrError("cr_quant_act_rmsnorm", status)


def cr_swiglu(h, F, out, stream=None):
    M, ld_h = _rows_ld(h)
    _, ld_out = _rows_ld(out)
    _check("cr_swiglu", lib().cr_swiglu(_ptr(h), _TORCH_TO_CR[h.dtype], ld_h, M, F, _ptr(out), ld_out,
                                        _stream(stream)))


def cr_gemm_s8_rowscale(a_s8, a_scale, b_s8, b_scale, c, stream=None, M=None, N=None):
    Ma, lda = _rows_ld(a_s8)
    Nb, ldb = _rows_ld(b_s8)
    _, ldc = _rows_ld(c)
    M = Ma if M is None else M
    N = Nb if N is None else N
    K_pad = a_s8.shape[1]
    _check("cr_gemm_s8_rowscale", lib().cr_gemm_s8_rowscale(
        _ptr(a_s8), lda, _ptr(a_scale), _ptr(b_s8), ldb, _ptr(b_scale), M, N, K_pad, _ptr(c),
        _TORCH_TO_CR[c.dtype], ldc, _stream(stream)))


def cr_linear_nvfp4_workspace_bytes(M, N, K, max_tile_bytes=0) -> int:
    return int(lib().cr_linear_nvfp4_workspace_bytes(M, N, K, max_tile_bytes))


def cr_gemm_s8_rowscale_bias(a_s8, a_scale, b_s8, b_scale, bias, c, stream=None):
    M, lda = _rows_ld(a_s8)
    N, ldb = _rows_ld(b_s8)
    _, ldc = _rows_ld(c)
    _check("cr_gemm_s8_rowscale_bias", lib().cr_gemm_s8_rowscale_bias(
        _ptr(a_s8), lda, _ptr(a_scale), _ptr(b_s8), ldb, _ptr(b_scale), _ptr(bias), M, N, a_s8.shape[1],
        _ptr(c), _TORCH_TO_CR[c.dtype], ldc, _stream(stream)))


def cr_linear_nvfp4_plan(M, N, K, max_tile_bytes=0) -> tuple[int, int]:
    """(rows per weight chunk, number of chunks) that cr_linear_nvfp4 uses on this device."""
    r, n = C.c_int64(0), C.c_int64(0)
    _check("cr_linear_nvfp4_plan", lib().cr_linear_nvfp4_plan(M, N, K, max_tile_bytes,
                                                              C.byref(r), C.byref(n)))
    return int(r.value), int(n.value)


def cr_linear_nvfp4(x, K, swiglu, w_fp4, w_sf, global_scale, out, workspace, max_tile_bytes=0,
                    flags=0, stream=None, aux_stream=None, pre_scale=None, bias=None):
    """cr_linear_nvfp4, or cr_linear_nvfp4_ex when a pre-scale or a bias is given."""
    M, ld_x = _rows_ld(x)
    N, ld_fp4 = _rows_ld(w_fp4)
    _, ld_sf = _rows_ld(w_sf)
    _, ldc = _rows_ld(out)
    aux = None if aux_stream is None else _stream(aux_stream)
    ws = (_ptr(workspace), workspace.numel() * workspace.element_size(), max_tile_bytes, flags,
          _stream(stream), aux)
    if pre_scale is None and bias is None:
        _check("cr_linear_nvfp4", lib().cr_linear_nvfp4(
            _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(w_fp4), ld_fp4,
            _ptr(w_sf), ld_sf, _ptr(global_scale), N, _ptr(out), _TORCH_TO_CR[out.dtype], ldc, *ws))
    else:
        _check("cr_linear_nvfp4_ex", lib().cr_linear_nvfp4_ex(
            _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(pre_scale), _ptr(w_fp4), ld_fp4,
            _ptr(w_sf), ld_sf, _ptr(global_scale), N, _ptr(bias), _ptr(out), _TORCH_TO_CR[out.dtype], ldc, *ws))


def cr_linear_nvfp4_noalloc(x, K, swiglu, w_fp4, w_sf, global_scale, out, max_tile_bytes=0, flags=0,
                            stream=None, pre_scale=None, bias=None):
    """The layer with the library's own device scratch as its workspace (nothing allocated)."""
    M, ld_x = _rows_ld(x)
    N, ld_fp4 = _rows_ld(w_fp4)
    _, ld_sf = _rows_ld(w_sf)
    _, ldc = _rows_ld(out)
    _check("cr_linear_nvfp4_noalloc", lib().cr_linear_nvfp4_noalloc(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(pre_scale), _ptr(w_fp4), ld_fp4,
        _ptr(w_sf), ld_sf, _ptr(global_scale), N, _ptr(bias), _ptr(out), _TORCH_TO_CR[out.dtype], ldc,
        max_tile_bytes, flags, _stream(stream)))


def cr_weight_amax_nvfp4(w_fp4, w_sf, global_scale, K, w_amax, flags=0, stream=None):
    n, ld_fp4 = _rows_ld(w_fp4)
    _, ld_sf = _rows_ld(w_sf)
    _check("cr_weight_amax_nvfp4", lib().cr_weight_amax_nvfp4(
        _ptr(w_fp4), ld_fp4, _ptr(w_sf), ld_sf, _ptr(global_scale), n, K, _ptr(w_amax), flags, _stream(stream)))


def cr_gemm_nvfp4_fused(a_s8, a_scale, w_fp4, w_sf, global_scale, w_amax, K, c, bias=None, flags=0,
                        stream=None):
    M, lda = _rows_ld(a_s8)
    N, ld_fp4 = _rows_ld(w_fp4)
    _, ld_sf = _rows_ld(w_sf)
    _, ldc = _rows_ld(c)
    _check("cr_gemm_nvfp4_fused", lib().cr_gemm_nvfp4_fused(
        _ptr(a_s8), lda, _ptr(a_scale), _ptr(w_fp4), ld_fp4, _ptr(w_sf), ld_sf, _ptr(global_scale),
        _ptr(w_amax), _ptr(bias), M, N, K, _ptr(c), _TORCH_TO_CR[c.dtype], ldc, flags, _stream(stream)))


def cr_quant_weight_w4(w, K, w_s4, w_scale, flags=0, stream=None):
    N, ld_w = _rows_ld(w)
    _, ld_s4 = _rows_ld(w_s4)
    _check("cr_quant_weight_w4", lib().cr_quant_weight_w4(
        _ptr(w), _TORCH_TO_CR[w.dtype], ld_w, N, K, _ptr(w_s4), ld_s4, _ptr(w_scale), flags, _stream(stream)))


def cr_gemm_s8s4_rowscale(a_s8, a_scale, b_s4, b_scale, c, bias=None, stream=None):
    M, lda = _rows_ld(a_s8)
    N, ldb = _rows_ld(b_s4)
    _, ldc = _rows_ld(c)
    _check("cr_gemm_s8s4_rowscale", lib().cr_gemm_s8s4_rowscale(
        _ptr(a_s8), lda, _ptr(a_scale), _ptr(b_s4), ldb, _ptr(b_scale), _ptr(bias), M, N, a_s8.shape[1],
        _ptr(c), _TORCH_TO_CR[c.dtype], ldc, _stream(stream)))


def cr_linear_w4a8_workspace_bytes(M, K) -> int:
    return int(lib().cr_linear_w4a8_workspace_bytes(M, K))


def cr_linear_w4a8(x, K, swiglu, w_s4, w_scale, out, workspace, bias=None, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    N, ld_s4 = _rows_ld(w_s4)
    _, ldc = _rows_ld(out)
    _check("cr_linear_w4a8", lib().cr_linear_w4a8(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(w_s4), ld_s4, _ptr(w_scale), N,
        _ptr(bias), _ptr(out), _TORCH_TO_CR[out.dtype], ldc, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), flags, _stream(stream)))


def cr_quant_act_w4(x, K, swiglu, x_s4, x_scale, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    _, ld_s4 = _rows_ld(x_s4)
    _check("cr_quant_act_w4", lib().cr_quant_act_w4(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(x_s4), ld_s4, _ptr(x_scale), flags,
        _stream(stream)))


def cr_gemm_s4s4_rowscale(a_s4, a_scale, b_s4, b_scale, c, bias=None, K_pad=None, stream=None):
    M, lda = _rows_ld(a_s4)
    N, ldb = _rows_ld(b_s4)
    _, ldc = _rows_ld(c)
    kp = 2 * a_s4.shape[1] if K_pad is None else K_pad
    _check("cr_gemm_s4s4_rowscale", lib().cr_gemm_s4s4_rowscale(
        _ptr(a_s4), lda, _ptr(a_scale), _ptr(b_s4), ldb, _ptr(b_scale), _ptr(bias), M, N, kp,
        _ptr(c), _TORCH_TO_CR[c.dtype], ldc, _stream(stream)))


def cr_linear_w4a4_workspace_bytes(M, K) -> int:
    return int(lib().cr_linear_w4a4_workspace_bytes(M, K))


def cr_linear_w4a4(x, K, swiglu, w_s4, w_scale, out, workspace, bias=None, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    N, ld_s4 = _rows_ld(w_s4)
    _, ldc = _rows_ld(out)
    _check("cr_linear_w4a4", lib().cr_linear_w4a4(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(w_s4), ld_s4, _ptr(w_scale), N,
        _ptr(bias), _ptr(out), _TORCH_TO_CR[out.dtype], ldc, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), flags, _stream(stream)))


def cr_quant_weight_w4_e2m3(w, K, w_f6, w_scale, flags=0, stream=None):
    N, ld_w = _rows_ld(w)
    _, ld_f6 = _rows_ld(w_f6)
    _check("cr_quant_weight_w4_e2m3", lib().cr_quant_weight_w4_e2m3(
        _ptr(w), _TORCH_TO_CR[w.dtype], ld_w, N, K, _ptr(w_f6), ld_f6, _ptr(w_scale), flags, _stream(stream)))


def cr_repack_w4_e2m3(w_s4, w_f6, K_pad=None, stream=None):
    N, ld_s4 = _rows_ld(w_s4)
    _, ld_f6 = _rows_ld(w_f6)
    kp = 2 * w_s4.shape[1] if K_pad is None else K_pad
    _check("cr_repack_w4_e2m3", lib().cr_repack_w4_e2m3(_ptr(w_s4), ld_s4, N, kp, _ptr(w_f6), ld_f6,
                                                          _stream(stream)))


def cr_quant_act_w4_e2m3(x, K, swiglu, x_f6, x_scale, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    _, ld_f6 = _rows_ld(x_f6)
    _check("cr_quant_act_w4_e2m3", lib().cr_quant_act_w4_e2m3(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(x_f6), ld_f6, _ptr(x_scale), flags,
        _stream(stream)))


def cr_gemm_e2m3_rowscale(a_f6, a_scale, b_f6, b_scale, c, bias=None, K_pad=None, stream=None):
    """E2M3-field operands are [quads, >= 3 K_pad] uint8 (four code rows per tensor row); M and N
    are the output's extents."""
    _, lda = _rows_ld(a_f6)
    _, ldb = _rows_ld(b_f6)
    M, ldc = _rows_ld(c)
    N = c.shape[1]
    kp = a_f6.shape[1] // 3 if K_pad is None else K_pad
    _check("cr_gemm_e2m3_rowscale", lib().cr_gemm_e2m3_rowscale(
        _ptr(a_f6), lda, _ptr(a_scale), _ptr(b_f6), ldb, _ptr(b_scale), _ptr(bias), M, N, kp,
        _ptr(c), _TORCH_TO_CR[c.dtype], ldc, _stream(stream)))


def cr_linear_w4a4_e2m3_workspace_bytes(M, K) -> int:
    return int(lib().cr_linear_w4a4_e2m3_workspace_bytes(M, K))


def cr_linear_w4a4_e2m3(x, K, swiglu, w_f6, w_scale, out, workspace, bias=None, flags=0, stream=None):
    M, ld_x = _rows_ld(x)
    _, ld_f6 = _rows_ld(w_f6)
    _, ldc = _rows_ld(out)
    N = out.shape[1]
    _check("cr_linear_w4a4_e2m3", lib().cr_linear_w4a4_e2m3(
        _ptr(x), _TORCH_TO_CR[x.dtype], ld_x, int(bool(swiglu)), M, K, _ptr(w_f6), ld_f6, _ptr(w_scale), N,
        _ptr(bias), _ptr(out), _TORCH_TO_CR[out.dtype], ldc, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), flags, _stream(stream)))


class Kv8Cache:
    """The 8-bit paged key/value cache: k [pages, Hkv, 64, D] and v [pages, Hkv, D, 64] uint8 (E4M3
    codes), k_scale and v_scale [pages, Hkv] fp32.  The caller deals out the pages: a page table
    [B, pages per sequence] int32 goes with every call."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4 or v.dim() != 4 or k.shape[2] != KV8_PAGE or v.shape != (*k.shape[:2], k.shape[3], KV8_PAGE):
            raise ValueError("expected k [pages, Hkv, 64, D] and v [pages, Hkv, D, 64]")
        for t, dtype, shape in ((k, torch.uint8, k.shape), (v, torch.uint8, v.shape),
                                (k_scale, torch.float32, k.shape[:2]), (v_scale, torch.float32, k.shape[:2])):
            if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
                raise ValueError("codes must be contiguous uint8, scales contiguous fp32 [pages, Hkv]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.Hkv, _, self.D = k.shape

    @classmethod
    def empty(cls, n_pages: int, Hkv: int, D: int, device="cuda") -> "Kv8Cache":
        codes = lambda *shape: torch.empty(n_pages, Hkv, *shape, dtype=torch.uint8, device=device)  # noqa: E731
        scales = lambda: torch.empty(n_pages, Hkv, dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(KV8_PAGE, D), codes(D, KV8_PAGE), scales(), scales())

    def _with_table(self, page_table: torch.Tensor) -> _Kv8:
        return _Kv8(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                    self.n_pages, page_table.data_ptr(), page_table.shape[1])


def _check_batch(cu_seqlens, kv_lens, page_table):
    B = kv_lens.numel()
    i32 = torch.int32
    if cu_seqlens.dtype is not i32 or kv_lens.dtype is not i32 or cu_seqlens.numel() != B + 1 \
            or not cu_seqlens.is_contiguous() or not kv_lens.is_contiguous():
        raise ValueError("cu_seqlens [B + 1] and kv_lens [B] must be contiguous int32 tensors")
    shape = page_table.shape
    if page_table.dtype is not i32 or len(shape) != 2 or shape[0] != B or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 tensor [B, pages per sequence]")
    return B


def cr_rope_append_kv8(qkv, cu_seqlens, kv_lens, max_new, Hq, q_weight, k_weight, eps, pos, freq, axis, q_out, cache,
                       page_table, flags=0, stream=None):
    B = _check_batch(cu_seqlens, kv_lens, page_table)
    D, Hkv = cache.D, cache.Hkv
    ld, width = _ld(qkv), Hq * D
    T, cols = qkv.shape
    if cols != width + 2 * Hkv * D:
        raise ValueError(f"qkv must hold {Hq} + 2 * {Hkv} heads of {D} elements a row")
    if q_out.dtype is not qkv.dtype or q_out.shape != (T, width):
        raise ValueError("q_out must be [T, Hq * D] of qkv's dtype")
    ld_pos = _ld(pos)
    n_pos, n_axes = pos.shape
    if pos.dtype is not torch.int32 or n_pos != T:
        raise ValueError("pos must be int32 [T, axes]")
    status = lib().cr_rope_append_kv8(
        qkv.data_ptr(), _TORCH_TO_CR.get(qkv.dtype, -1), ld, T, B, cu_seqlens.data_ptr(), kv_lens.data_ptr(), max_new,
        Hq, Hkv, D, _vector("q_weight", q_weight, D), _vector("k_weight", k_weight, D), eps, pos.data_ptr(),
        max(ld_pos, n_axes), n_axes, _vector("freq", freq, D // 2, torch.float64),
        _vector("axis", axis, D // 2, torch.int32), q_out.data_ptr(), max(_ld(q_out), width),
        cache._with_table(page_table), flags, _stream(stream))
    if status:
        raise CrError("cr_rope_append_kv8", status)


def cr_attn_kv8_workspace_bytes(T, B, max_q, max_kv, Hq, Hkv, D) -> int:
    return int(lib().cr_attn_kv8_workspace_bytes(T, B, max_q, max_kv, Hq, Hkv, D))


def cr_attn_kv8(q, cu_seqlens, kv_lens, max_q, max_kv, Hq, cache, page_table, sm_scale, out, workspace, flags=0,
                stream=None):
    B = _check_batch(cu_seqlens, kv_lens, page_table)
    ld_q, shape, D = _ld(q), q.shape, cache.D
    T, width = shape
    if width != Hq * D or out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("q and out must be [T, Hq * D] of one dtype")
    status = lib().cr_attn_kv8(
        q.data_ptr(), _TORCH_TO_CR.get(q.dtype, -1), max(ld_q, width), T, B, cu_seqlens.data_ptr(), kv_lens.data_ptr(),
        max_q, max_kv, Hq, cache.Hkv, D, cache._with_table(page_table), sm_scale, out.data_ptr(), max(_ld(out), width),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes, flags,
        _stream(stream))
    if status:
        raise CrError("cr_attn_kv8", status)


# ---------------------------------------------------------------- conveniences ----

def quant_act(x: torch.Tensor, K: int | None = None, swiglu: bool = False, flags: int = 0,
              pre_scale: torch.Tensor | None = None):
    """(x_s8 [M, K_pad] int8, x_scale [M] fp32) of X [M, K] or of SwiGLU(H [M, 2K]), with an
    optional [K] channel pre-scale."""
    if K is None:
        K = x.shape[1] // 2 if swiglu else x.shape[1]
    kp = padded_k(K)
    q = torch.empty(x.shape[0], kp, dtype=torch.int8, device=x.device)
    s = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    if pre_scale is not None:
        cr_quant_act_ex(x, K, swiglu, pre_scale, q, s, flags)
    else:
        (cr_quant_act_swiglu if swiglu else cr_quant_act)(x, K, q, s, flags)
    return q, s


def quant_act_rmsnorm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6,
                      residual: torch.Tensor | None = None, sum: torch.Tensor | None = None, flags: int = 0):
    """(x_s8 [M, K_pad] int8, x_scale [M] fp32, h) of the RMS norm of h = x + residual, the input
    of the INT8-activation GEMMs.  h [M, K] in x's type goes to `sum` (which may be x or
    residual: updated in place) or to a new tensor; None without a residual."""
    M, K = x.shape
    d = x.device
    q = torch.empty(M, (K + 255) // 256 * 256, dtype=torch.int8, device=d)
    s = torch.empty(M, dtype=torch.float32, device=d)
    if residual is not None and sum is None:
        n = 16 // x.element_size()                 # rows of 16-byte multiples
        sum = x.new_empty(M, K) if K % n == 0 else x.new_empty(M, (K + n - 1) // n * n)[:, :K]
    cr_quant_act_rmsnorm(x, residual, sum, weight, eps, K, q, s, flags)
    return q, s, sum


def prep_weight_nvfp4(w_fp4: torch.Tensor, w_sf: torch.Tensor, global_scale: torch.Tensor, K: int,
                      flags: int = 0):
    kp = padded_k(K)
    q = torch.empty(w_fp4.shape[0], kp, dtype=torch.int8, device=w_fp4.device)
    s = torch.empty(w_fp4.shape[0], dtype=torch.float32, device=w_fp4.device)
    cr_prep_weight_nvfp4(w_fp4, w_sf, global_scale, K, q, s, flags)
    return q, s


def gemm_s8_rowscale(a_s8, a_scale, b_s8, b_scale, out_dtype=torch.bfloat16, bias=None):
    c = torch.empty(a_s8.shape[0], b_s8.shape[0], dtype=out_dtype, device=a_s8.device)
    if bias is not None:
        cr_gemm_s8_rowscale_bias(a_s8, a_scale, b_s8, b_scale, bias, c)
    else:
        cr_gemm_s8_rowscale(a_s8, a_scale, b_s8, b_scale, c)
    return c


def linear_nvfp4(x, w_fp4, w_sf, global_scale, K, out_dtype=torch.bfloat16, swiglu=False, out=None,
                 max_tile_bytes=0, flags=0, aux_stream=None, workspace=None, pre_scale=None, bias=None):
    """y = x W^T (+ b) through the rotated S8 route (SwiGLU(x) W^T when swiglu); pre_scale
    multiplies the input channels before the rotation."""
    M, N = x.shape[0], w_fp4.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    need = cr_linear_nvfp4_workspace_bytes(M, N, K, max_tile_bytes)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    cr_linear_nvfp4(x, K, swiglu, w_fp4, w_sf, global_scale, out, workspace, max_tile_bytes, flags,
                    aux_stream=aux_stream, pre_scale=pre_scale, bias=bias)
    return out


def weight_amax_nvfp4(w_fp4: torch.Tensor, w_sf: torch.Tensor, global_scale: torch.Tensor, K: int,
                      flags: int = 0) -> torch.Tensor:
    """[N] fp32 row maxima of the rotated weight (input of gemm_nvfp4_fused)."""
    a = torch.empty(w_fp4.shape[0], dtype=torch.float32, device=w_fp4.device)
    cr_weight_amax_nvfp4(w_fp4, w_sf, global_scale, K, a, flags)
    return a


def gemm_nvfp4_fused(a_s8, a_scale, w_fp4, w_sf, global_scale, w_amax, K, out_dtype=torch.bfloat16,
                     bias=None, flags=0):
    c = torch.empty(a_s8.shape[0], w_fp4.shape[0], dtype=out_dtype, device=a_s8.device)
    cr_gemm_nvfp4_fused(a_s8, a_scale, w_fp4, w_sf, global_scale, w_amax, K, c, bias, flags)
    return c


def quant_weight_w4(w: torch.Tensor, K: int | None = None, flags: int = 0):
    """(packed 4-bit codes [N, K_pad / 2] uint8, scales [N] fp32) of a dense weight [N, K]."""
    if K is None:
        K = w.shape[1]
    kp = padded_k(K)
    q = torch.empty(w.shape[0], kp // 2, dtype=torch.uint8, device=w.device)
    s = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
    cr_quant_weight_w4(w, K, q, s, flags)
    return q, s


def linear_w4a8(x, w_s4, w_scale, K, out_dtype=torch.bfloat16, swiglu=False, bias=None, flags=0, out=None):
    """y = x W^T (+ b) through the W4A8 route against a prepared 4-bit weight."""
    M, N = x.shape[0], w_s4.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    ws = torch.empty(max(1, cr_linear_w4a8_workspace_bytes(M, K)), dtype=torch.uint8, device=x.device)
    cr_linear_w4a8(x, K, swiglu, w_s4, w_scale, out, ws, bias=bias, flags=flags)
    return out


def quant_act_w4(x: torch.Tensor, K: int | None = None, swiglu: bool = False, flags: int = 0):
    """(packed 4-bit codes [M, K_pad / 2] uint8, scales [M] fp32) of X [M, K] or of
    SwiGLU(H [M, 2K])."""
    if K is None:
        K = x.shape[1] // 2 if swiglu else x.shape[1]
    kp = padded_k(K)
    q = torch.empty(x.shape[0], kp // 2, dtype=torch.uint8, device=x.device)
    s = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    cr_quant_act_w4(x, K, swiglu, q, s, flags)
    return q, s


def linear_w4a4(x, w_s4, w_scale, K, out_dtype=torch.bfloat16, swiglu=False, bias=None, flags=0, out=None):
    """y = x W^T (+ b) through the W4A4 route against a prepared 4-bit weight."""
    M, N = x.shape[0], w_s4.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    ws = torch.empty(max(1, cr_linear_w4a4_workspace_bytes(M, K)), dtype=torch.uint8, device=x.device)
    cr_linear_w4a4(x, K, swiglu, w_s4, w_scale, out, ws, bias=bias, flags=flags)
    return out


def quant_weight_w4_e2m3(w: torch.Tensor, K: int | None = None, flags: int = 0):
    """(4-bit codes as E2M3 fields in quads of rows [ceil(N / 4), 3 K_pad] uint8, scales [N]
    fp32) of a dense weight; unused rows of the last quad are zero."""
    if K is None:
        K = w.shape[1]
    kp = padded_k(K)
    q = torch.zeros((w.shape[0] + 3) // 4, 3 * kp, dtype=torch.uint8, device=w.device)
    s = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
    cr_quant_weight_w4_e2m3(w, K, q, s, flags)
    return q, s


def quant_act_w4_e2m3(x: torch.Tensor, K: int | None = None, swiglu: bool = False, flags: int = 0):
    """(4-bit codes as E2M3 fields in quads of rows [ceil(M / 4), 3 K_pad] uint8, scales [M]
    fp32) of X or SwiGLU(H); unused rows of the last quad are zero."""
    if K is None:
        K = x.shape[1] // 2 if swiglu else x.shape[1]
    kp = padded_k(K)
    q = torch.zeros((x.shape[0] + 3) // 4, 3 * kp, dtype=torch.uint8, device=x.device)
    s = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    cr_quant_act_w4_e2m3(x, K, swiglu, q, s, flags)
    return q, s


def linear_w4a4_e2m3(x, w_f6, w_scale, K, out_dtype=torch.bfloat16, swiglu=False, bias=None, flags=0, out=None):
    """y = x W^T (+ b) through the W4A4 route on the 6-bit matrix cores."""
    M, N = x.shape[0], w_scale.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    ws = torch.empty(max(1, cr_linear_w4a4_e2m3_workspace_bytes(M, K)), dtype=torch.uint8, device=x.device)
    cr_linear_w4a4_e2m3(x, K, swiglu, w_f6, w_scale, out, ws, bias=bias, flags=flags)
    return out


def repack_w4_e2m3(w_s4: torch.Tensor, K_pad: int | None = None):
    """The E2M3 form [ceil(N / 4), 3 K_pad] uint8 of nibble-form 4-bit rows [N, K_pad / 2] (the
    row scales are unchanged); unused rows of the last quad are zero."""
    kp = 2 * w_s4.shape[1] if K_pad is None else K_pad
    out = torch.zeros((w_s4.shape[0] + 3) // 4, 3 * kp, dtype=torch.uint8, device=w_s4.device)
    cr_repack_w4_e2m3(w_s4, out, K_pad=kp)
    return out


def rope_table(D: int, sections=None, base: float = 10000.0, device="cuda"):
    """(freq [D/2] fp64, axis [D/2] int32) of a rotary embedding whose pairs are dealt to the
    position axes in runs of `sections` (default: one axis); pair i of an axis with n pairs turns
    by base^(-i/n) radians a position.  Pairs past the sections are left alone (frequency 0)."""
    sections = [D // 2] if sections is None else list(sections)
    if sum(sections) > D // 2 or not 1 <= len(sections) <= 4:
        raise ValueError("one to four sections of at most D/2 pairs in all")
    freq = [base ** (-i / n) for n in sections for i in range(n)]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    rest = D // 2 - len(freq)
    return (torch.tensor(freq + [0.0] * rest, dtype=torch.float64, device=device),
            torch.tensor(axis + [0] * rest, dtype=torch.int32, device=device))


def rope_append_kv8(qkv, cache: Kv8Cache, cu_seqlens, kv_lens, page_table, max_new: int, Hq: int, pos, freq, axis,
                    q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, out=None):
    """The rotated (and, with weights, per-head normed) queries [T, Hq * D] of the rows of a QKV
    projection; their keys and values go to the cache.  kv_lens counts the new tokens.  `out` may
    be qkv[:, : Hq * D]."""
    if out is None:
        out = qkv.new_empty(qkv.shape[0], Hq * cache.D)
    cr_rope_append_kv8(qkv, cu_seqlens, kv_lens, max_new, Hq, q_weight, k_weight, eps, pos, freq, axis, out, cache,
                       page_table, CR_FLAG_ROPE_INTERLEAVED if interleaved else 0)
    return out


def attn_kv8(q, cache: Kv8Cache, cu_seqlens, kv_lens, page_table, max_q: int, max_kv: int, Hq: int,
             sm_scale: float | None = None, causal: bool = True, out=None, workspace=None):
    """Attention of q [T, Hq * D] over the cached keys and values; sm_scale defaults to 1/sqrt(D)."""
    if out is None:
        out = q.new_empty(q.shape[0], Hq * cache.D)
    if workspace is None:
        need = cr_attn_kv8_workspace_bytes(q.shape[0], kv_lens.numel(), max_q, max_kv, Hq, cache.Hkv, cache.D)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    cr_attn_kv8(q, cu_seqlens, kv_lens, max_q, max_kv, Hq, cache, page_table,
                cache.D ** -0.5 if sm_scale is None else sm_scale, out, workspace, CR_FLAG_CAUSAL if causal else 0)
    return out
