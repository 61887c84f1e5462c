"""Python binding of libck.so (include/ck.h): argument marshalling only.

Every function takes CUDA tensors, passes their device pointers, sizes and the
current CUDA stream to the C entry point of the same name, and raises
``CKError`` on a non-OK status. All computation happens in the library's CUDA
kernels; there is no CPU fallback: importing this module without a built
libck.so raises ImportError.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libck.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m bit_quantized_linear_rotate_b200.build` "
        "(the ConvRot kernels have no CPU fallback)")

lib = ctypes.CDLL(LIB_PATH)

CK_OK, CK_ERR_INVALID_ARG, CK_ERR_UNSUPPORTED, CK_ERR_CUDA, CK_ERR_TIMEOUT = range(5)
CK_BF16, CK_FP16, CK_FP32 = 0, 1, 2
STATUS_NAMES = {0: "CK_OK", 1: "CK_ERR_INVALID_ARG", 2: "CK_ERR_UNSUPPORTED", 3: "CK_ERR_CUDA",
                4: "CK_ERR_TIMEOUT"}

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float

# name -> argument types (restype is ck_status = int unless listed below)
SIGNATURES = {
    "ck_rotate_quant_rowwise": [_p, _int, _i64, _i64, _i64, _int, _int, _p, _p, _p],
    "ck_rotate_quant_rowwise_i8": [_p, _int, _i64, _i64, _i64, _int, _int, _p, _p, _p],
    "ck_rotate_quant_rowwise_r": [_p, _int, _i64, _i64, _i64, _int, _p, _int, _p, _p, _p],
    "ck_rotate_quant_rowwise_scaled": [_p, _int, _i64, _i64, _i64, _int, _int, _f32, _p, _p, _p],
    "ck_gemm_w4a4": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p],
    "ck_gemm_w4a8": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p],
    "ck_unpack_int4": [_p, _i64, _i64, _p, _p],
    "ck_gemm_s8": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p],
    "ck_gemm_s8_i32": [_p, _p, _i64, _i64, _i64, _p, _p],
    "ck_linear_w4a4_workspace_bytes": [_i64, _i64],
    "ck_linear_w4a4": [_p, _int, _i64, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p, ctypes.c_size_t, _p],
    "ck_linear_w4a4_quantize": [_p, _int, _i64, _i64, _i64, _int, _p, ctypes.c_size_t, _p],
    "ck_linear_w4a4_matmul": [_i64, _i64, _i64, _p, _p, _p, _p, _p, ctypes.c_size_t, _p],
    "ck_linear_w4a4_scaled": [_p, _int, _i64, _i64, _i64, _i64, _int, _f32, _p, _p, _p, _p, _p, ctypes.c_size_t,
                              _p],
    "ck_linear_w4a4_static": [_p, _int, _i64, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p],
    "ck_linear_w4a8_workspace_bytes": [_i64, _i64],
    "ck_linear_w4a8": [_p, _int, _i64, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p, ctypes.c_size_t, _p],
    "ck_linear_w4a4_predecoded": [_p, _int, _i64, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p, ctypes.c_size_t,
                                  _p],
    "ck_gemv_w4a8": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p],
    "ck_gemv_w4a8_tc": [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p],
    "ck_gemv_awq_w4a16": [_p, _int, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p, _p],
    "ck_moe_route": [_p, _int, _i64, _i64, _int, _int, _p, _p, _p],
    "ck_moe_awq_w4a16_workspace_bytes": [_i64, _int, _i64, _i64],
    "ck_moe_awq_w4a16": [_p, _int, _i64, _i64, _i64, _i64, _i64, _int, _p, _int, _int, _int, _p, _p, _p, _p, _p, _p,
                         _p, _p, ctypes.c_size_t, _p],
    "ck_moe_experts_awq_w4a16": [_p, _int, _i64, _i64, _i64, _i64, _i64, _int, _p, _p, _int, _p, _p, _p, _p, _p, _p,
                                 _p, _p, ctypes.c_size_t, _p],
    "ck_lora_add_workspace_bytes": [_i64, _i64],
    "ck_lora_add": [_p, _int, _p, _int, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p,
                    ctypes.c_size_t, _p],
    "ck_gemm_w4a4_i32": [_p, _p, _i64, _i64, _i64, _p, _p],
    "ck_gemm_w4a8_i32": [_p, _p, _i64, _i64, _i64, _p, _p],
    "ck_device_error_check": [_p],
    "ck_selftest_bounded_wait": [_i64, _p],
    "ck_last_error": [],
    "ck_version": [],
}
_RESTYPES = {"ck_linear_w4a4_workspace_bytes": ctypes.c_size_t, "ck_linear_w4a8_workspace_bytes": ctypes.c_size_t,
             "ck_moe_awq_w4a16_workspace_bytes": ctypes.c_size_t, "ck_lora_add_workspace_bytes": ctypes.c_size_t,
             "ck_last_error": ctypes.c_char_p, "ck_version": ctypes.c_char_p}

for _name, _args in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _RESTYPES.get(_name, ctypes.c_int)


class CKError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.ck_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")


def _check(status: int, where: str) -> None:
    if status != CK_OK:
        raise CKError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None, device=None):
    """The stream handle for a call on `device`: the given stream (which must belong to that
    device) or that device's current stream."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt) -> int:
    if dt == torch.bfloat16:
        return CK_BF16
    if dt == torch.float16:
        return CK_FP16
    raise TypeError(f"unsupported dtype {dt} (bf16 or fp16)")


_BYTES = (torch.uint8, torch.int8)      # codes and packed nibbles: either view of the same bytes
_HALF = (torch.bfloat16, torch.float16)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_I32 = (torch.int32,)


def _types(where: str, **named) -> None:
    """TypeError unless each named tensor (None is skipped) has one of its allowed dtypes.

    The C entry points see raw bytes, so a tensor of the wrong dtype would be
    read as garbage rather than rejected."""
    for name, (t, allowed) in named.items():
        if t is not None and t.dtype not in allowed:
            want = " or ".join(str(a).replace("torch.", "") for a in allowed)
            raise TypeError(f"{where}: {name} must be {want}, got {str(t.dtype).replace('torch.', '')}")


def _cuda(*ts):
    """The one CUDA device all given tensors (None is skipped) live on; ValueError otherwise.

    The library launches on the calling thread's current device, so every call below runs with
    this device made current (``torch.cuda.device``)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"all tensors must be on one device ({dev} and {t.device} given)")
    return dev


def _rows(x):
    """(M, K, ldx) of a tensor whose last dim is contiguous; leading dims are flattened."""
    if x.stride(-1) != 1:
        raise ValueError("the last dimension must be contiguous")
    K = x.shape[-1]
    if x.dim() == 1:
        return 1, K, K, x
    x2 = x if x.dim() == 2 else x.reshape(-1, K)
    return x2.shape[0], K, x2.stride(0), x2


def version() -> str:
    return lib.ck_version().decode()


def last_error() -> str:
    return lib.ck_last_error().decode()


def _call(dev, name: str, *args, stream=None) -> None:
    """Calls the C entry point `name` with `dev` current and that device's stream appended."""
    with torch.cuda.device(dev):
        _check(getattr(lib, name)(*args, _stream(stream, dev)), name)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _codes_out(x, K, bits, q_out, scale_out):
    lead = tuple(x.shape[:-1])
    if q_out is None:
        q_out = torch.empty(lead + ((K // 2,) if bits == 4 else (K,)), device=x.device,
                            dtype=torch.uint8 if bits == 4 else torch.int8)
    if scale_out is None:
        scale_out = torch.empty(lead, device=x.device, dtype=torch.float32)
    return q_out, scale_out


def rotate_quant_rowwise(x, group_size: int, bits: int, q_out=None, scale_out=None, stream=None):
    """Returns (q, scale): q packed int4 (..., K/2) uint8 for bits=4, int8 (..., K) for bits=8."""
    _types("rotate_quant_rowwise", x=(x, _HALF), q_out=(q_out, _BYTES), scale_out=(scale_out, _F32))
    _cuda(x)
    M, K, ldx, x2 = _rows(x)
    q_out, scale_out = _codes_out(x, K, bits, q_out, scale_out)
    dev = _cuda(x, q_out, scale_out)
    _call(dev, "ck_rotate_quant_rowwise", _ptr(x2), _dtype_code(x.dtype), M, K, ldx, group_size, bits,
          _ptr(q_out), _ptr(scale_out), stream=stream)
    return q_out, scale_out


def rotate_quant_rowwise_i8(x, group_size: int, bits: int, q_out=None, scale_out=None, stream=None):
    """Returns (q, scale) with the codes stored one per byte: q (..., K) int8 for bits 4 or 8."""
    _types("rotate_quant_rowwise_i8", x=(x, _HALF), q_out=(q_out, _BYTES), scale_out=(scale_out, _F32))
    _cuda(x)
    M, K, ldx, x2 = _rows(x)
    q_out, scale_out = _codes_out(x, K, 8, q_out, scale_out)
    dev = _cuda(x, q_out, scale_out)
    _call(dev, "ck_rotate_quant_rowwise_i8", _ptr(x2), _dtype_code(x.dtype), M, K, ldx, group_size, bits,
          _ptr(q_out), _ptr(scale_out), stream=stream)
    return q_out, scale_out


def rotate_quant_rowwise_r(x, R, bits: int, q_out=None, scale_out=None, stream=None):
    """Rotation by a general (G, G) float32 matrix R (y_g = x_g @ R), then rowwise quantization.

    Returns (q, s) in the formats of rotate_quant_rowwise: bits=4 packed (..., K/2) uint8, bits=8
    (..., K) int8; s (...) float32.
    """
    _types("rotate_quant_rowwise_r", x=(x, _HALF), q_out=(q_out, _BYTES), scale_out=(scale_out, _F32))
    _cuda(x, R)
    if R.dtype != torch.float32 or R.dim() != 2 or R.shape[0] != R.shape[1] or not R.is_contiguous():
        raise ValueError("R must be a contiguous square float32 matrix")
    M, K, ldx, x2 = _rows(x)
    q_out, scale_out = _codes_out(x, K, bits, q_out, scale_out)
    dev = _cuda(x, R, q_out, scale_out)
    _call(dev, "ck_rotate_quant_rowwise_r", _ptr(x2), _dtype_code(x.dtype), M, K, ldx, R.shape[0], _ptr(R), bits,
          _ptr(q_out), _ptr(scale_out), stream=stream)
    return q_out, scale_out


def rotate_quant_rowwise_scaled(x, group_size: int, bits: int, input_scale: float, q_out=None,
                                scale_out=None, stream=None):
    """rotate_quant_rowwise of input_scale * x (a finite tensor-wise scale >= 0); same formats."""
    _types("rotate_quant_rowwise_scaled", x=(x, _HALF), q_out=(q_out, _BYTES), scale_out=(scale_out, _F32))
    _cuda(x)
    M, K, ldx, x2 = _rows(x)
    q_out, scale_out = _codes_out(x, K, bits, q_out, scale_out)
    dev = _cuda(x, q_out, scale_out)
    _call(dev, "ck_rotate_quant_rowwise_scaled", _ptr(x2), _dtype_code(x.dtype), M, K, ldx, group_size, bits,
          float(input_scale), _ptr(q_out), _ptr(scale_out), stream=stream)
    return q_out, scale_out


def unpack_int4(packed, out=None, stream=None):
    """(R, C/2) packed int4 -> (R, C) int8 with value u - 8."""
    _types("unpack_int4", packed=(packed, _BYTES), out=(out, _BYTES))
    _cuda(packed)
    R, Ch = packed.shape
    if out is None:
        out = torch.empty((R, 2 * Ch), device=packed.device, dtype=torch.int8)
    dev = _cuda(packed, out)
    _call(dev, "ck_unpack_int4", _ptr(packed), R, 2 * Ch, _ptr(out), stream=stream)
    return out


def _mn_out(a, M, N, out, dtype=torch.bfloat16):
    return torch.empty((M, N), device=a.device, dtype=dtype) if out is None else out


def gemm_w4a8(qa, a_scale, w_packed, w_scale, bias=None, out=None, stream=None):
    """int8 activation codes (M, K) x packed int4 weights (N, K/2) -> bf16 (M, N)."""
    _types("gemm_w4a8", qa=(qa, _BYTES), a_scale=(a_scale, _F32), w_packed=(w_packed, _BYTES),
           w_scale=(w_scale, _BF16), bias=(bias, _BF16), out=(out, _BF16))
    _cuda(qa, a_scale, w_packed, w_scale, bias, out)
    M, K = qa.shape
    N = w_packed.shape[0]
    out = _mn_out(qa, M, N, out)
    _call(_cuda(qa, out), "ck_gemm_w4a8", _ptr(qa), _ptr(a_scale), M, K, N, _ptr(w_packed), _ptr(w_scale),
          _ptr(bias), _ptr(out), stream=stream)
    return out


def gemm_s8(qa, a_scale, w8, w_scale, bias=None, out=None, stream=None):
    _types("gemm_s8", qa=(qa, _BYTES), a_scale=(a_scale, _F32), w8=(w8, _BYTES), w_scale=(w_scale, _BF16),
           bias=(bias, _BF16), out=(out, _BF16))
    _cuda(qa, a_scale, w8, w_scale, bias, out)
    M, K = qa.shape
    N = w8.shape[0]
    out = _mn_out(qa, M, N, out)
    _call(_cuda(qa, out), "ck_gemm_s8", _ptr(qa), _ptr(a_scale), M, K, N, _ptr(w8), _ptr(w_scale), _ptr(bias),
          _ptr(out), stream=stream)
    return out


def gemm_s8_i32(qa, w8, out=None, stream=None):
    _types("gemm_s8_i32", qa=(qa, _BYTES), w8=(w8, _BYTES), out=(out, _I32))
    _cuda(qa, w8, out)
    M, K = qa.shape
    N = w8.shape[0]
    out = _mn_out(qa, M, N, out, torch.int32)
    _call(_cuda(qa, out), "ck_gemm_s8_i32", _ptr(qa), _ptr(w8), M, K, N, _ptr(out), stream=stream)
    return out


def gemm_w4a4(qa_packed, a_scale, w_packed, w_scale, bias=None, out=None, stream=None):
    _types("gemm_w4a4", qa_packed=(qa_packed, _BYTES), a_scale=(a_scale, _F32), w_packed=(w_packed, _BYTES),
           w_scale=(w_scale, _BF16), bias=(bias, _BF16), out=(out, _BF16))
    _cuda(qa_packed, a_scale, w_packed, w_scale, bias, out)
    M, Kh = qa_packed.shape
    N = w_packed.shape[0]
    out = _mn_out(qa_packed, M, N, out)
    _call(_cuda(qa_packed, out), "ck_gemm_w4a4", _ptr(qa_packed), _ptr(a_scale), M, 2 * Kh, N, _ptr(w_packed),
          _ptr(w_scale), _ptr(bias), _ptr(out), stream=stream)
    return out


def linear_w4a4_workspace_bytes(M: int, K: int) -> int:
    return int(lib.ck_linear_w4a4_workspace_bytes(M, K))


def linear_w4a8_workspace_bytes(M: int, K: int) -> int:
    return int(lib.ck_linear_w4a8_workspace_bytes(M, K))


def _linear(name, x, w, w_scale, group_size, bias, workspace, out, stream, ws_fn, *extra, w_name="w_packed"):
    """Shared marshalling of the one-shot linears: (x, weights, scales) -> y (..., N) bf16."""
    _types(name, x=(x, _HALF), **{w_name: (w, _BYTES)}, w_scale=(w_scale, _BF16), bias=(bias, _BF16),
           out=(out, _BF16), workspace=(workspace, _BYTES))
    _cuda(x, w, w_scale, bias, workspace, out)
    M, K, ldx, x2 = _rows(x)
    N = w.shape[0]
    if workspace is None:
        workspace = torch.empty(ws_fn(M, K), device=x.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty(tuple(x.shape[:-1]) + (N,), device=x.device, dtype=torch.bfloat16)
    dev = _cuda(x, workspace, out)
    _call(dev, "ck_" + name, _ptr(x2), _dtype_code(x.dtype), M, K, N, ldx, group_size, *extra, _ptr(w),
          _ptr(w_scale), _ptr(bias), _ptr(out), _ptr(workspace), _nbytes(workspace), stream=stream)
    return out


def linear_w4a4(x, w_packed, w_scale, group_size: int, bias=None, workspace=None, out=None,
                stream=None):
    """ConvRot W4A4 linear: y (..., N) bf16 from x (..., K) bf16/fp16 and packed (N, K/2) weights."""
    return _linear("linear_w4a4", x, w_packed, w_scale, group_size, bias, workspace, out, stream,
                   linear_w4a4_workspace_bytes)


def linear_w4a8(x, w_packed, w_scale, group_size: int, bias=None, workspace=None, out=None,
                stream=None):
    """ConvRot W4A8 linear: x rotated and quantized to int8 codes, times packed (N, K/2) int4 weights."""
    return _linear("linear_w4a8", x, w_packed, w_scale, group_size, bias, workspace, out, stream,
                   linear_w4a8_workspace_bytes)


def linear_w4a4_predecoded(x, w_s8, w_scale, group_size: int, bias=None, workspace=None, out=None,
                           stream=None):
    """linear_w4a4 with the weights already unpacked to int8 (N, K) by unpack_int4 (same results)."""
    return _linear("linear_w4a4_predecoded", x, w_s8, w_scale, group_size, bias, workspace, out, stream,
                   linear_w4a4_workspace_bytes, w_name="w_s8")


def linear_w4a4_scaled(x, w_packed, w_scale, group_size: int, input_scale: float, bias=None, workspace=None,
                       out=None, stream=None):
    """linear_w4a4 of input_scale * x (a finite tensor-wise scale >= 0); the output is not rescaled."""
    return _linear("linear_w4a4_scaled", x, w_packed, w_scale, group_size, bias, workspace, out, stream,
                   linear_w4a4_workspace_bytes, ctypes.c_float(float(input_scale)))


# Size of the library's built-in scratch for linear_w4a4_static (CK_LINEAR_STATIC_SCRATCH_BYTES).
LINEAR_STATIC_SCRATCH_BYTES = 32 * 1024 * 1024


def linear_w4a4_static(x, w_packed, w_scale, group_size: int, bias=None, out=None, stream=None):
    """linear_w4a4 without a workspace argument: the library uses its own fixed per-device scratch.

    Same results as linear_w4a4. Calls on one device share that scratch, so calls that may run
    at the same time on the GPU (different streams, several threads) must not be mixed. The call
    runs with x's device current: the scratch it uses is that device's.
    """
    _types("linear_w4a4_static", x=(x, _HALF), w_packed=(w_packed, _BYTES), w_scale=(w_scale, _BF16),
           bias=(bias, _BF16), out=(out, _BF16))
    _cuda(x, w_packed, w_scale, bias, out)
    M, K, ldx, x2 = _rows(x)
    N = w_packed.shape[0]
    if out is None:
        out = torch.empty(tuple(x.shape[:-1]) + (N,), device=x.device, dtype=torch.bfloat16)
    _call(_cuda(x, out), "ck_linear_w4a4_static", _ptr(x2), _dtype_code(x.dtype), M, K, N, ldx, group_size,
          _ptr(w_packed), _ptr(w_scale), _ptr(bias), _ptr(out), stream=stream)
    return out


def linear_w4a4_quantize(x, group_size: int, workspace, stream=None):
    """Phase 1 of linear_w4a4: rotate + quantize x into `workspace` (opaque)."""
    _types("linear_w4a4_quantize", x=(x, _HALF), workspace=(workspace, _BYTES))
    dev = _cuda(x, workspace)
    M, K, ldx, x2 = _rows(x)
    _call(dev, "ck_linear_w4a4_quantize", _ptr(x2), _dtype_code(x.dtype), M, K, ldx, group_size, _ptr(workspace),
          _nbytes(workspace), stream=stream)
    return workspace


def linear_w4a4_matmul(M: int, K: int, w_packed, w_scale, workspace, bias=None, out=None, stream=None):
    """Phase 2 of linear_w4a4: GEMM of the workspace codes with the packed weights -> y (M, N) bf16."""
    _types("linear_w4a4_matmul", w_packed=(w_packed, _BYTES), w_scale=(w_scale, _BF16), bias=(bias, _BF16),
           out=(out, _BF16), workspace=(workspace, _BYTES))
    _cuda(w_packed, w_scale, workspace, bias, out)
    N = w_packed.shape[0]
    out = _mn_out(w_packed, M, N, out)
    _call(_cuda(w_packed, workspace, out), "ck_linear_w4a4_matmul", M, K, N, _ptr(w_packed), _ptr(w_scale),
          _ptr(bias), _ptr(out), _ptr(workspace), _nbytes(workspace), stream=stream)
    return out


def _gemv_w4a8(name, xq, x_scale, w_packed, w_scale, bias, out, stream):
    _types(name, xq=(xq, _BYTES), x_scale=(x_scale, _F32), w_packed=(w_packed, _BYTES),
           w_scale=(w_scale, _BF16), bias=(bias, _BF16), out=(out, _BF16))
    _cuda(xq, x_scale, w_packed, w_scale, bias, out)
    M, K = xq.shape
    N = w_packed.shape[0]
    out = _mn_out(xq, M, N, out)
    _call(_cuda(xq, out), "ck_" + name, _ptr(xq), _ptr(x_scale), M, K, N, _ptr(w_packed), _ptr(w_scale),
          _ptr(bias), _ptr(out), stream=stream)
    return out


def gemv_w4a8(xq, x_scale, w_packed, w_scale, bias=None, out=None, stream=None):
    return _gemv_w4a8("gemv_w4a8", xq, x_scale, w_packed, w_scale, bias, out, stream)


def gemv_w4a8_tc(xq, x_scale, w_packed, w_scale, bias=None, out=None, stream=None):
    """gemv_w4a8 on the tcgen05 tensor cores (the same results bit for bit; an alternative path)."""
    return _gemv_w4a8("gemv_w4a8_tc", xq, x_scale, w_packed, w_scale, bias, out, stream)


def gemv_awq_w4a16(x, qweight, wscales, wzeros, bias=None, group_size: int = 64, out=None, stream=None):
    """``ck.gemv_awq_w4a16(x, qdata, wscales, wzeros, bias=, group_size=)``."""
    same = (x.dtype,) if x.dtype in _HALF else _HALF
    _types("gemv_awq_w4a16", x=(x, _HALF), qweight=(qweight, _BYTES), wscales=(wscales, same),
           wzeros=(wzeros, same), bias=(bias, same), out=(out, same))
    _cuda(x, qweight, wscales, wzeros, bias, out)
    M, K = x.shape
    N = qweight.shape[0]
    out = _mn_out(x, M, N, out, x.dtype)
    _call(_cuda(x, out), "ck_gemv_awq_w4a16", _ptr(x), _dtype_code(x.dtype), M, K, N, group_size, _ptr(qweight),
          _ptr(wscales), _ptr(wzeros), _ptr(bias), _ptr(out), stream=stream)
    return out


# ------------------------------------------ weights chosen for each token
#
# These calls are short (some 5 us on the device), so their checks are one expression over cheap
# attributes; only where it fails does a slower function find out what is wrong and say so (or that the
# call is merely less usual).

_moe_bytes = functools.lru_cache(maxsize=1024)(lib.ck_moe_awq_w4a16_workspace_bytes)
_lora_bytes = functools.lru_cache(maxsize=1024)(lib.ck_lora_add_workspace_bytes)

_LOGITS = (torch.bfloat16, torch.float16, torch.float32)
_f32t, _i32t, _bf16t = torch.float32, torch.int32, torch.bfloat16
_byte_like = frozenset(_BYTES)


def _empty(like, shape, dtype, stream):
    """A tensor for the call's own use or its result, from the pool of the stream that the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _shape(where: str, **named) -> None:
    """ValueError unless each named tensor (None is skipped) is contiguous and has its shape."""
    for name, (t, shape) in named.items():
        if t is not None and (tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{where}: {name} must be a contiguous tensor of shape {shape}, got {tuple(t.shape)}"
                             f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _matrix(where: str, name: str, t, rows, cols) -> None:
    """ValueError unless t is (rows, cols) with a contiguous last dimension."""
    if tuple(t.shape) != (rows, cols) or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{where}: {name} must be ({rows}, {cols}) with contiguous rows, got {tuple(t.shape)} with "
                         f"strides {t.stride()}")


def _on(dev: int, *ts) -> bool:
    """Whether all given tensors (None is skipped) live on CUDA device `dev`."""
    for t in ts:
        if t is not None and t.get_device() != dev:
            return False
    return dev >= 0


def _run(fn, name: str, dev: int, stream, *args) -> None:
    """_call for a C function at hand and a device index."""
    if stream is None and torch._C._cuda_getDevice() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        device = torch.device("cuda", dev)
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream, device))
    if status != CK_OK:
        raise CKError(status, name)


def _no_route(logits, top_k, weights_out, ids_out):
    """Raises what is wrong with moe_route's arguments."""
    _types("moe_route", logits=(logits, _LOGITS), weights_out=(weights_out, _F32), ids_out=(ids_out, _I32))
    if logits.dim() != 2:
        raise ValueError(f"moe_route: logits must be (T, E), got {tuple(logits.shape)}")
    T, E = logits.shape
    _shape("moe_route", logits=(logits, (T, E)), weights_out=(weights_out, (T, top_k)), ids_out=(ids_out, (T, top_k)))
    _cuda(logits, weights_out, ids_out)


def moe_route(logits, top_k: int, renormalize: bool = True, weights_out=None, ids_out=None, stream=None):
    """The top_k largest of each row of logits (T, E): (weights (T, top_k) float32, ids (T, top_k) int32).

    weights are softmax shares among the chosen (renormalize) or among all E experts; ties go to the
    lowest index; a -inf or NaN logit is never chosen, and a slot left over has id -1 and weight 0."""
    top_k = int(top_k)
    dev = logits.get_device()
    if not (logits.dtype in _LOGITS and logits.dim() == 2 and logits.is_contiguous() and dev >= 0
            and weights_out is None and ids_out is None):
        _no_route(logits, top_k, weights_out, ids_out)
    T, E = logits.shape
    k = max(top_k, 0)
    weights = _empty(logits, (T, k), _f32t, stream) if weights_out is None else weights_out
    ids = _empty(logits, (T, k), _i32t, stream) if ids_out is None else ids_out
    _run(lib.ck_moe_route, "ck_moe_route", dev, stream, logits.data_ptr(), _LOGITS.index(logits.dtype), T, E, top_k,
         1 if renormalize else 0, weights.data_ptr(), ids.data_ptr())
    return weights, ids


def moe_awq_w4a16_workspace_bytes(T: int, top_k: int, K: int, I: int) -> int:
    return int(lib.ck_moe_awq_w4a16_workspace_bytes(T, top_k, K, I))


def _no_moe(name, x, given, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z, G, workspace, out):
    """Raises what is wrong with a mixture-of-experts call's arguments (its choice apart)."""
    same = (x.dtype,) if x.dtype in _HALF else _HALF
    _types(name, x=(x, _HALF), gate_up_q=(gate_up_q, _BYTES), gate_up_s=(gate_up_s, same), gate_up_z=(gate_up_z, same),
           down_q=(down_q, _BYTES), down_s=(down_s, same), down_z=(down_z, same), out=(out, same),
           workspace=(workspace, _BYTES))
    if x.dim() != 2 or gate_up_q.dim() != 3 or gate_up_q.shape[1] % 2:
        raise ValueError(f"{name}: x must be (T, K) and gate_up_q (E, 2 I, K / 2), got {tuple(x.shape)} and "
                         f"{tuple(gate_up_q.shape)}")
    T, K = x.shape
    E, I = gate_up_q.shape[0], gate_up_q.shape[1] // 2
    _matrix(name, "x", x, T, K)
    if G > 0:
        _shape(name, gate_up_q=(gate_up_q, (E, 2 * I, K // 2)), gate_up_s=(gate_up_s, (E, K // G, 2 * I)),
               gate_up_z=(gate_up_z, (E, K // G, 2 * I)), down_q=(down_q, (E, K, I // 2)),
               down_s=(down_s, (E, I // G, K)), down_z=(down_z, (E, I // G, K)), out=(out, (T, K)))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be contiguous")
    _cuda(x, *given, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z, workspace, out)


def _moe(fn, name, x, given, choice, top_k, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z, group_size,
         workspace, out, stream):
    """Shared marshalling of the mixture-of-experts calls; `given` are the tensors of the choice, `choice`
    the C arguments between the group size and the weights."""
    G = int(group_size)
    dt = x.dtype
    dev = x.get_device()
    try:
        (T, K), (E, rows, half), (Ed, Kd, Ih) = x.shape, gate_up_q.shape, down_q.shape
        I = rows >> 1
        fine = (G > 0 and half == K >> 1 and rows == 2 * I and Ed == E and Kd == K and Ih == I >> 1
                and gate_up_s.shape == (E, K // G, rows) and gate_up_z.shape == gate_up_s.shape
                and down_s.shape == (E, I // G, K) and down_z.shape == down_s.shape and dt in _HALF
                and gate_up_s.dtype == dt and gate_up_z.dtype == dt and down_s.dtype == dt and down_z.dtype == dt
                and gate_up_q.dtype in _byte_like and down_q.dtype in _byte_like and gate_up_q.is_contiguous()
                and gate_up_s.is_contiguous() and gate_up_z.is_contiguous() and down_q.is_contiguous()
                and down_s.is_contiguous() and down_z.is_contiguous() and x.is_contiguous()
                and workspace is None and out is None
                and _on(dev, *given, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z))
    except ValueError:                            # another number of dimensions
        fine = False
    if not fine:
        _no_moe(name, x, given, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z, G, workspace, out)
        (T, K), (E, rows) = x.shape, gate_up_q.shape[:2]
        I = rows >> 1
    if workspace is None:
        workspace = _empty(x, (_moe_bytes(T, top_k, K, I),), torch.uint8, stream)
    if out is None:
        out = torch.empty_like(x) if fine and stream is None else _empty(x, (T, K), dt, stream)
    _run(fn, name, dev, stream, x.data_ptr(), 0 if dt == _bf16t else 1, T, K, I, E, x.stride(0) if T > 1 else K, G,
         *choice, gate_up_q.data_ptr(), gate_up_s.data_ptr(), gate_up_z.data_ptr(), down_q.data_ptr(),
         down_s.data_ptr(), down_z.data_ptr(), out.data_ptr(), workspace.data_ptr(), _nbytes(workspace))
    return out


def moe_awq_w4a16(x, logits, top_k: int, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z,
                  group_size: int = 64, renormalize: bool = True, workspace=None, out=None, stream=None):
    """A mixture-of-experts layer for up to 64 tokens: each row of x (T, K) goes through the top_k experts of
    its logits (T, E) as moe_route chooses them, out = sum of weight * (silu(x Wgate^T) * (x Wup^T)) Wdown^T.

    The experts are AWQ W4A16: gate_up_q (E, 2 I, K/2) packed bytes, the gate rows first, with scales and
    zeros (E, K/G, 2 I); down_q (E, K, I/2) with scales and zeros (E, I/G, K), all in x's dtype."""
    name = "moe_awq_w4a16"
    top_k = int(top_k)
    if not (logits.dtype in _LOGITS and logits.is_contiguous() and logits.dim() == 2
            and logits.shape[0] == x.shape[0] and logits.shape[1] == gate_up_q.shape[0]):
        _types(name, logits=(logits, _LOGITS))
        _shape(name, logits=(logits, (x.shape[0], gate_up_q.shape[0])))
    choice = (logits.data_ptr(), _LOGITS.index(logits.dtype), top_k, 1 if renormalize else 0)
    return _moe(lib.ck_moe_awq_w4a16, name, x, (logits,), choice, top_k, gate_up_q, gate_up_s, gate_up_z, down_q,
                down_s, down_z, group_size, workspace, out, stream)


def moe_experts_awq_w4a16(x, ids, weights, gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z,
                          group_size: int = 64, workspace=None, out=None, stream=None):
    """moe_awq_w4a16 with the choice given: ids (T, top_k) int32 and weights (T, top_k) float32, used as they
    are. A slot whose id is outside [0, E) is empty; an expert named twice counts with both weights."""
    name = "moe_experts_awq_w4a16"
    if not (ids.dtype == _i32t and weights.dtype == _f32t and ids.dim() == 2 and ids.shape[0] == x.shape[0]
            and weights.shape == ids.shape and ids.is_contiguous() and weights.is_contiguous()):
        _types(name, ids=(ids, _I32), weights=(weights, _F32))
        if ids.dim() != 2:
            raise ValueError(f"{name}: ids must be (T, top_k), got {tuple(ids.shape)}")
        _shape(name, ids=(ids, (x.shape[0], ids.shape[1])), weights=(weights, (x.shape[0], ids.shape[1])))
    k = ids.shape[1]
    return _moe(lib.ck_moe_experts_awq_w4a16, name, x, (ids, weights), (ids.data_ptr(), weights.data_ptr(), k), k,
                gate_up_q, gate_up_s, gate_up_z, down_q, down_s, down_z, group_size, workspace, out, stream)


def lora_add_workspace_bytes(M: int, L: int) -> int:
    return int(lib.ck_lora_add_workspace_bytes(M, L))


def _no_lora(y, x, lora_a, lora_b, ids, scales, workspace, out):
    """Raises what is wrong with lora_add's arguments."""
    same = (x.dtype,) if x.dtype in _HALF else _HALF
    _types("lora_add", y=(y, same + _BF16), x=(x, _HALF), lora_a=(lora_a, same), lora_b=(lora_b, same), ids=(ids, _I32),
           scales=(scales, _F32), out=(out, (y.dtype,)), workspace=(workspace, _BYTES))
    if x.dim() != 2 or lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("lora_add: x must be (M, K), lora_a (L, R, K) and lora_b (L, N, R)")
    (M, K), (L, R) = x.shape, lora_a.shape[:2]
    N = lora_b.shape[1]
    _matrix("lora_add", "x", x, M, K)
    _matrix("lora_add", "y", y, M, N)
    if out is not None:
        _matrix("lora_add", "out", out, M, N)
    _shape("lora_add", lora_a=(lora_a, (L, R, K)), lora_b=(lora_b, (L, N, R)), ids=(ids, (M,)), scales=(scales, (L,)))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("lora_add: workspace must be contiguous")
    _cuda(y, x, lora_a, lora_b, ids, scales, workspace, out)


def lora_add(y, x, lora_a, lora_b, ids, scales=None, workspace=None, out=None, stream=None):
    """out[m] = y[m] + scales[a] * (x[m] A[a]^T) B[a]^T with a = ids[m]; out[m] = y[m] where a is no adapter.

    y (M, N) bf16 or x's dtype is a projection's output, x (M, K) its input; lora_a (L, R, K) and lora_b
    (L, N, R) are the adapters, ids (M,) int32 (-1: none), scales (L,) float32. `out` may be y: in place."""
    dt, ydt = x.dtype, y.dtype
    dev = x.get_device()
    try:
        (M, K), (L, R, Ka), (Lb, N, Rb), (My, Ny), (Mi,) = x.shape, lora_a.shape, lora_b.shape, y.shape, ids.shape
        fine = (Ka == K and Lb == L and Rb == R and My == M and Ny == N and Mi == M and dt in _HALF
                and lora_a.dtype == dt and lora_b.dtype == dt and (ydt == dt or ydt == _bf16t) and ids.dtype == _i32t
                and x.is_contiguous() and y.is_contiguous() and lora_a.is_contiguous() and lora_b.is_contiguous()
                and ids.is_contiguous() and workspace is None and (out is None or out is y) and dev >= 0
                and y.get_device() == dev and lora_a.get_device() == dev and lora_b.get_device() == dev
                and ids.get_device() == dev
                and (scales is None or (scales.dtype == _f32t and scales.shape == (L,) and scales.is_contiguous()
                                        and scales.get_device() == dev)))
    except ValueError:                            # another number of dimensions
        fine = False
    if not fine:
        _no_lora(y, x, lora_a, lora_b, ids, scales, workspace, out)
        (M, K), (L, N, R) = x.shape, lora_b.shape
    if out is None:
        out = torch.empty_like(y) if fine and stream is None else _empty(y, (M, N), ydt, stream)
    if workspace is None:
        need = _lora_bytes(M, L)
        if need:
            workspace = _empty(x, (need,), torch.uint8, stream)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), _nbytes(workspace))
    one = M <= 1                                  # the stride of a single row is its length, whatever the tensor says
    _run(lib.ck_lora_add, "ck_lora_add", dev, stream, y.data_ptr(), 0 if ydt == _bf16t else 1, x.data_ptr(),
         0 if dt == _bf16t else 1, M, K, N, R, L, K if one else x.stride(0), N if one else y.stride(0),
         N if one else out.stride(0), lora_a.data_ptr(), lora_b.data_ptr(), ids.data_ptr(),
         None if scales is None else scales.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    return out


def gemm_w4a4_i32(qa_packed, w_packed, out=None, stream=None):
    _types("gemm_w4a4_i32", qa_packed=(qa_packed, _BYTES), w_packed=(w_packed, _BYTES), out=(out, _I32))
    _cuda(qa_packed, w_packed, out)
    M, Kh = qa_packed.shape
    N = w_packed.shape[0]
    out = _mn_out(qa_packed, M, N, out, torch.int32)
    _call(_cuda(qa_packed, out), "ck_gemm_w4a4_i32", _ptr(qa_packed), _ptr(w_packed), M, 2 * Kh, N, _ptr(out),
          stream=stream)
    return out


def gemm_w4a8_i32(qa, w_packed, out=None, stream=None):
    _types("gemm_w4a8_i32", qa=(qa, _BYTES), w_packed=(w_packed, _BYTES), out=(out, _I32))
    _cuda(qa, w_packed, out)
    M, K = qa.shape
    N = w_packed.shape[0]
    out = _mn_out(qa, M, N, out, torch.int32)
    _call(_cuda(qa, out), "ck_gemm_w4a8_i32", _ptr(qa), _ptr(w_packed), M, K, N, _ptr(out), stream=stream)
    return out


def device_error_check(stream=None) -> None:
    """Synchronises the stream and raises CKError(CK_ERR_TIMEOUT) if a bounded wait gave up."""
    _check(lib.ck_device_error_check(_stream(stream)), "ck_device_error_check")


def selftest_bounded_wait(timeout_ns: int, stream=None) -> None:
    _check(lib.ck_selftest_bounded_wait(int(timeout_ns), _stream(stream)), "ck_selftest_bounded_wait")
