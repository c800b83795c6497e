"""Python binding of libmigemm (the gfx950 dense matrix-multiply library).

Argument marshalling only: every step of the product runs in the library's HIP
kernels.  The functions named ``migemm_*`` mirror the C ABI in
``include/migemm.h`` one for one (integers and raw device pointers);
``gemm`` is a convenience wrapper over torch tensors that derives the sizes,
leading dimensions, pointers and the current stream, lends the workspace that
``migemm_workspace_size`` asks for (a torch allocation on the same stream) and
calls ``migemm_gemm_ws``.

The library is loaded on first use from this package's directory.  If it has
not been built, every call raises ``RuntimeError``: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libmigemm.so")

F32, F16, BF16, I8, I32 = 0, 1, 2, 3, 4
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_HIP, ERR_WORKSPACE = 0, 1, 2, 3, 4
NOALLOC_SCRATCH_BYTES = 64 << 20  # the allocation-free entry point's scratch per GPU
OP_N, OP_T = 0, 1
VARIANT_AUTO, NAIVE, LDS_TILED, REGTILE_VALU, REGTILE_MFMA, MFMA16, MFMA_I8 = -1, 0, 1, 2, 3, 4, 5

# Every symbol the header declares (checked by the CPU test suite).
EXPORTS = ("migemm_gemm", "migemm_gemm_variant", "migemm_gemm_ex", "migemm_gemm_ex_variant",
           "migemm_gemm_ws", "migemm_gemm_noalloc", "migemm_workspace_size", "migemm_describe",
           "migemm_describe_ex",
           "migemm_convert", "migemm_quantize_mx", "migemm_dequantize_mx", "migemm_gemm_mx",
           "migemm_mx_config_count", "migemm_mx_config_name",
           "migemm_linear_loss_workspace_size", "migemm_linear_ce_forward",
           "migemm_linear_ce_backward", "migemm_linear_kd_forward", "migemm_linear_kd_backward",
           "migemm_variant_count", "migemm_variant_name",
           "migemm_variant_supports", "migemm_config_count", "migemm_config_name",
           "migemm_select", "migemm_status_string", "migemm_last_hip_error", "migemm_version")

_lib = None


class MigemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = migemm_status_string(status)
        if status == ERR_HIP:
            msg += f" (hipError_t {migemm_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def lib():
    """The loaded library (ctypes.CDLL); raises RuntimeError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise RuntimeError(f"libmigemm.so is not built ({LIBRARY_PATH}); run "
                           "`python dense_gemm_16_amd/build.py` or __graft_entry__.build()")
    L = ctypes.CDLL(LIBRARY_PATH)
    i64, i32, vp, cp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_char_p
    L.migemm_gemm.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_gemm.restype = i32
    L.migemm_gemm_variant.argtypes = [i32, i32, i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_gemm_variant.restype = i32
    f32 = ctypes.c_float
    L.migemm_gemm_ex.argtypes = [i32, i32, i64, i64, i64, i32, vp, i64, vp, i64, f32, f32, i32,
                                 vp, i64, vp]
    L.migemm_gemm_ex.restype = i32
    L.migemm_gemm_ex_variant.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32, vp, i64, vp, i64,
                                         f32, f32, i32, vp, i64, vp]
    L.migemm_gemm_ex_variant.restype = i32
    L.migemm_gemm_ws.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32, vp, i64, vp, i64,
                                 f32, f32, i32, vp, i64, vp, i64, vp]
    L.migemm_gemm_ws.restype = i32
    L.migemm_gemm_noalloc.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32, vp, i64, vp, i64,
                                      f32, f32, i32, vp, i64, vp]
    L.migemm_gemm_noalloc.restype = i32
    L.migemm_workspace_size.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32, vp, i64, vp,
                                        i64, ctypes.POINTER(i64)]
    L.migemm_workspace_size.restype = i32
    L.migemm_describe.argtypes = [i64, i64, i64, i32, i64, i64, i64, cp, i32]
    L.migemm_describe.restype = i32
    L.migemm_describe_ex.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32, vp, i64, vp, i64,
                                     i32, i64, i64, cp, i32]
    L.migemm_describe_ex.restype = i32
    L.migemm_convert.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp]
    L.migemm_convert.restype = i32
    L.migemm_quantize_mx.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_quantize_mx.restype = i32
    L.migemm_dequantize_mx.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_dequantize_mx.restype = i32
    L.migemm_gemm_mx.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, f32, f32, i32,
                                 vp, i64, vp]
    L.migemm_gemm_mx.restype = i32
    L.migemm_mx_config_count.argtypes = []
    L.migemm_mx_config_count.restype = i32
    L.migemm_mx_config_name.argtypes = [i32]
    L.migemm_mx_config_name.restype = cp
    layer = [i64, i64, i64, i32, vp, i64, vp, i64]  # T, V, D, dtype, X, ldx, W, ldw
    kd = [i64, i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp, i64, f32]
    L.migemm_linear_loss_workspace_size.argtypes = [i32, i64, i64, i64, i64, i32, vp, i64, vp, i64,
                                                    ctypes.POINTER(i64)]
    L.migemm_linear_loss_workspace_size.restype = i32
    L.migemm_linear_ce_forward.argtypes = layer + [vp, i64, vp, vp, vp, i64, vp]
    L.migemm_linear_ce_forward.restype = i32
    L.migemm_linear_ce_backward.argtypes = layer + [vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_linear_ce_backward.restype = i32
    L.migemm_linear_kd_forward.argtypes = kd + [vp, vp, vp, i64, vp, i64, vp]
    L.migemm_linear_kd_forward.restype = i32
    L.migemm_linear_kd_backward.argtypes = kd + [vp, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp]
    L.migemm_linear_kd_backward.restype = i32
    L.migemm_variant_count.argtypes = []
    L.migemm_variant_count.restype = i32
    L.migemm_variant_name.argtypes = [i32]
    L.migemm_variant_name.restype = cp
    L.migemm_variant_supports.argtypes = [i32, i32]
    L.migemm_variant_supports.restype = i32
    L.migemm_config_count.argtypes = [i32]
    L.migemm_config_count.restype = i32
    L.migemm_config_name.argtypes = [i32, i32]
    L.migemm_config_name.restype = cp
    L.migemm_select.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i64,
                                ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.migemm_select.restype = i32
    L.migemm_status_string.argtypes = [i32]
    L.migemm_status_string.restype = cp
    L.migemm_last_hip_error.argtypes = []
    L.migemm_last_hip_error.restype = i32
    L.migemm_version.argtypes = []
    L.migemm_version.restype = i32
    _lib = L
    return L


# ---------------------------------------------------------------- C ABI mirror

def migemm_gemm(M, N, K, dtype, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return lib().migemm_gemm(M, N, K, dtype, A, lda, B, ldb, C, ldc, stream)


def migemm_gemm_variant(variant, config, M, N, K, dtype, A, lda, B, ldb, C, ldc,
                        stream=None) -> int:
    return lib().migemm_gemm_variant(variant, config, M, N, K, dtype, A, lda, B, ldb, C, ldc,
                                     stream)


def migemm_gemm_ex(op_a, op_b, M, N, K, dtype, A, lda, B, ldb, alpha, beta, c_dtype, C, ldc,
                   stream=None) -> int:
    return lib().migemm_gemm_ex(op_a, op_b, M, N, K, dtype, A, lda, B, ldb, alpha, beta,
                                c_dtype, C, ldc, stream)


def migemm_gemm_ex_variant(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb, alpha,
                           beta, c_dtype, C, ldc, stream=None) -> int:
    return lib().migemm_gemm_ex_variant(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B,
                                        ldb, alpha, beta, c_dtype, C, ldc, stream)


def migemm_gemm_ws(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb, alpha, beta,
                   c_dtype, C, ldc, workspace, workspace_bytes, stream=None) -> int:
    return lib().migemm_gemm_ws(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb,
                                alpha, beta, c_dtype, C, ldc, workspace, workspace_bytes, stream)


def migemm_gemm_noalloc(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb, alpha,
                        beta, c_dtype, C, ldc, stream=None) -> int:
    return lib().migemm_gemm_noalloc(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb,
                                     alpha, beta, c_dtype, C, ldc, stream)


def migemm_workspace_size(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb):
    """(status, bytes) of the workspace migemm_gemm_ws would use."""
    n = ctypes.c_int64(-1)
    st = lib().migemm_workspace_size(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb,
                                     ctypes.byref(n))
    return st, n.value


def _parse_description(text: str) -> dict:
    out = {}
    for item in text.split(";"):
        if "=" in item:
            k, v = item.split("=", 1)
            out[k] = int(v) if v.lstrip("-").isdigit() else v
    return out


def migemm_describe(M, N, K, dtype, lda, ldb, ldc, buflen=8192):
    """(status, text) describing what migemm_gemm would run."""
    buf = ctypes.create_string_buffer(buflen)
    st = lib().migemm_describe(M, N, K, dtype, lda, ldb, ldc, buf, buflen)
    return st, buf.value.decode()


def migemm_describe_ex(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb, c_dtype,
                       ldc, workspace_bytes, buflen=8192):
    """(status, text) describing what migemm_gemm_ws would run."""
    buf = ctypes.create_string_buffer(buflen)
    st = lib().migemm_describe_ex(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb,
                                  c_dtype, ldc, workspace_bytes, buf, buflen)
    return st, buf.value.decode()


def describe(*args, **kw) -> dict:
    """migemm_describe_ex's text parsed into a dict (integers where numeric)."""
    st, text = migemm_describe_ex(*args, **kw)
    if st != OK:
        raise MigemmError(st, "migemm_describe_ex")
    return _parse_description(text)


def migemm_convert(src_dtype, dst_dtype, rows, cols, src, lds, dst, ldd, stream=None) -> int:
    return lib().migemm_convert(src_dtype, dst_dtype, rows, cols, src, lds, dst, ldd, stream)


def migemm_quantize_mx(src_dtype, op, rows, cols, src, lds, data, ldd, scales, ldsc,
                       stream=None) -> int:
    return lib().migemm_quantize_mx(src_dtype, op, rows, cols, src, lds, data, ldd, scales, ldsc,
                                    stream)


def migemm_dequantize_mx(dst_dtype, rows, cols, data, ldd, scales, ldsc, dst, ld,
                         stream=None) -> int:
    return lib().migemm_dequantize_mx(dst_dtype, rows, cols, data, ldd, scales, ldsc, dst, ld,
                                      stream)


def migemm_gemm_mx(config, M, N, K, A, lda, a_scales, ldas, B, ldb, b_scales, ldbs, alpha, beta,
                   c_dtype, C, ldc, stream=None) -> int:
    return lib().migemm_gemm_mx(config, M, N, K, A, lda, a_scales, ldas, B, ldb, b_scales, ldbs,
                                alpha, beta, c_dtype, C, ldc, stream)


def migemm_mx_config_count() -> int:
    return lib().migemm_mx_config_count()


def migemm_mx_config_name(config: int) -> str | None:
    s = lib().migemm_mx_config_name(config)
    return s.decode() if s is not None else None


def migemm_linear_loss_workspace_size(backward, T, V, D, top, dtype, X, ldx, W, ldw):
    """(status, bytes) of the workspace a loss's pass needs."""
    n = ctypes.c_int64(-1)
    st = lib().migemm_linear_loss_workspace_size(backward, T, V, D, top, dtype, X, ldx, W, ldw,
                                                 ctypes.byref(n))
    return st, n.value


def migemm_linear_ce_forward(T, V, D, dtype, X, ldx, W, ldw, target, ignore_index, loss, lse,
                             workspace, workspace_bytes, stream=None) -> int:
    return lib().migemm_linear_ce_forward(T, V, D, dtype, X, ldx, W, ldw, target, ignore_index,
                                          loss, lse, workspace, workspace_bytes, stream)


def migemm_linear_ce_backward(T, V, D, dtype, X, ldx, W, ldw, target, ignore_index, lse, grad, dX,
                              lddx, dW, lddw, workspace, workspace_bytes, stream=None) -> int:
    return lib().migemm_linear_ce_backward(T, V, D, dtype, X, ldx, W, ldw, target, ignore_index,
                                           lse, grad, dX, lddx, dW, lddw, workspace,
                                           workspace_bytes, stream)


def migemm_linear_kd_forward(T, V, D, top, dtype, X, ldx, W, ldw, teacher_dtype, teacher, ldt,
                             index, ldi, temperature, loss, lse, student, lds, workspace,
                             workspace_bytes, stream=None) -> int:
    return lib().migemm_linear_kd_forward(T, V, D, top, dtype, X, ldx, W, ldw, teacher_dtype,
                                          teacher, ldt, index, ldi, temperature, loss, lse, student,
                                          lds, workspace, workspace_bytes, stream)


def migemm_linear_kd_backward(T, V, D, top, dtype, X, ldx, W, ldw, teacher_dtype, teacher, ldt,
                              index, ldi, temperature, lse, student, lds, grad, dX, lddx, dW, lddw,
                              workspace, workspace_bytes, stream=None) -> int:
    return lib().migemm_linear_kd_backward(T, V, D, top, dtype, X, ldx, W, ldw, teacher_dtype,
                                           teacher, ldt, index, ldi, temperature, lse, student, lds,
                                           grad, dX, lddx, dW, lddw, workspace, workspace_bytes,
                                           stream)


def migemm_variant_count() -> int:
    return lib().migemm_variant_count()


def migemm_variant_name(variant: int) -> str | None:
    s = lib().migemm_variant_name(variant)
    return s.decode() if s is not None else None


def migemm_variant_supports(variant: int, dtype: int) -> bool:
    return bool(lib().migemm_variant_supports(variant, dtype))


def migemm_config_count(variant: int) -> int:
    return lib().migemm_config_count(variant)


def migemm_config_name(variant: int, config: int) -> str | None:
    s = lib().migemm_config_name(variant, config)
    return s.decode() if s is not None else None


def migemm_select(M, N, K, dtype, A, lda, B, ldb, C, ldc):
    """(status, variant, config) that migemm_gemm would use."""
    v, c = ctypes.c_int(-9), ctypes.c_int(-9)
    st = lib().migemm_select(M, N, K, dtype, A, lda, B, ldb, C, ldc, ctypes.byref(v),
                             ctypes.byref(c))
    return st, v.value, c.value


def migemm_status_string(status: int) -> str:
    return lib().migemm_status_string(status).decode()


def migemm_last_hip_error() -> int:
    return lib().migemm_last_hip_error()


def migemm_version() -> int:
    return lib().migemm_version()


# ---------------------------------------------------------- torch convenience

_codes = {}


def _dtype_code(t) -> int:
    if not _codes:
        import torch
        _codes.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16,
                       torch.int8: I8, torch.int32: I32})
    code = _codes.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}; expected float32, float16, bfloat16, "
                         "int8 (operands) or int32 (output of an int8 product)")
    return code


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("operands must have unit stride along rows (row-major)")
    if t.shape[0] <= 1:
        return max(1, t.shape[1])
    return _apart(t.stride(0), t.shape[1])


def _apart(stride, n) -> int:
    """The leading dimension of rows of `n` elements that lie `stride` apart.  Packed
    rows of no elements have stride 0 or 1; rows that share their elements
    (``expand``) have stride 0 too, but no leading dimension says so."""
    if stride == 0 and n > 0:
        raise ValueError("rows that share memory (stride 0) are not supported; copy them "
                         "with contiguous()")
    return max(1, stride)


def _operand(t):
    """(op, ld) of a 2-D operand: row-major (unit column stride) is OP_N with
    ld = stride(0); a transposed view (unit row stride) is OP_T with ld = stride(1)."""
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    rows, cols = t.shape
    if cols <= 1 or t.stride(1) == 1:
        return OP_N, _apart(t.stride(0), cols) if rows > 1 else max(1, cols)
    if rows <= 1 or t.stride(0) == 1:
        return OP_T, _apart(t.stride(1), rows)  # (cols > 1 here)
    raise ValueError("operands must be row-major or transposed views of row-major storage")


def convert(src, dtype, out=None, *, stream=None):
    """``src`` (a 2-D CUDA tensor, float32/float16/bfloat16, unit column stride)
    converted to ``dtype`` on the GPU (round to nearest even when narrowing);
    ``out`` is allocated if not given.  Returns ``out`` without synchronising."""
    import torch
    if src.device.type != "cuda":
        raise ValueError("src must be on the GPU")
    rows, cols = src.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=src.device)
    elif out.dtype != dtype or tuple(out.shape) != (rows, cols):
        raise ValueError("out must have src's shape and the requested dtype")
    if stream is None:
        stream = torch.cuda.current_stream(src.device).cuda_stream
    st = migemm_convert(_dtype_code(src), _dtype_code(out), rows, cols, src.data_ptr() or None,
                        _ld(src), out.data_ptr() or None, _ld(out), stream)
    if st != OK:
        raise MigemmError(st, "migemm_convert")
    return out


def _check_device(name, t, device):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")


def workspace(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb, device):
    """A torch byte tensor on `device` large enough for migemm_gemm_ws with these
    arguments (None when the call needs none)."""
    import torch
    st, n = migemm_workspace_size(variant, config, op_a, op_b, M, N, K, dtype, A, lda, B, ldb)
    if st != OK:
        raise MigemmError(st, "migemm_workspace_size")
    if n == 0:
        return None
    # torch's allocations are 512-byte aligned, beyond the 256 the library asks
    return torch.empty(n, dtype=torch.uint8, device=device)


def gemm(a, b, out=None, *, alpha: float = 1.0, beta: float = 0.0, out_dtype=None,
         variant: int = VARIANT_AUTO, config: int = -1, stream=None):
    """out = alpha * (A x B) + beta * out on the GPU for torch tensors.

    ``a`` (M x K) and ``b`` (K x N) are CUDA tensors of the same dtype
    (float32, float16, bfloat16, or int8 with an int32 ``out``) on one device,
    each row-major or a transposed view of row-major storage (``x.t()``, or a
    column-major tensor), passed as stored: no copy is made.  ``out`` (M x N,
    row-major, on the same device) may be float32, float16 or bfloat16; if not
    given it is allocated with ``out_dtype`` (default float32), which beta == 0
    requires.  The workspace the call asks for (migemm_workspace_size) is
    allocated by torch on the same stream and lent to migemm_gemm_ws.  Runs on
    ``stream`` (default: torch's current stream) and returns ``out`` without
    synchronising.
    """
    import torch
    device = a.device
    _check_device("a", a, device)
    _check_device("b", b, device)
    if a.dtype != b.dtype:
        raise ValueError(f"dtype mismatch: {a.dtype} vs {b.dtype}")
    dt = _dtype_code(a)
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(a.shape)} x {tuple(b.shape)}")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an existing out")
        default = torch.int32 if a.dtype == torch.int8 else torch.float32
        out = torch.empty((M, N), dtype=out_dtype or default, device=device)
    else:
        _check_device("out", out, device)
        if tuple(out.shape) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must have shape (M, N) (and out_dtype, if given)")
    cd = _dtype_code(out)
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    pa, pb, pc = a.data_ptr() or None, b.data_ptr() or None, out.data_ptr() or None
    (op_a, lda), (op_b, ldb) = _operand(a), _operand(b)
    ws = workspace(variant, config, op_a, op_b, M, N, K, dt, pa, lda, pb, ldb, device)
    if ws is not None and stream != torch.cuda.current_stream(device).cuda_stream:
        # the block goes back to torch's pool when `ws` dies; keep it from being
        # reused before the work queued on `stream` has finished
        ws.record_stream(torch.cuda.ExternalStream(stream, device=device))
    st = migemm_gemm_ws(variant, config, op_a, op_b, M, N, K, dt, pa, lda, pb, ldb,
                        float(alpha), float(beta), cd, pc, _ld(out),
                        ws.data_ptr() if ws is not None else None,
                        ws.numel() if ws is not None else 0, stream)
    if st != OK:
        raise MigemmError(st, "migemm_gemm_ws")
    return out


_torch = None


def _load_torch():
    """torch, kept in a global: an import statement costs a short call 0.2 us."""
    global _torch
    import torch
    _torch = torch
    return torch


# ---------------------------------------------------------------------- MXFP4

class MxMatrix(NamedTuple):
    """A matrix in microscaled 4-bit floating point (the format is described in
    ``include/migemm.h``).

    ``data``: uint8 CUDA tensor, rows x (16 bytes or more per block of 32
    elements); ``scales``: uint8, rows x (1 byte or more per block); both with unit
    column stride, 16-byte aligned rows and row strides a multiple of 16.
    ``cols``: elements per row (not bytes)."""
    data: "torch.Tensor"  # noqa: F821
    scales: "torch.Tensor"  # noqa: F821
    cols: int

    @property
    def shape(self):
        return self.data.shape[0], self.cols

    @property
    def device(self):
        return self.data.device


def _mx_operand(name, m, device):
    """(data pointer, ldd, scales pointer, ldsc) of an MxMatrix, checked."""
    torch = _torch or _load_torch()
    data, scales, cols = m
    blocks, u8 = (cols + 31) // 32, torch.uint8
    if not (data.is_cuda and scales.is_cuda and data.device == device == scales.device):
        _check_device(f"{name}.data", data, device)
        _check_device(f"{name}.scales", scales, device)
    if not (data.dtype is u8 and scales.dtype is u8 and data.dim() == 2 == scales.dim()):
        raise ValueError(f"{name} must hold uint8 matrices (got {data.dtype}, {tuple(data.shape)} "
                         f"and {scales.dtype}, {tuple(scales.shape)})")
    (rows, width), (srows, swidth) = data.shape, scales.shape
    (ldd, unit), (ldsc, sunit) = data.stride(), scales.stride()
    if srows != rows or width < 16 * blocks or swidth < blocks or (
            width > 1 and unit != 1) or (swidth > 1 and sunit != 1):
        raise ValueError(f"{name} must hold data and scales of as many rows, of at least "
                         f"{16 * blocks} and {blocks} bytes, with unit column stride (got "
                         f"{tuple(data.shape)} and {tuple(scales.shape)}, strides {data.stride()} "
                         f"and {scales.stride()})")
    if rows <= 1:
        ldd, ldsc = width, swidth
    elif ldd != width or ldsc != swidth:
        # a row occupies its whole stride, the last one too
        for t, ld in ((data, ldd), (scales, ldsc)):
            if t.untyped_storage().nbytes() - t.storage_offset() < rows * ld:
                raise ValueError(f"{name}: the storage ends inside the last row's stride")
    return data.data_ptr() or None, ldd, scales.data_ptr() or None, ldsc


class _Here:
    """The context of a call on torch's current device: nothing to change."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_here = _Here()


def _device_of(device):
    """A context that makes `device` torch's current one, where it is not."""
    torch = _torch or _load_torch()
    return _here if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _stream_of(stream, device):
    """(stream handle, whether it is another one than torch's current stream)."""
    torch = _torch or _load_torch()
    current = torch._C._cuda_getCurrentRawStream(device.index)
    return (current, False) if stream is None else (stream, stream != current)


def _run_on(stream, device, *tensors):
    """For a call on another stream than torch's current one: `stream` waits for what
    is queued on the current stream (new tensors may reuse memory that work there
    still reads), and the tensors, None apart, are kept from being reused before the
    work queued on `stream` has finished."""
    torch = _torch or _load_torch()
    s = torch.cuda.ExternalStream(stream, device=device)
    s.wait_stream(torch.cuda.current_stream(device))
    for t in tensors:
        if t is not None:
            t.record_stream(s)


def quantize_mx(src, *, out=None, stream=None):
    """``src`` (a 2-D CUDA tensor, float32/float16/bfloat16, row-major or a
    transposed view of row-major storage, read as stored) quantised to MXFP4 along
    its rows, as an ``MxMatrix`` (``out``, if given).  Quantise a weight stored K x N
    for ``gemm_mx`` as ``quantize_mx(w.t())``.  Does not synchronise."""
    torch = _torch or _load_torch()
    device = src.device
    _check_device("src", src, device)
    op, lds = _operand(src)
    rows, cols = src.shape
    blocks = (cols + 31) // 32
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        if out is None:
            ldd, ldsc = 16 * max(blocks, 1), max(16, (blocks + 15) // 16 * 16)
            out = MxMatrix(torch.empty((rows, ldd), dtype=torch.uint8, device=device),
                           torch.empty((rows, ldsc), dtype=torch.uint8, device=device), cols)
            data, scales = out.data.data_ptr() or None, out.scales.data_ptr() or None
        else:
            if out.shape != (rows, cols):
                raise ValueError("out must have src's shape")
            data, ldd, scales, ldsc = _mx_operand("out", out, device)
        if other:
            _run_on(stream, device, src, out.data, out.scales)
        st = lib().migemm_quantize_mx(_dtype_code(src), op, rows, cols, src.data_ptr() or None, lds,
                                data, ldd, scales, ldsc, stream)
        if st != OK:
            raise MigemmError(st, "migemm_quantize_mx")
    return out


def dequantize_mx(m, dtype, out=None, *, stream=None):
    """The values of an ``MxMatrix`` as a row-major ``dtype`` tensor (float32,
    float16 or bfloat16; ``out``, if given).  Does not synchronise."""
    torch = _torch or _load_torch()
    device = m.device
    rows, cols = m.shape
    data, ldd, scales, ldsc = _mx_operand("m", m, device)
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        if out is None:
            out = torch.empty((rows, cols), dtype=dtype, device=device)
        else:
            _check_device("out", out, device)
            if out.dtype != dtype or tuple(out.shape) != (rows, cols):
                raise ValueError("out must have m's shape and the requested dtype")
        if other:
            _run_on(stream, device, m.data, m.scales, out)
        st = lib().migemm_dequantize_mx(_dtype_code(out), rows, cols, data, ldd, scales, ldsc,
                                  out.data_ptr() or None, _ld(out), stream)
        if st != OK:
            raise MigemmError(st, "migemm_dequantize_mx")
    return out


def gemm_mx(a, b, out=None, *, alpha: float = 1.0, beta: float = 0.0, out_dtype=None,
            config: int = -1, stream=None):
    """out = alpha * (A x B^T) + beta * out for two ``MxMatrix`` operands: ``a`` is
    M x K, ``b`` N x K (quantised along k).  ``out`` (M x N, row-major, float32,
    float16 or bfloat16) is allocated with ``out_dtype`` (default float32) if not
    given, which beta == 0 requires.  Does not synchronise."""
    torch = _torch or _load_torch()
    device = a.device
    (M, K), (N, K2) = a.shape, b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {a.shape} x {b.shape} transposed")
    pa, lda, psa, ldsa = _mx_operand("a", a, device)
    pb, ldb, psb, ldsb = _mx_operand("b", b, device)
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        if out is None:
            if beta != 0.0:
                raise ValueError("beta != 0 needs an existing out")
            out = torch.empty((M, N), dtype=out_dtype or torch.float32, device=device)
        else:
            _check_device("out", out, device)
            if tuple(out.shape) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
                raise ValueError("out must have shape (M, N) (and out_dtype, if given)")
        if other:
            _run_on(stream, device, a.data, a.scales, b.data, b.scales, out)
        st = lib().migemm_gemm_mx(config, M, N, (K + 31) // 32 * 32, pa, lda, psa, ldsa, pb, ldb, psb,
                            ldsb, float(alpha), float(beta), _dtype_code(out),
                            out.data_ptr() or None, _ld(out), stream)
        if st != OK:
            raise MigemmError(st, "migemm_gemm_mx")
    return out


# ------------------------------------------------------- output-layer losses

def _layer(x, w):
    """(device, T, V, D, dtype code, (x pointer, ldx, w pointer, ldw)) of an output
    layer's operands, checked."""
    device = x.device
    if not (x.is_cuda and w.device == device):
        _check_device("x", x, device)
        _check_device("w", w, device)
    if x.dtype is not w.dtype:
        raise ValueError(f"dtype mismatch: {x.dtype} vs {w.dtype}")
    dt, ldx, ldw = _dtype_code(x), _ld(x), _ld(w)
    (T, D), (V, D2) = x.shape, w.shape
    if D != D2:
        raise ValueError(f"x has rows of {D}, w of {D2}")
    return device, T, V, D, dt, (x.data_ptr() or None, ldx, w.data_ptr() or None, ldw)


def _row_vector(name, t, device, dtype, rows):
    """Pointer of a contiguous vector of one value per row, checked."""
    if t.device != device:
        _check_device(name, t, device)
    if t.dtype is not dtype or t.shape != (rows,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {rows} (got {t.dtype}, "
                         f"{tuple(t.shape)}, strides {t.stride()})")
    return t.data_ptr() or None


def _row_gradient(grad, device, rows):
    """`grad` as one float32 per row: a number, a 0-d tensor or a vector."""
    torch = _torch or _load_torch()
    if not isinstance(grad, torch.Tensor):
        return torch.full((rows,), float(grad), dtype=torch.float32, device=device)
    _check_device("grad", grad, device)
    if grad.dtype is torch.float32 and grad.shape == (rows,) and grad.is_contiguous():
        return grad
    if grad.dim() > 1 or (grad.dim() == 1 and grad.shape[0] != rows):
        raise ValueError(f"grad must be a number or a vector of {rows}")
    return grad.to(torch.float32).expand(rows).contiguous()


def _gradient(name, wanted, given, like):
    """The tensor a gradient is written to: `given` (checked), a new one, or None."""
    torch = _torch or _load_torch()
    if given is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format) if wanted else None
    _check_device(name, given, like.device)
    if given.dtype != like.dtype or given.shape != like.shape:
        raise ValueError(f"{name} must have the shape and dtype of what it is the gradient of")
    return given


def _loss_workspace(backward, T, V, D, top, dt, ptrs, device):
    torch = _torch or _load_torch()
    st, n = migemm_linear_loss_workspace_size(backward, T, V, D, top, dt, *ptrs)
    if st != OK:
        raise MigemmError(st, "migemm_linear_loss_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _teacher(logits, index, T, device):
    """(dtype code, pointer, ldt, index pointer, ldi, entries per row), checked."""
    torch = _torch or _load_torch()
    _check_device("teacher_logits", logits, device)
    _check_device("teacher_index", index, device)
    if logits.dim() != 2 or logits.shape[0] != T or index.shape != logits.shape:
        raise ValueError(f"teacher_logits and teacher_index must both be {T} x entries")
    if index.dtype != torch.int64:
        raise ValueError("teacher_index must be int64")
    return (_dtype_code(logits), logits.data_ptr() or None, _ld(logits), index.data_ptr() or None,
            _ld(index)), logits.shape[1]


def linear_cross_entropy(x, w, target, *, ignore_index: int = -100, stream=None):
    """(loss, lse): per row of ``x`` (T x D) the softmax cross entropy of the logits
    ``x @ w.t()`` (``w``: V x D) against ``target`` (int64, T), and the logits'
    log-sum-exp (float64), which ``linear_cross_entropy_backward`` takes.  The
    logits are never stored.  Rows whose target is ``ignore_index`` have loss 0; a
    target outside the vocabulary gives NaN.  ``x`` and ``w``: CUDA tensors of one
    dtype (float32, float16, bfloat16), unit column stride.  Runs on ``stream``
    (default: torch's current stream; another one first waits for it) without
    synchronising.  Autograd does not see the call: the gradients come from the
    backward function."""
    torch = _torch or _load_torch()
    device, T, V, D, dt, ptrs = _layer(x, w)
    pt = _row_vector("target", target, device, torch.int64, T)
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        loss = torch.empty(T, dtype=torch.float32, device=device)
        lse = torch.empty(T, dtype=torch.float64, device=device)
        ws = _loss_workspace(0, T, V, D, 0, dt, ptrs, device)
        if other:
            _run_on(stream, device, x, w, target, loss, lse, ws)
        st = lib().migemm_linear_ce_forward(T, V, D, dt, *ptrs, pt, ignore_index, loss.data_ptr() or None,
                                      lse.data_ptr() or None, ws.data_ptr() or None, ws.numel(),
                                      stream)
    if st != OK:
        raise MigemmError(st, "migemm_linear_ce_forward")
    return loss, lse


def linear_cross_entropy_backward(x, w, target, lse, grad, *, ignore_index: int = -100, dx=None,
                                  dw=None, need_dx: bool = True, need_dw: bool = True,
                                  stream=None):
    """(dx, dw): the gradients of ``linear_cross_entropy``'s losses to ``x`` and ``w``
    in their dtype, for the upstream gradient ``grad`` of each row's loss (a number
    or a vector of T).  ``dx`` and ``dw`` are written into if given; one that is
    neither given nor needed is None."""
    torch = _torch or _load_torch()
    device, T, V, D, dt, ptrs = _layer(x, w)
    pt = _row_vector("target", target, device, torch.int64, T)
    pl = _row_vector("lse", lse, device, torch.float64, T)
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        grad = _row_gradient(grad, device, T)
        dx, dw = _gradient("dx", need_dx, dx, x), _gradient("dw", need_dw, dw, w)
        ws = _loss_workspace(1, T, V, D, 0, dt, ptrs, device)
        if other:
            _run_on(stream, device, x, w, target, lse, grad, dx, dw, ws)
        st = lib().migemm_linear_ce_backward(
            T, V, D, dt, *ptrs, pt, ignore_index, pl, grad.data_ptr() or None, *_out_matrix(dx),
            *_out_matrix(dw), ws.data_ptr() or None, ws.numel(), stream)
    if st != OK:
        raise MigemmError(st, "migemm_linear_ce_backward")
    return dx, dw


def _out_matrix(t):
    return (None, 1) if t is None else (t.data_ptr() or None, _ld(t))


def linear_distillation(x, w, teacher_logits, teacher_index, *, temperature: float = 1.0,
                        stream=None):
    """(loss, lse, student): per row of ``x`` (T x D) temperature^2 times the
    divergence of the student's softmax (logits ``x @ w.t()``, ``w``: V x D, never
    stored) from the softmax of the teacher's top logits (``teacher_logits``, T x
    entries, at the vocabulary indices ``teacher_index``, int64; a negative index
    marks an entry that is not held), both at ``temperature``.  ``lse`` and
    ``student`` (the student's logits at the indices) are what
    ``linear_distillation_backward`` takes.  ``lse`` is float64, the others float32.  A row that holds no entry
    has loss 0.  Otherwise as ``linear_cross_entropy``."""
    torch = _torch or _load_torch()
    device, T, V, D, dt, ptrs = _layer(x, w)
    teacher, top = _teacher(teacher_logits, teacher_index, T, device)
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        loss = torch.empty(T, dtype=torch.float32, device=device)
        lse = torch.empty(T, dtype=torch.float64, device=device)
        student = torch.empty((T, top), dtype=torch.float32, device=device)
        ws = _loss_workspace(0, T, V, D, top, dt, ptrs, device)
        if other:
            _run_on(stream, device, x, w, teacher_logits, teacher_index, loss, lse, student, ws)
        st = lib().migemm_linear_kd_forward(
            T, V, D, top, dt, *ptrs, *teacher, float(temperature), loss.data_ptr() or None,
            lse.data_ptr() or None, student.data_ptr() or None, max(1, top), ws.data_ptr() or None,
            ws.numel(), stream)
    if st != OK:
        raise MigemmError(st, "migemm_linear_kd_forward")
    return loss, lse, student


def linear_distillation_backward(x, w, teacher_logits, teacher_index, lse, student, grad, *,
                                 temperature: float = 1.0, dx=None, dw=None, need_dx: bool = True,
                                 need_dw: bool = True, stream=None):
    """(dx, dw): the gradients of ``linear_distillation``'s losses to ``x`` and ``w``;
    arguments as in ``linear_cross_entropy_backward``."""
    torch = _torch or _load_torch()
    device, T, V, D, dt, ptrs = _layer(x, w)
    teacher, top = _teacher(teacher_logits, teacher_index, T, device)
    pl = _row_vector("lse", lse, device, torch.float64, T)
    _check_device("student", student, device)
    if student.dtype != torch.float32 or tuple(student.shape) != (T, top):
        raise ValueError(f"student must be float32, {T} x {top}")
    with _device_of(device):
        stream, other = _stream_of(stream, device)
        grad = _row_gradient(grad, device, T)
        dx, dw = _gradient("dx", need_dx, dx, x), _gradient("dw", need_dw, dw, w)
        ws = _loss_workspace(1, T, V, D, top, dt, ptrs, device)
        if other:
            _run_on(stream, device, x, w, teacher_logits, teacher_index, lse, student, grad, dx,
                    dw, ws)
        st = lib().migemm_linear_kd_backward(
            T, V, D, top, dt, *ptrs, *teacher, float(temperature), pl, student.data_ptr() or None,
            _ld(student), grad.data_ptr() or None, *_out_matrix(dx), *_out_matrix(dw),
            ws.data_ptr() or None, ws.numel(), stream)
    if st != OK:
        raise MigemmError(st, "migemm_linear_kd_backward")
    return dx, dw
