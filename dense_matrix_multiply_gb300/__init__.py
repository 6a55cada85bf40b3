"""Python binding of the GB300 dense GEMM library (libgemm_gb300.so).

Argument marshalling only: every step of C = A·B runs in the library's CUDA
kernels.  The C entry points are exposed under the same names and take either
torch CUDA tensors (their data pointers are passed, and the library is pointed
at torch's current stream first) or raw device addresses as integers.

There is no CPU path.  If the shared library has not been built, or the device
is not a GB300, calls raise instead of computing anything elsewhere.
"""

from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

LIB_PATH = _build.LIB

GEMM_OK = 0
STATUS_NAMES = {
    0: "GEMM_OK",
    1: "GEMM_ERR_INVALID_VALUE",
    2: "GEMM_ERR_ALIAS",
    3: "GEMM_ERR_UNSUPPORTED_DEVICE",
    4: "GEMM_ERR_CUDA",
    5: "GEMM_ERR_TIMEOUT",
}

# Every symbol include/gemm.h declares, with its ctypes signature.
_VP, _I = ctypes.c_void_p, ctypes.c_int
SIGNATURES = {
    "gemm_f32_rm": ([_VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_f16_cm": ([_VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_bf16_rm": ([_VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_bf16_rm_noalloc": ([_VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_bf16_rm_silu_mul": ([_VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_ex": ([_I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _VP, ctypes.c_int64, ctypes.c_int64,
                 _VP, ctypes.c_int64, ctypes.c_int64, ctypes.c_float, _VP, ctypes.c_int64, ctypes.c_int64,
                 _I], _I),
    "gemm_quantize_rows_e4m3": ([_VP, _VP, _VP, _I, _I], _I),
    "gemm_e4m3_rowscale": ([_VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_e4m3_rowscale_fused": ([_VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_fp4_code_bytes": ([_I, _I], ctypes.c_int64),
    "gemm_fp4_scale_bytes": ([_I, _I, _I], ctypes.c_int64),
    "gemm_fp4_quantize": ([_I, _I, _VP, ctypes.c_int64, _VP, _VP, _VP, _I, _I], _I),
    "gemm_fp4_dequantize": ([_I, _I, _VP, _VP, _VP, _VP, ctypes.c_int64, _I, _I], _I),
    "gemm_fp4": ([_I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int64, _I, _I, _I], _I),
    "gemm_fp4_linear": ([_I, _I, _VP, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, ctypes.c_int64, _I, _I, _I], _I),
    "gemm_gated": ([_I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_gated_backward": ([_I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_rms_norm": ([_I, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _I, _I], _I),
    "gemm_rms_norm_e4m3": ([_I, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _I, _I], _I),
    "gemm_rms_norm_backward": ([_I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I], _I),
    "gemm_cross_entropy": ([_I, _VP, _VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_cross_entropy_backward": ([_I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I], _I),
    "gemm_orthogonalize": ([_I, _VP, ctypes.c_int64, _VP, ctypes.c_int64, _I, ctypes.c_float, ctypes.c_float,
                            ctypes.c_float, _I, _I], _I),
    "gemm_set_stream": ([_VP], _I),
    "gemm_get_stream": ([], _VP),
    "gemm_synchronize": ([], _I),
    "gemm_status_string": ([_I], ctypes.c_char_p),
    "gemm_last_kernel": ([], ctypes.c_char_p),
    "gemm_kernel_launches": ([], ctypes.c_ulonglong),
    "gemm_last_error": ([], ctypes.c_char_p),
    "gemm_force_kernel": ([ctypes.c_char_p], _I),
}

_lock = threading.Lock()
_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS_NAMES.get(status, status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


def ensure_built() -> str:
    """Compiles the library if it is missing or older than its sources."""
    return _build.build()


def load():
    """The loaded shared library (ctypes.CDLL).  Raises if it was never built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA extension missing: {LIB_PATH} has not been built "
                    "(run dense_matrix_multiply_gb300.ensure_built() or __graft_entry__.build())")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def _addr(x) -> int:
    if isinstance(x, int):
        return x
    if x is None:
        return 0
    return x.data_ptr()


_raw_stream = _raw_device = None


def _point_at(lib, device: int) -> None:
    """Points the library at torch's current stream of a device.  That has to be the current
    device, where the library launches; a call refused for it leaves the stream as it was."""
    global _raw_stream, _raw_device
    if _raw_stream is None:
        import torch
        _raw_device = torch._C._cuda_getDevice
        _raw_stream = torch._C._cuda_getCurrentRawStream
    if device != _raw_device():
        raise ValueError(f"tensors on cuda:{device}, the current device is cuda:{_raw_device()}")
    lib.gemm_set_stream(_raw_stream(device))


def _bind_torch_stream(*tensors) -> None:
    """Points the library at torch's current stream of the tensors' device.
    Every tensor argument must live on the current CUDA device: a kernel given
    another device's address would read memory it cannot reach."""
    dev = None
    for t in tensors:
        if t is None or type(t) is int or not hasattr(t, "get_device"):
            continue
        d = t.get_device()  # an index: cheaper than a torch.device per tensor
        if d < 0:
            raise ValueError("tensors must live on a CUDA device")
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"tensors on two devices: cuda:{dev} and cuda:{d}")
    if dev is not None:
        _point_at(_lib or load(), dev)


def _span(outer: int, inner: int, ld: int, stride: int = 0, batch: int = 1) -> int:
    """Elements from a stored matrix's first element to one past its last:
    `batch` matrices of `outer` lines of `inner` elements, lines `ld` apart and
    matrices `stride` apart.  0 for an empty matrix or a negative argument,
    which the library itself rejects."""
    if min(outer, inner, ld, stride, batch) < 0 or outer == 0 or inner == 0 or batch == 0:
        return 0
    return (batch - 1) * stride + (outer - 1) * ld + inner


def _check(name: str, t, elt_size: int, need: int, tight: bool = True) -> None:
    """Host-side check of one tensor argument before its address is passed on:
    the element size of the entry point, and room for the `need` elements the
    call reads or writes from the tensor's first element (the tensor's own
    elements for the tight layouts of the named entry points, which also need
    a contiguous tensor; the rest of its storage for gemm_ex, whose leading
    dimensions may step over a wider buffer).  A raw address (an int) or None
    is passed as it is."""
    if t is None or isinstance(t, int):
        return
    if t.element_size() != elt_size:
        raise ValueError(f"{name}: the entry point takes {elt_size}-byte elements, got {t.dtype}")
    if tight:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        room = t.numel()
    else:
        room = t.untyped_storage().nbytes() // elt_size - t.storage_offset()
    if room < need:
        raise ValueError(f"{name} holds {room} elements, the call needs {need}")


def _check_rows(name: str, t, ld: int, need: int) -> None:
    """A tensor in the place of a matrix with leading dimension ld that spans `need`
    elements: unit stride along a row and, if there are several, ld from one row to
    the next (through any further dimensions).  A flat buffer has no rows of its own."""
    if not need or t is None or type(t) is int or t.stride() == (ld, 1):
        return
    size, stride = t.shape, t.stride()
    good = not len(size) or size[-1] <= 1 or stride[-1] == 1
    if need > ld:
        step = ld
        for n, apart in zip(size[-2::-1], stride[-2::-1]):
            good = good and (n <= 1 or apart == step)
            step *= n
    if not good:
        raise ValueError(f"{name} must have rows of adjacent elements, {ld} elements apart; its strides are {stride}")


def _take(lib, name: str, *args):
    """Addresses of several tensor arguments (argument, tensor, element size,
    elements, tight), each checked as by _check -- a contiguous tensor with room
    passes without a message being built -- and all on the current CUDA device, to
    whose current torch stream the library is pointed."""
    out, dev, mixed = [], None, False
    for arg, t, size, need, tight in args:
        if t is None:
            out.append(0)
            continue
        if type(t) is int:
            out.append(t)
            continue
        if t.element_size() != size or not t.is_contiguous() or t.numel() < need:
            _check(f"{name}: {arg}", t, size, need, tight)
        d = t.get_device()
        if d != dev:
            mixed = dev is not None
            dev = d if dev is None or d < 0 else dev
        out.append(t.data_ptr())
    if dev is not None:
        if dev < 0:
            raise ValueError("tensors must live on a CUDA device")
        if mixed:
            raise ValueError("tensors on two devices")
        _point_at(lib, dev)
    return out


def _dims(M: int, N: int, K: int):
    """Elements of the tight A [M,K], B [K,N] and C [M,N] a call touches: none
    when M or N is 0 (a no-op) or a dimension is negative (the library rejects
    the call); C alone when K is 0 (zeros are written)."""
    M, N, K = int(M), int(N), int(K)
    if min(M, N, K) < 0 or M == 0 or N == 0:
        return 0, 0, 0
    return M * K, K * N, M * N


_ELT = {"gemm_f32_rm": 4, "gemm_f16_cm": 2, "gemm_bf16_rm": 2, "gemm_bf16_rm_noalloc": 2}


def _call(name: str, A, B, C, M: int, N: int, K: int) -> None:
    lib = load()
    na, nb, nc = _dims(M, N, K)
    for arg, t, need in (("A", A, na), ("B", B, nb), ("C", C, nc)):
        _check(f"{name}: {arg}", t, _ELT[name], need)
    _bind_torch_stream(A, B, C)
    st = getattr(lib, name)(_addr(A), _addr(B), _addr(C), int(M), int(N), int(K))
    if st != GEMM_OK:
        raise GemmError(st, name, lib.gemm_last_error().decode())


def gemm_f32_rm(A, B, C, M: int, N: int, K: int) -> None:
    """C[M,N] = A[M,K]·B[K,N], row-major float32, FP32 FFMA only."""
    _call("gemm_f32_rm", A, B, C, M, N, K)


def gemm_f16_cm(A, B, C, M: int, N: int, K: int) -> None:
    """C = A·B, column-major half (lda = M, ldb = K, ldc = M), FP32 accumulation."""
    _call("gemm_f16_cm", A, B, C, M, N, K)


def gemm_bf16_rm(A, B, C, M: int, N: int, K: int) -> None:
    """C[M,N] = A[M,K]·B[K,N], row-major bf16, FP32 accumulation."""
    _call("gemm_bf16_rm", A, B, C, M, N, K)


def gemm_bf16_rm_noalloc(A, B, C, M: int, N: int, K: int) -> None:
    """As gemm_bf16_rm, on the tensor-core kernel with its scratch in a static
    device array: the call allocates no device memory."""
    _call("gemm_bf16_rm_noalloc", A, B, C, M, N, K)


def gemm_bf16_rm_silu_mul(X, W_g, W_u, Z, M: int, N: int, K: int) -> None:
    """Z[M,N] = SiLU(X W_g) * (X W_u), bf16 row-major, the FFN gate/up projection."""
    lib = load()
    nx, nw, nz = _dims(M, N, K)
    for arg, t, need in (("X", X, nx), ("W_g", W_g, nw), ("W_u", W_u, nw), ("Z", Z, nz)):
        _check(f"gemm_bf16_rm_silu_mul: {arg}", t, 2, need)
    _bind_torch_stream(X, W_g, W_u, Z)
    st = lib.gemm_bf16_rm_silu_mul(_addr(X), _addr(W_g), _addr(W_u), _addr(Z), int(M), int(N), int(K))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_bf16_rm_silu_mul", lib.gemm_last_error().decode())


def gemm_quantize_rows_e4m3(A, Q, scale, M: int, K: int) -> None:
    """Row-wise E4M3 quantisation of a half [M,K] matrix: Q [M,K] codes (uint8),
    scale [M] float32, a_ik ~ Q[i,k] * scale_i."""
    lib = load()
    na = _dims(M, 1, K)[0]
    rows = max(int(M), 0)  # the scales are written even for K = 0 (scale 0)
    for arg, t, size, need in (("A", A, 2, na), ("Q", Q, 1, na), ("scale", scale, 4, rows)):
        _check(f"gemm_quantize_rows_e4m3: {arg}", t, size, need)
    _bind_torch_stream(A, Q, scale)
    st = lib.gemm_quantize_rows_e4m3(_addr(A), _addr(Q), _addr(scale), int(M), int(K))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_quantize_rows_e4m3", lib.gemm_last_error().decode())


def gemm_e4m3_rowscale(Q, scale, Wt, C, M: int, N: int, K: int) -> None:
    """C[M,N] (half) = diag(scale) Q[M,K] W[K,N], with the E4M3 weights given as Wt [N,K]."""
    lib = load()
    nq, nw, nc = _dims(M, N, K)
    rows = int(M) if nq else 0  # the scales are read only when the product has terms
    for arg, t, size, need in (("Q", Q, 1, nq), ("scale", scale, 4, rows), ("Wt", Wt, 1, nw), ("C", C, 2, nc)):
        _check(f"gemm_e4m3_rowscale: {arg}", t, size, need)
    _bind_torch_stream(Q, scale, Wt, C)
    st = lib.gemm_e4m3_rowscale(_addr(Q), _addr(scale), _addr(Wt), _addr(C), int(M), int(N), int(K))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_e4m3_rowscale", lib.gemm_last_error().decode())


def gemm_e4m3_rowscale_fused(A, Wt, C, M: int, N: int, K: int) -> None:
    """C[M,N] (half) = diag(amax/448) E4M3(diag(448/amax) A) W, the row-wise
    quantisation of the half A [M,K] fused into the product's load path; the
    E4M3 weights given as Wt [N,K]."""
    lib = load()
    na, nw, nc = _dims(M, N, K)
    for arg, t, size, need in (("A", A, 2, na), ("Wt", Wt, 1, nw), ("C", C, 2, nc)):
        _check(f"gemm_e4m3_rowscale_fused: {arg}", t, size, need)
    _bind_torch_stream(A, Wt, C)
    st = lib.gemm_e4m3_rowscale_fused(_addr(A), _addr(Wt), _addr(C), int(M), int(N), int(K))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_e4m3_rowscale_fused", lib.gemm_last_error().decode())


DTYPES = {"f32": 0, "f16": 1, "bf16": 2}
LAYOUTS = {"rm": 0, "cm": 1}
OPS = {"N": 0, "T": 1}


def gemm_ex(dtype: str, layout: str, op_a: str, op_b: str, M: int, N: int, K: int, alpha: float,
            A, lda: int, stride_a: int, B, ldb: int, stride_b: int, beta: float, C, ldc: int,
            stride_c: int, batch: int = 1) -> None:
    """C_b = alpha op(A_b) op(B_b) + beta C_b for b < batch.  dtype 'f32' | 'f16' |
    'bf16', layout 'rm' | 'cm', op_a / op_b 'N' | 'T'; leading dimensions and
    strides in elements (see include/gemm.h for the storage rules)."""
    lib = load()
    M, N, K, batch = int(M), int(N), int(K), int(batch)
    cm = layout == "cm"
    a_r, a_c = (M, K) if op_a == "N" else (K, M)
    b_r, b_c = (K, N) if op_b == "N" else (N, K)
    # (lines, elements per line) of each stored matrix in memory order
    (ao, ai), (bo, bi), (co, ci) = ((c, r) if cm else (r, c) for r, c in ((a_r, a_c), (b_r, b_c), (M, N)))
    # A and B are read only when the product has terms; C is written whenever
    # it has elements (and read when beta != 0)
    reads_ab = K > 0 and float(alpha) != 0.0 and M > 0 and N > 0
    size = {"f32": 4, "f16": 2, "bf16": 2}.get(dtype, 0)
    if size:
        _check("gemm_ex: A", A, size, _span(ao, ai, int(lda), int(stride_a), batch) if reads_ab else 0, tight=False)
        _check("gemm_ex: B", B, size, _span(bo, bi, int(ldb), int(stride_b), batch) if reads_ab else 0, tight=False)
        _check("gemm_ex: C", C, size, _span(co, ci, int(ldc), int(stride_c), batch), tight=False)
    _bind_torch_stream(A, B, C)
    st = lib.gemm_ex(DTYPES[dtype], LAYOUTS[layout], OPS[op_a], OPS[op_b], int(M), int(N), int(K),
                     float(alpha), _addr(A), int(lda), int(stride_a), _addr(B), int(ldb), int(stride_b),
                     float(beta), _addr(C), int(ldc), int(stride_c), int(batch))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_ex", lib.gemm_last_error().decode())


FP4_FORMATS = {"mx": 0, "nv": 1}
_DTYPES16 = {"f16": 1, "bf16": 2}


def _fp4_enums(name: str, dtype: str, fmt: str):
    if dtype not in _DTYPES16 or fmt not in FP4_FORMATS:
        raise ValueError(f"{name}: dtype 'f16' | 'bf16' and format 'mx' | 'nv', got {dtype!r} and {fmt!r}")
    return _DTYPES16[dtype], FP4_FORMATS[fmt]


def gemm_fp4_code_bytes(rows: int, K: int) -> int:
    """Bytes of the 4-bit codes of a [rows, K] matrix."""
    return int(load().gemm_fp4_code_bytes(int(rows), int(K)))


def gemm_fp4_scale_bytes(fmt: str, rows: int, K: int) -> int:
    """Bytes of the block scales of a [rows, K] matrix in format 'mx' or 'nv'."""
    if fmt not in FP4_FORMATS:
        raise ValueError(f"gemm_fp4_scale_bytes: format 'mx' | 'nv', got {fmt!r}")
    return int(load().gemm_fp4_scale_bytes(FP4_FORMATS[fmt], int(rows), int(K)))


def _fp4_sizes(fmt: int, rows: int, K: int):
    """Bytes of the codes and scales of a quantised [rows, K] operand, and the
    elements of its tensor scale (nothing where a size is 0 or negative: the
    library returns or rejects the call)."""
    if rows <= 0 or K <= 0:
        return 0, 0, 0
    return rows * ((K + 31) // 32 * 16), (rows + 127) // 128 * ((K + 255) // 256) * (2048 if fmt else 1024), 1


def _fp4_span(rows: int, cols: int, ld: int) -> int:
    """_span of one matrix."""
    return (rows - 1) * ld + cols if rows > 0 and cols > 0 and ld >= 0 else 0


def gemm_fp4_quantize(dtype: str, fmt: str, A, lda: int, tensor_scale, Q, S, M: int, K: int) -> None:
    """Quantises A [M,K] ('f16' | 'bf16', leading dimension lda) to 4-bit codes Q
    and block scales S, format 'mx' or 'nv'; tensor_scale: one FP32 value on the
    device for 'nv' (None: 1), None for 'mx'.  A tensor of two or more dimensions
    with other strides than lda's, a transposed view for one, is refused (as X, C and
    the read-back's A are below).  See include/gemm.h."""
    lib = _lib or load()
    d, f = _fp4_enums("gemm_fp4_quantize", dtype, fmt)
    M, K, lda = int(M), int(K), int(lda)
    nq, ns, ng = _fp4_sizes(f, M, K)
    na = _fp4_span(M, K, lda)
    _check_rows("gemm_fp4_quantize: A", A, lda, na)
    a, q, s, g = _take(lib, "gemm_fp4_quantize", ("A", A, 2, na, False),
                       ("Q", Q, 1, nq, True), ("S", S, 1, ns, True), ("tensor_scale", tensor_scale, 4, ng, True))
    st = lib.gemm_fp4_quantize(d, f, a, lda, g, q, s, M, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp4_quantize", lib.gemm_last_error().decode())


def gemm_fp4_dequantize(dtype: str, fmt: str, Q, S, tensor_scale, A, lda: int, M: int, K: int) -> None:
    """Writes the values that codes Q and scales S stand for to A [M,K]."""
    lib = _lib or load()
    d, f = _fp4_enums("gemm_fp4_dequantize", dtype, fmt)
    M, K, lda = int(M), int(K), int(lda)
    nq, ns, ng = _fp4_sizes(f, M, K)
    na = _fp4_span(M, K, lda)
    _check_rows("gemm_fp4_dequantize: A", A, lda, na)
    a, q, s, g = _take(lib, "gemm_fp4_dequantize", ("A", A, 2, na, False),
                       ("Q", Q, 1, nq, True), ("S", S, 1, ns, True), ("tensor_scale", tensor_scale, 4, ng, True))
    st = lib.gemm_fp4_dequantize(d, f, q, s, g, a, lda, M, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp4_dequantize", lib.gemm_last_error().decode())


def gemm_fp4(dtype: str, fmt: str, Qa, Sa, ga, Qb, Sb, gb, C, ldc: int, M: int, N: int, K: int) -> None:
    """C [M,N] ('f16' | 'bf16') = ga gb a b^T of two quantised matrices a [M,K] and
    b [N,K] of format 'mx' or 'nv'."""
    lib = _lib or load()
    d, f = _fp4_enums("gemm_fp4", dtype, fmt)
    M, N, K, ldc = int(M), int(N), int(K), int(ldc)
    some = M > 0 and N > 0  # else a no-op or a call that the library rejects
    qa, sa, na = _fp4_sizes(f, M, K if some else 0)
    qb, sb, nb = _fp4_sizes(f, N, K if some else 0)
    nc = _fp4_span(M, N, ldc)
    _check_rows("gemm_fp4: C", C, ldc, nc)
    pqa, psa, pga, pqb, psb, pgb, c = _take(
        lib, "gemm_fp4", ("Qa", Qa, 1, qa, True), ("Sa", Sa, 1, sa, True), ("ga", ga, 4, na, True),
        ("Qb", Qb, 1, qb, True), ("Sb", Sb, 1, sb, True), ("gb", gb, 4, nb, True),
        ("C", C, 2, nc, False))
    st = lib.gemm_fp4(d, f, pqa, psa, pga, pqb, psb, pgb, c, ldc, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp4", lib.gemm_last_error().decode())


def gemm_fp4_linear(dtype: str, fmt: str, X, ldx: int, gx, Qw, Sw, gw, C, ldc: int, M: int, N: int, K: int) -> None:
    """C [M,N] = X W^T with X [M,K] ('f16' | 'bf16', leading dimension ldx)
    quantised within the call (tensor scale gx) and W [N,K] quantised already."""
    lib = _lib or load()
    d, f = _fp4_enums("gemm_fp4_linear", dtype, fmt)
    M, N, K, ldx, ldc = int(M), int(N), int(K), int(ldx), int(ldc)
    some = M > 0 and N > 0  # else a no-op or a call that the library rejects
    qw, sw, nw = _fp4_sizes(f, N, K if some else 0)
    nx, nc = _fp4_span(M, K, ldx) if some else 0, _fp4_span(M, N, ldc)
    _check_rows("gemm_fp4_linear: X", X, ldx, nx)
    _check_rows("gemm_fp4_linear: C", C, ldc, nc)
    x, pgx, q, s, pgw, c = _take(
        lib, "gemm_fp4_linear", ("X", X, 2, nx, False), ("gx", gx, 4, nw, True),
        ("Qw", Qw, 1, qw, True), ("Sw", Sw, 1, sw, True), ("gw", gw, 4, nw, True),
        ("C", C, 2, nc, False))
    st = lib.gemm_fp4_linear(d, f, x, ldx, pgx, q, s, pgw, c, ldc, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp4_linear", lib.gemm_last_error().decode())


ACTIVATIONS = {"silu": 0, "gelu": 1}


def _gated_enums(name: str, dtype: str, act: str):
    if dtype not in _DTYPES16 or act not in ACTIVATIONS:
        raise ValueError(f"{name}: dtype 'f16' | 'bf16' and act 'silu' | 'gelu', got {dtype!r} and {act!r}")
    return _DTYPES16[dtype], ACTIVATIONS[act]


def gemm_gated(dtype: str, act: str, X, W_g, W_u, Z, G, U, M: int, N: int, K: int) -> None:
    """Z [M,N] = act(X W_g) * (X W_u) ('f16' | 'bf16', act 'silu' | 'gelu'); G and U
    (FP32 [M,N], or both None) keep the two products for gemm_gated_backward."""
    lib = _lib or load()
    d, a = _gated_enums("gemm_gated", dtype, act)
    M, N, K = int(M), int(N), int(K)
    nx, nw, nz = _dims(M, N, K)
    p = _take(lib, "gemm_gated", ("X", X, 2, nx, True), ("W_g", W_g, 2, nw, True), ("W_u", W_u, 2, nw, True),
              ("Z", Z, 2, nz, True), ("G", G, 4, nz, True), ("U", U, 4, nz, True))
    st = lib.gemm_gated(d, a, *p, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_gated", lib.gemm_last_error().decode())


def gemm_gated_backward(dtype: str, act: str, X, W_g, W_u, G, U, dZ, dX, dW_g, dW_u, M: int, N: int, K: int) -> None:
    """Gradients of gemm_gated from dZ [M,N] and the G and U it stored: dX [M,K],
    dW_g and dW_u [K,N]; None leaves one out."""
    lib = _lib or load()
    d, a = _gated_enums("gemm_gated_backward", dtype, act)
    M, N, K = int(M), int(N), int(K)
    nx, nw, nz = (M * K, K * N, M * N) if min(M, N, K) >= 0 else (0, 0, 0)
    p = _take(lib, "gemm_gated_backward", ("X", X, 2, nx, True), ("W_g", W_g, 2, nw, True), ("W_u", W_u, 2, nw, True),
              ("G", G, 4, nz, True), ("U", U, 4, nz, True), ("dZ", dZ, 2, nz, True), ("dX", dX, 2, nx, True),
              ("dW_g", dW_g, 2, nw, True), ("dW_u", dW_u, 2, nw, True))
    st = lib.gemm_gated_backward(d, a, *p, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_gated_backward", lib.gemm_last_error().decode())


def _dtype16(name: str, dtype: str) -> int:
    if dtype not in _DTYPES16:
        raise ValueError(f"{name}: dtype 'f16' | 'bf16', got {dtype!r}")
    return _DTYPES16[dtype]


def gemm_rms_norm(dtype: str, X, R, w, eps: float, H, Y, rstd, M: int, K: int) -> None:
    """H = X + R, Y = w H / sqrt(mean(H^2) + eps) over rows of K ('f16' | 'bf16').  R None:
    no residual (H None too); H None: the sum is not kept; H may be X or R itself; w
    None: ones; rstd (FP32 [M], or None) is kept for gemm_rms_norm_backward."""
    lib = _lib or load()
    d = _dtype16("gemm_rms_norm", dtype)
    M, K = int(M), int(K)
    n, m, k = _rows_dims(M, K)
    x, r, pw, h, y, rs = _take(lib, "gemm_rms_norm", ("X", X, 2, n, True), ("R", R, 2, n, True), ("w", w, 2, k, True),
                               ("H", H, 2, n, True), ("Y", Y, 2, n, True), ("rstd", rstd, 4, m, True))
    st = lib.gemm_rms_norm(d, x, r, pw, eps, h, y, rs, M, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_rms_norm", lib.gemm_last_error().decode())


def gemm_rms_norm_e4m3(dtype: str, X, R, w, eps: float, H, Q, scale, M: int, K: int) -> None:
    """gemm_rms_norm with Y as E4M3 codes Q [M,K] and row scales (FP32 [M]), the operand
    of gemm_e4m3_rowscale: Y ~ Q scale, scale = amax |Y| / 448."""
    lib = _lib or load()
    d = _dtype16("gemm_rms_norm_e4m3", dtype)
    M, K = int(M), int(K)
    n, m, k = _rows_dims(M, K)
    x, r, pw, h, q, sc = _take(lib, "gemm_rms_norm_e4m3", ("X", X, 2, n, True), ("R", R, 2, n, True),
                               ("w", w, 2, k, True), ("H", H, 2, n, True), ("Q", Q, 1, n, True),
                               ("scale", scale, 4, m, True))
    st = lib.gemm_rms_norm_e4m3(d, x, r, pw, eps, h, q, sc, M, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_rms_norm_e4m3", lib.gemm_last_error().decode())


def gemm_rms_norm_backward(dtype: str, H, w, rstd, dY, dH, dX, dw, M: int, K: int) -> None:
    """Gradients of gemm_rms_norm from dY and dH (None: 0): dX [M,K] of X and R alike (may
    be dH itself), dw FP32 [K]; None leaves one out."""
    lib = _lib or load()
    d = _dtype16("gemm_rms_norm_backward", dtype)
    M, K = int(M), int(K)
    n, m, k = _rows_dims(M, K)
    kw = max(K, 0) if M >= 0 else 0  # dw is written for M = 0 too
    p = _take(lib, "gemm_rms_norm_backward", ("H", H, 2, n, True), ("w", w, 2, k, True), ("rstd", rstd, 4, m, True),
              ("dY", dY, 2, n, True), ("dH", dH, 2, n, True), ("dX", dX, 2, n, True), ("dw", dw, 4, kw, True))
    st = lib.gemm_rms_norm_backward(d, *p, M, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_rms_norm_backward", lib.gemm_last_error().decode())


def gemm_cross_entropy(dtype: str, X, W, targets, loss, lse, M: int, N: int, K: int) -> None:
    """loss (FP32 [M]) = lse - Z[i, targets_i] of the logits Z = X W^T, never kept: X [M,K],
    W [N,K] ('f16' | 'bf16'), targets int64 [M] (outside 0 .. N-1: the row is left out, loss
    0); lse (FP32 [M], or None) is kept for gemm_cross_entropy_backward."""
    lib = _lib or load()
    d = _dtype16("gemm_cross_entropy", dtype)
    M, N, K = int(M), int(N), int(K)
    nx, nw, _ = _dims(M, N, K)
    m = M if min(M, N, K) >= 0 else 0
    p = _take(lib, "gemm_cross_entropy", ("X", X, 2, nx, True), ("W", W, 2, nw, True), ("targets", targets, 8, m, True),
              ("loss", loss, 4, m, True), ("lse", lse, 4, m, True))
    st = lib.gemm_cross_entropy(d, *p, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_cross_entropy", lib.gemm_last_error().decode())


def gemm_cross_entropy_backward(dtype: str, X, W, targets, lse, dloss, dX, dW, M: int, N: int, K: int) -> None:
    """Gradients of gemm_cross_entropy from dloss (FP32 [M]) and the lse it stored: dX [M,K]
    and dW [N,K]; None leaves one out."""
    lib = _lib or load()
    d = _dtype16("gemm_cross_entropy_backward", dtype)
    M, N, K = int(M), int(N), int(K)
    nx, nw, m = (M * K, N * K, M) if min(M, N, K) >= 0 else (0, 0, 0)
    p = _take(lib, "gemm_cross_entropy_backward", ("X", X, 2, nx, True), ("W", W, 2, nw, True),
              ("targets", targets, 8, m, True), ("lse", lse, 4, m, True), ("dloss", dloss, 4, m, True),
              ("dX", dX, 2, nx, True), ("dW", dW, 2, nw, True))
    st = lib.gemm_cross_entropy_backward(d, *p, M, N, K)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_cross_entropy_backward", lib.gemm_last_error().decode())


QUINTIC = (3.4445, -4.7750, 2.0315)


def gemm_orthogonalize(dtype: str, G, ldg: int, O, ldo: int, steps: int, M: int, N: int, coefficients=QUINTIC) -> None:
    """O [M,N] = G / |G|_F after `steps` times X <- a X + (b A + c A^2) X, A = X X^T (X^T X
    from the right for M > N), coefficients (a, b, c); 'f16' | 'bf16', leading dimensions
    ldg and ldo; O may be G itself.  A tensor of two or more dimensions with other strides
    than its leading dimension's is refused."""
    lib = _lib or load()
    d = _dtype16("gemm_orthogonalize", dtype)
    M, N, ldg, ldo = int(M), int(N), int(ldg), int(ldo)
    a, b, c = coefficients
    ng, no = _fp4_span(M, N, ldg), _fp4_span(M, N, ldo)
    _check_rows("gemm_orthogonalize: G", G, ldg, ng)
    _check_rows("gemm_orthogonalize: O", O, ldo, no)
    pg, po = _take(lib, "gemm_orthogonalize", ("G", G, 2, ng, False), ("O", O, 2, no, False))
    st = lib.gemm_orthogonalize(d, pg, ldg, po, ldo, int(steps), a, b, c, M, N)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_orthogonalize", lib.gemm_last_error().decode())


def _rows_dims(M: int, K: int):
    """Elements of an [M,K] operand, of a value a row and of one a column: none where M or
    K is 0 or negative (a no-op, or a call that the library rejects)."""
    return (M * K, M, K) if M > 0 and K > 0 else (0, 0, 0)


def gemm_set_stream(stream) -> None:
    """Stream for this thread's later calls: a torch.cuda.Stream, a raw handle or None."""
    handle = getattr(stream, "cuda_stream", stream)
    st = load().gemm_set_stream(ctypes.c_void_p(handle or 0))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_set_stream")


def gemm_get_stream() -> int:
    return load().gemm_get_stream() or 0


def gemm_synchronize() -> None:
    lib = load()
    st = lib.gemm_synchronize()
    if st != GEMM_OK:
        raise GemmError(st, "gemm_synchronize", lib.gemm_last_error().decode())


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(int(status)).decode()


def gemm_last_kernel() -> str:
    return load().gemm_last_kernel().decode()


def gemm_kernel_launches() -> int:
    return int(load().gemm_kernel_launches())


def gemm_last_error() -> str:
    return load().gemm_last_error().decode()


def gemm_force_kernel(family) -> None:
    st = load().gemm_force_kernel(family.encode() if family else None)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_force_kernel", str(family))


def matmul(a, b, out=None):
    """C = a @ b for 2-D row-major torch CUDA tensors of one dtype (float32,
    bfloat16 or float16).  float16 goes through the column-major entry point on
    the same buffers (row-major C = A·B is column-major C^T = B^T·A^T)."""
    import torch
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"bad shapes {tuple(a.shape)} @ {tuple(b.shape)}")
    if a.dtype != b.dtype:
        raise ValueError("a and b must share a dtype")
    a = a.contiguous()
    b = b.contiguous()
    M, K = a.shape
    N = b.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=a.dtype, device=a.device)
    elif out.shape != (M, N) or out.dtype != a.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M, N] tensor of the input dtype")
    if a.dtype == torch.float32:
        gemm_f32_rm(a, b, out, M, N, K)
    elif a.dtype == torch.bfloat16:
        gemm_bf16_rm(a, b, out, M, N, K)
    elif a.dtype == torch.float16:
        gemm_f16_cm(b, a, out, N, M, K)
    else:
        raise ValueError(f"unsupported dtype {a.dtype}")
    return out
