"""Products in 8-bit floating point for torch tensors: the entry points of
include/sgemm_f32_f8.h.

    w = f8_pack(codes, scales)             # or f8_quantize(B); a scale for each 128 x 128
    C = matmul_f8(A, w)                    # A: rows x K, float32 or bfloat16
    C = matmul_f8(A, w, offsets=offsets)   # rows by expert (a stack of matrices)

    w, wt = f8_quantize(B, both=True)      # a training step: the matrices and their transposes
    dA = matmul_f8(dC, wt, dtype=torch.float8_e5m2)
    dB = matmul_f8_ta(A, dC, dtypes=(torch.float8_e4m3fn, torch.float8_e5m2))

Rows are put into 8 bits by each call, with a power of two for each row and block of 128
as their scale (the formulas are in include/sgemm_f32_f8.h), or once for several products
by f8_rows().  Weights are laid out once; each call is enqueued on ``stream`` (default:
torch's current stream on the tensors' device) without synchronising.  A stream that is
passed in has to wait for the work that makes the inputs, and what reads the results for
that stream, as with torch's own operations on a stream.  There is no autograd here: a
result takes no part in a graph, also where an input requires a gradient; the gradients
are products of their own, as above.
"""
from __future__ import annotations

import torch

from ._binding import (F8_E4M3, F8_E5M2, F8_IN_BF16, F8_IN_F32, F8_IN_ROWS, F8_SCALE_E8M0,
                       F8_SCALE_F32, OP_N, OP_T, lib)
from ._tensors import MOST, call, dense, matrix, new, place
from .experts import _offsets, _stack

CODE_TYPES = {torch.float8_e4m3fn: F8_E4M3, torch.float8_e5m2: F8_E5M2}
NUMBER_TYPES = {torch.float32: F8_IN_F32, torch.bfloat16: F8_IN_BF16}
SCALE_TYPES = {torch.float32: F8_SCALE_F32, torch.float8_e8m0fnu: F8_SCALE_E8M0}


def _held(t, name, size):
    """Raises unless t holds `size` bytes as the library lays them out."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous uint8 torch tensor")
    if t.numel() < size:
        raise ValueError(f"{name} holds {t.numel()} bytes; {size} are needed")


class F8Weights:
    """8-bit matrices as the library lays them out: ``experts`` of K x N (``stacked``:
    made from a stack, else one matrix), with a scale for each 128 x 128."""

    def __init__(self, packed, experts, stacked, K, N, scale_type):
        _held(packed, "packed", lib().sgemm_f32_f8_packed_size(experts, N, K))
        self.packed = packed
        self.experts, self.stacked = experts, stacked
        self.K, self.N = K, N
        self.scale_type = scale_type

    def __repr__(self):
        kind = "fp32" if self.scale_type == F8_SCALE_F32 else "power of two"
        return f"F8Weights({self.experts} x {self.K} x {self.N}, {kind} scales)"


class F8Rows:
    """rows x K numbers in 8 bits (``code_type``: that of their codes), with a scale for
    each row and block of 128."""

    def __init__(self, data, rows, K, code_type):
        _held(data, "data", lib().sgemm_f32_f8_rows_size(rows, K))
        self.data = data
        self.rows, self.K = rows, K
        self.code_type = code_type

    def __repr__(self):
        return f"F8Rows({self.rows} x {self.K}, {'e4m3' if self.code_type == F8_E4M3 else 'e5m2'})"


def _code_type(dtype):
    kind = CODE_TYPES.get(dtype)
    if kind is None:
        raise TypeError(f"codes are float8_e4m3fn or float8_e5m2, not {dtype}")
    return kind


def _numbers(t, rows, cols, name, device=None):
    """(type, row stride) of a rows x cols float32 or bfloat16 tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in NUMBER_TYPES:
        raise TypeError(f"{name} must be a 2-D float32 or bfloat16 torch tensor")
    return NUMBER_TYPES[t.dtype], matrix(t, rows, cols, name, t.dtype, device)


def _weights(w):
    """The number of the GPU that holds the matrices w."""
    if not isinstance(w, F8Weights):
        raise TypeError("w must be F8Weights (f8_pack, f8_quantize)")
    device = w.packed.get_device()
    return device if device >= 0 else place(w.packed, "w", None)


def _new(experts, stacked, K, N, scale_type, like, stream):
    if max(experts, K, N) > MOST:
        raise ValueError("sizes beyond 32 bits")
    size = lib().sgemm_f32_f8_packed_size(experts, N, K)
    packed = new(like, size, stream, torch.uint8)
    return F8Weights(packed, experts, stacked, K, N, scale_type)


def _pointer(w):
    return (0, 0) if w is None else (w.packed.data_ptr(), w.packed.numel())


def f8_pack(codes, scales, stream=None):
    """F8Weights from codes ([experts x] K x N, float8_e4m3fn, row-major or transposed
    views) and scales ([experts x] ceil(K/128) x ceil(N/128), float32 or float8_e8m0fnu, in the
    codes' layout: contiguous, or with transposed codes the transposed view of a contiguous
    array, as in ``f8_pack(codes.t(), scales.t())``)."""
    if not isinstance(codes, torch.Tensor) or codes.dim() not in (2, 3):
        raise TypeError("codes must be a 2-D or 3-D float8_e4m3fn torch tensor")
    stacked = codes.dim() == 3
    stack = codes if stacked else codes[None]
    ld, stride, trans = _stack(stack, "codes", None, torch.float8_e4m3fn)
    experts, K, N = stack.shape
    if not isinstance(scales, torch.Tensor) or scales.dtype not in SCALE_TYPES:
        raise TypeError("scales must be a float32 or float8_e8m0fnu torch tensor")
    kind = SCALE_TYPES[scales.dtype]
    shape = (experts,) * stacked + (-(-K // 128), -(-N // 128))
    if scales.shape != shape:
        raise ValueError(f"scales has the shape {tuple(scales.shape)}; {shape} is needed")
    held = scales.transpose(-1, -2) if trans else scales
    if not held.is_contiguous():
        raise ValueError("scales must be " + ("the transposed view of a contiguous array, as codes is a "
                                              "transposed one" if trans else
                                              "contiguous, as codes is row-major"))
    dense(held, held.shape, "scales", scales.dtype, codes.get_device())
    w = _new(experts, stacked, K, N, kind, codes, stream)
    call("sgemm_f32_f8_pack", codes.get_device(), stream, experts, N, K, OP_T if trans else OP_N,
         codes.data_ptr(), ld, stride, scales.data_ptr(), kind, w.packed.data_ptr(),
         w.packed.numel())
    return w


def f8_quantize(B, both=False, stream=None):
    """F8Weights nearest to B ([experts x] K x N, float32, row-major or transposed views),
    with powers of two as scales; with ``both`` a pair of them and those of the transposes
    (N x K, for the product with a gradient)."""
    if not isinstance(B, torch.Tensor) or B.dim() not in (2, 3):
        raise TypeError("B must be a 2-D or 3-D float32 torch tensor")
    stacked = B.dim() == 3
    stack = B if stacked else B[None]
    ldb, strideb, trans = _stack(stack, "B", None)
    experts, K, N = stack.shape
    w = _new(experts, stacked, K, N, F8_SCALE_E8M0, B, stream)
    wt = _new(experts, stacked, N, K, F8_SCALE_E8M0, B, stream) if both else None
    call("sgemm_f32_f8_quantize", B.get_device(), stream, experts, N, K, OP_T if trans else OP_N,
         B.data_ptr(), ldb, strideb, *_pointer(w), *_pointer(wt))
    return (w, wt) if both else w


def f8_unpack(w, stream=None):
    """The float32 matrices that w stands for, [experts x] K x N."""
    device = _weights(w)
    out = new(w.packed, (w.experts, w.K, w.N), stream, torch.float32)
    call("sgemm_f32_f8_unpack", device, stream, w.experts, w.N, w.K,
         w.packed.data_ptr(), w.packed.numel(), out.data_ptr(), max(w.N, 1), w.K * w.N)
    return out if w.stacked else out[0]


def f8_rows(A, dtype=torch.float8_e4m3fn, stream=None):
    """F8Rows of A (rows x K, float32 or bfloat16), for several products with the same
    rows; ``dtype``: the type of the codes."""
    kind, lda = _numbers(A, None, None, "A")
    code = _code_type(dtype)
    rows, K = A.shape
    if max(rows, K) > MOST:
        raise ValueError("sizes beyond 32 bits")
    data = new(A, lib().sgemm_f32_f8_rows_size(rows, K), stream, torch.uint8)
    call("sgemm_f32_f8_rows", A.get_device(), stream, rows, K, A.data_ptr(), lda, kind, code,
         data.data_ptr(), data.numel())
    return F8Rows(data, rows, K, code)


def matmul_f8(A, w, offsets=None, out=None, out_dtype=torch.float32, dtype=torch.float8_e4m3fn,
              stream=None):
    """A @ W for rows A (rows x K, float32 or bfloat16, put into codes of ``dtype``; or
    F8Rows) and one 8-bit matrix, or with ``offsets`` (int32, experts + 1 values) row i
    times the matrix of its expert e, offsets[e] <= i < offsets[e+1].  The result is
    float32 or bfloat16 (``out_dtype``, or the type of ``out``), summed in float32 either
    way.  Rows of no expert are left as they are in ``out`` (and hold anything in a result
    allocated here)."""
    device = _weights(w)
    if isinstance(A, F8Rows):
        if A.K != w.K:
            raise ValueError(f"A has {A.K} columns; {w.K} are needed")
        rows, held, kind, code, lda = A.rows, A.data, F8_IN_ROWS, A.code_type, w.K
        dense(held, held.shape, "A", torch.uint8, device)
    else:
        kind, lda = _numbers(A, None, w.K, "A", device)
        rows, held, code = A.shape[0], A, _code_type(dtype)
    if offsets is None:
        if w.experts != 1:
            raise ValueError(f"{w.experts} matrices need offsets")
    elif _offsets(offsets, device) != w.experts:
        raise ValueError(f"{offsets.numel()} offsets for {w.experts} experts")
    if out is None:
        if out_dtype not in NUMBER_TYPES:
            raise TypeError(f"results are float32 or bfloat16, not {out_dtype}")
        out = new(held, (rows, w.N), stream, out_dtype)
        ldc = w.N or 1
    else:
        _, ldc = _numbers(out, rows, w.N, "out", device)
    need, workspace = 0, None
    if kind != F8_IN_ROWS:
        need = lib().sgemm_f32_f8_workspace_size(rows, w.N, w.K, w.experts, offsets is not None)
        if need:
            workspace = new(held, need, stream, torch.uint8)
    call("sgemm_f32_f8", device, stream, rows, w.N, w.K, w.experts,
         0 if offsets is None else offsets.data_ptr(), held.data_ptr(), lda, kind, code,
         w.packed.data_ptr(), w.scale_type, out.data_ptr(), ldc, NUMBER_TYPES[out.dtype],
         0 if workspace is None else workspace.data_ptr(), need)
    return out


def matmul_f8_ta(A, D, offsets=None, out=None, alpha=1.0, beta=0.0,
                 dtypes=(torch.float8_e4m3fn, torch.float8_e4m3fn), stream=None):
    """alpha * A.T @ D + beta * out in 8 bits (columns of A) x (columns of D), float32, A
    and D (rows x any, float32 or bfloat16) put into codes of ``dtypes`` along their
    columns; with ``offsets`` a stack of them, matrix e over rows offsets[e] ..
    offsets[e+1]-1: the gradient of matmul_f8(A, W, offsets) with respect to W for D = the
    gradient of its result.  An expert without rows gets zeros (beta * out[e])."""
    a_kind, lda = _numbers(A, None, None, "A")
    device = A.get_device()
    rows, M = A.shape
    d_kind, ldd = _numbers(D, rows, None, "D", device)
    N = D.shape[1]
    a_code, d_code = (_code_type(t) for t in dtypes)
    experts = 1 if offsets is None else _offsets(offsets, device)
    shape = (M, N) if offsets is None else (experts, M, N)
    if max(rows, M, N, experts) > MOST:
        raise ValueError("sizes beyond 32 bits")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = new(A, shape, stream, torch.float32)
        ldc, stridec = N or 1, M * N
    else:
        if not isinstance(out, torch.Tensor) or tuple(out.shape) != shape:
            raise ValueError("out has the wrong shape")
        ldc, stridec, trans = _stack(out[None] if offsets is None else out, "out", device)
        if trans:
            raise ValueError("out must hold row-major matrices")
    need = lib().sgemm_f32_f8_ta_workspace_size(rows, M, N, experts)
    workspace = new(A, need, stream, torch.uint8) if need else None
    call("sgemm_f32_f8_ta", device, stream, rows, M, N, experts,
         0 if offsets is None else offsets.data_ptr(), float(alpha), A.data_ptr(), lda, a_kind,
         a_code, D.data_ptr(), ldd, d_kind, d_code, float(beta), out.data_ptr(), ldc, stridec,
         0 if workspace is None else workspace.data_ptr(), need)
    return out
