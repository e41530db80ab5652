"""Products with 4-bit weights for torch tensors: the entry points of
include/sgemm_f32_w4.h.

    w = w4_quantize(B, group=128)          # or w4_pack(codes, scales, zeros, K=K, group=group)
    C = matmul_w4(A, w)                    # A: rows x K, float32
    C = matmul_w4(A, w, offsets=offsets)   # rows by expert (a stack of matrices)

Weights are laid out once; each call is enqueued on ``stream`` (default: torch's
current stream on the tensors' device) without synchronising.  A stream that is passed
in has to wait for the work that makes the inputs, and what reads the results for that
stream, as with torch's own operations on a stream.  There is no autograd here: a
result takes no part in a graph, also where an input requires a gradient, and the
product has no gradient of its own (w4_unpack() gives the matrices for one).
"""
from __future__ import annotations

import torch

from ._binding import W4_SCALE_BF16, W4_SCALE_F16, W4_SCALE_F32, lib
from ._tensors import INT_MAX, MOST, call, dense, matrix, new
from .experts import _offsets, _stack

SCALE_TYPES = {torch.float32: W4_SCALE_F32, torch.float16: W4_SCALE_F16,
               torch.bfloat16: W4_SCALE_BF16}


class W4Weights:
    """4-bit matrices as the library lays them out: ``experts`` of K x N (``stacked``:
    made from a stack, else one matrix), with scales for each ``group`` of k and zero
    points if ``zeros``."""

    def __init__(self, packed, experts, stacked, K, N, group, scale_type, zeros):
        self.packed = packed
        self.experts, self.stacked = experts, stacked
        self.K, self.N, self.group = K, N, group
        self.scale_type, self.zeros = scale_type, zeros

    def __repr__(self):
        return (f"W4Weights({self.experts} x {self.K} x {self.N}, group {self.group}, "
                f"{'with' if self.zeros else 'without'} zero points)")


def _new(experts, stacked, K, N, group, scale_dtype, zeros, like, stream):
    if scale_dtype not in SCALE_TYPES:
        raise TypeError("scales must be float32, float16 or bfloat16")
    if group not in (32, 64) and (group <= 0 or group % 128 != 0):
        raise ValueError(f"group must be 32, 64 or a multiple of 128, not {group}")
    if max(experts, K, N) > MOST or group > INT_MAX:
        raise ValueError("sizes beyond 32 bits")
    kind = SCALE_TYPES[scale_dtype]
    size = lib().sgemm_f32_w4_packed_size(experts, N, K, group, kind, int(zeros))
    packed = new(like, size, stream, torch.uint8)
    return W4Weights(packed, experts, stacked, K, N, group, kind, bool(zeros))


def w4_pack(codes, scales, zeros=None, *, K, group, stream=None):
    """W4Weights from codes (uint8, [experts x] ceil(K/2) x N, the code of an even k in
    the low four bits), scales ([experts x] ceil(K/group) x N, float32, float16 or
    bfloat16) and zero points (uint8, as scales, any byte; None: 8).  All contiguous."""
    if not isinstance(codes, torch.Tensor) or codes.dim() not in (2, 3):
        raise TypeError("codes must be a 2-D or 3-D uint8 torch tensor")
    stacked = codes.dim() == 3
    experts = codes.shape[0] if stacked else 1
    N = codes.shape[-1]
    lead = (experts,) if stacked else ()
    if K < 0 or group <= 0:
        raise ValueError(f"K = {K}, group = {group}")
    groups = -(-K // group)
    dense(codes, lead + (-(-K // 2), N), "codes", torch.uint8, None)
    if not isinstance(scales, torch.Tensor) or scales.dtype not in SCALE_TYPES:
        raise TypeError("scales must be a float32, float16 or bfloat16 torch tensor")
    dense(scales, lead + (groups, N), "scales", scales.dtype, codes.get_device())
    if zeros is not None:
        dense(zeros, lead + (groups, N), "zeros", torch.uint8, codes.get_device())
    w = _new(experts, stacked, K, N, group, scales.dtype, zeros is not None, codes, stream)
    call("sgemm_f32_w4_pack", codes.get_device(), stream, experts, N, K, group,
         codes.data_ptr(), scales.data_ptr(), w.scale_type,
         0 if zeros is None else zeros.data_ptr(), w.packed.data_ptr(), w.packed.numel())
    return w


def w4_quantize(B, group=128, zeros=False, scale_dtype=torch.float32, stream=None):
    """W4Weights nearest to B ([experts x] K x N, float32, row-major): each group's scale
    from its largest magnitude, or with ``zeros`` its scale and zero point from its
    range (the formulas are in include/sgemm_f32_w4.h)."""
    if not isinstance(B, torch.Tensor) or B.dim() not in (2, 3):
        raise TypeError("B must be a 2-D or 3-D float32 torch tensor")
    stacked = B.dim() == 3
    stack = B if stacked else B[None]
    ldb, strideb, trans = _stack(stack, "B", None)
    if trans:
        raise ValueError("B must hold row-major matrices")
    experts, K, N = stack.shape
    w = _new(experts, stacked, K, N, group, scale_dtype, zeros, B, stream)
    call("sgemm_f32_w4_quantize", B.get_device(), stream, experts, N, K, group,
         B.data_ptr(), ldb, strideb, w.scale_type, int(w.zeros), w.packed.data_ptr(),
         w.packed.numel())
    return w


def w4_unpack(w, stream=None):
    """The float32 matrices that w stands for, [experts x] K x N."""
    device = w.packed.get_device()
    out = new(w.packed, (w.experts, w.K, w.N), stream, torch.float32)
    call("sgemm_f32_w4_unpack", device, stream, w.experts, w.N, w.K, w.group, w.scale_type,
         int(w.zeros), w.packed.data_ptr(), w.packed.numel(), out.data_ptr(), max(w.N, 1),
         w.K * w.N)
    return out if w.stacked else out[0]


def matmul_w4(A, w, offsets=None, out=None, stream=None):
    """A @ W for rows A (rows x K, float32) and one 4-bit matrix, or with ``offsets``
    (int32, experts + 1 values) row i times the matrix of its expert e, offsets[e] <=
    i < offsets[e+1].  Rows of no expert are left as they are in ``out`` (and hold
    anything in a result allocated here)."""
    lda = matrix(A, None, w.K, "A", device=w.packed.get_device())
    device = A.get_device()
    rows = A.shape[0]
    if offsets is None:
        if w.experts != 1:
            raise ValueError(f"{w.experts} matrices need offsets")
    elif _offsets(offsets, device) != w.experts:
        raise ValueError(f"{offsets.numel()} offsets for {w.experts} experts")
    if out is None:
        out = new(A, (rows, w.N), stream)
        ldc = w.N or 1
    else:
        ldc = matrix(out, rows, w.N, "out", device=device)
    if offsets is None:
        call("sgemm_f32_w4", device, stream, rows, w.N, w.K, A.data_ptr(), lda,
             w.packed.data_ptr(), w.group, w.scale_type, int(w.zeros), out.data_ptr(), ldc)
    else:
        call("sgemm_f32_w4_experts", device, stream, rows, w.N, w.K, w.experts,
             offsets.data_ptr(), A.data_ptr(), lda, w.packed.data_ptr(), w.group, w.scale_type,
             int(w.zeros), out.data_ptr(), ldc)
    return out
