"""Products of several matrices in one call and the ordering of rows around them,
for torch tensors: the entry points of include/sgemm_f32_experts.h.

Each call is enqueued on ``stream`` (default: torch's current stream on the
tensors' device) without synchronising.  A stream that is passed in has to wait for
the work that makes the inputs, and what reads the results for that stream, as with
torch's own operations on a stream.  Float tensors are float32 with a unit column
stride; a row stride (a view of a wider tensor) is passed as it is.  There is no
autograd here: a result takes no part in a graph, also where an input requires a
gradient; the gradients are functions of their own.

    routing = sort_by_expert(ids, experts)            # ids: tokens x top, int32
    rows = gather_rows(x, routing)                    # backward: combine_rows(drows, routing)
    h = grouped_matmul(rows, B, routing.offsets)      # backward: grouped_matmul(dh, B.transpose(1, 2), ...)
                                                      #           grouped_matmul_ta(rows, dh, ...)
    y = combine_rows(h, routing, weights)             # backward: combine_rows_grad(dy, h, ...)
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._binding import lib
from ._tensors import INT_MAX, MOST, call, dense, matrix, new, place


class Routing(NamedTuple):
    """Where rows go: expert e's rows are places offsets[e] .. offsets[e+1]-1 (int32,
    experts + 1 values); order[p] is the pair token*top + choice at place p (int32,
    tokens*top values, -1 past the last); position[token, choice] is a pair's place
    (int32, -1 if it was dropped)."""
    offsets: torch.Tensor
    order: torch.Tensor
    position: torch.Tensor


def _pairs(routing):
    """(positions, tokens, top, GPU number) of a routing, whose positions are checked."""
    position = routing.position
    if (not isinstance(position, torch.Tensor) or position.dtype is not torch.int32
            or position.dim() != 2):
        raise TypeError("routing.position must be a 2-D int32 torch tensor")
    device = position.get_device()
    if device < 0:
        place(position, "routing.position", None)
    if not position.is_contiguous():
        raise ValueError("routing.position must be contiguous")
    return position, *position.shape, device


def _offsets(offsets, device):
    """The number of experts of an offsets tensor."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 1:
        raise TypeError("offsets must be a 1-D int32 torch tensor of experts + 1 values")
    dense(offsets, offsets.shape, "offsets", torch.int32, device)
    return offsets.numel() - 1


def sort_by_expert(ids, experts, stream=None):
    """The Routing of ids (tokens x top, int32, unit column stride): pairs in the order
    of their experts, and of (token, choice) within an expert.  An id outside
    [0, experts) drops its pair."""
    ld = matrix(ids, None, None, "ids", torch.int32)
    tokens, top = ids.shape
    experts = int(experts)
    if tokens * top > MOST or not 0 <= experts <= MOST:
        raise ValueError(f"{tokens} x {top} pairs for {experts} experts do not fit 32-bit numbers")
    device = ids.get_device()
    empty = ids.new_empty if stream is None else lambda shape: new(ids, shape, stream)
    offsets, order, position = empty(experts + 1), empty(tokens * top), empty((tokens, top))
    need = lib().sgemm_f32_route_workspace_size(tokens, top, experts)
    workspace = empty(need // 4) if need else None
    call("sgemm_f32_route_sort", device, stream, tokens, top, experts, ids.data_ptr(), ld,
         offsets.data_ptr(), order.data_ptr(), position.data_ptr(),
         workspace.data_ptr() if need else 0, need)
    return Routing(offsets, order, position)


def gather_rows(x, routing, out=None, stream=None):
    """Row p of the result is the row of x (tokens x width) whose token is at place p
    of the routing.  Rows past the last place are left as they are in ``out`` (and
    hold anything in a result allocated here)."""
    position, tokens, top, device = _pairs(routing)
    ldx = matrix(x, tokens, None, "x", device=device)
    width = x.shape[1]
    if out is None:
        out = new(x, (tokens * top, width), stream)
        ldo = width or 1
    else:
        ldo = matrix(out, tokens * top, width, "out", device=device)
    call("sgemm_f32_route_gather", device, stream, tokens, top, width,
         position.data_ptr(), x.data_ptr(), ldx, out.data_ptr(), ldo)
    return out


def combine_rows(rows, routing, weights=None, out=None, stream=None):
    """Each token's rows, times its weights (tokens x top; None: 1), added in the order of
    its choices: tokens x width.  Dropped pairs add nothing.  Without weights this is
    the gradient of gather_rows."""
    position, tokens, top, device = _pairs(routing)
    ldr = matrix(rows, tokens * top, None, "rows", device=device)
    width = rows.shape[1]
    ldw = 1 if weights is None else matrix(weights, tokens, top, "weights", device=device)
    if out is None:
        out = new(rows, (tokens, width), stream)
        ldo = width or 1
    else:
        ldo = matrix(out, tokens, width, "out", device=device)
    call("sgemm_f32_route_combine", device, stream, tokens, top, width,
         position.data_ptr(), 0 if weights is None else weights.data_ptr(), ldw,
         rows.data_ptr(), ldr, out.data_ptr(), ldo)
    return out


def combine_rows_grad(dout, rows, routing, weights=None, drows=None, stream=None):
    """(drows, dweights), the gradient of combine_rows(rows, routing, weights) for the
    gradient dout of its result.  dweights is None without weights.  Rows past the
    last place are left as they are in ``drows`` (and hold anything in a tensor
    allocated here)."""
    position, tokens, top, device = _pairs(routing)
    ldd = matrix(dout, tokens, None, "dout", device=device)
    width = dout.shape[1]
    ldr = matrix(rows, tokens * top, width, "rows", device=device)
    dweights, ldw = None, 1
    if weights is not None:
        ldw = matrix(weights, tokens, top, "weights", device=device)
        if ldw == max(top, 1):
            dweights = new(weights, (tokens, top), stream)
        else:  # the library gives the gradient the weights' row stride
            dweights = new(weights, (tokens, ldw), stream)[:, :top]
    if drows is None:
        drows = new(rows, (tokens * top, width), stream)
        lddr = width or 1
    else:
        lddr = matrix(drows, tokens * top, width, "drows", device=device)
    call("sgemm_f32_route_combine_grad", device, stream, tokens, top, width,
         position.data_ptr(), 0 if weights is None else weights.data_ptr(), ldw,
         rows.data_ptr(), ldr, dout.data_ptr(), ldd, drows.data_ptr(), lddr,
         0 if dweights is None else dweights.data_ptr())
    return drows, dweights


def _stack(B, name, device):
    """(leading dimension, stride between matrices, transposed) of an experts x rows x
    cols tensor whose matrices are row-major or transposes of row-major ones."""
    if not isinstance(B, torch.Tensor) or B.dtype != torch.float32 or B.dim() != 3:
        raise TypeError(f"{name} must be a 3-D float32 torch tensor")
    if B.get_device() != device:
        place(B, name, device)
    e, r, c = B.shape
    se, s0, s1 = B.stride()
    if e == 0 or r == 0 or c == 0:
        return max(c, 1), 0, False
    if (c == 1 or s1 == 1) and (r == 1 or s0 >= c):
        ld, trans = (s0 if r > 1 else c), False
    elif (r == 1 or s0 == 1) and (c == 1 or s1 >= r):
        ld, trans = (s1 if c > 1 else r), True
    else:
        raise ValueError(f"{name} needs matrices with a unit stride in one dimension that do not "
                         "overlap themselves")
    if ld > INT_MAX:
        raise ValueError(f"{name} is too large: row stride {ld}")
    return ld, se if e > 1 else 0, trans


def grouped_matmul(A, B, offsets, out=None, alpha=1.0, beta=0.0, stream=None):
    """Row i of the result is alpha * A[i] @ B[e] + beta * out[i] for its expert e,
    offsets[e] <= i < offsets[e+1].  B is experts x K x N; a transposed view
    (``B.transpose(1, 2)``) is passed as transposed matrices, without a copy, and an
    expanded first dimension as one shared matrix.  Rows of no expert are left as
    they are in ``out`` (and hold anything in a result allocated here)."""
    lda = matrix(A, None, None, "A")
    device = A.get_device()
    rows, K = A.shape
    ldb, strideb, trans = _stack(B, "B", device)
    experts, K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if _offsets(offsets, device) != experts:
        raise ValueError(f"{offsets.numel()} offsets for {experts} experts")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = new(A, (rows, N), stream)
        ldc = N or 1
    else:
        ldc = matrix(out, rows, N, "out", device=device)
    call("sgemm_f32_grouped", device, stream, int(trans), rows, N, K, experts,
         offsets.data_ptr(), float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb, strideb,
         float(beta), out.data_ptr(), ldc)
    return out


def grouped_matmul_ta(A, D, offsets, out=None, alpha=1.0, beta=0.0, stream=None):
    """Matrix e of the result is alpha * A_e.T @ D_e + beta * out[e], A_e and D_e being
    rows offsets[e] .. offsets[e+1]-1: experts x (columns of A) x (columns of D),
    the gradient of grouped_matmul(A, B, offsets) with respect to B for D = the
    gradient of its result.  An expert without rows gets zeros (beta * out[e])."""
    lda = matrix(A, None, None, "A")
    device = A.get_device()
    rows, M = A.shape
    ldd = matrix(D, rows, None, "D", device=device)
    N = D.shape[1]
    experts = _offsets(offsets, device)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = new(A, (experts, M, N), stream)
        ldc, stridec = N or 1, M * N
    else:
        if tuple(out.shape) != (experts, M, N):
            raise ValueError("out has the wrong shape")
        ldc, stridec, trans = _stack(out, "out", device)
        if trans:
            raise ValueError("out must hold row-major matrices")
    call("sgemm_f32_grouped_ta", device, stream, rows, M, N, experts, offsets.data_ptr(),
         float(alpha), A.data_ptr(), lda, D.data_ptr(), ldd, float(beta), out.data_ptr(), ldc,
         stridec)
    return out
