"""What the torch layer of the operators shares: checks of tensors, the stream of a
call, and the library call itself on the tensors' device."""
from __future__ import annotations

import torch

from torch._C import _cuda_getCurrentRawStream as raw_stream
from torch._C import _cuda_getDevice as current_device

from ._binding import SgemmError, lib

INT_MAX = 2**31 - 1
MOST = 2**31 - 65537   # the largest size that the operators take


def matrix(t, rows, cols, name, dtype=torch.float32, device=None):
    """The row stride of a rows x cols tensor with unit column stride (rows or cols
    None: any number) on GPU number `device` (None: any); raises where it is not
    one."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D {str(dtype).split('.')[-1]} torch tensor")
    if t.get_device() != device:
        place(t, name, device)
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} has the shape {r} x {c}; "
                         f"{'any' if rows is None else rows} x {'any' if cols is None else cols} "
                         "is needed")
    s0, s1 = t.stride()
    if s1 == 1 and 0 < c <= s0 <= INT_MAX and 0 < r <= INT_MAX:
        return s0
    if r == 0 or c == 0:
        return max(c, 1)
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} needs a unit column stride")
    if r > 1 and s0 < c:
        raise ValueError(f"{name}: row stride {s0} is shorter than a row ({c}); "
                         "broadcast or overlapping views are not supported")
    ld = s0 if r > 1 else c
    if ld > INT_MAX or r > INT_MAX:
        raise ValueError(f"{name} is too large: {r} rows, row stride {ld}")
    return ld


def place(t, name, device):
    """The number of the GPU t lives on; raises unless it is on one (on `device`, if
    given)."""
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if device is not None and index != device:
        raise ValueError(f"{name} lives on GPU {index}, the other tensors on GPU {device}")
    return index


def dense(t, shape, name, dtype, device):
    """Raises unless t is a contiguous tensor of this shape and type on GPU number
    `device` (None: any)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {str(dtype).split('.')[-1]} torch tensor")
    if t.get_device() != device:
        place(t, name, device)
    if t.shape != shape:
        raise ValueError(f"{name} has the shape {tuple(t.shape)}; {tuple(shape)} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def launch_stream(stream, index):
    """`stream`, which a caller passed, as a torch stream; raises where it says that it is
    not one of GPU number `index`, whose memory a kernel on it could not reach."""
    device = getattr(stream, "device", None)
    if device is not None and device.index != index:
        raise ValueError(f"the stream is one of {device}, the tensors live on GPU {index}")
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if not stream.cuda_stream:  # ExternalStream would make a new one of the null handle
        return torch.cuda.default_stream(index)
    return torch.cuda.ExternalStream(stream.cuda_stream, device=index)


def new(like, shape, stream, dtype=None):
    """A tensor on like's GPU, of its type unless `dtype` is given, for a call on `stream`
    to write.  torch's allocator hands memory freed on a stream to the next allocation for
    that stream without waiting for the work there that still uses it.  So what a
    stream that is passed in is to write is allocated for that stream, and marked as
    used on the current one, where the caller reads and frees it."""
    if stream is None:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    index = like.get_device()
    stream = launch_stream(stream, index)
    if stream.cuda_stream == raw_stream(index):
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream(index)
    if index == current_device():
        # as torch.cuda.stream() does, without its context: 6.4 instead of 9.9 us
        torch.cuda.set_stream(stream)
        try:
            t = like.new_empty(shape, dtype=dtype)
        finally:
            torch.cuda.set_stream(current)
    else:
        with torch.cuda.stream(stream):
            t = like.new_empty(shape, dtype=dtype)
    t.record_stream(current)
    return t


_entries = {}   # library functions by name, looked up once


def call(entry, index, stream, *args):
    """entry(*args, stream) on GPU number `index`, on `stream` (default: torch's
    current stream there)."""
    f = _entries.get(entry)
    if f is None:
        f = _entries[entry] = getattr(lib(), entry)
    # the current stream's handle without a Stream object: 0.1 instead of 1.9 us
    handle = raw_stream(index) if stream is None else launch_stream(stream, index).cuda_stream
    if index == current_device():
        status = f(*args, handle)
    else:
        with torch.cuda.device(index):
            status = f(*args, handle)
    if status != 0:
        raise SgemmError(status, entry)
