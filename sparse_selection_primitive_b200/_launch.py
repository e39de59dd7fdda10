"""What the expert and cache calls share: the launch on the tensors' own device,
and the checks of tensor arguments."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import LapSumError

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def launch(fn, device, *args):
    """Calls the library function with the current stream of ``device`` as its last
    argument, on that device whatever the current one is; raises on an error.

    The device and the stream come from the calls behind torch.cuda.current_device and
    current_stream, which build no Stream; a torch without CUDA does not have them, and the
    package has to be imported there too."""
    index, stream = device.index, torch._C._cuda_getCurrentRawStream
    if index == torch._C._cuda_getDevice():
        code = fn(*args, stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream(index))
    if code != 0:
        raise LapSumError(code, fn.__name__)


def need(x, name: str, dtypes, dim: int, device=None):
    """x must be a CUDA tensor of one of ``dtypes`` with ``dim`` dimensions, on ``device``."""
    if isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in dtypes and x.dim() == dim and \
            (device is None or x.device == device):
        return
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in dtypes:
        kinds = ", ".join(str(d).replace("torch.", "") for d in dtypes)
        raise TypeError(f"{name} must be a CUDA tensor of {kinds}")
    if x.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    raise ValueError(f"{name} is on {x.device}, not on {device}")


def extent(x: torch.Tensor):
    """First and one past the last byte that x's elements span."""
    start, span = x.data_ptr(), 1
    if x.is_contiguous():
        return start, start + x.numel() * x.element_size()
    for n, s in zip(x.shape, x.stride()):
        if n == 0:
            return start, start
        span += (n - 1) * s
    return start, start + span * x.element_size()


def overlap(x: torch.Tensor, y: torch.Tensor) -> bool:
    a, b = extent(x), extent(y)
    return a[0] < b[1] and b[0] < a[1]


def apart(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether x and y are known to share no memory: their extents do not overlap, or they lie
    side by side in one structure (the same steps in their first dimensions, and inside one
    step parts that do not overlap and together are no longer than it)."""
    if not overlap(x, y):
        return True
    steps = []
    for d in range(min(x.dim(), y.dim()) - 1):
        if x.shape[d] != y.shape[d]:
            break
        if x.shape[d] > 1:
            step = x.stride(d) * x.element_size()
            if step != y.stride(d) * y.element_size():
                break
            steps.append((step, x.shape[d]))
        (a0, a1), (b0, b1) = extent(x[(0,) * (d + 1)]), extent(y[(0,) * (d + 1)])
        if a1 <= b0 or b1 <= a0:
            span = max(a1, b1) - min(a0, b0)
            for step, n in sorted(steps):
                if step < span:
                    break
                span += step * (n - 1)
            else:
                return True
    return False


def distinct(x: torch.Tensor) -> bool:
    """Whether no two of x's elements share memory (strides nest without overlap)."""
    if x.is_contiguous():
        return True
    need_stride = 1
    for s, n in sorted((s, n) for n, s in zip(x.shape, x.stride()) if n > 1):
        if s < need_stride:
            return False
        need_stride = s * (n - 1) + need_stride
    return True


def no_tangents(name: str, *tensors):
    """Refuses forward-mode inputs: the library reads their values and would drop their
    tangents unnoticed."""
    if forward_ad._current_level < 0:  # no dual tensors outside a level (unpack_dual's own test)
        return
    if any(forward_ad.unpack_dual(x).tangent is not None for x in tensors):
        raise NotImplementedError(f"{name} has no forward-mode derivative")


def no_gradient(name: str):
    """Refuses tensors that require a gradient: a call without a backward pass must not cut
    a graph unnoticed."""
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no gradient: call it under torch.no_grad() or on "
                           "detached tensors")
