"""Argument checks and the call itself, shared by ``experts`` and ``w4``.

A decode step's kernels take a few microseconds, so a call must not spend more
than that on its arguments: one test per tensor decides whether all is well,
and only a tensor that fails it is looked at again for the message.
"""

import torch

from .binding import _check, _need_cuda, _need_shape


def device_of(t, name):
    """Index of the HIP device that a tensor is on; others have to be there too."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t.get_device()


def need(dev, t, name, dtype, shape):
    """Refuses `t` unless it is a contiguous tensor of this dtype and shape on
    device `dev`, all of which the library relies on."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        return
    _need_cuda(t, name, dtype)
    _need_shape(t, name, shape)
    raise ValueError(f"{name} must be on cuda:{dev} as the other tensors, got {t.device}")


def call(dev, fn, *args):
    """fn(*args, stream) on device `dev` and its current stream; a kernel can
    only be launched on a stream of the current device."""
    if torch.cuda.current_device() == dev:
        _check(fn(*args, _raw_stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _raw_stream(dev)))


def _public_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without the Python object around it, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
