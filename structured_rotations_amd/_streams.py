"""Streams, devices and memory of a call: which GPU it goes to, which stream
allocates what it makes, and which streams the allocator has to wait for before
it gives the memory of the call's tensors to others.
"""
from __future__ import annotations

import torch

from ._lib import check

# torch's own short way to the handle, where this build has it (a decoding step
# is a few calls of 5 us each; the Stream object alone costs 1 us)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def new(shape, dtype, like, stream):
    """A new tensor beside `like`.  The allocator hands out memory that earlier
    work of the allocating stream may still use, so with an explicit stream,
    which the call's work follows, it is that stream that allocates."""
    if stream is None or like.device.type == "cpu":
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def new_like(like, stream):
    """torch.empty_like, allocated as new() does."""
    if stream is None or like.device.type == "cpu":
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        return torch.empty_like(like)


def stream_of(stream, dev, tensors):
    """The given stream's handle, or that of the current stream.  Any of the
    call's tensors may be dropped when the call returns: the allocator is told
    that both streams use them."""
    if stream is None:
        return _current_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on GPU {stream.device.index}, the arguments on GPU {dev}")
    here = torch.cuda.current_stream(dev)
    if stream.cuda_stream != here.cuda_stream:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
                t.record_stream(here)
    return stream.cuda_stream


def launch(fn, stream, dev, tensors, *args):
    """fn(*args, stream handle) on GPU dev, which holds every tensor: the
    library launches on the current GPU, and handle 0 is that one's default
    stream."""
    handle = stream_of(stream, dev, tensors)
    if dev == _current_device():
        check(fn(*args, handle))
    else:
        with torch.cuda.device(dev):
            check(fn(*args, handle))
