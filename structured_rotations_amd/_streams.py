"""Streams and memory of a call: which stream allocates what the call makes,
and which streams the allocator has to wait for before it gives the memory of
the call's tensors to others.
"""
from __future__ import annotations

import torch

# torch's own short way to the handle, where this build has it (a decoding step
# is a few calls of 5 us each; the Stream object alone costs 1 us)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def new(shape, dtype, like, stream):
    """A new tensor beside `like`.  The allocator hands out memory that earlier
    work of the allocating stream may still use, so with an explicit stream,
    which the call's work follows, it is that stream that allocates."""
    if stream is None or like.device.type == "cpu":
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def stream_of(stream, dev, tensors):
    """The given stream's handle, or that of the current stream.  Any of the
    call's tensors may be dropped when the call returns: the allocator is told
    that both streams use them."""
    if stream is None:
        return _current_stream(dev)
    here = torch.cuda.current_stream(dev)
    if stream.cuda_stream != here.cuda_stream:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
                t.record_stream(here)
    return stream.cuda_stream
