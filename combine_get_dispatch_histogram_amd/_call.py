"""Pointer marshalling and argument checks shared by the package's calls."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib


class _Args:
    """Pointer marshalling for one library call: every tensor it passes must be
    a contiguous device tensor on one and the same GPU, and the call runs with
    that GPU current and on its current stream."""

    def __init__(self):
        self.dev = None

    def _see(self, t: torch.Tensor) -> None:
        if not t.is_cuda:
            raise ValueError("miep expects device tensors")
        if self.dev is None:
            self.dev = t.device
        elif t.device != self.dev:
            raise ValueError("miep expects every tensor of a call on one device (%s and %s)" % (self.dev, t.device))

    def p(self, t: Optional[torch.Tensor]):
        if t is None:
            return None
        self._see(t)
        if not t.is_contiguous():
            raise ValueError("miep expects contiguous tensors")
        return t.data_ptr()

    def handle(self, h) -> None:
        for t in h.tensors():
            self.p(t)


# The current stream of a device as an integer, without building a Stream
# object for every call (10 us a call became 6, more than a small kernel takes).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(a: _Args, name: str, *args) -> None:
    if a.dev is None:
        raise ValueError("miep call without device tensors")
    call = getattr(_lib.load(), name)
    index = a.dev.index
    if torch.cuda.current_device() == index:
        _lib.check(call(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(a.dev):
            _lib.check(call(*args, _raw_stream(index)))


def _want(t: Optional[torch.Tensor], name: str, dtype, shape=None):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def check_status(status: torch.Tensor) -> None:
    """Read a dispatch's device status word (synchronous: waits for the
    current stream); raises MiepError(MIEP_ECAPACITY) if the receive rows
    exceeded their fixed capacity."""
    _want(status, "status", torch.int32, (1,))
    a = _Args()
    _run(a, "miep_check_status", a.p(status))
