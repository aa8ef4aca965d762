"""Pointer marshalling and argument checks shared by the package's calls."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib


class _Args:
    """Pointer marshalling for one library call: every tensor it passes must be
    a contiguous device tensor on one and the same GPU, and the call runs with
    that GPU current and on its current stream."""

    __slots__ = ("dev", "index", "astray")

    def __init__(self):
        self.dev = self.index = self.astray = None

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
        index = t.get_device()                             # -1 on the host
        if index != self.index:
            self._see(t)
            self.index = index
        if not t.is_contiguous():
            raise ValueError("miep expects contiguous tensors")
        return t.data_ptr()

    def arg(self, t: torch.Tensor, name: str, dtype, shape=None) -> int:
        """_want and p in one step.  Where the tensor lies is looked at by _run
        (``astray``), so that wrong types and shapes are reported first."""
        if t.dtype != dtype or (shape is not None and t.shape != shape):
            _want(t, name, dtype, shape)
        index = t.get_device()                             # -1 on the host
        if index != self.index:
            if self.index is None and index >= 0:
                self._see(t)
                self.index = index
            elif self.astray is None:
                self.astray = t
        if not t.is_contiguous():
            raise ValueError("miep expects contiguous tensors")
        return t.data_ptr()

    def opt(self, t: Optional[torch.Tensor], name: str, dtype, shape=None) -> Optional[int]:
        return None if t is None else self.arg(t, name, dtype, shape)

    def handle(self, h) -> None:
        for t in h.tensors():
            self.p(t)


# The current stream of a device as an integer, without building a Stream
# object for every call, and the current device without torch's check that the
# GPU is set up, as tensors on it show (a small swiglu_fp8 call took 10.1 us, of
# which its launch is 3.8; 7.4 with the first, 6.8 with both, 6.1 with `arg`).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(a: _Args, name: str, *args) -> None:
    if a.astray is not None:
        a._see(a.astray)
    if a.dev is None:
        raise ValueError("miep call without device tensors")
    call = getattr(_lib.load(), name)
    index = a.index
    if _current_device() == index:
        _lib.check(call(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            _lib.check(call(*args, _raw_stream(index)))


def _want(t: Optional[torch.Tensor], name: str, dtype, shape=None):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def check_status(status: torch.Tensor) -> None:
    """Read a dispatch's device status word (synchronous: waits for the
    current stream); raises MiepError(MIEP_ECAPACITY) if the receive rows
    exceeded their fixed capacity."""
    _want(status, "status", torch.int32, (1,))
    a = _Args()
    _run(a, "miep_check_status", a.p(status))
