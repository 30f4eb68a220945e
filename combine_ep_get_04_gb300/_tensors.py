"""Checks on the tensors whose addresses go to the C ABI."""
from __future__ import annotations

import torch


# The raw handle of a device's current stream, without a Stream object around it.
# (A torch without CUDA has neither: the package can be imported there all the same.)
_raw_stream, _current_device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
# Whether a tensor may be on another device than the current one, on which the kernels run.
_SEVERAL = _current_device is not None and torch.cuda.device_count() > 1


def _on_current(t: torch.Tensor, name: str) -> None:
    if _SEVERAL and t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "tensor",
         numel: int | None = None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr() or None


def _rows_ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str, shape: tuple[int, int]) -> tuple[int | None, int]:
    """Address and row stride (in elements) of a [rows, cols] tensor whose rows
    may lie further apart than their length."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.shape == shape and t.is_cuda:
        ld, step = t.stride()
        if step == 1 or shape[1] <= 1:
            if _SEVERAL:
                _on_current(t, name)
            return t.data_ptr() or None, ld if shape[0] > 1 else shape[1]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous rows")


def _shaped_ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str, shape: tuple) -> int | None:
    """Address of a contiguous tensor of exactly this shape."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        if _SEVERAL:
            _on_current(t, name)
        return t.data_ptr() or None
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    return _ptr(t, dtype, name)


def _int32(n: int, name: str) -> int:
    """A size that the C ABI takes as 32 bits, which ctypes would cut to its low ones."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} = {n} does not fit 32 bits")
    return n


def _stream(stream: torch.cuda.Stream | None) -> int | None:
    return (_raw_stream(_current_device()) if stream is None else stream.cuda_stream) or None


def _empty(shape, dtype: torch.dtype, device: torch.device, stream: torch.cuda.Stream | None) -> torch.Tensor:
    """Memory that is written on `stream`.  Of that stream's own: what the
    allocator has for the current one may still be read there, and would go
    back to it while `stream` writes."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)
