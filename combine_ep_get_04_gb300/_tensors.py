"""Checks on the tensors whose addresses go to the C ABI."""
from __future__ import annotations

import torch


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


def _rows_ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str, rows: int, cols: int) -> tuple[int | None, int]:
    """Address and row stride (in elements) of a [rows, cols] tensor whose rows
    may lie further apart than their length."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr() or None, t.stride(0) if rows > 1 else cols


def _shaped_ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str, shape: tuple) -> int | None:
    """Address of a contiguous tensor of exactly this shape."""
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    return _ptr(t, dtype, name)


def _stream(stream: torch.cuda.Stream | None) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream or None
