"""Low-rank adapters of many requests beside a shared projection: binding of
f16_lora (``include/w4a16.h``)::

    adapters = Adapters(a, b, scale, columns=(2048, 256, 256))   # once per projection
    y = w4_gemv(x, ...)                                          # or w4_gemm, f16_gemm
    f16_lora(x, adapters, ids, y)                                # ids int32 [rows], negative: none
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _dev, _here, _on, _stream, lib

__all__ = ["Adapters", "f16_lora", "lora_workspace", "lora_workspace_bytes"]

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class _Adapters(ctypes.Structure):
    _fields_ = [("a", _P), ("b", _P), ("scale", _P), ("a_adapter", _L), ("b_adapter", _L), ("adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("slices", ctypes.c_int32),
                ("columns", ctypes.c_int32 * 4)]


lib.f16_lora.argtypes = [_P, _L, _P, _L, _P, _L, _P, _P, _I, _P, ctypes.c_size_t, _P]
lib.f16_lora_workspace_bytes.argtypes = [_P, _I]
lib.f16_lora_workspace_bytes.restype = ctypes.c_size_t


def _half(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float16:
        raise TypeError(f"{name} must be a float16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t


def _rows(t: torch.Tensor, name: str, shape):
    """(device pointer, row stride) of a float16 tensor of this shape with contiguous rows."""
    _half(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be [{shape[0]}][{shape[1]}]")
    strides = t.stride()
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), strides[0] if shape[0] > 1 else 8  # (of one row the stride is never used)


class Adapters:
    """The adapters of one projection, checked and marshalled once.  Keeps its tensors;
    their contents may change between calls (an adapter's place taken by another).

    a        float16 [adapters][slices][rank][K], or [adapters][rank][K] for one slice
    b        float16 [adapters][N][rank]
    scale    float32 [adapters], 1 when None
    columns  widths of the slices, which add up to N; one slice of all when None
    """

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor | None = None, columns=None):
        a, b = _half(a, "a"), _half(b, "b")
        if a.dim() == 3:
            a = a.unsqueeze(1)
        if a.dim() != 4 or b.dim() != 3:
            raise ValueError("a must be [adapters][slices][rank][K] and b [adapters][N][rank]")
        n, slices, rank, k = a.shape
        columns = (b.shape[1],) if columns is None else tuple(columns)
        if b.shape[0] != n or b.shape[2] != rank:
            raise ValueError(f"b must be [{n}][N][{rank}]")
        if len(columns) != slices or not 1 <= slices <= 4 or min(columns) < 1 or sum(columns) != b.shape[1]:
            raise ValueError(f"columns must be the widths of 1 to 4 slices, one for each of a's, that add up to {b.shape[1]}")
        for t, name in ((a, "a"), (b, "b")):
            if n > 0 and not t[0].is_contiguous():
                raise ValueError(f"each adapter of {name} must be contiguous")
        if scale is not None and scale.numel() != n:
            raise ValueError(f"scale must be [{n}]")
        self.a, self.b, self.scale = a, b, scale
        self.K, self.N = k, b.shape[1]
        ends = [sum(columns[:i + 1]) for i in range(slices)]
        self.struct = _Adapters(a.data_ptr(), b.data_ptr(),
                                None if scale is None else _dev(scale, "scale", (torch.float32,)),
                                a.stride(0) if n > 1 else 8, b.stride(0) if n > 1 else 8, n, rank, k, self.N, slices,
                                (ctypes.c_int32 * 4)(*ends))
        self.ptr = ctypes.addressof(self.struct)
        self.device = a.device
        self.sized = None  # (rows, workspace bytes) asked last


def lora_workspace_bytes(adapters: Adapters, rows: int) -> int:
    sized = adapters.sized
    if sized is None or sized[0] != rows:
        adapters.sized = sized = rows, int(lib.f16_lora_workspace_bytes(adapters.ptr, rows))
    return sized[1]


def lora_workspace(adapters: Adapters, rows: int) -> torch.Tensor:
    """A workspace for f16_lora with up to this many rows, for calls that do not overlap."""
    return torch.empty(max(lora_workspace_bytes(adapters, rows), 16), dtype=torch.uint8, device=adapters.device)


def f16_lora(x: torch.Tensor, adapters: Adapters, ids: torch.Tensor, y: torch.Tensor, out: torch.Tensor | None = None,
             stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out[m] = y[m] + scale[a] * (x[m] @ A_a.T) @ B_a.T with a = ids[m] (int32; negative: y[m]).
    x float16 [rows][K], y and out [rows][N], any row strides that are multiples of 8 (out's rows apart); out is y itself when None.
    workspace: from lora_workspace; a fresh one is made when None."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    m = ids.numel()
    px, xs = _rows(x, "x", (m, adapters.K))
    _here(x)
    if x.device != adapters.device:
        raise ValueError(f"x is on {x.device}, the adapters on {adapters.device}")
    py, ys = _rows(y, "y", (m, adapters.N))
    po, os = (py, ys) if out is None else _rows(out, "out", (m, adapters.N))
    if workspace is None:
        with _on(stream):
            workspace = lora_workspace(adapters, m)
    _check("f16_lora", lib.f16_lora(px, xs, py, ys, po, os, adapters.ptr, _dev(ids, "ids", (torch.int32,)), m,
                                    _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(), _stream(stream)))
    return y if out is None else out
