"""Attention with a paged key/value cache: binding of f16_rope, f16_kv_append
(both with norms of the heads) and f16_attention (``include/w4a16.h``).

A decode or prefill step of a layer, between its q/k/v projections and its o
projection::

    cache = KVCache(k_pages, v_pages)            # once: [pages][page_size][heads][dim]
    rope = Rope(*rope_turns(128, base=1e6))      # once
    ws = attention_workspace(cache, q_heads, max_q_len)   # once
    batch = KVBatch(block_table, q_offsets, kv_lens, total_q, max_q_len)  # once per step
    q = f16_kv_append(k, v, cache, batch, rope=rope, q=q, y=q)
    y = f16_attention(q, cache, batch, workspace=ws)

Activations are float16 [tokens][heads][dim] with any strides whose heads
start on 16 bytes (views of one projection's output among them).  The batch's
index tensors are read on the device when the kernels run.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _dev, _here, _on, _result, _stream, lib

__all__ = ["HeadNorm", "KVBatch", "KVCache", "Rope", "attention_workspace", "attention_workspace_bytes", "f16_attention",
           "f16_kv_append", "f16_rope", "rope_turns"]

_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", _P), ("q_offsets", _P), ("kv_lens", _P), ("batch", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_strides", _L * 3), ("v_strides", _L * 3),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("box_rows", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k_map", ctypes.c_uint64 * 16), ("v_map", ctypes.c_uint64 * 16), ("k_wide", ctypes.c_uint64 * 16),
                ("v_wide", ctypes.c_uint64 * 16)]


class _Rotation(ctypes.Structure):
    _fields_ = [("turns", _P), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", _F)]


class _Norm(ctypes.Structure):
    _fields_ = [("weight", _P), ("eps", _F)]


lib.f16_kv_cache_init.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I]
lib.f16_rope.argtypes = [_P, _L, _L, _P, _L, _L, _P, _P, _I, _I, _I, _P]
lib.f16_kv_append.argtypes = [_P, _L, _L, _P, _L, _L, _P, _P, _P, _P, _P, _L, _L, _P, _L, _L, _I, _P]
lib.f16_rope_ex.argtypes = [_P, _L, _L, _P, _L, _L, _P, _P, _P, _I, _I, _I, _P]
lib.f16_kv_append_ex.argtypes = [_P, _L, _L, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, _L, _L, _P, _L, _L, _I, _P]
lib.f16_attention.argtypes = [_P, _L, _L, _P, _L, _L, _P, _I, _F, _I, _I, _P, _P, _P, _Z, _P]
lib.f16_attention_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.f16_attention_workspace_bytes.restype = _Z


def _heads(t: torch.Tensor, name: str):
    """(device pointer, token stride, head stride) of a float16 [tokens][heads][dim] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.float16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][dim]")
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"the dim elements of {name} must be contiguous")
    # The stride of a dimension of one entry is never used; any value torch keeps there will do.
    return t.data_ptr(), (st if n > 1 else 8), (sh if h > 1 else 8)


def _ints(t: torch.Tensor, name: str) -> int:
    return _dev(t, name, (torch.int32,))


def rope_turns(rot: int, base: float = 10000.0, method: str | None = None, stretch: float = 1.0,
               original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, low: float = 1.0,
               high: float = 4.0, device="cuda"):
    """(turns int64 [rot / 2], factor), the first arguments of Rope, for angles
    theta_i = base ** (-2 i / rot) per position and, with method, for a context
    `stretch` times the original one:

    None      theta_i;
    "linear"  theta_i / stretch;
    "ntk"     base * stretch ** (rot / (rot - 2)) in place of base;
    "yarn"    theta_i where a pair turns more than beta_fast times in
              original_len positions, theta_i / stretch where fewer than
              beta_slow times, linear in i between the whole i at or beyond
              these (within 0 .. rot - 1, past the last pair where it still
              turns more often); factor 0.1 ln stretch + 1;
    "bands"   theta_i for wavelengths below original_len / high, theta_i /
              stretch above original_len / low, interpolated in
              original_len / wavelength between.
    """
    if rot < 8 or rot % 8 != 0:
        raise ValueError("rot must be a positive multiple of 8")
    if not stretch > 0:
        raise ValueError("stretch must be positive")
    if method not in (None, "linear", "ntk", "yarn", "bands"):
        raise ValueError(f"unknown method {method!r}")
    if method in ("yarn", "bands") and original_len < 1:
        raise ValueError(f"method {method!r} needs original_len")
    factor = 1.0
    if method == "ntk":
        base = base * stretch ** (rot / (rot - 2))
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if method == "linear":
        theta = [t / stretch for t in theta]
    elif method == "yarn":
        def index(turns):  # of the pair that turns so many times over the original context
            return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        # (Past the last pair, rot // 2 - 1, where every pair turns more than beta_slow times.)
        lo, hi = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
        theta = [t * (1 - r) + t / stretch * r for t, r in zip(theta, ramp)]
        factor = 0.1 * math.log(stretch) + 1.0
    elif method == "bands":
        def band(t):
            mix = (original_len * t / (2 * math.pi) - low) / (high - low)
            mix = min(max(mix, 0.0), 1.0)
            return t * mix + t / stretch * (1 - mix)
        theta = [band(t) for t in theta]
    turns = [round(t / (2 * math.pi) * 2.0**64) % 2**64 for t in theta]
    turns = [t - 2**64 if t >= 2**63 else t for t in turns]
    return torch.tensor(turns, dtype=torch.int64, device=device), factor


class Rope:
    """A rotation of positions: pair i of a head's first 2 * len(turns) elements
    turns by position * turns[i] / 2**64 of a full turn and is scaled by
    factor; pairs are (2i, 2i + 1) when interleaved, else (i, i + len(turns))."""

    def __init__(self, turns: torch.Tensor, factor: float = 1.0, interleaved: bool = False):
        self.turns = turns
        self.rot = 2 * turns.numel()
        self.struct = _Rotation(_dev(turns, "turns", (torch.int64,)), self.rot, 1 if interleaved else 0, factor)
        self.ptr = ctypes.addressof(self.struct)


class HeadNorm:
    """A norm of heads, before their rotation: x * weight / sqrt(mean x**2 + eps)
    over a head's elements.  weight: float32 [dim] on the GPU (a float16 or
    bfloat16 one is widened once, here, on the current stream)."""

    def __init__(self, weight: torch.Tensor, eps: float = 1e-6):
        if isinstance(weight, torch.Tensor) and weight.dtype in (torch.float16, torch.bfloat16):
            weight = weight.float()
        pointer = _dev(weight, "weight", (torch.float32,))
        if weight.dim() != 1:
            raise ValueError("weight must be [dim]")
        self.weight, self.eps, self.dim = weight, eps, weight.numel()
        self.struct = _Norm(pointer, eps)
        self.ptr = ctypes.addressof(self.struct)

    def _of(self, dim: int) -> int:
        """The descriptor's address, for heads of dim elements."""
        if dim != self.dim:
            raise ValueError(f"a norm of {self.dim} elements for heads of {dim}")
        return self.ptr


class KVCache:
    """A paged cache over k and v, float16 [pages][page_size][heads][dim] with any
    order of strides (a permuted view of [pages][heads][page_size][dim] is
    fine): checked and described once, for every later call.  Keeps k and v."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        strides = []
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.float16:
                raise TypeError(f"{name} must be a float16 tensor")
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dim() != 4 or t.shape != k.shape:
                raise ValueError("k and v must be [pages][page_size][heads][dim] of one shape")
            if t.stride(3) != 1 and t.shape[3] > 1:
                raise ValueError(f"the dim elements of {name} must be contiguous")
            strides.append((_L * 3)(*(t.stride(i) if t.shape[i] > 1 else 8 for i in range(3))))
        self.k, self.v = k, v
        self.num_pages, self.page_size, self.heads, self.head_dim = k.shape
        self.struct = _Cache()
        self.ptr = ctypes.addressof(self.struct)
        _check("f16_kv_cache_init",
               lib.f16_kv_cache_init(self.ptr, k.data_ptr(), v.data_ptr(), strides[0], strides[1], *k.shape))


class KVBatch:
    """The sequences of one step.

    block_table  int32 [batch][pages]: page of each page_size positions of a sequence
    q_offsets    int32 [batch + 1]: sequence b has the new tokens q_offsets[b] .. q_offsets[b + 1] - 1
    kv_lens      int32 [batch]: its tokens in the cache, the new ones (its last) included
    total_q      tokens of the q, k and v tensors
    max_q_len    the most new tokens of one sequence

    Checked and marshalled once, for every layer of the step; the tensors'
    contents may change between calls (a captured graph replayed)."""

    def __init__(self, block_table: torch.Tensor, q_offsets: torch.Tensor, kv_lens: torch.Tensor, total_q: int,
                 max_q_len: int):
        if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32:
            raise TypeError("block_table must be an int32 tensor")
        if not block_table.is_cuda:
            raise ValueError("block_table must be a CUDA tensor")
        n = kv_lens.numel()
        if block_table.dim() != 2 or block_table.shape[0] != n or q_offsets.numel() != n + 1:
            raise ValueError("block_table must be [batch][pages], q_offsets [batch + 1] and kv_lens [batch]")
        pages = block_table.shape[1]
        if pages > 1 and block_table.stride(1) != 1:
            raise ValueError("the rows of block_table must be contiguous")
        self.tensors = (block_table, q_offsets, kv_lens)
        self.total_q, self.max_q_len = total_q, max_q_len
        self.struct = _Batch(block_table.data_ptr(), _ints(q_offsets, "q_offsets"), _ints(kv_lens, "kv_lens"), n,
                             pages, block_table.stride(0) if n > 1 else pages, total_q, max_q_len)
        self.ptr = ctypes.addressof(self.struct)


def f16_rope(x: torch.Tensor, rope: Rope | None, positions: torch.Tensor | None = None, y: torch.Tensor | None = None,
             stream=None, norm: HeadNorm | None = None) -> torch.Tensor:
    """y[t][h] = x[t][h] turned to positions[t] (int32; token t is at position t
    when None), normed before with norm (rope may be None then).  y may be x."""
    px, xt, xh = _heads(x, "x")
    _here(x)
    if y is None:
        y = _result(x.shape, x.device, stream)
    py, yt, yh = _heads(y, "y")
    n, h, d = x.shape
    if y.shape != x.shape:
        raise ValueError("y must have the shape of x")
    if positions is not None and positions.numel() != n:
        raise ValueError("positions must be [tokens]")
    pp = None if positions is None else _ints(positions, "positions")
    if norm is None and rope is not None:
        status = lib.f16_rope(px, xt, xh, py, yt, yh, pp, rope.ptr, n, h, d, _stream(stream))
    else:
        status = lib.f16_rope_ex(px, xt, xh, py, yt, yh, pp, None if rope is None else rope.ptr,
                                 None if norm is None else norm._of(d), n, h, d, _stream(stream))
    _check("f16_rope", status)
    return y


def f16_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, batch: KVBatch, rope: Rope | None = None,
                  q: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  positions: torch.Tensor | None = None, stream=None, q_norm: HeadNorm | None = None,
                  k_norm: HeadNorm | None = None) -> torch.Tensor | None:
    """Write the new tokens' k (rotated) and v [total_q][heads][dim] into the cache;
    returns the rotated q in y (None without q).  positions: int32 [total_q]
    for the rotation, where they are not those in the cache.  q_norm, k_norm:
    norms of the query and the key heads, before they are rotated.  y may be q."""
    pk, kt, kh = _heads(k, "k")
    _here(k)
    pv, vt, vh = _heads(v, "v")
    n, d = batch.total_q, cache.head_dim
    if k.shape != (n, cache.heads, d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{n}][{cache.heads}][{d}]")
    if positions is not None and positions.numel() != n:
        raise ValueError("positions must be [total_q]")
    pq = py = None
    qt = qh = yt = yh = hq = 0
    if q is not None:
        pq, qt, qh = _heads(q, "q")
        if y is None:
            y = _result(q.shape, q.device, stream)
        py, yt, yh = _heads(y, "y")
        hq = q.shape[1]
        if q.shape[0] != n or q.shape[2] != d or y.shape != q.shape:
            raise ValueError(f"q and y must be [{n}][heads][{d}]")
    elif y is not None or q_norm is not None:
        raise ValueError("y is the rotated q, and q_norm norms it: they need q")
    pr = None if rope is None else rope.ptr
    pp = None if positions is None else _ints(positions, "positions")
    if q_norm is None and k_norm is None:
        status = lib.f16_kv_append(pk, kt, kh, pv, vt, vh, cache.ptr, batch.ptr, pr, pp, pq, qt, qh, py, yt, yh, hq,
                                   _stream(stream))
    else:
        status = lib.f16_kv_append_ex(pk, kt, kh, pv, vt, vh, cache.ptr, batch.ptr, pr, pp,
                                      None if q_norm is None else q_norm._of(d), None if k_norm is None else k_norm._of(d),
                                      pq, qt, qh, py, yt, yh, hq, _stream(stream))
    _check("f16_kv_append", status)
    return y


def attention_workspace_bytes(q_heads: int, kv_heads: int, head_dim: int, max_q_len: int) -> int:
    return int(lib.f16_attention_workspace_bytes(q_heads, kv_heads, head_dim, max_q_len))


def attention_workspace(cache: KVCache, q_heads: int, max_q_len: int) -> torch.Tensor:
    """A zero-filled workspace for f16_attention on this cache with up to
    max_q_len new tokens of a sequence (reusable by every later call that needs
    no more).  Filled on the current stream: calls on another one have to come after it."""
    need = attention_workspace_bytes(q_heads, cache.heads, cache.head_dim, max_q_len)
    return torch.zeros(max(need, 16), dtype=torch.uint8, device=cache.k.device)


def f16_attention(q: torch.Tensor, cache: KVCache, batch: KVBatch, y: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, scale: float | None = None, causal: bool = True, window: int = 0,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t][h]: attention of q [total_q][heads][dim] over the positions of its
    sequence in the cache up to its own (all of them with causal False; the
    last `window` of them where that is not 0).  scale: 1 / sqrt(dim) when
    None.  lse: float32 [total_q][heads], receives log sum exp of the scaled
    scores.  workspace: from attention_workspace (zero-filled once, then
    reused); a fresh one is made when None."""
    pq, qt, qh = _heads(q, "q")
    _here(q)
    n, h, d = q.shape
    window = max(min(window, 2**31 - 1), -1)  # (passed as 32 bits; every position is below, a negative one is refused)
    if y is None:
        y = _result(q.shape, q.device, stream)
    py, yt, yh = _heads(y, "y")
    if n != batch.total_q or d != cache.head_dim or y.shape != q.shape:
        raise ValueError(f"q and y must be [{batch.total_q}][heads][{cache.head_dim}]")
    if lse is not None and lse.shape != (n, h):
        raise ValueError(f"lse must be [{n}][{h}]")
    if workspace is None:
        with _on(stream):
            workspace = attention_workspace(cache, h, batch.max_q_len)
    _check("f16_attention",
           lib.f16_attention(pq, qt, qh, py, yt, yh, None if lse is None else _dev(lse, "lse", (torch.float32,)), h,
                             d**-0.5 if scale is None else scale, 1 if causal else 0, window, cache.ptr, batch.ptr,
                             _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(), _stream(stream)))
    return y
