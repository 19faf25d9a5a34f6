"""Rules of token selection: binding of w4_logit_rules and w4_token_counts
(``include/w4a16.h``).

A decoding loop over requests in slots::

    counts = TokenCounts.new(slots, vocabulary)        # once
    token_counts_add(counts, slots, prompts, offsets, prompt=True, reset=True)   # requests take their slots
    rules = LogitRules(counts, slots, repetition, presence, frequency, biases, allowed)   # once per batch
    idx, val = lm_head_argmax_topk(x, ..., rules=rules)      # each step
    token_counts_add(counts, slots, chosen)                  # int32 [rows], idx[:, 0] where greedy

Everything but the shapes is read on the device when the kernels run: a
captured graph can be replayed with other slots, penalties, masks and biases.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _dev, _here, _stream, lib

__all__ = ["LogitRules", "TokenCounts", "token_counts_add"]

_P, _L = ctypes.c_void_p, ctypes.c_int64
_PROMPT, _RESET = 1, 2


class _Rules(ctypes.Structure):
    _fields_ = [("counts", _P), ("counts_stride", _L), ("slot", _P), ("repetition", _P), ("presence", _P),
                ("frequency", _P), ("bias_offsets", _P), ("bias_tokens", _P), ("bias_values", _P), ("allowed", _P),
                ("allowed_stride", _L), ("slots", ctypes.c_int32), ("bias_entries", ctypes.c_int32)]


class TokenCounts:
    """The tokens that requests have seen, over an int16 tensor [slots][vocabulary]
    (rows may be wider apart): bit 15 "in the prompt", the low 15 bits the times
    in the output.  Keeps the tensor."""

    def __init__(self, counts: torch.Tensor):
        if not isinstance(counts, torch.Tensor) or counts.dtype is not torch.int16:
            raise TypeError("counts must be an int16 tensor")
        if not counts.is_cuda:
            raise ValueError("counts must be a CUDA tensor")
        if counts.dim() != 2 or (counts.shape[1] > 1 and counts.stride(1) != 1):
            raise ValueError("counts must be [slots][vocabulary] with contiguous rows")
        self.counts = counts
        self.slots, self.vocabulary = counts.shape
        self.stride = counts.stride(0) if self.slots > 1 else max(self.vocabulary, 1)
        self.ptr = counts.data_ptr()

    @classmethod
    def new(cls, slots: int, vocabulary: int, device="cuda") -> "TokenCounts":
        """Zeroed counts, rows on 16 bytes (read fastest)."""
        wide = (vocabulary + 7) // 8 * 8
        return cls(torch.zeros(slots, wide, dtype=torch.int16, device=device)[:, :vocabulary])


def token_counts_add(counts: TokenCounts, slots: torch.Tensor, tokens: torch.Tensor,
                     offsets: torch.Tensor | None = None, prompt: bool = False, reset: bool = False,
                     stream=None) -> None:
    """Count tokens (int32, one after the other; negative ones are skipped) in their
    sequences' rows: sequence b, in slot slots[b] (int32; negative: none), has the
    tokens offsets[b] .. offsets[b + 1] - 1 (int32 [batch + 1]), or token b where
    offsets is None.  prompt: they are a prompt's, else the output's.  reset: the
    rows are cleared before (requests take their slots; of equal ones the last takes it, and device_status reports it)."""
    _here(counts.counts)
    batch = slots.numel()
    if offsets is not None and offsets.numel() != batch + 1:
        raise ValueError("offsets must be [batch + 1]")
    if offsets is None and tokens.numel() != batch:
        raise ValueError("without offsets, tokens must be [batch]")
    ints = (torch.int32,)
    _check("token_counts_add",
           lib.w4_token_counts(counts.ptr, counts.stride, counts.slots, counts.vocabulary, _dev(slots, "slots", ints),
                               _dev(tokens, "tokens", ints), None if offsets is None else _dev(offsets, "offsets", ints),
                               batch, tokens.numel(), (_PROMPT if prompt else 0) | (_RESET if reset else 0),
                               _stream(stream)))


class LogitRules:
    """Rules of a batch of rows, checked and marshalled once for
    lm_head_argmax_topk(rules=); any part may be None.  Keeps its tensors.

    counts, slots          TokenCounts and int32 [rows]: the slot of each row (negative: no penalties)
    repetition             float32 [rows]: seen tokens' logits are divided (positive) or multiplied by it
    presence, frequency    float32 [rows]: taken off the logits of output tokens, once, and per occurrence
    biases                 (offsets int32 [rows + 1], tokens int32, values float32): added to row r's tokens
                           offsets[r] .. offsets[r + 1] - 1, one entry after the other
    allowed                int32 [rows][words], bit n % 32 of word n // 32: token n can be selected
    """

    def __init__(self, counts: TokenCounts | None = None, slots: torch.Tensor | None = None,
                 repetition: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                 frequency: torch.Tensor | None = None, biases=None, allowed: torch.Tensor | None = None):
        self.struct = s = _Rules()
        self.tensors = [counts, slots, repetition, presence, frequency, biases, allowed]
        self.rows, self.counts, self.words = None, counts, None
        if (counts is None) != (slots is None):
            raise ValueError("counts and slots come together")
        if counts is None and not (repetition is None and presence is None and frequency is None):
            raise ValueError("penalties need counts")
        if counts is not None:
            s.counts, s.counts_stride, s.slots = counts.ptr, counts.stride, counts.slots
            s.slot = self._row(slots, "slots", torch.int32)
            for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
                if t is not None:
                    setattr(s, name, self._row(t, name, torch.float32))
        if biases is not None:
            offsets, tokens, values = biases
            if tokens.numel() != values.numel():
                raise ValueError("bias tokens and values must be as many")
            s.bias_offsets = self._row(offsets, "bias offsets", torch.int32, 1)
            if tokens.numel():
                s.bias_tokens = _dev(tokens, "bias tokens", (torch.int32,))
                s.bias_values = _dev(values, "bias values", (torch.float32,))
            else:  # (no entry is read; empty tensors have no address)
                s.bias_tokens = s.bias_values = s.bias_offsets
            s.bias_entries = tokens.numel()
        if allowed is not None:
            if allowed.dim() != 2:
                raise ValueError("allowed must be [rows][words]")
            s.allowed = self._row(allowed, "allowed", torch.int32, rows=allowed.shape[0])
            s.allowed_stride = self.words = allowed.shape[1]
        self.ptr = ctypes.addressof(s)

    def _row(self, t: torch.Tensor, name: str, dtype, more: int = 0, rows: int | None = None) -> int:
        pointer = _dev(t, name, (dtype,))
        n = t.numel() - more if rows is None else rows
        if self.rows is None:
            self.rows = n
        if n != self.rows or n < 1:
            raise ValueError(f"{name} is for {n} rows, not {self.rows}")
        return pointer

    def _of(self, rows: int, vocabulary: int) -> int:
        """The struct's address, for a call on these rows and tokens."""
        if self.rows is not None and rows != self.rows:
            raise ValueError(f"rules of {self.rows} rows for {rows}")
        if self.counts is not None and self.counts.vocabulary != vocabulary:
            raise ValueError(f"counts of {self.counts.vocabulary} tokens for {vocabulary}")
        if self.words is not None and self.words < (vocabulary + 31) // 32:
            raise ValueError(f"allowed needs {(vocabulary + 31) // 32} words a row")
        return self.ptr
