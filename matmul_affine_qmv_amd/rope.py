"""Rotary positions of queries and keys: marshalling for qmx_rope (include/qmx.h
says what it computes), and the frequencies that models stretch for long contexts.
"""
from __future__ import annotations

import math

import torch

from .f8 import _HALVES, _MOST, _WHOLE, _check, _current_device, _function, _like, _raw_stream


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 0, low: float = 1.0, high: float = 4.0, fast: float = 32.0,
                     slow: float = 1.0, device="cuda") -> torch.Tensor:
    """Radians a position of each pair, float64 [rotary_dim / 2] on `device`:
    f_i = base ** (-2 i / rotary_dim), and for contexts `factor` times as long as
    the original_length that a model was trained on:

    scaling "linear": f_i / factor.
    scaling "base":   base * factor ** (d / (d - 2)) for the base, which divides the
                      last frequency by factor and leaves the first (d = rotary_dim > 2).
    scaling "bands":  f_i / factor where a turn takes more than original_length / low
                      positions, f_i where it takes less than original_length / high,
                      and between them a blend, linear in turns (low < high).
    scaling "yarn":   f_i / factor and f_i blended linearly in i, between the pairs
                      that make `fast` and `slow` turns in original_length positions
                      (fast > slow); YaRN also scales what it turns by 0.1 ln(factor)
                      + 1 (rope's `scale`).  The published method blends linearly in
                      turns.  Blending in i, from the pair rounded down to the one
                      rounded up, these held to 0 .. rotary_dim - 1 and at least 0.001
                      apart, is what the programs do that models are trained and run
                      with, whose frequencies a model needs."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and at least 2, got {rotary_dim}")
    if not base > 1 or not factor >= 1:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "base", "bands", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'base', 'bands' or 'yarn', got {scaling!r}")
    if scaling in ("bands", "yarn") and original_length < 1:
        raise ValueError(f"scaling {scaling!r} needs original_length")
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling 'base' needs a rotary_dim of at least 4")
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    f = float(base) ** (-2 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if not 0 < low < high:
            raise ValueError("bands need 0 < low < high")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    elif scaling == "yarn":
        if not 0 < slow < fast:
            raise ValueError("yarn needs 0 < slow < fast")

        def pair_of(turns):  # the (fractional) pair that makes so many turns
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        first = max(math.floor(pair_of(fast)), 0)
        last = max(first + 0.001, min(math.ceil(pair_of(slow)), rotary_dim - 1))
        stretched = ((i - first) / (last - first)).clamp(0, 1)
        f = (1 - stretched) * f + stretched * f / factor
    return f.to(device)


def _heads(t, name, shape, dtype, index):
    """Address, token and head stride."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {tuple(shape)} of dtype {dtype} on HIP device {index}")
    token, head, last = t.stride()
    if last != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have a unit last stride")
    return t.data_ptr(), token, head


def rope(q, k, positions, frequencies, *, interleaved=False, scale=1.0, out=None):
    """(q, k) turned by their tokens' positions (qmx_rope).

    q, k: [tokens, heads, head_dim] and [tokens, kv_heads, head_dim] (any strides,
    the last 1), k may be None; positions: int32 [tokens], below 0 for tokens that
    are left as they are; frequencies: float64 [pairs] (rope_frequencies), the first
    2 * pairs elements of a head turn, element i with pairs + i or, interleaved, 2i
    with 2i + 1.  scale: of what turns.  out: the (q, k) to write into, q and k
    themselves to turn them in place.  Returns (q, k), contiguous if made here."""
    code = _HALVES.get(q.dtype)
    if code is None or q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim] in float16 or bfloat16, got {q.dim()}-D {q.dtype}")
    if not q.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    index, shape, dtype = q.get_device(), q.shape, q.dtype
    if index != _current_device():
        with torch.cuda.device(index):
            return rope(q, k, positions, frequencies, interleaved=interleaved, scale=scale, out=out)
    T, heads, D = shape
    if T > _MOST or heads > _MOST or D > _MOST:
        raise ValueError("q must have sizes below 2^31")
    if positions.dtype is not torch.int32 or positions.shape != (T,) or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 vector of {T}")
    if frequencies.dtype is not torch.float64 or frequencies.dim() != 1 or not frequencies.is_contiguous():
        raise ValueError("frequencies must be a contiguous float64 vector")
    pairs = frequencies.shape[0]
    if not 2 <= 2 * pairs <= D:
        raise ValueError(f"frequencies must have 1 to {D // 2} elements, got {pairs}")
    if positions.get_device() != index or frequencies.get_device() != index:
        raise ValueError(f"positions and frequencies must be on {q.device}")
    from_q = _heads(q, "q", shape, dtype, index)
    from_k = to_k = (None, 0, 0)
    kv_heads = 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be [tokens, kv_heads, head_dim]")
        kv_heads = k.shape[1]
        if kv_heads > _MOST:
            raise ValueError("k must have sizes below 2^31")
        from_k = _heads(k, "k", (T, kv_heads, D), dtype, index)
    if out is None:
        q_out, k_out = _like(q, memory_format=_WHOLE), None
        to_q = (q_out.data_ptr(), heads * D, D)
        if k is not None:
            k_out = _like(k, memory_format=_WHOLE)
            to_k = (k_out.data_ptr(), kv_heads * D, D)
    else:
        q_out, k_out = out
        if (k_out is None) != (k is None):
            raise ValueError("out must be as many tensors as q and k")
        to_q = _heads(q_out, "q's out", shape, dtype, index)
        if k is not None:
            to_k = _heads(k_out, "k's out", (T, kv_heads, D), dtype, index)
    _check(_function("qmx_rope")(*from_q, *to_q, heads, *from_k, *to_k, kv_heads, positions.data_ptr(),
                                 frequencies.data_ptr(), T, D, pairs, int(interleaved), scale, code,
                                 _raw_stream(index)), "qmx_rope")
    return q_out, k_out
