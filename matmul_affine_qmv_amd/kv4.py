"""The paged 4-bit key/value cache: marshalling for qmx_kv_maps, qmx_kv4_write,
qmx_kv4_read and qmx_kv4_attention (include/qmx.h says what they compute).

As in the package itself, every function checks its tensors, allocates what is
not given and calls the C ABI on torch's current HIP stream; nothing here
synchronises or copies to the host, so a step can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _WORD_DTYPES, QMX_BF16, QMX_F16, _check, _ptr, _stream, lib

_HALVES = {torch.float16: QMX_F16, torch.bfloat16: QMX_BF16}


class _CCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_sb", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_sb", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("group_size", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class KvMaps(NamedTuple):
    """What kv_maps writes, int32 tensors: query_offsets [R + 1], kv_lens [R],
    slots, positions and request_ids [tokens], counts [2]."""
    query_offsets: torch.Tensor
    kv_lens: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    request_ids: torch.Tensor
    counts: torch.Tensor

    @classmethod
    def empty(cls, requests: int, tokens: int, device) -> "KvMaps":
        return cls(*(torch.empty(n, dtype=torch.int32, device=device)
                     for n in (requests + 1, requests, tokens, tokens, tokens, 2)))


class Kv4Cache:
    """One layer's cache: k_codes and v_codes [pages, kv_heads, page_size * D / 8]
    uint32 words, k_sb and v_sb [pages, kv_heads, page_size, D / group_size, 2]
    (scale, bias) in float16 or bfloat16."""

    def __init__(self, k_codes, k_sb, v_codes, v_sb):
        if k_sb.dim() != 5 or k_sb.shape[-1] != 2 or v_sb.shape != k_sb.shape or v_sb.dtype != k_sb.dtype:
            raise ValueError("k_sb and v_sb must be [pages, kv_heads, page_size, groups, 2] of one dtype")
        if k_sb.dtype not in _HALVES:
            raise ValueError(f"unsupported dtype {k_sb.dtype}")
        if k_codes.dtype not in _WORD_DTYPES or v_codes.dtype not in _WORD_DTYPES:
            raise ValueError("k_codes and v_codes must hold uint32 words (torch.int32 or torch.uint32)")
        pages, heads, page, groups, _ = k_sb.shape
        if (k_codes.dim() != 3 or tuple(k_codes.shape[:2]) != (pages, heads) or v_codes.shape != k_codes.shape
                or page < 1 or groups < 1 or k_codes.shape[2] * 8 % page):
            raise ValueError("k_codes and v_codes must be [pages, kv_heads, page_size * head_dim / 8]")
        dim = k_codes.shape[2] * 8 // page
        if dim % groups:
            raise ValueError(f"head_dim {dim} is not cut into {groups} groups")
        for t in (k_codes, k_sb, v_codes, v_sb):
            if not t.is_cuda or t.device != k_codes.device:
                raise ValueError("all tensors must be on one HIP device")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
        if dim not in (64, 128, 256):
            raise ValueError(f"head_dim must be 64, 128 or 256, got {dim}")
        if dim // groups not in (32, 64, 128):
            raise ValueError(f"group_size must be 32, 64 or 128, got {dim // groups}")
        if page not in (16, 32, 64, 128, 256, 512, 1024):
            raise ValueError(f"page_size must be a power of two from 16 to 1024, got {page}")
        self.k_codes, self.k_sb, self.v_codes, self.v_sb = k_codes, k_sb, v_codes, v_sb
        self.num_pages, self.kv_heads, self.page_size = pages, heads, page
        self.head_dim, self.group_size = dim, dim // groups
        self.dtype, self.device = k_sb.dtype, k_codes.device
        self._c = _CCache(k_codes.data_ptr(), k_sb.data_ptr(), v_codes.data_ptr(), v_sb.data_ptr(), pages, heads,
                          dim, page, self.group_size, _HALVES[k_sb.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def zeros(cls, num_pages: int, kv_heads: int, head_dim: int, *, page_size=64, group_size=64,
              dtype=torch.bfloat16, device="cuda") -> "Kv4Cache":
        """A cache of num_pages pages whose every element is 0."""
        codes = (num_pages, kv_heads, page_size * head_dim // 8)
        pairs = (num_pages, kv_heads, page_size, head_dim // group_size, 2)
        return cls(*(t for _ in range(2) for t in (torch.zeros(codes, dtype=torch.int32, device=device),
                                                   torch.zeros(pairs, dtype=dtype, device=device))))


def _ints(device, **tensors):
    for name, t in tensors.items():
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 vector")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _table(t, requests, device):
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != requests or (t.numel() > 1 and t.shape[1] > 1
                                                                            and t.stride(1) != 1):
        raise ValueError(f"block_table must be int32 [{requests}, columns] with a unit last stride")
    if t.device != device:
        raise ValueError(f"block_table must be on {device}")
    if requests > 1 and t.numel() and t.stride(0) < t.shape[1]:
        raise ValueError("block_table's rows must not overlap")


def kv_maps(past, new, block_table, free_pages, *, page_size, tokens=None, out=None) -> KvMaps:
    """Enters the pages that the requests' new tokens need into block_table (in
    place) and returns the step's offsets, lengths and slot maps (qmx_kv_maps).

    past, new: int32 [R]; block_table: int32 [R, columns]; free_pages: int32
    [F], handed out from its front.  tokens: the room for new tokens, when no
    `out` (a KvMaps to write into) gives it.  counts[1] of the result is how
    many of free_pages were wanted."""
    if not past.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    dev, R = past.device, past.numel()
    _ints(dev, past=past, new=new, free_pages=free_pages)
    if new.numel() != R:
        raise ValueError("past and new must have one length")
    _table(block_table, R, dev)
    if out is None:
        if tokens is None:
            raise ValueError("kv_maps needs tokens or out")
        out = KvMaps.empty(R, tokens, dev)
    else:
        _ints(dev, **out._asdict())
        T = out.slots.numel()
        if [t.numel() for t in out] != [R + 1, R, T, T, T, 2] or (tokens is not None and tokens != T):
            raise ValueError("out's tensors must have R + 1, R, tokens, tokens, tokens and 2 elements")
    _check(lib().qmx_kv_maps(_ptr(past), _ptr(new), _ptr(block_table), _ptr(free_pages), R, block_table.shape[1],
                             block_table.stride(0), free_pages.numel(), page_size, out.slots.numel(),
                             *map(_ptr, out), _stream(past)), "qmx_kv_maps")
    return out


def _new_tokens(cache, x, name):
    if x.dim() != 3 or tuple(x.shape[1:]) != (cache.kv_heads, cache.head_dim):
        raise ValueError(f"{name} must be [tokens, {cache.kv_heads}, {cache.head_dim}]")
    if x.dtype != cache.dtype:
        raise ValueError(f"{name} must have the cache's dtype {cache.dtype}")
    if x.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}")
    if x.stride(2) != 1:
        raise ValueError(f"{name} must have a unit last stride")


def kv4_write(cache: Kv4Cache, k, v, slots) -> None:
    """Quantises k and v [tokens, kv_heads, head_dim] (any strides, the last 1)
    into the cache at `slots` (int32 [tokens], distinct; below 0: skipped)."""
    _new_tokens(cache, k, "k")
    _new_tokens(cache, v, "v")
    _ints(cache.device, slots=slots)
    if not k.shape[0] == v.shape[0] == slots.numel():
        raise ValueError("k, v and slots must have one length")
    _check(lib().qmx_kv4_write(cache._ref, _ptr(k), _ptr(v), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                               _ptr(slots), slots.numel(), _stream(k)), "qmx_kv4_write")


def kv4_read(cache: Kv4Cache, slots, out=None):
    """(k, v) [tokens, kv_heads, head_dim]: what the cache holds at `slots`
    (zeros where a slot is below 0)."""
    _ints(cache.device, slots=slots)
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    if out is None:
        out = tuple(torch.empty(shape, dtype=cache.dtype, device=cache.device) for _ in range(2))
    for t in out:
        if tuple(t.shape) != shape or t.dtype != cache.dtype or t.device != cache.device or not t.is_contiguous():
            raise ValueError(f"out must be two contiguous {shape} tensors of dtype {cache.dtype}")
    _check(lib().qmx_kv4_read(cache._ref, _ptr(out[0]), _ptr(out[1]), _ptr(slots), slots.numel(), _stream(slots)),
           "qmx_kv4_read")
    return out


def kv4_attention_workspace_bytes(cache: Kv4Cache, requests, tokens, heads, max_query_len, max_kv_len,
                                  window=0) -> int:
    return lib().qmx_kv4_attention_workspace_bytes(cache.kv_heads, cache.head_dim, requests, tokens, heads,
                                                   max_query_len, max_kv_len, window)


def kv4_attention(cache: Kv4Cache, q, block_table, kv_lens, query_offsets, *, max_query_len, max_kv_len, window=0,
                  scale=None, return_lse=False, out=None, workspace=None):
    """Causal attention of q [tokens, heads, head_dim] over the cache, which
    holds the same tokens already (qmx_kv4_attention).

    block_table: int32 [R, columns]; kv_lens: int32 [R]; query_offsets: int32
    [R + 1], request r's queries being the last of its kv_lens[r] tokens.
    max_query_len, max_kv_len: host bounds of both.  window: 0, or how many
    tokens a query sees, itself among them.  scale: above 0, head_dim ** -0.5 by default.
    Returns out, or (out, lse) with float32 lse [tokens, heads]."""
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.shape[1] % cache.kv_heads or q.shape[1] < 1:
        raise ValueError(f"q must be [tokens, a multiple of {cache.kv_heads}, {cache.head_dim}]")
    if q.dtype != cache.dtype:
        raise ValueError(f"q must have the cache's dtype {cache.dtype}")
    if q.device != cache.device:
        raise ValueError(f"q must be on {cache.device}")
    if q.stride(2) != 1:
        raise ValueError("q must have a unit last stride")
    T, heads, D = q.shape
    R = kv_lens.numel()
    _ints(q.device, kv_lens=kv_lens, query_offsets=query_offsets)
    if query_offsets.numel() != R + 1:
        raise ValueError("query_offsets must have one element more than kv_lens")
    _table(block_table, R, q.device)
    if out is None:
        out = torch.empty((T, heads, D), dtype=q.dtype, device=q.device)
    elif tuple(out.shape) != (T, heads, D) or out.dtype != q.dtype or out.device != q.device \
            or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {(T, heads, D)} of dtype {q.dtype}")
    lse = torch.empty((T, heads), dtype=torch.float32, device=q.device) if return_lse else None
    max_query_len = min(max_query_len, T)
    if workspace is None:
        need = lib().qmx_kv4_attention_workspace_bytes(cache.kv_heads, D, R, T, heads, max_query_len, max_kv_len,
                                                       window)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {q.device}")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().qmx_kv4_attention(cache._ref, _ptr(q), q.stride(0), q.stride(1), _ptr(out), _ptr(lse),
                                   _ptr(block_table), block_table.shape[1], block_table.stride(0), _ptr(kv_lens),
                                   _ptr(query_offsets), R, T, heads, max_query_len, max_kv_len, window,
                                   D ** -0.5 if scale is None else scale, _ptr(workspace), ws_bytes, _stream(q)),
           "qmx_kv4_attention")
    return (out, lse) if return_lse else out
