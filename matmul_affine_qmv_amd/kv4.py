"""The paged 4-bit key/value cache: marshalling for qmx_kv_maps, qmx_kv4_write,
qmx_kv4_read and qmx_kv4_attention (include/qmx.h says what they compute).

As in the package itself, every function checks its tensors, allocates what is
not given and calls the C ABI on torch's current HIP stream; nothing here
synchronises or copies to the host, so a step can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple
from functools import lru_cache

import torch

from . import _WORD_DTYPES, QMX_BF16, QMX_F16, QmxError, lib

_HALVES = {torch.float16: QMX_F16, torch.bfloat16: QMX_BF16}
_INT = torch.int32

# A call's own cost on the host counts beside kernels of a few microseconds: the
# stream is asked for as a number, and pointers go to the library as numbers.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(status: int, func: str) -> None:
    if status:
        raise QmxError(status, func)


class _CCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_sb", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_sb", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("group_size", ctypes.c_int),
                ("dtype", ctypes.c_int)]


_MAPS = ("query_offsets", "kv_lens", "slots", "positions", "request_ids", "counts")


class KvMaps(namedtuple("KvMaps", _MAPS)):
    """What kv_maps writes, int32 tensors on one device: query_offsets [R + 1],
    kv_lens [R], slots, positions and request_ids [tokens], counts [2]."""

    def __new__(cls, *args, **kwargs):
        self = super().__new__(cls, *args, **kwargs)
        if not self.slots.is_cuda:
            raise ValueError("all tensors must be on a HIP device")
        _ints(self.slots.get_device(), **self._asdict())
        R, T = self.kv_lens.numel(), self.slots.numel()
        if [t.numel() for t in self] != [R + 1, R, T, T, T, 2]:
            raise ValueError("the tensors must have R + 1, R, tokens, tokens, tokens and 2 elements")
        self.requests, self.tokens, self.device_index = R, T, self.slots.get_device()
        return self

    @classmethod
    def _make(cls, tensors) -> "KvMaps":
        return cls(*tensors)

    @classmethod
    def empty(cls, requests: int, tokens: int, device) -> "KvMaps":
        return cls(*(torch.empty(n, dtype=_INT, device=device)
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
        self.dtype, self.device, self.device_index = k_sb.dtype, k_codes.device, k_codes.get_device()
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


def _ints(index, **tensors):
    for name, t in tensors.items():
        if t.dtype is not _INT or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 vector")
        if t.get_device() != index:
            raise ValueError(f"{name} must be on HIP device {index}")


def _table(t, requests, index):
    """Columns and row stride of a block table."""
    if t.dtype is not _INT or t.dim() != 2:
        raise ValueError("block_table must be int32 [requests, columns]")
    rows, columns = t.shape
    stride, last = t.stride()
    if rows != requests or (last != 1 and rows and columns > 1):
        raise ValueError(f"block_table must be int32 [{requests}, columns] with a unit last stride")
    if t.get_device() != index:
        raise ValueError(f"block_table must be on HIP device {index}")
    if rows > 1 and columns and stride < columns:
        raise ValueError("block_table's rows must not overlap")
    return columns, stride


def kv_maps(past, new, block_table, free_pages, *, page_size, tokens=None, out=None) -> KvMaps:
    """Enters the pages that the requests' new tokens need into block_table (in
    place) and returns the step's offsets, lengths and slot maps (qmx_kv_maps).

    past, new: int32 [R]; block_table: int32 [R, columns]; free_pages: int32
    [F], handed out from its front.  tokens: the room for new tokens, when no
    `out` (a KvMaps to write into) gives it.  counts[1] of the result is how
    many of free_pages were wanted.  Outputs share no memory with the inputs:
    the next step's past is a copy of kv_lens, or past + new in place."""
    if not past.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    index, R = past.get_device(), past.numel()
    _ints(index, past=past, new=new, free_pages=free_pages)
    if new.numel() != R:
        raise ValueError("past and new must have one length")
    columns, stride = _table(block_table, R, index)
    if out is None:
        if tokens is None:
            raise ValueError("kv_maps needs tokens or out")
        out = KvMaps.empty(R, tokens, past.device)
    elif out.requests != R or (tokens is not None and tokens != out.tokens):
        raise ValueError("out's tensors must have R + 1, R, tokens, tokens, tokens and 2 elements")
    elif out.device_index != index:
        raise ValueError(f"out must be on HIP device {index}")
    _check(lib().qmx_kv_maps(past.data_ptr(), new.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), R,
                             columns, stride, free_pages.numel(), page_size, out.tokens,
                             *[t.data_ptr() for t in out], _raw_stream(index)), "qmx_kv_maps")
    return out


def _new_tokens(cache, x, name):
    """Token and head strides of new keys or values."""
    if x.dim() != 3 or x.shape[1:] != (cache.kv_heads, cache.head_dim):
        raise ValueError(f"{name} must be [tokens, {cache.kv_heads}, {cache.head_dim}]")
    if x.dtype is not cache.dtype:
        raise ValueError(f"{name} must have the cache's dtype {cache.dtype}")
    if x.get_device() != cache.device_index:
        raise ValueError(f"{name} must be on {cache.device}")
    token, head, last = x.stride()
    if last != 1:
        raise ValueError(f"{name} must have a unit last stride")
    return token, head


def kv4_write(cache: Kv4Cache, k, v, slots) -> None:
    """Quantises k and v [tokens, kv_heads, head_dim] (any strides, the last 1)
    into the cache at `slots` (int32 [tokens], distinct; below 0: skipped)."""
    kt, kh = _new_tokens(cache, k, "k")
    vt, vh = _new_tokens(cache, v, "v")
    _ints(cache.device_index, slots=slots)
    T = slots.numel()
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError("k, v and slots must have one length")
    _check(lib().qmx_kv4_write(cache._ref, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), T,
                               _raw_stream(cache.device_index)), "qmx_kv4_write")


def kv4_read(cache: Kv4Cache, slots, out=None):
    """(k, v) [tokens, kv_heads, head_dim]: what the cache holds at `slots`
    (zeros where a slot is below 0)."""
    _ints(cache.device_index, slots=slots)
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    if out is None:
        k = torch.empty(shape, dtype=cache.dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        for t in out:
            if t.shape != shape or t.dtype is not cache.dtype or t.get_device() != cache.device_index \
                    or not t.is_contiguous():
                raise ValueError(f"out must be two contiguous {shape} tensors of dtype {cache.dtype}")
    _check(lib().qmx_kv4_read(cache._ref, k.data_ptr(), v.data_ptr(), slots.data_ptr(), shape[0],
                              _raw_stream(cache.device_index)), "qmx_kv4_read")
    return k, v


@lru_cache(maxsize=4096)
def _workspace_bytes(device_index, *sizes):
    return lib().qmx_kv4_attention_workspace_bytes(*sizes)


def kv4_attention_workspace_bytes(cache: Kv4Cache, requests, tokens, heads, max_query_len, max_kv_len,
                                  window=0) -> int:
    """Bytes of workspace that kv4_attention needs for these sizes (a host rule);
    as there, max_query_len may be above the number of tokens."""
    return _workspace_bytes(cache.device_index, cache.kv_heads, cache.head_dim, requests, tokens, heads,
                            max_query_len, max_kv_len, window)


def kv4_attention(cache: Kv4Cache, q, block_table, kv_lens, query_offsets, *, max_query_len, max_kv_len, window=0,
                  scale=None, return_lse=False, out=None, workspace=None):
    """Causal attention of q [tokens, heads, head_dim] over the cache, which
    holds the same tokens already (qmx_kv4_attention).

    block_table: int32 [R, columns]; kv_lens: int32 [R]; query_offsets: int32
    [R + 1], request r's queries being the last of its kv_lens[r] tokens.
    max_query_len, max_kv_len: host bounds of both; what a request has past them
    is not computed: its later queries' outputs are zeros, its later keys
    unseen.  window: 0, or how many tokens a query sees, itself among them.
    scale: above 0, head_dim ** -0.5 by default.  workspace: of
    kv4_attention_workspace_bytes bytes, where the caller keeps one.  Returns
    out, or (out, lse) with float32 lse [tokens, heads]."""
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.shape[1] % cache.kv_heads or q.shape[1] < 1:
        raise ValueError(f"q must be [tokens, a multiple of {cache.kv_heads}, {cache.head_dim}]")
    if q.dtype is not cache.dtype:
        raise ValueError(f"q must have the cache's dtype {cache.dtype}")
    index = cache.device_index
    if q.get_device() != index:
        raise ValueError(f"q must be on {cache.device}")
    token, head, last = q.stride()
    if last != 1:
        raise ValueError("q must have a unit last stride")
    T, heads, D = q.shape
    R = kv_lens.numel()
    _ints(index, kv_lens=kv_lens, query_offsets=query_offsets)
    if query_offsets.numel() != R + 1:
        raise ValueError("query_offsets must have one element more than kv_lens")
    columns, stride = _table(block_table, R, index)
    if out is None:
        out = torch.empty((T, heads, D), dtype=q.dtype, device=cache.device)
    elif out.shape != (T, heads, D) or out.dtype is not q.dtype or out.get_device() != index \
            or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {(T, heads, D)} of dtype {q.dtype}")
    lse = torch.empty((T, heads), dtype=torch.float32, device=cache.device) if return_lse else None
    max_query_len = min(max_query_len, T)
    need = _workspace_bytes(index, cache.kv_heads, D, R, T, heads, max_query_len, max_kv_len, window)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    elif workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be contiguous on {cache.device}")
    _check(lib().qmx_kv4_attention(cache._ref, q.data_ptr(), token, head, out.data_ptr(),
                                   lse.data_ptr() if return_lse else None, block_table.data_ptr(), columns, stride,
                                   kv_lens.data_ptr(), query_offsets.data_ptr(), R, T, heads, max_query_len,
                                   max_kv_len, window, D ** -0.5 if scale is None else scale,
                                   workspace.data_ptr() if workspace is not None else None,
                                   workspace.nbytes if workspace is not None else 0, _raw_stream(index)),
           "qmx_kv4_attention")
    return (out, lse) if return_lse else out
