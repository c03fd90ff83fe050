"""8-bit floats: marshalling for qmx_rms_norm, qmx_f8_quantize, qmx_f8_dequantize
and qmx_qmm_f8 (include/qmx.h says what they compute).

Codes are torch.float8_e4m3fn; their scales torch.float8_e8m0fnu (torch.uint8 is
taken for the same bytes), or float32 for weights.  As in the package itself,
every function checks its tensors, allocates what is not given and calls the C
ABI on torch's current HIP stream of the tensors' device; nothing here
synchronises or copies to the host, so a step can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import QMX_BF16, QMX_F16, QmxError, lib

_HALVES = {torch.float16: QMX_F16, torch.bfloat16: QMX_BF16}
_CODES, _SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
_BYTES = (_SCALES, torch.uint8)
_ANY_SCALES = (*_BYTES, torch.float32)
_SCALE_E8M0, _SCALE_F32 = 0, 1
_MOST = 2 ** 31 - 1   # sizes go to the library as ints

# A call's own cost on the host counts beside kernels of a few microseconds: the
# checks are written out where they are made, the stream is asked for as a number,
# and pointers go to the library as numbers.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_like = torch.empty_like
_WHOLE = torch.contiguous_format


@lru_cache(maxsize=None)
def _function(name):
    return getattr(lib(), name)


def _check(status, name):
    if status:
        raise QmxError(status, name)


def _rows(t, name, dtype, shape, index):
    """Row stride of another 16-bit matrix with unit element stride."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} of dtype {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on HIP device {index}")
    stride, last = t.stride()
    if last != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have a unit last stride")
    return stride


def _first(x):
    """dtype code, shape, row stride and device index of a 16-bit matrix."""
    code = _HALVES.get(x.dtype)
    if code is None or x.dim() != 2:
        raise ValueError(f"x must be [rows, width] in float16 or bfloat16, got {x.dim()}-D {x.dtype}")
    if not x.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    stride, last = x.stride()
    shape = x.shape
    if last != 1 and shape[1] > 1:
        raise ValueError("x must have a unit last stride")
    if shape[0] > _MOST or shape[1] > _MOST:
        raise ValueError("x must have below 2^31 rows and columns")
    return code, shape, stride, x.get_device()


def _dense(t, name, shape, dtypes, index):
    if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} of dtype {' or '.join(str(d) for d in dtypes)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on HIP device {index}")


def _norm(x, first, weight, residual, eps, sum_out, out, scales):
    code, shape, stride, index = first
    weight_at = residual_at = sum_at = None
    r_stride = s_stride = 0
    if weight is not None:
        if weight.dtype is not x.dtype or weight.shape != shape[1:] or not weight.is_contiguous() \
                or weight.get_device() != index:
            raise ValueError(f"weight must be a contiguous [{shape[1]}] of dtype {x.dtype} on {x.device}")
        weight_at = weight.data_ptr()
    if residual is not None:
        r_stride = _rows(residual, "residual", x.dtype, shape, index)
        residual_at = residual.data_ptr()
        if sum_out is None:
            sum_out = _like(x, memory_format=_WHOLE)
            s_stride = shape[1]
        else:
            s_stride = _rows(sum_out, "sum_out", x.dtype, shape, index)
        sum_at = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    _check(_function("qmx_rms_norm")(x.data_ptr(), stride, residual_at, r_stride, weight_at, sum_at, s_stride,
                                     out.data_ptr(), scales, *shape, eps, code, _raw_stream(index)), "qmx_rms_norm")
    return sum_out


def rms_norm(x, weight=None, residual=None, *, eps=1e-6, sum_out=None, out=None):
    """Root mean square norm of x [rows, width] times weight [width] (None: ones),
    into x's dtype (qmx_rms_norm).  x and residual may have any row stride.

    residual: added to x before; then (out, sum) are returned, sum being what was
    normed.  sum_out: where it goes, x or residual itself for instance.  out:
    contiguous, x or residual itself for instance.  Over anything else of the call's
    tensors both are refused."""
    first = _first(x)
    if first[3] != _current_device():
        with torch.cuda.device(first[3]):
            return rms_norm(x, weight, residual, eps=eps, sum_out=sum_out, out=out)
    if out is None:
        out = _like(x, memory_format=_WHOLE)
    else:
        _dense(out, "out", x.shape, (x.dtype,), first[3])
    total = _norm(x, first, weight, residual, eps, sum_out, out, None)
    return out if residual is None else (out, total)


def rms_norm_f8(x, weight=None, residual=None, *, eps=1e-6, sum_out=None, out=None):
    """rms_norm into 8 bits: (codes [rows, width], scales [rows, width / 128]), or
    (codes, scales, sum) with a residual.  width is a multiple of 128.  out: the
    two to write into."""
    first = _first(x)
    if first[3] != _current_device():
        with torch.cuda.device(first[3]):
            return rms_norm_f8(x, weight, residual, eps=eps, sum_out=sum_out, out=out)
    codes, scales = _outputs(x, first, 1, out)
    total = _norm(x, first, weight, residual, eps, sum_out, codes, scales.data_ptr())
    return (codes, scales) if residual is None else (codes, scales, total)


def _outputs(x, first, block_rows, out):
    """Codes and scales for x, made or checked."""
    rows, width = first[1]
    if width % 128:
        raise ValueError("x must be [rows, a multiple of 128]")
    shape = (-(-rows // block_rows), width // 128)
    if out is None:
        return _like(x, dtype=_CODES, memory_format=_WHOLE), x.new_empty(shape, dtype=_SCALES)
    codes, scales = out
    _dense(codes, "codes", (rows, width), (_CODES,), first[3])
    _dense(scales, "scales", shape, _BYTES, first[3])
    return codes, scales


def f8_quantize(x, *, block_rows=1, out=None):
    """(codes, scales) of x [rows, width] in float16 or bfloat16, rows any stride
    apart, width a multiple of 128: a scale for each 128 of a row, as qmm_f8 takes
    activations, or of each block of 128 x 128 (block_rows=128), as it takes
    weights (qmx_f8_quantize)."""
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
    first = code, shape, stride, index = _first(x)
    if index != _current_device():
        with torch.cuda.device(index):
            return f8_quantize(x, block_rows=block_rows, out=out)
    codes, scales = _outputs(x, first, block_rows, out)
    _check(_function("qmx_f8_quantize")(x.data_ptr(), stride, codes.data_ptr(), scales.data_ptr(), *shape, block_rows,
                                        code, _raw_stream(index)), "qmx_f8_quantize")
    return codes, scales


def f8_dequantize(codes, scales, *, dtype=torch.bfloat16, out=None):
    """The values that codes [rows, width] stand for, in float16 or bfloat16.
    scales: [rows, width / 128], or [ceil(rows / 128), width / 128] of blocks; E8M0
    or float32 (qmx_f8_dequantize)."""
    if codes.dtype is not _CODES or codes.dim() != 2 or codes.shape[1] % 128:
        raise ValueError("codes must be float8_e4m3fn [rows, a multiple of 128]")
    if not codes.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    rows, width = codes.shape
    if rows > _MOST or width > _MOST:
        raise ValueError("codes must have below 2^31 rows and columns")
    index = codes.get_device()
    if index != _current_device():
        with torch.cuda.device(index):
            return f8_dequantize(codes, scales, dtype=dtype, out=out)
    block_rows = 1 if scales.dim() != 2 or scales.shape[0] == rows else 128
    _dense(scales, "scales", (-(-rows // block_rows), width // 128), _ANY_SCALES, index)
    if out is None:
        code = _HALVES.get(dtype)
        if code is None:
            raise ValueError(f"unsupported dtype {dtype}")
        out = _like(codes, dtype=dtype)
    else:
        _dense(out, "out", codes.shape, tuple(_HALVES), index)
        code = _HALVES[out.dtype]
    kind = _SCALE_F32 if scales.dtype is torch.float32 else _SCALE_E8M0
    _check(_function("qmx_f8_dequantize")(codes.data_ptr(), scales.data_ptr(), kind, out.data_ptr(), rows, width,
                                          block_rows, code, _raw_stream(index)), "qmx_f8_dequantize")
    return out


def plan_f8(M, N, K, num_cus=0):
    """(tile rows, tile columns, parts of K) that qmm_f8 takes (qmx_plan_f8, a host rule)."""
    tile_rows, tile_cols, splits = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    if not all(abs(size) <= _MOST for size in (M, N, K)):
        raise ValueError("M, N and K must be below 2^31")
    _check(lib().qmx_plan_f8(M, N, K, num_cus, ctypes.byref(tile_rows), ctypes.byref(tile_cols), ctypes.byref(splits)),
           "qmx_plan_f8")
    return tile_rows.value, tile_cols.value, splits.value


@lru_cache(maxsize=4096)
def _workspace_bytes(index, M, N, K):
    with torch.cuda.device(index):
        return lib().qmx_qmm_f8_workspace_bytes(M, N, K)


def qmm_f8_workspace_bytes(M, N, K, device="cuda") -> int:
    """Bytes of workspace that qmm_f8 needs for these sizes (a host rule)."""
    if not all(0 <= size <= _MOST for size in (M, N, K)):
        raise ValueError("M, N and K must be 0 or more and below 2^31")
    index = torch.device(device).index
    return _workspace_bytes(_current_device() if index is None else index, M, N, K)


def qmm_f8(w, w_scales, x, x_scales, out=None, *, dtype=torch.bfloat16, workspace=None):
    """out[M, N] = x @ w.T of 8-bit floats, in float16 or bfloat16 (qmx_qmm_f8).

    w: codes [N, K], w_scales [ceil(N / 128), K / 128] E8M0 or float32;
    x: codes [M, K], x_scales [M, K / 128] E8M0; all contiguous.  workspace: of
    qmm_f8_workspace_bytes bytes, where the caller keeps one."""
    if x.dtype is not _CODES or w.dtype is not _CODES or x.dim() != 2 or w.dim() != 2:
        raise ValueError("w and x must be float8_e4m3fn [N, K] and [M, K]")
    M, K = x.shape
    N, K_w = w.shape
    index = x.get_device()
    if K_w != K or K % 128:
        raise ValueError(f"w and x must have one K, a multiple of 128; got {K_w} and {K}")
    if index < 0 or w.get_device() != index:
        raise ValueError("all tensors must be on one HIP device")
    if M > _MOST or N > _MOST or K > _MOST:
        raise ValueError("M, N and K must be below 2^31")
    if index != _current_device():
        with torch.cuda.device(index):
            return qmm_f8(w, w_scales, x, x_scales, out, dtype=dtype, workspace=workspace)
    if not w.is_contiguous() or not x.is_contiguous():
        raise ValueError("w and x must be contiguous")
    _dense(w_scales, "w_scales", (-(-N // 128), K // 128), _ANY_SCALES, index)
    _dense(x_scales, "x_scales", (M, K // 128), _BYTES, index)
    if out is None:
        code = _HALVES.get(dtype)
        if code is None:
            raise ValueError(f"unsupported dtype {dtype}")
        out = x.new_empty((M, N), dtype=dtype)
    else:
        _dense(out, "out", (M, N), tuple(_HALVES), index)
        code = _HALVES[out.dtype]
    need = _workspace_bytes(index, M, N, K)
    room, size = None, 0
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {x.device}")
        room, size = workspace.data_ptr(), workspace.nbytes
    elif need:
        workspace = x.new_empty(need, dtype=torch.uint8)
        room, size = workspace.data_ptr(), need
    kind = _SCALE_F32 if w_scales.dtype is torch.float32 else _SCALE_E8M0
    _check(_function("qmx_qmm_f8")(w.data_ptr(), w_scales.data_ptr(), kind, x.data_ptr(), x_scales.data_ptr(),
                                   out.data_ptr(), M, N, K, code, room, size, _raw_stream(index)), "qmx_qmm_f8")
    return out
