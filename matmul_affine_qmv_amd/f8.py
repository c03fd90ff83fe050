"""8-bit floats: marshalling for qmx_rms_norm, qmx_f8_quantize, qmx_f8_dequantize
and qmx_qmm_f8 (include/qmx.h says what they compute).

Codes are torch.float8_e4m3fn; their scales torch.float8_e8m0fnu (torch.uint8 is
taken for the same bytes), or float32 for weights.  As in the package itself,
every function checks its tensors, allocates what is not given and calls the C
ABI on torch's current HIP stream of the tensors' device; nothing here
synchronises or copies to the host, so a step can be captured into a graph.
"""
from __future__ import annotations

from functools import lru_cache

import torch

from . import QMX_BF16, QMX_F16, QmxError, lib

_HALVES = {torch.float16: QMX_F16, torch.bfloat16: QMX_BF16}
_CODES, _SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
_BYTES = (_SCALES, torch.uint8)
_SCALE_E8M0, _SCALE_F32 = 0, 1

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _on(index, name, *args):
    """The library's function on a device, which is made the current one if it is not."""
    if index == _current_device():
        return getattr(lib(), name)(*args)
    with torch.cuda.device(index):
        return getattr(lib(), name)(*args)


def _call(index, name, *args):
    """The same on its current stream, its status checked."""
    status = _on(index, name, *args, _raw_stream(index))
    if status:
        raise QmxError(status, name)


def _rows(t, name, dtype=None, shape=None):
    """Row stride of a 16-bit matrix with unit element stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, width]")
    if not t.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    if t.dtype not in _HALVES:
        raise ValueError(f"{name} has an unsupported dtype {t.dtype}")
    stride, last = t.stride()
    if last != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have a unit last stride")
    if dtype is not None and (t.dtype is not dtype or t.shape != shape):
        raise ValueError(f"{name} must be {tuple(shape)} of dtype {dtype}")
    return stride


def _dense(t, name, shape, dtypes, index):
    if tuple(t.shape) != shape or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {shape} of dtype {' or '.join(str(d) for d in dtypes)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on HIP device {index}")


def _norm(x, weight, residual, eps, sum_out, out, scales):
    stride = _rows(x, "x")
    shape, index = x.shape, x.get_device()
    rows, width = shape
    if weight is not None:
        _dense(weight, "weight", (width,), (x.dtype,), index)
    r_stride = s_stride = 0
    if residual is not None:
        r_stride = _rows(residual, "residual", x.dtype, shape)
        if sum_out is None:
            sum_out = torch.empty((rows, width), dtype=x.dtype, device=x.device)
        s_stride = _rows(sum_out, "sum_out", x.dtype, shape)
        if residual.get_device() != index or sum_out.get_device() != index:
            raise ValueError(f"residual and sum_out must be on {x.device}")
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    _call(index, "qmx_rms_norm", x.data_ptr(), stride, residual.data_ptr() if residual is not None else None, r_stride,
          weight.data_ptr() if weight is not None else None, sum_out.data_ptr() if sum_out is not None else None,
          s_stride, out.data_ptr(), scales.data_ptr() if scales is not None else None, rows, width, eps,
          _HALVES[x.dtype])
    return sum_out


def rms_norm(x, weight=None, residual=None, *, eps=1e-6, sum_out=None, out=None):
    """Root mean square norm of x [rows, width] times weight [width] (None: ones),
    into x's dtype (qmx_rms_norm).  x and residual may have any row stride.

    residual: added to x before; then (out, sum) are returned, sum being what was
    normed.  sum_out: where it goes, x or residual itself for instance.  out:
    contiguous, x itself for instance."""
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif x.is_cuda:
        _dense(out, "out", tuple(x.shape), (x.dtype,), x.get_device())
    total = _norm(x, weight, residual, eps, sum_out, out, None)
    return out if residual is None else (out, total)


def rms_norm_f8(x, weight=None, residual=None, *, eps=1e-6, sum_out=None, out=None):
    """rms_norm into 8 bits: (codes [rows, width], scales [rows, width / 128]), or
    (codes, scales, sum) with a residual.  width is a multiple of 128.  out: the
    two to write into."""
    codes, scales = _outputs(x, 1, out)
    total = _norm(x, weight, residual, eps, sum_out, codes, scales)
    return (codes, scales) if residual is None else (codes, scales, total)


def _outputs(x, block_rows, out):
    """Codes and scales for x, made or checked."""
    if x.dim() != 2 or x.shape[1] % 128:
        raise ValueError("x must be [rows, a multiple of 128]")
    rows, width = x.shape
    shape = (-(-rows // block_rows), width // 128)
    if out is None:
        return (torch.empty((rows, width), dtype=_CODES, device=x.device),
                torch.empty(shape, dtype=_SCALES, device=x.device))
    codes, scales = out
    _dense(codes, "codes", (rows, width), (_CODES,), x.get_device())
    _dense(scales, "scales", shape, _BYTES, x.get_device())
    return codes, scales


def f8_quantize(x, *, block_rows=1, out=None):
    """(codes, scales) of x [rows, width] in float16 or bfloat16, rows any stride
    apart, width a multiple of 128: a scale for each 128 of a row, as qmm_f8 takes
    activations, or of each block of 128 x 128 (block_rows=128), as it takes
    weights (qmx_f8_quantize)."""
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
    stride = _rows(x, "x")
    codes, scales = _outputs(x, block_rows, out)
    _call(x.get_device(), "qmx_f8_quantize", x.data_ptr(), stride, codes.data_ptr(), scales.data_ptr(), *x.shape,
          block_rows, _HALVES[x.dtype])
    return codes, scales


def _coded(codes, scales, name, types):
    """Rows of codes to a scale, and the scales' type."""
    if codes.dim() != 2 or codes.dtype is not _CODES or codes.shape[1] % 128:
        raise ValueError(f"{name} must be float8_e4m3fn [rows, a multiple of 128]")
    if not codes.is_cuda:
        raise ValueError("all tensors must be on a HIP device")
    if not codes.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    rows, width = codes.shape
    block_rows = 1 if scales.dim() != 2 or scales.shape[0] == rows else 128
    _dense(scales, f"{name}_scales", (-(-rows // block_rows), width // 128), types, codes.get_device())
    return block_rows, _SCALE_F32 if scales.dtype is torch.float32 else _SCALE_E8M0


def f8_dequantize(codes, scales, *, dtype=torch.bfloat16, out=None):
    """The values that codes [rows, width] stand for, in float16 or bfloat16.
    scales: [rows, width / 128], or [ceil(rows / 128), width / 128] of blocks; E8M0
    or float32 (qmx_f8_dequantize)."""
    block_rows, kind = _coded(codes, scales, "codes", (*_BYTES, torch.float32))
    if out is None:
        if dtype not in _HALVES:
            raise ValueError(f"unsupported dtype {dtype}")
        out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    else:
        _dense(out, "out", tuple(codes.shape), tuple(_HALVES), codes.get_device())
    _call(codes.get_device(), "qmx_f8_dequantize", codes.data_ptr(), scales.data_ptr(), kind, out.data_ptr(),
          *codes.shape, block_rows, _HALVES[out.dtype])
    return out


@lru_cache(maxsize=4096)
def _workspace_bytes(index, M, N, K):
    return _on(index, "qmx_qmm_f8_workspace_bytes", M, N, K)


def qmm_f8_workspace_bytes(M, N, K, device="cuda") -> int:
    """Bytes of workspace that qmm_f8 needs for these sizes (a host rule)."""
    index = torch.device(device).index
    return _workspace_bytes(_current_device() if index is None else index, M, N, K)


def qmm_f8(w, w_scales, x, x_scales, out=None, *, dtype=torch.bfloat16, workspace=None):
    """out[M, N] = x @ w.T of 8-bit floats, in float16 or bfloat16 (qmx_qmm_f8).

    w: codes [N, K], w_scales [ceil(N / 128), K / 128] E8M0 or float32;
    x: codes [M, K], x_scales [M, K / 128] E8M0; all contiguous.  workspace: of
    qmm_f8_workspace_bytes bytes, where the caller keeps one."""
    if x.dim() != 2 or w.dim() != 2 or w.dtype is not _CODES or x.dtype is not _CODES:
        raise ValueError("w and x must be float8_e4m3fn [N, K] and [M, K]")
    M, K = x.shape
    N, index = w.shape[0], x.get_device()
    if w.shape[1] != K or K % 128:
        raise ValueError(f"w and x must have one K, a multiple of 128; got {w.shape[1]} and {K}")
    if not x.is_cuda or w.get_device() != index:
        raise ValueError("all tensors must be on one HIP device")
    if not w.is_contiguous() or not x.is_contiguous():
        raise ValueError("w and x must be contiguous")
    _dense(w_scales, "w_scales", (-(-N // 128), K // 128), (*_BYTES, torch.float32), index)
    _dense(x_scales, "x_scales", (M, K // 128), _BYTES, index)
    if out is None:
        if dtype not in _HALVES:
            raise ValueError(f"unsupported dtype {dtype}")
        out = torch.empty((M, N), dtype=dtype, device=x.device)
    else:
        _dense(out, "out", (M, N), tuple(_HALVES), index)
    need = _workspace_bytes(index, M, N, K)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be contiguous on {x.device}")
    _call(index, "qmx_qmm_f8", w.data_ptr(), w_scales.data_ptr(),
          _SCALE_F32 if w_scales.dtype is torch.float32 else _SCALE_E8M0, x.data_ptr(), x_scales.data_ptr(),
          out.data_ptr(), M, N, K, _HALVES[out.dtype], workspace.data_ptr() if workspace is not None else None,
          workspace.nbytes if workspace is not None else 0)
    return out
