"""8-bit floats, the norm and rotary positions in 64 bits and more, from their
definitions (include/qmx.h), on the CPU: what the GPU's results are held against.
"""
import math

import numpy as np
import torch

# every e4m3 code's value
CODE = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
_POS = np.array(sorted({abs(v) for v in CODE.tolist() if not math.isnan(v)}))   # 127 magnitudes


def two(e):
    return torch.from_numpy(np.ldexp(1.0, np.asarray(e)))


def scale_values(scales):
    """What scales (E8M0 or float32) are, in 64 bits."""
    if scales.dtype == torch.float32:
        return scales.double()
    b = scales.view(torch.uint8).int()
    return torch.where(b == 255, math.nan, two(b.numpy() - 127))


def nearest_code(v):
    """Codes (as uint8) of values of at most 448 in 64 bits: to nearest, to the even code at a middle."""
    a = np.abs(v.numpy())
    hi = np.clip(np.searchsorted(_POS, a), 1, len(_POS) - 1)
    lo = hi - 1
    below, above = a - _POS[lo], _POS[hi] - a
    pick = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)   # magnitude i has code i
    return torch.from_numpy((pick + 128 * np.signbit(v.numpy())).astype(np.uint8))


def quantize(x, block_rows=1):
    """(codes, scale bytes) of x [M, K] in 64 bits."""
    x = x.double()
    M, K = x.shape
    over = -M % block_rows
    g = torch.cat((x, x.new_zeros(over, K))).view((M + over) // block_rows, block_rows, K // 128, 128)
    amax = g.abs().amax((1, 3))
    bad = ~torch.isfinite(g).all(3).all(1)
    m, e = np.frexp(torch.where(bad, 1.0, amax).numpy())
    e = np.maximum(np.where(m > 0, np.where(m > 0.875, e - 8, e - 9), -127), -127)
    v = torch.where(bad[:, None, :, None], 0.0, g) * two(-e)[:, None, :, None]
    codes = torch.where(bad[:, None, :, None], 0x7f, nearest_code(v)).to(torch.uint8)
    return codes.view(M + over, K)[:M], torch.where(bad, 255, torch.from_numpy(e + 127)).to(torch.uint8)


def values(codes, scales):
    """What codes stand for, in 64 bits (exact for E8M0)."""
    s = scale_values(scales)
    if len(s) != len(codes):
        s = s.repeat_interleave(128, 0)[:len(codes)]
    c = CODE[codes.view(torch.uint8).long()]
    return (c.unflatten(1, (-1, 128)) * s[..., None]).flatten(1)


def norm(x, weight, residual, eps):
    """(y in 64 bits, h in the type)"""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = h.double()
    y = v / torch.sqrt((v * v).sum(1, keepdim=True) / x.shape[1] + eps)
    return (y if weight is None else y * weight.double()), h


def product(w, ws, x, xs):
    """(out in 64 bits, bound of the matrix instruction's and float32's own errors).

    Of 8 neighbouring k each product is cut 2^-13 below the largest exponent, which is at most the largest
    product; a sum of 8 and all that follows is float32: G sums of groups, each from 16 sums of 8 (at most 2^-23
    of the sum of magnitudes a step, cut or rounded)."""
    X, W = values(x, xs), values(w, ws)
    out = X @ W.T
    G = X.shape[1] // 128
    size = X.abs() @ W.abs().T
    bound = (G + 20) * 2.0 ** -23 * size
    for m in range(len(X)):   # the largest of 8 products
        p = (X[m].abs()[None] * W.abs()).unflatten(1, (-1, 8)).amax(2).sum(1)
        bound[m] += 7 * 2.0 ** -13 * p
    return out, bound


def half_step(y, dtype):
    """The most that rounding y (64 bits) to a type moves it."""
    fi = torch.finfo(dtype)
    return y.abs() * (fi.eps / 2) + fi.tiny * fi.eps / 2


def rope(x, positions, frequencies, interleaved, scale):
    """(y in 64 bits, |a| + |b| of each result); angles in 80 bits."""
    n = len(frequencies)
    t = positions.numpy().astype(np.longdouble)[:, None] * frequencies.numpy().astype(np.longdouble)[None]
    full = 2 * np.longdouble("3.14159265358979323846264338327950288")
    t = t - full * np.rint(t / full)
    c = torch.from_numpy(np.cos(t).astype(np.float64))[:, None]
    s = torch.from_numpy(np.sin(t).astype(np.float64))[:, None]
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., first], x[..., second]
    turned = (positions >= 0)[:, None, None]
    y[..., first] = torch.where(turned, scale * (a * c - b * s), a)
    y[..., second] = torch.where(turned, scale * (b * c + a * s), b)
    size[..., first] = size[..., second] = torch.where(turned, abs(scale) * (a.abs() + b.abs()), 0.0)
    return y, size
