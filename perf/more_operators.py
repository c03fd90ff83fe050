"""Operators around the products and the cache of one layer's step in 8-bit floats, as cases to time and compare.

* norm:     root mean square norm, with the residual's addition before it, into the type or into 8 bits;
* quantise: activations (groups of 128 of a row) or weights (blocks of 128 x 128) into 8 bits, and back as values;
* product:  matrix product of both in 8 bits;
* rope:     rotary positions of queries and keys.

8 bits.  An element is an e4m3 number (torch.float8_e4m3fn), with one scale for each 128 of a row, or each block of
128 rows by 128: a power of two 2^e held as e + 127 (torch.float8_e8m0fnu), e the least whole number from -127 on with
amax <= 448 * 2^e.  An element is x * 2^-e rounded to nearest even.  A product's weights may have float32 scales.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def _norm(name, rows, width, type="bf16", residual=True, f8=True, gap=0):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "type": type, "residual": residual, "f8": f8,
            "gap": gap}


def _quantise(name, rows, width, type="bf16", block=1, gap=0):
    return {"name": name, "op": "quantise", "rows": rows, "width": width, "type": type, "block": block, "gap": gap}


def _product(name, M, N, K, type="bf16", scales="e8m0"):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "type": type, "scales": scales}


def _rope(name, tokens, heads, kv_heads, dim, rotary, far, type="bf16", interleaved=False, factor=1.0, pad=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "far": far, "type": type, "interleaved": interleaved, "factor": factor, "pad": pad}


def listed():
    return [
        # one user, one token: latency
        _norm("norm token", 1, 5120),
        # a prompt's chunk, on its way to an 8-bit product
        _norm("norm prompt", 8192, 5120),
        # an odd width, rows apart, no residual, the result in the type
        _norm("norm odd", 2500, 4097, "f16", residual=False, f8=False, gap=7),
        # the gated activation of a decode batch
        _quantise("quantise batch", 40, 14336, "f16"),
        # a layer's weights when a program loads them
        _quantise("quantise weights", 17408, 5120, block=128),
        # one token through the widest projection: the weights' bytes
        _product("product token", 1, 27648, 5120),
        # a decode batch, float32 scales as a checkpoint has them
        _product("product batch", 33, 5120, 14336, "f16", scales="f32"),
        # drafted tokens through a small projection: latency
        _product("product drafts", 5, 2048, 2048),
        # a chunk of ragged prompts, with rows of weights that do not fill a block
        _product("product chunk", 300, 4100, 4096),
        # a whole prompt
        _product("product prompt", 8192, 14336, 5120),
        # a decode batch far into long documents, frequencies stretched by 4, room for more tokens in the graph
        _rope("rope batch", 40, 40, 8, 128, 128, 131072, factor=4.0, pad=24),
        # a prompt, neighbours paired, a part of the head
        _rope("rope prompt", 8192, 32, 8, 128, 64, 8192, "f16", interleaved=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "quantise", "product", "product", "product", "rope"])
    type = rng.choice(["bf16", "f16"])
    gap = rng.choice([0, 0, 8, rng.randrange(1, 100)])
    if op == "norm":
        f8 = rng.random() < 0.6
        width = 128 * _spread(rng, 1, 128) if f8 or rng.random() < 0.4 else _spread(rng, 1, 16384)
        case = _norm("", _spread(rng, 1, min(40000, 40000000 // width)), width, type, rng.random() < 0.7, f8, gap)
    elif op == "quantise":
        width, block = 128 * _spread(rng, 1, 200), rng.choice([1, 1, 128])
        case = _quantise("", _spread(rng, 1, min(40000, 80000000 // width)), width, type, block, gap)
    elif op == "product":
        N, K = _spread(rng, 16, 32000), 128 * _spread(rng, 1, 136)
        M = rng.choice([1, _spread(rng, 2, 64), _spread(rng, 65, 1000), _spread(rng, 500, 8192)])
        N = max(1, min(N, 140000000 // K, 600000000000 // (M * K)))
        case = _product("", M, N, K, type, rng.choice(["e8m0", "f32"]))
    else:
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        tokens = _spread(rng, 1, max(2, 42000000 // ((heads + kv_heads) * dim)))
        case = _rope("", tokens, heads, kv_heads, dim, rng.choice([dim, dim, dim // 2, dim // 4]),
                     _spread(rng, tokens, 1000000), type, rng.random() < 0.5, rng.choice([1.0, 4.0, 32.0]),
                     rng.choice([0, 0, rng.randrange(1, 100)]))
    del case["name"]
    return case


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        out = n + n // 128 if case["f8"] else 0  # codes and scales, written and read back
        return {"bytes": 2 * n * (4 if case["residual"] else 2) + 2 * out + 2 * case["width"], "flops": 5 * n}
    if case["op"] == "quantise":
        n = case["rows"] * case["width"]
        return {"bytes": 4 * n + 2 * (n + n // (128 * case["block"])), "flops": 3 * n}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        each = 4 if case["scales"] == "f32" else 1
        return {"bytes": (M + N) * K + M * K // 128 + each * -(-N // 128) * K // 128 + 2 * M * N,
                "flops": 2 * M * N * K}
    cells = (case["tokens"] + case["pad"]) * (case["heads"] + case["kv_heads"])
    return {"bytes": 4 * cells * case["dim"] + 4 * case["tokens"], "flops": 3 * cells * case["rotary"]}


# ---------------------------------------------------------------------------------------------- inputs
def _rows(rows, width, gap, gen, dtype, outliers=0.0):
    """Rows `gap` elements apart; a few channels are several times larger than the others."""
    x = torch.randn((rows, width + gap), generator=gen, device=DEVICE)
    x *= 1 + outliers * (torch.rand(width + gap, generator=gen, device=DEVICE) < 0.01)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEVICE))
    return x.to(dtype)[:, :width]


def _eight(x, block):
    """Codes and scales of finite values x [M, K] in groups of 128 of `block` rows."""
    M, K = x.shape
    over = -M % block
    g = torch.nn.functional.pad(x, (0, 0, 0, over)).view(-1, block, K // 128, 128)
    m, e = torch.frexp(g.abs().amax((1, 3)))
    e = torch.where(m > 0, torch.where(m > 0.875, e - 8, e - 9), -127).clamp(min=-127)
    v = (g.double() * _two(-e)[:, None, :, None]).view(-1, K)[:M]
    return _nearest(v).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _nearest(v):
    """The e4m3 number next to each v of at most 448, in 64 bits: even at middles."""
    step = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4
    return torch.round(v * _two(-step)) * _two(step)


def _two(e):
    """2^e in 64 bits, exactly (a power function is off by a last digit here and there)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _power(scales):
    return _two(scales.view(torch.uint8).int() - 127)


def _frequencies(case):
    n = case["rotary"] // 2
    return 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=DEVICE) / n) / case["factor"]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, dtype = case["op"], TYPES[case["type"]]
    st = {"op": op, "dtype": dtype}
    if op == "norm":
        rows, width, gap = case["rows"], case["width"], case["gap"]
        st["x"] = _rows(rows, width, gap, gen, dtype)
        st["residual"] = _rows(rows, width, gap, gen, dtype, 20.0) if case["residual"] else None
        st["weight"] = (1 + 0.2 * torch.randn(width, generator=gen, device=DEVICE)).to(dtype)
        st["f8"] = case["f8"]
    elif op == "quantise":
        st["x"] = _rows(case["rows"], case["width"], case["gap"], gen, dtype, 20.0)
        st["block"] = case["block"]
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        st["x"], st["x_scales"] = _eight(_rows(M, K, 0, gen, torch.bfloat16, 20.0), 1)
        w = torch.randn((N, K), generator=gen, device=DEVICE) * K ** -0.5
        st["w"], st["w_scales"] = _eight(w.to(torch.bfloat16), 128)
        if case["scales"] == "f32":
            more = 0.5 + torch.rand(st["w_scales"].shape, generator=gen, device=DEVICE)
            st["w_scales"] = _power(st["w_scales"]).float() * more
    else:
        T, H, G, D = case["tokens"] + case["pad"], case["heads"], case["kv_heads"], case["dim"]
        # parts of the rows that a fused projection of queries, keys and values gives
        fused = torch.randn((T, H + 2 * G, D), generator=gen, device=DEVICE).to(dtype)
        st["q"], st["k"] = fused[:, :H], fused[:, H:H + G]
        at = torch.randint(0, case["far"], (case["tokens"],), generator=gen, device=DEVICE)
        st["positions"] = torch.cat((at, at.new_full((case["pad"],), -1))).int()
        st["frequencies"] = _frequencies(case)
        st["interleaved"], st["scale"] = case["interleaved"], 1 + 0.1 * math.log(case["factor"])
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["op"]
    if own:
        import matmul_affine_qmv_amd as qmx
        if op == "norm":
            if not st["f8"]:
                return qmx.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS)
            codes, scales, *total = qmx.rms_norm_f8(st["x"], st["weight"], st["residual"], eps=EPS)
            return [qmx.f8_dequantize(codes, scales, dtype=st["dtype"]), *total]
        if op == "quantise":
            codes, scales = qmx.f8_quantize(st["x"], block_rows=st["block"])
            return qmx.f8_dequantize(codes, scales, dtype=st["dtype"])
        if op == "product":
            return qmx.qmm_f8(st["w"], st["w_scales"], st["x"], st["x_scales"], dtype=st["dtype"])
        return qmx.rope(st["q"], st["k"], st["positions"], st["frequencies"], interleaved=st["interleaved"],
                        scale=st["scale"])
    if op == "norm":
        return _plain_norm(st)
    if op == "quantise":
        return _values(*_eight(st["x"], st["block"])).to(st["dtype"])
    if op == "product":
        return (_values(st["x"], st["x_scales"]) @ _values(st["w"], st["w_scales"]).T).to(st["dtype"])
    return _plain_rope(st)


def _values(codes, scales):
    """What codes [M, K] stand for, in 32 bits."""
    s = scales if scales.dtype == torch.float32 else _power(scales).float()
    if len(s) != len(codes):
        s = s.repeat_interleave(128, 0)[:len(codes)]
    return (codes.float().unflatten(1, (-1, 128)) * s[..., None]).flatten(1)


def _plain_norm(st):
    x, residual, total = st["x"], st["residual"], []
    if residual is not None:
        x = (x.float() + residual.float()).to(x.dtype)
        total = [x]
    if not st["f8"]:
        v = x.float()
        y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
        return [y.to(x.dtype), *total] if total else y.to(x.dtype)
    v = x.double()  # for what lies next to a border between two codes
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * st["weight"].double()
    return [_values(*_eight(y, 1)).to(x.dtype), *total]


def _plain_rope(st):
    n = len(st["frequencies"])
    angle = st["positions"].clamp(min=0).double()[:, None, None] * st["frequencies"]
    there = (st["positions"] >= 0)[:, None, None]
    cos, sin = (angle.cos() * st["scale"]).float(), (angle.sin() * st["scale"]).float()
    out = []
    for x in (st["q"], st["k"]):
        a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if st["interleaved"] else (x[..., :n], x[..., n:2 * n])
        a, b = a.float(), b.float()
        a, b = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((a, b), -1).flatten(-2) if st["interleaved"] else torch.cat((a, b), -1)
        out.append(torch.where(there, torch.cat((y.to(x.dtype), x[..., 2 * n:]), -1), x))
    return out


# ---------------------------------------------------------------------------------------------- in 64 bits
def _exact_eight(x, block):
    """What x stands for in 8 bits, value by value from the definition."""
    M, K = x.shape
    powers = torch.tensor([2.0 ** e for e in range(-128, 130)], dtype=torch.float64, device=x.device)
    out = torch.empty(M, K, dtype=torch.float64, device=x.device)
    for r in range(0, M, 128 if block == 128 else 4096):
        part = x[r:r + (128 if block == 128 else 4096)].double().unflatten(1, (K // 128, 128))
        most = part.abs().amax(2, keepdim=True)
        if block == 128:
            most = most.amax(0, keepdim=True)
        unit = powers[1 + torch.searchsorted(448 * powers[1:], most)]
        size = part.abs() / unit
        grid = torch.full_like(size, 2.0 ** -9)
        for e in range(-5, 9):
            grid[size >= 2.0 ** e] = 2.0 ** (e - 3)
        out[r:r + len(part)] = ((part / unit / grid).round() * grid * unit).flatten(1)
    return out


def _exact_product(st):
    M, K = st["x"].shape
    N = len(st["w"])
    ws = st["w_scales"]
    powers = torch.tensor([2.0 ** e for e in range(-127, 128)] + [math.nan], dtype=torch.float64, device=DEVICE)
    ws = ws.double() if ws.dtype == torch.float32 else powers[ws.view(torch.uint8).long()]
    xs = powers[st["x_scales"].view(torch.uint8).long()]
    x = (st["x"].double().view(M, K // 128, 128) * xs[:, :, None]).view(M, K)
    out = torch.empty(M, N, dtype=torch.float64, device=DEVICE)
    for n in range(0, N, 128):
        w = st["w"][n:n + 128].double().view(-1, K // 128, 128) * ws[n // 128][None, :, None]
        out[:, n:n + 128] = x @ w.view(-1, K).T
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h, total = st["x"], []
        if case["residual"]:
            h = (h.double() + st["residual"].double()).to(h.dtype)
            total = [h.double()]
        h = h.double()
        y = st["weight"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["width"] + EPS)
        if case["f8"]:
            return [_exact_eight(y, 1), *total]
        return [y, *total] if total else y
    if case["op"] == "quantise":
        return _exact_eight(st["x"], case["block"])
    if case["op"] == "product":
        return _exact_product(st)
    n, got = case["rotary"] // 2, []
    turn = st["positions"].double()[:, None] * _frequencies(case)[None]
    turn = torch.polar(torch.full_like(turn, st["scale"]), turn)[:, None]
    for x in (st["q"].double(), st["k"].double()):
        y = x.clone()
        first = slice(0, 2 * n, 2) if case["interleaved"] else slice(0, n)
        second = slice(1, 2 * n, 2) if case["interleaved"] else slice(n, 2 * n)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        got.append(torch.where((st["positions"] >= 0)[:, None, None], y, x))
    return got
