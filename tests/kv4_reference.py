"""The paged 4-bit key/value cache in 64 bits on the CPU, from the definition in
include/qmx.h: one token, head or request at a time, with numpy.

``attention`` also returns how far a result may be off, from the kernels'
roundings alone (``u`` is half a step of the type, 2^-24 that of float32):

* the output's rounding, u |out|;
* that of each p_t s_tg to the type before it meets the code, taken about the
  middle of the codes: u sum_t p_t s_tg |c_td - 8| (in float16 also half the
  smallest subnormal step, 2^-25, for each of the keys);
* 32-bit sums: every product is rounded and added at most `steps` times, with
  codes offset by up to OFF + 15: steps 2^-24 sum_t p_t (s_tg (OFF + 23) + |b|);
* the scores' 32-bit error E_t (the same count on q's side, and the exponent's
  argument): p_t moves by a factor of at most exp(2 max E), so the output by
  expm1(2 max E) sum_t p_t |v_t - out|.

``prompt``: the kernel of many rows rounds other things.  Values and
probabilities to float16, 2 * 2^-11 sum_t p_t |v_td|, in place of p_t s_tg, or
2^-24 of the request's largest value each (a power of two above it at most twice
it; probabilities down to 2^-25 a key, and those scaled with it); queries to
float16, 2^-24 of the row's largest, and bfloat16 keys' scaled codes, 2^-24 of
their block's largest, which enters E_t.
"""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # the largest rounding, relative
U32 = 2.0 ** -24
OFF = 128.0


def key_place(D, t, d):
    """(word, bit) of element d of token t in a block of keys."""
    h, j, e = d // 8 % 4, d // 32, d % 8
    return (h * 16 + t) * (D // 32) + j, 4 * (e // 2) + 16 * (e % 2)


def value_place(D, t, d):
    a, f, n = d // 64, d // 16 % 4, d % 16
    half = ((t // 4 * 16 + n) * (D // 64) + a) * 4 + t % 4
    return half // 2, 16 * (half % 2) + 4 * f


def quantise(x, group, dtype):
    """Codes, scales and biases (float64 numpy) of x [..., D] (torch, dtype)."""
    g = x.double().numpy().reshape(*x.shape[:-1], -1, group)
    lo, hi = g.min(-1), g.max(-1)
    s = torch.from_numpy((hi - lo) / 15).to(dtype).double().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.clip(np.rint((g - lo[..., None]) / s[..., None]), 0, 15)
    c = np.where(s[..., None] == 0, 0, c)
    return c.reshape(x.shape).astype(np.int64), s, lo


class Cache:
    """Codes, scales and biases [pages, heads, page, ...] and their packed form."""

    def __init__(self, pages, heads, dim, page, group, dtype, rng):
        self.page, self.group, self.dtype, self.dim = page, group, TYPES[dtype], dim
        self.type, self.heads, self.pages = dtype, heads, pages
        cells = (pages, heads, page)
        self.codes = [rng.integers(0, 16, (*cells, dim)) for _ in range(2)]
        self.s, self.b = [], []
        for _ in range(2):
            s = torch.from_numpy(rng.uniform(0.05, 0.4, (*cells, dim // group))).to(self.dtype)
            b = torch.from_numpy(rng.normal(0, 0.4, s.shape)).to(self.dtype).double() - 7.5 * s.double()
            self.s.append(s.double().numpy())
            self.b.append(b.to(self.dtype).double().numpy())

    def packed(self):
        """k_codes, k_sb, v_codes, v_sb as CPU tensors."""
        out = []
        for which, place in ((0, key_place), (1, value_place)):
            c, D = self.codes[which], self.dim
            P, H, page, _ = c.shape
            words = np.zeros((P, H, page // 16, 2 * D), dtype=np.uint64)
            for t in range(16):
                w, bit = zip(*(place(D, t, d) for d in range(D)))
                at = c[:, :, t::16, :].astype(np.uint64) << np.array(bit, dtype=np.uint64)
                for d in range(D):
                    words[..., w[d]] |= at[..., d]
            words = words.reshape(P, H, -1).astype(np.uint32).view(np.int32)
            sb = torch.from_numpy(np.stack((self.s[which], self.b[which]), -1)).to(self.dtype)
            out += [torch.from_numpy(words), sb]
        return out

    def values(self, which, page, head):
        rep = lambda x: np.repeat(x[page, head], self.group, -1)  # noqa: E731
        return self.codes[which][page, head] * rep(self.s[which]) + rep(self.b[which])


def maps(past, new, table, free, page, T):
    """offsets, kv_lens, slots, positions, request ids, counts; `table` changes."""
    R, columns = table.shape
    offsets, kv, slots, at_, ids = [0], [], [-1] * T, [-1] * T, [-1] * T
    used = 0
    for r in range(R):
        p, n = max(past[r], 0), max(new[r], 0)
        n = min(n, T - offsets[-1])
        held = min(-(-p // page), columns)
        for c in range(held, min(-(-(p + n) // page), columns)):
            table[r, c] = free[used] if used < len(free) else -1
            used += 1
        for i in range(n):
            t, at = offsets[-1] + i, p + i
            ids[t], at_[t] = r, at
            if at // page < columns and table[r, at // page] >= 0:
                slots[t] = table[r, at // page] * page + at % page
        kv.append(p + n)
        offsets.append(offsets[-1] + n)
    return offsets, kv, slots, at_, ids, [sum(max(x, 0) for x in new), used]


def attention(cache, q, table, kv_lens, offsets, window=0, scale=None, prompt=False):
    """(out, lse, bound of out, bound of lse), float64, q [T, heads, D] torch on the CPU."""
    T, heads, D = q.shape
    each = heads // cache.heads
    scale = D ** -0.5 if scale is None else scale
    q = q.double().numpy()
    out, lse = np.zeros((T, heads, D)), np.full((T, heads), -np.inf)
    tol, lse_tol = np.zeros((T, heads, D)), np.zeros((T, heads))
    u = HALF[cache.type]
    for r in range(len(kv_lens)):
        n, kv = offsets[r + 1] - offsets[r], kv_lens[r]
        for h in range(cache.heads):
            pages = [int(x) for x in table[r]]
            ok = np.repeat([0 <= x < cache.pages for x in pages], cache.page)[:kv]
            got = [x if 0 <= x < cache.pages else 0 for x in pages]
            flat = lambda a: a[got, h].reshape(-1, a.shape[-1])[:kv]  # noqa: E731
            rep = lambda a: np.repeat(a, cache.group, -1)  # noqa: E731
            ks, kb, vs, vb = (rep(flat(x[i])) for i in (0, 1) for x in (cache.s, cache.b))
            kc, vc = flat(cache.codes[0]), flat(cache.codes[1])
            for i in range(n):
                pos = kv - n + i
                key = np.arange(len(ok))
                see = ok & (key <= pos) & (key > (pos - window if window else -1))
                if not see.any():
                    continue
                k = kc[see] * ks[see] + kb[see]
                v = vc[see] * vs[see] + vb[see]
                for a in range(h * each, (h + 1) * each):
                    t = offsets[r] + i
                    x = q[t, a]
                    s = k @ x * scale
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    p /= total
                    out[t, a] = p @ v
                    lse[t, a] = m + np.log(total)
                    size = ((OFF + 15) * ks[see] + np.abs(kb[see]) + OFF * ks[see]) @ np.abs(x) * abs(scale)
                    err = (D + 8) * U32 * size.max() + 8 * U32 * (np.abs(s).max() + 1)
                    if prompt:
                        err += 2.0 ** -24 * scale * (np.abs(x).max() * np.abs(k).sum(-1).max()
                                                     + np.abs(x).sum() * (ks[see] * 8 + np.abs(kb[see])).max())
                    steps = see.sum() / 32 + 64
                    spread = p @ np.abs(v - out[t, a])
                    held = u * (p @ (vs[see] * np.abs(vc[see] - 8)))
                    if prompt:
                        held = 2.0 ** -10 * (p @ np.abs(v)) + 2.0 ** -24 * np.abs(vc * vs + vb).max() * (1 + see.sum() / total)
                    tol[t, a] = (u * np.abs(out[t, a]) + held
                                 + steps * U32 * (p @ (vs[see] * (OFF + 23) + np.abs(vb[see])))
                                 + np.expm1(2 * err) * spread)
                    if cache.type == "f16":
                        tol[t, a] += 4 * see.sum() * 2.0 ** -25 * 8 / total
                    lse_tol[t, a] = err + steps * U32 + 2 * U32 * abs(lse[t, a])
    return out, lse, tol, lse_tol
