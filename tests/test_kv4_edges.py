"""The paged 4-bit key/value cache where types, lengths and arguments end: tokens of no request at either end,
subnormal groups, long tails, magnitudes far apart, and arguments that the entries refuse.

Bounds.  ``u`` is half a step of the type, 2^-24 that of float32.  For a token, with p its keys' probabilities:

* the output's rounding, u |out| (and half a subnormal step);
* few rows: p s enters the product with its code, taken about the middle of the codes, to ``held`` of itself;
* many rows: values and probabilities are float16, 2^-11 each; values also to 2^-18 of their token's largest, and a
  probability times a value to 2^-26 of the largest value that the token sees, for each key (the sum of exponentials
  is at least 1 of them);
* 32-bit sums, every product rounded and added at most ``steps`` times;
* key t's score is off by E_t, D products on 32-bit sums and the exponent's argument (many rows: and 2^-31 of the
  largest elements), which moves the output by sum p_t expm1(2 E_t) |v_t - out| and the logarithm of the sum by
  log sum p_t exp(E_t) at most.
"""
import math

import numpy as np
import pytest
import torch

import kv4_reference as ref
import matmul_affine_qmv_amd as qmx
from test_kv4 import DEV, FAKE, device_cache, fake_ptr_test, ints, on_gpu, say

U32 = ref.U32


def expected(c, q, table, kv, offsets, window=0, scale=None, prompt=False, held=2.0 ** -16):
    """(out, lse, bound of out, bound of lse) in float64 of q [T, heads, D] (torch, on the CPU)."""
    T, heads, D = q.shape
    each, scale = heads // c.heads, D ** -0.5 if scale is None else scale
    u, q = ref.HALF[c.type], q.double().numpy()
    out, lse = np.zeros((T, heads, D)), np.full((T, heads), -np.inf)
    tol, ltol = np.zeros((T, heads, D)), np.zeros((T, heads))
    rep = lambda a: np.repeat(a, c.group, -1)  # noqa: E731
    for r, length in enumerate(kv):
        n = offsets[r + 1] - offsets[r]
        pages = [int(x) for x in table[r]]
        ok = np.repeat([0 <= x < c.pages for x in pages], c.page)[:length]
        got = [x if 0 <= x < c.pages else 0 for x in pages]
        for a in range(heads):
            flat = lambda x: x[got, a // each].reshape(-1, x.shape[-1])[:length]  # noqa: E731
            ks, kb, vs, vb = (rep(flat(x[i])) for i in (0, 1) for x in (c.s, c.b))
            kc, vc = flat(c.codes[0]), flat(c.codes[1])
            for i in range(n):
                t, pos, key = offsets[r] + i, length - n + i, np.arange(len(ok))
                see = ok & (key <= pos) & (key > (pos - window if window else -1))
                if not see.any():
                    continue
                x, v = q[t, a], vc[see] * vs[see] + vb[see]
                s = (kc[see] * ks[see] + kb[see]) @ x * scale
                size = 16 * ks[see] + np.abs(kb[see])
                p = np.exp(s - s.max())
                total = p.sum()
                p /= total
                out[t, a], lse[t, a] = p @ v, s.max() + np.log(total)
                E = (D + 8) * U32 * scale * (size @ np.abs(x)) + 8 * U32 * (np.abs(s) + np.abs(s.max()) + 1)
                if prompt:
                    E += 2.0 ** -31 * scale * (np.abs(x).max() * size.sum(-1) + np.abs(x).sum() * size.max(-1))
                eps = np.where(p > 0, np.expm1(2 * np.minimum(E, 10)), 0)
                steps = see.sum() / 32 + 64
                if prompt:
                    most = np.abs(vs[see] * 15 + vb[see]).max(-1, keepdims=True)
                    most = np.maximum(most, np.abs(vb[see]).max(-1, keepdims=True))
                    lost = 2.0 ** -10 * np.abs(v) + 2.0 ** -18 * most
                    rounded = p @ lost + 2.0 ** -26 * most.max() * see.sum() / total
                else:
                    rounded = held * (p @ (vs[see] * np.abs(vc[see] - 8)))
                tol[t, a] = (u * np.abs(out[t, a]) + (2.0 ** -25 if c.type == "f16" else 2.0 ** -134) + rounded
                             + steps * U32 * (p @ (vs[see] * (ref.OFF + 23) + np.abs(vb[see])))
                             + (p * eps) @ np.abs(v - out[t, a]) / max(1 - (p * eps).sum(), 0.01))
                up = s - lse[t, a] + E
                ltol[t, a] = up.max() + np.log(np.exp(up - up.max()).sum()) + steps * U32 + 2 * U32 * abs(lse[t, a])
    return out, lse, tol, ltol


def tables(lens, page):
    """A block table that hands pages out in order, and the number of pages."""
    need = [-(-x // page) for x in lens]
    table, first = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = np.arange(first, first + n)
        first += n
    return table, first


def held_to(c, q, table, kv, offsets, scale=None, window=0, **bound):
    """A call's outputs against `expected`, which it has to meet and to repeat."""
    each, n = q.shape[1] // c.heads, int(np.diff(offsets).max())
    prompt = n * each > 64
    for x in (*c.s, *c.b):
        x[:] = torch.from_numpy(x).to(c.dtype).double().numpy()
    args = (device_cache(c), q.to(DEV), torch.from_numpy(table).to(DEV), ints(kv), ints(offsets))
    kw = dict(max_query_len=n, max_kv_len=max(kv), scale=scale, window=window)
    out, lse = qmx.kv4_attention(*args, return_lse=True, **kw)
    o, l, tol, ltol = expected(c, q, table, kv, offsets, window, scale, prompt, **bound)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all(), "not finite"
    over = np.abs(got - o) - tol
    assert (over <= 0).all(), (over.max(), tol.flat[over.argmax()], np.unravel_index(over.argmax(), over.shape))
    none = np.isneginf(l)
    assert np.array_equal(np.isneginf(got_lse), none)
    assert (np.abs(got_lse[~none] - l[~none]) <= ltol[~none]).all(), np.abs(got_lse - l)[~none].max()
    assert torch.equal(out, qmx.kv4_attention(*args, **kw)), "rerun not bit-identical"


@on_gpu
@pytest.mark.parametrize("new,past", [(1, 40), (2, 3000), (50, 10), (60, 3000)])
@pytest.mark.parametrize("before,behind", [(3, 0), (2, 4)])
def test_tokens_before_the_first_offset(new, past, before, behind):
    """Tokens before query_offsets[0] belong to no request, as those behind the last: zeros, and -inf."""
    say("before", new, past, before, behind)
    rng = np.random.default_rng(30)
    kv = [past + new, 20]
    table, pages = tables(kv, 16)
    cache = device_cache(ref.Cache(pages, 2, 64, 16, 32, "bf16", rng))
    T = before + 2 * new + behind
    q = torch.from_numpy(rng.normal(0, 1, (T, 4, 64))).bfloat16().to(DEV)
    table = torch.from_numpy(table).to(DEV)
    kw = dict(max_query_len=new, max_kv_len=max(kv), return_lse=True)
    want, want_lse = qmx.kv4_attention(cache, q[before:], table, ints(kv), ints([0, new, 2 * new]), **kw)
    left = torch.full((T, 4), 7.0, device=DEV)   # what lse's memory may hold
    del left
    out, lse = qmx.kv4_attention(cache, q, table, ints(kv), ints([before, before + new, before + 2 * new]),
                                 out=torch.full_like(q, 7.0), **kw)
    assert torch.equal(out[before:], want) and torch.equal(lse[before:], want_lse)
    assert not out[:before].any() and torch.isneginf(lse[:before]).all()


@on_gpu
@pytest.mark.parametrize("first", [0, 2, 9])
def test_no_requests_and_a_first_offset(first):
    """No request, or a first offset behind all tokens: nothing but zeros."""
    say("no requests", first)
    cache = qmx.Kv4Cache.zeros(2, 1, 64, page_size=16, group_size=32, device=DEV)
    q = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = qmx.kv4_attention(cache, q, torch.zeros(0, 1, dtype=torch.int32, device=DEV), none, ints([first]),
                            max_query_len=1, max_kv_len=16, out=torch.full_like(q, 7.0))
    assert not out.any()
    out = qmx.kv4_attention(cache, q, ints([[0]]), ints([3]), ints([first + 5, first + 6]), max_query_len=1,
                            max_kv_len=16, out=torch.full_like(q, 7.0))
    assert not out.any()


@on_gpu
def test_maps_of_all_the_tokens_that_an_int_counts():
    """Room for 2^31 - 1 tokens: the last step of a group's walk passes that number."""
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    say("maps of 2^31 - 1 tokens")
    got = qmx.kv_maps(ints([0, 5]), ints([100, T - 150]), ints([[0, -1], [1, 2]]), ints([7]), page_size=64, tokens=T)
    assert got.query_offsets.tolist() == [0, 100, T - 50] and got.kv_lens.tolist() == [100, T - 145]
    assert got.counts.tolist() == [T - 50, 3]
    step = 1 << 28
    for begin in range(0, T, step):
        t = torch.arange(begin, min(T, begin + step), dtype=torch.int32, device=DEV)
        part = slice(begin, begin + t.numel())
        behind, second = t >= T - 50, t >= 100
        ids = second.int().masked_fill_(behind, -1)
        assert torch.equal(got.request_ids[part], ids)
        at = torch.where(second, t - 95, t).masked_fill_(behind, -1)
        assert torch.equal(got.positions[part], at)
        slot = torch.where(second, at.clamp(max=64) + 64, at.clamp(max=64) + 7 * 64)   # each request has one page
        slot = slot.masked_fill_((at >= 64) | behind, -1)
        assert torch.equal(got.slots[part], slot)


EOVERLAP, ELAUNCH = -12, -9


def maps_status(at, R=3, columns=4, stride=7, nfree=5, T=8):
    """qmx_kv_maps on placeholder pointers, by the first int of each argument."""
    place = dict(past=0, fresh=100, table=200, free=300, query_offsets=400, kv_lens=500, slots=600, positions=700,
                 request_ids=800, counts=900)
    place.update(at)
    p = {k: FAKE + 4 * v for k, v in place.items()}
    return qmx.lib().qmx_kv_maps(p["past"], p["fresh"], p["table"], p["free"], R, columns, stride, nfree, 16, T,
                                 p["query_offsets"], p["kv_lens"], p["slots"], p["positions"], p["request_ids"],
                                 p["counts"], None)


@fake_ptr_test
def test_maps_refuse_outputs_over_inputs():
    """The launch's groups read the lengths while one of them writes: kv_lens as the next step's past, in place, gave
    slots that depended on which came first."""
    assert maps_status({}) != EOVERLAP                                    # no device here: the launch fails
    for bad in (dict(past=500), dict(past=502), dict(past=498), dict(fresh=500), dict(free=402), dict(past=599),
                dict(past=607), dict(free=901), dict(counts=304), dict(slots=701), dict(request_ids=705),
                dict(positions=593), dict(kv_lens=403), dict(kv_lens=200), dict(kv_lens=203), dict(kv_lens=206),
                dict(kv_lens=217), dict(slots=193), dict(past=214), dict(free=199), dict(counts=206),
                dict(fresh=215)):
        assert maps_status(bad) == EOVERLAP, bad
    # inputs may share memory; what stands beside, between the table's rows, or behind its last row does not overlap
    for good in (dict(past=100), dict(past=301), dict(kv_lens=404), dict(kv_lens=204), dict(past=211), dict(past=218),
                 dict(past=197), dict(slots=192), dict(counts=204), dict(counts=198)):
        assert maps_status(good) == ELAUNCH, good
    assert maps_status(dict(kv_lens=200), columns=0) == ELAUNCH
    assert maps_status(dict(kv_lens=201), R=1, stride=0) == EOVERLAP
    assert maps_status(dict(kv_lens=204), R=1, stride=0) == ELAUNCH
    assert maps_status({}, stride=2 ** 62) == ELAUNCH and maps_status(dict(past=199), stride=2 ** 62) == EOVERLAP
    assert "overlaps" in qmx.strerror(EOVERLAP)


@on_gpu
def test_binding_refuses_outputs_over_inputs():
    """The lengths that a step wrote, given back to the same KvMaps as the next step's past."""
    say("maps over their inputs")
    table, free, one = ints([[0, -1], [1, -1]]), ints([2, 3]), ints([1, 1])
    maps = qmx.kv_maps(ints([15, 3]), one, table, free, page_size=16, tokens=2)
    with pytest.raises(qmx.QmxError, match="overlaps"):
        qmx.kv_maps(maps.kv_lens, one, table, free, page_size=16, out=maps)
    with pytest.raises(qmx.QmxError, match="overlaps"):
        qmx.kv_maps(one, one, maps.slots.view(2, 1), free, page_size=16, out=maps)
    assert maps.kv_lens.tolist() == [16, 4] and table.tolist() == [[0, -1], [1, -1]]
    maps = qmx.kv_maps(maps.kv_lens.clone(), one, table, free, page_size=16, out=maps)
    assert maps.kv_lens.tolist() == [17, 5] and maps.slots.tolist() == [32, 20]


SIZES = [(8, 128, 64, 64, 32, 4096, 8000, 0), (8, 128, 64, 64, 32, 512, 8192, 0), (2, 64, 3, 5, 4, 9, 4000, 0),
         (4, 256, 1, 40, 16, 2048, 70000, 0), (1, 64, 20, 20, 8, 300, 9000, 2000)]


@pytest.mark.parametrize("sizes", SIZES)
def test_workspace_of_a_bound_above_the_tokens(sizes):
    """kv4_attention takes no more queries a request than there are tokens; the size it is given has to be for that."""
    bytes_ = qmx.lib().qmx_kv4_attention_workspace_bytes
    kv_heads, dim, R, T, heads, most, kv, window = sizes
    assert bytes_(*sizes) == bytes_(kv_heads, dim, R, T, heads, T, kv, window) > 0


@on_gpu
@pytest.mark.parametrize("each,D,most", [(4, 64, 512), (1, 128, 3), (2, 256, 2000)])
@pytest.mark.parametrize("new", [1, 2, 40])
def test_workspace_of_the_caller(each, D, most, new):
    """A workspace of the size that kv4_attention_workspace_bytes says, with a bound of the queries above the tokens and
    without, gives what the call's own gives; one byte less is refused."""
    say("workspace", each, D, most, new)
    rng = np.random.default_rng(33)
    kv = [3000, 1700, 9]
    table, pages = tables(kv, 64)
    cache = device_cache(ref.Cache(pages, 2, D, 64, 64, "bf16", rng))
    offsets = [0, new, 2 * new, 2 * new + 1]
    T, heads = offsets[-1], 2 * each
    q = torch.from_numpy(rng.normal(0, 1, (T, heads, D))).bfloat16().to(DEV)
    args = (cache, q, torch.from_numpy(table).to(DEV), ints(kv), ints(offsets))
    need = qmx.kv4_attention_workspace_bytes(cache, 3, T, heads, most, 3000)
    assert need > 0
    kw = dict(max_query_len=most, max_kv_len=3000)
    want = qmx.kv4_attention(*args, **kw)
    room = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(want, qmx.kv4_attention(*args, workspace=room, **kw))
    assert torch.equal(want, qmx.kv4_attention(*args, workspace=room, **kw))   # over what the last call left there
    with pytest.raises(qmx.QmxError, match="workspace"):
        qmx.kv4_attention(*args, workspace=room[:need - 1], **kw)


@on_gpu
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("power", range(-133, -95, 3))
def test_write_of_tiny_groups(D, group, power):
    """bfloat16 groups whose scale is subnormal, or just above: codes, scales and biases bit for bit, and back.  Reading
    rounds to bfloat16, half a step of which is 2^-134 down there."""
    say("tiny", D, group, power)
    rng = np.random.default_rng(200 - power)
    T, H = 40, 2
    x = [rng.normal(0, 1, (T, H, D)) * 2.0 ** power for _ in range(2)]
    x[0][::2] = rng.integers(0, 31, x[0][::2].shape) * 2.0 ** power    # middles between codes
    x[1][::2] = rng.integers(-200, 200, x[1][::2].shape) * 2.0 ** power
    x[1][1] = 2.0 ** (power + 20)                                       # one value
    k, v = (torch.from_numpy(a).bfloat16() for a in x)
    c = ref.Cache(3, H, D, 16, group, "bf16", rng)
    cache = device_cache(c)
    slots = np.arange(5, 5 + T)
    qmx.kv4_write(cache, k.to(DEV), v.to(DEV), ints(slots.tolist()))
    got = qmx.kv4_read(cache, ints(slots.tolist()))
    P, at = slots // 16, slots % 16
    for which, a in ((0, k), (1, v)):
        c.codes[which][P, :, at], c.s[which][P, :, at], c.b[which][P, :, at] = ref.quantise(a, group, torch.bfloat16)
    for name, g, w in zip(("k_codes", "k_sb", "v_codes", "v_sb"),
                          (cache.k_codes, cache.k_sb, cache.v_codes, cache.v_sb), c.packed()):
        assert torch.equal(g.cpu(), w), name
    for which, g in enumerate(got):
        exact = np.stack([[c.values(which, P[t], h)[at[t]] for h in range(H)] for t in range(T)])
        size = (ref.HALF["bf16"] + 32 * U32) * np.abs(exact) + 2.0 ** -134
        assert (np.abs(g.double().cpu().numpy() - exact) <= size + 15 * U32 * np.abs(exact).max()).all()


@on_gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("keys,above,size", [(1200, 9.0, 2.0 ** -13), (6000, 9.0, 1e-3), (30000, 10.0, 5e-4),
                                             (60000, 11.0, 1e-3)])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_long_tail_behind_one_key(dtype, D, group, keys, above, size):
    """One key far above a long tail of keys, whose values are small: each of the tail's products is tiny and their sum
    is not.  The codes are alike from token to token, so nothing that is lost cancels.  p s is held in 16 bits."""
    say("tail", dtype, D, group, keys, above)
    rng = np.random.default_rng(keys + D)
    page = 64
    table, pages = tables([keys], page)
    c = ref.Cache(pages, 1, D, page, group, dtype, rng)
    q = torch.from_numpy(rng.uniform(0.5, 1.5, (1, 1, D))).to(ref.TYPES[dtype])
    round_ = lambda x: torch.from_numpy(np.asarray(x)).to(ref.TYPES[dtype]).double().numpy()  # noqa: E731
    x = q.double().numpy()[0, 0]
    c.s[0][:] = round_(rng.uniform(0.02, 0.06, c.s[0].shape) * 8 / D ** 0.5)
    c.b[0][:] = round_(-7.5 * c.s[0])
    c.s[0][0, :, 0], c.b[0][0, :, 0] = 0, round_(above / (x.sum() * D ** -0.5))
    c.codes[1][:] = rng.choice([0, 15], D)
    c.s[1][:] = round_(rng.uniform(0.5, 1.5, c.s[1].shape) * size)
    c.b[1][:] = round_(-7.5 * c.s[1])
    c.s[1][0, :, 0] = c.b[1][0, :, 0] = 0
    held_to(c, q, table, [keys], [0, 1])


@on_gpu
@pytest.mark.parametrize("new,past", [(40, 50), (1, 90), (60, 2000), (2, 2000)])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("power,key_power", [(-40, None), (-120, None), (-76, -76), (-130, 0), (-100, 90), (90, -100),
                                             (-20, -120), (120, -130)])
def test_scores_that_vanish(new, past, D, group, power, key_power):
    """Keys that are all zeros, or queries and keys whose powers of two together leave the range of float32: finite
    inputs give finite outputs, and scores of nothing the mean of what is seen."""
    say("vanish", new, past, D, group, power, key_power)
    rng = np.random.default_rng(41)
    kv = [past + new, 7]
    table, pages = tables(kv, 32)
    c = ref.Cache(pages, 1, D, 32, group, "bf16", rng)
    for x in (c.s[0], c.b[0]):
        x *= 0.0 if key_power is None else 2.0 ** key_power
        x[:] = torch.from_numpy(x).bfloat16().double().numpy()
    offsets = [0, new, new + min(new, 7)]
    q = torch.from_numpy(rng.normal(0, 1, (offsets[-1], 2, D)) * 2.0 ** power).bfloat16()
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30])
def test_tiny_softmax_scales(dtype, new, scale):
    say("scale", dtype, new, scale)
    rng = np.random.default_rng(42)
    kv = [100 + new]
    table, pages = tables(kv, 16)
    c = ref.Cache(pages, 1, 64, 16, 32, dtype, rng)
    q = torch.from_numpy(rng.normal(0, 2.0 ** -12, (new, 2, 64))).to(ref.TYPES[dtype])
    held_to(c, q, table, kv, [0, new], scale=scale)


def spread_case(dtype, D, group, lens, seed, page=32, heads=1):
    rng = np.random.default_rng(seed)
    kv = [p + n for p, n in lens]
    table, pages = tables(kv, page)
    c = ref.Cache(pages, heads, D, page, group, dtype, rng)
    offsets = [0] + np.cumsum([n for _, n in lens]).tolist()
    q = torch.from_numpy(rng.normal(0, 1, (offsets[-1], 2 * heads, D))).to(ref.TYPES[dtype])
    return rng, c, q, table, kv, offsets


def at(table, page, r, t):
    return table[r, t // page], slice(None), t % page


FAR = {"bf16": 2.0 ** 60, "f16": 2.0 ** 12}


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 128), (256, 32), (256, 64)])
@pytest.mark.parametrize("lens", [[(0, 50), (70, 33)], [(1900, 40)]])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
def test_hidden_tokens_cost_nothing(dtype, D, group, lens, what):
    """Tokens of huge keys or values that only the last queries see leave the others' digits alone."""
    say("hidden", dtype, D, group, lens, what)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, lens, 50)
    for x in (c.s[0], c.b[0], c.s[1], c.b[1]):
        x *= 2.0 ** -6
    for r, length in enumerate(kv):
        for t in (length - 1, length - 7, length - 12):
            for i in ((0,), (1,), (0, 1))[("keys", "values", "both").index(what)]:
                c.s[i][at(table, 32, r, t)] *= FAR[dtype]
                c.b[i][at(table, 32, r, t)] *= FAR[dtype]
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("new", [1, 50])
def test_keys_far_above_their_neighbours(dtype, D, group, new):
    """Keys of huge elements whose scores are far below the others': they take part in no output and in no rounding."""
    say("neighbours", dtype, D, group, new)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, [(90, new)], 53)
    q = q.abs() + 0.25
    big = {"bf16": 2.0 ** 30, "f16": 2.0 ** 11}[dtype]
    for t in (3, 17, 40, 41):
        c.s[0][at(table, 32, 0, t)], c.b[0][at(table, 32, 0, t)] = big, -16 * big
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("new", [1, 50])
def test_queries_with_elements_that_meet_zeros(dtype, D, group, new):
    """A group of large query elements on keys that are zeros there: the others' products keep their digits."""
    say("queries", dtype, D, group, new)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, [(90, new)], 54)
    c.s[0][..., 0] = c.b[0][..., 0] = 0
    q[..., :group] *= 2.0 ** 13
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("window", [20, 100])
def test_tokens_before_the_window_cost_nothing(dtype, D, group, window):
    say("window", dtype, D, group, window)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, [(160, 40), (0, 50)], 51)
    for x in (c.s[0], c.b[0], c.s[1], c.b[1]):
        x *= 2.0 ** -6
    for r, t in ((0, 62), (0, 145), (0, 150), (1, 1)):
        for x in (c.s[0], c.b[0], c.s[1], c.b[1]):
            x[at(table, 32, r, t)] *= FAR[dtype]
    held_to(c, q, table, kv, offsets, window=window)


@on_gpu
@pytest.mark.parametrize("dtype,powers", [("bf16", 1), ("bf16", 4), ("bf16", 12), ("bf16", 40), ("f16", 1), ("f16", 4),
                                          ("f16", 7)])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("lens", [[(0, 70), (90, 40)], [(1800, 50)]])
def test_magnitudes_of_every_token(dtype, powers, D, group, lens):
    """Values that differ from token to token by up to 4 ** powers; a stretch of zeros."""
    say("powers", dtype, powers, D, group, lens)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, lens, 52 + powers)
    factor = 2.0 ** rng.integers(-powers, powers + 1, (*c.s[1].shape[:3], 1))
    for x in (c.s[1], c.b[1]):
        x *= factor
        x[:] = torch.from_numpy(x).to(ref.TYPES[dtype]).double().numpy()
        x[1] = 0
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("lens", [[(0, 70), (90, 40)], [(1800, 50)]])
def test_rising_and_falling_values(D, group, lens):
    """Values that rise by 2^40 over a request, and fall again."""
    say("rising", D, group, lens)
    rng, c, q, table, kv, offsets = spread_case("bf16", D, group, lens, 60)
    for r, length in enumerate(kv):
        for t in range(length):
            for x in (c.s[1], c.b[1]):
                x[at(table, 32, r, t)] *= 2.0 ** round(40 * math.sin(math.pi * t / length))
    held_to(c, q, table, kv, offsets)


@on_gpu
@pytest.mark.parametrize("dtype,limit", [("f16", 0.60), ("bf16", 0.45)])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 128)])
def test_prompts_add_little_to_the_rounding_of_the_output(dtype, limit, D, group):
    """The root mean square of what a prompt's outputs are off, beside that of their own rounding. A rounding is off
    by u / sqrt(3) at a mantissa of 1 and half that at 2, r = 0.424 u over log-even mantissas, and a sum of random
    signs keeps that relative to itself. A float16 output has r of its own; one more, the values', gives sqrt(2) r =
    0.60 u (a third, the probabilities' as one float16 number, gave 0.63 to 0.66 u). A bfloat16 output's own r is of
    2^-8, whose square two at 2^-11 raise by 2 / 64: 0.43, under 0.45 of 2^-8 with 9000 and more outputs drawn."""
    say("rounding", dtype, D, group)
    rng, c, q, table, kv, offsets = spread_case(dtype, D, group, [(400, 64), (0, 90)], 70)
    for x in (c.s[0], c.b[0]):   # scores of about 1
        x *= 0.3
    for x in (*c.s, *c.b):
        x[:] = torch.from_numpy(x).to(c.dtype).double().numpy()
    out = qmx.kv4_attention(device_cache(c), q.to(DEV), torch.from_numpy(table).to(DEV), ints(kv), ints(offsets),
                            max_query_len=90, max_kv_len=max(kv)).double().cpu().numpy()
    want = expected(c, q, table, kv, offsets, prompt=True)[0]
    off = np.sqrt(((out - want) ** 2).mean() / (want ** 2).mean())
    assert off <= limit * ref.HALF[dtype], off / ref.HALF[dtype]
