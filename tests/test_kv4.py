"""The paged 4-bit key/value cache: refusals, and the reference's own layout, on
the CPU; the operators against the 64-bit reference of kv4_reference.py on a GPU.
"""
import ctypes
import math
import os
import sys

import numpy as np
import pytest
import torch

import kv4_reference as ref
import matmul_affine_qmv_amd as qmx
from matmul_affine_qmv_amd.kv4 import _CCache

if not os.path.exists(qmx.LIB_PATH):
    pytest.skip("libqmx.so not built", allow_module_level=True)

OK, ENULL, ESHAPE, EGROUP, EDTYPE, EALIGN, EWS = 0, -1, -2, -4, -5, -6, -7
F32, F16, BF16 = 0, 1, 2
FAKE, ODD = 0x10000, 0x10001
DEV = "cuda:0"


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


# ---------------------------------------------------------------- on the CPU
# Placeholder pointers must never reach a kernel: with a GPU in sight these are skipped.
fake_ptr_test = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder pointers: CPU-only checks")


def ccache(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=4, heads=2, dim=128, page=16, group=64, dt=BF16):
    return ctypes.byref(_CCache(kc, ks, vc, vs, pages, heads, dim, page, group, dt))


BAD_CACHES = [(dict(dt=F32), EDTYPE), (dict(dt=7), EDTYPE), (dict(dim=96), ESHAPE), (dict(dim=0), ESHAPE),
              (dict(group=16), EGROUP), (dict(dim=64, group=128), EGROUP), (dict(page=8), ESHAPE),
              (dict(page=48), ESHAPE), (dict(page=2048), ESHAPE), (dict(pages=-1), ESHAPE), (dict(heads=0), ESHAPE),
              (dict(kc=None), ENULL), (dict(vs=None), ENULL), (dict(ks=0x10004), EALIGN), (dict(vc=0x10008), EALIGN)]


@fake_ptr_test
@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=lambda x: str(x))
def test_cache_refusals(bad, status):
    L, c = qmx.lib(), ccache(**bad)
    assert L.qmx_kv4_write(c, FAKE, FAKE, 256, 128, 256, 128, FAKE, 4, None) == status
    assert L.qmx_kv4_read(c, FAKE, FAKE, FAKE, 4, None) == status
    assert attention(c) == status


def attention(c, q=FAKE, out=FAKE, lse=None, table=FAKE, columns=8, stride=8, lens=FAKE, offsets=FAKE, R=2, T=2,
              heads=8, max_q=1, max_kv=100, window=0, scale=0.1, ws=None, wsb=0):
    return qmx.lib().qmx_kv4_attention(c, q, 1024, 128, out, lse, table, columns, stride, lens, offsets, R, T, heads,
                                       max_q, max_kv, window, scale, ws, wsb, None)


@fake_ptr_test
def test_attention_refusals():
    c = ccache()
    for bad in (dict(heads=7), dict(heads=0), dict(R=-1), dict(T=-1), dict(columns=-1), dict(max_q=-1),
                dict(max_q=3), dict(max_kv=-1), dict(window=-1), dict(scale=math.nan), dict(scale=math.inf), dict(scale=0.0), dict(scale=-0.1),
                dict(stride=7), dict(max_kv=2 ** 31 - 1), dict(columns=2 ** 30, stride=2 ** 30)):
        assert attention(c, **bad) == ESHAPE, bad
    for bad in (dict(q=None), dict(out=None), dict(offsets=None), dict(lens=None), dict(table=None)):
        assert attention(c, **bad) == ENULL, bad
    for bad in (dict(q=ODD), dict(out=0x10008), dict(lse=0x10002), dict(table=0x10002), dict(lens=0x10001),
                dict(offsets=0x10002)):
        assert attention(c, **bad) == EALIGN, bad
    need = qmx.lib().qmx_kv4_attention_workspace_bytes(2, 128, 2, 2, 8, 1, 100000, 0)
    assert need > 0
    assert attention(c, max_kv=100000) == EWS
    assert attention(c, max_kv=100000, ws=FAKE, wsb=need - 1) == EWS
    assert attention(c, max_kv=100000, ws=0x10008, wsb=need) == EWS
    assert attention(c, T=0, max_q=0, q=None, out=None) == OK
    assert attention(None) == ENULL
    for bad in ((0, 128, 2, 2, 8, 1, 9999, 0), (3, 128, 2, 2, 8, 1, 9999, 0), (2, 96, 2, 2, 8, 1, 9999, 0),
                (2, 128, 2, 2, 8, 1, -1, 0), (2, 128, 2, 2, 8, 1, 9999, -1)):
        assert qmx.lib().qmx_kv4_attention_workspace_bytes(*bad) == 0


@fake_ptr_test
def test_maps_write_read_refusals():
    L = qmx.lib()

    def maps(past=FAKE, fresh=FAKE, table=FAKE, free=FAKE, R=2, columns=4, stride=4, nfree=3, page=16, T=8,
             out=(FAKE,) * 6):
        return L.qmx_kv_maps(past, fresh, table, free, R, columns, stride, nfree, page, T, *out, None)

    for bad in (dict(R=-1), dict(columns=-1), dict(nfree=-1), dict(T=-1), dict(page=0), dict(stride=3),
                dict(R=2 ** 16, columns=2 ** 16, stride=2 ** 16)):
        assert maps(**bad) == ESHAPE, bad
    for bad in (dict(past=None), dict(fresh=None), dict(table=None), dict(free=None)):
        assert maps(**bad) == ENULL, bad
    for i in range(6):
        assert maps(out=tuple(None if j == i else FAKE for j in range(6))) == ENULL
        assert maps(out=tuple(ODD if j == i else FAKE for j in range(6))) == EALIGN
    assert maps(past=ODD) == EALIGN and maps(table=0x10002) == EALIGN

    c = ccache()
    assert L.qmx_kv4_write(c, FAKE, FAKE, 1, 1, 1, 1, FAKE, -1, None) == ESHAPE
    assert L.qmx_kv4_write(c, None, FAKE, 1, 1, 1, 1, FAKE, 1, None) == ENULL
    assert L.qmx_kv4_write(c, FAKE, FAKE, 1, 1, 1, 1, None, 1, None) == ENULL
    assert L.qmx_kv4_write(c, FAKE, ODD, 1, 1, 1, 1, FAKE, 1, None) == EALIGN
    assert L.qmx_kv4_write(c, None, None, 1, 1, 1, 1, None, 0, None) == OK
    assert L.qmx_kv4_write(None, FAKE, FAKE, 1, 1, 1, 1, FAKE, 1, None) == ENULL
    assert L.qmx_kv4_read(c, FAKE, None, FAKE, 1, None) == ENULL
    assert L.qmx_kv4_read(c, FAKE, 0x10008, FAKE, 1, None) == EALIGN
    assert L.qmx_kv4_read(c, FAKE, FAKE, FAKE, 2 ** 31 - 1, None) == ESHAPE
    assert L.qmx_kv4_read(c, None, None, None, 0, None) == OK


def test_binding_refuses_host_tensors():
    codes, sb = torch.zeros(2, 2, 256, dtype=torch.int32), torch.zeros(2, 2, 16, 2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        qmx.Kv4Cache(codes, sb, codes, sb)
    with pytest.raises(ValueError, match="dtype"):
        qmx.Kv4Cache(codes, sb.float(), codes, sb.float())
    with pytest.raises(ValueError, match="words"):
        qmx.Kv4Cache(codes.float(), sb, codes, sb)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        qmx.kv_maps(i, i, torch.zeros(2, 2, dtype=torch.int32), i, page_size=16, tokens=2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_is_a_permutation(D):
    """Every nibble of a block belongs to one (token, element)."""
    for place in (ref.key_place, ref.value_place):
        got = {place(D, t, d) for t in range(16) for d in range(D)}
        assert got == {(w, 4 * b) for w in range(2 * D) for b in range(8)}


def test_layout_of_the_header():
    """The header's two formulas, written out for a few places."""
    assert ref.key_place(128, 5, 0) == (5 * 4, 0) and ref.key_place(128, 5, 1) == (5 * 4, 16)
    assert ref.key_place(128, 5, 8) == ((16 + 5) * 4, 0) and ref.key_place(128, 5, 32 + 3) == (5 * 4 + 1, 20)
    assert ref.value_place(128, 0, 0) == (0, 0) and ref.value_place(128, 1, 0) == (0, 16)
    assert ref.value_place(128, 0, 16) == (0, 4) and ref.value_place(128, 2, 64) == (3, 0)
    assert ref.value_place(128, 4, 1) == ((16 + 1) * 4, 0)


# ---------------------------------------------------------------- on the GPU
gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def on_gpu(test):
    for m in gpu:
        test = m(test)
    return test


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def device_cache(c):
    return qmx.Kv4Cache(*(x.to(DEV) for x in c.packed()))


@on_gpu
@pytest.mark.parametrize("R,columns,page,T,nfree,seed", [
    (1, 1, 16, 0, 0, 0), (1, 4, 16, 5, 4, 1), (3, 8, 32, 40, 9, 2), (7, 3, 16, 100, 2, 3), (64, 9, 16, 700, 300, 4),
    (1024, 6, 64, 5000, 2000, 5), (1025, 5, 32, 9001, 3000, 6), (2500, 7, 48, 40001, 9000, 7), (5, 4, 1, 12, 9, 8),
    (0, 3, 16, 6, 2, 9), (40, 12, 1000, 3000, 50, 10)])
def test_maps(R, columns, page, T, nfree, seed):
    """Lengths of zero, more tokens than room, more pages than there are, tables too narrow, holes."""
    say("maps", R, columns, page, T, nfree)
    rng = np.random.default_rng(seed)
    past = rng.integers(-1, columns * page + 3, R).tolist()
    new = rng.integers(-2, max(2, 2 * T // max(R, 1)) + 1, R).tolist()
    wide = rng.integers(0, 5000, (R, columns + 3)).astype(np.int32)
    wide[rng.random(wide.shape) < 0.05] = -1
    free = rng.permutation(6000)[:nfree].astype(np.int32)
    want_table = wide.copy()
    want = ref.maps(past, new, want_table[:, :columns], free, page, T)
    dev_wide = torch.from_numpy(wide).to(DEV)
    got = qmx.kv_maps(ints(past), ints(new), dev_wide[:, :columns], ints(free.tolist()), page_size=page, tokens=T)
    for name, g, w in zip(got._fields, got, want):
        assert g.tolist() == list(map(int, w)), name
    assert np.array_equal(dev_wide.cpu().numpy(), want_table)
    again = qmx.kv_maps(ints(past), ints(new), torch.from_numpy(wide).to(DEV)[:, :columns], ints(free.tolist()),
                        page_size=page, out=qmx.KvMaps.empty(R, T, DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def awkward(rng, shape, dtype):
    """Rows of noise, and rows with ties, one value, tiny and huge values, and wide spans."""
    x = rng.normal(0, 1, shape)
    rows = x.reshape(-1, shape[-1])
    for i in range(0, len(rows), 8):
        rows[i] = rng.integers(0, 31, shape[-1]) / 2                          # middles between codes
        if i + 5 < len(rows):
            rows[i + 1] = 0.375
            rows[i + 2] *= 2.0 ** -14                                         # subnormal in float16
            rows[i + 3] = np.where(rng.random(shape[-1]) < 0.5, -1, rng.normal(0, 2.0 ** -13, shape[-1]))
            rows[i + 4] *= 8000.0
            rows[i + 5] = rng.integers(0, 2, shape[-1]) * 2.0 ** -24
    return torch.from_numpy(x).to(dtype)


@on_gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64),
                                     (256, 128)])
@pytest.mark.parametrize("tokens,page,fused", [(1, 16, False), (37, 32, True), (150, 64, False), (95, 1024, True)])
def test_write_and_read(dtype, D, group, tokens, page, fused):
    """Codes, scales and biases bit for bit; other slots stay; reads give c s + b rounded."""
    say("write", dtype, D, group, tokens, page, fused)
    rng = np.random.default_rng(D + group + tokens)
    H = 3
    pages = 2 + -(-tokens // page)
    c = ref.Cache(pages, H, D, page, group, dtype, rng)
    cache = device_cache(c)
    T = ref.TYPES[dtype]
    k, v = awkward(rng, (tokens, H, D), T), awkward(rng, (tokens, H, D), T)
    slots = rng.permutation(pages * page)[:tokens]
    if tokens == 150:
        slots = np.arange(7, 157)                       # neighbours, from inside a block on
    slots = slots.astype(np.int32)
    drop = rng.random(tokens) < (0.15 if tokens > 1 else 0)
    slots[drop] = rng.choice([-1, -5, pages * page, 2 ** 31 - 1], int(drop.sum()))
    kd, vd = k.to(DEV), v.to(DEV)
    if fused:                                           # rows of a wider product, not 16-byte aligned
        wide = torch.zeros(tokens, 2 * H * D + 13, dtype=T, device=DEV)
        wide[:, 3:3 + H * D], wide[:, 5 + H * D:5 + 2 * H * D] = kd.flatten(1), vd.flatten(1)
        kd = wide[:, 3:3 + H * D].unflatten(1, (H, D))
        vd = wide[:, 5 + H * D:5 + 2 * H * D].unflatten(1, (H, D))
    qmx.kv4_write(cache, kd, vd, ints(slots.tolist()))
    keep = ~drop
    for which, x in ((0, k), (1, v)):
        code, s, b = ref.quantise(x, group, T)
        P, at = slots[keep] // page, slots[keep] % page
        c.codes[which][P, :, at], c.s[which][P, :, at], c.b[which][P, :, at] = code[keep], s[keep], b[keep]
    want = c.packed()
    for name, g, w in zip(("k_codes", "k_sb", "v_codes", "v_sb"),
                          (cache.k_codes, cache.k_sb, cache.v_codes, cache.v_sb), want):
        assert torch.equal(g.cpu(), w), name
    got = qmx.kv4_read(cache, ints(slots.tolist()))
    for which, g in enumerate(got):
        exact = np.zeros((tokens, H, D))
        for t in np.flatnonzero(keep):
            for h in range(H):
                exact[t, h] = c.values(which, slots[t] // page, h)[slots[t] % page]
        off = np.abs(g.double().cpu().numpy() - exact)
        # c s is exact in float32, its sum with b rounded there and then to the type (down to half a subnormal step)
        size = (ref.HALF[dtype] + 2 * ref.U32) * np.abs(exact) + (2.0 ** -25 if dtype == "f16" else 0)
        cancel = ref.U32 * (15 * np.abs(exact).max(-1, keepdims=True))
        assert (off <= size + cancel).all(), off.max()


@on_gpu
def test_write_keeps_nan_and_infinity_to_their_group():
    say("write nan")
    x = torch.randn(4, 1, 128, dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 70], x[2, 0, 5], x[3, 0, 6] = math.nan, math.inf, -math.inf, -math.nan
    cache = qmx.Kv4Cache.zeros(1, 1, 128, page_size=16, group_size=64, device=DEV)
    slots = ints([0, 1, 2, 3])
    qmx.kv4_write(cache, x.to(DEV), x.to(DEV), slots)
    for got in qmx.kv4_read(cache, slots):
        bad = ~torch.isfinite(got.float().cpu())[:, 0]
        assert bad[0, :64].all() and not bad[0, 64:].any()
        assert bad[1, 64:].all() and not bad[1, :64].any()
        assert bad[2, :64].all() and not bad[2, 64:].any()
        assert bad[3, :64].all() and not bad[3, 64:].any()


def attention_case(dtype, D, group, page, each, H, lens, window=0, pad=0, holes=(), spoil=False, strided=False,
                   seed=0, scale=None, table_extra=0, uneven=False):
    """lens: (past, new) of each request.  holes: (request, column) entries without a page."""
    say("attention", dtype, D, group, page, each, H, lens, window, pad, holes, spoil, strided)
    rng = np.random.default_rng(seed)
    need = [-(-(p + n) // page) for p, n in lens]
    pages = sum(need) + 2
    c = ref.Cache(pages, H, D, page, group, dtype, rng)
    if uneven:   # keys far above and queries far below 1, values that differ from token to token
        for x in (c.s[0], c.b[0]):
            x *= 2.0 ** 40
        factor = 2.0 ** rng.integers(-6, 7, (pages, H, page, 1))
        c.s[1] *= factor
        c.b[1] *= factor
    R, columns = len(lens), max(1, max(need)) + table_extra
    order = rng.permutation(pages)[:sum(need)]
    table = np.full((R, columns), -1, dtype=np.int32)
    first = 0
    for r, n in enumerate(need):
        table[r, :n] = order[first:first + n]
        first += n
    for i, (r, col) in enumerate(holes):
        table[r, col] = (-1, pages, 2 ** 30)[i % 3]
    kv = [p + n for p, n in lens]
    offsets = [0]
    for _, n in lens:
        offsets.append(offsets[-1] + n)
    T, heads = offsets[-1] + pad, each * H
    q = torch.from_numpy(rng.normal(0, 1.3, (T, heads, D)) * (2.0 ** -40 if uneven else 1)).to(ref.TYPES[dtype])
    packed = c.packed()
    if spoil:   # whatever no request sees holds NaN
        seen = np.zeros((pages, page), dtype=bool)
        for r, n in enumerate(kv):
            for at in range(n):
                if 0 <= table[r, at // page] < pages:
                    seen[table[r, at // page], at % page] = True
        for i in (1, 3):
            packed[i].transpose(1, 2)[torch.from_numpy(~seen)] = math.nan
    cache = qmx.Kv4Cache(*(x.to(DEV) for x in packed))
    qd = q.to(DEV)
    if strided:
        wide = torch.zeros(T, heads * D + 24, dtype=q.dtype, device=DEV)
        wide[:, 5:5 + heads * D] = qd.flatten(1)
        qd = wide[:, 5:5 + heads * D].unflatten(1, (heads, D))
    kw = dict(max_query_len=max([n for _, n in lens] + [0]), max_kv_len=max(kv + [0]), window=window, scale=scale)
    args = (cache, qd, torch.from_numpy(table).to(DEV), ints(kv), ints(offsets))
    out, lse = qmx.kv4_attention(*args, return_lse=True, **kw)
    prompt = kw["max_query_len"] * each > 64   # the kernel of many rows
    o, l, tol, ltol = ref.attention(c, q, table, kv, offsets, window, scale, prompt)
    out_, lse_ = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out_).all()
    over = np.abs(out_ - o) - tol
    assert (over <= 0).all(), (over.max(), tol.flat[over.argmax()], np.unravel_index(over.argmax(), over.shape))
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(lse_), empty)
    assert (np.abs(lse_[~empty] - l[~empty]) <= ltol[~empty]).all()
    assert torch.equal(out, qmx.kv4_attention(*args, **kw)), "rerun not bit-identical"
    return args, kw, out


FORMATS = [(t, d, g) for t in ("bf16", "f16") for d, g in ((64, 32), (64, 64), (128, 32), (128, 64), (128, 128),
                                                           (256, 32), (256, 64), (256, 128))]


@on_gpu
@pytest.mark.parametrize("dtype,D,group", FORMATS)
def test_attention_single_tokens(dtype, D, group):
    """Lengths 1 and up, an empty request, tokens of no request."""
    attention_case(dtype, D, group, 16, 4, 2, [(0, 1), (14, 1), (15, 1), (16, 1), (30, 1), (31, 1), (0, 0), (99, 1)],
                   pad=3, seed=1)


@on_gpu
@pytest.mark.parametrize("dtype,D,group", FORMATS)
def test_attention_prompts(dtype, D, group):
    """Rows of several waves and tiles; prompts beside chunks behind a cached prefix."""
    attention_case(dtype, D, group, 32, 2, 1, [(0, 70), (45, 33), (3, 0), (200, 1)], pad=1, seed=2, spoil=True)


@on_gpu
@pytest.mark.parametrize("dtype,D,group", FORMATS)
def test_attention_prompts_of_many_tiles(dtype, D, group):
    """Several work-groups' rows, keys shared among work-groups, an odd number of query heads a key head."""
    attention_case(dtype, D, group, 64, 5, 1, [(1200, 61), (0, 0), (7, 110), (30, 1)], pad=5, seed=12, spoil=True)


@on_gpu
@pytest.mark.parametrize("dtype,D,group", FORMATS)
def test_attention_prompts_cut(dtype, D, group):
    """Prompts behind a long prefix, whose units are cut and joined."""
    attention_case(dtype, D, group, 64, 2, 2, [(1777, 61), (0, 0), (7, 90), (700, 1)], pad=3, seed=13, spoil=True)


@on_gpu
@pytest.mark.parametrize("dtype,D,group", FORMATS)
def test_attention_split_keys(dtype, D, group):
    """Keys cut over work-groups, requests that end in the first part."""
    attention_case(dtype, D, group, 64, 3, 1, [(2500, 1), (10, 2), (0, 0), (1111, 4)], pad=2, seed=3, spoil=True)


@on_gpu
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100])
@pytest.mark.parametrize("lens", [[(150, 1), (5, 1)], [(90, 9), (0, 3)], [(40, 65), (0, 90)], [(1700, 2)]])
def test_attention_window(window, lens):
    attention_case("bf16", 64, 32, 16, 2, 2, lens, window=window, seed=4, spoil=True)


@on_gpu
@pytest.mark.parametrize("each,H", [(1, 1), (1, 5), (5, 2), (7, 1), (8, 3), (16, 1), (17, 1), (40, 1)])
@pytest.mark.parametrize("new", [1, 3])
def test_attention_shared_heads(each, H, new):
    attention_case("f16", 128, 64, 128, each, H, [(60, new), (131, new)], seed=5)


@on_gpu
@pytest.mark.parametrize("lens", [[(70, 1), (40, 1)], [(60, 40), (35, 50)], [(1700, 1), (600, 2)]])
def test_attention_missing_pages(lens):
    """Entries without a page inside a request; a request whose every page is missing sees nothing."""
    holes = [(0, 0), (0, 2), (1, 1)]
    attention_case("bf16", 128, 64, 16, 4, 2, lens + [(20, 2)], holes=holes + [(2, 0), (2, 1)], spoil=True, seed=6)


@on_gpu
@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
def test_attention_page_sizes(page):
    attention_case("bf16", 64, 64, page, 2, 1, [(page - 1, 1), (page, 1), (2 * page - 20, 30)], seed=7, table_extra=2)


@on_gpu
@pytest.mark.parametrize("lens", [[(77, 1)], [(10, 80)], [(1500, 1)]])
def test_attention_strided_queries_and_scale(lens):
    attention_case("f16", 64, 32, 16, 3, 2, lens, strided=True, scale=0.3, seed=8)
    attention_case("bf16", 128, 128, 16, 3, 2, lens, scale=0.05, seed=9)


@on_gpu
def test_attention_spread_scores():
    """Scores far apart: the running maximum rises often, and most probabilities vanish."""
    attention_case("bf16", 128, 32, 16, 4, 1, [(700, 1)], scale=3.0, seed=10)
    attention_case("f16", 128, 64, 16, 4, 1, [(300, 30)], scale=3.0, seed=11)


@on_gpu
@pytest.mark.parametrize("lens", [[(90, 1), (33, 3)], [(50, 75), (0, 40)], [(2000, 1), (1700, 2)], [(1900, 70)]])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
def test_attention_uneven_magnitudes(lens, D, group):
    attention_case("bf16", D, group, 32, 2, 1, lens, seed=14, spoil=True, uneven=True)


@on_gpu
def test_attention_nan_stays_with_its_rows():
    say("attention nan")
    rng = np.random.default_rng(12)
    c = ref.Cache(6, 1, 64, 16, 32, "bf16", rng)
    packed = c.packed()
    packed[3][2, 0, 4, 1, 0] = math.nan        # one value group of request 0's token 20
    cache = qmx.Kv4Cache(*(x.to(DEV) for x in packed))
    table = ints([[1, 2, 3], [4, 5, -1]])
    q = torch.randn(25, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = qmx.kv4_attention(cache, q, table, ints([30, 20]), ints([0, 20, 25]), max_query_len=20, max_kv_len=30)
    bad = torch.isnan(out.float()).cpu()
    assert bad[10:20, :, 32:].all()            # positions 20..29
    assert not bad[:10].any() and not bad[20:].any() and not bad[:, :, :32].any()
    # the same through the kernel of many rows, and an infinite bias
    packed[3][2, 0, 4, 1] = torch.tensor([0.0, math.inf])
    cache = qmx.Kv4Cache(*(x.to(DEV) for x in packed))
    q = torch.randn(25, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = qmx.kv4_attention(cache, q, table, ints([30, 20]), ints([0, 20, 25]), max_query_len=20, max_kv_len=30)
    bad = torch.isinf(out.float()).cpu()
    assert bad[10:20, :, 32:].all()
    assert torch.isfinite(out[:10].float()).all() and torch.isfinite(out[20:].float()).all()
    assert torch.isfinite(out[:, :, :32].float()).all()


@on_gpu
def test_step_under_a_graph():
    """Maps, write and attention captured once and replayed over new lengths, with eager work between."""
    say("graph")
    torch.manual_seed(0)
    H, each, D, page, R, T, columns = 2, 3, 128, 16, 5, 8, 120
    cache = qmx.Kv4Cache.zeros(200, H, D, page_size=page, group_size=64, device=DEV)
    other = qmx.Kv4Cache.zeros(200, H, D, page_size=page, group_size=64, device=DEV)
    tables = [torch.full((R, columns), -1, dtype=torch.int32, device=DEV) for _ in range(2)]
    past, new = ints([0] * R), ints([1] * R)
    free = ints(list(range(200)))
    qkv = torch.randn(T, (each + 2) * H, D, dtype=torch.bfloat16, device=DEV)
    maps = qmx.KvMaps.empty(R, T, DEV)

    def step(cache, table, maps):
        m = qmx.kv_maps(past, new, table, free, page_size=page, out=maps)
        qmx.kv4_write(cache, qkv[:, each * H:each * H + H], qkv[:, each * H + H:], m.slots)
        return qmx.kv4_attention(cache, qkv[:, :each * H], table, m.kv_lens, m.query_offsets, max_query_len=4,
                                 max_kv_len=columns * page, return_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, tables[0], maps)
    torch.cuda.current_stream().wait_stream(side)
    cache.k_sb.zero_(), cache.v_sb.zero_(), cache.k_codes.zero_(), cache.v_codes.zero_()
    tables[0].fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(cache, tables[0], maps)
    used = 0
    rng = np.random.default_rng(0)
    for i in range(6):
        count = torch.from_numpy(rng.multinomial(6, [0.2] * R).clip(0, 4).astype(np.int32)).to(DEV)
        new.copy_(count)
        free.copy_(torch.roll(torch.arange(200, dtype=torch.int32, device=DEV), -used))
        qkv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = step(other, tables[1], qmx.KvMaps.empty(R, T, DEV))
        assert torch.equal(tables[0], tables[1])
        for a, b in zip(captured, want):
            assert torch.equal(a, b)
        assert torch.equal(cache.k_codes, other.k_codes) and torch.equal(cache.v_sb, other.v_sb)
        used += int(maps.counts[1])
        past.add_(count)


@on_gpu
def test_other_stream():
    """The calls go to torch's current stream, behind what is queued there."""
    say("stream")
    cache = qmx.Kv4Cache.zeros(4, 1, 64, page_size=16, group_size=32, dtype=torch.float16, device=DEV)
    k = torch.randn(40, 1, 64, dtype=torch.float16, device=DEV)
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        x = (big @ big)[:40, :64].mul(0).reshape(40, 1, 64).half() + k
        qmx.kv4_write(cache, x, x, slots)
        got = qmx.kv4_read(cache, slots)[0]
    torch.cuda.current_stream().wait_stream(side)
    again = qmx.Kv4Cache.zeros(4, 1, 64, page_size=16, group_size=32, dtype=torch.float16, device=DEV)
    qmx.kv4_write(again, k, k, slots)
    assert torch.equal(got, qmx.kv4_read(again, slots)[0])


@on_gpu
@pytest.mark.parametrize("new", [1, 90])
def test_cache_without_pages(new):
    """Nothing is there: attention and reads give zeros, writes do nothing."""
    say("no pages", new)
    cache = qmx.Kv4Cache.zeros(0, 2, 128, page_size=16, group_size=64, device=DEV)
    q = torch.randn(new, 4, 128, dtype=torch.bfloat16, device=DEV)
    out, lse = qmx.kv4_attention(cache, q, ints([[0, 1, 2, 3, 4, 5]]), ints([90]), ints([0, new]), max_query_len=new,
                                 max_kv_len=2000, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    slots = ints(list(range(new)))
    qmx.kv4_write(cache, q[:, :2], q[:, 2:], slots)
    assert not any(t.any() for t in qmx.kv4_read(cache, slots))


@on_gpu
@pytest.mark.parametrize("new,max_kv", [(1, 50), (70, 90), (1, 5000)])
def test_bounds_of_the_host_hold(new, max_kv):
    """Keys past max_kv_len, or past the table's columns, are not seen whatever kv_lens says; tokens of no request,
    and all of them where there are no requests, get zeros."""
    say("bounds", new, max_kv)
    rng = np.random.default_rng(20)
    c = ref.Cache(8, 1, 64, 16, 32, "f16", rng)
    cache = device_cache(c)
    table = np.arange(6, dtype=np.int32)[None]
    q = torch.from_numpy(rng.normal(0, 1, (new + 2, 2, 64))).half()
    seen = min(max_kv, 96)
    out = qmx.kv4_attention(cache, q.to(DEV), ints(table.tolist()), ints([300]), ints([0, new]), max_query_len=new,
                            max_kv_len=max_kv)
    # every query is at position 300 - new or later, so it sees all that is there
    for t in range(new):
        want, _, tol, _ = ref.attention(c, q[t:t + 1], table, [seen], [0, 1], prompt=2 * new > 64)
        assert (np.abs(out[t].double().cpu().numpy() - want[0]) <= tol[0]).all()
    assert not out[new:].any()
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = qmx.kv4_attention(cache, q.to(DEV), torch.zeros(0, 6, dtype=torch.int32, device=DEV), none, ints([0]),
                            max_query_len=new, max_kv_len=max_kv)
    assert not out.any()


@on_gpu
def test_example_of_a_serving_loop():
    """Prompts, then graph replays of one token each, against float64 on what the cache reads back as.  Reading back
    rounds keys and values to bfloat16 (half a step 2^-8 each, scores of at most a few units move p by that much again),
    the kernel's probabilities and outputs are rounded alike: 8 such roundings of the row's largest output bound them."""
    say("example")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import kv4_decode
    errors = kv4_decode.main(steps=20)
    assert len(errors) == 21 and max(errors) <= 8 * 2.0 ** -8, errors


@on_gpu
def test_binding_refusals():
    cache = qmx.Kv4Cache.zeros(2, 2, 64, page_size=16, group_size=32, device=DEV)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    s = ints([0, 1, 2])
    for k, v, slots in ((x.half(), x, s), (x[:2], x, s), (x, x[:, :1], s), (x, x, s.long()), (x, x, s[:2]),
                        (x.transpose(1, 2).contiguous().transpose(1, 2), x, s), (x.cpu(), x, s)):
        with pytest.raises(ValueError):
            qmx.kv4_write(cache, k, v, slots)
    with pytest.raises(ValueError):
        qmx.kv4_read(cache, s.float())
    with pytest.raises(ValueError):
        qmx.kv4_read(cache, s, out=(x, x.half()))
    table, lens, offsets = ints([[0], [1]]), ints([2, 1]), ints([0, 2, 3])
    kw = dict(max_query_len=2, max_kv_len=2)
    for args in ((x[:, :1], table, lens, offsets), (x.half(), table, lens, offsets), (x, table[:1], lens, offsets),
                 (x, table, lens, offsets[:2]), (x, table.long(), lens, offsets), (x, table, lens.cpu(), offsets)):
        with pytest.raises(ValueError):
            qmx.kv4_attention(cache, *args, **kw)
    with pytest.raises(ValueError):
        qmx.kv4_attention(cache, x, table, lens, offsets, out=x.half(), **kw)
    with pytest.raises(qmx.QmxError):
        qmx.kv4_attention(cache, x, table, lens, offsets, window=-1, **kw)
    with pytest.raises(ValueError):
        qmx.kv_maps(lens, lens[:1], table, lens, page_size=16, tokens=3)
    with pytest.raises(ValueError):
        qmx.kv_maps(lens, lens, table, lens, page_size=16)
    with pytest.raises(ValueError):
        qmx.kv_maps(lens, lens, table, lens, page_size=16, out=qmx.KvMaps.empty(3, 3, DEV))
    with pytest.raises(qmx.QmxError):
        qmx.kv_maps(lens, lens, table, lens, page_size=0, tokens=3)
    with pytest.raises(ValueError):
        qmx.Kv4Cache.zeros(2, 2, 96, page_size=16, group_size=32, device=DEV)
    with pytest.raises(ValueError):
        qmx.Kv4Cache.zeros(2, 2, 64, page_size=48, group_size=32, device=DEV)
