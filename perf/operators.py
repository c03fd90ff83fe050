"""The operators of a paged key/value cache held in 4 bits, as cases to time and compare.

Four operators, as one layer's step of a serving program uses them:

* maps:   block tables and slot maps from the requests' lengths;
* write:  new keys and values quantised into the cache (the case reads the same slots back, as values);
* read:   cached keys and values gathered by slot, as values;
* attend: attention of the new queries over the cache.

The cache.  A token's keys (and values) of one head are cut into groups of `group` elements; a group has a
scale s and a bias b in the cache's type and a 4-bit code c per element, and stands for c * s + b.  With
lo and hi the group's least and greatest element: b = lo, s = (hi - lo) / 15 rounded to the type, and
c = (x - b) / s rounded to nearest even and kept within 0..15 (0 where s is 0).  Tokens live in pages of
`page` tokens; a page holds blocks of 16 tokens per head, each block's codes as 2 * D 32-bit words:

* keys:   word (h * 16 + token) * (D / 32) + j holds elements 32j + 8h + e, e = 0..7, element e at
          bit 4 * (e / 2) + 16 * (e % 2)                                           (h = 0..3);
* values: 16-bit half ((h * 16 + n) * (D / 64) + a) * 4 + i holds token 4h + i's elements 16 * (4a + f) + n,
          f = 0..3, at bit 4f                                                      (n = 0..15).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"


# ---------------------------------------------------------------------------------------------- cases
def _case(name, op, requests, past, new, ragged, heads=32, kv_heads=8, dim=128, group=64, page=16, type="bf16",
          window=0, lse=False, pad=0):
    return {"name": name, "op": op, "requests": requests, "past": past, "new": new, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "group": group, "page": page, "type": type, "window": window,
            "lse": lse, "pad": pad}


def listed():
    return [
        # one decoded token for each of a small batch, under a captured graph that has room for 32
        _case("maps decode", "maps", 24, 4000, 1, 3, pad=8),
        # a scheduler's step over many requests: prompts and chunks of prompts of every length
        _case("maps prompts", "maps", 3000, 20000, 200, 5, page=32, pad=1111),
        # the tokens of one decode step
        _case("write decode", "write", 40, 5000, 1, 7, heads=40),
        # a long prompt, with the finer groups
        _case("write prompt", "write", 4, 1000, 14000, 9, group=32, page=64, type="f16"),
        # a cached prefix taken up by another program
        _case("read prefix", "read", 1, 0, 777, 0, page=32),
        # many prefixes at once, to be copied elsewhere
        _case("read many", "read", 50, 0, 6000, 11, dim=64, type="f16", page=16),
        # one user, one token: latency
        _case("attend one", "attend", 1, 640, 1, 0),
        # a full decode batch of every length, five query heads to a key head
        _case("attend batch", "attend", 48, 8000, 1, 13, heads=40, lse=True),
        # two users deep into very long documents
        _case("attend long", "attend", 2, 131000, 1, 17, heads=64, group=128, page=64, type="f16"),
        # drafted tokens checked at once, a key head for each query head, sliding window, an idle request
        _case("attend drafts", "attend", 16, 4000, 5, 19, heads=16, kv_heads=16, dim=64, group=32, page=32,
              type="f16", window=1500, lse=True),
        # a whole prompt
        _case("attend prompt", "attend", 1, 0, 8192, 0, page=64),
        # chunks of several prompts beside each other, wide heads
        _case("attend chunks", "attend", 12, 4000, 512, 23, heads=16, kv_heads=4, dim=256, type="f16", pad=100),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["maps", "write", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    kind = {"ragged": rng.randrange(1, 10 ** 6) if rng.random() < 0.8 else 0, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "group": group, "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "f16"]),
            "pad": rng.choice([0, 0, rng.randrange(1, 300)])}
    if op == "maps":
        requests = _spread(rng, 1, 3000)
        case = _case("", op, requests, _spread(rng, 1, 20000), _spread(rng, 1, max(1, 600000 // requests)), 0)
        case["new"] = min(case["new"], 20000)
    elif op in ("write", "read"):
        tokens = _spread(rng, 1, 48000000 // (kv_heads * dim))
        requests = _spread(rng, 1, min(64, tokens))
        case = _case("", op, requests, 0 if op == "read" else _spread(rng, 1, 4000), max(1, tokens // requests), 0)
    else:
        new = rng.choice([1, 1, rng.randrange(2, 9), _spread(rng, 9, 2000)])
        requests = _spread(rng, 1, 64 if new < 9 else 8)
        keys = min(131072, 250000000 // (requests * kv_heads * dim), 120000000000 // (requests * heads * new * dim))
        past = max(0, _spread(rng, 1, max(1, keys)) - new)
        case = _case("", op, requests, past, new, 0, window=rng.choice([0, 0, 0, _spread(rng, 1, 4096)]),
                     lse=rng.random() < 0.5)
    case.update(kind)
    del case["name"]
    return case


def _lengths(case):
    """(past, new) of each request.  Ragged: the first has the full lengths, and of four or more the last idles."""
    rng = random.Random(case["ragged"])
    past, new = [], []
    for r in range(case["requests"]):
        full = r == 0 or not case["ragged"]
        past.append(case["past"] if full else int(math.exp(rng.uniform(0, math.log(case["past"] + 1)))) - 1)
        new.append(case["new"] if full else rng.randint(1, case["new"]))
    if case["ragged"] and case["requests"] >= 4:
        past[-1] = new[-1] = 0
    return past, new


def _pairs(case):
    """Cached tokens that an attention has to read, and its (query, key) pairs, for one head."""
    tokens = pairs = 0
    for p, n in zip(*_lengths(case)):
        w = case["window"] or p + n
        if n:
            tokens += p + n - max(0, p + 1 - w)
            pairs += sum(min(p + i + 1, w) for i in range(n))
    return tokens, pairs


def work(case):
    past, new = _lengths(case)
    n, page = sum(new), case["page"]
    cells = case["kv_heads"] * case["dim"]
    codes = 2 * case["kv_heads"] * (case["dim"] // 2 + 4 * case["dim"] // case["group"])  # keys and values of a token
    if case["op"] == "maps":
        pages = sum(-(-(p + m) // page) - -(-p // page) for p, m in zip(past, new))
        return {"bytes": 16 * case["requests"] + 12 * (n + case["pad"]) + 8 * pages, "flops": n + case["pad"]}
    if case["op"] == "write":
        return {"bytes": 4 * n + n * (4 * cells + codes) + n * (codes + 4 * cells), "flops": 8 * n * cells}
    if case["op"] == "read":
        return {"bytes": 4 * n + n * (codes + 4 * cells), "flops": 4 * n * cells}
    tokens, pairs = _pairs(case)
    return {"bytes": tokens * codes + 4 * n * case["heads"] * case["dim"] + 4 * (tokens // page),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _quantise(x, group, dtype):
    """Codes [..., D] (int32), scales and biases [..., D / group] of x [..., D]: in 64 bits, for what lies next
    to a border between two codes."""
    g = x.double().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    s, b = ((hi - lo) / 15).to(dtype), lo.to(dtype)
    c = torch.round((g - b.double()[..., None]) / s.double()[..., None]).clamp(0, 15)
    c = torch.where(s[..., None] == 0, torch.zeros_like(c), c)
    return c.int().flatten(-2), s, b


_ELEMENT_BIT = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]


def _pack_keys(c):
    """[..., 16 tokens, D] codes as [..., 2 * D] words."""
    D = c.shape[-1]
    c = c.unflatten(-1, (D // 32, 4, 8)) << _ints(_ELEMENT_BIT)
    return c.sum(-1, dtype=torch.int32).movedim(-1, -3).flatten(-3)


def _pack_values(c):
    D = c.shape[-1]
    c = c.unflatten(-1, (D // 64, 4, 16)).unflatten(-4, (4, 2, 2))  # h, i / 2, i % 2, a, f, n
    c = c << (16 * _ints([0, 1])[:, None, None, None] + 4 * _ints([0, 1, 2, 3])[:, None])
    c = c.sum((-4, -2), dtype=torch.int32)  # h, i / 2, a, n
    return c.movedim(-1, -3).transpose(-1, -2).flatten(-4)


def _unpack_keys(w, D):
    """[..., 2 * D] words as [..., 16 tokens, D] codes."""
    w = w.unflatten(-1, (4, 16, D // 32)).movedim(-3, -1)  # token, j, h
    return ((w[..., None] >> _ints(_ELEMENT_BIT)) & 15).flatten(-3)


def _unpack_values(w, D):
    w = w.unflatten(-1, (4, 16, D // 64, 2))[..., None, None]  # h, n, a, i / 2
    c = (w >> (16 * _ints([0, 1])[:, None] + 4 * _ints([0, 1, 2, 3]))) & 15  # h, n, a, i / 2, i % 2, f
    return c.permute(*range(c.dim() - 6), -6, -3, -2, -4, -1, -5).flatten(-3).flatten(-4, -2)


def _noise(case, shape, gen, outliers):
    x = torch.randn(shape, generator=gen, device=DEVICE)
    if outliers:  # a few channels of the keys are several times larger than the others
        x = x * (1 + 3 * (torch.rand(shape[-1], generator=gen, device=DEVICE) < 0.06))
    return x.to(TYPES[case["type"]])


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    past, new = _lengths(case)
    page, D, H, R = case["page"], case["dim"], case["kv_heads"], case["requests"]
    dtype = TYPES[case["type"]]
    kv = [p + n for p, n in zip(past, new)]
    tokens = sum(new) + case["pad"]
    columns = max(1, max(-(-x // page) for x in kv))
    st = {"op": case["op"], "past": _ints(past), "new": _ints(new), "kv_lens": _ints(kv), "tokens": tokens,
          "page": page, "group": case["group"], "dim": D, "max_new": max(new), "max_kv": max(kv),
          "window": case["window"], "lse": case["lse"]}
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    st["offsets"] = _ints(offsets)
    need = [-(-x // page) for x in kv]
    held = [-(-x // page) for x in past] if case["op"] == "maps" else need
    num_pages = sum(need) + 3
    order = torch.randperm(num_pages, generator=gen, device=DEVICE).int()
    table = torch.full((R, columns), -1, dtype=torch.int32, device=DEVICE)
    table[torch.arange(columns, device=DEVICE) < _ints(held)[:, None]] = order[:sum(held)]
    st["table"] = table
    if case["op"] == "maps":
        st["free"] = order[sum(held):].contiguous()
        for name, size in (("query_offsets", R + 1), ("kv_lens_out", R), ("slots", tokens), ("positions", tokens),
                           ("request_ids", tokens), ("counts", 2)):
            st[name] = torch.zeros(size, dtype=torch.int32, device=DEVICE)
        if own:
            import matmul_affine_qmv_amd as qmx
            st["maps"] = qmx.KvMaps(st["query_offsets"], st["kv_lens_out"], st["slots"], st["positions"],
                                    st["request_ids"], st["counts"])
        return st
    # the cache, with what an earlier program left in the pages that nobody holds
    cells = (num_pages, H, page)
    sb = []
    for name, pack in (("k", _pack_keys), ("v", _pack_values)):
        c, s, b = _quantise(_noise(case, (*cells, D), gen, name == "k"), case["group"], dtype)
        st[name + "_codes"] = pack(c.unflatten(-2, (-1, 16))).flatten(-2).contiguous()
        st[name + "_sb"] = torch.stack((s, b), -1).contiguous()
        del c, s, b
    if own:
        import matmul_affine_qmv_amd as qmx
        st["cache"] = qmx.Kv4Cache(st["k_codes"], st["k_sb"], st["v_codes"], st["v_sb"])
    if case["op"] == "attend":
        st["q"] = _noise(case, (tokens, case["heads"], D), gen, False)
        st["q"].mul_(1.5)
        return st
    row = torch.repeat_interleave(torch.arange(R, device=DEVICE), _ints(new).long())
    at = torch.arange(sum(new), device=DEVICE) - st["offsets"].long()[row] + st["past"].long()[row]
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=DEVICE)
    slots[:sum(new)] = table[row, at // page] * page + (at % page).int()
    st["slots"] = slots
    if case["op"] == "write":  # parts of the rows that a fused projection of queries, keys and values gives
        fused = _noise(case, (tokens, case["heads"] + 2 * H, D), gen, False)
        st["k"], st["v"] = fused[:, case["heads"]:case["heads"] + H], fused[:, case["heads"] + H:]
        st["k"].mul_(1 + 3 * (torch.rand(D, generator=gen, device=DEVICE) < 0.06))
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["op"]
    if own:
        import matmul_affine_qmv_amd as qmx
        if op == "maps":
            m = qmx.kv_maps(st["past"], st["new"], st["table"], st["free"], page_size=st["page"], out=st["maps"])
            return [*m, st["table"]]
        if op == "write":
            qmx.kv4_write(st["cache"], st["k"], st["v"], st["slots"])
            return qmx.kv4_read(st["cache"], st["slots"])
        if op == "read":
            return qmx.kv4_read(st["cache"], st["slots"])
        return qmx.kv4_attention(st["cache"], st["q"], st["table"], st["kv_lens"], st["offsets"],
                                 max_query_len=st["max_new"], max_kv_len=st["max_kv"], window=st["window"],
                                 return_lse=st["lse"])
    if op == "maps":
        return _maps(st)
    if op == "write":
        _write(st)
    return _attend(st) if op == "attend" else _read(st)


def _maps(st):
    past, new, page, T = st["past"].long(), st["new"].long(), st["page"], st["tokens"]
    table, columns = st["table"], st["table"].shape[1]
    ends = new.cumsum(0).clamp(max=T)
    offsets = torch.cat((ends.new_zeros(1), ends))
    kv = past + ends - offsets[:-1]
    held = ((past + page - 1) // page).clamp(max=columns)
    take = ((kv + page - 1) // page).clamp(max=columns) - held
    first = take.cumsum(0) - take
    column = torch.arange(columns, device=past.device)
    fresh = column - held[:, None]
    fresh = torch.where((fresh >= 0) & (fresh < take[:, None]), fresh + first[:, None], -1)
    pages = torch.cat((st["free"], st["free"].new_full((1,), -1)))
    table.copy_(torch.where(fresh >= 0, pages[fresh.clamp(max=len(st["free"]))], table))
    t = torch.arange(T, device=past.device)
    row = torch.searchsorted(ends, t, right=True)
    there = row < len(new)
    row = row.clamp(max=len(new) - 1)
    at = t - offsets[row] + past[row]
    got = table[row, (at // page).clamp(max=columns - 1)].long()
    slot = torch.where((got >= 0) & (at < columns * page), got * page + at % page, -1)
    out = [offsets, kv, torch.where(there, slot, -1), torch.where(there, at, -1), torch.where(there, row, -1),
           torch.stack((new.sum(), take.sum()))]
    return [x.int() for x in out] + [table]


def _write(st):
    H, page, D = st["k_sb"].shape[1], st["page"], st["dim"]
    there = (st["slots"] >= 0).nonzero()[:, 0]
    slot = st["slots"][there].long()
    P, at = slot // page, slot % page
    for name in ("k", "v"):
        c, s, b = _quantise(st[name][there], st["group"], st["k"].dtype)
        if name == "k":
            words = (c.unflatten(-1, (D // 32, 4, 8)) << _ints(_ELEMENT_BIT)).sum(-1, dtype=torch.int32)
            to = st["k_codes"].view(-1, H, page // 16, 4, 16, D // 32)
            to[P, :, at // 16, :, at % 16] = words.transpose(-1, -2)
        else:
            halves = (c.unflatten(-1, (D // 64, 4, 16)) << 4 * _ints([0, 1, 2, 3])[:, None]).sum(-2, dtype=torch.int32)
            to = st["v_codes"].view(torch.int16).view(-1, H, page // 16, 4, 16, D // 64, 4)
            to[P, :, at // 16, at % 16 // 4, :, :, at % 4] = halves.transpose(-1, -2).to(torch.int16)
        st[name + "_sb"][P, :, at] = torch.stack((s, b), -1)


def _values(codes, sb):
    """What codes [..., D] with scales and biases [..., D / group, 2] stand for, in 32 bits."""
    c = codes.float().unflatten(-1, (sb.shape[-2], -1))
    return (c * sb[..., :1].float() + sb[..., 1:].float()).flatten(-2)


def _read(st):
    H, page, D = st["k_sb"].shape[1], st["page"], st["dim"]
    slot = st["slots"].long().clamp(min=0)
    P, at = slot // page, slot % page
    words = st["k_codes"].view(-1, H, page // 16, 4, 16, D // 32)[P, :, at // 16, :, at % 16]
    keys = (words.transpose(-1, -2)[..., None] >> _ints(_ELEMENT_BIT)) & 15  # tokens, heads, j, h, e
    halves = st["v_codes"].view(torch.int16).view(-1, H, page // 16, 4, 16, D // 64, 4)
    halves = halves[P, :, at // 16, at % 16 // 4, :, :, at % 4].int()  # tokens, heads, n, a
    values = (halves.transpose(-1, -2)[..., None, :] >> 4 * _ints([0, 1, 2, 3])[:, None]) & 15
    there = (st["slots"] >= 0)[:, None, None]
    return [torch.where(there, _values(c.flatten(2), st[name + "_sb"][P, :, at]), 0).to(st["k_sb"].dtype)
            for name, c in (("k", keys), ("v", values))]


def _attend(st):
    q, page, D, n, window = st["q"], st["page"], st["dim"], st["max_new"], st["window"]
    T, heads, _ = q.shape
    pages, H = st["k_sb"].shape[:2]
    table = st["table"][:, :-(-st["max_kv"] // page)]
    R, L, each = len(table), table.shape[1] * page, heads // H
    held = table.long().clamp(0, pages - 1)
    kv = []
    for name, unpack in (("k", _unpack_keys), ("v", _unpack_values)):
        codes = unpack(st[name + "_codes"][held].unflatten(-1, (page // 16, -1)), D).flatten(-3, -2)
        kv.append(_values(codes, st[name + "_sb"][held]).transpose(1, 2).flatten(2, 3))  # requests, heads, tokens, D
        del codes
    start, lens = st["offsets"][:-1].long(), st["kv_lens"].long()
    count = st["offsets"][1:].long() - start
    i = torch.arange(n, device=q.device)
    rows = (start[:, None] + i).clamp(max=T - 1)
    x = q[rows].float().unflatten(2, (H, each)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # requests, heads, n * each, D
    s = (x @ kv[0].transpose(-1, -2)).mul_(D ** -0.5).unflatten(2, (n, each))
    key = torch.arange(L, device=q.device)
    at = (lens - count)[:, None] + i
    seen = (key <= at[..., None]) & (key < lens[:, None, None])
    if window:
        seen = seen & (key > at[..., None] - window)
    seen = (seen & ((table >= 0) & (table < pages)).repeat_interleave(page, 1)[:, None])[:, None, :, None]
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ kv[1]).unflatten(2, (n, each)) / torch.where(total > 0, total, 1)
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(st["offsets"][1:].long(), t, right=True)
    there = (r < R)[:, None]
    r = r.clamp(max=R - 1)
    i = (t - start[r]).clamp(max=n - 1)
    out = torch.where(there[..., None], o[r, :, i].flatten(1, 2), 0).to(q.dtype)
    if not st["lse"]:
        return out
    lse = (m + total.log())[..., 0]
    return out, torch.where(there, lse[r, :, i].flatten(1, 2), -math.inf)


# ---------------------------------------------------------------------------------------------- in 64 bits
def _cell(words, sb, token, d, group, keys):
    """Values of tokens (within a page) and elements d of one page and head, from the definition of the layout."""
    D = words.shape[-1] * 8 // sb.shape[-3]
    block, t = token // 16, token % 16
    if keys:
        h, j, e = d // 8 % 4, d // 32, d % 8
        word, bit = (h * 16 + t) * (D // 32) + j, 4 * (e // 2) + 16 * (e % 2)
    else:
        a, f, n = d // 64, d // 16 % 4, d % 16
        half = ((t // 4 * 16 + n) * (D // 64) + a) * 4 + t % 4
        word, bit = half // 2, 16 * (half % 2) + 4 * f
    code = (words[..., block * 2 * D + word].long() >> bit) & 15
    return code.double() * sb[..., token, d // group, 0].double() + sb[..., token, d // group, 1].double()


def exact(case, seed):
    if case["op"] == "maps":
        return None
    st = prepare(case, seed)
    page, D, group, H = st["page"], st["dim"], st["group"], case["kv_heads"]
    d = torch.arange(D, device=DEVICE)
    if case["op"] == "write":
        got = []
        for x in (st["k"], st["v"]):
            g = x.double().reshape(len(x), H, D // group, group)
            low, high = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
            step = ((high - low) / 15).to(x.dtype).double()
            code = ((g - low) / step).nan_to_num(0).round().clamp(0, 15)
            got.append((code * step + low).reshape(len(x), H, D) * (st["slots"] >= 0).double()[:, None, None])
        return got
    if case["op"] == "read":
        got = []
        for name, keys in (("k", True), ("v", False)):
            out = torch.zeros(st["tokens"], H, D, dtype=torch.float64, device=DEVICE)
            for part in torch.arange(st["tokens"], device=DEVICE).split(4096):
                slot = st["slots"][part].long()
                at = slot.clamp(min=0)
                words, sb = st[name + "_codes"][at // page], st[name + "_sb"][at // page]
                row = torch.arange(len(part), device=DEVICE)[:, None, None]
                head = torch.arange(H, device=DEVICE)[None, :, None]
                t = (at % page)[:, None, None]
                block, w = t // 16, t % 16
                if keys:
                    word = (d // 8 % 4 * 16 + w) * (D // 32) + d // 32
                    bit = 4 * (d % 8 // 2) + 16 * (d % 2)
                else:
                    half = ((w // 4 * 16 + d % 16) * (D // 64) + d // 64) * 4 + w % 4
                    word, bit = half // 2, 16 * (half % 2) + 4 * (d // 16 % 4)
                code = (words[row, head, block * 2 * D + word].long() >> bit) & 15
                pair = sb[row, head, t, d // group].double()
                out[part] = (code.double() * pair[..., 0] + pair[..., 1]) * (slot >= 0).double()[:, None, None]
            got.append(out)
        return got
    heads, T, window = case["heads"], st["tokens"], case["window"]
    each = heads // H
    out = torch.zeros(T, heads, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=DEVICE)
    token = torch.arange(page, device=DEVICE)[:, None]
    begin = 0
    for r, (p, n) in enumerate(zip(*_lengths(case))):
        rows = slice(begin, begin + n)
        begin += n
        if not n:
            continue
        held = st["table"][r, :-(-(p + n) // page)].long()
        for h in range(H):
            k = _cell(st["k_codes"][held, h], st["k_sb"][held, h], token, d, group, True).flatten(0, 1)[:p + n]
            v = _cell(st["v_codes"][held, h], st["v_sb"][held, h], token, d, group, False).flatten(0, 1)[:p + n]
            for first in range(0, n, 1024):
                part = torch.arange(first, min(n, first + 1024), device=DEVICE)
                at = p + part[:, None]
                key = torch.arange(p + n, device=DEVICE)
                hidden = (key > at) | (key <= at - window) if window else key > at
                for g in range(h * each, (h + 1) * each):
                    s = st["q"][rows, g].double()[part] @ k.T / math.sqrt(D)
                    s = s.masked_fill(hidden, -math.inf)
                    total = torch.logsumexp(s, -1)
                    out[begin - n + part, g] = torch.exp(s - total[:, None]) @ v
                    lse[begin - n + part, g] = total
    return (out, lse) if case["lse"] else out
