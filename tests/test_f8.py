"""8-bit floats, the norm before them and rotary positions: refusals on the CPU; the
operators against the 64-bit reference of f8_reference.py on a GPU.
"""
import math
import os
import sys

import pytest
import torch

import f8_reference as ref
import matmul_affine_qmv_amd as qmx

if not os.path.exists(qmx.LIB_PATH):
    pytest.skip("libqmx.so not built", allow_module_level=True)

OK, ENULL, ESHAPE, EGROUP, EDTYPE, EALIGN, EWS, EOVER = 0, -1, -2, -4, -5, -6, -7, -12
F32, F16, BF16 = 0, 1, 2
E8M0, SF32 = 0, 1
FAKE, ODD = 0x10000, 0x10001
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same(a, b):
    """Bits equal, NaNs of 16-bit types any."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    assert a.shape == b.shape and a.element_size() == b.element_size()
    if a.dtype in TYPES:
        assert a.dtype is b.dtype
        nan = torch.isnan(a)
        return torch.equal(nan, torch.isnan(b)) and torch.equal(a[~nan].view(torch.int16), b[~nan].view(torch.int16))
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- on the CPU
# Placeholder pointers must never reach a kernel: with a GPU in sight these are skipped.
fake_ptr_test = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder pointers: CPU-only checks")


@fake_ptr_test
def test_norm_refusals():
    def norm(x=FAKE, r=None, w=FAKE, s=None, out=FAKE, sc=None, rows=2, width=256, eps=1e-6, dt=BF16, ss=256):
        return qmx.lib().qmx_rms_norm(x, 256, r, 256, w, s, ss, out, sc, rows, width, eps, dt, None)

    assert norm(dt=F32) == EDTYPE and norm(dt=9) == EDTYPE
    for bad in (dict(rows=-1), dict(width=-1), dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf)):
        assert norm(**bad) == ESHAPE, bad
    for stride in (255, 0, -255):
        assert norm(r=FAKE, s=FAKE + 2 ** 20, ss=stride) == EOVER
    for both in (dict(r=FAKE + 2 ** 20, s=FAKE), dict(sc=FAKE), dict(r=FAKE, s=FAKE + 2 ** 20, x=FAKE + 2 ** 20, sc=FAKE)):
        assert norm(**both) == EOVER, both
    assert norm(sc=FAKE, width=200) == EGROUP
    for bad in (dict(x=None), dict(out=None), dict(r=FAKE), dict(s=FAKE)):
        assert norm(**bad) == ENULL, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(out=ODD), dict(r=ODD, s=FAKE), dict(r=FAKE, s=ODD),
                dict(out=0x10004, sc=FAKE)):
        assert norm(**bad) == EALIGN, bad
    assert norm(rows=0, x=None) == OK and norm(width=0, x=None) == OK


@fake_ptr_test
def test_codes_refusals():
    L = qmx.lib()

    def quantize(x=FAKE, c=FAKE, s=FAKE, rows=3, width=256, block=1, dt=F16):
        return L.qmx_f8_quantize(x, 256, c, s, rows, width, block, dt, None)

    def dequantize(c=FAKE, s=FAKE, kind=E8M0, o=FAKE, rows=3, width=256, block=1, dt=F16):
        return L.qmx_f8_dequantize(c, s, kind, o, rows, width, block, dt, None)

    for f in (quantize, dequantize):
        assert f(dt=F32) == EDTYPE
        assert f(rows=-1) == ESHAPE and f(width=-128) == ESHAPE and f(rows=2 ** 31 - 1, width=256) == ESHAPE
        assert f(rows=2 ** 29 + 1, width=128) == ESHAPE
        assert f(width=100) == EGROUP and f(block=2) == EGROUP and f(block=0) == EGROUP
        assert f(c=None) == ENULL and f(s=None) == ENULL
        assert f(c=0x10008) == EALIGN
        assert f(rows=0, c=None) == OK and f(width=0, c=None) == OK
    assert quantize(x=None) == ENULL and quantize(x=ODD) == EALIGN
    assert dequantize(o=None) == ENULL and dequantize(o=0x10008) == EALIGN
    assert dequantize(kind=2) == EDTYPE and dequantize(kind=-1) == EDTYPE
    assert dequantize(kind=SF32, s=0x10002) == EALIGN


@fake_ptr_test
def test_product_refusals():
    L = qmx.lib()

    def mm(w=FAKE, ws=FAKE, kind=E8M0, x=FAKE, xs=FAKE, out=FAKE, M=2, N=256, K=256, dt=BF16, work=None, size=0):
        return L.qmx_qmm_f8(w, ws, kind, x, xs, out, M, N, K, dt, work, size, None)

    assert mm(dt=F32) == EDTYPE and mm(kind=2) == EDTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K=-128), dict(K=2 ** 24), dict(M=2 ** 31 - 1, N=2 ** 31 - 1),
                dict(N=2 ** 25 + 1), dict(M=2 ** 30 + 1, N=1), dict(M=2 ** 30, N=1024)):
        assert mm(**bad) == ESHAPE, bad
    assert mm(K=200) == EGROUP and mm(K=64) == EGROUP
    for bad in (dict(w=None), dict(ws=None), dict(x=None), dict(xs=None), dict(out=None)):
        assert mm(**bad) == ENULL, bad
    for bad in (dict(w=0x10008), dict(x=0x10008), dict(out=ODD), dict(kind=SF32, ws=0x10002)):
        assert mm(**bad) == EALIGN, bad
    assert mm(M=0, out=None) == OK and mm(N=0, out=None) == OK
    need = L.qmx_qmm_f8_workspace_bytes(100, 128, 8192)
    assert need > 0 and need % (100 * 128 * 4) == 0
    big = dict(M=100, N=128, K=8192)
    assert mm(**big) == EWS and mm(**big, work=FAKE, size=need - 1) == EWS and mm(**big, work=0x10008, size=need) == EWS
    for sizes in ((-1, 128, 128), (1, -1, 128), (1, 1, 100), (0, 128, 8192), (100, 0, 8192), (100, 128, 0)):
        assert L.qmx_qmm_f8_workspace_bytes(*sizes) == 0


@fake_ptr_test
def test_rope_refusals():
    def rope(q=FAKE, qo=FAKE, heads=4, k=FAKE, ko=FAKE, kv=2, pos=FAKE, f=FAKE, T=3, D=128, pairs=64, scale=1.0,
             dt=BF16, out=(512, 128), kout=(256, 128)):
        return qmx.lib().qmx_rope(q, 512, 128, qo, *out, heads, k, 256, 128, ko, *kout, kv, pos, f, T, D, pairs,
                                  0, scale, dt, None)

    assert rope(dt=F32) == EDTYPE
    for bad in (dict(heads=-1), dict(kv=-1), dict(heads=8193), dict(kv=8193), dict(T=-1), dict(D=0), dict(D=4097),
                dict(pairs=0), dict(pairs=65), dict(scale=math.nan), dict(scale=math.inf)):
        assert rope(**bad) == ESHAPE, bad
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None), dict(f=None)):
        assert rope(**bad) == ENULL, bad
    for bad in (dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(ko=ODD), dict(pos=0x10002), dict(f=0x10004)):
        assert rope(**bad) == EALIGN, bad
    for bad in (dict(out=(0, 128)), dict(out=(512, 0)), dict(out=(511, 128)), dict(out=(512, 127)), dict(out=(128, 383)),
                dict(kout=(255, 128)), dict(kout=(-255, 128)), dict(kout=(256, 2 ** 62), D=129, pairs=1, T=2 ** 31 - 1)):
        assert rope(**bad) == EOVER, bad
    assert rope(T=0, q=None) == OK and rope(heads=0, kv=0, q=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes = torch.zeros(2, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(2, 2, dtype=torch.uint8)
    for call in (lambda: qmx.rms_norm(x, x[0]), lambda: qmx.rms_norm_f8(x, x[0]), lambda: qmx.f8_quantize(x),
                 lambda: qmx.f8_dequantize(codes, s), lambda: qmx.qmm_f8(codes, s, codes, s),
                 lambda: qmx.rope(x[None], None, torch.zeros(1, dtype=torch.int32), torch.zeros(2).double())):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_reference_codes():
    """The reference's own rounding: every code is its own, middles go to even codes."""
    finite = ~torch.isnan(ref.CODE)
    assert torch.equal(ref.nearest_code(ref.CODE[finite]).int(), torch.arange(256)[finite].int())
    v = ref.CODE[:126]
    middle = (v + ref.CODE[1:127]) / 2
    got = ref.nearest_code(middle).int()
    assert torch.equal(got, (torch.arange(126).int() + 1) // 2 * 2)
    # a type's own rounding agrees with torch's
    x = torch.randn(20, 384, generator=gen(1)).double() * 30
    x[0, 0] = 448
    assert torch.equal(ref.nearest_code(x.clamp(-448, 448)).view(torch.float8_e4m3fn).double(),
                       x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double())


def test_rope_frequencies():
    d, base, L = 128, 10000.0, 4096
    i = torch.arange(d // 2).double()
    plain = qmx.rope_frequencies(d, base, device="cpu")
    assert plain.dtype == torch.float64
    torch.testing.assert_close(plain, base ** (-2 * i / d), rtol=1e-14, atol=0)
    torch.testing.assert_close(qmx.rope_frequencies(d, base, scaling="linear", factor=4, device="cpu"), plain / 4,
                               rtol=1e-14, atol=0)
    f = qmx.rope_frequencies(d, base, scaling="base", factor=8, device="cpu")
    assert f[0] == 1 and abs(f[-1] * 8 / plain[-1] - 1) < 1e-12
    f = qmx.rope_frequencies(d, base, scaling="bands", factor=8, original_length=L, device="cpu")
    turns = L * plain / (2 * math.pi)
    assert torch.equal(f[turns >= 4], plain[turns >= 4])
    torch.testing.assert_close(f[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14, atol=0)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (f[mid] < plain[mid]).all() and (f[mid] > plain[mid] / 8).all()
    f = qmx.rope_frequencies(d, base, scaling="yarn", factor=8, original_length=L, device="cpu")
    assert torch.equal(f[turns >= 33], plain[turns >= 33])
    torch.testing.assert_close(f[turns < 0.8], plain[turns < 0.8] / 8, rtol=1e-14, atol=0)
    assert (f.diff() < 0).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(scaling="other"), dict(factor=0.5), dict(base=1.0),
                dict(scaling="yarn"), dict(scaling="bands"), dict(scaling="bands", original_length=9, low=4, high=4),
                dict(scaling="yarn", original_length=9, fast=1, slow=1), dict(rotary_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            qmx.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **bad})


# ---------------------------------------------------------------- on a GPU: the norm
def apart(t, gap=0, offset=0):
    """The same matrix on the GPU in rows `gap` elements apart, `offset` elements from an aligned address."""
    rows, width = t.shape
    room = torch.full((offset + rows * (width + gap) + 8,), float("nan"), dtype=t.dtype, device=DEV)
    v = room[offset:offset + rows * (width + gap)].view(rows, width + gap)[:, :width]
    v.copy_(t)
    return v


def norm_bound(y, w, dtype):
    """Half a step of the type, and float32's: the root, the product with it and that with w are each rounded by 2^-24 of
    themselves, the first product also by 2^-150 where it leaves the normal numbers."""
    return ref.half_step(y, dtype) * (1 + 1e-6) + 3 * 2.0 ** -24 * y.abs() + 2.0 ** -150 * (1 if w is None else w.double().abs())


def check_norm(x, w, r, y, eps, got, total):
    want, h = ref.norm(x, w, r, eps)
    if r is not None:
        assert same(total, h)
    off = (got.cpu().double() - want).abs()
    over = off - norm_bound(want, w, x.dtype)
    assert (over <= 0).all(), f"{over.max().item()} over half a step"


NORM_WIDTHS = [1, 2, 7, 8, 9, 127, 128, 130, 511, 512, 513, 1000, 2048, 2049, 4096, 4097, 8192, 8199, 16384, 16385, 40001]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("width", NORM_WIDTHS)
def test_norm_widths(width, dtype):
    say("norm", width, dtype)
    g = gen(width)
    for rows, gap, offset, res in ((1, 0, 0, True), (5, 3, 1, True), (6, 0, 5, False)):
        x = (torch.randn(rows, width, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(dtype)
        r = (30 * torch.randn(rows, width, generator=g)).to(dtype) if res else None
        w = torch.randn(width, generator=g).to(dtype)
        got = qmx.rms_norm(apart(x, gap, offset), w.to(DEV), apart(r, gap, offset) if res else None, eps=1e-5)
        check_norm(x, w, r, None, 1e-5, got[0] if res else got, got[1] if res else None)


def check_codes(codes, scales, y):
    """Codes and scales of y in 64 bits, which both sides have but for a sum's and five more roundings: (width + 10) *
    2^-53 of it.  What lies nearer than that to a middle (a row of one value times a weight that is one) may go
    either way."""
    near = (y.shape[1] + 10) * 2.0 ** -53
    fits = torch.zeros(y.shape, dtype=torch.bool)
    for z in (y * (1 - near), y, y * (1 + near)):
        c, s = ref.quantize(z)
        fits |= (codes.cpu().view(torch.uint8) == c) & (scales.cpu().view(torch.uint8) == s).repeat_interleave(128, 1)
    assert fits.all(), (~fits).nonzero()[:4]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("width", [128, 384, 512, 640, 2048, 2176, 4096, 5120, 8192, 8320, 16384, 16512, 33024])
def test_norm_f8(width, dtype):
    """Codes and scales are those of 64 bits."""
    say("norm f8", width, dtype)
    g = gen(width + 1)
    for rows, gap, offset, res in ((1, 0, 0, True), (7, 5, 3, False), (9, 0, 0, True)):
        x = torch.randn(rows, width, generator=g).to(dtype)
        x[:, ::17] *= 40
        r = torch.randn(rows, width, generator=g).to(dtype) if res else None
        w = (1 + 0.3 * torch.randn(width, generator=g)).to(dtype)
        codes, scales, *total = qmx.rms_norm_f8(apart(x, gap, offset), w.to(DEV), apart(r, gap, offset) if res else None)
        y, h = ref.norm(x, w, r, 1e-6)
        check_codes(codes, scales, y)
        if res:
            assert same(total[0], h)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [600, 1500, 8300])
@pytest.mark.parametrize("width", [64, 512, 1000, 1536, 2048, 2049, 2560, 4096, 4097, 5120, 8192, 9216, 12290, 16384])
def test_norm_many_rows(width, rows):
    """Lanes and elements a lane are picked by rows and width; large sums are stored another way."""
    say("norm many", rows, width)
    g = torch.Generator(device=DEV).manual_seed(width)
    x = torch.randn(rows, width, device=DEV, generator=g).bfloat16()
    r = torch.randn(rows, width, device=DEV, generator=g).bfloat16()
    w = (1 + 0.3 * torch.randn(width, device=DEV, generator=g)).bfloat16()
    some = torch.cat((torch.arange(20), torch.randint(rows, (20,), generator=gen(1)), torch.arange(rows - 20, rows)))
    got, total = qmx.rms_norm(x, w, r)
    y, h = ref.norm(x[some].cpu(), w.cpu(), r[some].cpu(), 1e-6)
    assert torch.equal(total, x + r)
    check_norm(x[some].cpu(), w.cpu(), r[some].cpu(), None, 1e-6, got[some], total[some])
    if width % 128 == 0:
        codes, scales, total = qmx.rms_norm_f8(x, w, r)
        assert torch.equal(total, x + r)
        check_codes(codes.view(torch.uint8)[some].view(codes.dtype), scales.view(torch.uint8)[some].view(scales.dtype), y)
        codes, scales = qmx.rms_norm_f8(total, w)
        check_codes(codes.view(torch.uint8)[some].view(codes.dtype), scales.view(torch.uint8)[some].view(scales.dtype), y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_norm_ranges(dtype):
    """Rows of the largest, of the smallest and of no magnitude, and rows that hold a NaN or an infinity, which
    touch no other row."""
    fi = torch.finfo(dtype)
    small = fi.tiny * fi.eps
    for width in (256, 3000 // 128 * 128, 20480):
        x = torch.randn(9, width, generator=gen(width)).to(dtype)
        x[0] = fi.max
        x[1] = 0
        x[2] = small
        x[3, ::3] = -fi.max
        x[4] = x[4] * fi.tiny * 4
        x[6, 5] = math.nan
        x[7, 130] = -math.inf
        w = torch.randn(width, generator=gen(3)).to(dtype)
        for weight in (w, None):
            for eps in (1e-6, 1e-30, 1e-300):
                say("range", dtype, width, eps)
                y, _ = ref.norm(x, weight, None, eps)
                dw = weight.to(DEV) if weight is not None else None
                got = qmx.rms_norm(x.to(DEV), dw, eps=eps).cpu().double()
                bad = ~torch.isfinite(y)
                assert torch.equal(torch.isnan(got), torch.isnan(y))
                fine = torch.where(bad, 0.0, got - y).abs()
                most = norm_bound(torch.where(bad, 0.0, y), weight, dtype)
                # past the largest number what is rounded is infinite
                beyond = y.abs() > fi.max
                assert ((fine <= most) | beyond).all()
                codes, scales = qmx.rms_norm_f8(x.to(DEV), dw, eps=eps)
                check_codes(codes, scales, torch.where(y.abs() > torch.finfo(torch.float32).max, math.inf, y))


@pytest.mark.gpu
def test_norm_of_nothing_and_next_to_nothing():
    """Groups of zeros, with weights of any kind, and groups that only a large weight brings back into range."""
    x = torch.zeros(6, 640)
    x[:, :128] = 2.0 ** 30
    x[1, 128:256] = 2.0 ** -133
    x[2, 256::3] = 2.0 ** -120
    x[3, 130] = -2.0 ** -133
    x[4, 128:] = -0.0
    x[5] = 0
    x = x.bfloat16()
    w = torch.ones(640)
    w[128:] = 2.0 ** 59
    w[384:512] = 2.0 ** 127
    w[512:514] = torch.tensor([math.inf, math.nan])
    w = w.bfloat16()
    for weight in (w, w.flip(0), None):
        for lead in (1, 400):   # few rows and many
            codes, scales = qmx.rms_norm_f8(x.to(DEV).repeat(lead, 1), None if weight is None else weight.to(DEV))
            y, _ = ref.norm(x, weight, None, 1e-6)
            y = torch.where(y.abs() > torch.finfo(torch.float32).max, math.inf, y)
            check_codes(codes.view(torch.uint8)[-6:].view(codes.dtype), scales.view(torch.uint8)[-6:].view(scales.dtype), y)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [640, 5000, 20480])
def test_norm_in_place(width):
    """The sum over x or over the residual, the result over x."""
    g = gen(5)
    x, r = torch.randn(33, width, generator=g).bfloat16(), torch.randn(33, width, generator=g).bfloat16()
    w = torch.randn(width, generator=g).bfloat16().to(DEV)
    y, h = (t.cpu() for t in qmx.rms_norm(x.to(DEV), w, r.to(DEV)))
    dx, dr = apart(x, 3, 1), apart(r, 8)
    y1, h1 = qmx.rms_norm(dx, w, dr, sum_out=dr)
    assert h1 is dr and same(y1, y) and same(dr, h) and same(dx, x)
    dx, dr = apart(x, 3, 1), apart(r, 8)
    y1, h1 = qmx.rms_norm(dx, w, dr, sum_out=dx)
    assert same(y1, y) and same(dx, h) and same(dr, r)
    dx = x.to(DEV)
    dr = r.to(DEV)
    y1, h1 = qmx.rms_norm(dx, w, dr, sum_out=dr, out=dx)
    assert same(dx, y) and same(dr, h)
    plain = qmx.rms_norm(x.to(DEV), w)
    dx = x.to(DEV)
    assert same(qmx.rms_norm(dx, w, out=dx), plain) and same(dx, plain)
    if width % 128 == 0:
        dr = r.to(DEV)
        c, s, h1 = qmx.rms_norm_f8(x.to(DEV), w, dr, sum_out=dr)
        c2, s2, _ = qmx.rms_norm_f8(x.to(DEV), w, r.to(DEV))
        assert same(c, c2) and same(s, s2) and same(dr, h) and same(h1, h)


@pytest.mark.gpu
def test_norm_shared_rows_and_nothing():
    """A row that stands for all (stride 0), no rows, no columns."""
    x = torch.randn(1, 300, generator=gen(6)).half()
    w = torch.randn(300, generator=gen(7)).half().to(DEV)
    one = qmx.rms_norm(x.to(DEV), w)
    many = qmx.rms_norm(x.to(DEV).expand(70, 300), w)
    assert same(many, one.expand(70, 300))
    total, sums = qmx.rms_norm(x.to(DEV).expand(70, 300), w, x.to(DEV).expand(70, 300))
    assert total.is_contiguous() and sums.is_contiguous() and same(sums, (x + x).expand(70, 300))
    for f in (qmx.rms_norm_f8, qmx.f8_quantize):
        part = x[:, :256].to(DEV)
        for a, b in zip(f(part.expand(70, 256)), f(part)):
            assert a.is_contiguous() and same(a, b.view(torch.uint8).expand(70, b.shape[1]).view(b.dtype))
    with pytest.raises(qmx.QmxError):
        qmx.rms_norm(x.to(DEV).expand(70, 300), w, x.to(DEV).expand(70, 300), sum_out=x.to(DEV).expand(70, 300))
    assert qmx.rms_norm(torch.empty(0, 300, device=DEV, dtype=torch.half), w).shape == (0, 300)
    assert qmx.rms_norm(torch.empty(4, 0, device=DEV, dtype=torch.half), w[:0]).shape == (4, 0)


# ---------------------------------------------------------------- codes
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_every_value(dtype, block):
    """Every 16-bit pattern, in groups of like and of unlike magnitudes."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    g = gen(11)
    orders = [bits, bits[torch.randperm(65536, generator=g)], bits.view(512, 128).T.reshape(-1)]
    for order in orders:
        x = order.view(dtype).view(-1, 256 if block == 1 else 128)
        if block == 1:
            x = torch.cat((x, x.nan_to_num(0, 0, 0)))
        else:
            x = x.nan_to_num(0, 0, 0) if order is orders[1] else x
        codes, scales = qmx.f8_quantize(x.to(DEV), block_rows=block)
        want = ref.quantize(x, block)
        assert same(scales, want[1]) and same(codes, want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width,block,gap,offset", [
    (1, 128, 1, 0, 0), (3, 384, 1, 5, 1), (67, 1152, 1, 0, 3), (1, 128, 128, 0, 0), (127, 256, 128, 1, 0),
    (128, 384, 128, 0, 0), (129, 128, 128, 8, 7), (300, 640, 128, 0, 0), (1000, 128, 1, 0, 0), (0, 256, 1, 0, 0),
    (0, 256, 128, 0, 0), (5, 0, 1, 0, 0)])
def test_quantize_shapes(rows, width, block, gap, offset, dtype):
    say("quantize", rows, width, block, gap, offset)
    x = torch.randn(rows, width, generator=gen(rows + width)) * torch.exp(4 * torch.randn(rows, 1, generator=gen(1)))
    x = x.to(dtype)
    x[rows // 2:rows // 2 + 1] = 0
    codes, scales = qmx.f8_quantize(apart(x, gap, offset), block_rows=block)
    if width == 0:
        assert codes.shape == (rows, 0) and qmx.f8_dequantize(codes, scales).shape == (rows, 0)
        return
    want = ref.quantize(x, block)
    assert same(scales, want[1]) and same(codes, want[0])
    for to in TYPES:
        back = qmx.f8_dequantize(codes, scales, dtype=to)
        assert same(back, ref.values(want[0], want[1]).to(torch.float32).to(to))
    f = (torch.rand(scales.shape, generator=gen(2)) + 0.1).to(DEV)
    back = qmx.f8_dequantize(codes, f, dtype=dtype)
    s = f.cpu() if block == 1 else f.cpu().repeat_interleave(128, 0)[:rows]
    c = codes.cpu().float().unflatten(1, (-1, 128))
    assert same(back, (c * s[..., None]).flatten(1).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_dequantize_every_code(dtype):
    """Every code under every scale."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2)
    got = qmx.f8_dequantize(codes.to(DEV).view(torch.float8_e4m3fn), scales.to(DEV), dtype=dtype).cpu()
    # exact in 64 bits and in 32; then one rounding
    want = ref.values(codes, scales).float().to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine].view(torch.int16), want[fine].view(torch.int16))


@pytest.mark.gpu
def test_codes_into_given_tensors():
    x = torch.randn(40, 512, generator=gen(3)).half().to(DEV)
    codes, scales = qmx.f8_quantize(x)
    c = torch.empty_like(codes)
    s = torch.empty(40, 4, dtype=torch.uint8, device=DEV)
    assert qmx.f8_quantize(x, out=(c, s))[0] is c and same(c, codes) and same(s, scales)
    o = torch.empty(40, 512, dtype=torch.bfloat16, device=DEV)
    assert qmx.f8_dequantize(c, s, out=o) is o and same(o, qmx.f8_dequantize(codes, scales))
    for call in (lambda: qmx.f8_quantize(x, out=(c[:39], s)), lambda: qmx.f8_quantize(x, block_rows=64),
                 lambda: qmx.f8_quantize(x.float()), lambda: qmx.f8_quantize(x[:, :100]),
                 lambda: qmx.f8_quantize(x.T), lambda: qmx.f8_dequantize(c, s[:2]),
                 lambda: qmx.f8_dequantize(c, s, dtype=torch.float32), lambda: qmx.f8_dequantize(x, s),
                 lambda: qmx.f8_dequantize(c.T, s)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- products
def coded(rows, K, block, seed, spread=1.0):
    """Random codes and E8M0 scales of numbers of unlike magnitudes."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    x = x * (1 + 20 * (torch.rand(K, generator=g) < 0.02))
    codes, scales = ref.quantize(x.bfloat16(), block)
    return codes.view(torch.float8_e4m3fn), scales


def check_product(M, N, K, dtype, f32=False, seed=0, most_rows=None, out=None):
    say("product", M, N, K, dtype, f32)
    x, xs = coded(M, K, 1, seed + 1)
    w, ws = coded(N, K, 128, seed + 2, 0.3)
    if f32:
        ws = (ref.scale_values(ws) * (0.5 + torch.rand(ws.shape, generator=gen(seed + 3)))).float()
    args = [t.to(DEV) for t in (w, ws, x, xs)]
    got = qmx.qmm_f8(*args, dtype=dtype, out=out)
    assert got.shape == (M, N) and got.dtype == dtype
    again = qmx.qmm_f8(*args, dtype=dtype)
    assert same(got, again)
    rows = torch.arange(M) if most_rows is None or M <= most_rows else torch.randperm(M, generator=gen(seed))[:most_rows]
    want, bound = ref.product(w, ws, x[rows], xs[rows])
    off = (got.cpu()[rows].double() - want).abs()
    most = bound + ref.half_step(want.abs() + bound, dtype)
    assert (off <= most).all(), (off / most).max().item()
    norm = want.norm().item()
    if norm:
        # half a step of every element, spread evenly, is 1 / sqrt(3) of it; the matrix instruction's own 1.6e-5 twice
        rounding = ref.half_step(want, dtype).norm().item() / norm
        assert off.norm().item() / norm <= rounding + 4e-5


SIZES = [(1, 1, 128), (1, 16, 128), (1, 129, 640), (2, 300, 256), (3, 128, 384), (15, 100, 512), (16, 257, 1152),
         (17, 64, 128), (31, 130, 640), (32, 48, 2048), (33, 200, 896), (47, 131, 1280), (48, 256, 512), (49, 90, 640),
         (63, 260, 384), (64, 128, 1024), (65, 129, 640), (100, 128, 8192), (127, 384, 1152), (128, 128, 128),
         (129, 500, 256), (200, 1, 2048), (257, 255, 640), (300, 1030, 1024), (1000, 3, 256), (513, 640, 384)]


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, dtype, f32):
    check_product(M, N, K, dtype, f32, seed=M + N + K, most_rows=48)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,f32", [(4096, 4096, 128, False), (4100, 4099, 384, True), (3900, 5000, 640, False),
                                       (8200, 2050, 256, False)])
def test_product_many_tiles(M, N, K, f32):
    check_product(M, N, K, torch.bfloat16, f32, seed=M, most_rows=24)


# On 256 compute units: of each kernel, whole and cut calls whose scales fit in LDS at once, and others.
EVERY = [(1, 512, 2048), (30, 2048, 2048), (16, 1001, 8192), (17, 8192, 5120), (1, 1000, 5120), (16, 4100, 12800),
         (640, 4100, 128), (33, 14001, 5120), (33, 2048, 5120), (40, 4100, 12800), (33, 20000, 1024), (48, 20004, 5120),
         (160, 2047, 12800), (1300, 512, 12800), (1300, 14000, 128), (512, 4100, 5120), (128, 4097, 12800),
         (640, 2048, 12800), (800, 14008, 1024), (2048, 4100, 5120), (300, 8192, 12800), (192, 20000, 12800)]


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "f32"])
@pytest.mark.parametrize("M,N,K", EVERY)
def test_product_every_kernel(M, N, K, f32):
    """Rows at both ends and every 61st, against 64 bits, with the reference's bound of the kernel's own errors, in which
    the largest of 8 products is at most the sum of their magnitudes; half a step of bfloat16 is 2^-8 of the result."""
    say("product every", M, N, K, f32)
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    w, ws = qmx.f8_quantize((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).bfloat16(), block_rows=128)
    x, xs = qmx.f8_quantize(torch.randn(M, K, generator=g, device=DEV).bfloat16())
    if f32:
        ws = ws.float() * (0.5 + torch.rand(ws.shape, generator=g, device=DEV))
    got = qmx.qmm_f8(w, ws, x, xs)
    X = x.double().view(M, -1, 128) * xs.double()[:, :, None]
    rows = torch.cat((torch.arange(min(M, 24)), torch.arange(max(0, M - 24), M), torch.arange(0, M, 61))).unique().to(DEV)
    X = X.view(M, K)[rows]
    step = 2048
    for n in range(0, N, step):
        W = w[n:n + step].double().view(-1, K // 128, 128)
        W = (W * ws[n // 128:(n + step) // 128].double().repeat_interleave(128, 0)[:len(W), :, None]).view(-1, K)
        want, most = X @ W.T, X.abs() @ W.abs().T * (7 * 2.0 ** -13 + (K // 128 + 20) * 2.0 ** -23)
        off = (got[rows, n:n + step].double() - want).abs()
        assert (off <= most + 2.0 ** -8 * (want.abs() + most)).all(), (n, (off - most).max().item())
        assert off.norm() <= (2.0 ** -8 / 3 ** 0.5 + 4e-5) * want.norm()
    assert same(got, qmx.qmm_f8(w, ws, x, xs))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_product_long_rows(M):
    check_product(M, 70, 17408 + 128, torch.float16, False, seed=M, most_rows=8)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(3, 64), (20, 64), (130, 128), (3, 65), (130, 131)])
def test_product_out_at_any_element(M, N):
    """An output between others', on an address that is no multiple of 8: nothing beside it changes."""
    room = torch.full((M * N + 9,), 7.0, dtype=torch.half, device=DEV)
    check_product(M, N, 512, torch.half, out=room[3:3 + M * N].view(M, N))
    assert (room[:3] == 7).all() and (room[3 + M * N:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 40, 150])
def test_product_special_values(M):
    """Scales at both ends, groups that are NaN, codes that are, and no groups at all."""
    N, K = 260, 512
    x, xs = coded(M, K, 1, 5)
    w, ws = coded(N, K, 128, 6)
    xs, ws = xs.clone(), ws.clone()
    xs[0] = 0
    ws[1] = 254       # with x's 2^-127 products of ordinary size
    if M > 2:
        xs[2, 1] = 255
        x = x.clone()
        x.view(torch.uint8)[3, 200] = 0xff
    got = qmx.qmm_f8(*[t.to(DEV) for t in (w, ws, x, xs)], dtype=torch.bfloat16).cpu().double()
    want = ref.values(x, xs) @ ref.values(w, ws).T
    # where magnitudes sum up beyond float32, parts of a sum may be infinities of both signs
    inside = ref.values(x, xs).abs() @ ref.values(w, ws).abs().T <= torch.finfo(torch.float32).max
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got)[inside | nan], nan[inside | nan])
    if M > 2:
        assert torch.isnan(got[2:4]).all()
    row0, bound = ref.product(w, ws, x[:1], xs[:1])
    assert ((got[:1] - row0).abs() <= bound + ref.half_step(row0.abs() + bound, torch.bfloat16) + 2.0 ** -133).all()
    # 2^127 and numbers beside 1: beyond the type
    big = want[1, 128:256].abs() > 3.5e38
    assert big.any() and not torch.isfinite(got[1, 128:256][big]).any()
    empty = torch.zeros(M, 0, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    none = torch.zeros(300, 0, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    zero = qmx.qmm_f8(none, torch.zeros(3, 0, dtype=torch.uint8, device=DEV), empty,
                      torch.zeros(M, 0, dtype=torch.uint8, device=DEV), out=torch.ones(M, 300, device=DEV).half())
    assert (zero == 0).all()


@pytest.mark.gpu
def test_product_binding():
    w, ws = (t.to(DEV) for t in coded(256, 1024, 128, 1))
    x, xs = (t.to(DEV) for t in coded(100, 1024, 1, 2))
    need = qmx.qmm_f8_workspace_bytes(100, 256, 1024)
    y = qmx.qmm_f8(w, ws, x, xs)
    if need:
        room = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
        assert same(qmx.qmm_f8(w, ws, x, xs, workspace=room), y)
        with pytest.raises(qmx.QmxError):
            qmx.qmm_f8(w, ws, x, xs, workspace=room[:need - 16])
    assert same(qmx.qmm_f8(w, ws.view(torch.float8_e8m0fnu), x, xs.view(torch.float8_e8m0fnu)), y)
    assert qmx.qmm_f8(w, ws, x[:0], xs[:0]).shape == (0, 256)
    assert qmx.qmm_f8(w[:0], ws[:0], x, xs).shape == (100, 0)
    for call in (lambda: qmx.qmm_f8(w, ws[:1], x, xs), lambda: qmx.qmm_f8(w, ws, x, xs[:9]),
                 lambda: qmx.qmm_f8(w, ws, x, xs.float()), lambda: qmx.qmm_f8(w, ws, x, xs, dtype=torch.float32),
                 lambda: qmx.qmm_f8(w, ws, x[:, :512], xs), lambda: qmx.qmm_f8(w, ws, x.view(torch.uint8), xs),
                 lambda: qmx.qmm_f8(w, ws, x, xs, out=torch.empty(100, 255, device=DEV).half()),
                 lambda: qmx.qmm_f8(w.T, ws, x, xs)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- rotary positions
def check_rope(q, k, positions, f, interleaved, scale, got):
    """Half a step of the type; and, of |a| + |b|, an angle off by 2^-23 (a turn's rest rounded to 24 digits, times
    2 pi), sine and cosine by 2^-22, their products with the scale and the sum by 3 * 2^-24."""
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        want, size = ref.rope(x, positions, f, interleaved, scale)
        off = (y.cpu().double() - want).abs()
        turned = size > 0
        most = torch.where(turned, ref.half_step(want, x.dtype) * (1 + 1e-6) + size * 2.0 ** -21, 0.0)
        assert (off <= most).all(), (off - most).max().item()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("T,heads,kv,D,n", [(1, 1, 1, 2, 1), (1, 32, 8, 128, 64), (3, 5, 1, 64, 32), (7, 4, 2, 128, 32),
                                            (5, 3, 3, 80, 40), (2, 2, 1, 81, 40), (4, 6, 2, 96, 13), (9, 1, 0, 256, 128),
                                            (6, 0, 4, 100, 3), (130, 40, 8, 128, 64), (300, 3, 1, 48, 20),
                                            (2049, 5, 2, 64, 32), (2050, 2, 1, 70, 9), (2, 2, 2, 4096, 2048),
                                            (2050, 1, 1, 1200, 600), (6, 1, 0, 3056, 1528), (3, 1, 0, 3080, 1532),
                                            (1030, 40, 8, 128, 64), (4100, 24, 4, 40, 20), (4099, 30, 9, 64, 30)])
def test_rope(T, heads, kv, D, n, interleaved, dtype):
    say("rope", T, heads, kv, D, n, interleaved, dtype)
    g = gen(T + D)
    q, k = torch.randn(T, heads, D, generator=g).to(dtype), torch.randn(T, kv, D, generator=g).to(dtype)
    at = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32)
    at[T // 2] = -1 if T > 2 else 0
    f = qmx.rope_frequencies(2 * n, 500000.0, device="cpu")
    scale = 1.0 if T % 2 else 1.2
    got = qmx.rope(q.to(DEV), k.to(DEV), at.to(DEV), f.to(DEV), interleaved=interleaved, scale=scale)
    check_rope(q, k, at, f, interleaved, scale, got)
    if heads:
        alone = qmx.rope(q.to(DEV), None, at.to(DEV), f.to(DEV), interleaved=interleaved, scale=scale)
        assert alone[1] is None and same(alone[0], got[0])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_rope_far(interleaved):
    """Positions to the end of 32 bits, and rates of half a turn and more a position."""
    at = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 1234567891, -1, -2 ** 31], dtype=torch.int32)
    f = torch.tensor([1.0, math.pi, 2 * math.pi, 6.0, 1e-3, 1e-9, 0.0, 0.37], dtype=torch.float64)
    q = torch.randn(7, 2, 16, generator=gen(4)).half()
    got = qmx.rope(q.to(DEV), None, at.to(DEV), f.to(DEV), interleaved=interleaved)
    for x, y in ((q, got[0]),):
        want, size = ref.rope(x, at, f, interleaved, 1.0)
        off = (y.cpu().double() - want).abs()
        # an angle of up to 2^31 * 2 pi in 64 bits is off by three roundings of 2^-53 of itself: 2^-18.7
        most = ref.half_step(want, x.dtype) * (1 + 1e-6) + size * (2.0 ** -21 + 2.0 ** -18)
        assert (off <= torch.where(size > 0, most, torch.zeros_like(most))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("T", [6, 2100])
def test_rope_strides_and_in_place(T, interleaved):
    """Parts of a fused projection's rows, at any element, turned where they are: nothing else changes."""
    H, G, D, n = 6, 2, 72, 24
    g = gen(8)
    fused = torch.randn(T, H + 2 * G, D, generator=g).bfloat16()
    at = torch.randint(-1, 5000, (T,), generator=g, dtype=torch.int32)
    f = qmx.rope_frequencies(2 * n, device="cpu")
    room = torch.zeros(fused.numel() + 3, dtype=torch.bfloat16, device=DEV)
    there = room[3:].view(fused.shape)
    there.copy_(fused)
    q, k = there[:, :H], there[:, H:H + G]
    out = qmx.rope(q, k, at.to(DEV), f.to(DEV), interleaved=interleaved, scale=0.7)
    check_rope(fused[:, :H], fused[:, H:H + G], at, f, interleaved, 0.7, out)
    assert same(there, fused)
    got = qmx.rope(q, k, at.to(DEV), f.to(DEV), interleaved=interleaved, scale=0.7, out=(q, k))
    assert got[0] is q and same(q, out[0]) and same(k, out[1]) and same(there[:, H + G:], fused[:, H + G:])
    assert (room[:3] == 0).all()
    # heads before tokens, as some programs keep them
    t = fused[:, :H].to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    assert same(qmx.rope(t, None, at.to(DEV), f.to(DEV), interleaved=interleaved, scale=0.7)[0], out[0])


@pytest.mark.gpu
def test_rope_binding():
    q = torch.zeros(4, 2, 64, dtype=torch.half, device=DEV)
    at, f = torch.zeros(4, dtype=torch.int32, device=DEV), qmx.rope_frequencies(64, device=DEV)
    for call in (lambda: qmx.rope(q, q[:3], at, f), lambda: qmx.rope(q, None, at[:3], f),
                 lambda: qmx.rope(q, None, at.long(), f), lambda: qmx.rope(q, None, at, f.float()),
                 lambda: qmx.rope(q, None, at, torch.cat((f, f))), lambda: qmx.rope(q, None, at, f[:0]),
                 lambda: qmx.rope(q.float(), None, at, f), lambda: qmx.rope(q[:, :, ::2], None, at, f[:8]),
                 lambda: qmx.rope(q, None, at, f, out=(q, q)), lambda: qmx.rope(q, q, at, f, out=(q, None)),
                 lambda: qmx.rope(q, None, at, f, out=(q[:2], None)), lambda: qmx.rope(q, None, at.cpu(), f)):
        with pytest.raises(ValueError):
            call()
    assert qmx.rope(q[:0], q[:0], at[:0], f)[0].shape == (0, 2, 64)
    wide = q[:1].expand(4, 2, 64)
    assert same(qmx.rope(wide, wide, at, f)[1], q)
    with pytest.raises(qmx.QmxError):
        qmx.rope(wide, None, at, f, out=(wide, None))


@pytest.mark.gpu
def test_more_rows_than_a_grid_holds():
    """2^32 threads and more would be needed at once: the same as of the rows in parts."""
    say("norm")
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(2 ** 22 + 2 ** 21 + 5, 128, device=DEV, generator=g).half()
    w = torch.randn(128, device=DEV, generator=g).half()
    cuts = [0, 3, 2 ** 20 + 1, 2 ** 21 + 7, 2 ** 22 - 1, 2 ** 22 + 1, len(x)]
    parts = list(zip(cuts, cuts[1:]))
    whole = qmx.rms_norm_f8(x, w, x)
    for a, b in parts:
        for one, every in zip(qmx.rms_norm_f8(x[a:b], w, x[a:b]), whole):
            assert torch.equal(one.view(torch.uint8), every[a:b].view(torch.uint8))
    y = qmx.rms_norm(x[:, :9])
    assert all(torch.equal(qmx.rms_norm(x[a:b, :9]), y[a:b]) for a, b in parts)
    say("rope")
    q = x.view(-1)[:4 * (2 ** 24 + 3)].view(-1, 2, 2)
    at = torch.randint(-1, 2 ** 20, (len(q),), device=DEV, generator=g, dtype=torch.int32)
    f = qmx.rope_frequencies(2, device=DEV)
    turned = qmx.rope(q, q[:, :1], at, f)
    cuts = [0, 5, 2 ** 23 - 1, 2 ** 23 + 9, 2 ** 24 - 2, len(q)]
    for a, b in zip(cuts, cuts[1:]):
        for one, every in zip(qmx.rope(q[a:b], q[a:b, :1], at[a:b], f), turned):
            assert torch.equal(one.view(torch.uint8), every[a:b].view(torch.uint8))


@pytest.mark.gpu
def test_sizes_past_an_int():
    x = torch.ones(1, 1, dtype=torch.half, device=DEV).expand(2 ** 31, 1)
    codes = torch.empty(2 ** 31, 0, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(2 ** 31, 0, dtype=torch.uint8, device=DEV)
    at, f = torch.zeros(1, dtype=torch.int32, device=DEV), qmx.rope_frequencies(2, device=DEV)
    q = x.view(-1, 1, 1).expand(-1, 1, 2)
    for call in (lambda: qmx.rms_norm(x), lambda: qmx.rms_norm_f8(x), lambda: qmx.f8_quantize(x),
                 lambda: qmx.f8_dequantize(codes, scales), lambda: qmx.qmm_f8(codes[:1], scales[:1], codes, scales),
                 lambda: qmx.qmm_f8(codes, scales[:2 ** 24], codes[:1], scales[:1]),
                 lambda: qmx.qmm_f8_workspace_bytes(2 ** 32 + 1, 128, 128),
                 lambda: qmx.rope(q, None, at.expand(2 ** 31), f)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- together
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 150])
def test_a_layer_in_a_graph_and_on_a_stream(T):
    """Norm, product, rotation, quantiser and product, as one layer runs them: the same from a side stream and from a
    captured graph, replayed over new inputs between other work."""
    width, H, D = 1024, 6, 64
    g = gen(T)
    weight = torch.randn(width, generator=g).bfloat16().to(DEV)
    w1 = qmx.f8_quantize((torch.randn(H * D, width, generator=g) / 32).bfloat16().to(DEV), block_rows=128)
    w2 = qmx.f8_quantize((torch.randn(width, H * D, generator=g) / 20).bfloat16().to(DEV), block_rows=128)
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    f = qmx.rope_frequencies(D, device=DEV)

    def layer(x, r):
        codes, scales, total = qmx.rms_norm_f8(x, weight, r)
        q = qmx.qmm_f8(*w1, codes, scales).view(T, H, D)
        q, _ = qmx.rope(q, None, at, f, out=(q, None))
        y = qmx.qmm_f8(*w2, *qmx.f8_quantize(q.view(T, H * D)))
        return qmx.rms_norm(y, weight, total)

    inputs = [[torch.randn(T, width, generator=g).bfloat16().to(DEV) for _ in range(2)] for _ in range(4)]
    wanted = [[t.clone() for t in layer(*i)] for i in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(*inputs[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(same(a, b) for a, b in zip(got, wanted[0]))
    x, r = (t.clone() for t in inputs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, r)
    for i, want in zip(inputs, wanted):
        x.copy_(i[0])
        r.copy_(i[1])
        layer(*inputs[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_example_of_layers():
    """Prompts, then graph replays of one token each.  Of a row's largest output a product is off by half a step of
    bfloat16, 2^-9, and by the matrix instruction's cuts: at most 7 * 2^-13 of the largest of each 8 products, of which a
    row of 512 or 1024 has 64 or 128 of some 3 (or 6 with its outliers) deviations, beside outputs of 3 * sqrt(512): again
    2^-9; a rotation is off by half a step; attention by 8 roundings, as examples/kv4_decode.py."""
    say("example")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import f8_layers
    errors = f8_layers.main(steps=12)
    assert len(errors) == 13 and max(errors) <= 8 * 2.0 ** -8, errors
