"""8-bit floats, the norm and rotary positions where arguments end: outputs laid over
inputs, and what every product kernel does at its edges.  References and bounds are
those of f8_reference.py.
"""
import itertools

import pytest
import torch

import f8_reference as ref
import matmul_affine_qmv_amd as qmx
from test_f8 import BF16, DEV, EOVER, F16, TYPES, apart, check_codes, check_norm, fake_ptr_test, gen, same, say

ELAUNCH = -9
BASE = 1 << 40   # placeholder addresses in bytes


# ---------------------------------------------------------------- outputs over inputs, on the CPU
def elements(at, n, rows, stride, size=2, sets=1, set_stride=0):
    """Every byte of `rows` rows of n elements, `sets` times."""
    return {at + size * (s * set_stride + r * stride + i) + b
            for s in range(sets) for r in range(rows) for i in range(n) for b in range(size)}


@fake_ptr_test
def test_norm_refuses_outputs_over_rows():
    """The sum may be x or the residual and a 16-bit result x or the residual, row for row; anything else that shares a
    byte is refused, and what shares none is not (there is no device here, so the launch fails)."""
    rows, width = 4, 128

    def norm(x=0, xs=width, r=10000, rs=width, s=20000, ss=width, out=30000, sc=None, w=40000, rows=rows):
        at = [None if v is None else BASE + v for v in (x, r, w, s, out, sc)]
        if r is None:
            at[3] = None
        return qmx.lib().qmx_rms_norm(at[0], xs, at[1], rs, at[2], at[3], ss, at[4], at[5], rows, width, 1e-6, BF16, None)

    good = [dict(), dict(s=0), dict(s=10000), dict(out=0), dict(out=10000), dict(s=10000, out=0), dict(s=0, out=10000),
            dict(s=0, xs=200, ss=200), dict(s=10000, rs=130, ss=130), dict(r=None, out=0), dict(x=10000), dict(x=10000, xs=0),
            dict(x=0, xs=256, s=256, ss=256), dict(x=0, xs=384, r=256, rs=384, s=512, ss=384),   # columns side by side
            dict(rows=1, xs=999, s=0, ss=5), dict(rows=1, xs=999, out=0), dict(sc=31000), dict(r=None, sc=31000),
            dict(x=0, xs=-width, out=2 * width), dict(x=0, xs=300, s=256, ss=300), dict(w=256 * rows, x=0)]
    bad = [dict(x=0, xs=256, r=256, rs=256, s=512, ss=512), dict(s=0, xs=200), dict(s=10000, rs=200), dict(s=0, xs=200, ss=201), dict(out=0, xs=200), dict(out=10000, rs=200),
           dict(out=0, xs=0), dict(s=0, xs=0, ss=width), dict(s=2), dict(s=256), dict(out=2), dict(out=254), dict(out=20000),
           dict(out=20000 + 2 * width * rows - 2), dict(s=40000), dict(out=40000), dict(w=20254), dict(sc=0, r=None),
           dict(sc=20002), dict(sc=30000 + width * rows - 1), dict(sc=40001), dict(sc=31000, out=0), dict(sc=31000, out=8),
           dict(sc=31000, out=10008), dict(sc=31000, out=20000), dict(x=0, xs=256, s=254, ss=256), dict(x=0, xs=-width, out=0),
           dict(x=0, xs=300, s=600, ss=250), dict(r=None, out=0, xs=width + 1), dict(r=None, out=2 * width),
           dict(x=0, xs=2 ** 40, s=2 * 2 ** 40 + 2, ss=200)]
    for case in good:
        assert norm(**case) == ELAUNCH, case
    for case in bad:
        assert norm(**case) == EOVER, case


@fake_ptr_test
def test_norm_overlaps_by_their_bytes():
    """Against the bytes themselves, for every small distance and stride."""
    rows, width = 3, 4
    for xs, ss, off in itertools.product((-9, -4, 0, 1, 3, 4, 5, 6, 8, 9, 13), (-9, 4, 5, 8, 9), range(-40, 41, 3)):
        x, s = BASE, BASE + 2 * off
        shared = elements(x, width, rows, xs) & elements(s, width, rows, ss)
        got = qmx.lib().qmx_rms_norm(x, xs, BASE + 10000, width, None, s, ss, BASE + 20000, None, rows, width, 1e-6, F16, None)
        assert got == (EOVER if shared and (off or xs != ss) else ELAUNCH), (xs, ss, off)


@pytest.mark.gpu
def test_norm_refuses_views_over_their_own_rows():
    """A contiguous view over the start of rows that are apart."""
    room = torch.randn(9 * 300, generator=gen(1)).half().to(DEV)
    x, w = room.view(9, 300)[:, :256], torch.ones(256, dtype=torch.half, device=DEV)
    view, other = room[:9 * 256].view(9, 256), torch.randn(9, 256, generator=gen(2)).half().to(DEV)
    before = room.clone()
    for call in (lambda: qmx.rms_norm(x, w, out=view), lambda: qmx.rms_norm(x, w, other, sum_out=view),
                 lambda: qmx.rms_norm(other, w, x, sum_out=view), lambda: qmx.rms_norm(other, w, x, out=view),
                 lambda: qmx.rms_norm_f8(x, w, other, sum_out=view)):
        with pytest.raises(qmx.QmxError, match="overlap"):
            call()
    assert same(room, before)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [640, 5000, 20480])
def test_norm_into_the_residual(width):
    """A result over the residual, row for row, the sum over x or by itself."""
    say("into the residual", width)
    g = gen(width)
    x, r = torch.randn(33, width, generator=g).bfloat16(), torch.randn(33, width, generator=g).bfloat16()
    w = torch.randn(width, generator=g).bfloat16().to(DEV)
    y, h = (t.cpu() for t in qmx.rms_norm(x.to(DEV), w, r.to(DEV)))
    for over in (True, False):
        dx, dr = apart(x, 3, 1) if over else x.to(DEV), r.to(DEV)
        got, total = qmx.rms_norm(dx, w, dr, sum_out=dx if over else None, out=dr)
        assert got is dr and same(dr, y) and same(total, h) and same(dx, h if over else x)


@fake_ptr_test
def test_rope_refuses_outputs_over_heads():
    """An output may be its own input, stride for stride; anything else that shares a byte is refused."""
    T, H, G, D = 3, 4, 2, 64
    fused = dict(qs=(512, 64), os=(512, 64), ks=(512, 64), kos=(512, 64))   # of 8 heads

    def rope(q=0, qs=(H * D, D), qo=20000, os=(H * D, D), k=40000, ks=(G * D, D), ko=60000, kos=(G * D, D), pos=80000,
             f=80104, T=T, H=H, G=G):
        at = [BASE + v for v in (q, qo, k, ko, pos, f)]
        return qmx.lib().qmx_rope(at[0], *qs, at[1], *os, H, at[2], *ks, at[3], *kos, G, at[4], at[5], T, D, D // 2, 0, 1.0,
                                  BF16, None)

    good = [dict(), dict(qo=0), dict(ko=40000), dict(qo=0, ko=40000), dict(q=40000), dict(fused, qo=0, k=512, ko=512),
            dict(fused, qo=0, k=512), dict(fused, k=512, ko=512), dict(fused, k=512, qo=40000, ko=40512),
            dict(fused, q=0, k=512, qo=768, os=(512, 64), H=2, G=2, ko=1000000),   # each its own quarter of a token
            dict(T=1, qs=(5, 64), qo=0, os=(9999, 64)), dict(H=1, qs=(64, 7), qo=0, os=(64, 64)), dict(H=0, qo=40000, G=2),
            dict(G=0, ko=0), dict(qs=(0, 64)), dict(k=0, ks=(H * D, D), ko=40000),
            dict(qs=(192 * 4, 192), k=128, ks=(192 * 4, 192), G=4, qo=0, os=(192 * 4, 192), ko=128, kos=(192 * 4, 192))]
    bad = [dict(fused, qo=40000, ko=40512), dict(qo=0, os=(512, 64)), dict(qs=(512, 64), qo=0), dict(qs=(64, 256), qo=0, os=(256, 64)), dict(qo=2),
           dict(qo=512), dict(qo=2 * H * D * T - 2), dict(qo=40000), dict(ko=0), dict(qo=60000), dict(qo=60000 + 128),
           dict(qo=0, ko=0), dict(qo=79000), dict(ko=80000), dict(ko=80104 - 2), dict(qo=80000 - 2 * H * D * T + 4),
           dict(fused, qo=0, k=510, ko=1000000), dict(fused, qo=0, k=512, ko=514), dict(fused, qo=0, k=512, ko=512 - 128),
           dict(ko=40000, kos=(128, 64), ks=(129, 64)), dict(T=2, qs=(5, 64), qo=0, os=(9999, 64)), dict(qo=0, qs=(0, 64)),
           dict(q=40000, ko=40000), dict(k=0, ks=(H * D, D), qo=0, ko=0, kos=(H * D, D))]
    for case in good:
        assert rope(**case) == ELAUNCH, case
    for case in bad:
        assert rope(**case) == EOVER, case


@fake_ptr_test
def test_rope_overlaps_by_their_bytes():
    """Keys turned into places among the queries', against the bytes themselves."""
    T, D = 3, 2
    layouts = [(2, 8, 2), (3, 6, 2), (2, 12, 5), (2, 2, 9), (1, 4, 0), (4, 8, 2), (2, -8, 2)]   # heads, token and head strides
    for (H, ts, hs), (G, kts, khs), off in itertools.product(layouts, layouts, range(-60, 61, 7)):
        q, ko = BASE, BASE + 2 * off
        shared = elements(q, D, H, hs, 2, T, ts) & elements(ko, D, G, khs, 2, T, kts)
        got = qmx.lib().qmx_rope(q, ts, hs, BASE + 10000, 8, 2, H, BASE + 20000, 8, 2, ko, kts, khs, G, BASE + 30000,
                                 BASE + 31000, T, D, 1, 0, 1.0, F16, None)
        assert got == (EOVER if shared else ELAUNCH), (H, ts, hs, G, kts, khs, off)


@pytest.mark.gpu
def test_rope_refuses_views_over_their_own_heads():
    T, H, D = 5, 4, 64
    room = torch.randn(T * H * 96, generator=gen(3)).half().to(DEV)
    q, view = room.view(T, H, 96)[..., :D], room[:T * H * D].view(T, H, D)
    at, f = torch.arange(T, dtype=torch.int32, device=DEV), qmx.rope_frequencies(D, device=DEV)
    other, before = torch.empty_like(view), room.clone()
    for call in (lambda: qmx.rope(q, None, at, f, out=(view, None)), lambda: qmx.rope(q, q, at, f, out=(q, q)),
                 lambda: qmx.rope(q, q, at, f, out=(other, other)), lambda: qmx.rope(q, q, at, f, out=(q, other)),
                 lambda: qmx.rope(q[:, :2], q[:, 1:], at, f, out=(q[:, :2], q[:, 1:]))):
        with pytest.raises(qmx.QmxError, match="overlap"):
            call()
    assert same(room, before)
