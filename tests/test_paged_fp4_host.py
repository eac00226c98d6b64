"""Host side of the 4-bit pages and of eviction: argument checks before any CUDA call, and pins of the oracle
(CPU only)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F4

P = 1 << 20   # a fake, aligned address that is never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def strides(x):
    return None if x is None else (ctypes.c_int64 * len(x))(*x)


def _append(fa, at=False, **kw):
    a = dict(q=P, k=P, v=P, q_out=P, k_out=P, k_pages=P, v_pages=P, k_scale=P, v_scale=P, table=P, stride=4, lens=P,
             cu=None, offsets=P, turns=P, qw=None, kw=None, strides=[512, 64] * 5, B=2, T=2, H=8, Hkv=2, d=64, pages=8,
             page=16, width=4, rot=64, inter=0, rs=1.0, eps=1e-6, max_new=0)
    a.update(kw)
    a["strides"] = strides(a["strides"])
    v = list(a.values())
    if at:  # with a flag for e4m3 pages
        v.insert(list(a).index("width") + 1, 1)
    return (fa.lib.fa_append_paged_at if at else fa.lib.fa_append_paged_fp4)(*v, None)


@pytest.mark.parametrize("at", [False, True], ids=["fp4", "e4m3 at"])
@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k_pages=None), INVALID), (dict(table=None), INVALID),
    (dict(turns=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(H=7), INVALID),
    (dict(T=3), INVALID), (dict(stride=3), INVALID), (dict(eps=-1.0), INVALID), (dict(offsets=P + 2), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(v_pages=P + 8), UNSUPPORTED),
    (dict(strides=[512, 64] * 3 + [512, 0] + [512, 64]), UNSUPPORTED), (dict(T=0, q=None, k=None, v=None, q_out=None), 0),
])
def test_append_refusals(fa, kw, want, at):
    assert _append(fa, at, **kw) == want, fa.lib.fa_last_error_detail()


def test_append_scale_alignment(fa):
    assert _append(fa, k_scale=P + 8) == UNSUPPORTED and b"16-byte" in fa.lib.fa_last_error_detail()


def _decode(fa, **kw):
    a = dict(q=P, qs=[512, 64, 512], k=P, v=P, ks=P, vs=P, table=P, stride=64, lens=P, o=P, os=[512, 64, 64],
             lse=P, B=2, H=8, Hkv=2, Nq=1, d=64, pages=8, page=16, max_len=1000, scale=0.125, splits=4, ws=P,
             bytes=1 << 30)
    a.update(kw)
    a["qs"], a["os"] = strides(a["qs"]), strides(a["os"])
    return fa.lib.fa_decode_paged_fp4(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(B=0), INVALID), (dict(H=9), INVALID), (dict(max_len=-1), INVALID),
    (dict(splits=1025), INVALID), (dict(scale=float("inf")), INVALID), (dict(stride=62), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(Nq=33), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(vs=P + 4), UNSUPPORTED),
    (dict(os=[512, 0, 64]), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(bytes=64), WORKSPACE),
])
def test_decode_refusals(fa, kw, want):
    assert _decode(fa, **kw) == want, fa.lib.fa_last_error_detail()


def _read(fa, **kw):
    a = dict(k=P, v=P, ks=P, vs=P, kind=2, table=P, stride=4, lens=P, cu=P, ko=P, vo=P, strides=[128, 64] * 2, B=2, total=10,
             Hkv=2, d=64, pages=8, page=16, width=4)
    a.update(kw)
    a["strides"] = strides(a["strides"])
    return fa.lib.fa_read_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
    (dict(ko=None), INVALID), (dict(vo=None), INVALID), (dict(strides=None), INVALID), (dict(kind=3), INVALID),
    (dict(kind=-1), INVALID), (dict(kind=1, ks=None), INVALID), (dict(ks=None), INVALID), (dict(B=0), INVALID),
    (dict(total=-1), INVALID), (dict(Hkv=0), INVALID), (dict(width=0), INVALID), (dict(stride=3), INVALID),
    (dict(pages=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(k=P + 8), UNSUPPORTED),
    (dict(ko=P + 8), UNSUPPORTED), (dict(cu=P + 2), UNSUPPORTED), (dict(strides=[128, 60, 128, 64]), UNSUPPORTED),
    (dict(strides=[128, 64, 64, 64]), UNSUPPORTED), (dict(total=0, cu=None, ko=None, vo=None), 0),
])
def test_read_refusals(fa, kw, want):
    assert _read(fa, **kw) == want, fa.lib.fa_last_error_detail()


def _weigh(fa, **kw):
    a = dict(q=P, qs=[512, 64, 512], lse=P, k=P, ks=P, kind=2, table=P, stride=64, lens=P, w=P, ws=1000, B=2, H=8, Hkv=2, Nq=1,
             d=64, pages=8, page=16, max_len=1000, scale=0.125)
    a.update(kw)
    a["qs"] = strides(a["qs"])
    return fa.lib.fa_weigh_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(qs=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID),
    (dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(kind=7), INVALID), (dict(B=0), INVALID), (dict(H=9), INVALID),
    (dict(Nq=0), INVALID), (dict(max_len=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(ws=999), INVALID),
    (dict(stride=62), INVALID), (dict(d=80), UNSUPPORTED), (dict(Nq=33), UNSUPPORTED), (dict(H=1 << 20, Nq=1 << 20), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(q=P + 8), UNSUPPORTED), (dict(w=P + 2), UNSUPPORTED), (dict(qs=[512, 60, 512]), UNSUPPORTED),
])
def test_weigh_refusals(fa, kw, want):
    assert _weigh(fa, **kw) == want, fa.lib.fa_last_error_detail()


def _evict(fa, **kw):
    a = dict(w=P, ws=1000, k=P, v=P, ks=P, vs=P, kind=2, table=P, stride=64, lens=P, offsets=None, nt=2 * P, ns=8, kept=P,
             nl=2 * P, no=P, nw=2 * P, nws=128, width=128, B=2, Hkv=2, d=64, pages=8, page=16, max_len=1000, keep=100, first=4,
             recent=20)
    a.update(kw)
    return fa.lib.fa_evict_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=None), INVALID),
    (dict(nt=None), INVALID), (dict(kept=None), INVALID), (dict(nl=None), INVALID), (dict(no=None), INVALID),
    (dict(nw=None), INVALID), (dict(table=None), INVALID), (dict(kind=3), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(keep=0), INVALID), (dict(first=-1), INVALID), (dict(recent=-1), INVALID), (dict(first=90), INVALID),
    (dict(first=101), INVALID), (dict(recent=2147483647), INVALID), (dict(width=99), INVALID), (dict(ws=999), INVALID),
    (dict(nws=127), INVALID), (dict(stride=62), INVALID), (dict(ns=6), INVALID), (dict(max_len=(1 << 30) + 1), INVALID),
    (dict(nw=P), INVALID), (dict(nl=P), INVALID), (dict(nt=P), INVALID), (dict(B=1 << 20, Hkv=1 << 12), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(page=12), UNSUPPORTED), (dict(k=P + 8), UNSUPPORTED), (dict(vs=P + 8), UNSUPPORTED),
    (dict(kept=P + 2), UNSUPPORTED), (dict(offsets=P + 1), UNSUPPORTED),
])
def test_evict_refusals(fa, kw, want):
    assert _evict(fa, **kw) == want, fa.lib.fa_last_error_detail()


def test_workspace_of_the_fp4_decode(fa):
    for a in ((3, 4, 2, 1, 64, 1000, 4), (1, 32, 8, 1, 128, 1 << 20, 0)):
        assert fa.decode_paged_fp4_workspace_size(*a) > 0
    assert fa.decode_paged_fp4_workspace_size(3, 8, 3, 2, 64, 100, 4) == 0


def test_scale_bytes_are_the_upper_bytes_of_f16():
    b = np.arange(256, dtype=np.uint8)
    want = (b.astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    got = F4.scale_decode(b)
    assert np.array_equal(got, want, equal_nan=True)


def test_every_held_value_is_exact_in_f16_and_bf16():
    s = F4.scale_decode(np.arange(F4.nearest_even(np.array(F4.SCALE_MAX), F4._SCALES) + 1))
    x = (s[:, None] * F4.LEVELS).ravel()
    t = torch.from_numpy(x)
    assert x.max() == 61440 and torch.equal(t.to(torch.float16).double(), t) and torch.equal(t.to(torch.bfloat16).double(), t)


@pytest.mark.parametrize("value,scale,code", [
    (6.0, 1.0, 7), (6.375, 1.0, 7), (6.5, 1.125, 7), (0.0, 0.0, 0), (2.0 ** -130, 2.0 ** -17, 0), (1e30, 10240.0, 7),
    (61440.0, 10240.0, 7), (2.0 ** -17 * 6, 2.0 ** -17, 7), (2.0 ** -14 * 6, 2.0 ** -14, 7), (9 * 2.0 ** -17, 2.0 ** -16, 6),
])
def test_encode_pins(value, scale, code):
    """A group whose only element that is not 0 is `value`."""
    x = np.zeros(16)
    x[3] = value
    c, s = F4.encode(x)
    assert F4.scale_decode(s)[0] == scale and c[3] == code and (np.delete(c, 3) == 0).all()
    x[3] = -value
    assert F4.encode(x)[0][3] == (code | 8 if value else 8 * np.signbit(-value)) and F4.encode(x)[1][0] == s[0]


def test_ties_go_to_the_even_code():
    x = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.26, 0.74, 5.1, 4.9, 0.0])
    c, s = F4.encode(x)
    assert F4.scale_decode(s)[0] == 1.0
    assert c.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 1, 7, 6, 0]


def test_not_finite_makes_its_group_nan():
    x = np.ones(48)
    x[20], x[40] = np.inf, np.nan
    y = F4.held(x)
    assert np.isnan(y[16:]).all() and np.isfinite(y[:16]).all()


def test_error_of_a_row_is_bounded():
    """A step of the codes is at most 2 scales, so half a step at most 1 scale: max / 6, and 1/16 more for the scale's
    rounding; beyond 6 scales (the scale rounded down) by at most 1/16 of 6."""
    x = np.random.default_rng(0).standard_normal((200, 128))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    off = np.abs(F4.held(x) - x).reshape(200, 8, 16)
    most = np.abs(x).reshape(200, 8, 16).max(axis=-1, keepdims=True)
    assert (off <= most / 6 * (1 + 1 / 16)).all()


def test_kept_rows_pins():
    w = [5.0, 1.0, 9.0, 9.0, 0.0, math.nan, 9.0, -1.0, 7.0, 2.0]
    assert F4.kept_rows(w, 10, 10, 0, 0) == list(range(10))
    assert F4.kept_rows(w, 10, 4, 1, 1) == [0, 2, 3, 9]
    assert F4.kept_rows(w, 10, 4, 0, 0) == [2, 3, 6, 8]
    assert F4.kept_rows(w, 10, 9, 0, 0) == [0, 1, 2, 3, 4, 6, 7, 8, 9]
    assert F4.kept_rows(w, 8, 5, 2, 3) == [0, 1, 5, 6, 7]
    assert F4.kept_rows([0.0] * 6, 6, 3, 0, 1) == [0, 1, 5]
