"""GPU parity of the paged operators (fa_append_paged, fa_decode_paged) against
the fp64 oracle, alone and in a run of steps as a serving program makes them.

Tolerances. q and k of the append are computed in fp32 (a rotation is two
products and a sum of values no larger than the pair, a norm adds a factor: below
16 roundings of 2^-24 of the row's largest value) and rounded once to bf16, at
most half a step, 2^-8 of the value. An e4m3 code is off by at most half a step:
2^-4 of the value, or 2^-10 of the scale below the smallest normal code; codes
that were rounded again when their scale grew, by two of those. Values that are
not computed (v, bf16 rows) must match exactly. Attention has the forward pass's
tolerances (tests/parity.py).
"""

import math

import numpy as np
import pytest
import torch

from oracle import fp8 as FP8
from oracle import paged as OP
from parity import compare, to64

pytestmark = pytest.mark.gpu

BASE = 500000.0


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def near_bf16(got, ref, what=""):
    """Within the fp32 computation's error and half a bf16 step of the exact values [.., d]."""
    bound = 2.0 ** -8 * np.abs(ref) + 16 * 2.0 ** -24 * np.abs(ref).max(axis=-1, keepdims=True) + 1e-37
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - ref).max():.3e}"


def make_table(rng, B, count, width, spare=2):
    """A block table of shuffled pages, -1 past each sequence's own; returns it and the pool's size."""
    ids = rng.permutation(sum(count) + spare)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :count[b]] = ids[at:at + count[b]]
        at += count[b]
    return table, sum(count) + spare


def cuda(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


class Cache:
    """A pool with random earlier contents, and its fp64 mirror."""

    def __init__(self, rng, n, Hkv, page, d, f8):
        self.f8, g = f8, torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        self.gpu, self.scale = [], []
        for _ in range(2):
            x = torch.randn(n, Hkv, page, d, generator=g)
            if f8:
                e = torch.randint(-9, -5, (n, Hkv), generator=g)
                self.scale.append(torch.exp2(e.float()).cuda())
                self.gpu.append((x * 128).clamp(-448, 448).to(torch.float8_e4m3fn).cuda())
            else:
                self.scale.append(None)
                self.gpu.append(x.to(torch.bfloat16).cuda())

    def codes(self, i):
        return self.gpu[i].view(torch.uint8).cpu().numpy().copy()

    def scales(self, i):
        return to64(self.scale[i])

    def values(self, i):
        """Real values [n, Hkv, page, d] in fp64."""
        if not self.f8:
            return to64(self.gpu[i])
        return FP8.e4m3_decode(self.codes(i)) * self.scales(i)[:, :, None, None]

    def kw(self):
        return dict(k_scale=self.scale[0], v_scale=self.scale[1])


# new tokens and lengths (with them) of each sequence, heads, page, d, rot
APPEND = [
    # one token each: at a page's first row, its last, in the middle, and the very first token
    dict(new=[1, 1, 1, 1], lens=[17, 16, 5, 1], H=8, Hkv=2, page=16, d=64, rot=64),
    dict(new=[1, 1, 1], lens=[129, 64, 1000], H=8, Hkv=2, page=64, d=128, rot=128),
    # several tokens each (uniform), crossing a page
    dict(new=[3, 3], lens=[17, 130], H=6, Hkv=6, page=16, d=128, rot=32),
    # ragged prompts: none, one, a page, past a page, continuing a page
    dict(new=[0, 1, 32, 70, 45], lens=[40, 1, 32, 70, 60], H=4, Hkv=2, page=32, d=64, rot=48),
    dict(new=[300, 2, 129], lens=[300, 131, 257], H=7, Hkv=1, page=128, d=128, rot=64),
    dict(new=[5, 200], lens=[5, 210], H=2, Hkv=1, page=64, d=64, rot=16),
    # no rotation at all
    dict(new=[2, 9], lens=[9, 9], H=2, Hkv=2, page=16, d=64, rot=0),
    # far positions: the angle of every pair is exact there too (positions a table could not hold)
    dict(new=[2, 1], lens=[1000003, 777777], H=2, Hkv=1, page=128, d=128, rot=128),
]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("inter,norm", [(False, True), (True, False)], ids=["half-norm", "interleaved"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "n{}h{}kv{}p{}d{}r{}".format(
    "-".join(map(str, c["new"])), c["H"], c["Hkv"], c["page"], c["d"], c["rot"]))
def test_append(fa, case, inter, norm, f8):
    new, lens, H, Hkv, page, d, rot = (case[k] for k in ("new", "lens", "H", "Hkv", "page", "d", "rot"))
    rng = np.random.default_rng(sum(lens) * 7 + d + 2 * inter + f8)
    B, T = len(new), sum(new)
    first = [(L - n) // page for n, L in zip(new, lens)]
    count = [(L + page - 1) // page for L in lens]
    used, pool = make_table(rng, B, [c - f for c, f in zip(count, first)], max(c - f for c, f in zip(count, first)) + 1)
    table = np.full((B, max(count)), -1, dtype=np.int32)
    for b in range(B):
        table[b, first[b]:count[b]] = used[b, :count[b] - first[b]]
    cache = Cache(rng, pool, Hkv, page, d, f8)
    before = [cache.codes(i) if f8 else cache.values(i) for i in range(2)]
    scales = [cache.scales(i).copy() if f8 else None for i in range(2)]
    # parts of one projection, with tokens behind the last sequence that nobody touches
    qkv = torch.randn(T + 3, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    w = [cuda(1 + 0.3 * rng.standard_normal(d), torch.bfloat16) if norm else None for _ in range(2)]
    turns = fa.rotary_turns(rot, BASE) if rot else None
    uniform = len(set(new)) == 1
    cu = None if uniform else cuda(np.concatenate([[0], np.cumsum(new)]), torch.int32)
    if uniform:
        q, k, v = q[:T], k[:T], v[:T]
    qo = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full(k.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    fa.append_paged(q, k, v, cache.gpu[0], cache.gpu[1], cuda(table), cuda(lens, torch.int32), cu_seqlens=cu, turns=turns,
                    interleaved=inter, q_weight=w[0], k_weight=w[1], eps=1e-5, q_out=qo, k_out=ko, **cache.kw())
    assert fa.device_status() == fa.FA_OK

    tl = [] if turns is None else turns.tolist()
    rq, rk, pos = OP.append(to64(q[:T]), to64(k[:T]), to64(v[:T]), new, lens, tl, inter,
                            *[None if x is None else to64(x) for x in w], eps=1e-5)
    near_bf16(to64(qo)[:T], rq, "q")
    near_bf16(to64(ko)[:T], rk, "k")
    assert (qo[T:] == 7).all() and (ko[T:] == 7).all()
    seq = np.repeat(np.arange(B), new)
    for i, x in ((0, rk), (1, to64(v[:T]))):
        if not f8:
            want = before[i].copy()
            for t in range(T):
                want[table[seq[t], pos[t] // page], :, pos[t] % page] = x[t]
            got = cache.values(i)
            if i == 1:
                assert np.array_equal(got, want)
            else:
                near_bf16(got, want, "k pages")
            continue
        codes, sc = before[i].copy(), scales[i].copy()
        OP.store_e4m3(x, new, lens, table, page, codes, sc)
        assert np.array_equal(cache.scales(i), sc)
        if i == 1:
            assert np.array_equal(cache.codes(1), codes)   # v: every code
            continue
        got = cache.values(0)
        fresh = np.zeros(codes.shape, dtype=bool)
        ref = np.zeros(codes.shape)
        for t in range(T):
            at = (table[seq[t], pos[t] // page], slice(None), pos[t] % page)
            fresh[at], ref[at] = True, x[t]
        same = codes == cache.codes(0)
        assert same[~fresh].all()                          # rows written earlier, rounded again or not
        half = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc[:, :, None, None]) * (1 + 2.0 ** -16)
        assert np.all(np.abs(got - ref)[fresh] <= half[fresh])
        assert same[fresh].mean() > 0.999


def test_append_in_place_and_strided_outputs(fa):
    """q and k may be turned where they lie, and the outputs may be parts of a larger tensor; both give the bytes of
    separate contiguous outputs."""
    rng = np.random.default_rng(3)
    T, H, Hkv, d, page = 37, 4, 2, 128, 32
    table, pool = make_table(rng, 1, [2], 2)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    turns = fa.rotary_turns(d, BASE)
    got = []
    for mode in range(3):
        x = qkv.clone()
        cache = Cache(np.random.default_rng(5), pool, Hkv, page, d, True)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        kw = {}
        if mode == 1:
            kw = dict(q_out=q, k_out=k)
        elif mode == 2:
            big = torch.zeros(T, 2 * (H + Hkv) + 1, d, dtype=torch.bfloat16, device="cuda")
            kw = dict(q_out=big[:, 1:2 * H + 1:2], k_out=big[:, 2 * H + 1:2 * H + 1 + Hkv])
        qo, ko = fa.append_paged(q, k, v, *cache.gpu, cuda(table), cuda([T], torch.int32), turns=turns, **cache.kw(), **kw)
        got.append([qo.contiguous(), ko.contiguous(), cache.gpu[0].view(torch.uint8), cache.gpu[1].view(torch.uint8),
                    *cache.scale])
        assert torch.equal(x[:, H + Hkv:], qkv[:, H + Hkv:])
    assert fa.device_status() == fa.FA_OK
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("ragged", [False, True])
def test_padded_batch(fa, ragged):
    """Sequences of length 0 are padding: their tokens are left alone, their table rows not read, and decode gives their
    rows zeros; the others' results are those of the batch without them."""
    rng = np.random.default_rng(14)
    H, Hkv, d, page = 4, 2, 64, 16
    lens, new = [0, 20, 0, 5, 0], [2, 2, 2, 2, 2]
    table = np.full((5, 2), 99, dtype=np.int32)
    table[1], table[3, 0] = [2, 0], 4
    cache = Cache(rng, 5, Hkv, page, d, True)
    before = [c.view(torch.uint8).clone() for c in cache.gpu] + [s.clone() for s in cache.scale]
    x = torch.randn(10, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    split = lambda y: (y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:])   # noqa: E731
    turns = fa.rotary_turns(d)
    cu = cuda(np.arange(0, 11, 2), torch.int32) if ragged else None
    qo, ko = torch.full((10, H, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((10, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.append_paged(*split(x), *cache.gpu, cuda(table), cuda(lens, torch.int32), cu_seqlens=cu, turns=turns, q_out=qo, k_out=ko,
                    **cache.kw())
    o, lse = fa.decode_paged(qo.view(5, 2, H, d).transpose(1, 2), *cache.gpu, cuda(table), cuda(lens, torch.int32), **cache.kw())
    assert fa.device_status() == fa.FA_OK
    pad = [0, 1, 4, 5, 8, 9]
    assert (qo[pad] == 7).all() and (ko[pad] == 7).all()
    assert (o[[0, 2, 4]] == 0).all() and torch.isneginf(lse[[0, 2, 4]]).all()
    after = [c.view(torch.uint8).clone() for c in cache.gpu] + [s.clone() for s in cache.scale]
    for t, b in zip([*cache.gpu, *cache.scale], before):
        t.view(b.dtype).copy_(b)
    live = [2, 3, 6, 7]
    q2, k2 = fa.append_paged(*split(x[live]), *cache.gpu, cuda(table[[1, 3]]), cuda([20, 5], torch.int32), turns=turns, **cache.kw())
    o2, l2 = fa.decode_paged(q2.view(2, 2, H, d).transpose(1, 2), *cache.gpu, cuda(table[[1, 3]]), cuda([20, 5], torch.int32), **cache.kw())
    assert fa.device_status() == fa.FA_OK
    assert torch.equal(q2, qo[live]) and torch.equal(k2, ko[live])
    assert all(torch.equal(a, b.view(a.dtype)) for a, b in zip(after, [*cache.gpu, *cache.scale]))
    # other ranges of tiles, so other roundings: each within the tolerance of the exact result
    assert (o2 - o[[1, 3]]).abs().max() <= 2e-2 and (l2 - lse[[1, 3]]).abs().max() <= 2e-3


def test_tokens_before_the_first_sequence(fa):
    """Offsets that do not start at 0: the tokens before the first sequence are nobody's. Sequences that begin inside a
    page whose scale was never set keep to their own rows, and the page before it is not touched."""
    H, Hkv, d, page, skip = 2, 1, 64, 16, 100
    rng = np.random.default_rng(15)
    new, lens = [20, 3], [41, 40]
    cu = [skip, skip + 20, skip + 23]
    table = np.array([[3, 1, 4], [5, 0, 2]], dtype=np.int32)
    cache = Cache(rng, 6, Hkv, page, d, True)
    for s in cache.scale:
        s.fill_(float("nan"))
    codes, sc = cache.codes(1), cache.scales(1)
    x = torch.randn(150, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    qo = torch.full((150, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.append_paged(x[:, :H], x[:, H:H + 1], x[:, H + 1:], *cache.gpu, cuda(table), cuda(lens, torch.int32),
                    cu_seqlens=cuda(cu, torch.int32), max_new=20, q_out=qo, **cache.kw())
    # without max_new as well: the blocks are then found through the offsets
    qo2 = torch.full((150, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.append_paged(x[:, :H], x[:, H:H + 1], x[:, H + 1:], *cache.gpu, cuda(table), cuda(lens, torch.int32),
                    cu_seqlens=cuda(cu, torch.int32), q_out=qo2, **cache.kw())
    assert fa.device_status() == fa.FA_OK
    live = slice(skip, skip + 23)
    assert torch.equal(qo, qo2) and torch.equal(qo[live], x[live, :H])
    assert (qo[:skip] == 7).all() and (qo[skip + 23:] == 7).all()
    with np.errstate(invalid="ignore"):
        sc = np.where(np.isnan(sc), 0.0, sc)            # no scale yet: any new one replaces it, held codes stay
        ref = codes.copy()
        OP.store_e4m3(to64(x[live, H + 1:]), new, lens, table, page, codes, sc)
    got = cache.codes(1)
    fresh = np.zeros(codes.shape, dtype=bool)
    for b, (n, L) in enumerate(zip(new, lens)):
        for p in range(L - n, L):
            fresh[table[b][p // page], :, p % page] = True
    assert np.array_equal(got[fresh], codes[fresh]) and np.array_equal(got[~fresh], ref[~fresh])
    untouched = [3, 5, 0]                               # pages before the sequences' first new rows
    assert np.isnan(to64(cache.scale[1])[untouched]).all()


def test_append_scale_growth_and_odd_values(fa):
    """Token by token into one e4m3 page: the scale follows the largest value so far; infinities and NaN become the NaN
    code and leave the scale alone; an all-zero page has the least scale; a page that starts over forgets its old one."""
    d, page = 64, 16
    rng = np.random.default_rng(4)
    mags = [0.0, 1e-3, 1e-3, 2.0, 0.5, 700.0, 1e-9, 3e4, 1.0]
    rows = np.array([rng.uniform(-1, 1, (1, d)) * m for m in mags])
    rows[4, 0, 3], rows[4, 0, 7] = np.inf, np.nan
    x = cuda(rows, torch.bfloat16)
    ref = to64(x)
    pages = [torch.full((3, 1, page, d), 0x40, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.full((3, 1), float("nan"), device="cuda") for _ in range(2)]
    codes, sc = np.full((3, 1, page, d), 0x40, dtype=np.uint8), np.full((3, 1), np.nan)
    for i in range(len(mags)):
        t = x[i:i + 1]
        fa.append_paged(t, t, t, *pages, cuda([[1]], torch.int32), cuda([i + 1], torch.int32), k_scale=scale[0],
                        v_scale=scale[1])
        OP.store_e4m3(ref[i:i + 1], [1], [i + 1], [[1]], page, codes, sc)
        for p, s in zip(pages, scale):
            assert np.array_equal(p.cpu().numpy(), codes), i
            assert to64(s)[1, 0] == sc[1, 0] and np.isnan(to64(s)[[0, 2]]).all()
    assert sc[1, 0] == 2.0 ** OP.scale_exponent(float(np.abs(ref[7]).max())) and (codes[1, 0, 4] == 0x7F).sum() == 2
    assert fa.device_status() == fa.FA_OK


DECODE = [
    # B, H, Hkv, Nq, page, lens, splits
    dict(H=4, Hkv=4, Nq=1, page=16, lens=[300, 1], splits=1),
    dict(H=8, Hkv=2, Nq=1, page=16, lens=[1000, 517, 0], splits=3),      # ends inside a page; an empty sequence
    dict(H=8, Hkv=1, Nq=2, page=64, lens=[0, 1, 700], splits=2),         # a token that sees nothing
    dict(H=16, Hkv=4, Nq=4, page=32, lens=[129, 1999], splits=0),
    dict(H=32, Hkv=2, Nq=8, page=128, lens=[640, 9], splits=2),          # 128 rows a K/V head
    dict(H=6, Hkv=3, Nq=5, page=16, lens=[257, 5, 4], splits=7),
    dict(H=7, Hkv=1, Nq=1, page=64, lens=[64, 63, 65], splits=1),        # G = 7: a padded row
    dict(H=9, Hkv=1, Nq=1, page=64, lens=[128, 127, 129, 4000], splits=0),  # 9 rows: two 8-row tiles
    dict(H=17, Hkv=1, Nq=1, page=32, lens=[300], splits=2),              # a second row tile of one row
    dict(H=2, Hkv=2, Nq=3, page=128, lens=[2, 3, 900], splits=1024),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "h{}kv{}nq{}p{}l{}s{}".format(
    c["H"], c["Hkv"], c["Nq"], c["page"], "-".join(map(str, c["lens"])), c["splits"]))
def test_decode(fa, case, f8, d):
    H, Hkv, Nq, page, lens, splits = (case[k] for k in ("H", "Hkv", "Nq", "page", "lens", "splits"))
    rng = np.random.default_rng(H * 100 + d + f8)
    B = len(lens)
    count = [(L + page - 1) // page for L in lens]
    table, pool = make_table(rng, B, count, max(count) + 2)
    cache = Cache(rng, pool, Hkv, page, d, f8)
    # rows past each sequence's end hold NaN: they are never read into a result
    for b, L in enumerate(lens):
        if L % page:
            for g in cache.gpu:
                g.view(torch.uint8 if f8 else torch.int16)[int(table[b, L // page]), :, L % page:] = 0x7F if f8 else 0x7FFF
    q = torch.randn(B, Nq, H, d, generator=torch.Generator().manual_seed(H)).to(torch.bfloat16).cuda().transpose(1, 2)
    o, lse = fa.decode_paged(q, *cache.gpu, cuda(table), cuda(lens, torch.int32), num_splits=splits, **cache.kw())
    assert fa.device_status() == fa.FA_OK
    ro, rl = OP.attend(to64(q), cache.values(0), cache.values(1), table, lens, 1 / math.sqrt(d))
    compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1), f"{case} f8={f8} d={d}")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_decode_negative_zero_and_large_scores(fa, f8):
    """A negative scale, scale 0 (uniform weights), and rows whose scores sit near +-1e3."""
    rng = np.random.default_rng(8)
    B, H, Hkv, Nq, page, d, lens = 2, 8, 2, 1, 32, 128, [500, 333]
    count = [(L + page - 1) // page for L in lens]
    table, pool = make_table(rng, B, count, max(count))
    cache = Cache(rng, pool, Hkv, page, d, f8)
    q = torch.randn(B, H, Nq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    for scale, mul in ((-0.1, 1.0), (0.0, 1.0), (1 / math.sqrt(d), 200.0), (1 / math.sqrt(d), 2.0 ** -120)):
        x = (q.float() * mul).to(torch.bfloat16)
        o, lse = fa.decode_paged(x, *cache.gpu, cuda(table), cuda(lens, torch.int32), scale=scale, **cache.kw())
        assert fa.device_status() == fa.FA_OK
        ro, rl = OP.attend(to64(x), cache.values(0), cache.values(1), table, lens, scale)
        # fp32 scores near 1e3 are exact to 2^-24 of their size: their weights to 1e3 * 2^-22, and lse likewise
        d_o, d_l = np.abs(to64(o) - ro), np.abs(to64(lse) - rl)
        assert d_o.max() <= 1e-2 + 2.0 ** -8 * np.abs(ro).max() and d_l.max() <= 1e-3 + 2.0 ** -22 * np.abs(rl).max()


def test_decode_scales_far_apart(fa):
    """e4m3 pages whose value scales span 2^36: the products run on the codes, so rows that attend to a page of small
    values are as exact as rows that attend to a large one. The query picks a page through one key component."""
    B, H, Hkv, page, d, P = 1, 8, 1, 16, 64, 6
    rng = np.random.default_rng(12)
    codes = [torch.randn(P, 1, page, d, generator=torch.Generator().manual_seed(s)).mul(64).clamp(-400, 400).to(torch.float8_e4m3fn)
             for s in (1, 2)]
    kv = codes[0].float()
    kv[:, :, :, :P] = 0
    for i in range(P):
        kv[i, :, :, i] = 256
    codes[0] = kv.to(torch.float8_e4m3fn)
    ks = torch.full((P, 1), 2.0 ** -8)
    vs = torch.exp2(torch.tensor([-26.0, 10.0, -3.0, -26.0, 4.0, -12.0]))[:, None]
    q = torch.zeros(B, H, 1, d)
    for h in range(H):
        q[0, h, 0, :P] = 0.0
        q[0, h, 0, h % P] = 3.0e2     # exp(-300 / 8) of the weight elsewhere
        q[0, h, 0, P:] = torch.from_numpy(rng.standard_normal(d - P)).float()
    q = q.to(torch.bfloat16)
    table = np.arange(P)[None]
    o, lse = fa.decode_paged(q.cuda(), codes[0].cuda(), codes[1].cuda(), cuda(table, torch.int32),
                             cuda([P * page], torch.int32), k_scale=ks.cuda(), v_scale=vs.cuda())
    assert fa.device_status() == fa.FA_OK
    vals = [FP8.e4m3_decode(c.view(torch.uint8).numpy()) * to64(s)[:, :, None, None] for c, s in zip(codes, (ks, vs))]
    ro, rl = OP.attend(to64(q), *vals, table, [P * page], 1 / math.sqrt(d))
    # per row: half a bf16 step of the value, and fp32/f16 weight errors (2^-11) of the row's largest
    bound = 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * np.abs(ro).max(axis=-1, keepdims=True)
    assert np.all(np.abs(to64(o) - ro) <= bound)
    assert np.abs(to64(lse) - rl).max() <= 1e-3


def test_decode_arbitrary_positive_scales_and_shared_pages(fa):
    """Scales that are no powers of two, and two sequences that share their first pages."""
    page, d, H, Hkv, lens = 16, 128, 8, 2, [77, 90]
    rng = np.random.default_rng(21)
    cache = Cache(rng, 12, Hkv, page, d, True)
    for i in range(2):
        cache.scale[i] = (torch.rand(12, Hkv, generator=torch.Generator().manual_seed(i)) * 0.01 + 0.002).cuda()
    table = np.array([[3, 5, 7, 1, 0, 2], [3, 5, 7, 9, 11, 10]], dtype=np.int32)
    q = torch.randn(2, H, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    o, lse = fa.decode_paged(q, *cache.gpu, cuda(table), cuda(lens, torch.int32), **cache.kw())
    assert fa.device_status() == fa.FA_OK
    ro, rl = OP.attend(to64(q), cache.values(0), cache.values(1), table, lens, 1 / math.sqrt(d))
    compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))


def test_bad_pages_and_lengths_are_reported(fa):
    """A table entry outside the pool hides its keys (decode) or is not written (append); lengths outside the cache are
    clipped. Nothing else changes, and the status names it once. (The lookup itself is tested on the host.)"""
    page, d, H, Hkv = 16, 64, 4, 2
    rng = np.random.default_rng(30)
    for f8 in (False, True):
        cache = Cache(rng, 6, Hkv, page, d, f8)
        q = torch.randn(1, H, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        good = [0, 2, 3]
        for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
            t = cuda([[0, bad, 2, 3]], torch.int32)
            o, lse = fa.decode_paged(q, *cache.gpu, t, cuda([4 * page], torch.int32), **cache.kw())
            assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
            ro, rl = OP.attend(to64(q), cache.values(0), cache.values(1), [good], [3 * page], 1 / math.sqrt(d))
            compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))
            x = torch.randn(2, Hkv, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
            before = [c.view(torch.uint8).clone() for c in cache.gpu]
            qo, ko = fa.append_paged(x, x, x, *cache.gpu, t, cuda([page + 2], torch.int32), **cache.kw())
            assert fa.device_status() == fa.FA_ERR_INVALID_ARG
            assert torch.equal(qo, x) and torch.equal(ko, x)
            assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, cache.gpu))
        t = cuda([[0, 2, 3]], torch.int32)
        for L, seen in ((1000, 48), (-3, 0)):
            o, lse = fa.decode_paged(q, *cache.gpu, t, cuda([L], torch.int32), **cache.kw())
            assert fa.device_status() == fa.FA_ERR_INVALID_ARG
            ro, rl = OP.attend(to64(q), cache.values(0), cache.values(1), [good], [seen], 1 / math.sqrt(d))
            compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))
        # appends past the cache, before position 0, with offsets outside T and with more tokens than max_new
        x = torch.randn(4, Hkv, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
        for L, cu, mx in ((49, None, 0), (2, None, 0), (8, [0, 9], 0), (8, [-1, 3], 0), (8, [3, 1], 0), (8, [0, 4], 2)):
            kw = {} if cu is None else dict(cu_seqlens=cuda(cu, torch.int32), max_new=mx)
            fa.append_paged(x, x, x, *cache.gpu, t, cuda([L], torch.int32), **kw, **cache.kw())
            assert fa.device_status() == fa.FA_ERR_INVALID_ARG, (L, cu)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_offsets_past_32_bits(fa, f8):
    """A pool of more than 2^32 bytes a tensor (2^31 elements in bf16): the pages at its far end."""
    page, d, Hkv, H, L = 128, 128, 8, 8, 200
    n = (1 << 15 if f8 else 1 << 14) + 3 + (1 << 10)
    assert n * Hkv * page * d * (1 if f8 else 2) > 1 << 32
    pages = [torch.zeros(n, Hkv, page, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16, device="cuda") for _ in range(2)]
    scale = [torch.ones(n, Hkv, device="cuda") if f8 else None for _ in range(2)]
    table = cuda([[n - 1, n - 2]], torch.int32)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(L, 3 * H, d, generator=g).to(torch.bfloat16).cuda()
    turns = fa.rotary_turns(d, BASE)
    q, k = fa.append_paged(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], *pages, table, cuda([L], torch.int32), turns=turns,
                           k_scale=scale[0], v_scale=scale[1])
    o, lse = fa.decode_paged(q[-1:].view(1, 1, H, d).transpose(1, 2), *pages, table, cuda([L], torch.int32),
                             k_scale=scale[0], v_scale=scale[1])
    assert fa.device_status() == fa.FA_OK
    small = []
    for p, s in zip(pages, scale):
        c = p[-2:].flip(0) if not f8 else p[-2:].view(torch.uint8).flip(0)
        small.append(to64(c) if not f8 else FP8.e4m3_decode(c.cpu().numpy()) * to64(s[-2:].flip(0))[:, :, None, None])
    assert not pages[0][:-2].view(torch.uint8).any()
    ro, rl = OP.attend(to64(q[-1:]).reshape(1, 1, H, d).transpose(0, 2, 1, 3), *small, [[0, 1]], [L], 1 / math.sqrt(d))
    compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))
    if not f8:
        assert torch.equal(pages[1][n - 1].transpose(0, 1).contiguous(), x[:128, 2 * H:].contiguous())


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_steps_and_graph_replay(fa, f8):
    """A prompt and decode steps as a serving loop runs them, against attention over the turned keys of the whole
    sequence; then the step captured once, on another stream, and replayed with new inputs and lengths."""
    H, Hkv, d, page, B = 8, 2, 128, 16, 2
    rng = np.random.default_rng(40)
    prompt = [21, 40]
    width = 6
    table, pool = make_table(rng, B, [width, width], width)
    cache = Cache(rng, pool, Hkv, page, d, f8)
    dt = cuda(table)
    turns = fa.rotary_turns(d, BASE)
    g = torch.Generator().manual_seed(1)
    draw = lambda T: torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()   # noqa: E731
    split = lambda x: (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:])                            # noqa: E731
    lens = cuda(prompt, torch.int32)
    x = draw(sum(prompt))
    fa.append_paged(*split(x), *cache.gpu, dt, lens, cu_seqlens=cuda([0, 21, 61], torch.int32), turns=turns, **cache.kw())
    side = torch.cuda.Stream()
    static = draw(B)
    qo = torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda")
    o = torch.empty(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H, 1, device="cuda")
    ws = torch.empty(fa.decode_paged_workspace_size(B, H, Hkv, 1, d, width * page, 3), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        fa.append_paged(*split(static), *cache.gpu, dt, lens, turns=turns, q_out=qo, with_k=False, **cache.kw())
        fa.decode_paged(qo.view(B, 1, H, d).transpose(1, 2), *cache.gpu, dt, lens, num_splits=3, workspace=ws, out=o,
                        lse=lse, **cache.kw())

    def check(what):
        assert fa.device_status() == fa.FA_OK
        ro, rl = OP.attend(to64(qo)[:, :, None], cache.values(0), cache.values(1), table, lens.tolist(), 1 / math.sqrt(d))
        compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1), what)

    for i in range(3):
        static.copy_(draw(B))
        step()
        check(f"step {i}")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        static.copy_(draw(B))
        graph.replay()
        torch.cuda.synchronize()
        check(f"replay {i}")
    assert lens.tolist() == [28, 47]


def test_decode_deterministic_on_another_stream(fa):
    """Two calls on the same inputs, one of them on a stream that is not current, give the same bytes."""
    rng = np.random.default_rng(50)
    lens, page, d = [900, 333], 64, 128
    table, pool = make_table(rng, 2, [15, 6], 15)
    cache = Cache(rng, pool, 2, page, d, True)
    q = torch.randn(2, 8, 2, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    a = fa.decode_paged(q, *cache.gpu, cuda(table), cuda(lens, torch.int32), num_splits=4, **cache.kw())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    dt, dl = cuda(table), cuda(lens, torch.int32)
    torch.cuda.synchronize()
    b = fa.decode_paged(q, *cache.gpu, dt, dl, num_splits=4, stream=s, **cache.kw())
    s.synchronize()
    assert fa.device_status() == fa.FA_OK
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refusals(fa):
    """What the binding turns down before the library is called."""
    page, d, H, Hkv = 16, 64, 4, 2
    cache = Cache(np.random.default_rng(1), 4, Hkv, page, d, True)
    plain = Cache(np.random.default_rng(1), 4, Hkv, page, d, False)
    t, L = cuda([[0, 1]], torch.int32), cuda([5], torch.int32)
    q = torch.zeros(1, H, 1, d, dtype=torch.bfloat16, device="cuda")
    dec = lambda **kw: fa.decode_paged(**{**dict(q=q, k_pages=cache.gpu[0], v_pages=cache.gpu[1], block_table=t,  # noqa: E731
                                                 seqlens_k=L, **cache.kw()), **kw})
    dec()
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., ::2]), dict(k_scale=None), dict(seqlens_k=L.long()),
                dict(seqlens_k=cuda([5, 5], torch.int32)), dict(block_table=t.cpu()), dict(max_len=33), dict(max_len=-1),
                dict(v_pages=plain.gpu[1]), dict(k_pages=plain.gpu[0], v_pages=plain.gpu[1]),
                dict(k_pages=cache.gpu[0][:, :1], v_pages=cache.gpu[1][:, :1]), dict(out=q[:, :2]),
                dict(lse=torch.zeros(4, device="cuda")), dict(k_scale=cache.scale[0][:, :1])):
        with pytest.raises(ValueError):
            dec(**bad)
    with pytest.raises(fa.FAError):
        dec(num_splits=2000)
    x = torch.zeros(1, Hkv, d, dtype=torch.bfloat16, device="cuda")
    app = lambda **kw: fa.append_paged(**{**dict(q=q[:, :, 0], k=x, v=x, k_pages=cache.gpu[0], v_pages=cache.gpu[1],  # noqa: E731
                                                 block_table=t, seqlens_k=L, **cache.kw()), **kw})
    app()
    for bad in (dict(q=q), dict(k=x.float()), dict(v=x[:, :1]), dict(cu_seqlens=L), dict(turns=L), dict(k_scale=None),
                dict(q_weight=x[0, 0].float()), dict(k_weight=x[0, 0, :32]), dict(q_out=x), dict(k_out=q[:, :, 0])):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(fa.FAError):
        app(turns=torch.zeros(4, dtype=torch.int64, device="cuda"))   # rot = 8
    assert fa.device_status() == fa.FA_OK


def _attend_bound(q, vals, table, lens, scale, ro):
    """How far a decode over e4m3 pages may be from the exact ``ro``: half a bf16 step of the output, and of each
    term p_j |v_j| half an f16 step of its weight (2^-11), as much again for the rounding of the sum it is divided by,
    of the fp32 score in its exponent and of the fp32 sums."""
    spread, _ = OP.attend(q, vals[0], np.abs(vals[1]), table, lens, scale)
    return 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * spread


# exponent by which one page's value scale lies above the others', and by how many nats its only visible key leads
@pytest.mark.parametrize("span,lead", [(12, 8.0), (16, 6.0), (16, 6.5), (20, 3.5), (7, 9.0), (8, 9.0), (60, 3.0)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("d,H,Nq", [(64, 4, 1), (64, 4, 3), (128, 4, 1), (128, 7, 2)])
def test_decode_small_values_beside_a_large_page(fa, d, H, Nq, where, span, lead):
    """The mass lies on pages of small values, and a page of a far larger scale, whose keys' codes are zero, has the
    largest score: its scale must not cost the other pages' weights their bits."""
    page, L = 16, 2000
    P = L // page
    rng = np.random.default_rng(span * 100 + d)
    big = {"first": 0, "middle": P // 2, "last": P - 1}[where]
    kv = rng.standard_normal((P, 1, page, d)) * 16
    kv[..., 0] = 0.0
    kv[big, 0, :, 0] = -256.0                       # the page's other keys are far below
    kv[big, 0, 0, 0] = 256.0
    vv = rng.standard_normal((P, 1, page, d)) * 64
    vv[big] = 0.0
    table = rng.permutation(P)[None]
    at = np.argsort(table[0])                       # the position of each page of the pool
    kc, vc = (torch.from_numpy(np.clip(x[at], -400, 400)).float().to(torch.float8_e4m3fn) for x in (kv, vv))
    ks, vs = torch.full((P, 1), 2.0 ** -4), torch.full((P, 1), 2.0 ** -6)
    vs[table[0, big]] = 2.0 ** (span - 6)
    scale = 1 / math.sqrt(d)
    q = torch.from_numpy(rng.standard_normal((1, H, Nq, d)) * 0.1)
    q[..., 0] = lead / (256 * 2.0 ** -4 * scale)
    q = q.to(torch.bfloat16)
    vals = [FP8.e4m3_decode(c.view(torch.uint8).numpy()) * to64(s)[:, :, None, None] for c, s in ((kc, ks), (vc, vs))]
    ro, rl = OP.attend(to64(q), *vals, table, [L], scale)
    bound = _attend_bound(to64(q), vals, table, [L], scale, ro)
    for splits in (1, 0):
        o, lse = fa.decode_paged(q.cuda(), kc.cuda(), vc.cuda(), cuda(table, torch.int32), cuda([L], torch.int32),
                                 k_scale=ks.cuda(), v_scale=vs.cuda(), scale=scale, num_splits=splits)
        assert fa.device_status() == fa.FA_OK
        off = np.abs(to64(o) - ro) - bound
        assert off.max() <= 0, f"splits {splits}: {off.max():.3e} past the bound, outputs up to {np.abs(ro).max():.3e}"
        assert np.abs(to64(lse) - rl).max() <= 1e-3


@pytest.mark.parametrize("d,H,Nq", [(64, 8, 1), (64, 8, 2), (128, 8, 1), (128, 8, 2)])
def test_decode_value_scales_of_every_size(fa, d, H, Nq):
    """Pages whose value scales lie anywhere in 2^-40 .. 2^20, in any order; the larger ones hold zeros but for one
    element, so every other element comes from the small pages alone."""
    page, L = 32, 1500
    P = (L + page - 1) // page
    rng = np.random.default_rng(d + Nq)
    e = rng.integers(-40, 21, P)
    e[3] = 20
    kv = rng.standard_normal((P, 1, page, d)) * 32
    vv = rng.standard_normal((P, 1, page, d)) * 64
    vv[e > -34, :, :, 1:] = 0.0
    kc, vc = (torch.from_numpy(np.clip(x, -400, 400)).float().to(torch.float8_e4m3fn) for x in (kv, vv))
    ks, vs = torch.full((P, 1), 2.0 ** -5), torch.exp2(torch.from_numpy(e).float())[:, None]
    scale = 1 / math.sqrt(d)
    q = torch.from_numpy(rng.standard_normal((1, H, Nq, d))).to(torch.bfloat16)
    table = np.arange(P)[None]
    vals = [FP8.e4m3_decode(c.view(torch.uint8).numpy()) * to64(s)[:, :, None, None] for c, s in ((kc, ks), (vc, vs))]
    ro, rl = OP.attend(to64(q), *vals, table, [L], scale)
    bound = _attend_bound(to64(q), vals, table, [L], scale, ro)
    for splits in (1, 5, 0):
        o, lse = fa.decode_paged(q.cuda(), kc.cuda(), vc.cuda(), cuda(table, torch.int32), cuda([L], torch.int32),
                                 k_scale=ks.cuda(), v_scale=vs.cuda(), scale=scale, num_splits=splits)
        assert fa.device_status() == fa.FA_OK
        bad = np.abs(to64(o) - ro) > bound
        assert not bad.any(), f"splits {splits}: {bad.sum()} of {bad.size} past the bound"
        assert np.abs(to64(lse) - rl).max() <= 1e-3


def test_decode_hidden_page_beside_large_scales(fa):
    """A table entry outside the pool hides its keys also where the other pages' scales lie far above 1."""
    page, d, H, Hkv = 16, 128, 8, 2
    cache = Cache(np.random.default_rng(31), 6, Hkv, page, d, True)
    for s in cache.scale:
        s.mul_(2.0 ** 20)
    cache.scale[0].mul_(2.0 ** -20)
    q = torch.randn(1, H, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    o, lse = fa.decode_paged(q, *cache.gpu, cuda([[0, -1, 2, 3]], torch.int32), cuda([4 * page], torch.int32), **cache.kw())
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
    vals = cache.values(0), cache.values(1)
    ro, rl = OP.attend(to64(q), *vals, [[0, 2, 3]], [3 * page], 1 / math.sqrt(d))
    assert np.all(np.abs(to64(o) - ro) <= _attend_bound(to64(q), vals, [[0, 2, 3]], [3 * page], 1 / math.sqrt(d), ro))
    assert np.abs(to64(lse) - rl).max() <= 1e-3


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("cu,T,max_new,lens", [
    ([0, 4], 4, 2, [8]),                     # more than max_new
    ([0, 9], 4, 0, [20]),                    # more than there are
    ([0, 4, 40], 40, 20, [21, 47]),          # both pages of a clipped sequence
    ([0, 50, 120], 100, 0, [50, 130]),       # blocks found through the offsets
    ([0, 2 ** 31 - 1], 4, 0, [2 ** 31 - 1]),
    ([0, 2 ** 31 - 1], 4, 0, [-2 ** 31]),    # nothing of it has a place
])
def test_append_clipped_tokens_keep_their_positions(fa, cu, T, max_new, lens, f8):
    """A sequence with more new tokens than the call covers is reported; the tokens that the call does cover go to the
    positions that its length and its offsets give them, and nothing else is written."""
    H, Hkv, page, d, width = 4, 2, 16, 64, 9
    rng = np.random.default_rng(6)
    B = len(lens)
    table, pool = make_table(rng, B, [width] * B, width)
    cache = Cache(rng, pool, Hkv, page, d, f8)
    before = [cache.codes(i) if f8 else cache.values(i) for i in range(2)]
    scales = [cache.scales(i).copy() if f8 else None for i in range(2)]
    x = torch.randn(T, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    qo = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    turns = fa.rotary_turns(d, BASE)
    fa.append_paged(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], *cache.gpu, cuda(table), cuda(lens, torch.int32),
                    cu_seqlens=cuda(cu, torch.int32), max_new=max_new, turns=turns, q_out=qo, k_out=ko, **cache.kw())
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
    most = max_new if max_new else T
    covered = np.zeros(T, dtype=bool)
    want = [b.copy() for b in before]
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        m = min(n, most, T - cu[b])
        t = np.arange(cu[b], cu[b] + m)
        start = L - n
        placed = start >= 0 and start + m <= width * page
        if not placed:                       # (none of these cases places a part of a sequence)
            assert start < -m or start > width * page
            covered[t] = True                # turned all the same, by positions outside the cache
            continue
        covered[t] = True
        rq, rk, pos = OP.append(to64(x[t, :H]), to64(x[t, H:H + Hkv]), None, [m], [start + m], turns.tolist(), False)
        near_bf16(to64(qo)[t], rq, f"q {b}")
        near_bf16(to64(ko)[t], rk, f"k {b}")
        v = to64(x[t, H + Hkv:])
        if f8:
            OP.store_e4m3(v, [m], [start + m], table[b:b + 1], page, want[1], scales[1])
        else:
            for i, p in enumerate(pos):
                want[1][table[b, p // page], :, p % page] = v[i]
    assert (to64(qo)[~covered] == 7).all() and (to64(ko)[~covered] == 7).all()
    if f8:
        assert np.array_equal(cache.codes(1), want[1]) and np.array_equal(cache.scales(1), scales[1])
    else:
        assert np.array_equal(cache.values(1), want[1])


def test_append_to_a_page_of_tiny_scale(fa):
    """A page whose scale lies below every scale that append writes: zeros stay zeros, and the scale becomes one that
    append writes."""
    page, d = 16, 64
    pages = [torch.zeros(1, 1, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for p in pages:
        p[0, 0, 0, :5] = 0x40
    scale = [torch.full((1, 1), 2.0 ** -140, device="cuda") for _ in range(2)]
    x = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    fa.append_paged(x, x, x, *pages, cuda([[0]], torch.int32), cuda([2], torch.int32), k_scale=scale[0], v_scale=scale[1])
    assert fa.device_status() == fa.FA_OK
    for p, s in zip(pages, scale):
        assert (p == 0).all() and (s == 2.0 ** -40).all()   # (2 * 2^-140 is below half of the least code)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_rows_that_see_nothing_beside_nan(fa, d, f8):
    """A token before the sequence's first key gets zeros and -inf, whatever v holds; the tokens that see the keys get
    what v holds."""
    page, H, Hkv, Nq, lens = 16, 4, 2, 5, [3, 2]
    cache = Cache(np.random.default_rng(2), 3, Hkv, page, d, f8)
    cache.gpu[1].view(torch.uint8 if f8 else torch.int16).fill_(0x7F if f8 else 0x7FC0)
    q = torch.randn(2, H, Nq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    for splits in (0, 1, 3):
        o, lse = fa.decode_paged(q, *cache.gpu, cuda([[2], [0]], torch.int32), cuda(lens, torch.int32), num_splits=splits,
                                 **cache.kw())
        assert fa.device_status() == fa.FA_OK
        for b, L in enumerate(lens):
            assert (o[b, :, :Nq - L] == 0).all() and torch.isneginf(lse[b, :, :Nq - L]).all()
            assert torch.isnan(o[b, :, Nq - L:]).all() and torch.isfinite(lse[b, :, Nq - L:]).all()


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("inter,norm,rot_scale", [(True, True, 1.0), (False, False, 1.0), (False, True, 1.3688879454),
                                                 (True, True, 0.25), (True, False, -2.5), (False, True, 0.0)])
@pytest.mark.parametrize("d,rot", [(64, 48), (128, 128)])
def test_append_rotation_scale_and_weights_in_every_layout(fa, d, rot, inter, norm, rot_scale, f8):
    """A factor on the turned elements (the others keep their size), and norm weights in both layouts."""
    new, lens, H, Hkv, page = [3, 20], [50, 20], 3, 1, 16
    rng = np.random.default_rng(d + 2 * inter + norm)
    T = sum(new)
    count = [(L + page - 1) // page for L in lens]
    table, pool = make_table(rng, 2, count, max(count))
    cache = Cache(rng, pool, Hkv, page, d, f8)
    codes, sc = cache.codes(0) if f8 else None, cache.scales(0).copy() if f8 else None
    x = torch.randn(T, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16).cuda()
    w = [cuda(1 + 0.3 * rng.standard_normal(d), torch.bfloat16) if norm else None for _ in range(2)]
    turns = fa.rotary_turns(rot, BASE)
    q, k = fa.append_paged(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], *cache.gpu, cuda(table), cuda(lens, torch.int32),
                           cu_seqlens=cuda([0, 3, 23], torch.int32), turns=turns, interleaved=inter, rot_scale=rot_scale,
                           q_weight=w[0], k_weight=w[1], eps=1e-5, **cache.kw())
    assert fa.device_status() == fa.FA_OK
    rq, rk, pos = OP.append(to64(x[:, :H]), to64(x[:, H:H + Hkv]), None, new, lens, turns.tolist(), inter,
                            *[None if y is None else to64(y) for y in w], eps=1e-5, rot_scale=float(np.float32(rot_scale)))
    near_bf16(to64(q), rq, "q")
    near_bf16(to64(k), rk, "k")
    seq = np.repeat(np.arange(2), new)
    got = np.stack([cache.values(0)[table[s, p // page], :, p % page] for s, p in zip(seq, pos)])
    if not f8:
        near_bf16(got, rk, "k pages")
        return
    OP.store_e4m3(rk, new, lens, table, page, codes, sc)
    assert np.array_equal(cache.scales(0), sc)
    step = np.stack([sc[table[s, p // page]] for s, p in zip(seq, pos)])[:, :, None]
    assert np.all(np.abs(got - rk) <= np.maximum(2.0 ** -4 * np.abs(rk), 2.0 ** -10 * step) * (1 + 2.0 ** -16))
