"""GPU parity of the 4-bit pages (fa_append_paged_fp4, fa_decode_paged_fp4, fa_read_paged) against the fp64 oracle.

Tolerances. q and k of the append as for bf16 pages (tests/test_paged_gpu.py: half a bf16 step and the fp32
computation). What the pages then hold is a function of bf16 values that are at hand (v, and k as the call returned
it), so it must be exactly the oracle's, but for the sign of a zero. Reading back is exact for bf16 pages, 4-bit rows
and e4m3 pages of power-of-two scales. Attention has the forward pass's tolerances (tests/parity.py).
"""

import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F4
from oracle import fp8 as FP8
from oracle import paged as OP
from parity import compare, to64
from test_paged_gpu import APPEND, BASE, cuda, make_table, near_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


class Cache4:
    """A pool of 4-bit pages with random earlier contents."""

    def __init__(self, rng, n, Hkv, page, d, spread=1.0):
        x = [rng.standard_normal((n, Hkv, page, d)) * np.exp2(rng.integers(-6, 4, (n, Hkv, page, 1)) * spread) for _ in range(2)]
        enc = [F4.encode(torch.from_numpy(y).to(torch.bfloat16).double().numpy()) for y in x]
        self.gpu = [torch.from_numpy(F4.pack(c)).cuda() for c, _ in enc]
        self.scale = [torch.from_numpy(s).cuda() for _, s in enc]

    def bytes(self):
        return [x.cpu().numpy().copy() for x in (*self.gpu, *self.scale)]

    def values(self, i):
        return F4.decode(self.gpu[i].cpu().numpy(), self.scale[i].cpu().numpy())

    @property
    def all(self):
        return (*self.gpu, *self.scale)


@pytest.mark.parametrize("inter,norm", [(False, True), (True, False), (False, False)], ids=["half-norm", "interleaved", "half"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "n{}h{}kv{}p{}d{}r{}".format(
    "-".join(map(str, c["new"])), c["H"], c["Hkv"], c["page"], c["d"], c["rot"]))
def test_append(fa, case, inter, norm):
    new, lens, H, Hkv, page, d, rot = (case[k] for k in ("new", "lens", "H", "Hkv", "page", "d", "rot"))
    rng = np.random.default_rng(sum(lens) * 7 + d + 2 * inter + norm)
    B, T = len(new), sum(new)
    first = [(L - n) // page for n, L in zip(new, lens)]
    count = [(L + page - 1) // page for L in lens]
    used, pool = make_table(rng, B, [c - f for c, f in zip(count, first)], max(c - f for c, f in zip(count, first)) + 1)
    table = np.full((B, max(count)), -1, dtype=np.int32)
    for b in range(B):
        table[b, first[b]:count[b]] = used[b, :count[b] - first[b]]
    cache = Cache4(rng, pool, Hkv, page, d)
    before = cache.bytes()
    held = [cache.values(i) for i in range(2)]
    # parts of one projection, with tokens behind the last sequence that nobody touches; channels of unlike size
    qkv = torch.randn(T + 3, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(T))
    qkv = (qkv * torch.exp2(torch.randint(-5, 5, (d,), generator=torch.Generator().manual_seed(d)))).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    w = [cuda(1 + 0.3 * rng.standard_normal(d), torch.bfloat16) if norm else None for _ in range(2)]
    turns = fa.rotary_turns(rot, BASE) if rot else None
    uniform = len(set(new)) == 1
    cu = None if uniform else cuda(np.concatenate([[0], np.cumsum(new)]), torch.int32)
    if uniform:
        q, k, v = q[:T], k[:T], v[:T]
    offsets = rng.integers(0, 1 << 20, B) if norm else None
    qo = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full(k.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    fa.append_paged_fp4(q, k, v, *cache.all, cuda(table), cuda(lens, torch.int32), cu_seqlens=cu, turns=turns,
                        interleaved=inter, q_weight=w[0], k_weight=w[1], eps=1e-5, q_out=qo, k_out=ko,
                        offsets=None if offsets is None else cuda(offsets, torch.int32))
    assert fa.device_status() == fa.FA_OK
    tl = [] if turns is None else turns.tolist()
    at = lens if offsets is None else [L + int(o) for L, o in zip(lens, offsets)]
    rq, rk, pos = OP.append(to64(q[:T]), to64(k[:T]), to64(v[:T]), new, at, tl, inter,
                            *[None if x is None else to64(x) for x in w], eps=1e-5)
    near_bf16(to64(qo)[:T], rq, "q")
    near_bf16(to64(ko)[:T], rk, "k")
    assert (qo[T:] == 7).all() and (ko[T:] == 7).all()
    seq = np.repeat(np.arange(B), new)
    rows = [p - (0 if offsets is None else int(offsets[b])) for p, b in zip(pos, seq)]
    for i, x in ((0, to64(ko)[:T]), (1, to64(v[:T]))):
        want, fresh, y = held[i], np.zeros(before[i].shape[:3], dtype=bool), F4.held(x)
        for t in range(T):
            place = (table[seq[t], rows[t] // page], slice(None), rows[t] % page)
            want[place], fresh[place] = y[t], True
        assert np.array_equal(cache.values(i), want)
        after = cache.bytes()
        for j in (i, 2 + i):     # every other row's bytes are untouched
            assert np.array_equal(after[j][~fresh], before[j][~fresh])


def test_append_odd_values(fa):
    """Infinities and NaN make their group of 16 NaN and no other; zeros, the least and the largest scales; ties."""
    H, Hkv, d, page, T = 2, 1, 128, 16, 12
    rng = np.random.default_rng(3)
    x = rng.standard_normal((T, Hkv, d))
    x[0, 0, 5], x[1, 0, 127], x[2, 0, 64] = np.inf, np.nan, -np.inf
    x[3] = 0.0
    x[4] *= 2.0 ** -20
    x[5] *= 2.0 ** 14                                        # groups over 61440 saturate
    x[6] = 3e38
    x[7, 0, :16] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 4.0]
    x[8, 0, 16:32] = x[7, 0, :16] * 1.125 * 2.0 ** -9
    x[9] = 2.0 ** -130
    x[10, 0, ::2] = -0.0
    x[11] = np.where(rng.random((Hkv, d)) < 0.5, 2.0 ** -16 * 1.5, -2.0 ** -17)
    x = torch.from_numpy(x).to(torch.bfloat16)
    cache = Cache4(rng, 2, Hkv, page, d)
    q = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    fa.append_paged_fp4(q, x.cuda(), x.flip(-1).cuda(), *cache.all, cuda([[1]], torch.int32), cuda([T], torch.int32))
    assert fa.device_status() == fa.FA_OK
    for i, y in ((0, x), (1, x.flip(-1))):
        want, got = F4.held(y.double().numpy()), cache.values(i)[1, :, :T].transpose(1, 0, 2)
        assert np.array_equal(got, want, equal_nan=True)
        assert np.isnan(got).sum() == 3 * 16


def test_quantisation_of_every_bf16_value(fa):
    """Every finite bf16 magnitude as the largest of its group, and every one below a fixed largest: the bytes of the
    oracle (65,536 groups)."""
    d, page = 128, 128
    bits = torch.arange(0x7f80, dtype=torch.int32)
    big = bits.to(torch.int16).view(torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    a = (big.float()[:, None] * torch.rand(len(big), 16, generator=g)).to(torch.bfloat16)
    a[:, 3] = big
    b = torch.zeros(65536 - len(big), 16)
    b[:, 1:] = torch.randn(len(b), 15, generator=g) * 2
    b[:, 0] = 6.0 * (1 + torch.arange(len(b)) % 8 / 8)
    # exact borders between the codes: 0.25, 0.75, .. 5 scales
    b[:, 1:8] = (b[:, :1] / 6) * torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.cat([a, b.to(torch.bfloat16)]).reshape(-1, 1, d)
    T = x.shape[0]
    n = T // page
    cache = Cache4(np.random.default_rng(0), n, 1, page, d)
    q = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
    fa.append_paged_fp4(q, x.cuda(), x.cuda(), *cache.all, torch.arange(n, dtype=torch.int32, device="cuda")[None],
                        cuda([T], torch.int32))
    assert fa.device_status() == fa.FA_OK
    code, byte = F4.encode(x.double().numpy())
    for i in range(2):
        assert np.array_equal(cache.scale[i].cpu().numpy().reshape(T, 1, -1), byte)
        packed = cache.gpu[i].cpu().numpy().reshape(T, 1, -1)
        assert np.array_equal(F4.decode(packed, byte), F4.decode(F4.pack(code), byte))


# lengths, heads, page, new tokens, splits
DECODE = [
    dict(lens=[1, 16, 17, 0, 64, 65], H=4, Hkv=2, Nq=1, page=16, splits=0),
    dict(lens=[700], H=32, Hkv=8, Nq=1, page=16, splits=0),
    dict(lens=[63, 1000, 2, 333], H=8, Hkv=1, Nq=3, page=32, splits=3),
    dict(lens=[129, 4000], H=20, Hkv=4, Nq=5, page=128, splits=0),
    dict(lens=[5, 3, 500], H=14, Hkv=2, Nq=4, page=64, splits=7),
    dict(lens=[200], H=16, Hkv=1, Nq=8, page=64, splits=1),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "L{}h{}kv{}q{}p{}".format("-".join(map(str, c["lens"])), c["H"], c["Hkv"],
                                                                            c["Nq"], c["page"]))
def test_decode(fa, case, d):
    lens, H, Hkv, Nq, page, splits = (case[k] for k in ("lens", "H", "Hkv", "Nq", "page", "splits"))
    rng = np.random.default_rng(sum(lens) + H + d)
    B, count = len(lens), [(L + page - 1) // page for L in lens]
    table, pool = make_table(rng, B, count, max(count) + 2)
    cache = Cache4(rng, pool, Hkv, page, d, spread=0.3)
    # rows past each sequence's end hold NaN: they are never read into a result
    for b, L in enumerate(lens):
        if L % page:
            for s in cache.scale:
                s[int(table[b, L // page]), :, L % page:] = 0xFF
    q = torch.randn(B, Nq, H, d, generator=torch.Generator().manual_seed(H)).to(torch.bfloat16).cuda().transpose(1, 2)
    o, lse = fa.decode_paged_fp4(q, *cache.all, cuda(table), cuda(lens, torch.int32), num_splits=splits)
    assert fa.device_status() == fa.FA_OK
    kv = [np.nan_to_num(cache.values(i)) for i in range(2)]
    ro, rl = OP.attend(to64(q), *kv, table, lens, 1 / math.sqrt(d))
    # fp16 weights: half a step of each, 2^-11 of the largest value in the row's keys; past what compare allows for |v| near 1
    big = max(1.0, np.abs(kv[1]).max())
    compare(to64(o).reshape(-1, d) / big, to64(lse).reshape(-1), ro.reshape(-1, d) / big, rl.reshape(-1), f"{case} d={d}")


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scales_of_every_size(fa, d):
    """Rows of the least and the largest scales side by side, a negative softmax scale, large scores."""
    rng = np.random.default_rng(5)
    page, H, Hkv, lens = 16, 8, 2, [300, 77]
    table, pool = make_table(rng, 2, [19, 5], 19)
    cache = Cache4(rng, pool, Hkv, page, d)
    cache.scale[1].copy_(torch.from_numpy(rng.integers(1, 227, tuple(cache.scale[1].shape)).astype(np.uint8)))
    q = torch.randn(2, H, 1, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for scale, mul in ((-0.05, 1.0), (0.0, 1.0), (1 / math.sqrt(d), 30.0), (1 / math.sqrt(d), 2.0 ** -120)):
        x = (q.float() * mul).to(torch.bfloat16)
        o, lse = fa.decode_paged_fp4(x, *cache.all, cuda(table), cuda(lens, torch.int32), scale=scale)
        assert fa.device_status() == fa.FA_OK
        kv = [cache.values(i) for i in range(2)]
        ro, rl = OP.attend(to64(x), *kv, table, lens, scale)
        # weights are off by half an f16 step (2^-11, or 2^-25 of the row's largest) and the scores' fp32 error: 2^-20 of
        # the largest; values by nothing; the result by half a bf16 step of itself
        most = max(abs(scale) * np.abs(to64(x)).max() * np.abs(kv[0]).max() * d, 1.0)
        err = 2.0 ** -11 + 2.0 ** -20 * most
        bound = 2.0 ** -8 * np.abs(ro) + 2 * err * np.abs(kv[1]).max()
        assert np.all(np.abs(to64(o) - ro) <= bound) and np.abs(to64(lse) - rl).max() <= 1e-3 + 2.0 ** -20 * most


def test_decode_rows_that_see_nothing_beside_nan(fa):
    """Tokens before a sequence's beginning get zeros, whatever the values hold; NaN reaches the tokens that see a key."""
    rng = np.random.default_rng(9)
    page, d, H, Hkv = 16, 128, 4, 2
    cache = Cache4(rng, 2, Hkv, page, d)
    cache.scale[1][1, :, 0, 3] = 0xFF
    q = torch.randn(1, H, 3, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    o, lse = fa.decode_paged_fp4(q, *cache.all, cuda([[1]], torch.int32), cuda([2], torch.int32))
    assert fa.device_status() == fa.FA_OK
    assert (o[:, :, 0] == 0).all() and torch.isneginf(lse[:, :, 0]).all()
    assert torch.isnan(o[:, :, 1:, 48:64]).all() and torch.isfinite(o[:, :, 1:, :48]).all() and torch.isfinite(lse[:, :, 1:]).all()


def test_decode_bad_pages_and_lengths(fa):
    rng = np.random.default_rng(10)
    page, d, H, Hkv = 16, 64, 4, 2
    cache = Cache4(rng, 6, Hkv, page, d, spread=0.3)
    q = torch.randn(1, H, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    kv = [cache.values(i) for i in range(2)]
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        o, lse = fa.decode_paged_fp4(q, *cache.all, cuda([[0, bad, 2, 3]], torch.int32), cuda([64], torch.int32))
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
        ro, rl = OP.attend(to64(q), *kv, [[0, 2, 3]], [48], 1 / math.sqrt(d))
        compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))
        before = cache.bytes()
        x = torch.randn(1, Hkv, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        fa.append_paged_fp4(q[:, :, 0], x, x, *cache.all, cuda([[bad]], torch.int32), cuda([1], torch.int32))
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        assert all(np.array_equal(a, b) for a, b in zip(before, cache.bytes()))
    o, lse = fa.decode_paged_fp4(q, *cache.all, cuda([[0, 1, 2, 3]], torch.int32), cuda([2 ** 31 - 1], torch.int32))
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG
    ro, rl = OP.attend(to64(q), *kv, [[0, 1, 2, 3]], [64], 1 / math.sqrt(d))
    compare(to64(o).reshape(-1, d), to64(lse).reshape(-1), ro.reshape(-1, d), rl.reshape(-1))


def pool_of(rng, kind, n, Hkv, page, d):
    """(k_pages, v_pages, k_scale, v_scale, values of K, of V) of any kind of pages."""
    if kind == "fp4":
        c = Cache4(rng, n, Hkv, page, d, spread=0.3)
        return (*c.all, c.values(0), c.values(1))
    x = [torch.from_numpy(rng.standard_normal((n, Hkv, page, d))) for _ in range(2)]
    if kind == "bf16":
        x = [y.to(torch.bfloat16) for y in x]
        return (x[0].cuda(), x[1].cuda(), None, None, *(y.double().numpy() for y in x))
    s = [torch.from_numpy(np.exp2(rng.integers(-10, -6, (n, Hkv)))).float() for _ in range(2)]
    x = [(y * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for y in x]
    return (x[0].cuda(), x[1].cuda(), s[0].cuda(), s[1].cuda(),
            *(FP8.e4m3_decode(y.view(torch.uint8).numpy()) * to64(z)[:, :, None, None] for y, z in zip(x, s)))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("d,page,Hkv,lens,rows", [
    (64, 16, 2, [1, 40, 0, 17, 33], [1, 40, 0, 5, 0]), (128, 64, 8, [200, 1, 65], [200, 1, 65]), (128, 16, 1, [50], [1]),
    (64, 128, 3, [129, 700], [2, 699]), (128, 32, 5, [0, 0, 7], [3, 0, 7]),
], ids=str)
def test_read(fa, kind, d, page, Hkv, lens, rows):
    """All rows, the last ones, none; tokens of a sequence of length 0 are padding; strided outputs; rows behind the last."""
    rng = np.random.default_rng(sum(lens) + d)
    B, count = len(lens), [(L + page - 1) // page for L in lens]
    table, n = make_table(rng, B, count, max(count) + 1)
    kp, vp, ks, vs, kv, vv = pool_of(rng, kind, n, Hkv, page, d)
    cu = np.concatenate([[0], np.cumsum(rows)])
    total = int(cu[-1]) + 2
    big = torch.full((total, 2 * Hkv + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = fa.read_paged(kp, vp, cuda(table), cuda(lens, torch.int32), cuda(cu, torch.int32), total, k_scale=ks, v_scale=vs,
                         k_out=big[:, :Hkv], v_out=big[:, Hkv:2 * Hkv])
    assert fa.device_status() == fa.FA_OK
    want = np.full((2, total, Hkv, d), 7.0)
    for b in range(B):
        for i in range(rows[b] if lens[b] else 0):
            r = lens[b] - rows[b] + i
            for x, y in enumerate((kv, vv)):
                want[x, cu[b] + i] = y[table[b, r // page], :, r % page]
    want = torch.from_numpy(want).to(torch.bfloat16)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1]) and (big[:, 2 * Hkv] == 7).all()
    k2, v2 = fa.read_paged(kp, vp, cuda(table), cuda(lens, torch.int32), cuda(cu, torch.int32), int(cu[-1]), k_scale=ks, v_scale=vs)
    live = np.concatenate([np.full(r, L > 0) for r, L in zip(rows, lens)])
    assert k2.is_contiguous() and torch.equal(k2.cpu()[live], want[0, :-2][live]) and torch.equal(v2.cpu()[live], want[1, :-2][live])


def test_read_rows_that_are_not_there(fa):
    """More rows than a sequence holds, pages outside the pool, offsets that decrease or pass the outputs: the other rows
    are read, these are left as they were, and the call is reported."""
    rng = np.random.default_rng(1)
    kp, vp, ks, vs, kv, _ = pool_of(rng, "fp4", 4, 2, 16, 64)
    for table, lens, cu, good in (
            ([[0, 1], [2, 3]], [20, 5], [0, 22, 25], {2 + i: (0 if i < 16 else 1, i % 16) for i in range(20)} | {22 + i: (2, 2 + i) for i in range(3)}),
            ([[0, 9], [2, 3]], [20, 5], [0, 20, 25], {i: (0, i) for i in range(16)} | {20 + i: (2, i) for i in range(5)}),
            ([[0, -7], [2, 3]], [20, 5], [0, 20, 25], {i: (0, i) for i in range(16)} | {20 + i: (2, i) for i in range(5)}),
            ([[0, 1], [2, 3]], [20, 40], [0, 20, 25], {i: (0 if i < 16 else 1, i % 16) for i in range(20)}),
            ([[0, 1], [2, 3]], [20, 5], [-3, 17, 22], {i: (0 if i < 13 else 1, (i + 3) % 16) for i in range(17)} | {17 + i: (2, i) for i in range(5)}),
            ([[0, 1], [2, 3]], [20, 20], [0, 20, 40], {i: (0 if i < 16 else 1, i % 16) for i in range(20)} | {20 + i: (2, i) for i in range(10)})):
        out = [torch.full((30, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        fa.read_paged(kp, vp, cuda(table, torch.int32), cuda(lens, torch.int32), cuda(cu, torch.int32), 30, k_scale=ks, v_scale=vs,
                      k_out=out[0], v_out=out[1])
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        got = to64(out[0])
        for t in range(30):
            if t in good:
                assert np.array_equal(got[t], kv[good[t][0], :, good[t][1]]), (cu, t)
            elif not (lens[1] == 40 and 20 <= t < 25):   # (a length past the table: rows that lie in it are read)
                assert (got[t] == 7).all(), (cu, t)


def test_offsets_past_32_bits(fa):
    """A pool of more than 2^32 bytes of codes: rows far into it are written, read and attended to."""
    d, Hkv, page = 128, 8, 128
    n = (1 << 32) // (Hkv * page * d // 2) + 40
    kp, vp = (torch.zeros(n, Hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n, Hkv, page, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table, L, H = [n - 1, 3, n - 2], 300, 16
    x = torch.randn(L, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    t, lens = cuda([table], torch.int32), cuda([L], torch.int32)
    fa.append_paged_fp4(q, k, v, kp, vp, ks, vs, t, lens)
    kh, vh = fa.read_paged(kp, vp, t, lens, cuda([0, L], torch.int32), L, k_scale=ks, v_scale=vs)
    o, lse = fa.decode_paged_fp4(q[-1:].transpose(0, 1)[None], kp, vp, ks, vs, t, lens)
    assert fa.device_status() == fa.FA_OK
    assert np.array_equal(to64(kh), F4.held(to64(k))) and np.array_equal(to64(vh), F4.held(to64(v)))
    assert not kp[:3].any() and not kp[4:n - 3].any()
    from oracle import attention as A
    for h in range(H):
        ro, rl = A.attend_head(to64(q[-1:, h]), to64(kh[:, h // 2]), to64(vh[:, h // 2]), 1 / math.sqrt(d))
        compare(to64(o[0, h]), to64(lse[0, h]), ro, rl)


def test_binding_refusals(fa):
    rng = np.random.default_rng(4)
    c = Cache4(rng, 4, 2, 16, 64)
    kp, vp, ks, vs = c.all
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, lens = cuda([[0, 1], [2, 3]], torch.int32), cuda([3, 4], torch.int32)
    app = lambda **kw: fa.append_paged_fp4(*[kw.get(n, x) for n, x in dict(  # noqa: E731
        q=q, k=kv, v=kv, kp=kp, vp=vp, ks=ks, vs=vs, t=t, lens=lens).items()])
    app()
    for kw in (dict(kp=kp.float()), dict(kp=kp[:, :, :, :16]), dict(ks=ks.float()), dict(ks=ks[:, :1]), dict(vs=vs[:3]),
               dict(vp=vp[:, :, :8]), dict(t=t.long()), dict(lens=lens[:1]), dict(kp=kp.cpu()), dict(q=q.cpu()), dict(vs=None),
               dict(ks=ks.transpose(2, 3)), dict(k=kv[:, :1], v=kv[:, :1])):
        with pytest.raises(ValueError):
            app(**kw)
    with pytest.raises(ValueError):
        fa.append_paged_fp4(q, kv, kv, kp, vp, ks, vs, t, lens, offsets=cuda([1], torch.int32))
    q4 = q.view(2, 1, 4, 64).transpose(1, 2)
    fa.decode_paged_fp4(q4, kp, vp, ks, vs, t, lens)
    for bad in (dict(max_len=33), dict(out=q4.float())):
        with pytest.raises(ValueError):
            fa.decode_paged_fp4(q4, kp, vp, ks, vs, t, lens, **bad)
    with pytest.raises(fa.FAError):
        fa.decode_paged_fp4(q4, kp, vp, ks, vs, t, lens, scale=float("nan"))
    cu = cuda([0, 3, 7], torch.int32)
    fa.read_paged(kp, vp, t, lens, cu, 7, k_scale=ks, v_scale=vs)
    for args in ((kp, vp, t, lens, cu[:2], 7), (kp, vp[:2], t, lens, cu, 7), (kp, vp, t, lens, cu, -1), (kp[0], vp, t, lens, cu, 7)):
        with pytest.raises(ValueError):
            fa.read_paged(*args, k_scale=ks, v_scale=vs)
    with pytest.raises(ValueError):
        fa.read_paged(kp, vp, t, lens, cu, 7)                     # (uint8 pages without scales are no bf16 pages)
    with pytest.raises(ValueError):
        fa.read_paged(kp, vp, t, lens, cu, 7, k_scale=ks, v_scale=None)
    assert fa.device_status() == fa.FA_OK
