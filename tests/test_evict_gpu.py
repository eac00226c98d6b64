"""GPU parity of eviction by accumulated attention weight (fa_weigh_paged, fa_evict_paged) against the fp64 oracle,
alone and in a run of steps over caches of every kind.

Tolerances. Eviction copies: everything it returns must be exactly the oracle's (codes of an e4m3 page whose scale grew
are rounded once, to nearest even). An attention weight is exp(y - lse): a score's products are exact and summed in
fp32 in at most d / 16 + 4 steps, each off by at most 2^-22 of the sum of their magnitudes (the tensor cores do not round to
nearest), q's smallest elements by 2^-25 of its largest; y, lse and their difference are rounded three times (2^-24 of
each); the exponential is off by 2^-22 of itself. The sum over at most 128 rows adds 128 half steps of fp32.
"""

import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F4
from oracle import fp8 as FP8
from oracle import paged as OP
from parity import to64
from test_paged_fp4_gpu import pool_of
from test_paged_gpu import cuda, make_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def near_weights(got, base, q, kv, table, lens, lse, scale):
    """`got` [B,Hkv,W] against `base` plus the oracle's weights, within the error derived above."""
    B, H, Nq, d = q.shape
    Hkv, page = kv.shape[1], kv.shape[2]
    want = base.copy()
    for b, rows in enumerate(F4.weigh(q, kv, table, lens, lse, scale)):
        for hk, w in enumerate(rows):
            L, G = lens[b], H // Hkv
            if L == 0:
                continue
            k = np.array([kv[int(table[b][j // page]), hk, j % page] for j in range(L)])
            rel = np.zeros(L)
            for h in range(hk * G, (hk + 1) * G):
                for t in range(Nq):
                    if np.isfinite(lse[b, h, t]):
                        x = q[b, h, t]
                        size = abs(scale) * (np.abs(k) @ np.abs(x))
                        off = size * (d / 16 + 4) * 2.0 ** -22 + abs(scale) * np.abs(x).max() * np.abs(k).sum(axis=1) * 2.0 ** -25
                        rel = np.maximum(rel, off + 3 * 2.0 ** -24 * (size + abs(lse[b, h, t])))
            want[b, hk, :L] += w
            bound = w * (np.expm1(rel) + 2.0 ** -22 + 128 * 2.0 ** -24) + np.abs(want[b, hk, :L]) * 2.0 ** -24 + 1e-37
            assert np.all(np.abs(got[b, hk, :L] - want[b, hk, :L]) <= bound), (b, hk, np.abs(got[b, hk, :L] - want[b, hk, :L]).max())
    for b, L in enumerate(lens):
        assert np.array_equal(got[b, :, L:], base[b, :, L:])


def lse_of(q, kv, table, lens, scale):
    return OP.attend(q, kv, kv, table, lens, scale)[1]


# lengths, heads, tokens, page
WEIGH = [
    dict(lens=[1, 16, 17, 0, 65], H=4, Hkv=2, Nq=1, page=16),
    dict(lens=[700, 3], H=32, Hkv=8, Nq=1, page=64),
    dict(lens=[63, 1000, 2], H=5, Hkv=1, Nq=3, page=32),
    dict(lens=[300, 130], H=8, Hkv=2, Nq=16, page=128),       # 64 rows
    dict(lens=[200, 40], H=4, Hkv=1, Nq=32, page=16),         # 128 rows
    dict(lens=[150], H=14, Hkv=2, Nq=18, page=64),            # 126
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", WEIGH, ids=lambda c: "L{}h{}kv{}q{}p{}".format("-".join(map(str, c["lens"])), c["H"], c["Hkv"],
                                                                           c["Nq"], c["page"]))
def test_weigh(fa, case, d, kind):
    lens, H, Hkv, Nq, page = (case[k] for k in ("lens", "H", "Hkv", "Nq", "page"))
    rng = np.random.default_rng(sum(lens) + H + d)
    B, count = len(lens), [(L + page - 1) // page for L in lens]
    table, n = make_table(rng, B, count, max(count) + 2)
    kp, _, ks, _, kv, _ = pool_of(rng, kind, n, Hkv, page, d)
    # rows past each sequence's end hold NaN
    for b, L in enumerate(lens):
        if L % page:
            where = (int(table[b, L // page]), slice(None), slice(L % page, None))
            if kind == "fp4":
                ks[where] = 0xFF
            else:
                kp.view(torch.int16 if kind == "bf16" else torch.uint8)[where] = 0x7FFF if kind == "bf16" else 0x7F
    q = torch.randn(B, Nq, H, d, generator=torch.Generator().manual_seed(H)).to(torch.bfloat16).cuda().transpose(1, 2)
    scale = 1 / math.sqrt(d)
    lse = lse_of(to64(q), np.nan_to_num(kv), table, lens, scale)
    W = max(lens) + 5
    base = rng.random((B, Hkv, W)).astype(np.float32)
    big = torch.full((B, Hkv, W + 3), -1.0, device="cuda")
    w = big[:, :, :W]
    w.copy_(torch.from_numpy(base))
    got = fa.weigh_paged(q, cuda(lse, torch.float32), kp, cuda(table), cuda(lens, torch.int32), w, k_scale=ks)
    assert fa.device_status() == fa.FA_OK and got is w and (big[:, :, W:] == -1).all()
    near_weights(to64(w), base.astype(np.float64), to64(q), kv, table, lens, to64(cuda(lse, torch.float32)), scale)
    # twice the same bytes: nothing depends on an order
    again = torch.from_numpy(base).cuda()
    fa.weigh_paged(q, cuda(lse, torch.float32), kp, cuda(table), cuda(lens, torch.int32), again, k_scale=ks)
    assert torch.equal(again, w)


def test_weigh_after_decode_sums_to_the_rows(fa):
    """With the decode's own log-sum-exp the weights of all keys sum to the number of query rows that see a key."""
    rng = np.random.default_rng(2)
    lens, H, Hkv, Nq, page, d = [900, 2, 77], 8, 2, 3, 32, 128
    count = [(L + page - 1) // page for L in lens]
    table, n = make_table(rng, 3, count, max(count))
    kp, vp, ks, vs, _, _ = pool_of(rng, "fp4", n, Hkv, page, d)
    q = torch.randn(3, H, Nq, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    t, ln = cuda(table), cuda(lens, torch.int32)
    _, lse = fa.decode_paged_fp4(q, kp, vp, ks, vs, t, ln)
    w = torch.zeros(3, Hkv, max(lens), device="cuda")
    fa.weigh_paged(q, lse, kp, t, ln, w, k_scale=ks)
    assert fa.device_status() == fa.FA_OK
    # each weight is off by a few 2^-20 of itself, so is their sum
    rows = np.array([12.0, 8.0, 12.0])[:, None]       # (of the second sequence the first token sees nothing)
    assert np.abs(to64(w).sum(axis=-1) / rows - 1).max() <= 2.0 ** -16


def test_weigh_odd_rows(fa):
    """Rows with lse = -inf add nothing, whatever q and the keys hold; NaN keys reach their own weights only; a negative
    scale; pages outside the pool; lengths past max_len are clipped."""
    rng = np.random.default_rng(3)
    page, d, H, Hkv = 16, 64, 4, 2
    kp, _, _, _, kv, _ = pool_of(rng, "bf16", 6, Hkv, page, d)
    q = torch.randn(1, H, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    t, ln = cuda([[0, 2, 3]], torch.int32), cuda([40], torch.int32)
    lse = cuda(lse_of(to64(q), kv, [[0, 2, 3]], [40], -0.2), torch.float32)
    w = torch.zeros(1, Hkv, 48, device="cuda")
    fa.weigh_paged(q, lse, kp, t, ln, w, scale=-0.2)
    near_weights(to64(w), np.zeros((1, Hkv, 48)), to64(q), kv, [[0, 2, 3]], [40], to64(lse), -0.2)
    # the first group's rows are dead: weights of K/V head 0 stay 0 beside NaN and infinity in q and k
    dead, qn, kn = lse.clone(), q.clone(), kp.clone()
    dead[:, :2] = -math.inf
    qn[:, :2] = math.nan
    kn[2, 0, 3] = math.inf
    kn[2, 1, 3] = math.nan
    w.zero_()
    fa.weigh_paged(qn, dead, kn, t, ln, w, scale=-0.2)
    assert fa.device_status() == fa.FA_OK
    assert (w[:, 0] == 0).all() and torch.isnan(w[0, 1, 19]) and torch.isfinite(w[0, 1]).sum() == 47
    # a page outside the pool: its keys get nothing, the rest what it had
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        w2 = torch.zeros(1, Hkv, 48, device="cuda")
        fa.weigh_paged(q, lse, kp, cuda([[0, bad, 3]], torch.int32), ln, w2, scale=-0.2)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        assert (w2[..., 16:32] == 0).all() and (w2[..., :16] > 0).all() and (w2[..., 32:40] > 0).all()
    # clipped: the keys past max_len are not written (their weights count from the same lse)
    w3 = torch.zeros(1, Hkv, 20, device="cuda")
    fa.weigh_paged(q, lse, kp, t, ln, w3, scale=-0.2)
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG and (w3 > 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("d,page,Hkv,lens,keep,first,recent", [
    (64, 16, 2, [100, 7, 0, 33, 32], 32, 4, 8), (128, 64, 4, [1000, 129], 100, 0, 0), (64, 128, 1, [500], 500, 1, 1),
    (128, 16, 2, [50, 51], 50, 50, 0), (64, 32, 3, [40, 300], 39, 0, 39), (128, 128, 2, [3], 1, 0, 0),
    (64, 64, 1, [9000, 4097], 130, 10, 100), (128, 16, 8, [700, 2, 18], 17, 1, 3),
], ids=str)
def test_evict(fa, kind, d, page, Hkv, lens, keep, first, recent):
    rng = np.random.default_rng(sum(lens) + d + keep)
    B, count = len(lens), [(L + page - 1) // page for L in lens]
    more = [(min(L, keep) + page - 1) // page for L in lens]
    both, n = make_table(rng, B, [a + b for a, b in zip(count, more)], max(a + b for a, b in zip(count, more)))
    table = np.full((B, max(count) + 1), -1, dtype=np.int32)
    new = np.full((B, max(max(more), 1) + 1), -1, dtype=np.int32)
    for b in range(B):
        table[b, :count[b]], new[b, :more[b]] = both[b, :count[b]], both[b, count[b]:count[b] + more[b]]
    kp, vp, ks, vs, _, _ = pool_of(rng, kind, n, Hkv, page, d)
    before = [None if x is None else (x if x.dtype == torch.uint8 or x.dtype == torch.float32 else x.view(torch.uint8)).cpu().numpy().copy()
              for x in (kp, vp, ks, vs)]
    W = max(lens) + 3
    # many ties, zeros of both signs, infinities, NaN
    w = rng.integers(0, 12, (B, Hkv, W)).astype(np.float32) / 4
    w[rng.random(w.shape) < 0.05] = np.nan
    w[rng.random(w.shape) < 0.03] = np.inf
    w[rng.random(w.shape) < 0.1] = -0.0
    w[rng.random(w.shape) < 0.02] = -np.inf
    w[:, :, ::3] = rng.random((B, Hkv, (W + 2) // 3))
    offsets = rng.integers(0, 1000, B)
    nw = torch.full((B, Hkv, keep + 9), 5.0, device="cuda")
    kept, nl, nw2, no = fa.evict_paged(cuda(w), kp, vp, cuda(table), cuda(lens, torch.int32), cuda(new), keep, first=first,
                                       recent=recent, k_scale=ks, v_scale=vs, offsets=cuda(offsets, torch.int32),
                                       new_weights=nw[:, :, :keep + 4])
    assert fa.device_status() == fa.FA_OK
    assert nl.tolist() == [min(L, keep) for L in lens]
    assert no.tolist() == [int(o) + L - min(L, keep) for o, L in zip(offsets, lens)]
    assert (nw[:, :, keep + 4:] == 5).all()
    want = [None if x is None else x.copy() for x in before]
    want_kept, want_w = np.full((B, Hkv, keep), -1), np.zeros((B, Hkv, keep + 4), dtype=np.float32)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            rows = F4.kept_rows(w[b, h], L, keep, first, recent)
            want_kept[b, h, :len(rows)] = rows
            want_w[b, h, :len(rows)] = w[b, h, rows]
            for x in range(2):
                for p0 in range(0, len(rows), page):
                    part, dst = rows[p0:p0 + page], new[b, p0 // page]
                    src = [(table[b, j // page], j % page) for j in part]
                    if kind == "e4m3":
                        old = np.array([before[2 + x][s, h] for s, _ in src])
                        want[2 + x][dst, h] = old.max()
                        for i, (s, r) in enumerate(src):
                            v = FP8.e4m3_decode(before[x][s, h, r]) * (old[i] / old.max())
                            want[x][dst, h, i] = before[x][s, h, r] if old[i] == old.max() else OP.e4m3_encode(v)
                    else:
                        for i, (s, r) in enumerate(src):
                            want[x][dst, h, i] = before[x][s, h, r]
                            if kind == "fp4":
                                want[2 + x][dst, h, i] = before[2 + x][s, h, r]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(nw2.cpu().numpy(), want_w, equal_nan=True)
    for x, y in zip((kp, vp, ks, vs), want):
        if y is not None:
            assert np.array_equal((x if x.dtype in (torch.uint8, torch.float32) else x.view(torch.uint8)).cpu().numpy(), y)


@pytest.mark.parametrize("B,Hkv,L,keep,first,recent", [
    (1, 1, 400000, 1000, 5, 100), (1, 2, 131072, 32768, 0, 2048), (40, 8, 5000, 1250, 4, 64), (3, 1, 45000, 44999, 0, 0),
    (300, 1, 50000, 25000, 10, 10)])
def test_evict_selection_of_long_rows(fa, B, Hkv, L, keep, first, recent):
    """The selection alone at lengths that take clusters of every size, keys held or read again: weights with few
    different values, so that ties decide, and random ones, against a stable sort."""
    g = torch.Generator(device="cuda").manual_seed(L)
    for few in (True, False):
        w = torch.randint(0, 3, (B, Hkv, L), device="cuda", generator=g).float() if few else torch.rand(B, Hkv, L, device="cuda", generator=g)
        lens = torch.randint(keep + 1, L + 1, (B,), device="cuda", generator=g).int()
        page, d = 128, 64
        width = (L + page - 1) // page
        # (all rows come from page 0, which every entry shares: what is copied does not matter here)
        count = (keep + page - 1) // page
        pool = [torch.zeros(1 + B * count, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        new = 1 + torch.arange(B * count, dtype=torch.int32, device="cuda").view(B, count)
        kept, nl, nw, _ = fa.evict_paged(w, *pool, table, lens, new, keep, first=first, recent=recent)
        assert fa.device_status() == fa.FA_OK and (nl == keep).all()
        j = torch.arange(L, device="cuda")
        sure = (j < first) | ((j >= lens[:, None] - recent) & (j < lens[:, None]))
        x = torch.where(sure[:, None], 10.0, w)
        x = torch.where((j >= lens[:, None])[:, None], -1.0, x)
        top = x.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(dim=-1).values
        assert torch.equal(kept, top.int())
        assert torch.equal(nw, w.gather(2, top))


def test_evict_bad_pages_and_lengths(fa):
    """Pages outside the pool are skipped and reported, on either side; lengths past max_len are clipped."""
    rng = np.random.default_rng(7)
    page, d, Hkv = 16, 64, 2
    for kind in ("bf16", "e4m3", "fp4"):
        for bad in (-1, 8, 2 ** 31 - 1, -2 ** 31):
            kp, vp, ks, vs, kv, _ = pool_of(rng, kind, 8, Hkv, page, d)
            w = torch.rand(1, Hkv, 48, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
            for table, new, missing in (([[0, bad, 2]], [[3, 4]], "old"), ([[0, 1, 2]], [[3, bad]], "new")):
                was = kp.view(torch.uint8).clone()
                kept, nl, _, _ = fa.evict_paged(w, kp, vp, cuda(table, torch.int32), cuda([48], torch.int32), cuda(new, torch.int32),
                                                30, k_scale=ks, v_scale=vs)
                assert fa.device_status() == fa.FA_ERR_INVALID_ARG and nl.tolist() == [30]
                got = kp.view(torch.uint8)
                for h in range(Hkv):
                    rows = F4.kept_rows(w[0, h].tolist(), 48, 30, 0, 0)
                    assert kept[0, h].tolist() == rows
                    for i, j in enumerate(rows):
                        gone = (missing == "old" and 16 <= j < 32) or (missing == "new" and i >= 16)
                        if not (missing == "new" and i >= 16) and kind != "e4m3":
                            dst = got[new[0][i // page], h, i % page]
                            src = was[table[0][j // page], h, j % page] if not gone else was[new[0][i // page], h, i % page]
                            assert torch.equal(dst, src)
                assert torch.equal(got[[5, 6, 7]], was[[5, 6, 7]])
    kept, nl, _, _ = fa.evict_paged(w, kp, vp, cuda([[0, 1, 2]], torch.int32), cuda([49], torch.int32), cuda([[3, 4]], torch.int32), 20,
                                    k_scale=ks, v_scale=vs)
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG and nl.tolist() == [20] and int(kept.max()) < 48


def test_binding_refusals(fa):
    rng = np.random.default_rng(5)
    kp, vp, ks, vs, _, _ = pool_of(rng, "fp4", 6, 2, 16, 64)
    t, new, ln = cuda([[0, 1], [2, 3]], torch.int32), cuda([[4], [5]], torch.int32), cuda([20, 9], torch.int32)
    w = torch.rand(2, 2, 32, device="cuda")
    ok = dict(weights=w, k_pages=kp, v_pages=vp, block_table=t, seqlens_k=ln, new_table=new, keep=16, k_scale=ks, v_scale=vs)
    fa.evict_paged(**ok)
    for kw in (dict(weights=w.double()), dict(weights=w[:, :1]), dict(weights=w.transpose(0, 1)), dict(weights=w[:, :, ::2]), dict(keep=17), dict(keep=0),
               dict(new_table=new[:1]), dict(new_table=new.long()), dict(v_pages=vp[:5]), dict(v_scale=None), dict(max_len=33),
               dict(offsets=cuda([1], torch.int32)), dict(seqlens_k=ln.cpu()), dict(new_weights=w[:1])):
        with pytest.raises(ValueError):
            fa.evict_paged(**{**ok, **kw})
    for kw in (dict(first=10, recent=7), dict(first=-1), dict(new_weights=w), dict(new_weights=torch.rand(2, 2, 15, device="cuda"))):
        with pytest.raises(fa.FAError):
            fa.evict_paged(**{**ok, **kw})
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 4, 1, device="cuda")
    okw = dict(q=q, lse=lse, k_pages=kp, block_table=t, seqlens_k=ln, weights=w, k_scale=ks)
    fa.weigh_paged(**okw)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(lse=lse[:, :2]), dict(lse=lse.double()), dict(k_scale=None), dict(weights=w[:, :, 0]),
               dict(weights=w.expand(2, 2, 32)[:1]), dict(max_len=-1), dict(max_len=40), dict(block_table=t[:1]),
               dict(weights=torch.rand(1, 1, 32, device="cuda").expand(2, 2, 32))):
        with pytest.raises(ValueError):
            fa.weigh_paged(**{**okw, **kw})
    with pytest.raises(fa.FAError):
        fa.weigh_paged(**okw, scale=float("inf"))
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_a_run_of_them(fa, kind):
    """What a serving program does with a cache that is cut: two prompts in chunks (append, read back, attend, weigh), cut to
    a budget, then single tokens (append at their true positions, decode, weigh) captured into a graph and replayed, another
    cut, more tokens. Compared with the same steps on lists of rows in 64 bits."""
    H, Hkv, d, page, keep, first, recent = 8, 2, 128, 16, 40, 2, 8
    lens0, B = [70, 90], 2
    rng = np.random.default_rng(11)
    n = 64
    free = list(rng.permutation(n))
    kp, vp, ks, vs, _, _ = pool_of(rng, kind, n, Hkv, page, d)
    turns = fa.rotary_turns(d, 10000.0)
    scale = 1 / math.sqrt(d)
    W = 128
    table = torch.full((B, W // page), -1, dtype=torch.int32, device="cuda")

    def new_pages(t):
        for b in range(B):
            t[b] = torch.tensor([free.pop() for _ in range(t.shape[1])], dtype=torch.int32)

    new_pages(table)
    weights = torch.zeros(B, Hkv, W, device="cuda")
    lens, offsets = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def append(x, cu):
        part = (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:])
        if kind == "fp4":
            return fa.append_paged_fp4(*part, kp, vp, ks, vs, table, lens, cu_seqlens=cu, turns=turns, offsets=offsets)
        return fa.append_paged(*part, kp, vp, table, lens, cu_seqlens=cu, turns=turns, k_scale=ks, v_scale=vs, offsets=offsets)

    def decode(q):
        if kind == "fp4":
            return fa.decode_paged_fp4(q, kp, vp, ks, vs, table, lens)
        return fa.decode_paged(q, kp, vp, table, lens, k_scale=ks, v_scale=vs)

    def rows_held():
        """What the cache holds, read back: [b] -> (k, v) [L, Hkv, d] in 64 bits."""
        cu = [0]
        for L in lens.tolist():
            cu.append(cu[-1] + L)
        k, v = fa.read_paged(kp, vp, table, lens, cuda(cu, torch.int32), cu[-1], k_scale=ks, v_scale=vs)
        return [(to64(k[a:b]), to64(v[a:b])) for a, b in zip(cu, cu[1:])]

    def check(q, o, lse, before, held):
        """q, o [B,H,Nq,d]: attention and weights of these tokens, against the rows held."""
        qs, want = to64(q), before.copy()
        for b, (k, v) in enumerate(held):
            L, Nq = k.shape[0], q.shape[2]
            for h in range(H):
                s = scale * qs[b, h] @ k[:, h // 4].T
                s[np.arange(L)[None] > (L - Nq + np.arange(Nq))[:, None]] = -np.inf
                m = s.max(axis=-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(axis=-1, keepdims=True)
                # weights of 16 bits over values of order 1 (the tolerance of tests/parity.py), result in bf16
                assert np.abs(to64(o[b, h]) - p / l @ v[:, h // 4]).max() <= 2e-2
                assert np.abs(to64(lse[b, h]) - (m + np.log(l))[:, 0]).max() <= 1e-3
                want[b, h // 4, :L] += (p / l).sum(axis=0)
        assert np.abs(to64(weights) - want).max() <= 1e-3

    step = 0
    for part in ([30, 50], [25, 30], [15, 10]):           # chunks of the prompts
        T = sum(part)
        x = torch.randn(T, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(step)).to(torch.bfloat16).cuda()
        step += 1
        lens += cuda(part, torch.int32)
        cu = cuda([0, part[0], T], torch.int32)
        q, _ = append(x, cu)
        total = int(lens.sum())
        cu_k = cuda([0, int(lens[0]), total], torch.int32)
        k, v = fa.read_paged(kp, vp, table, lens, cu_k, total, k_scale=ks, v_scale=vs)
        o, lse = fa.fwd_packed(q, k, v, cu, cu_k, causal=True)
        # the chunk's last five tokens are weighed (q and lse as the decode takes them)
        tail = torch.stack([q[:part[0]][-5:], q[part[0]:][-5:]]).transpose(1, 2)
        tail_o = torch.stack([o[:part[0]][-5:], o[part[0]:][-5:]]).transpose(1, 2)
        tail_lse = torch.stack([lse[:, :part[0]][:, -5:], lse[:, part[0]:][:, -5:]]).contiguous()
        before = to64(weights)
        fa.weigh_paged(tail, tail_lse, kp, table, lens, weights, k_scale=ks)
        check(tail, tail_o, tail_lse, before, rows_held())
    assert lens.tolist() == lens0

    def cut():
        nonlocal table, weights, lens, offsets
        old, old_lens, old_w = rows_held(), lens.tolist(), to64(weights)
        new = torch.full((B, W // page), -1, dtype=torch.int32, device="cuda")
        new_pages(new)
        kept, lens, weights, offsets = fa.evict_paged(weights, kp, vp, table, lens, new, keep, first=first, recent=recent,
                                                      k_scale=ks, v_scale=vs, offsets=offsets,
                                                      new_weights=torch.empty(B, Hkv, W, device="cuda"))
        free.extend(table.flatten().tolist())
        table = new
        assert lens.tolist() == [min(L, keep) for L in old_lens]
        for b, (k, v) in enumerate(rows_held()):
            for h in range(Hkv):
                rows = F4.kept_rows(old_w[b, h], old_lens[b], keep, first, recent)
                assert kept[b, h, :len(rows)].tolist() == rows
                for x, y in zip((k, v), old[b]):
                    # e4m3: rounded again where the page's scale grew, half a step of 2^-4, or 2^-10 of that scale (values
                    # below 448 of it, of which the largest row has some over 224)
                    tol = (2.0 ** -4 * np.abs(y[rows, h]) + 2.0 ** -10 / 224 * np.abs(y).max()) if kind == "e4m3" else 0.0
                    assert np.all(np.abs(x[:, h] - y[rows, h]) <= tol)

    def token(x):
        lens.add_(1)
        q, _ = append(x, None)
        q = q.view(B, 1, H, d).transpose(1, 2)
        o, lse = decode(q)
        fa.weigh_paged(q, lse, kp, table, lens, weights, k_scale=ks)
        return q, o, lse

    for rounds in range(2):
        cut()
        assert offsets.tolist() == [L - keep + 4 * rounds for L in lens0]
        x = torch.randn(B, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(100 + rounds)).to(torch.bfloat16).cuda()
        before = to64(weights)
        q, o, lse = token(x)
        check(q, o, lse, before, rows_held())
        # the true position: the row and what was evicted before it
        rq, _, _ = OP.append(to64(x[:, :H]), to64(x[:, H:H + Hkv]), None, [1] * B,
                             [int(L) + int(p) for L, p in zip(lens, offsets)], turns.tolist(), False)
        assert np.abs(to64(q)[:, :, 0] - rq).max() <= 2.0 ** -7 * np.abs(rq).max()
        # three more through a captured graph
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gq, go, gl = token(x)
        for i in range(3):
            x.copy_(torch.randn(B, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(200 + 10 * rounds + i)).to(torch.bfloat16))
            before = to64(weights)
            graph.replay()
            torch.cuda.synchronize()
            check(gq, go, gl, before, rows_held())
        assert fa.device_status() == fa.FA_OK


def test_captured_eviction(fa):
    """A captured weigh and evict follows new lengths and weights, on another stream than the tensors' own."""
    rng = np.random.default_rng(12)
    B, Hkv, H, d, page, keep = 2, 2, 4, 64, 16, 20
    kp, vp, ks, vs, kv, _ = pool_of(rng, "fp4", 20, Hkv, page, d)
    table = cuda([[0, 1, 2, 3], [4, 5, 6, 7]], torch.int32)
    new = cuda([[10, 11], [12, 13]], torch.int32)
    lens, w = cuda([50, 18], torch.int32), torch.rand(B, Hkv, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.evict_paged(w, kp, vp, table, lens, new, keep, k_scale=ks, v_scale=vs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept, nl, nw, no = fa.evict_paged(w, kp, vp, table, lens, new, keep, k_scale=ks, v_scale=vs)
    for seed, L in ((1, [64, 1]), (2, [20, 21]), (3, [0, 40])):
        w.copy_(torch.rand(B, Hkv, 64, generator=torch.Generator().manual_seed(seed)))
        lens.copy_(torch.tensor(L, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.device_status() == fa.FA_OK and nl.tolist() == [min(x, keep) for x in L]
        assert no.tolist() == [x - min(x, keep) for x in L]
        for b in range(B):
            for h in range(Hkv):
                rows = F4.kept_rows(w[b, h].tolist(), L[b], keep, 0, 0)
                assert kept[b, h].tolist() == rows + [-1] * (keep - len(rows))
