"""GPU parity of the packed prefill (fa_fwd_packed) against the fp64 oracle: every
element of small batches of ragged sequences, with grouped heads, prefixes, empty
sequences and rows, foreign values beside every sequence, and tokens behind the
last one. Tolerances are those of the forward pass (tests/parity.py)."""

import math

import numpy as np
import pytest
import torch

from oracle import paged as OP
from parity import compare, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def cum(xs):
    return [0] + np.cumsum(xs).tolist()


def i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def inputs(tq, tk, H, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(t, h, d, generator=g).to(torch.bfloat16).cuda() for t, h in ((tq, H), (tk, Hkv), (tk, Hkv))]


CASES = [
    # lq, lk (None: the same), H, Hkv
    ([1], None, 2, 2),
    ([128, 128], None, 4, 2),
    ([5, 1, 190, 127, 129], None, 8, 2),
    ([0, 300, 0, 77, 0], None, 4, 1),                        # empty sequences
    ([260, 513], None, 6, 2),                                # an odd group: two row tiles of a head
    ([100, 30, 257], None, 5, 1),
    ([40, 1, 200], [300, 129, 200], 8, 4),                   # behind prefixes
    ([200, 130, 3], [70, 0, 2], 4, 2),                       # fewer keys than queries: rows that see nothing
    ([300, 10], [0, 0], 2, 1),                               # no key at all
    ([17] * 40, None, 2, 2),                                 # many short sequences
    ([700], None, 7, 7),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "q{}k{}h{}kv{}".format(
    "-".join(map(str, c[0][:5])), "same" if c[1] is None else "-".join(map(str, c[1])), c[2], c[3]))
def test_packed(fa, case, causal, d):
    lq, lk, H, Hkv = case
    cu_q, cu_k = cum(lq), cum(lq if lk is None else lk)
    more = 3  # rows behind the last sequence
    q, k, v = inputs(cu_q[-1] + more, cu_k[-1] + more, H, Hkv, d, seed=len(lq) + d)
    for x in (q, k, v):
        x[-more:] = float("nan")
    out = torch.full_like(q, 7.0)
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    fa.fwd_packed(q, k, v, i32(cu_q), None if lk is None else i32(cu_k), causal=causal, out=out, lse=lse)
    assert fa.device_status() == fa.FA_OK
    n = cu_q[-1]
    ro, rl = OP.packed(to64(q[:n]), to64(k[:cu_k[-1]]), to64(v[:cu_k[-1]]), cu_q, cu_k, 1 / math.sqrt(d), causal)
    compare(to64(out[:n]).reshape(-1, d), to64(lse[:, :n]).T.reshape(-1), ro.reshape(-1, d), rl.T.reshape(-1),
            f"{case} causal={causal} d={d}")
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 1)])
def test_sequences_do_not_reach_one_another(fa, H, Hkv, d):
    """Infinities and NaN in every other sequence leave the others' results bit for bit as they are without them."""
    lq = [70, 130, 5, 257, 64]
    cu = cum(lq)
    q, k, v = inputs(cu[-1], cu[-1], H, Hkv, d, seed=5)
    clean, lse0 = fa.fwd_packed(q, k, v, i32(cu), causal=True)
    for b in (1, 3):
        for x in (q, k, v):
            x[cu[b]:cu[b + 1]] = float("inf")
            x[cu[b]:cu[b + 1], :, ::3] = float("nan")
    dirty, lse1 = fa.fwd_packed(q, k, v, i32(cu), causal=True)
    assert fa.device_status() == fa.FA_OK
    for b in (0, 2, 4):
        assert torch.equal(clean[cu[b]:cu[b + 1]], dirty[cu[b]:cu[b + 1]])
        assert torch.equal(lse0[:, cu[b]:cu[b + 1]], lse1[:, cu[b]:cu[b + 1]])


@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_of_every_tile(fa, d):
    """Two long sequences and a short one, grouped heads, more units than SMs: seeded rows of every head, the first and
    last rows of the sequences among them."""
    lq, H, Hkv = [3000, 40, 4100], 32, 8
    cu = cum(lq)
    q, k, v = inputs(cu[-1], cu[-1], H, Hkv, d, seed=9)
    o, lse = fa.fwd_packed(q, k, v, i32(cu), causal=True)
    assert fa.device_status() == fa.FA_OK
    from oracle import attention as A
    rng = np.random.default_rng(0)
    for b in range(3):
        a0, a1 = cu[b], cu[b + 1]
        for h in range(0, H, 3):
            rows = np.unique(np.concatenate([[0, lq[b] - 1], rng.integers(0, lq[b], 6)]))
            ro, rl = A.attend_head(to64(q[a0:a1, h]), to64(k[a0:a1, h // 4]), to64(v[a0:a1, h // 4]), 1 / math.sqrt(d),
                                   True, rows=rows)
            compare(to64(o[a0:a1, h])[rows], to64(lse[h, a0:a1])[rows], ro, rl, f"b={b} h={h}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (4, 2)])
def test_many_short_units(fa, H, Hkv, d):
    """Several times more units than SMs, most of them of one row block whose second tile (odd groups) has no row, with
    a few that see no key at all: every CTA walks a run of such units."""
    rng = np.random.default_rng(2)
    B = 700
    lq = rng.integers(1, 60, B)
    lq[::7] = 200
    lk = lq + rng.integers(-3, 40, B)
    lk[::5] = 0
    lk = np.maximum(lk, 0)
    cu_q, cu_k = cum(lq), cum(lk)
    q, k, v = inputs(cu_q[-1], cu_k[-1], H, Hkv, d, seed=d)
    o, lse = fa.fwd_packed(q, k, v, i32(cu_q), i32(cu_k), causal=True)
    assert fa.device_status() == fa.FA_OK
    some = [0, 1, 5, 7, 35, *rng.integers(0, B, 40).tolist()]
    for b in some:
        a0, a1, b0, b1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        ro, rl = OP.packed(to64(q[a0:a1]), to64(k[b0:b1]), to64(v[b0:b1]), [0, a1 - a0], [0, b1 - b0], 1 / math.sqrt(d), True)
        compare(to64(o[a0:a1]).reshape(-1, d), to64(lse[:, a0:a1]).T.reshape(-1), ro.reshape(-1, d), rl.T.reshape(-1), f"{b}")


@pytest.mark.parametrize("d", [64, 128])
def test_against_the_dense_forward(fa, d):
    """One sequence, one head per K/V head: the same attention as fa_fwd on the same rows, bit for bit where both walk
    the same tiles (an odd group takes the dense kernel's tiles)."""
    N, H = 600, 3
    q, k, v = inputs(N, N, H, H, d, seed=3)
    o, lse = fa.fwd_packed(q, k, v, i32([0, N]), causal=True)
    dense = [x.transpose(0, 1).contiguous()[None] for x in (q, k, v)]
    od, ld = fa.fwd(*dense, causal=True)
    assert fa.device_status() == fa.FA_OK
    assert torch.equal(o.transpose(0, 1)[None], od) and torch.equal(lse[None], ld)


def test_negative_and_zero_scale(fa):
    lq, d, H, Hkv = [150, 20], 64, 4, 2
    cu = cum(lq)
    q, k, v = inputs(cu[-1], cu[-1], H, Hkv, d, seed=4)
    for scale in (-0.125, 0.0):
        o, lse = fa.fwd_packed(q, k, v, i32(cu), scale=scale, causal=True)
        assert fa.device_status() == fa.FA_OK
        ro, rl = OP.packed(to64(q), to64(k), to64(v), cu, cu, scale, True)
        compare(to64(o).reshape(-1, d), to64(lse).T.reshape(-1), ro.reshape(-1, d), rl.T.reshape(-1))


def test_parts_of_one_projection(fa):
    """q, k, v taken from one tensor [T, H + 2 Hkv, d] and o written into a larger one: the bytes of separate tensors,
    and nothing else written."""
    lq, d, H, Hkv = [140, 300, 9], 128, 8, 2
    cu = cum(lq)
    qkv = torch.randn(cu[-1], H + 2 * Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    parts = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    want, lse = fa.fwd_packed(*(x.contiguous() for x in parts), i32(cu), causal=True)
    big = torch.full((cu[-1], 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse2 = fa.fwd_packed(*parts, i32(cu), causal=True, out=big[:, ::2])
    head_major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in parts]
    got3, lse3 = fa.fwd_packed(*head_major, i32(cu), causal=True)
    assert fa.device_status() == fa.FA_OK
    assert torch.equal(want, got) and torch.equal(lse, lse2) and (big[:, 1::2] == 7).all()
    assert torch.equal(want, got3) and torch.equal(lse, lse3)


def test_graph_follows_new_offsets(fa):
    """A captured call replayed with other offsets in the same tensors; another call between replays uses its own
    workspace."""
    d, H, Hkv, T = 128, 8, 2, 700
    q, k, v = inputs(T, T, H, Hkv, d, seed=8)
    cu = i32([0, 100, 650, 700])
    ws = [torch.empty(fa.fwd_packed_workspace_size(3, T, H, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out, lse = torch.empty_like(q), torch.empty(H, T, device="cuda")
    fa.fwd_packed(q, k, v, cu, causal=True, workspace=ws[0], out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fwd_packed(q, k, v, cu, causal=True, workspace=ws[0], out=out, lse=lse)
    for offs in ([0, 100, 650, 700], [0, 700, 700, 700], [0, 1, 2, 3], [0, 350, 351, 620]):
        cu.copy_(i32(offs))
        out.fill_(7.0)
        graph.replay()
        want, lw = fa.fwd_packed(q, k, v, i32(offs), causal=True, workspace=ws[1])
        torch.cuda.synchronize()
        n = offs[-1]
        assert fa.device_status() == fa.FA_OK
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:, :n], lw[:, :n]) and (out[n:] == 7).all()


def test_bad_offsets_are_clipped_and_reported(fa):
    d, H, Hkv, T = 64, 4, 2, 200
    q, k, v = inputs(T, T, H, Hkv, d, seed=8)
    for offs in ([0, 300], [-5, 100], [100, 50], [0, 2 ** 31 - 1]):
        out = torch.full_like(q, 7.0)
        fa.fwd_packed(q, k, v, i32(offs), causal=True, out=out)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
        a, b = max(offs[0], 0), min(max(offs[1], 0), T)
        if b > a:
            ro, _ = OP.packed(to64(q), to64(k), to64(v), [a, b], [a, b], 1 / math.sqrt(d), True)
            assert np.abs(to64(out[a:b]) - ro[a:b]).max() <= 2e-2
        assert (out[:a] == 7).all() and (out[max(a, b):] == 7).all()


def test_serving_run(fa):
    """A prompt step as a server makes it: append (norms and rotation) of a packed batch, attention among the new
    tokens, then single decode steps over the cache. A sequence's decode row equals the packed attention of the same
    tokens given as one longer prompt."""
    H, Hkv, d, page, lens = 8, 2, 128, 32, [90, 33]
    T = sum(lens)
    g = torch.Generator().manual_seed(1)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    turns = fa.rotary_turns(d, 500000.0, scaling=("by_parts", 4.0, 4096, 1.0, 32.0))
    kw = dict(turns=turns, q_weight=w[0], k_weight=w[1])
    pool = [torch.zeros(16, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = i32([[4, 2, 9, 1], [7, 3, 11, 0]])
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    split = lambda x: (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:])   # noqa: E731
    cu, L = i32(cum(lens)), i32(lens)
    q, k = fa.append_paged(*split(qkv), *pool, table, L, cu_seqlens=cu, **kw)
    o, lse = fa.fwd_packed(q, k, split(qkv)[2], cu, causal=True)
    ro, rl = OP.packed(to64(q), to64(k), to64(split(qkv)[2]), cum(lens), cum(lens), 1 / math.sqrt(d), True)
    compare(to64(o).reshape(-1, d), to64(lse).T.reshape(-1), ro.reshape(-1, d), rl.T.reshape(-1))
    step = torch.randn(2, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    L1 = L + 1
    q1, k1 = fa.append_paged(*split(step), *pool, table, L1, **kw)
    od, ld = fa.decode_paged(q1.view(2, 1, H, d).transpose(1, 2), *pool, table, L1)
    # the same as one prompt
    whole = torch.cat([qkv[:90], step[:1], qkv[90:], step[1:]])
    cu2 = i32([0, 91, 125])
    q2, k2 = fa.append_paged(*split(whole), *[torch.zeros_like(x) for x in pool], table, L1, cu_seqlens=cu2, **kw)
    op, lp = fa.fwd_packed(q2, k2, split(whole)[2], cu2, causal=True)
    assert fa.device_status() == fa.FA_OK
    for b, t in ((0, 90), (1, 124)):
        assert torch.equal(q2[t], q1[b]) and torch.equal(k2[t], k1[b])
        # each within the tolerance of the exact result
        assert (od[b, :, 0].float() - op[t].float()).abs().max() <= 2e-2
        assert (ld[b, :, 0] - lp[:, t]).abs().max() <= 2e-3


def test_plan_of_many_sequences(fa):
    """More sequences than the list's CTA has threads, empty ones and a long one among them: every row is computed once,
    with its own sequence's keys. (Each sequence's values are one constant of its own, so its rows return that constant.)"""
    rng = np.random.default_rng(7)
    B, d = 2600, 64
    lq = rng.integers(0, 5, B)
    lq[1500], lq[2599] = 1000, 130
    cu = cum(lq)
    T = cu[-1]
    q, k, _ = inputs(T, T, 2, 2, d, seed=1)
    own = torch.repeat_interleave(torch.arange(B) % 251, torch.tensor(lq)).cuda()
    v = own.to(torch.bfloat16)[:, None, None].expand(T, 2, d).contiguous()
    o, lse = fa.fwd_packed(q, k, v, i32(cu))
    assert fa.device_status() == fa.FA_OK
    # integers up to 250 are bf16 values; the weights' sum and the sum of the rounded weights differ by at most 2^-8
    assert ((o.float() - v.float()).abs() <= 2.0 ** -8 * v.float() * 2).all() and torch.isfinite(lse).all()


def test_calls_on_another_stream(fa):
    """Outputs and workspaces that a call makes stay its own while it runs on a stream that is not current."""
    lq = [300, 200, 100] * 6
    cu = i32(cum(lq))
    q, k, v = inputs(sum(lq), sum(lq), 8, 2, 128, seed=6)
    want, lse = fa.fwd_packed(q, k, v, cu, causal=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(fa.fwd_packed(q, k, v, cu, causal=True, stream=side))
        torch.full((1 << 20,), 3.0, device="cuda")   # current-stream work that takes memory the side stream still uses, if let
    side.synchronize()
    assert fa.device_status() == fa.FA_OK
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, lse)


def test_binding_refusals(fa):
    q, k, v = inputs(10, 10, 4, 2, 64, seed=1)
    cu = i32([0, 10])
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(k=k[:, :, :32]), dict(v=v[:5]), dict(cu_seqlens_q=cu.long()),
               dict(cu_seqlens_q=cu[:1]), dict(cu_seqlens_k=i32([0, 5, 10])), dict(out=q[:5]),
               dict(lse=torch.zeros(10, 4, device="cuda"))):
        with pytest.raises(ValueError):
            fa.fwd_packed(**{**dict(q=q, k=k, v=v, cu_seqlens_q=cu), **kw})
    with pytest.raises(fa.FAError):
        fa.fwd_packed(q, k, v, cu, scale=float("nan"))
    with pytest.raises(fa.FAError):
        fa.fwd_packed(q, k, v, cu, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FAError):
        fa.fwd_packed(q, k[:5], v[:5], cu)   # other rows without their offsets
    assert fa.fwd_packed(q[:0], k[:0], v[:0], cu)[0].shape == (0, 4, 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 1)])
def test_rows_that_see_nothing_beside_nan(fa, H, Hkv, d):
    """Queries before a sequence's first key get zeros and -inf, whatever v holds; a query of NaN gets NaN in both."""
    lq, lk = [150, 40], [20, 40]
    cu_q, cu_k = cum(lq), cum(lk)
    q, k, v = inputs(cu_q[-1], cu_k[-1], H, Hkv, d, seed=12)
    v[:20] = float("nan")
    q[160] = float("nan")
    o, lse = fa.fwd_packed(q, k, v, i32(cu_q), i32(cu_k), causal=True)
    assert fa.device_status() == fa.FA_OK
    assert (o[:130] == 0).all() and torch.isneginf(lse[:, :130]).all()
    assert torch.isnan(o[130:150]).all() and torch.isfinite(lse[:, 130:150]).all()
    assert torch.isnan(o[160]).all() and torch.isnan(lse[:, 160]).all()
    rest = [t for t in range(150, 190) if t != 160]
    assert torch.isfinite(o[rest]).all() and torch.isfinite(lse[:, rest]).all()
