"""The paged calls where their other tests do not look: the keys' position behind rows that were lost, two streams with every
call in flight, refusals made by the compiled and by the Python checks, weights that are nearly alike."""

import numpy as np
import pytest
import torch

from oracle import paged as OP
from parity import to64
from test_paged_gpu import APPEND, BASE, Cache, cuda, make_table, near_bf16
from test_paged_long_gpu import same, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


@pytest.mark.parametrize("inter,norm", [(False, True), (True, False)], ids=["half-norm", "interleaved"])
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", [c for c in APPEND if c["rot"]], ids=lambda c: "n{}p{}d{}r{}".format(
    "-".join(map(str, c["new"])), c["page"], c["d"], c["rot"]))
def test_keys_behind_lost_rows(fa, case, f8, inter, norm):
    """Queries, keys and held rows are those of position row + offset; the rows are where the lengths say."""
    new, lens, H, Hkv, page, d, rot = (case[k] for k in ("new", "lens", "H", "Hkv", "page", "d", "rot"))
    rng = np.random.default_rng(sum(lens) + d + inter)
    B, T = len(new), sum(new)
    count = [(L + page - 1) // page for L in lens]
    table, n = make_table(rng, B, count, max(count))
    cache = Cache(rng, n, Hkv, page, d, f8)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    w = [cuda(1 + 0.3 * rng.standard_normal(d), torch.bfloat16) if norm else None for _ in range(2)]
    turns = fa.rotary_turns(rot, BASE)
    cu = None if len(set(new)) == 1 else cuda(np.concatenate([[0], np.cumsum(new)]), torch.int32)
    offsets = rng.integers(1, 1 << 20, B)
    qo, ko = fa.append_paged(q, k, v, *cache.gpu, cuda(table), cuda(lens, torch.int32), cu_seqlens=cu, max_new=max(new),
                             turns=turns, interleaved=inter, q_weight=w[0], k_weight=w[1], eps=1e-5,
                             offsets=cuda(offsets, torch.int32), **cache.kw())
    assert fa.device_status() == fa.FA_OK
    rq, rk, pos = OP.append(to64(q), to64(k), to64(v), new, [L + int(o) for L, o in zip(lens, offsets)], turns.tolist(), inter,
                            *[None if x is None else to64(x) for x in w], eps=1e-5)
    near_bf16(to64(qo), rq, "q")
    near_bf16(to64(ko), rk, "k")
    held, scale = cache.values(0), None if not f8 else cache.scales(0)
    for t, b in enumerate(np.repeat(np.arange(B), new)):
        row = pos[t] - int(offsets[b])
        pid = table[b, row // page]
        x = held[pid, :, row % page]
        if not f8:
            assert np.array_equal(x, to64(ko)[t])
        else:  # half a step of e4m3 (2^-4 of a value, 2^-10 of the scale at least), of the fp32 key
            tol = 2.0 ** -4 * np.abs(rk[t]) + 2.0 ** -10 * scale[pid][:, None] + 16 * 2.0 ** -24 * np.abs(rk[t]).max(axis=-1, keepdims=True)
            assert np.all(np.abs(x - rk[t]) <= tol)


def test_two_streams_with_every_call_in_flight(fa):
    """Two 4-bit caches, each on a stream of its own, all calls issued in turn before anything is waited for."""
    def calls(s, out):
        pool = (s["kp"], s["vp"], s["ks"], s["vs"])
        kw = dict(k_scale=s["ks"], v_scale=s["vs"])
        yield lambda: out.extend(fa.append_paged_fp4(s["qt"], s["k"], s["v"], *pool, s["table"], s["lens"], turns=s["turns"],
                                                     q_weight=s["norm"], k_weight=s["norm"]))
        yield lambda: out.extend(fa.decode_paged_fp4(s["q"], *pool, s["table"], s["lens"], workspace=s["ws"]))
        yield lambda: out.extend(fa.read_paged(s["kp"], s["vp"], s["table"], s["lens"], s["cu"], 431, **kw))
        yield lambda: out.append(fa.weigh_paged(s["q"], out[3], s["kp"], s["table"], s["lens"], s["w"], k_scale=s["ks"]))
        yield lambda: out.extend(fa.evict_paged(s["w"], s["kp"], s["vp"], s["table"], s["lens"], s["new"], 64, first=3, recent=20, **kw))
        yield lambda: out.extend(pool)

    alone = []
    for seed in (7, 8):
        out = []
        for call in calls(state(fa, "fp4", seed), out):
            call()
        torch.cuda.synchronize()
        alone.append([x.clone() for x in out])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        states, outs = [state(fa, "fp4", seed) for seed in (7, 8)], [[], []]
        torch.cuda.synchronize()
        for pair in zip(*(calls(s, o) for s, o in zip(states, outs))):
            for call, st in zip(pair, streams):
                with torch.cuda.stream(st):
                    call()
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            same(a, b)
    assert fa.device_status() == fa.FA_OK


class Off:
    def __getattr__(self, name):
        return lambda *a: NotImplemented


def bad_calls(fa, s):
    """Calls that are refused, each a name and a call."""
    f4 = dict(q=s["qt"], k=s["k"], v=s["v"], k_pages=s["kp"], v_pages=s["vp"], k_scale=s["ks"], v_scale=s["vs"],
              block_table=s["table"], seqlens_k=s["lens"], turns=s["turns"])
    dec = dict(q=s["q"], k_pages=s["kp"], v_pages=s["vp"], k_scale=s["ks"], v_scale=s["vs"], block_table=s["table"],
               seqlens_k=s["lens"], workspace=s["ws"])
    rd = dict(k_pages=s["kp"], v_pages=s["vp"], block_table=s["table"], seqlens_k=s["lens"], cu_seqlens=s["cu"], total=431,
              k_scale=s["ks"], v_scale=s["vs"])
    wg = dict(q=s["q"], lse=s["lse"], k_pages=s["kp"], block_table=s["table"], seqlens_k=s["lens"], weights=s["w"], k_scale=s["ks"])
    ev = dict(weights=s["w"], k_pages=s["kp"], v_pages=s["vp"], block_table=s["table"], seqlens_k=s["lens"], new_table=s["new"],
              keep=20, k_scale=s["ks"], v_scale=s["vs"])
    pools = [dict(k_pages=s["kp"][:, :1]), dict(v_pages=s["vp"][1:]), dict(k_pages=s["kp"].float()), dict(k_scale=s["ks"][..., :1]),
             dict(v_scale=s["vs"].float()), dict(k_pages=s["kp"].transpose(1, 2)), dict(k_pages=s["kp"].cpu()), dict(k_pages=None)]
    tables = [dict(block_table=s["table"].long()), dict(block_table=s["table"][0]), dict(block_table=s["table"].t()),
              dict(block_table=s["table"].cpu()), dict(seqlens_k=s["lens"].long()), dict(seqlens_k=s["lens"][:2]),
              dict(seqlens_k=s["lens"].cpu())]
    some = {
        fa.append_paged_fp4: (f4, pools + tables + [
            dict(q=s["qt"].float()), dict(q=s["qt"][:5]), dict(k=s["k"][:, :1]), dict(k=s["k"][0]), dict(v=s["v"][..., :64]),
            dict(turns=s["turns"].int()), dict(turns=s["turns"][:3]), dict(q_weight=s["norm"][:64]), dict(k_weight=s["norm"].float()),
            dict(offsets=s["lens"].long()), dict(offsets=s["lens"][:1]), dict(cu_seqlens=s["lens"]), dict(max_new=-1),
            dict(q_out=s["qt"][:5]), dict(k_out=s["k"].float()), dict(q_out=s["qt"][:, :1].expand(-1, 8, -1)), dict(eps=-1.0)]),
        fa.decode_paged_fp4: (dec, pools + tables + [
            dict(q=s["q"].half()), dict(q=s["q"][0]), dict(q=s["q"][:2]), dict(q=s["q"][:, :3]), dict(workspace=s["ws"][:16]),
            dict(out=s["q"][:2]), dict(lse=s["lse"].double()), dict(lse=s["lse"][:, :2]), dict(max_len=-1), dict(max_len=1 << 20),
            dict(num_splits=-1), dict(scale=float("nan")), dict(workspace=s["ws"].cpu())]),
        fa.read_paged: (rd, pools + tables + [
            dict(cu_seqlens=s["cu"][:3]), dict(cu_seqlens=s["cu"].long()), dict(total=-1), dict(k_out=s["k"]), dict(v_out=s["v"].float())]),
        fa.weigh_paged: (wg, [p for p in pools if "v_pages" not in p and "v_scale" not in p] + tables + [
            dict(q=s["q"].half()), dict(q=s["q"][:2]), dict(lse=s["lse"][:, :2]), dict(lse=s["lse"].double()), dict(weights=s["w"][:2]),
            dict(weights=s["w"].double()), dict(weights=s["w"][..., ::2]), dict(max_len=-1), dict(max_len=314), dict(scale=float("inf")),
            dict(k_scale=None)]),
        fa.evict_paged: (ev, pools + tables + [
            dict(weights=s["w"].double()), dict(weights=s["w"][:, :1]), dict(keep=0), dict(keep=65), dict(first=-1), dict(recent=21),
            dict(first=15, recent=6), dict(new_table=s["new"][:1]), dict(new_table=s["new"].long()), dict(new_table=s["table"]),
            dict(offsets=s["lens"][:1]), dict(max_len=314), dict(new_weights=s["w"][:2]), dict(new_weights=s["w"][..., :19]),
            dict(new_weights=s["w"])]),
    }
    for fn, (ok, wrong) in some.items():
        for kw in wrong:
            yield fn.__name__, sorted(kw), (lambda fn=fn, ok=ok, kw=kw: fn(**{**ok, **kw}))


def test_compiled_and_python_checks_refuse_alike(fa, monkeypatch):
    def refusals():
        s = state(fa, "fp4", 1)
        out = []
        for name, what, call in bad_calls(fa, s):
            try:
                call()
                out.append((name, what, None))
            except Exception as e:
                out.append((name, what, type(e)))
        return out

    fast = refusals()
    monkeypatch.setattr(fa, "_binding", Off())
    slow = refusals()
    assert fast == slow
    assert all(e in (ValueError, fa.FAError) for _, _, e in fast), [x for x in fast if x[2] not in (ValueError, fa.FAError)]
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("spread", [0.05, 0.5, 1.0])
@pytest.mark.parametrize("B,Hkv,L,keep", [(2, 4, 131072, 32768), (32, 8, 16384, 4001), (4, 4, 1400, 1024), (1, 1, 400000, 1000), (300, 1, 50000, 25000)])
def test_selection_of_weights_that_are_nearly_alike(fa, B, Hkv, L, keep, spread):
    """Weights within an octave or so, most of which share the border's first digit: against a stable sort."""
    g = torch.Generator(device="cuda").manual_seed(L + B)
    w = torch.exp(spread * torch.randn(B, Hkv, L, device="cuda", generator=g))
    w[..., ::5] = w[..., ::5].to(torch.bfloat16).float()                       # with some ties
    page, d, count = 128, 64, (keep + 127) // 128
    pool = [torch.zeros(1 + B * count, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.zeros(B, (L + page - 1) // page, dtype=torch.int32, device="cuda")
    new = 1 + torch.arange(B * count, dtype=torch.int32, device="cuda").view(B, count)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    kept, _, nw, _ = fa.evict_paged(w, *pool, table, lens, new, keep)
    assert fa.device_status() == fa.FA_OK
    top = w.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(dim=-1).values
    assert torch.equal(kept, top.int()) and torch.equal(nw, w.gather(2, top))


@pytest.mark.skipif(not hasattr(torch, "float4_e2m1fn_x2"), reason="a torch without the type")
def test_pairs_of_4bit_values_as_their_own_type(fa):
    """Pages of float4_e2m1fn_x2 are taken by the compiled checks too, and read as the same bytes."""
    s = state(fa, "fp4", 3)
    pages = [x.view(torch.float4_e2m1fn_x2) for x in (s["kp"], s["vp"])]
    want = fa.read_paged(s["kp"], s["vp"], s["table"], s["lens"], s["cu"], 431, k_scale=s["ks"], v_scale=s["vs"])
    r = fa._binding.read(*pages, s["table"], s["lens"], s["cu"], 431, s["ks"], s["vs"], None, None, None)
    if hasattr(fa._binding, "__file__"):
        assert r is not NotImplemented and r[0] == fa.FA_OK
        assert all(torch.equal(a, b) for a, b in zip(want, r[1]))
    got = fa.read_paged(*pages, s["table"], s["lens"], s["cu"], 431, k_scale=s["ks"], v_scale=s["vs"])
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and fa.device_status() == fa.FA_OK
