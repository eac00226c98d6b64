"""Cases of the operators that make a paged cache smaller: 4-bit pages (`fa.append_paged_fp4`, `fa.read_paged`,
`fa.decode_paged_fp4`) and eviction by accumulated attention weight (`fa.weigh_paged`, `fa.evict_paged`).

Every case is a dict of plain values. `prepare` makes its inputs on the GPU from a seed, `run` makes one pass: the plain
form in elementary torch operations, or (with `own` set) this package's calls. `exact` computes the same outputs in 64
bits, written apart from the plain form.

The operators, in short:

fill    New tokens are normalised and turned as `fa.append_paged` does it (token i of sequence b, n_b new ones, is at row
        p = L_b - n_b + i and turned for position p + offset_b), q and k are returned in bf16, and k (as returned) and v go
        to 4-bit pages. A row is held in groups of 16 neighbours: one scale s, the nearest value to max|x| / 6 with 5
        exponent and 3 mantissa bits (an f16's upper byte without the sign; 2^-17 <= s <= 10240, 0 for a group of zeros),
        and 16 codes, the nearest to x / s of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (ties to the even code,
        saturating). Then the rows that a prompt's attention needs are read back as bf16, code times scale: the last m_b
        rows of every sequence, packed.
decode  q [B, H, n, d] are the last n positions of each sequence; query head h reads K/V head h / (H / Hkv); token t sees
        key j iff j <= L_b - n + t.
weigh   weights[b, hk, j] += sum over the query rows (h, t) of K/V head hk that see j of exp(scale <q, k_j> - lse).
evict   Of a sequence with L > keep rows, every K/V head keeps rows j < first, j >= L - recent, and those of the others
        with the largest weights, keep in all (ties to the lowest index), in order; a shorter one keeps all. The kept rows
        go to the pages of a new table. An e4m3 page's scale is the largest of its rows' old scales, and codes are rounded
        again to it. New lengths, weights (0 behind the kept ones) and positions of row 0 come back.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # of the codes 0 .. 7; codes 8 .. 15 are their negatives


# ---------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # One decode step of a small batch: one token each, read back for the tokens' own attention. Latency.
        dict(name="fill_step_b8", op="fill", B=8, new_lo=1, new_hi=1, past_lo=40, past_hi=2000, H=16, Hkv=4, d=64,
             page=16, rot=64, inter=False, norm=False, whole=False, moved=0, uniform=True, lens_seed=1),
        # Prompts of different lengths, with the norms of queries and keys; their own rows are read back.
        dict(name="fill_prompts", op="fill", B=12, new_lo=1, new_hi=4096, past_lo=0, past_hi=500, H=32, Hkv=8, d=128,
             page=64, rot=128, inter=False, norm=True, whole=False, moved=0, uniform=False, lens_seed=3),
        # Chunks of long prompts behind prefixes that lost rows before; the whole cache is read back for their attention.
        dict(name="fill_chunks_prefix", op="fill", B=9, new_lo=500, new_hi=2048, past_lo=0, past_hi=9000, H=28, Hkv=4,
             d=128, page=32, rot=64, inter=True, norm=False, whole=True, moved=200000, uniform=False, lens_seed=4),
        # One user, a short context: the latency of a single decode step.
        dict(name="decode_b1_short", op="decode", B=1, H=32, Hkv=8, d=128, nq=1, page=16, len_lo=700, len_hi=700,
             lens_seed=5),
        # A serving batch, ragged lengths.
        dict(name="decode_b64_ragged", op="decode", B=64, H=32, Hkv=8, d=128, nq=1, page=64, len_lo=4096, len_hi=8192,
             lens_seed=6),
        # A few users with long contexts and drafts of four tokens to check, d = 64.
        dict(name="decode_b6_long_nq4_d64", op="decode", B=6, H=32, Hkv=8, d=64, nq=4, page=128, len_lo=30001,
             len_hi=131072, lens_seed=7),
        # A decode step's weights, short contexts, a 16-bit cache. Latency.
        dict(name="weigh_b8_short_bf16", op="weigh", B=8, H=16, Hkv=4, d=64, nq=1, page=16, kind="bf16", len_lo=5,
             len_hi=1500, lens_seed=8),
        # The same for a serving batch with a 4-bit cache.
        dict(name="weigh_b64_fp4", op="weigh", B=64, H=32, Hkv=8, d=128, nq=1, page=64, kind="fp4", len_lo=4096,
             len_hi=8192, lens_seed=9),
        # The last sixteen tokens of prompts, weighed before their caches are cut; e4m3 pages.
        dict(name="weigh_b16_window_e4m3", op="weigh", B=16, H=32, Hkv=8, d=128, nq=16, page=64, kind="e4m3", len_lo=1000,
             len_hi=16384, lens_seed=10),
        # A few sequences a little over their budget, a 16-bit cache.
        dict(name="evict_b4_bf16", op="evict", B=4, Hkv=4, d=64, page=16, kind="bf16", len_lo=1025, len_hi=1400,
             keep=1024, first=4, recent=128, read=False, lens_seed=11),
        # Prompts of a serving batch cut to a quarter, e4m3 pages, an odd budget that ends inside a page.
        dict(name="evict_b32_e4m3", op="evict", B=32, Hkv=8, d=128, page=64, kind="e4m3", len_lo=8000, len_hi=16384,
             keep=4001, first=16, recent=512, read=False, lens_seed=12),
        # Two very long contexts in a 4-bit cache, cut between chunks; the kept rows are read back for the next chunk.
        dict(name="evict_b2_long_fp4", op="evict", B=2, Hkv=8, d=128, page=128, kind="fp4", len_lo=90001, len_hi=131072,
             keep=32768, first=64, recent=2048, read=True, lens_seed=13),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fill", "decode", "weigh", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["bf16", "e4m3", "fp4", "fp4"])
    seed = rng.randrange(1 << 30)
    if op == "fill":
        B = _log(rng, 1, 256)
        uniform = rng.random() < 0.5
        if uniform:
            lo = hi = rng.choice([1, 1, 2, 3, 5])
        else:
            lo, hi = 1, _log(rng, 2, max(2, 24000 // B))
        whole = rng.random() < 0.4
        past = _log(rng, 10, max(10, min(100000, 60000 // B)) if whole else 100000)
        return dict(op=op, B=B, new_lo=lo, new_hi=hi, past_lo=0, past_hi=past, H=Hkv * G, Hkv=Hkv, d=d, page=page,
                    rot=rng.choice([d, d, d // 2, 16, 48]), inter=rng.random() < 0.4, norm=rng.random() < 0.5,
                    whole=whole, moved=rng.choice([0, 0, 1000, 400000]), uniform=uniform, lens_seed=seed)
    if op == "decode":
        B = _log(rng, 1, 96)
        hi = _log(rng, 20, min(131072, 390000 // B))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, nq=rng.choice([1, 1, 1, 2, 3, 5]), page=page,
                    len_lo=max(1, hi // rng.choice([1, 2, 50])), len_hi=hi, lens_seed=seed)
    if op == "weigh":
        B = _log(rng, 1, 96)
        hi = _log(rng, 20, min(131072, 190000 // B))
        nq = rng.choice([1, 1, 2, 5, 16, 128 // G])
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, nq=nq if nq * G <= 128 else 128 // G, page=page, kind=kind,
                    len_lo=max(1, hi // rng.choice([1, 2, 50])), len_hi=hi, lens_seed=seed)
    B = _log(rng, 1, 64)
    hi = _log(rng, 40, min(131072, 250000 // B))
    keep = max(8, int(hi * rng.choice([0.1, 0.25, 0.5, 0.9])))
    return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, kind=kind, len_lo=max(1, hi // rng.choice([1, 2, 10])), len_hi=hi,
                keep=keep, first=rng.choice([0, 1, keep // 50]), recent=rng.choice([0, keep // 16, keep // 3]),
                read=kind == "fp4", lens_seed=seed)


def _lens(c):
    """The case's lengths, a pair for each sequence: new tokens and length of fill, else (0, length)."""
    rng = random.Random(c["lens_seed"])
    out = []
    for _ in range(c["B"]):
        if c["op"] == "fill":
            n = rng.randint(c["new_lo"], c["new_hi"])
            out.append((n, n + rng.randint(c["past_lo"], c["past_hi"])))
        else:
            out.append((0, rng.randint(c["len_lo"], c["len_hi"])))
    return out


def _cum(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _row_bytes(kind, d):
    """Bytes of one row (keys or values) of one K/V head; an e4m3 page's scale is not counted."""
    return {"bf16": 2 * d, "e4m3": d, "fp4": d // 2 + d // 16}[kind]


def work(c):
    lens = _lens(c)
    Hkv, d, B = c["Hkv"], c["d"], c["B"]
    if c["op"] == "fill":
        T, H, row = sum(n for n, _ in lens), c["H"], _row_bytes("fp4", d)
        # q read and written, k read and written, v read, the cache rows written; the rows read back: those that were
        # there before read, all of them written in bf16
        R = sum(L for _, L in lens) if c["whole"] else T
        nbytes = T * (2 * 2 * H * d + 3 * 2 * Hkv * d + 2 * Hkv * row) + (R - T) * 2 * Hkv * row + R * 2 * Hkv * 2 * d
        return {"bytes": nbytes, "flops": T * (H + Hkv) * (3 * c["rot"] + (4 * d if c["norm"] else 0)) + 4 * T * Hkv * d}
    total = sum(L for _, L in lens)
    if c["op"] == "evict":
        row = _row_bytes(c["kind"], d)
        kept = sum(min(L, c["keep"]) for _, L in lens)
        # the weights read, the kept rows read and written, their indices and weights written
        nbytes = Hkv * (4 * total + kept * (2 * 2 * row + 8))
        return {"bytes": nbytes + (kept * 2 * Hkv * 2 * d if c["read"] else 0), "flops": Hkv * total}
    H, nq = c["H"], c["nq"]
    seen = sum(sum(max(0, L - nq + t + 1) for t in range(nq)) for _, L in lens)
    if c["op"] == "decode":
        nbytes = total * Hkv * 2 * _row_bytes("fp4", d) + 2 * B * H * nq * d * 2 + B * H * nq * 4
        return {"bytes": nbytes, "flops": 4 * H * d * seen}
    nbytes = total * Hkv * (_row_bytes(c["kind"], d) + 8) + B * H * nq * (2 * d + 4)
    return {"bytes": nbytes, "flops": 2 * H * d * seen + H * seen}


# ---------------------------------------------------------------------------------------------------------------------
# the 4-bit rows

def _quantize(x):
    """x [..., d] fp32 -> (codes 0 .. 15 [..., d], scales [..., d / 16]) as whole numbers and fp32."""
    g = x.unflatten(-1, (-1, 16))
    most = g.abs().amax(dim=-1)
    y = most / 6.0
    step = torch.exp2((torch.frexp(y).exponent - 4).clamp(min=-17).float())
    s = (torch.round(y / step) * step).clamp(min=2.0 ** -17, max=10240.0)
    s = torch.where(most > 0, s, torch.zeros_like(s))
    a = g.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    unit = 0.5 + 0.5 * (a >= 2) + (a >= 4)
    v = (torch.round(a / unit) * unit).clamp(max=6.0)
    code = (v >= 0.5).int() + (v >= 1) + (v >= 1.5) + (v >= 2) + (v >= 3) + (v >= 4) + (v >= 6)
    code = code + 8 * torch.signbit(g)
    return code.flatten(-2), s


def _scale_bytes(s):
    """The byte of a scale: an f16's sign is 0 and its lower seven bits are 0."""
    return (s.half().view(torch.int16) >> 7).to(torch.uint8)


def _pack(code):
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def _values(codes, scale):
    """Rows [..., d / 2] and [..., d / 16] of bytes -> values [..., d] in fp32."""
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1).flatten(-2)
    s = (scale.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------------------------------------------------
# inputs

def _i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _turns(rot, base=500000.0):
    """Frequency j, base^(-2j / rot) radians a token, as a fraction of a turn in units of 2^-64 (mod 2^64)."""
    out = []
    for j in range(rot // 2):
        t = int(base ** (-2.0 * j / rot) / (2.0 * math.pi) * 2.0 ** 64) % (1 << 64)
        out.append(t - (1 << 64) if t >= 1 << 63 else t)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def _outliers(Hkv, d, g):
    """Factors of the channels of each head: a few are far larger than the rest, as in the keys of trained models."""
    f = torch.ones(Hkv, d, device="cuda")
    at = torch.rand(Hkv, d, device="cuda", generator=g).argsort(dim=-1)[:, :max(2, d // 32)]
    return f.scatter_(1, at, 20.0)


def _page_pool(n, Hkv, page, d, kind, g):
    """Pages that hold earlier tokens. Rows of different pages differ in magnitude, as tokens do."""
    x = torch.randn(n, Hkv, page, d, device="cuda", generator=g)
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    x = x * torch.exp2(torch.randn(n, Hkv, 1, 1, device="cuda", generator=g) * 0.7)
    if kind == "fp4":
        code, s = _quantize(x.to(torch.bfloat16).float())
        return _pack(code), _scale_bytes(s)
    m, e = torch.frexp(x.abs().amax(dim=(2, 3)) / E4M3_MAX)
    s = torch.exp2(torch.where(m > 0.5, e, e - 1).float())
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    lens = _lens(c)
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    kind = c.get("kind", "fp4")
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    st = dict(c, kind=kind)
    # the pages that a call touches, at random places of the pool: all of a sequence's, or those from the first new row on
    part = c["op"] == "fill" and not c["whole"]
    count = [(L + page - 1) // page for _, L in lens]
    start = [(L - n) // page if part else 0 for n, L in lens]
    more = [(min(L, c["keep"]) + page - 1) // page if c["op"] == "evict" else 0 for _, L in lens]
    need = sum(count) - sum(start)
    ids = list(range(need + sum(more) + 3))
    rng.shuffle(ids)

    def table(lo, hi):
        t = torch.full((B, max(1, max(hi))), -1, dtype=torch.int32)
        for b in range(B):
            t[b, lo[b]:hi[b]] = torch.tensor([ids.pop() for _ in range(lo[b], hi[b])], dtype=torch.int32)
        return t.cuda()

    pool = len(ids)
    st["table"], st["lens"] = table(start, count), _i32([L for _, L in lens])
    st["max_len"] = max(L for _, L in lens)
    st["k_pages"], st["k_scale"] = _page_pool(pool, Hkv, page, d, kind, g)
    st["v_pages"], st["v_scale"] = _page_pool(pool, Hkv, page, d, kind, g)
    if c["op"] == "evict":
        st["new_table"] = table([0] * B, more)
        # accumulated weights: a few keys have far more than the rest, and many that were never looked at have exactly 0
        w = torch.exp(2.0 * rand(B, Hkv, st["max_len"])) * (torch.rand(B, Hkv, st["max_len"], device="cuda", generator=g) > 0.05)
        st["weights"] = w
        st["offsets"] = _i32([rng.randint(0, 100000) for _ in range(B)])
        st["width"] = c["keep"] + 512                       # room for the tokens to come until the next eviction
        cu = _cum([min(L, c["keep"]) for _, L in lens])
        st["read_cu"], st["read_total"] = _i32(cu), cu[-1]
        return st
    if c["op"] in ("decode", "weigh"):
        H, nq = c["H"], c["nq"]
        # token-major memory, as the append returns it, seen as [B, H, nq, d]
        st["q"] = (1.5 * rand(B, nq, H, d)).to(torch.bfloat16).transpose(1, 2)
        if c["op"] == "weigh":
            # the decode call before returned the log-sum-exp
            st["lse"] = _log_sums(st)
            st["weights"] = torch.zeros(B, Hkv, st["max_len"], device="cuda")
        return st
    n, H = [a for a, _ in lens], c["H"]
    T = sum(n)
    qkv = rand(T, H + 2 * Hkv, d)  # one projection's output; q, k and v are views of it
    qkv[:, H:H + Hkv] *= _outliers(Hkv, d, g)
    qkv = qkv.to(torch.bfloat16)
    st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    st["cu"] = None if c["uniform"] else _i32(_cum(n))
    st["max_new"] = max(n)
    st["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
    st["row"] = torch.cat([torch.arange(L - a, L, device="cuda") for a, L in lens])
    st["offsets"] = _i32([rng.randint(0, c["moved"]) for _ in range(B)]) if c["moved"] else None
    st["turns"] = _turns(c["rot"])
    st["q_weight"] = (1 + 0.2 * rand(d)).to(torch.bfloat16) if c["norm"] else None
    st["k_weight"] = (1 + 0.2 * rand(d)).to(torch.bfloat16) if c["norm"] else None
    st["eps"] = 1e-6
    cu = _cum([L if c["whole"] else a for a, L in lens])
    st["read_cu"], st["read_total"] = _i32(cu), cu[-1]
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass

def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _own_fill(st):
    from io_aware_exact_fa_gb300 import fa
    cache = (st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
    q, k = fa.append_paged_fp4(st["q"], st["k"], st["v"], *cache, cu_seqlens=st["cu"], max_new=st["max_new"],
                               turns=st["turns"], interleaved=st["inter"], q_weight=st["q_weight"],
                               k_weight=st["k_weight"], eps=st["eps"], offsets=st["offsets"])
    ks, vs = fa.read_paged(st["k_pages"], st["v_pages"], st["table"], st["lens"], st["read_cu"], st["read_total"],
                           k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"q": q, "k": k, "k_held": ks, "v_held": vs}


def _own_decode(st):
    from io_aware_exact_fa_gb300 import fa
    if "ws" not in st:  # a serving program keeps its workspace
        st["ws"] = torch.empty(max(1, fa.decode_paged_fp4_workspace_size(st["B"], st["H"], st["Hkv"], st["nq"], st["d"],
                                                                         st["max_len"])), dtype=torch.uint8, device="cuda")
    return fa.decode_paged_fp4(st["q"], st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["table"], st["lens"],
                               max_len=st["max_len"], workspace=st["ws"])


def _own_weigh(st):
    from io_aware_exact_fa_gb300 import fa
    return fa.weigh_paged(st["q"], st["lse"], st["k_pages"], st["table"], st["lens"], st["weights"],
                          k_scale=st["k_scale"])


def _own_evict(st):
    from io_aware_exact_fa_gb300 import fa
    if "new_weights" not in st:  # a buffer of the cache that the rows move to
        st["new_weights"] = torch.empty(st["B"], st["Hkv"], st["width"], device="cuda")
    kept, lens, weights, offsets = fa.evict_paged(
        st["weights"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["new_table"], st["keep"],
        first=st["first"], recent=st["recent"], k_scale=st["k_scale"], v_scale=st["v_scale"], offsets=st["offsets"],
        new_weights=st["new_weights"])
    out = {"kept": kept, "lens": lens, "weights": weights, "offsets": offsets}
    if st["read"]:
        out["k"], out["v"] = fa.read_paged(st["k_pages"], st["v_pages"], st["new_table"], lens, st["read_cu"],
                                           st["read_total"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        return out
    return _pool_outputs(st, out)


def _pool_outputs(st, out):
    # (float8 values beside the scales they count in)
    out["k_pages"], out["v_pages"] = st["k_pages"], st["v_pages"]
    if st["kind"] == "e4m3":
        out["k_scale"], out["v_scale"] = st["k_scale"], st["v_scale"]
    return out


def _rotate(x, pos, st, weight):
    """Norm and rotation of [T, heads, d] in 32 bits (angles in 64)."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + st["eps"]) * weight.float()
    rot = st["rot"]
    freq = torch.where(st["turns"] < 0, st["turns"].double() + 2.0 ** 64, st["turns"].double()) * (2.0 * math.pi / 2.0 ** 64)
    ang = pos.double()[:, None] * freq
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    y = x.clone()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if st["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _store(x, pages, scale, st):
    """Writes x [T, Hkv, d] (bf16) to 4-bit pages."""
    code, s = _quantize(x.float())
    pid, row = st["table"][st["seq"], st["row"] // st["page"]].long(), st["row"] % st["page"]
    pages[pid, :, row] = _pack(code)
    scale[pid, :, row] = _scale_bytes(s)


def _packed_rows(lens, cu, total):
    """Of every packed output row: its sequence and its row there (the last cu[b + 1] - cu[b] rows of sequence b)."""
    n = cu.long().diff()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=total)
    return seq, torch.arange(total, device=cu.device) - cu.long()[seq + 1] + lens.long()[seq]


def _read(st, table, lens):
    seq, row = _packed_rows(lens, st["read_cu"], st["read_total"])
    pid, row = table[seq, row // st["page"]].long(), row % st["page"]
    return (_values(st["k_pages"][pid, :, row], st["k_scale"][pid, :, row]).to(torch.bfloat16),
            _values(st["v_pages"][pid, :, row], st["v_scale"][pid, :, row]).to(torch.bfloat16))


def _plain_fill(st):
    pos = st["row"] if st["offsets"] is None else st["row"] + st["offsets"].long()[st["seq"]]
    q, k = _rotate(st["q"], pos, st, st["q_weight"]), _rotate(st["k"], pos, st, st["k_weight"])
    _store(k, st["k_pages"], st["k_scale"], st)
    _store(st["v"], st["v_pages"], st["v_scale"], st)
    ks, vs = _read(st, st["table"], st["lens"])
    return {"q": q, "k": k, "k_held": ks, "v_held": vs}


def _gathered(pages, scale, st):
    """All rows of each sequence's table as fp32 [B, Hkv, keys, d]."""
    at = st["table"].clamp(min=0).long()
    if st["kind"] == "bf16":
        x = pages[at].float()
    elif st["kind"] == "e4m3":
        x = pages.view(torch.uint8)[at].view(pages.dtype).float() * scale[at][:, :, :, None, None]
    else:
        x = _values(pages[at], scale[at])
    return x.transpose(1, 2).flatten(2, 3)


def _scores(st, k):
    """Scaled scores [B, Hkv, rows, keys] (row = head of the group, token) and which of them count."""
    q = st["q"].float()
    B, H, n, d = q.shape
    s = (q.reshape(B, st["Hkv"], -1, d) * d ** -0.5) @ k.transpose(-1, -2)
    last = st["lens"][:, None] - n + torch.arange(n, device=q.device)             # [B, n]: last visible key
    vis = torch.arange(k.shape[2], device=q.device) <= last[..., None]            # [B, n, keys]
    return s, vis.repeat(1, H // st["Hkv"], 1)[:, None]


def _plain_decode(st):
    k, v = _gathered(st["k_pages"], st["k_scale"], st), _gathered(st["v_pages"], st["v_scale"], st)
    s, vis = _scores(st, k)
    s.masked_fill_(~vis, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    o = s @ v
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    shape = st["q"].shape
    return o.reshape(shape).to(torch.bfloat16), (m + l.log()).reshape(shape[:3])


def _log_sums(st):
    s, vis = _scores(st, _gathered(st["k_pages"], st["k_scale"], st))
    return torch.logsumexp(s.masked_fill_(~vis, -math.inf), dim=-1).reshape(st["q"].shape[:3])


def _plain_weigh(st):
    s, vis = _scores(st, _gathered(st["k_pages"], st["k_scale"], st))
    lse = st["lse"].reshape(st["B"], st["Hkv"], -1, 1)
    p = s.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    p = p.masked_fill_(~(vis & (lse > -math.inf)), 0.0).sum(dim=2)
    st["weights"] += p[..., :st["max_len"]]
    return st["weights"]


def _plain_evict(st):
    B, Hkv, keep, page = st["B"], st["Hkv"], st["keep"], st["page"]
    w, lens = st["weights"], st["lens"].long()
    j = torch.arange(w.shape[2], device=w.device)
    inside = j < lens[:, None]
    sure = inside & ((j < st["first"]) | (j >= lens[:, None] - st["recent"]) | (lens <= keep)[:, None])
    rank = (inside.int() + sure.int())[:, None].expand_as(w)                       # 2 always kept, 1 by weight, 0 no row
    order = torch.sort(torch.where(torch.isnan(w), -math.inf, w), dim=-1, descending=True, stable=True).indices
    order = order.gather(2, torch.sort(rank.gather(2, order), dim=-1, descending=True, stable=True).indices)
    new_lens = lens.clamp(max=keep)
    i = torch.arange(min(keep, w.shape[2]), device=w.device)
    held = (i < new_lens[:, None])[:, None]                                        # [B, 1, keep]
    at = torch.where(held, order[..., :i.numel()], w.shape[2]).sort(dim=-1).values
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=w.device)
    kept[..., :i.numel()] = torch.where(held, at, -1)
    at = torch.where(held, at, 0)
    weights = torch.zeros(B, Hkv, st["width"], device=w.device)
    weights[..., :i.numel()] = torch.where(held, w.gather(2, at), 0.0)
    # rows: from (page, head, row) to (page, head, row)
    b, h, i = torch.nonzero(held.expand_as(at), as_tuple=True)
    src = at[b, h, i]
    sp, sr, dp, dr = st["table"][b, src // page].long(), src % page, st["new_table"][b, i // page].long(), i % page
    _move(st["k_pages"], st["k_scale"], st["kind"], h, sp, sr, dp, dr)
    _move(st["v_pages"], st["v_scale"], st["kind"], h, sp, sr, dp, dr)
    offsets = st["offsets"] + (lens - new_lens).int()
    out = {"kept": kept, "lens": new_lens.int(), "weights": weights, "offsets": offsets}
    if st["read"]:
        out["k"], out["v"] = _read(st, st["new_table"], out["lens"])
        return out
    return _pool_outputs(st, out)


def _move(pages, scale, kind, h, sp, sr, dp, dr):
    if kind == "e4m3":
        n, heads = scale.shape
        most = torch.zeros(n * heads, device=scale.device).index_reduce_(0, dp * heads + h, scale[sp, h], "amax").view(n, heads)
        x = pages.view(torch.uint8)[sp, h, sr].view(pages.dtype).float() * (scale[sp, h] / most[dp, h])[:, None]
        pages.view(torch.uint8)[dp, h, dr] = x.to(pages.dtype).view(torch.uint8)
        scale.copy_(torch.where(most > 0, most, scale))
        return
    pages[dp, h, dr] = pages[sp, h, sr]
    if kind == "fp4":
        scale[dp, h, dr] = scale[sp, h, sr]


_plain = {"fill": _plain_fill, "decode": _plain_decode, "weigh": _plain_weigh, "evict": _plain_evict}
_own = {"fill": _own_fill, "decode": _own_decode, "weigh": _own_weigh, "evict": _own_evict}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits

def exact(c, seed):
    st = prepare(c, seed)
    d, page, Hkv, B, kind = c["d"], c["page"], c["Hkv"], c["B"], st["kind"]
    dev = "cuda"
    grid = torch.tensor(sorted(set(LEVELS + tuple(-x for x in LEVELS))), dtype=torch.float64, device=dev)
    parity = torch.tensor([1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1], device=dev)   # of the codes: -6 .. 0 .. 6

    def real(name, ids, hk, rows=None):
        """Rows of pages `ids` of one head as 64-bit values [pages, page, d], or row `rows` of each."""
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        pick = (lambda x: x[ids, hk]) if rows is None else (lambda x: x[ids, hk, rows])
        if kind == "bf16":
            return pick(pages).double()
        if kind == "e4m3":
            x = pick(pages.view(torch.uint8)).view(pages.dtype).double()
            return x * scale[ids, hk].double().view(-1, *[1] * (x.dim() - 1))
        byte, s = pick(pages).long(), pick(scale).long()
        x = torch.stack([byte % 16, byte // 16], dim=-1).flatten(-2)
        mag = torch.tensor(LEVELS, dtype=torch.float64, device=dev)[x % 8] * torch.where(x >= 8, -1.0, 1.0)
        e, m = s // 8, (s % 8).double()
        s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 15), m / 8 * 2.0 ** -14)
        return mag * s.repeat_interleave(16, dim=-1)

    def held(x):
        """What a 4-bit row holds of x [..., d] (bf16 values)."""
        z = x.double().unflatten(-1, (-1, 16))
        most = z.abs().amax(dim=-1)
        want = most / 6
        e = torch.floor(torch.log2(want.clamp(min=1e-30))).clamp(min=-14)
        n = want / torch.exp2(e - 3)
        s = (torch.round(n) * torch.exp2(e - 3)).clamp(2.0 ** -17, 10240.0)
        y = z / s[..., None]
        hi = torch.searchsorted(grid, y.contiguous()).clamp(max=14)
        lo = (hi - 1).clamp(min=0)
        up, down = (grid[hi] - y).abs(), (y - grid[lo]).abs()
        v = torch.where((up < down) | ((up == down) & (parity[hi] == 0)), grid[hi], grid[lo])
        return torch.where(most[..., None] > 0, v * s[..., None], 0.0).flatten(-2)

    lens = [L for _, L in _lens(c)]
    if c["op"] == "fill":
        news, rot = [n for n, _ in _lens(c)], c["rot"]
        pos = st["row"] + (0 if st["offsets"] is None else st["offsets"].long()[st["seq"]])
        # the angle from the product mod 2^64: the fraction of a turn that is left
        frac = (pos[:, None] * st["turns"][None, :]).double() / 2.0 ** 64
        spin = torch.polar(torch.ones_like(frac), 2 * math.pi * frac)[:, None]
        one = torch.arange(0, rot, 2, device=dev) if c["inter"] else torch.arange(rot // 2, device=dev)
        two = one + (1 if c["inter"] else rot // 2)
        heads = []
        for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + st["eps"]) * w.double()
            z = torch.complex(x[..., one], x[..., two]) * spin
            y = x.clone()
            y[..., one], y[..., two] = z.real, z.imag
            heads.append(y)
        out = {"q": heads[0], "k": heads[1]}
        at = _cum(news)
        for name, x in (("k", heads[1].to(torch.bfloat16)), ("v", st["v"])):
            new, parts = held(x), []
            for b, (n, L) in enumerate(zip(news, lens)):
                if c["whole"] and L > n:
                    ids = st["table"][b, :(L - n + page - 1) // page].long()
                    old = [real(name, ids, hk).reshape(-1, d)[:L - n] for hk in range(Hkv)]
                    parts.append(torch.stack(old, dim=1))
                parts.append(new[at[b]:at[b + 1]])
            out[name + "_held"] = torch.cat(parts)
        return out

    def scores(b, hk):
        """Scores of the rows of one K/V head (head of the group, token) in 64 bits, -inf where a row does not see a key."""
        L, nq, G = lens[b], c["nq"], c["H"] // Hkv
        ids = st["table"][b, :(L + page - 1) // page].long()
        k = real("k", ids, hk).reshape(-1, d)[:L]
        s = st["q"][b, hk * G:(hk + 1) * G].double().reshape(-1, d) @ k.t() / math.sqrt(d)
        last = (torch.arange(nq, device=dev) + L - nq).repeat(G)
        return s.masked_fill(torch.arange(L, device=dev) > last[:, None], -math.inf), ids

    if c["op"] == "decode":
        G = c["H"] // Hkv
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(st["q"].shape[:3], dtype=torch.float64, device=dev)
        for b in range(B):
            for hk in range(Hkv):
                s, ids = scores(b, hk)
                total = torch.logsumexp(s, dim=-1)
                p = torch.exp(s - torch.where(total == -math.inf, 0.0, total)[:, None])
                o[b, hk * G:(hk + 1) * G] = (p @ real("v", ids, hk).reshape(-1, d)[:lens[b]]).view(G, c["nq"], d)
                lse[b, hk * G:(hk + 1) * G] = total.view(G, c["nq"])
        return o, lse
    if c["op"] == "weigh":
        w = st["weights"].double()
        for b in range(B):
            for hk in range(Hkv):
                s, _ = scores(b, hk)
                G = c["H"] // Hkv
                lse = st["lse"][b, hk * G:(hk + 1) * G].double().reshape(-1, 1)
                w[b, hk, :lens[b]] += torch.exp(s - lse)[lse[:, 0] > -math.inf].sum(dim=0)
        return w

    # evict
    keep, first, recent = c["keep"], c["first"], c["recent"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    weights = torch.zeros(B, Hkv, st["width"], dtype=torch.float64)
    w = st["weights"].double().cpu()
    new_lens = [min(L, keep) for L in lens]
    for b, L in enumerate(lens):
        for hk in range(Hkv):
            rows = list(range(L))
            if L > keep:
                row = w[b, hk, :L].tolist()
                rows = sorted(range(first, L - recent), key=lambda x: (-row[x], x))[:keep - first - recent]
                rows = sorted(rows + list(range(first)) + list(range(L - recent, L)))
            rows = torch.tensor(rows)
            kept[b, hk, :len(rows)] = rows.int()
            weights[b, hk, :len(rows)] = w[b, hk, rows]
    out = {"kept": kept.cuda(), "lens": _i32(new_lens), "weights": weights.cuda(),
           "offsets": st["offsets"] + st["lens"] - _i32(new_lens)}
    moved = {}
    for name in ("k", "v"):
        for b in range(B):
            for hk in range(Hkv):
                at = kept[b, hk, :new_lens[b]].long().cuda()
                moved[name, b, hk] = real(name, st["table"][b, at // page].long(), hk, at % page)
    if c["read"]:
        for name in ("k", "v"):
            out[name] = torch.cat([torch.stack([moved[name, b, hk] for hk in range(Hkv)], dim=1) for b in range(B)])
        return out
    for name in ("k", "v"):
        pages = st[name + "_pages"].double()
        scale = None if kind == "bf16" else st[name + "_scale"].double()
        for b in range(B):
            for hk in range(Hkv):
                old = None if scale is None else st[name + "_scale"][st["table"][b, kept[b, hk, :new_lens[b]].long().cuda() // page].long(), hk].double()
                for p in range((new_lens[b] + page - 1) // page):
                    x = moved[name, b, hk][p * page:(p + 1) * page]
                    pid = int(st["new_table"][b, p])
                    if scale is not None:
                        s = old[p * page:(p + 1) * page].max()
                        scale[pid, hk] = s
                        x = (x / s).to(torch.float8_e4m3fn).double()
                    pages[pid, hk, :x.shape[0]] = x
        out[name + "_pages"] = pages
        if scale is not None:
            out[name + "_scale"] = scale
    return out
