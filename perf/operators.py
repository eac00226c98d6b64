"""Cases of the serving operators: appending rotated keys and values to a paged cache (`fa.append_paged`), attention of
new tokens over that cache (`fa.decode_paged`) and attention over packed prompts (`fa.fwd_packed`).

Every case is a dict of plain values. `prepare` makes its inputs on the GPU from a seed, `run` makes one pass: the plain
form in elementary torch operations, or (with `own` set) this package's calls. `exact` computes the same outputs in 64
bits, written apart from the plain form.

The operators, in short:

append  Token i of sequence b is at position p = L_b - n_b + i, where n_b tokens are new and L_b counts them too. Each
        head of q and k is normalised, x / sqrt(mean(x^2) + eps) * weight (where weights are given), and its first `rot`
        elements are turned by the angle 2 pi frac(p * turns_j / 2^64) for pair j: elements (j, j + rot / 2) in the half
        layout, (2j, 2j + 1) in the interleaved one. q and k are returned; k and v go to row p % page of page
        table[b, p / page]. An e4m3 cache holds codes with one power-of-two scale for each page and head, the least
        2^e >= 2^-40 with |x| <= 448 * 2^e for the page's rows so far; when a page's scale grows, the codes it already
        holds are rounded again to the new one.
decode  q [B, H, n, d] are the last n positions of each sequence; query head h reads K/V head h / (H / Hkv); token t sees
        key j iff j <= L_b - n + t. A token that sees nothing gets o = 0 and lse = -inf.
packed  Sequence b owns rows cu_q[b] .. cu_q[b + 1] of q and cu_k[b] .. cu_k[b + 1] of k and v; with `causal` its query i
        sees its key j iff j <= i + Lk_b - Lq_b. Rows that see nothing get o = 0 and lse = -inf.
"""

import math
import random

import torch

own = False

E_MIN = -40   # least exponent of a page's scale
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # One decode step of a small batch: eight sequences, one token each, a 16-bit cache. Launch and host latency.
        dict(name="append_step_b8_bf16", op="append", B=8, new_lo=1, new_hi=1, past_lo=40, past_hi=2000, H=16, Hkv=4,
             d=64, page=16, f8=False, rot=64, inter=False, norm=False, uniform=True, lens_seed=1),
        # One decode step of a large batch into an e4m3 cache, with the norms of queries and keys.
        dict(name="append_step_b256_e4m3", op="append", B=256, new_lo=1, new_hi=1, past_lo=100, past_hi=8000, H=32,
             Hkv=8, d=128, page=64, f8=True, rot=128, inter=False, norm=True, uniform=True, lens_seed=2),
        # Prompts of different lengths written to an e4m3 cache, some of them continuing a page begun earlier.
        dict(name="append_prompts_e4m3", op="append", B=12, new_lo=1, new_hi=4096, past_lo=0, past_hi=500, H=32, Hkv=8,
             d=128, page=64, f8=True, rot=128, inter=False, norm=True, uniform=False, lens_seed=3),
        # Chunks of long prompts, far positions, half of each head rotated in the interleaved layout, a 16-bit cache.
        dict(name="append_chunks_bf16_partial", op="append", B=9, new_lo=500, new_hi=2048, past_lo=0, past_hi=500000,
             H=28, Hkv=4, d=128, page=32, f8=False, rot=64, inter=True, norm=False, uniform=False, lens_seed=4),
        # One user, a short context: the latency of a single decode step.
        dict(name="decode_b1_short_e4m3", op="decode", B=1, H=32, Hkv=8, d=128, nq=1, page=16, f8=True, len_lo=700,
             len_hi=700, lens_seed=5),
        # A serving batch, ragged lengths of the grouped-decode benchmark, e4m3 pages.
        dict(name="decode_b64_ragged_e4m3", op="decode", B=64, H=32, Hkv=8, d=128, nq=1, page=64, f8=True, len_lo=4096,
             len_hi=8192, lens_seed=6),
        # Four new tokens a sequence (a draft being checked), a 16-bit cache, d = 64.
        dict(name="decode_b48_nq4_bf16_d64", op="decode", B=48, H=32, Hkv=8, d=64, nq=4, page=32, f8=False, len_lo=5,
             len_hi=8192, lens_seed=7),
        # Two users with very long contexts: the keys of one sequence are shared out over the whole GPU.
        dict(name="decode_b2_long_e4m3", op="decode", B=2, H=32, Hkv=8, d=128, nq=1, page=128, f8=True, len_lo=90001,
             len_hi=131072, lens_seed=8),
        # A few short prompts: latency.
        dict(name="packed_short_d64", op="packed", B=5, H=16, Hkv=4, d=64, lq_lo=1, lq_hi=190, lk_more=0, causal=True,
             lens_seed=9),
        # An ordinary prefill batch of ragged prompts.
        dict(name="packed_ragged_d128", op="packed", B=8, H=32, Hkv=8, d=128, lq_lo=200, lq_hi=2048, lk_more=0,
             causal=True, lens_seed=10),
        # Chunks of prompts behind prefixes that were computed before; an odd group of five heads.
        dict(name="packed_prefix_g5_d128", op="packed", B=6, H=20, Hkv=4, d=128, lq_lo=100, lq_hi=1024, lk_more=2500,
             causal=True, lens_seed=11),
        # Two long prompts.
        dict(name="packed_long_d128", op="packed", B=2, H=32, Hkv=8, d=128, lq_lo=7000, lq_hi=8192, lk_more=0,
             causal=True, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "packed"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    seed = rng.randrange(1 << 30)
    if op == "append":
        B = _log(rng, 1, 256)
        uniform = rng.random() < 0.5
        if uniform:
            lo = hi = rng.choice([1, 1, 2, 3, 5])
        else:
            lo, hi = 1, _log(rng, 2, max(2, 24000 // B))
        rot = rng.choice([d, d, d // 2, 16, 48])
        return dict(op=op, B=B, new_lo=lo, new_hi=hi, past_lo=0, past_hi=_log(rng, 10, 400000), H=Hkv * G, Hkv=Hkv, d=d,
                    page=rng.choice([16, 32, 64, 128]), f8=rng.random() < 0.6, rot=rot, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.5, uniform=uniform, lens_seed=seed)
    if op == "decode":
        B = _log(rng, 1, 96)
        f8 = rng.random() < 0.6
        hi = _log(rng, 20, min(131072, (390000 if f8 else 190000) // B))
        nq = rng.choice([1, 1, 1, 2, 3, 5])
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, nq=nq, page=rng.choice([16, 32, 64, 128]), f8=f8,
                    len_lo=max(1, hi // rng.choice([1, 2, 50])), len_hi=hi, lens_seed=seed)
    B = _log(rng, 1, 40)
    hi = _log(rng, 16, min(8192, int(math.sqrt(1.9e9 / (B * Hkv * G)))))
    more = rng.choice([0, 0, hi // 2])
    if more:
        hi = max(8, hi // 2)
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, lq_lo=1, lq_hi=hi, lk_more=more, causal=rng.random() < 0.8,
                lens_seed=seed)


def _lens(c):
    """The case's lengths, a list for each sequence: (n, L) of append, L of decode, (Lq, Lk) of packed."""
    rng = random.Random(c["lens_seed"])
    out = []
    for _ in range(c["B"]):
        if c["op"] == "append":
            n = rng.randint(c["new_lo"], c["new_hi"])
            out.append((n, n + rng.randint(c["past_lo"], c["past_hi"])))
        elif c["op"] == "decode":
            out.append(rng.randint(c["len_lo"], c["len_hi"]))
        else:
            lq = rng.randint(c["lq_lo"], c["lq_hi"])
            out.append((lq, lq + (rng.randint(0, c["lk_more"]) if c["lk_more"] else 0)))
    return out


def _cum(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _pairs(lq, lk, causal):
    """Visible (query, key) pairs of one head of one sequence (lk >= lq)."""
    return lq * lk - (lq * (lq - 1) // 2 if causal else 0)


def work(c):
    lens = _lens(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] == "append":
        T = sum(n for n, _ in lens)
        kv = 1 if c["f8"] else 2
        # q read and written, k read and written (for the prompt's own attention), v read, the cache rows written
        nbytes = T * d * (2 * 2 * H + 2 * 2 * Hkv + 2 * Hkv + 2 * Hkv * kv)
        return {"bytes": nbytes, "flops": T * (H + Hkv) * (3 * c["rot"] + (4 * d if c["norm"] else 0))}
    if c["op"] == "decode":
        esz = 1 if c["f8"] else 2
        nbytes = sum(lens) * Hkv * d * 2 * esz + 2 * c["B"] * H * c["nq"] * d * 2 + c["B"] * H * c["nq"] * 4
        flops = sum(4 * H * d * sum(max(0, L - c["nq"] + t + 1) for t in range(c["nq"])) for L in lens)
        return {"bytes": nbytes, "flops": flops}
    tq, tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    nbytes = 2 * tq * H * d * 2 + 2 * tk * Hkv * d * 2 + tq * H * 4
    return {"bytes": nbytes, "flops": sum(4 * H * d * _pairs(a, b, c["causal"]) for a, b in lens)}


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


def _exponents(amax):
    """Least e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9), elementwise; E_MIN for amax = 0."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _page_pool(n, Hkv, page, d, f8, g):
    """Pages that hold earlier tokens: bf16 values, or e4m3 codes and scales. Keys and values of different pages differ
    in magnitude, as they do between layers' outliers and ordinary tokens."""
    x = torch.randn(n, Hkv, page, d, device="cuda", generator=g)
    if not f8:
        return x.to(torch.bfloat16), None
    x = x * torch.exp2(torch.randn(n, Hkv, 1, 1, device="cuda", generator=g) * 0.7)
    s = torch.exp2(_exponents(x.abs().amax(dim=(2, 3))).float())
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    lens = _lens(c)
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    st = dict(c)
    if c["op"] == "packed":
        st["cu_q"], st["cu_k"] = _i32(_cum([a for a, _ in lens])), _i32(_cum([b for _, b in lens]))
        tq, tk = sum(a for a, _ in lens), sum(b for _, b in lens)
        st["q"], st["k"], st["v"] = rand(tq, H, d), rand(tk, Hkv, d), rand(tk, Hkv, d)
        st["max_q"], st["max_k"] = max(a for a, _ in lens), max(b for _, b in lens)
        return st
    page = c["page"]
    ends = lens if c["op"] == "decode" else [L for _, L in lens]
    # pages that the call touches: all of a sequence's for decode, those from its first new token on for append
    first = [0 if c["op"] == "decode" else (L - n) // page for (n, L) in (lens if c["op"] == "append" else [(L, L) for L in lens])]
    count = [(L + page - 1) // page for L in ends]
    need = sum(k - f for k, f in zip(count, first))
    pool = need + 3
    ids = list(range(pool))
    rng.shuffle(ids)
    width = max(1, max(count))
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        k = count[b] - first[b]
        table[b, first[b]:count[b]] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    st["table"], st["lens"] = table.cuda(), _i32(ends)
    st["max_len"] = max(ends)
    st["k_pages"], st["k_scale"] = _page_pool(pool, Hkv, page, d, c["f8"], g)
    st["v_pages"], st["v_scale"] = _page_pool(pool, Hkv, page, d, c["f8"], g)
    if c["op"] == "decode":
        # token-major memory, as the append returns it, seen as [B, H, nq, d]
        st["q"] = rand(B, c["nq"], H, d).transpose(1, 2)
        return st
    n = [a for a, _ in lens]
    T = sum(n)
    qkv = rand(T, H + 2 * Hkv, d)  # one projection's output; q, k and v are views of it
    st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    st["cu"] = None if c["uniform"] else _i32(_cum(n))
    st["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
    st["start"] = torch.tensor([L - a for a, L in lens], dtype=torch.int64, device="cuda")
    st["pos"] = torch.cat([torch.arange(L - a, L, device="cuda") for a, L in lens])
    st["max_new"] = max(n)
    st["turns"] = _turns(c["rot"])
    st["q_weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16) if c["norm"] else None
    st["k_weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16) if c["norm"] else None
    st["eps"] = 1e-6
    st["q_out"] = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda")
    st["k_out"] = torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass

def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _own_append(st):
    from io_aware_exact_fa_gb300 import fa
    q, k = fa.append_paged(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                           cu_seqlens=st["cu"], max_new=st["max_new"], turns=st["turns"], interleaved=st["inter"],
                           q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"], k_scale=st["k_scale"],
                           v_scale=st["v_scale"], q_out=st["q_out"], k_out=st["k_out"])
    return _append_outputs(st, q, k)


def _append_outputs(st, q, k):
    # An e4m3 cache comes back as its codes' values (float8) beside the power-of-two scales they count in.
    out = {"q": q, "k": k, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if st["f8"]:
        out["k_scale"], out["v_scale"] = st["k_scale"], st["v_scale"]
    return out


def _own_decode(st):
    from io_aware_exact_fa_gb300 import fa
    if "ws" not in st:  # a serving program keeps its workspace
        st["ws"] = torch.empty(max(1, fa.decode_paged_workspace_size(st["B"], st["H"], st["Hkv"], st["nq"], st["d"],
                                                                     st["max_len"])), dtype=torch.uint8, device="cuda")
    return fa.decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], k_scale=st["k_scale"],
                           v_scale=st["v_scale"], max_len=st["max_len"], workspace=st["ws"])


def _own_packed(st):
    from io_aware_exact_fa_gb300 import fa
    if "ws" not in st:
        st["ws"] = torch.empty(fa.fwd_packed_workspace_size(st["B"], st["q"].shape[0], st["H"], st["Hkv"]),
                               dtype=torch.uint8, device="cuda")
    return fa.fwd_packed(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], causal=st["causal"], workspace=st["ws"])


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
    if st["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _store(x, pages, scale, st):
    """Writes x [T, Hkv, d] (fp32) to the cache."""
    page, pos, seq = st["page"], st["pos"], st["seq"]
    pid = st["table"][seq, pos // page].long()
    row = pos % page
    if scale is None:
        pages[pid, :, row] = x.to(torch.bfloat16)
        return
    # largest magnitude of the new rows of each page, and of what the sequence's first page held before
    new = torch.zeros_like(scale).index_reduce_(0, pid, x.abs().amax(dim=-1), "amax")
    e = _exponents(new)
    begun = st["start"] % page                                      # rows of the first page held before
    p0 = st["table"].gather(1, (st["start"] // page)[:, None])[:, 0].long()
    old = torch.frexp(scale[p0]).exponent - 1
    merged = torch.where((begun > 0)[:, None], torch.maximum(e[p0], old), e[p0])
    e[p0] = merged
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, pid, True)
    raw = pages.view(torch.uint8)
    rows = torch.arange(page, device=x.device)
    held = (rows[None, :] < begun[:, None])[:, None, :, None]
    grown = pages[p0].float() * torch.exp2((old - merged).float())[:, :, None, None]
    raw[p0] = torch.where(held, grown.to(torch.float8_e4m3fn).view(torch.uint8), raw[p0])
    scale.copy_(torch.where(touched[:, None], torch.exp2(e.float()), scale))
    raw[pid, :, row] = (x / scale[pid][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(st):
    q = _rotate(st["q"], st["pos"], st, st["q_weight"])
    k = _rotate(st["k"], st["pos"], st, st["k_weight"])
    _store(k, st["k_pages"], st["k_scale"], st)
    _store(st["v"].float(), st["v_pages"], st["v_scale"], st)
    return _append_outputs(st, q.to(torch.bfloat16), k.to(torch.bfloat16))


def _attend(s, vis, v):
    """softmax over the visible entries of s [..., r, n] times v [..., n, d], and the log of the sum; zero and -inf
    where a row sees nothing. s is overwritten."""
    s.masked_fill_(~vis, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    o = s @ v
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o, (m + l.log())[..., 0]


def _gathered(pages, scale, table):
    B, width = table.shape
    _, Hkv, page, d = pages.shape
    at = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[at].view(pages.dtype).float() if scale is not None else pages[at].float()
    if scale is not None:
        x = x * scale[at][:, :, :, None, None]
    return x.transpose(1, 2).reshape(B, Hkv, width * page, d)


def _plain_decode(st):
    q = st["q"].float()
    B, H, n, d = q.shape
    Hkv = st["Hkv"]
    k, v = _gathered(st["k_pages"], st["k_scale"], st["table"]), _gathered(st["v_pages"], st["v_scale"], st["table"])
    s = (q.reshape(B, Hkv, (H // Hkv) * n, d) * d ** -0.5) @ k.transpose(-1, -2)
    last = st["lens"][:, None] - n + torch.arange(n, device=q.device)             # [B, n]: last visible key
    vis = torch.arange(k.shape[2], device=q.device) <= last[..., None]            # [B, n, keys]
    vis = vis.repeat(1, H // Hkv, 1)[:, None]
    o, lse = _attend(s, vis, v)
    return o.reshape(B, H, n, d).to(torch.bfloat16), lse.reshape(B, H, n)


def _plain_packed(st):
    # padded to the longest sequence: [B, heads, rows, d]
    H, Hkv, d, B = st["H"], st["Hkv"], st["d"], st["B"]
    Lq, Lk = st["max_q"], st["max_k"]
    iq, ik = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    nq, nk = st["cu_q"].diff()[:, None], st["cu_k"].diff()[:, None]
    in_q, in_k = iq < nq, ik < nk                                                 # [B, L]
    at_q = torch.where(in_q, st["cu_q"][:-1, None] + iq, 0)
    at_k = torch.where(in_k, st["cu_k"][:-1, None] + ik, 0)
    q = st["q"][at_q].float().transpose(1, 2).reshape(B, Hkv, H // Hkv * Lq, d)
    k = st["k"][at_k].float().transpose(1, 2)
    v = st["v"][at_k].float().transpose(1, 2)
    s = ((q * d ** -0.5) @ k.transpose(-1, -2)).view(B, Hkv, H // Hkv, Lq, Lk)
    vis = in_k[:, None, :] & in_q[:, :, None]
    if st["causal"]:
        vis = vis & (ik <= iq[:, None] + (nk - nq)[:, :, None])
    vis = vis[:, None, None]
    s.masked_fill_(~vis, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    o = (s.view(B, Hkv, H // Hkv * Lq, Lk) @ v).view(B, H, Lq, d)
    l, m = l.view(B, H, Lq, 1), m.view(B, H, Lq, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    return o.transpose(1, 2)[in_q].to(torch.bfloat16), lse.transpose(1, 2)[in_q].t().contiguous()


_plain = {"append": _plain_append, "decode": _plain_decode, "packed": _plain_packed}
_own = {"append": _own_append, "decode": _own_decode, "packed": _own_packed}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits

def exact(c, seed):
    st = prepare(c, seed)
    return {"append": _exact_append, "decode": _exact_decode, "packed": _exact_packed}[c["op"]](c, st)


def _rows(q, k, v, last):
    """Attention of one head: row i of q [r, d] sees keys 0 .. last[i] of k and v (all in 64 bits)."""
    s = (q @ k.t()) / math.sqrt(q.shape[-1])
    s = torch.where(torch.arange(k.shape[0], device=k.device)[None, :] > last[:, None], torch.full_like(s, -math.inf), s)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.where(torch.isinf(lse)[:, None], torch.zeros_like(s), torch.exp(s - lse[:, None]))
    return p @ v, lse


def _exact_packed(c, st):
    cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["H"], st["q"].shape[0], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        a0, a1, b0, b1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        last = torch.arange(a1 - a0, device="cuda") + (b1 - b0) - (a1 - a0)
        if not c["causal"]:
            last = torch.full_like(last, b1 - b0)
        for h in range(c["H"]):
            kh = h // (c["H"] // c["Hkv"])
            o[a0:a1, h], lse[h, a0:a1] = _rows(st["q"][a0:a1, h].double(), st["k"][b0:b1, kh].double(),
                                               st["v"][b0:b1, kh].double(), last)
    return o, lse


def _exact_decode(c, st):
    page, nq = c["page"], c["nq"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, L in enumerate(st["lens"].tolist()):
        ids = st["table"][b, :(L + page - 1) // page].long()
        last = torch.arange(L - nq, L, device="cuda")
        for kh in range(c["Hkv"]):
            kv = []
            for pages, scale in ((st["k_pages"], st["k_scale"]), (st["v_pages"], st["v_scale"])):
                x = (pages[:, kh].view(torch.uint8)[ids].view(pages.dtype) if c["f8"] else pages[:, kh][ids]).double()
                if c["f8"]:
                    x = x * scale[ids, kh].double()[:, None, None]
                kv.append(x.reshape(-1, c["d"])[:L])
            for h in range(kh * (c["H"] // c["Hkv"]), (kh + 1) * (c["H"] // c["Hkv"])):
                o[b, h], lse[b, h] = _rows(st["q"][b, h].double(), kv[0], kv[1], last)
    return o, lse


def _exact_append(c, st):
    page, rot, d = c["page"], c["rot"], c["d"]
    # the angle from the product mod 2^64: the fraction of a turn that is left
    frac = (st["pos"][:, None] * st["turns"][None, :]).double() / 2.0 ** 64
    cos, sin = torch.cos(2 * math.pi * frac)[:, None], torch.sin(2 * math.pi * frac)[:, None]
    first = torch.arange(0, rot, 2, device="cuda") if c["inter"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if c["inter"] else rot // 2)
    heads = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + st["eps"]) * w.double()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos, sin)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        heads.append(y)
    q, k = heads
    out = {"q": q, "k": k}
    lens = _lens(c)
    cu = _cum([n for n, _ in lens])
    for name, x in (("k", k), ("v", st["v"].double())):
        pages, scale = st[name + "_pages"].double(), st[name + "_scale"]
        if scale is not None:
            scale = scale.double()
        table = st["table"].tolist()
        for b, (n, L) in enumerate(lens):
            p = L - n
            while p < L:  # page by page
                end = min(L, (p // page + 1) * page)
                pid, r0 = table[b][p // page], p % page
                new = x[cu[b] + p - (L - n):cu[b] + end - (L - n)].transpose(0, 1)     # [Hkv, rows, d]
                if scale is None:
                    pages[pid, :, r0:r0 + end - p] = new
                else:
                    need = new.abs().amax(dim=(1, 2)) / E4M3_MAX
                    s = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** E_MIN))))
                    if r0 > 0:
                        s = torch.maximum(s, scale[pid])
                        held = pages[pid, :, :r0] * (scale[pid] / s)[:, None, None]
                        pages[pid, :, :r0] = held.to(torch.float8_e4m3fn).double()
                    scale[pid] = s
                    pages[pid, :, r0:r0 + end - p] = (new / s[:, None, None]).to(torch.float8_e4m3fn).double()
                p = end
        out[name + "_pages"] = pages
        if scale is not None:
            out[name + "_scale"] = scale
    return out
