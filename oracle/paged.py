"""fp64 oracle of the paged serving operators (test infrastructure only).

``append`` writes out, token by token, what a step does to its projections and
to the cache: the norm of each head, the rotation of its pairs by the position,
and the row of the page that holds the position. ``attend`` gathers a sequence's
rows back and calls the pinned forward definition. ``packed`` calls it once per
sequence and head of a packed batch.
"""

from __future__ import annotations

import math

import numpy as np

from . import attention as A
from . import fp8 as FP8

E_MIN = -40
_CODES = np.arange(127, dtype=np.uint8)             # the non-negative finite codes, in order of value
_VALUES = FP8.e4m3_decode(_CODES)


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code (ties to the even one) of |x| <= 448; the NaN code for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(_VALUES, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _VALUES[hi] - a, a - _VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code = code | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """Least e >= E_MIN with amax <= 448 * 2**e."""
    e = E_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def turn(x: np.ndarray, pos: int, turns, interleaved: bool, rot_scale: float = 1.0) -> np.ndarray:
    """One head [d] with its first 2 * len(turns) elements turned for position pos (Python integers: exact)."""
    y = np.array(x, dtype=np.float64)
    n = len(turns)
    for j, t in enumerate(turns):
        ang = 2.0 * math.pi * (((int(pos) * int(t)) % (1 << 64)) / 2.0 ** 64)
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        c, s = math.cos(ang), math.sin(ang)
        y[ia], y[ib] = rot_scale * (x[ia] * c - x[ib] * s), rot_scale * (x[ib] * c + x[ia] * s)
    return y


def head_norm(x: np.ndarray, w, eps: float) -> np.ndarray:
    return x if w is None else x / math.sqrt(float(np.mean(x * x)) + eps) * w


def append(q, k, v, new, lens, turns, interleaved, q_w=None, k_w=None, eps=1e-6, rot_scale=1.0):
    """q [T,H,d], k, v [T,Hkv,d] fp64, new tokens and lengths per sequence -> turned q, k (fp64) and the position
    of every token."""
    oq, ok, pos = np.array(q), np.array(k), []
    t = 0
    for n, L in zip(new, lens):
        for i in range(n):
            p = L - n + i
            pos.append(p)
            for h in range(q.shape[1]):
                oq[t, h] = turn(head_norm(q[t, h], q_w, eps), p, turns, interleaved, rot_scale)
            for h in range(k.shape[1]):
                ok[t, h] = turn(head_norm(k[t, h], k_w, eps), p, turns, interleaved, rot_scale)
            t += 1
    return oq, ok, pos


def store_e4m3(x, new, lens, table, page, codes, scale):
    """Appends x [T,Hkv,d] fp64 to codes [pages,Hkv,page,d] uint8 and scale [pages,Hkv] (both changed in place)."""
    t = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        p = L - n
        while p < L:
            end = min(L, (p // page + 1) * page)
            pid, r0 = int(table[b][p // page]), p % page
            for h in range(x.shape[1]):
                rows = x[t:t + end - p, h]
                fin = np.abs(rows[np.isfinite(rows)])
                s = 2.0 ** scale_exponent(float(fin.max(initial=0.0)))
                if r0 > 0:
                    old = float(scale[pid, h])
                    s = max(s, old)
                    if s != old:
                        held = FP8.e4m3_decode(codes[pid, h, :r0]) * (old / s)
                        codes[pid, h, :r0] = e4m3_encode(held)
                scale[pid, h] = s
                with np.errstate(invalid="ignore"):
                    codes[pid, h, r0:r0 + end - p] = e4m3_encode(rows / s)
            t += end - p
            p = end


def gather(pages, table_row, L, h):
    """Rows 0 .. L-1 of K/V head h from pages [pages,Hkv,page,d] (real values)."""
    page = pages.shape[2]
    out = [pages[int(table_row[i // page]), h, i % page] for i in range(L)]
    return np.array(out).reshape(L, pages.shape[3])


def attend(q, k_pages, v_pages, table, lens, scale):
    """q [B,H,Nq,d]: the last Nq tokens of each sequence; pages hold real values. -> o, lse."""
    B, H, Nq, d = q.shape
    Hkv = k_pages.shape[1]
    o, lse = np.zeros((B, H, Nq, d)), np.full((B, H, Nq), -np.inf)
    for b in range(B):
        for h in range(H):
            hk = h // (H // Hkv)
            if lens[b] > 0:
                o[b, h], lse[b, h] = A.attend_head(q[b, h], gather(k_pages, table[b], lens[b], hk),
                                                   gather(v_pages, table[b], lens[b], hk), scale, True)
    return o, lse


def packed(q, k, v, cu_q, cu_k, scale, causal):
    """q [Tq,H,d], k, v [Tk,Hkv,d] -> o [Tq,H,d], lse [H,Tq]."""
    o, lse = np.zeros(q.shape), np.full((q.shape[1], q.shape[0]), -np.inf)
    G = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        a0, a1, b0, b1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        for h in range(q.shape[1]):
            if a1 > a0 and b1 > b0:
                o[a0:a1, h], lse[h, a0:a1] = A.attend_head(q[a0:a1, h], k[b0:b1, h // G], v[b0:b1, h // G], scale, causal)
    return o, lse
