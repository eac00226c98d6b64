"""fp64 oracle of 4-bit rows and of eviction by attention weight (test infrastructure only).

A row is held in groups of 16 neighbours: a scale with 5 exponent bits (bias 15) and 3 mantissa bits, unsigned, and 16
e2m1 codes. ``encode`` finds both by comparing with every representable value, ``decode`` writes the formats out.
"""

from __future__ import annotations

import math

import numpy as np

GROUP = 16
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALE_MIN, SCALE_MAX = 2.0 ** -17, 10240.0


def scale_decode(byte: np.ndarray) -> np.ndarray:
    b = np.asarray(byte).astype(np.int64)
    e, m = b >> 3, (b & 7).astype(np.float64)
    x = np.where(e > 0, (1 + m / 8) * np.exp2(e - 15.0), m / 8 * 2.0 ** -14)
    return np.where(e == 31, np.where(m == 0, np.inf, np.nan), x)


_SCALES = scale_decode(np.arange(248))          # the finite ones, in order


def nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest value of an increasing grid, ties to the even index, clamped to its ends."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x, side="left"), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(grid[hi] - x), np.abs(x - grid[lo])
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def encode(x: np.ndarray):
    """x [..., d] (values of the row's own type) -> codes [..., d] (0 .. 15), scale bytes [..., d / 16]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    fine = np.isfinite(g).all(axis=-1)
    most = np.where(fine, np.abs(np.where(np.isfinite(g), g, 0.0)).max(axis=-1), 0.0)
    byte = nearest_even(most / 6, _SCALES)
    byte = np.clip(byte, 1, int(np.searchsorted(_SCALES, SCALE_MAX)))
    byte = np.where(most == 0, 0, byte)
    s = scale_decode(byte)
    with np.errstate(invalid="ignore", divide="ignore"):
        a = np.where(s[..., None] > 0, np.abs(g) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    code = nearest_even(np.where(np.isfinite(a), a, 0.0), LEVELS) + np.where(np.signbit(g), 8, 0)
    byte = np.where(fine, byte, 0xFF)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def decode(packed: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Rows of bytes [..., d / 2] and [..., d / 16] -> values [..., d]."""
    c = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)
    x = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        return x * np.repeat(scale_decode(scale), GROUP, axis=-1)


def held(x: np.ndarray) -> np.ndarray:
    """What a row holds of x."""
    c, s = encode(x)
    return decode(pack(c), s)


def kept_rows(weights, L: int, keep: int, first: int, recent: int):
    """Rows that stay of one K/V head, in order. weights: a sequence of floats (Python's comparison of each pair)."""
    if L <= keep:
        return list(range(L))
    between = list(range(first, L - recent))
    value = lambda j: -math.inf if math.isnan(weights[j]) else float(weights[j])   # noqa: E731
    chosen = sorted(between, key=lambda j: (-value(j), j))[:keep - first - recent]
    return sorted(list(range(first)) + chosen + list(range(L - recent, L)))


def weigh(q, k_pages, table, lens, lse, scale):
    """q [B,H,Nq,d], pages of real values [pages,Hkv,page,d] -> the weights added, [B][Hkv] arrays of L_b."""
    B, H, Nq, _ = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    out = []
    for b in range(B):
        rows = []
        for hk in range(Hkv):
            k = np.array([k_pages[int(table[b][j // page]), hk, j % page] for j in range(lens[b])]).reshape(lens[b], q.shape[3])
            w = np.zeros(lens[b])
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                for t in range(Nq):
                    n = lens[b] - Nq + t + 1           # keys that the token sees
                    if n > 0 and not np.isneginf(lse[b, h, t]):
                        with np.errstate(invalid="ignore", over="ignore"):
                            w[:n] += np.exp(scale * (k[:n] @ q[b, h, t]) - lse[b, h, t])
            rows.append(w)
        out.append(rows)
    return out
