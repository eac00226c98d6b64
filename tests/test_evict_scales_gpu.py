"""Eviction from e4m3 pages whose scales are no powers of two, or 0.

Tolerance: code * (old / new) has two roundings of fp32, 2^-24 of it each, before the one to e4m3. So a code is that of the
exact value, or of one within 2^-22 of it (a border between codes lies between them)."""

import numpy as np
import pytest
import torch

from oracle import fp4 as F4
from oracle import fp8 as FP8
from oracle import paged as OP
from test_paged_gpu import cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def cut(fa, codes, scales, L, keep, page, seed):
    """Evicts from one sequence on the pages 0 ..; (weights, kept rows, pools, new pages' first)."""
    n = codes[0].shape[0]
    Hkv, count = codes[0].shape[1], (L + page - 1) // page
    w = torch.rand(1, Hkv, L, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    pools = [torch.from_numpy(c).cuda() for c in codes]
    sc = [cuda(s, torch.float32) for s in scales]
    table = torch.arange(count, dtype=torch.int32, device="cuda")[None]
    new = torch.arange(count, n, dtype=torch.int32, device="cuda")[None]
    kept, _, _, _ = fa.evict_paged(w, *pools, table, cuda([L], torch.int32), new, keep, k_scale=sc[0], v_scale=sc[1])
    assert fa.device_status() == fa.FA_OK
    for h in range(Hkv):
        assert kept[0, h].tolist() == F4.kept_rows(w[0, h].tolist(), L, keep, 0, 0)
    return kept[0].cpu().numpy(), [x.cpu().numpy() for x in pools], [x.cpu().numpy() for x in sc], count


@pytest.mark.parametrize("d,page,spread", [(64, 16, 1.0), (128, 64, 1.0), (128, 16, 14.0), (64, 32, 25.0)])
def test_any_scales(fa, d, page, spread):
    rng = np.random.default_rng(d + page)
    L, keep, Hkv = 2000, 700, 3
    n = (L + page - 1) // page + (keep + page - 1) // page
    codes = [rng.integers(0, 256, (n, Hkv, page, d)).astype(np.uint8) for _ in range(2)]      # (NaN codes among them)
    scales = [np.exp2(-spread * rng.random((n, Hkv))).astype(np.float32) for _ in range(2)]
    kept, got, sc, first = cut(fa, codes, scales, L, keep, page, 1)
    for x in range(2):
        for h in range(Hkv):
            for p0 in range(0, keep, page):
                rows = kept[h, p0:p0 + page]
                old = scales[x][rows // page, h].astype(np.float64)
                assert sc[x][first + p0 // page, h] == old.max()
                src = codes[x][rows // page, h, rows % page]
                v = FP8.e4m3_decode(src) * (old / old.max())[:, None]
                y = got[x][first + p0 // page, h, :len(rows)]
                near = [OP.e4m3_encode(v * f) for f in (1.0, 1 - 2.0 ** -22, 1 + 2.0 ** -22)]
                nan = np.isnan(v)
                assert np.array_equal(np.isnan(FP8.e4m3_decode(y)), nan)
                ok = (y == near[0]) | (y == near[1]) | (y == near[2]) | nan
                ok |= (FP8.e4m3_decode(y) == 0) & (FP8.e4m3_decode(near[0]) == 0)              # (a zero's sign)
                same = (old == old.max())[:, None]
                assert np.all(np.where(same, y == src, ok))


def test_scales_of_zero(fa):
    """A new page whose rows all have scale 0 keeps their codes and a scale of 0 (read as zeros); among others' rows they are 0."""
    rng = np.random.default_rng(4)
    page, d, Hkv, L, keep = 16, 64, 2, 96, 64
    codes = [rng.integers(0, 0x7f, (10, Hkv, page, d)).astype(np.uint8) for _ in range(2)]
    scales = [np.zeros((10, Hkv), dtype=np.float32) for _ in range(2)]
    scales[1][4:, 1] = 0.3                                              # values of head 1: its last rows are not zero
    kept, got, sc, first = cut(fa, codes, scales, L, keep, page, 2)
    for x in range(2):
        for h in range(Hkv):
            for i, j in enumerate(kept[h]):
                y, dst = got[x][first + i // page, h, i % page], first + i // page
                if sc[x][dst, h] == 0 or scales[x][j // page, h] > 0:
                    assert np.array_equal(y, codes[x][j // page, h, j % page])
                else:
                    assert (y == 0).all()
    assert (sc[0][first:, 0] == 0).all() and (sc[1][first:, 1] != 0).any()
