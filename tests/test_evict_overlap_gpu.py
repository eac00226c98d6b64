"""Evicted weights beside the weights that are read: columns of one buffer are taken, overlapping ones refused."""

import pytest
import torch

from oracle import fp4 as F4
from test_paged_gpu import cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


@pytest.mark.parametrize("B,Hkv", [(2, 3), (1, 1)])
def test_columns_of_one_buffer(fa, B, Hkv):
    L, keep, page, d = 60, 20, 16, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.rand(B, Hkv, 64 + 32, device="cuda", generator=g)
    w = big[..., :64].clone()
    pools = [torch.randn(B * 6, Hkv, page, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    new = torch.arange(B * 4, B * 6, dtype=torch.int32, device="cuda").view(B, 2)
    lens = cuda([L] * B, torch.int32)
    args = (*pools, table, lens, new, keep)
    for bad in (big[..., 60:92], big[..., 1:33], big[..., 44:76]):
        if B * Hkv > 1 or bad.data_ptr() < big[..., 64:].data_ptr():
            with pytest.raises(fa.FAError):
                fa.evict_paged(big[..., :64], *args, new_weights=bad)
    assert torch.equal(big[..., :64], w)
    kept, _, nw, _ = fa.evict_paged(big[..., :64], *args, new_weights=big[..., 64:])
    assert fa.device_status() == fa.FA_OK and torch.equal(big[..., :64], w)
    for b in range(B):
        for h in range(Hkv):
            rows = F4.kept_rows(w[b, h].tolist(), L, keep, 0, 0)
            assert kept[b, h].tolist() == rows and torch.equal(nw[b, h, :keep], w[b, h, rows]) and (nw[b, h, keep:] == 0).all()
