"""The keys of a 4-bit append, bit for bit: every operation from the input to the bf16 key is fixed (fa.h), and a plain fp32
computation of the same steps gives the same keys and so the same codes.

Tolerance. Cosines and sines are off by less than 2^-30 of themselves before they are rounded, half a step of fp32 being
2^-25 or 2^-24 of them: at most 2 * 2^-30 / 2^-24 = 2^-5 of them round to the other neighbour. Each moves a key by at most
a step of fp32 (2^-23 of it), which crosses a border between bf16 values (2^-8 apart) for 2^-15 of the keys; a key has two
products. So at most 2 * 2^-5 * 2^-15 = 2^-19 of the keys differ, by one bf16 step, or, where the two products cancel, by
the products' own: 2 * 2^-23 of a turned pair's length, which is at most twice the row's largest key. The sums of a norm
leave no freedom.
"""

import math

import pytest
import torch

from test_paged_gpu import BASE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def plain_keys(x, pos, turns, inter, weight, eps):
    x = x.float()
    d, rot = x.shape[-1], 2 * turns.numel()
    if weight is not None:
        chain = (x * x).unflatten(-1, (d // 32, 32))
        s = chain[..., 0, :]
        for j in range(1, d // 32):                                 # elements 32 apart in order
            s = s + chain[..., j, :]
        while s.shape[-1] > 1:                                      # then neighbours in pairs
            s = s[..., 0::2] + s[..., 1::2]
        x = x * torch.rsqrt(s / d + eps) * weight.float()
    ang = (pos[:, None] * turns).double() * (2 * math.pi / 2.0 ** 64)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    at = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y, a, b = x.clone(), x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("d,rot,inter,T,Hkv,page", [
    (128, 128, False, 24000, 8, 64), (128, 48, False, 3001, 3, 32), (128, 64, True, 3001, 5, 128), (64, 64, False, 9001, 8, 64),
    (64, 32, True, 3001, 1, 16), (64, 48, False, 777, 2, 128), (128, 128, False, 7, 2, 16)])
def test_keys(fa, d, rot, inter, T, Hkv, page, norm):
    g = torch.Generator(device="cuda").manual_seed(d + rot + T + norm)
    qkv = torch.randn(T, 3 * Hkv, d, device="cuda", generator=g)
    qkv[:, Hkv:2 * Hkv] *= torch.exp2(torch.randint(-3, 5, (Hkv, d), device="cuda", generator=g))
    qkv = qkv.to(torch.bfloat16)
    q, k, v = qkv[:, :Hkv], qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16) if norm else None
    n = (T + page - 1) // page
    pages = [torch.zeros(n, Hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.zeros(n, Hkv, page, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    turns, offset = fa.rotary_turns(rot, BASE), 100003
    _, ko = fa.append_paged_fp4(q, k, v, *pages, *scale, table, torch.tensor([T], dtype=torch.int32, device="cuda"), turns=turns,
                                interleaved=inter, q_weight=w, k_weight=w, eps=1e-6,
                                offsets=torch.tensor([offset], dtype=torch.int32, device="cuda"))
    assert fa.device_status() == fa.FA_OK
    want = plain_keys(k, torch.arange(T, device="cuda") + offset, turns, inter, w, 1e-6)
    off = (ko != want)
    assert int(off.sum()) <= math.ceil(T * Hkv * d * 2.0 ** -19)
    step = torch.maximum(ko.float().abs(), want.float().abs()) * 2.0 ** -7 + 2.0 ** -21 * want.float().abs().amax(dim=-1, keepdim=True)
    assert bool(((ko.float() - want.float()).abs() <= step).all())
