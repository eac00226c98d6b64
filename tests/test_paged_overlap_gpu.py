"""Reads launched beside the tail of the append that writes their rows, over caches of every kind: rows, and the scales that
blocks of other pages and heads write to the same 32 bytes, are those that the append left."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


@pytest.mark.parametrize("Hkv,page", [(2, 16), (4, 64)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_a_captured_append_and_its_read(fa, kind, Hkv, page):
    d, H, B = 128, 2 * Hkv, 70
    g = torch.Generator(device="cuda").manual_seed(page)
    lens = torch.randint(250, 700, (B,), device="cuda", generator=g).int()
    new = torch.minimum(torch.randint(1, 300, (B,), device="cuda", generator=g).int(), lens)      # most begin inside a page
    width = (int(lens.max()) + page - 1) // page
    n = B * width
    table = torch.randperm(n, device="cuda", generator=g).int().view(B, width)
    T, total = int(new.sum()), int(lens.sum())
    assert total >= 512 * 32                                                                    # a read of over 512 blocks
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0)).int()
    rcu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int()
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if kind == "bf16":
        base = [rand(n, Hkv, page, d).to(torch.bfloat16) for _ in range(2)]
    elif kind == "e4m3":
        base = [rand(n, Hkv, page, d).to(torch.float8_e4m3fn) for _ in range(2)]
        base += [torch.exp2(torch.randint(-9, -4, (n, Hkv), device="cuda", generator=g).float()) for _ in range(2)]
    else:
        base = [torch.randint(0, 256, (n, Hkv, page, d // 2), device="cuda", generator=g).to(torch.uint8) for _ in range(2)]
        base += [torch.randint(40, 90, (n, Hkv, page, d // 16), device="cuda", generator=g).to(torch.uint8) for _ in range(2)]
    pool = [x.clone() for x in base]
    scales = dict(zip(("k_scale", "v_scale"), pool[2:]))
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    turns = fa.rotary_turns(d)

    def append():
        if kind == "fp4":
            return fa.append_paged_fp4(q, k, v, *pool, table, lens, cu_seqlens=cu, turns=turns)
        return fa.append_paged(q, k, v, *pool[:2], table, lens, cu_seqlens=cu, max_new=300, turns=turns, **scales)

    def read():
        return fa.read_paged(*pool[:2], table, lens, rcu, total, **scales)

    append()
    read()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append()
        got = read()
    for size in (1.0, 30.0, 0.1, 5.0, 300.0, 1.0):                  # scales grow in some pages and are kept in others
        for x in (q, k, v):
            x.copy_((rand(*x.shape) * size).to(torch.bfloat16))
        for x, y in zip(pool, base):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        once = [x.clone() for x in got]
        held = [x.clone() for x in pool]
        for x, y in zip(pool, base):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        torch.cuda.synchronize()
        append()
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(pool, held))
        for a, b in zip(once, read()):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert fa.device_status() == fa.FA_OK
