"""The device-checking build on packed batches: every TMA coordinate, TMEM range
and barrier phase count of the packed prefill kernel checks out on ragged
sequences (empty ones, rows that see no key, tiles without rows, several units a
CTA), and the outputs are the release library's bits."""

import ctypes
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_fa_gb300 import build
    build.build()
    build.build(debug=True)
    from io_aware_exact_fa_gb300 import fa
    return fa, fa.lib, fa.debug_library()


def _run(lib, q, k, v, cu_q, cu_k, ws, causal):
    (Tq, H, d), (Tk, Hkv, _) = q.shape, k.shape
    o = torch.full_like(q, 7.0)
    lse = torch.full((H, Tq), 7.0, device="cuda")
    st = (ctypes.c_int64 * 8)(H * d, d, Hkv * d, d, Hkv * d, d, H * d, d)
    rc = lib.fa_fwd_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), st, cu_q.data_ptr(),
                           cu_k.data_ptr(), cu_q.numel() - 1, Tq, Tk, H, Hkv, d, 1 / math.sqrt(d), int(causal),
                           ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, lib.fa_last_error_detail()
    torch.cuda.synchronize()
    return o, lse


def _record(lib):
    out = (ctypes.c_uint32 * 8)()
    assert lib.fa_debug_record(out, None) == 0
    return list(out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk,H,Hkv,causal", [
    ([5, 0, 190, 127, 129], [5, 0, 190, 127, 129], 8, 2, True),
    ([200, 130, 3], [70, 0, 2], 4, 2, True),
    ([260, 513, 1], [300, 600, 700], 6, 2, False),
    ([40, 300] * 150, [50, 200] * 150, 3, 1, True),
])
def test_debug_build_packed(libs, lq, lk, H, Hkv, causal, d):
    fa, rel, dbg = libs
    cu = [torch.tensor([0] + np.cumsum(x).tolist(), dtype=torch.int32, device="cuda") for x in (lq, lk)]
    g = torch.Generator().manual_seed(d)
    q = torch.randn(sum(lq) + 2, H, d, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(sum(lk) + 1, Hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ws = torch.empty(fa.fwd_packed_workspace_size(len(lq), q.shape[0], H, Hkv), dtype=torch.uint8, device="cuda")
    _record(dbg)
    o_d, l_d = _run(dbg, q, k, v, *cu, ws, causal)
    rec = _record(dbg)
    assert rec == [0] * 8, f"debug checks failed: {rec}"
    assert dbg.fa_get_device_status(None) == 0
    o_r, l_r = _run(rel, q, k, v, *cu, ws, causal)
    assert torch.equal(o_d, o_r) and torch.equal(l_d, l_r)
