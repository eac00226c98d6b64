"""Host side of the paged operators: argument checks before any CUDA call, the
page lookup of the kernels compiled for the host, the frequency tables, and pins
of the paged oracle (CPU only)."""

import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import fp8 as FP8
from oracle import paged as OP

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # a fake, aligned address that is never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_fa_gb300 import build
    build.build()
    from io_aware_exact_fa_gb300 import fa as lib
    return lib


def _append(fa, **kw):
    a = dict(q=P, k=P, v=P, q_out=P, k_out=P, k_pages=P, v_pages=P, k_scale=P, v_scale=P, table=P, stride=4, lens=P,
             cu=None, turns=P, qw=None, kw=None, strides=[512, 64] * 5, B=2, T=2, H=8, Hkv=2, d=64, pages=8, page=16,
             width=4, e4m3=0, rot=64, inter=0, rs=1.0, eps=1e-6, max_new=0)
    a.update(kw)
    a["strides"] = None if a["strides"] is None else (ctypes.c_int64 * 10)(*a["strides"])
    return fa.lib.fa_append_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID), (dict(k_pages=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(turns=None), INVALID), (dict(strides=None), INVALID),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(T=3), INVALID), (dict(H=7), INVALID), (dict(Hkv=0), INVALID),
    (dict(width=0), INVALID), (dict(pages=0), INVALID), (dict(rot=80), INVALID), (dict(rot=-16), INVALID),
    (dict(rs=float("nan")), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(max_new=-1), INVALID), (dict(stride=3), INVALID), (dict(e4m3=1, k_scale=None), INVALID),
    (dict(e4m3=1, v_scale=None), INVALID), (dict(width=1 << 27, stride=1 << 27, page=64), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
    (dict(q=P + 2), UNSUPPORTED), (dict(k_out=P + 8), UNSUPPORTED), (dict(v_pages=P + 8), UNSUPPORTED),
    (dict(turns=P + 4), UNSUPPORTED), (dict(table=P + 2), UNSUPPORTED), (dict(qw=P + 8), UNSUPPORTED),
    (dict(strides=[512, 60] + [512, 64] * 4), UNSUPPORTED), (dict(strides=[512, -64] + [512, 64] * 4), UNSUPPORTED),
    (dict(strides=[512, 64] * 3 + [512, 0] + [512, 64]), UNSUPPORTED), (dict(strides=[512, 64] * 4 + [0, 64]), UNSUPPORTED),
    (dict(T=0, q=None, k=None, v=None, q_out=None), 0),
])
def test_append_refusals(fa, kw, want):
    assert _append(fa, **kw) == want, fa.lib.fa_last_error_detail()


def _decode(fa, **kw):
    a = dict(q=P, qs=[512, 64, 512], k=P, v=P, ks=None, vs=None, table=P, stride=64, lens=P, o=P, os=[512, 64, 64],
             lse=P, B=2, H=8, Hkv=2, Nq=1, d=64, pages=8, page=16, max_len=1000, e4m3=0, scale=0.125, splits=4, ws=P,
             bytes=1 << 30)
    a.update(kw)
    for s in ("qs", "os"):
        a[s] = None if a[s] is None else (ctypes.c_int64 * 3)(*a[s])
    return fa.lib.fa_decode_paged(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(qs=None), INVALID), (dict(k=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(B=0), INVALID), (dict(H=9), INVALID),
    (dict(Nq=0), INVALID), (dict(max_len=-1), INVALID), (dict(max_len=(1 << 30) + 1), INVALID),
    (dict(splits=-1), INVALID), (dict(splits=1025), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(e4m3=1), INVALID), (dict(stride=62), INVALID), (dict(d=32), UNSUPPORTED), (dict(Nq=33), UNSUPPORTED),
    (dict(H=1 << 20, Nq=1 << 20), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(q=P + 8), UNSUPPORTED),
    (dict(o=P + 4), UNSUPPORTED), (dict(lse=P + 2), UNSUPPORTED), (dict(qs=[512, 64, 65], Nq=2), UNSUPPORTED),
    (dict(os=[512, 0, 64]), UNSUPPORTED),
    (dict(k=P + 8), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(bytes=64), WORKSPACE),
])
def test_decode_refusals(fa, kw, want):
    assert _decode(fa, **kw) == want, fa.lib.fa_last_error_detail()


def test_decode_workspace(fa):
    # a partial (o, m, l) for each range, and one more for each sequence and K/V head: 4 splits a pair on average, two
    # rows a pair padded to eight
    n = fa.decode_paged_workspace_size(3, 4, 2, 1, 64, 1000, 4)
    assert n % 256 == 0 and 0 <= n - (3 * 2 * 4 + 3 * 2) * 8 * (64 + 2) * 4 < 3 * 256
    # 18 rows: two tiles of sixteen
    n = fa.decode_paged_workspace_size(3, 18, 2, 2, 128, 1000, 1)
    assert n % 256 == 0 and 0 <= n - (3 * 2 + 3 * 2) * 2 * 16 * (128 + 2) * 4 < 3 * 256
    assert fa.decode_paged_workspace_size(3, 8, 3, 2, 64, 100, 4) == 0
    assert fa.decode_paged_workspace_size(3, 8, 2, 2, 80, 100, 4) == 0
    assert fa.decode_paged_workspace_size(1, 8, 2, 64, 64, 100, 4) == 0     # 256 rows
    # the library's own choice does not grow with the lengths
    assert (fa.decode_paged_workspace_size(1, 1, 1, 1, 64, 1 << 30) == fa.decode_paged_workspace_size(1, 1, 1, 1, 64, 10)
            < 16 << 20)


def _packed(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, strides=[512, 64, 128, 64, 128, 64, 512, 64], cu_q=P, cu_k=None, B=2, tq=100,
             tk=100, H=8, Hkv=2, d=64, scale=0.125, causal=1, ws=P, bytes=1 << 20)
    a.update(kw)
    a["strides"] = None if a["strides"] is None else (ctypes.c_int64 * 8)(*a["strides"])
    return fa.lib.fa_fwd_packed(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(strides=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(B=0), INVALID), (dict(H=7), INVALID), (dict(Hkv=0), INVALID),
    (dict(tq=-1), INVALID), (dict(tk=99), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(B=1 << 30, H=64), INVALID), (dict(d=80), UNSUPPORTED), (dict(q=P + 8), UNSUPPORTED),
    (dict(o=P + 2), UNSUPPORTED), (dict(lse=P + 1), UNSUPPORTED), (dict(cu_q=P + 2), UNSUPPORTED),
    (dict(cu_k=P + 2), UNSUPPORTED), (dict(strides=[512, 60, 128, 64, 128, 64, 512, 64]), UNSUPPORTED),
    (dict(strides=[512, 64, 0, 64, 128, 64, 512, 64]), UNSUPPORTED),
    (dict(strides=[512, 64, 128, 64, 128, -64, 512, 64]), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=P + 128), WORKSPACE), (dict(bytes=256), WORKSPACE), (dict(tq=0, tk=0, q=None, k=None, v=None, o=None), 0),
])
def test_packed_refusals(fa, kw, want):
    assert _packed(fa, **kw) == want, fa.lib.fa_last_error_detail()


def test_packed_workspace(fa):
    # pairs of heads: 128-row blocks; an odd group: 256-row blocks; at most one ragged block a sequence
    assert fa.fwd_packed_workspace_size(3, 1000, 8, 2) == 256 + (1000 // 128 + 3) * 32
    assert fa.fwd_packed_workspace_size(3, 1000, 6, 2) == 256 + (1000 // 256 + 3) * 32
    assert fa.fwd_packed_workspace_size(3, 1000, 6, 4) == 0 and fa.fwd_packed_workspace_size(0, 1, 1, 1) == 0


def test_page_lookup_on_the_host(tmp_path):
    """The kernels' page lookup and length clipping, compiled for the host: entries outside the pool are refused,
    offsets do not wrap at 2^31 or 2^32 elements."""
    src = tmp_path / "lookup.cu"
    src.write_text("""
#include <cstdio>
#include "paged.cuh"
int main() {
  long long id, pages, hkv, hk, page, row, d;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &id, &pages, &hkv, &hk, &page, &row, &d) == 7)
    std::printf("%lld\\n", fa::paged_row_offset((int)id, (int)pages, (int)hkv, (int)hk, (int)page, (int)row, (int)d));
  std::printf("%d %d %d\\n", fa::paged_clip_len(-5, 10), fa::paged_clip_len(7, 10), fa::paged_clip_len(2147483647, 10));
}
""")
    from io_aware_exact_fa_gb300 import build
    exe = tmp_path / "lookup"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                    build.INCLUDE, str(src), "-o", str(exe)], check=True, capture_output=True)
    rows = [(0, 4, 2, 1, 16, 3, 64), (3, 4, 2, 0, 16, 15, 64), (4, 4, 2, 0, 16, 0, 64), (-1, 4, 2, 0, 16, 0, 64),
            (-2147483648, 4, 2, 0, 16, 0, 64), (2147483647, 2147483647, 8, 7, 128, 127, 128),
            (1 << 20, (1 << 20) + 1, 8, 3, 64, 5, 128)]
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, r)) for r in rows), text=True,
                         capture_output=True, check=True).stdout.split()
    for (i, n, hkv, hk, page, row, d), got in zip(rows, out):
        assert int(got) == (((i * hkv + hk) * page + row) * d if 0 <= i < n else -1)
    assert out[len(rows):] == ["0", "7", "10"]


def test_rotary_turns(fa):
    # entries are whole units of 2^-64 turns, cut off: one unit besides the double's own rounding
    one = 2.0 ** 64
    t = fa.rotary_turns(64, 10000.0, device="cpu")
    assert t.dtype == torch.int64 and t.shape == (32,)
    for j in (0, 5, 31):
        assert math.isclose(int(t[j]) % (1 << 64) / one, 10000.0 ** (-2 * j / 64) / (2 * math.pi), rel_tol=1e-15,
                            abs_tol=1 / one)
    lin = fa.rotary_turns(64, scaling=("linear", 4.0), device="cpu")
    assert all(math.isclose(int(a), int(b) / 4, rel_tol=1e-15, abs_tol=2) for a, b in zip(lin, t))
    nb = fa.rotary_turns(64, scaling=("base", 8.0), device="cpu")
    assert int(nb[0]) == int(t[0]) and math.isclose(int(nb[31]), int(t[31]) / 8, rel_tol=1e-12)
    bp = fa.rotary_turns(64, scaling=("by_parts", 8.0, 4096, 1.0, 32.0), device="cpu")
    for a, b in zip(bp.tolist(), t.tolist()):
        turned = b / one * 4096
        want = b if turned >= 32 else b / 8 if turned <= 1 else None
        assert b / 8 * (1 - 1e-12) <= a <= b * (1 + 1e-12) if want is None else math.isclose(a, want, rel_tol=1e-12)
    for bad in ((0,), (63,), (64, 1e4, ("cubic", 2.0)), (64, 1e4, ("linear", 0.5))):
        with pytest.raises(ValueError):
            fa.rotary_turns(*bad, device="cpu")


def test_binding_refuses_host_tensors(fa):
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.append_paged(x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.decode_paged(x[None], x, x, x, x)


# --------------------------------------------------------------------------- pins of the oracle

def test_oracle_encode_matches_torch():
    x = torch.randn(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(0)) * 60
    x = torch.cat([x.clamp(-448, 448), torch.tensor([0.0, -0.0, 2 ** -10, 3 * 2 ** -10, 2 ** -9 * 1.5, 448.0, 17.0, 19.0])])
    # fp32 first: torch rounds a double through fp32
    x = x.float().double()
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OP.e4m3_encode(x.numpy()), want)
    assert list(OP.e4m3_encode(np.array([np.nan, np.inf, -np.inf]))) == [0x7F] * 3


def test_oracle_scale_exponent():
    assert OP.scale_exponent(0.0) == -40 and OP.scale_exponent(448.0) == 0
    assert OP.scale_exponent(np.nextafter(448.0, 1e9)) == 1 and OP.scale_exponent(1.0) == -8
    assert OP.scale_exponent(1e-30) == -40


def test_oracle_turn():
    """Turning by positions composes: the product of a turned query and key depends on their distance alone."""
    rng = np.random.default_rng(0)
    turns = [int(2.0 ** 64 * 10000.0 ** (-2 * j / 16) / (2 * math.pi)) for j in range(8)]
    q, k = rng.standard_normal(24), rng.standard_normal(24)
    for inter in (False, True):
        a = OP.turn(q, 70, turns, inter) @ OP.turn(k, 50, turns, inter)
        b = OP.turn(q, 20, turns, inter) @ OP.turn(k, 0, turns, inter)
        far = OP.turn(q, 10 ** 9 + 20, turns, inter) @ OP.turn(k, 10 ** 9, turns, inter)
        assert math.isclose(a, b, rel_tol=1e-12) and math.isclose(far, b, rel_tol=1e-11)
        y = OP.turn(q, 33, turns, inter)
        assert np.array_equal(y[16:], q[16:]) and math.isclose(y @ y, q @ q, rel_tol=1e-12)
    # the first pair turns one radian a position
    y = OP.turn(np.array([1.0, 0.0] + [0.0] * 14), 1, turns, True)
    assert math.isclose(y[0], math.cos(1), rel_tol=1e-12) and math.isclose(y[1], math.sin(1), rel_tol=1e-12)
    h = OP.turn(np.eye(16)[0], 1, turns, False)
    assert math.isclose(h[0], math.cos(1), rel_tol=1e-12) and math.isclose(h[8], math.sin(1), rel_tol=1e-12)


def test_oracle_store_matches_whole_quantisation():
    """Appending token by token ends with the scale of the whole page, and every value within the two roundings."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 1, 64)) * np.exp(rng.standard_normal((16, 1, 1)) * 2)
    codes, scale = np.full((2, 1, 16, 64), 0x55, dtype=np.uint8), np.full((2, 1), 7.0)
    for i in range(16):
        OP.store_e4m3(x[i:i + 1], [1], [i + 1], [[1]], 16, codes, scale)
    s = 2.0 ** OP.scale_exponent(np.abs(x).max())
    assert scale[1, 0] == s and scale[0, 0] == 7.0
    got = FP8.e4m3_decode(codes[1, 0]) * s
    assert np.all(np.abs(got - x[:, 0]) <= 2 * np.maximum(2.0 ** -4 * np.abs(x[:, 0]), 2.0 ** -10 * s))


# What the output may not be: rows of d elements that overlap, which several threads would write in any order.
@pytest.mark.parametrize("kw,bad", [
    (dict(strides=[512, 64] * 3 + [512, 8] + [512, 64]), True),             # heads 8 elements apart
    (dict(strides=[512, 64] * 3 + [504, 64] + [512, 64]), True),            # a token's last head over the next's first
    (dict(strides=[512, 64] * 3 + [64, 64] + [512, 64]), True),
    (dict(strides=[512, 64] * 3 + [64, 72] + [512, 64]), True),             # head-major, one row too close
    (dict(strides=[512, 64] * 4 + [120, 64]), True),                        # k_out: 2 heads
    (dict(strides=[512, 64] * 4 + [1 << 61, 1 << 62]), True),               # past any address
    (dict(T=0, strides=[512, 64] * 5), False),
])
def test_append_refuses_overlapping_outputs(fa, kw, bad):
    assert _append(fa, **kw) == (UNSUPPORTED if bad else 0)
    if bad:
        assert b"overlap" in fa.lib.fa_last_error_detail()


@pytest.mark.parametrize("kw", [
    dict(os=[512, 8, 64]), dict(os=[504, 64, 64]), dict(os=[64, 64, 64]), dict(os=[512, 64, 64], Nq=2),
    dict(os=[1024, 64, 504], Nq=2), dict(os=[1016, 64, 512], Nq=2),
])
def test_decode_refuses_overlapping_outputs(fa, kw):
    assert _decode(fa, **kw, qs=[1024, 64, 512]) == UNSUPPORTED and b"overlap" in fa.lib.fa_last_error_detail()


@pytest.mark.parametrize("o", [[512, 8], [504, 64], [64, 64], [64, 6328], [8, 512]])
def test_packed_refuses_overlapping_outputs(fa, o):
    assert _packed(fa, strides=[512, 64, 128, 64, 128, 64, *o]) == UNSUPPORTED
    assert b"overlap" in fa.lib.fa_last_error_detail()


def test_outputs_apart_are_taken(fa):
    """The layouts that do not overlap pass the check: the next refusal is another one (no workspace)."""
    for o, nq in (([512, 64, 64], 1), ([1024, 128, 64], 2), ([1024, 64, 512], 2), ([64, 256, 128], 2), ([8192, 64, 1024], 2)):
        assert _decode(fa, os=o, Nq=nq, qs=[1024, 64, 512], ws=None) == WORKSPACE
    for o in ([512, 64], [1024, 128], [64, 6400], [64, 1 << 20]):
        assert _packed(fa, strides=[512, 64, 128, 64, 128, 64, *o], ws=None) == WORKSPACE


def test_import_on_a_torch_without_cuda(fa):
    """The binding imports where torch was built without CUDA (its C module then has none of the CUDA entry points):
    workspace sizes and refusals need no GPU."""
    code = """
import torch
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
if hasattr(torch._C._dynamo.guards, "_empty_strided_cuda"):
    del torch._C._dynamo.guards._empty_strided_cuda
from io_aware_exact_fa_gb300 import fa
assert fa.fwd_packed_workspace_size(3, 1000, 8, 2) == 256 + (1000 // 128 + 3) * 32
assert fa.decode_paged_workspace_size(1, 8, 2, 1, 64, 100) > 0
x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
try:
    fa.fwd_packed(x, x, x, torch.zeros(2, dtype=torch.int32))
except ValueError as e:
    print("refused:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("refused: q must be a CUDA tensor"), r.stderr


def test_decode_ranges_follow_the_device(tmp_path):
    """The decode's ranges, compiled for the host: their warps fit the SMs that the device has in one wave, and the
    workspace, sized without a device, holds the ranges of any."""
    src = tmp_path / "ranges.cu"
    src.write_text("""
#include <cstdio>
#include "paged.cuh"
int main() {
  for (int d : {64, 128})
    for (int R = 1; R <= 128; ++R) {
      const int tiles = fa::decode_paged_row_tiles(R), warps = 4 * fa::decode_paged_ctas(d, fa::decode_paged_rows(R));
      const int most = fa::decode_paged_ranges(fa::DECODE_PAGED_SMS, 3, 2, R, d, 0);
      for (int sms : {1, 20, 76, 100, 148, 152, 160, 300}) {
        const int n = fa::decode_paged_ranges(sms, 3, 2, R, d, 0);
        if (n < 1 || n > most || (n > 1 && n * tiles > sms * warps)) return 1;
        if (sms <= fa::DECODE_PAGED_SMS && (n + 1) * tiles <= sms * warps) return 2;
        if (fa::decode_paged_ranges(sms, 3, 2, R, d, 7) != 42) return 3;
      }
    }
  if (fa::decode_paged_ranges(152, 1 << 20, 8, 1, 64, 1024) != 1 << 20) return 4;
  std::puts("ok");
}
""")
    from io_aware_exact_fa_gb300 import build
    exe = tmp_path / "ranges"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                    build.INCLUDE, str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert (r.returncode, r.stdout.strip()) == (0, "ok")


@pytest.mark.parametrize("parts", [(4096, 2.0, 2.0), (4096, 32.0, 1.0), (4096, -1.0, 2.0), (0, 1.0, 32.0)])
def test_rotary_turns_refuses_bad_parts(fa, parts):
    with pytest.raises(ValueError, match="by_parts"):
        fa.rotary_turns(64, 10000.0, ("by_parts", 4.0, *parts), device="cpu")
