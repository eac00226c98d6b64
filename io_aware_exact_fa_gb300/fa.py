"""Thin ctypes binding over libfa_gb300.so (include/fa.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels. PyTorch supplies device memory and the current
stream. Importing this module raises ImportError when the library has not
been built (there is no fallback path).
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m io_aware_exact_fa_gb300.build` "
        "(or __graft_entry__.build()); there is no non-CUDA fallback")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_u64 = ctypes.c_uint64
_f = ctypes.c_float
_sz = ctypes.c_size_t

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_WORKSPACE = range(6)

EXPORTS = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_fwd_masked": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _i64, _i64, _i64, _vp]),
    "fa_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _f, _f, _i, _vp]),
    "fa_fwd_host_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_fwd_host": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "fa_decode_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_decode_splitkv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_decode_splitkv_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_decode_grouped_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_decode_grouped": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_fwd_packed_workspace_size": (_sz, [_i] * 4),
    "fa_fwd_packed": (_i, [_vp] * 8 + [_i] * 6 + [_f, _i, _vp, _sz, _vp]),
    "fa_append_paged": (_i, [_vp] * 9 + [_vp, _i64] + [_vp] * 6 + [_i] * 11 + [_f, _f, _i, _vp]),
    "fa_decode_paged_workspace_size": (_sz, [_i] * 7),
    "fa_decode_paged": (_i, [_vp] * 7 + [_i64, _vp, _vp, _vp, _vp] + [_i] * 9 + [_f, _i, _vp, _sz, _vp]),
    "fa_materialized_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_fwd_materialized": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_get_device_status": (_i, [_vp]),
    "fa_set_wait_limit_ns": (None, [_u64]),
    "fa_get_wait_limit_ns": (_u64, []),
    "fa_selftest_wait_timeout": (_i, [_u64, _vp]),
    "fa_selftest_exp2": (_i, [_vp, _vp, _i, _vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_last_error_detail": (ctypes.c_char_p, []),
    "fa_launch_count": (_u64, []),
    "fa_debug_enabled": (_i, []),
    "fa_debug_record": (_i, [_vp, _vp]),
    "fa_debug_selftest": (_i, [_vp]),
}
for _name, (_res, _args) in EXPORTS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def debug_library() -> ctypes.CDLL:
    """The device-checking build (libfa_gb300_debug.so, FA_DEBUG=1; see
    include/fa.h), with the same entry points as the release library. Build it
    with ``build.build(debug=True)``."""
    path = os.path.join(_HERE, "libfa_gb300_debug.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m io_aware_exact_fa_gb300.build --debug`")
    dl = ctypes.CDLL(path)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(dl, name)
        fn.restype = res
        fn.argtypes = args
    return dl


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = _lib.fa_last_error_detail().decode()
        super().__init__(f"{where}: {_lib.fa_status_string(status).decode()} {detail}".strip())


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=torch.bfloat16) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
        causal: bool = False, keep_bits: Optional[torch.Tensor] = None,
        mask_strides: Tuple[int, int, int] = (0, 0, 0), out: Optional[torch.Tensor] = None,
        lse: Optional[torch.Tensor] = None, with_lse: bool = True,
        stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Exact attention forward pass: q [B,H,Nq,d], k/v [B,H,Nk,d] bf16 -> (o bf16, lse fp32).

    ``keep_bits`` (int32 words, bit j%32 of word j//32 = key j, 1 = attend)
    with ``mask_strides`` = (b, h, q) strides in words; q stride 0 broadcasts.
    """
    _need(q, "q"); _need(k, "k"); _need(v, "v")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d):
        raise ValueError("k and v must be [B, H, Nk, d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out")
    if with_lse and lse is None:
        lse = torch.empty(B, H, Nq, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    st = _stream_ptr(stream)
    lp = lse.data_ptr() if lse is not None else None
    if keep_bits is None:
        rc = _lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp,
                         B, H, Nq, Nk, d, float(scale), int(bool(causal)), st)
        _check(rc, "fa_fwd")
    else:
        _need(keep_bits, "keep_bits", torch.int32)
        sb, sh, sq = mask_strides
        rc = _lib.fa_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp,
                                B, H, Nq, Nk, d, float(scale), int(bool(causal)),
                                keep_bits.data_ptr(), int(sb), int(sh), int(sq), st)
        _check(rc, "fa_fwd_masked")
    return out, lse


def fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, descale_q: float, descale_k: float,
            descale_v: float, scale: Optional[float] = None, causal: bool = False,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, with_lse: bool = True,
            stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Forward pass on e4m3 inputs (fa_fwd_fp8): q8 [B,H,Nq,d], k8/v8 [B,H,Nk,d]
    as uint8 codes (or torch.float8_e4m3fn), each with one descale factor
    (real value = code value * descale) -> (o bf16, lse fp32)."""
    q8, k8, v8 = (t.view(torch.uint8) if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn else t
                  for t in (q8, k8, v8))
    _need(q8, "q8", torch.uint8); _need(k8, "k8", torch.uint8); _need(v8, "v8", torch.uint8)
    B, H, Nq, d = q8.shape
    Nk = k8.shape[2]
    if k8.shape != (B, H, Nk, d) or v8.shape != (B, H, Nk, d):
        raise ValueError("k8 and v8 must be [B, H, Nk, d] matching q8")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(B, H, Nq, d, dtype=torch.bfloat16, device=q8.device)
    _need(out, "out")
    if with_lse and lse is None:
        lse = torch.empty(B, H, Nq, dtype=torch.float32, device=q8.device)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    rc = _lib.fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(),
                         lse.data_ptr() if lse is not None else None, B, H, Nq, Nk, d, float(scale),
                         float(descale_q), float(descale_k), float(descale_v), int(bool(causal)),
                         _stream_ptr(stream))
    _check(rc, "fa_fwd_fp8")
    return out, lse


def fwd_host_workspace_size(B: int, H: int, Nq: int, Nk: int, d: int, chunk_heads: int = 0) -> int:
    return int(_lib.fa_fwd_host_workspace_size(B, H, Nq, Nk, d, chunk_heads))


def _need_host(t: torch.Tensor, name: str, dtype=torch.bfloat16) -> None:
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
             causal: bool = False, chunk_heads: int = 0, workspace: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, with_lse: bool = True,
             stream: Optional[torch.cuda.Stream] = None,
             sync: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """fa_fwd_host: the forward pass on HOST tensors (q [B,H,Nq,d], k/v [B,H,Nk,d]
    bf16; pin them for overlap). The library copies chunks of heads to the
    current CUDA device, runs the fused kernel there and copies o and lse
    back. With ``sync`` the call waits for ``stream`` before returning;
    otherwise the host outputs are complete once the stream is synchronised."""
    _need_host(q, "q"); _need_host(k, "k"); _need_host(v, "v")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d):
        raise ValueError("k and v must be [B, H, Nk, d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    pin = q.is_pinned()
    if out is None:
        out = torch.empty(tuple(q.shape), dtype=q.dtype, pin_memory=pin)
    _need_host(out, "out")
    if with_lse and lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, pin_memory=pin)
    if lse is not None:
        _need_host(lse, "lse", torch.float32)
    if workspace is None:
        workspace = torch.empty(max(1, fwd_host_workspace_size(B, H, Nq, Nk, d, chunk_heads)), dtype=torch.uint8,
                                device="cuda")
    _need(workspace, "workspace", torch.uint8)
    st = _stream_ptr(stream)
    rc = _lib.fa_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          lse.data_ptr() if lse is not None else None, B, H, Nq, Nk, d, float(scale),
                          int(bool(causal)), int(chunk_heads), workspace.data_ptr(),
                          workspace.numel(), st)
    _check(rc, "fa_fwd_host")
    if sync:
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return out, lse


def decode_workspace_size(B: int, H: int, d: int, num_splits: int) -> int:
    return int(_lib.fa_decode_workspace_size(B, H, d, num_splits))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, scale: Optional[float] = None,
           num_splits: int = 16, workspace: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, with_lse: bool = True,
           stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Split-KV decode: q [B,H,1,d], caches [B,H,Nk,d] bf16 -> (o [B,H,1,d] bf16, lse [B,H] fp32)."""
    _need(q, "q"); _need(k_cache, "k_cache"); _need(v_cache, "v_cache")
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per (b, h): q must be [B, H, 1, d]")
    Nk = k_cache.shape[2]
    if k_cache.shape != (B, H, Nk, d) or v_cache.shape != (B, H, Nk, d):
        raise ValueError("k_cache and v_cache must be [B, H, Nk, d]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = decode_workspace_size(B, H, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out")
    if with_lse and lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    rc = _lib.fa_decode_splitkv(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                                lse.data_ptr() if lse is not None else None, B, H, Nk, d, float(scale),
                                int(num_splits), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream))
    _check(rc, "fa_decode_splitkv")
    return out, lse


def decode_grouped_workspace_size(B: int, H: int, Nq: int, d: int, num_splits: int) -> int:
    return int(_lib.fa_decode_grouped_workspace_size(B, H, Nq, d, num_splits))


def decode_grouped(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   seqlens_k: Optional[torch.Tensor] = None, scale: Optional[float] = None, num_splits: int = 8,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, with_lse: bool = True,
                   stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode with grouped K/V heads, Nq new tokens and per-sequence lengths (fa.h fa_decode_grouped):
    q [B,H,Nq,d], caches [B,Hkv,Nk,d] bf16, seqlens_k int32 [B] or None -> (o [B,H,Nq,d], lse [B,H,Nq])."""
    _need(q, "q"); _need(k_cache, "k_cache"); _need(v_cache, "v_cache")
    B, H, Nq, d = q.shape
    Hkv, Nk = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Nk, d) or v_cache.shape != (B, Hkv, Nk, d):
        raise ValueError("k_cache and v_cache must be [B, Hkv, Nk, d]")
    if seqlens_k is not None:
        _need(seqlens_k, "seqlens_k", torch.int32)
        if seqlens_k.shape != (B,):
            raise ValueError("seqlens_k must be int32 [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = decode_grouped_workspace_size(B, H, Nq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out")
    if with_lse and lse is None:
        lse = torch.empty(B, H, Nq, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    rc = _lib.fa_decode_grouped(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                seqlens_k.data_ptr() if seqlens_k is not None else None, out.data_ptr(),
                                lse.data_ptr() if lse is not None else None, B, H, Hkv, Nq, Nk, d, float(scale),
                                int(num_splits), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream))
    _check(rc, "fa_decode_grouped")
    return out, lse


# --------------------------------------------------------------------------- paged caches

def rotary_turns(rot: int, base: float = 10000.0, scaling: Optional[Tuple] = None,
                 device: Optional[torch.device] = None) -> torch.Tensor:
    """Rotation frequencies for ``append_paged``: int64 [rot / 2], each base**(-2j / rot) radians a
    position as a fraction of a turn in units of 2**-64.

    ``scaling`` stretches them for contexts longer than a model was trained on:
      ("linear", f)                 every frequency divided by f (positions interpolated);
      ("base", f)                   the base raised to base * f**(rot / (rot - 2)), which divides the
                                    lowest frequency by f and leaves the highest alone;
      ("by_parts", f, n, slow, fast) frequencies that turn fewer than ``slow`` times in the n positions
                                    of training are divided by f, those that turn more than ``fast``
                                    times are left alone, linearly blended (in turns) between.
    """
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be positive and even")
    kind = scaling[0] if scaling else None
    if kind not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {kind!r}")
    if kind and not scaling[1] >= 1:
        raise ValueError("the scaling factor must be >= 1")
    if kind == "by_parts" and not (scaling[2] > 0 and 0 <= scaling[3] < scaling[4]):
        raise ValueError("by_parts scaling needs n > 0 and 0 <= slow < fast")
    if kind == "base":
        if rot < 4:
            raise ValueError("base scaling needs rot >= 4")
        base = base * scaling[1] ** (rot / (rot - 2))
    out = []
    for j in range(rot // 2):
        t = base ** (-2.0 * j / rot) / (2.0 * math.pi)      # turns a position
        if kind == "linear":
            t /= scaling[1]
        elif kind == "by_parts":
            _, f, n, slow, fast = scaling
            keep = min(1.0, max(0.0, (t * n - slow) / (fast - slow)))
            t = t / f * (1.0 - keep) + t * keep
        u = int(t * 2.0 ** 64) % (1 << 64)
        out.append(u - (1 << 64) if u >= 1 << 63 else u)
    return torch.tensor(out, dtype=torch.int64, device=device if device is not None else "cuda")


# The checks below run before every call of a serving step: each tensor's properties are asked for once, a device is
# compared by its index (-1 for host tensors), and the reason of a refusal is worked out only once there is one.

_BF16, _F32, _I32, _CODES = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _refusal(t, name: str, dtype, dev: int, shape, layout: str) -> ValueError:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        return ValueError(f"{name} is on {t.device}, q on cuda:{dev}")
    if shape is not None and t.shape != shape:
        return ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return ValueError(f"{name} must {layout}")


def _whole(t: torch.Tensor, name: str, dtype, dev: int, shape=None) -> int:
    """A contiguous tensor (of the given shape) on the call's device; returns its address."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()
            or (shape is not None and t.shape != shape)):
        raise _refusal(t, name, dtype, dev, shape, "be contiguous")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, dev: int, shape) -> Tuple[int, ...]:
    """A bf16 tensor whose last dimension is contiguous; its other strides may be any multiple of 8. Returns them for the
    C ABI (which does not look at the stride of a dimension of one element)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.get_device() != dev or t.shape != shape:
        raise _refusal(t, name, _BF16, dev, shape, "")
    st = t.stride()
    if st[-1] != 1:
        raise _refusal(t, name, _BF16, dev, shape, "have a contiguous last dimension")
    return st[:-1]


def _pool(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, Hkv: int, d: int, dev: int):
    """Checks the paged cache; returns (its addresses as the C ABI takes them, pages, page size, e4m3?, B, width)."""
    if not isinstance(k_pages, torch.Tensor):
        raise ValueError("k_pages must be a CUDA tensor")
    kind = k_pages.dtype
    e4m3 = kind is _CODES or kind is torch.uint8
    if not e4m3:
        kind = _BF16
    kp = _whole(k_pages, "k_pages", kind, dev)
    shape = k_pages.shape
    if len(shape) != 4 or shape[1] != Hkv or shape[3] != d:
        raise ValueError(f"k_pages and v_pages must be [num_pages, {Hkv}, page, {d}]")
    vp = _whole(v_pages, "v_pages", kind, dev, shape)
    n, _, page, _ = shape
    ks = vs = None
    if e4m3:
        if k_scale is None or v_scale is None:
            raise ValueError("e4m3 pages need k_scale and v_scale")
        ks = _whole(k_scale, "k_scale", _F32, dev, (n, Hkv))
        vs = _whole(v_scale, "v_scale", _F32, dev, (n, Hkv))
    elif k_scale is not None or v_scale is not None:
        raise ValueError("bf16 pages take no scales")
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not _I32 or block_table.get_device() != dev:
        raise _refusal(block_table, "block_table", _I32, dev, None, "")
    tab, ts = block_table.shape, block_table.stride()
    if len(tab) != 2 or (ts[1] != 1 and tab[1] > 1):
        raise ValueError("block_table must be [B, width] with contiguous rows")
    B, width = tab
    lens = _whole(seqlens_k, "seqlens_k", _I32, dev, (B,))
    return (kp, vp, ks, vs, block_table.data_ptr(), ts[0], lens), n, page, e4m3, B, width


# (a torch without CUDA has neither, and no tensor for the calls that ask; sizes and refusals work there all the same)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
try:  # the allocator without the dispatcher before it (half the time of torch.empty); on the current device
    _empty_here = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _empty_here = None


def _empty(shape: Tuple[int, ...], strides: Tuple[int, ...], dtype, dev: int) -> torch.Tensor:
    """A new tensor on device ``dev``; shape and strides are plain tuples."""
    if _empty_here is not None and _current_device() == dev:
        return _empty_here(shape, strides, dtype)
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


def _call(dev: int, stream: Optional[torch.cuda.Stream], fn, args, where: str, made=()) -> None:
    """Calls the library with the tensors' device current, on ``stream`` or that device's current stream. ``made``:
    tensors that were made for the call, or None; another stream than the current one is made known to the allocator,
    which would otherwise hand their memory out again while the call still runs."""
    if stream is None:
        st = _raw_stream(dev)
    elif stream.device.index == dev:
        st = stream.cuda_stream
        if st != _raw_stream(dev):
            for t in made:
                if t is not None:
                    t.record_stream(stream)
    else:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    if _current_device() == dev:
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc != FA_OK:
        raise FAError(rc, where)


_I64x10 = ctypes.c_int64 * 10
_I64x3 = ctypes.c_int64 * 3


def append_paged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, seqlens_k: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                 max_new: int = 0, turns: Optional[torch.Tensor] = None, interleaved: bool = False,
                 rot_scale: float = 1.0, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, with_k: bool = True,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norms, rotates and appends a step's tokens to a paged cache (fa.h fa_append_paged).

    q [T,H,d], k/v [T,Hkv,d] bf16 (parts of one projection are taken as they are); k_pages/v_pages
    [num_pages,Hkv,page,d] bf16, or float8_e4m3fn / uint8 codes with fp32 scales [num_pages,Hkv]; block_table int32
    [B,width]; seqlens_k int32 [B] with the new tokens counted; cu_seqlens int32 [B+1], or None for T / B tokens each.
    ``turns`` (``rotary_turns``) sets the rotation, None for none; the weights bf16 [d] the norms, None for none.
    Returns the turned q [T,H,d] and k [T,Hkv,d] (None without ``with_k``), contiguous unless given."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise ValueError("q must be a CUDA tensor [T, H, d]")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a CUDA tensor [T, Hkv, d]")
    dev = q.get_device()
    T, H, d = q_shape = q.shape
    kv_shape = (T, k.shape[1], d)
    Hkv = kv_shape[1]
    st = _heads(q, "q", dev, q_shape) + _heads(k, "k", dev, kv_shape) + _heads(v, "v", dev, kv_shape)
    pool, n, page, e4m3, B, width = _pool(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, Hkv, d, dev)
    kp, vp, ks, vs, table, table_stride, lens = pool
    cu = None if cu_seqlens is None else _whole(cu_seqlens, "cu_seqlens", _I32, dev, (B + 1,))
    rot, tp = 0, None
    if turns is not None:
        tp = _whole(turns, "turns", torch.int64, dev)
        rot = 2 * turns.numel()
    qw = None if q_weight is None else _whole(q_weight, "q_weight", _BF16, dev, (d,))
    kw = None if k_weight is None else _whole(k_weight, "k_weight", _BF16, dev, (d,))
    if q_out is None:
        q_out = _empty((T, H, d), (H * d, d, 1), _BF16, dev)
        st += (H * d, d)
    else:
        st += _heads(q_out, "q_out", dev, q_shape)
    if k_out is not None:
        st += _heads(k_out, "k_out", dev, kv_shape)
    elif with_k:
        k_out = _empty((T, Hkv, d), (Hkv * d, d, 1), _BF16, dev)
        st += (Hkv * d, d)
    else:
        st += (0, 0)
    _call(dev, stream, _lib.fa_append_paged,
          (q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), None if k_out is None else k_out.data_ptr(), kp, vp,
           ks, vs, table, table_stride, lens, cu, tp, qw, kw, _I64x10(*st), B, T, H, Hkv, d, n, page, width, e4m3, rot,
           bool(interleaved), rot_scale, eps, max_new), "fa_append_paged", (q_out, k_out))
    return q_out, k_out


def decode_paged_workspace_size(B: int, H: int, Hkv: int, Nq: int, d: int, max_len: int, num_splits: int = 0) -> int:
    return int(_lib.fa_decode_paged_workspace_size(B, H, Hkv, Nq, d, max_len, num_splits))


def decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                 seqlens_k: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                 max_len: Optional[int] = None, num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, with_lse: bool = True,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Grouped decode over a paged cache (fa.h fa_decode_paged): q [B,H,Nq,d] bf16, any strides with d contiguous
    (``append_paged``'s q of B x Nq tokens is ``q.view(B, Nq, H, d).transpose(1, 2)``), the pool and table as for
    ``append_paged`` -> (o [B,H,Nq,d] bf16, lse [B,H,Nq] fp32). ``max_len`` bounds the lengths (default: all that a
    row of the table covers); ``num_splits`` 0 lets the library choose. Without ``out``, o is token-major where q is, else contiguous."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
        raise ValueError("q must be a CUDA tensor [B, H, Nq, d]")
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a CUDA tensor [num_pages, Hkv, page, d]")
    dev = q.get_device()
    B, H, Nq, d = q_shape = q.shape
    qs = _heads(q, "q", dev, q_shape)
    Hkv = k_pages.shape[1]
    pool, n, page, e4m3, rows, width = _pool(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, Hkv, d, dev)
    if rows != B:
        raise ValueError("seqlens_k and block_table must have B rows")
    kp, vp, ks, vs, table, table_stride, lens = pool
    if max_len is None:
        max_len = width * page
    elif not 0 <= max_len <= width * page:
        raise ValueError(f"max_len must be in [0, {width * page}], what a row of block_table covers")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        # laid out like q where that is token-major, else contiguous
        os_ = (Nq * H * d, d, H * d) if qs[1] == d and qs[2] == H * d else (H * Nq * d, Nq * d, d)
        out = _empty((B, H, Nq, d), os_ + (1,), _BF16, dev)
    else:
        os_ = _heads(out, "out", dev, q_shape)
    lp = None
    if lse is not None:
        lp = _whole(lse, "lse", _F32, dev, (B, H, Nq))
    elif with_lse:
        lse = _empty((B, H, Nq), (H * Nq, Nq, 1), _F32, dev)
        lp = lse.data_ptr()
    if workspace is None:
        workspace = q.new_empty(max(1, decode_paged_workspace_size(B, H, Hkv, Nq, d, max_len, num_splits)),
                                dtype=torch.uint8)
    wp = _whole(workspace, "workspace", workspace.dtype, dev)
    _call(dev, stream, _lib.fa_decode_paged,
          (q.data_ptr(), _I64x3(*qs), kp, vp, ks, vs, table, table_stride, lens, out.data_ptr(), _I64x3(*os_), lp, B, H,
           Hkv, Nq, d, n, page, max_len, e4m3, scale, num_splits, wp, workspace.nbytes), "fa_decode_paged",
          (out, lse, workspace))
    return out, lse


# --------------------------------------------------------------------------- packed prefill

def fwd_packed_workspace_size(B: int, total_q: int, H: int, Hkv: int) -> int:
    return int(_lib.fa_fwd_packed_workspace_size(B, total_q, H, Hkv))


_I64x8 = ctypes.c_int64 * 8


def fwd_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = False,
               workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, with_lse: bool = True,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention inside each of B packed sequences, grouped K/V heads (fa.h fa_fwd_packed): q [total_q,H,d], k/v
    [total_k,Hkv,d] bf16 (parts of one projection are taken as they are), cu_seqlens int32 [B+1] ->
    (o [total_q,H,d] bf16, lse [H,total_q] fp32). Rows behind the last sequence are left as they were."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise ValueError("q must be a CUDA tensor [total_q, H, d]")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a CUDA tensor [total_k, Hkv, d]")
    dev = q.get_device()
    Tq, H, d = q_shape = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    kv_shape = (Tk, Hkv, d)
    st = _heads(q, "q", dev, q_shape) + _heads(k, "k", dev, kv_shape) + _heads(v, "v", dev, kv_shape)
    cq = _whole(cu_seqlens_q, "cu_seqlens_q", _I32, dev)
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_q.dim() != 1 or B < 1:
        raise ValueError("cu_seqlens_q must be int32 [B + 1], B >= 1")
    ck = None if cu_seqlens_k is None else _whole(cu_seqlens_k, "cu_seqlens_k", _I32, dev, (B + 1,))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        st += (H * d, d)
        out = _empty((Tq, H, d), (H * d, d, 1), _BF16, dev)
    else:
        st += _heads(out, "out", dev, q_shape)
    lp = None
    if lse is not None:
        lp = _whole(lse, "lse", _F32, dev, (H, Tq))
    elif with_lse:
        lse = _empty((H, Tq), (Tq, 1), _F32, dev)
        lp = lse.data_ptr()
    if workspace is None:
        workspace = q.new_empty(max(1, fwd_packed_workspace_size(B, Tq, H, Hkv)), dtype=torch.uint8)
    wp = _whole(workspace, "workspace", workspace.dtype, dev)
    _call(dev, stream, _lib.fa_fwd_packed,
          (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp, _I64x8(*st), cq, ck, B, Tq, Tk, H, Hkv, d, scale,
           bool(causal), wp, workspace.nbytes), "fa_fwd_packed", (out, lse, workspace))
    return out, lse


NOALLOC_SCRATCH_BYTES = 20 << 20


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, scale: Optional[float] = None,
                   num_splits: int = 16, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   with_lse: bool = True, stream: Optional[torch.cuda.Stream] = None):
    """Split-KV decode using the library's static scratch (no workspace); see fa.h."""
    _need(q, "q"); _need(k_cache, "k_cache"); _need(v_cache, "v_cache")
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per (b, h): q must be [B, H, 1, d]")
    Nk = k_cache.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if with_lse and lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    rc = _lib.fa_decode_splitkv_noalloc(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                                        lse.data_ptr() if lse is not None else None, B, H, Nk, d, float(scale),
                                        int(num_splits), _stream_ptr(stream))
    _check(rc, "fa_decode_splitkv_noalloc")
    return out, lse


def materialized_workspace_size(B: int, H: int, Nq: int, Nk: int) -> int:
    return int(_lib.fa_materialized_workspace_size(B, H, Nq, Nk))


def fwd_materialized(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                     causal: bool = False, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The materialising baseline (fa.h fa_fwd_materialized): S and P through HBM in bf16."""
    _need(q, "q"); _need(k, "k"); _need(v, "v")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d):
        raise ValueError("k and v must be [B, H, Nk, d]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = materialized_workspace_size(B, H, Nq, Nk)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, H, Nq, dtype=torch.float32, device=q.device)
    _need(out, "out"); _need(lse, "lse", torch.float32)
    rc = _lib.fa_fwd_materialized(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Nq,
                                  Nk, d, float(scale), int(bool(causal)), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(rc, "fa_fwd_materialized")
    return out, lse


def bwd_workspace_size(B: int, H: int, Nq: int, d: int) -> int:
    return int(_lib.fa_bwd_workspace_size(B, H, Nq, d))


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
        dout: torch.Tensor, scale: Optional[float] = None, causal: bool = False,
        workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
        grads: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """Backward pass of ``fwd`` (no key mask): returns (dq, dk, dv), bf16, shaped like q, k, v
    (written into ``grads`` when given)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n)
    _need(lse, "lse", torch.float32)
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d) or o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("shapes: q, o, dout [B,H,Nq,d]; k, v [B,H,Nk,d]")
    if lse.shape != (B, H, Nq):
        raise ValueError("lse must be [B, H, Nq]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = bwd_workspace_size(B, H, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if grads is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = grads
        for t, ref, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
            _need(t, n)
            if t.shape != ref.shape:
                raise ValueError(f"{n} must be shaped like its input")
    rc = _lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Nq, Nk, d, float(scale), int(bool(causal)),
                     workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(rc, "fa_bwd")
    return dq, dk, dv


def device_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise and return (then clear) the library's device status (FA_OK or FA_ERR_TIMEOUT)."""
    return int(_lib.fa_get_device_status(_stream_ptr(stream)))


def selftest_wait_timeout(limit_ns: int, stream: Optional[torch.cuda.Stream] = None) -> int:
    return int(_lib.fa_selftest_wait_timeout(int(limit_ns), _stream_ptr(stream)))


def selftest_exp2(x: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """2^x through the device FMA-pipe exponential used inside the prefill softmax."""
    _need(x, "x", torch.float32)
    y = torch.empty_like(x)
    _check(_lib.fa_selftest_exp2(x.data_ptr(), y.data_ptr(), x.numel(), _stream_ptr(stream)), "fa_selftest_exp2")
    return y


def set_wait_limit_ns(ns: int) -> None:
    _lib.fa_set_wait_limit_ns(int(ns))


def get_wait_limit_ns() -> int:
    return int(_lib.fa_get_wait_limit_ns())


def launch_count() -> int:
    return int(_lib.fa_launch_count())


def status_string(s: int) -> str:
    return _lib.fa_status_string(s).decode()


# raw handle for callers that pass their own pointers (host-buffer end-to-end timing, tests)
lib = _lib
