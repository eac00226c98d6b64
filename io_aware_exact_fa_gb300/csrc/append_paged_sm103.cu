// Norm, position rotation and append to a paged K/V cache for sm_103a.
//
// New token i of sequence b (n_b new tokens, length L_b with them) is at
// position p = L_b - n_b + i. For every head of q and k:
//     x' = x / sqrt(mean(x^2) + eps) * w                          (where weights are given)
//     (a, b) -> (a cos - b sin, b cos + a sin),  angle 2 pi frac(p t_j / 2^64)
// on the pairs j of its first `rot` elements: (j, j + rot / 2), or (2j, 2j + 1)
// interleaved. q' and k' are written out in bf16; k' and v go to the row of
// position p in the cache, in bf16 or as e4m3 codes.
//
// The frequency t_j is a fraction of a turn in 64-bit fixed point, so p t_j mod
// 2^64 is the exact angle, in turns, for any position: one integer product in
// place of a range reduction, with nothing lost at far positions and no table of
// angles to read. sincospi of the fraction is good to an ulp or two of fp32.
//
// e4m3 pages have one scale for each K/V head, a power of two: the least 2^e with
// amax <= 448 2^e over the rows the page holds. The codes are floating point, so
// a finer scale would not make them more exact, and when a later token makes the
// scale grow, dividing the codes already held by a power of two rounds again
// only where they fall below the smallest normal code. The values are rounded
// once, from the fp32 result, not through bf16.
//
// A block takes the new rows of one page of one sequence and one K/V head: G
// query heads, the key and the value head. Its rows are the rows of one page, so
// the page's scales are this block's alone and no sum or maximum goes through
// global atomics. What bounds it: HBM for prompts (q read and written, k and v
// read, the cache written), launch and load latency for a step of single tokens:
// there the heads run side by side in the block instead of one after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

constexpr int AP_MAX_THREADS = 256;
#ifndef AP_BATCH
#define AP_BATCH 2      // heads whose loads a thread has in flight
#endif
#ifndef AP_CTAS
#define AP_CTAS 3       // blocks an SM should hold
#endif

__device__ __forceinline__ uint4 ldg16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// bf16 pairs to fp32
__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Largest magnitude among 16 values, infinities and NaN left out (they are stored as the NaN code).
__device__ __forceinline__ float finite_amax(const float* x) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(x[i]);
    m = a <= FLT_MAX ? fmaxf(m, a) : m;
  }
  return m;
}

// Least 2^e, e >= -40, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, PAGED_SCALE_EXP_MIN);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The scale of a page whose new rows reach amax: that of the rows it already holds where it suffices.
__device__ __forceinline__ float merged_scale(float amax, float old, bool holds) {
  if (holds && old > 0.f && old <= FLT_MAX && amax <= 448.f * old) return old;
  return scale_for(amax);
}

// Four values to four e4m3 codes (nearest even); infinities and NaN give the NaN code.
__device__ __forceinline__ uint32_t to_codes4(const float* x, float inv) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fabsf(x[i]) <= FLT_MAX ? x[i] * inv : __uint_as_float(0x7fffffffu);
  return pack_e4m3x4(y[0], y[1], y[2], y[3]);
}

}  // namespace

template <int D, bool F8>
__global__ void __launch_bounds__(AP_MAX_THREADS, AP_CTAS) fa_append_paged_kernel(const AppendPagedParams p) {
  constexpr int LPR = D / 16;  // lanes of a row, 16 elements each
  extern __shared__ __align__(16) float ap_stash[];  // F8: rotated keys, [stash_rows][D]
  __shared__ int s_seq;
  __shared__ unsigned int s_amax[2];

  const int hk = static_cast<int>(blockIdx.x) % p.Hkv;
  const int c = static_cast<int>(blockIdx.x) / p.Hkv;
  const int tid = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);

  // ---- which sequence, and which of its pages
  int b, i;
  if (p.per_seq > 0) {
    b = c / p.per_seq;
    i = c - b * p.per_seq;
  } else {
    // sequence b owns the blocks from cu[b] / page + 2 b on: at least as many
    // as its tokens can touch pages
    if (tid == 0) s_seq = 0;
    __syncthreads();
    int last = 0;
    for (int x = tid; x < p.B; x += nt)
      if ((max(__ldg(p.cu + x), 0) >> p.page_shift) + 2 * x <= c) last = x;
    atomicMax(&s_seq, last);
    __syncthreads();
    b = s_seq;
    i = c - ((max(__ldg(p.cu + b), 0) >> p.page_shift) + 2 * b);
  }
  int t0, n;
  if (p.cu != nullptr) {
    t0 = __ldg(p.cu + b);
    n = __ldg(p.cu + b + 1) - t0;
    const int most = min(p.max_new, p.T - t0);
    if (t0 < 0 || n < 0 || n > most) {
      if (tid == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
      n = t0 < 0 ? 0 : max(0, min(n, most));
    }
  } else {
    n = p.T / p.B;
    t0 = b * n;
  }
  const int L = __ldg(p.seqlens + b);
  const int start = L - n;
  const int page0 = (start >> p.page_shift) + i;                // this block's page of the sequence
  const long long first = static_cast<long long>(page0) << p.page_shift;
  if (n == 0 || first >= L) return;                             // (uniform over the block)
  const int r0 = start > first ? start - static_cast<int>(first) : 0;           // its new rows r0 .. r1 - 1
  const int r1 = static_cast<int>(L - first < p.page ? L - first : p.page);
  const int nrows = r1 - r0;
  const int tok0 = t0 + static_cast<int>(first + r0 - start);   // token of row r0

  // ---- the page
  const bool in_table = page0 >= 0 && page0 < p.width;
  const int id = in_table ? __ldg(p.table + b * p.table_stride + page0) : -1;
  const long long pbase = paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, 0, D);
  const bool store = pbase >= 0;
  if (!store && tid == 0 && hk == 0) atomicOr(p.status, in_table ? FA_DEV_BAD_PAGE : FA_DEV_BAD_LENS);
  float old_k = 0.f, old_v = 0.f;
  const long long sidx = static_cast<long long>(id) * p.Hkv + hk;
  if constexpr (F8) {
    if (store) {
      old_k = p.k_scale[sidx];
      old_v = p.v_scale[sidx];
    }
    if (tid < 2) s_amax[tid] = 0u;
    __syncthreads();
  }

  // ---- thread (row in parallel, head slot, unit): unit u has 8 pairs, or 16 elements that are not turned
  const int grp = tid / LPR, u = tid % LPR;
  const int row_lane = grp % p.rows_par, slot = grp / p.rows_par;
  const unsigned gmask = ((LPR == 32) ? 0xffffffffu : ((1u << LPR) - 1u)) << ((tid & 31) & ~(LPR - 1));
  const bool turned = u < p.rot / 16;
  const int c0 = p.interleaved ? 16 * u : (turned ? 8 * u : p.rot + 16 * (u - p.rot / 16));
  const int c1 = p.interleaved || !turned ? c0 + 8 : p.rot / 2 + 8 * u;
  float am_k = 0.f, am_v = 0.f;
  if (slot < p.head_slots) {
    for (int r = row_lane; r < nrows; r += p.rows_par) {
      const long long tok = tok0 + r;
      float cs[8], sn[8];
      for (int h0 = slot; h0 < p.G + 2; h0 += AP_BATCH * p.head_slots) {
        // the loads of AP_BATCH heads are in flight together
        uint4 raw[AP_BATCH][2];
#pragma unroll
        for (int j = 0; j < AP_BATCH; ++j) {
          const int hh = h0 + j * p.head_slots;
          if (hh < p.G + 2) {
            const uint16_t* src = hh == p.G + 1 ? static_cast<const uint16_t*>(p.v) + tok * p.vst + hk * p.vsh
                                  : hh == p.G   ? static_cast<const uint16_t*>(p.k) + tok * p.kst + hk * p.ksh
                                                : static_cast<const uint16_t*>(p.q) + tok * p.qst + (hk * p.G + hh) * p.qsh;
            raw[j][0] = ldg16(src + c0);
            raw[j][1] = ldg16(src + c1);
          }
        }
        if (h0 == slot && turned) {
          const unsigned long long pos = static_cast<unsigned long long>(first + r0 + r);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // signed 64-bit fraction of a turn in [-1/2, 1/2)
            const long long a = static_cast<long long>(pos * static_cast<unsigned long long>(__ldg(p.turns + 8 * u + j)));
            const float hi = static_cast<float>(static_cast<int>(a >> 32)), lo = static_cast<float>(static_cast<uint32_t>(a));
            const float f = fmaf(lo, 5.42101086242752217e-20f, hi * 2.3283064365386963e-10f);  // 2^-64, 2^-32
            sincospif(2.f * f, &sn[j], &cs[j]);
            sn[j] *= p.rot_scale;
            cs[j] *= p.rot_scale;
          }
        }
#pragma unroll
        for (int j = 0; j < AP_BATCH; ++j) {
          const int hh = h0 + j * p.head_slots;
          if (hh >= p.G + 2) break;
          const bool is_v = hh == p.G + 1, is_k = hh == p.G;
          if (!F8 && is_v) {
            if (store) {
              uint16_t* dst = static_cast<uint16_t*>(p.v_pages) + pbase + static_cast<long long>(r0 + r) * D;
              *reinterpret_cast<uint4*>(dst + c0) = raw[j][0];
              *reinterpret_cast<uint4*>(dst + c1) = raw[j][1];
            }
            continue;
          }
          float x[16];
          unpack8(raw[j][0], x);
          unpack8(raw[j][1], x + 8);
          if (is_v) {
            am_v = fmaxf(am_v, finite_amax(x));
            continue;
          }
          const void* wt = is_k ? p.k_weight : p.q_weight;
          if (wt != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
            const float rs = __frsqrt_rn(fmaf(ss, 1.f / D, p.eps));
            float w[16];
            unpack8(ldg16(static_cast<const uint16_t*>(wt) + c0), w);
            unpack8(ldg16(static_cast<const uint16_t*>(wt) + c1), w + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * rs * w[e];
          }
          if (turned) {
            if (p.interleaved) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float ya = fmaf(x[2 * e], cs[e], -x[2 * e + 1] * sn[e]);
                x[2 * e + 1] = fmaf(x[2 * e + 1], cs[e], x[2 * e] * sn[e]);
                x[2 * e] = ya;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float ya = fmaf(x[e], cs[e], -x[e + 8] * sn[e]);
                x[e + 8] = fmaf(x[e + 8], cs[e], x[e] * sn[e]);
                x[e] = ya;
              }
            }
          }
          const uint4 y0 = pack8(x), y1 = pack8(x + 8);
          uint16_t* out = is_k ? (p.k_out == nullptr ? nullptr : static_cast<uint16_t*>(p.k_out) + tok * p.kost + hk * p.kosh)
                               : static_cast<uint16_t*>(p.q_out) + tok * p.qost + (hk * p.G + hh) * p.qosh;
          if (out != nullptr) {
            *reinterpret_cast<uint4*>(out + c0) = y0;
            *reinterpret_cast<uint4*>(out + c1) = y1;
          }
          if (is_k && store) {
            if constexpr (F8) {
              am_k = fmaxf(am_k, finite_amax(x));
              float* st = ap_stash + r * D;
#pragma unroll
              for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4*>(st + c0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                *reinterpret_cast<float4*>(st + c1 + e) = make_float4(x[8 + e], x[9 + e], x[10 + e], x[11 + e]);
              }
            } else {
              uint16_t* dst = static_cast<uint16_t*>(p.k_pages) + pbase + static_cast<long long>(r0 + r) * D;
              *reinterpret_cast<uint4*>(dst + c0) = y0;
              *reinterpret_cast<uint4*>(dst + c1) = y1;
            }
          }
        }
      }
    }
  }
  if constexpr (F8) {
    if (!store) return;  // (uniform)
    // magnitudes order as unsigned integers; a maximum does not depend on its order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      am_k = fmaxf(am_k, __shfl_xor_sync(0xffffffffu, am_k, o));
      am_v = fmaxf(am_v, __shfl_xor_sync(0xffffffffu, am_v, o));
    }
    if ((tid & 31) == 0) {
      atomicMax(&s_amax[0], __float_as_uint(am_k));
      atomicMax(&s_amax[1], __float_as_uint(am_v));
    }
    __syncthreads();
    const float sk = merged_scale(__uint_as_float(s_amax[0]), old_k, r0 > 0);
    const float sv = merged_scale(__uint_as_float(s_amax[1]), old_v, r0 > 0);
    uint8_t* kp = static_cast<uint8_t*>(p.k_pages) + pbase;
    uint8_t* vp = static_cast<uint8_t*>(p.v_pages) + pbase;
    // the codes already held, where the scale grew
    const bool rk = r0 > 0 && sk != old_k, rvv = r0 > 0 && sv != old_v;
    if (rk || rvv) {
      const float fk = old_k > 0.f && old_k <= FLT_MAX ? old_k / sk : 1.f;
      const float fv = old_v > 0.f && old_v <= FLT_MAX ? old_v / sv : 1.f;
      for (int x = tid; x < r0 * (D / 4); x += nt) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!(w ? rvv : rk)) continue;
          uint32_t* at = reinterpret_cast<uint32_t*>(w ? vp : kp) + x;
          const uint32_t old = *at;
          const uint32_t h0 = e4m3x2_to_f16x2(old), h1 = e4m3x2_to_f16x2(old >> 16);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
          const float y[4] = {f0.x, f0.y, f1.x, f1.y};
          *at = to_codes4(y, w ? fv : fk);
        }
      }
    }
    const float ik = 1.f / sk, iv = 1.f / sv;  // exact: powers of two
    for (int x = tid; x < nrows * LPR; x += nt) {
      const int r = x / LPR, e0 = (x % LPR) * 16;
      const float* st = ap_stash + r * D + e0;
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(st + e);
        y[e] = f.x, y[e + 1] = f.y, y[e + 2] = f.z, y[e + 3] = f.w;
      }
      const long long ro = static_cast<long long>(r0 + r) * D + e0;
      *reinterpret_cast<uint4*>(kp + ro) =
          make_uint4(to_codes4(y, ik), to_codes4(y + 4, ik), to_codes4(y + 8, ik), to_codes4(y + 12, ik));
      const uint16_t* src = static_cast<const uint16_t*>(p.v) + static_cast<long long>(tok0 + r) * p.vst + hk * p.vsh + e0;
      unpack8(ldg16(src), y);
      unpack8(ldg16(src + 8), y + 8);
      *reinterpret_cast<uint4*>(vp + ro) =
          make_uint4(to_codes4(y, iv), to_codes4(y + 4, iv), to_codes4(y + 8, iv), to_codes4(y + 12, iv));
    }
    if (tid == 0) {
      p.k_scale[sidx] = sk;
      p.v_scale[sidx] = sv;
    }
  }
}

cudaError_t append_paged_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(fa_append_paged_kernel<64, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 64 * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(fa_append_paged_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 128 * 4);
}

template <int D, bool F8>
static cudaError_t ap_launch(const AppendPagedParams& p, cudaStream_t stream) {
  const long long blocks = (p.per_seq > 0 ? static_cast<long long>(p.B) * p.per_seq : p.T / p.page + 2ll * p.B) * p.Hkv;
  const int groups = p.rows_par * p.head_slots;
  const int threads = (groups * (D / 16) + 31) / 32 * 32;
  const size_t smem = F8 ? static_cast<size_t>(p.stash_rows) * D * 4 : 0;
  fa_append_paged_kernel<D, F8><<<static_cast<unsigned>(blocks), threads, smem, stream>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_append_paged(bool f8, const AppendPagedParams& p, cudaStream_t stream) {
  if (p.d == 64) return f8 ? ap_launch<64, true>(p, stream) : ap_launch<64, false>(p, stream);
  return f8 ? ap_launch<128, true>(p, stream) : ap_launch<128, false>(p, stream);
}

}  // namespace fa
