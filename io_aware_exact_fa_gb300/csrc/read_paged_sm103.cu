// Rows of a paged cache (bf16, e4m3 or 4-bit pages) as packed bf16 keys and values
// for sm_103a: packed row cu[b] + i is row L_b - n_b + i of sequence b, where
// n_b = cu[b + 1] - cu[b] rows are asked for, its last ones (all of them, or a
// call's new tokens).
//
// An e4m3 value is code * scale, rounded once to bf16 (exact for a power of two); a
// 4-bit value is exact in bf16. What bounds it: HBM, mostly the writes (d = 128,
// 4-bit: 144 bytes read and 512 written for each row and K/V head). A block takes 32
// packed rows of all heads: its first threads find their sequence (by bisection of
// the offsets) and page, then every thread turns 8 elements of a key and of a value
// into 16 bytes each, which a warp writes side by side (with 16 elements a thread, two
// stores 32 bytes apart, L1 was the bound: 76 us in place of 55 for 65.5k rows of 8 heads, d = 128).
// Neighbouring threads take a row's units, then the next row of the same head, so
// reads run along the page.
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

// All loads are __ldcg, past L1 and never through the read-only path: a large launch begins while the launch that writes these
// rows, scales and lengths still runs, so the memory is not constant for its duration, and an SM's L1 may hold what that one
// read there before (the scales of eight pages and heads share a sector).
constexpr int RD_THREADS = 256;
constexpr int RD_ROWS = 32;      // packed rows of a block
constexpr int RD_FLIGHT = 4;     // units of K and V whose loads a thread has in flight
// Blocks from which on the launch is a dependent one, beside the tail of what comes before: it saves the GPU 1 to 3 us (143.5 ->
// 142 us for 26k rows appended and read back, 64 -> 62 for 9 chunks, 122 -> 120 behind an eviction) and costs the host 3 to 5 (12 -> 16 us for 8 rows).
constexpr unsigned RD_BESIDE = 512;

// Eight elements as they lie in the page: 16, 8 or 4 bytes, and their scale (4-bit rows: its byte).
struct Unit {
  uint4 a;
  float scale;
  uint32_t byte;
};

template <int D, int KIND>
__device__ __forceinline__ void rd_load(Unit& x, const void* pages, const void* scales, long long row, long long ph, int u) {
  constexpr int RB = paged_row_bytes(KIND, D);
  const uint8_t* at = static_cast<const uint8_t*>(pages) + row * RB + u * (RB / (D / 8));
  if constexpr (KIND == PAGES_BF16) {
    x.a = __ldcg(reinterpret_cast<const uint4*>(at));
  } else if constexpr (KIND == PAGES_E4M3) {
    const uint2 c = __ldcg(reinterpret_cast<const uint2*>(at));
    x.a.x = c.x, x.a.y = c.y;
    x.scale = __ldcg(static_cast<const float*>(scales) + ph);
  } else {
    x.a.x = __ldcg(reinterpret_cast<const uint32_t*>(at));
    x.byte = __ldcg(static_cast<const uint8_t*>(scales) + row * (D / 16) + u / 2);
  }
}

__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h, float f) {
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(y.x * f, y.y * f);
}

template <int KIND>
__device__ __forceinline__ uint4 rd_bf16(const Unit& x) {
  if constexpr (KIND == PAGES_BF16) {
    return x.a;
  } else {
    uint32_t h[4];
    float f = 1.f;
    if constexpr (KIND == PAGES_E4M3) {
      f = x.scale;
      e4m3x4_to_f16x2x2(x.a.x, h[0], h[1]);
      e4m3x4_to_f16x2x2(x.a.y, h[2], h[3]);
    } else {
      const uint32_t s2 = fp4_scale2<0>(x.byte);
      e2m1x8_to_f16x2x4(x.a.x, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = hmul2_bits(h[i], s2);
    }
    return make_uint4(half2_to_bf16x2(h[0], f), half2_to_bf16x2(h[1], f), half2_to_bf16x2(h[2], f), half2_to_bf16x2(h[3], f));
  }
}

}  // namespace

template <int D, int KIND>
__global__ void __launch_bounds__(RD_THREADS) fa_read_paged_kernel(const ReadPagedParams p) {
  constexpr int UNITS = D / 8;
  __shared__ long long s_base[RD_ROWS];  // its row of K/V head 0 in the pool, or -1
  const int tid = threadIdx.x;
  const int t0 = static_cast<int>(blockIdx.x) * RD_ROWS;
  pdl_wait();  // (launched beside the tail of what comes before it, most often what writes these rows)
  if (blockIdx.x == 0) {  // offsets that decrease or pass the tensors are reported; rows outside are left alone below
    bool bad = false;
    for (int b = tid; b < p.B; b += RD_THREADS) {
      const int lo = __ldcg(p.cu + b), hi = __ldcg(p.cu + b + 1), L = __ldcg(p.seqlens + b);
      bad = bad || lo < 0 || hi < lo || hi > p.total || L < 0 || L > static_cast<long long>(p.width) * p.page ||
            (L > 0 && hi - lo > L);
    }
    if (bad) atomicOr(p.status, FA_DEV_BAD_LENS);
  }
  if (tid < RD_ROWS) {
    const int t = t0 + tid;
    long long base = -1;
    if (t < p.total) {
      int lo = 0, n = p.B;  // the last sequence that starts at or before row t
      while (n > 1) {
        const int half = n / 2;
        if (__ldcg(p.cu + lo + half) <= t) {
          lo += half;
          n -= half;
        } else {
          n = half;
        }
      }
      const int first = __ldcg(p.cu + lo), end = __ldcg(p.cu + lo + 1);
      const int L = __ldcg(p.seqlens + lo);
      const long long row = static_cast<long long>(L) - (static_cast<long long>(end) - t);
      if (t >= first && t < end && row >= 0 && row < static_cast<long long>(p.width) * p.page) {
        const int id = __ldcg(p.table + lo * p.table_stride + (row >> p.page_shift));
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages))
          base = static_cast<long long>(id) * p.Hkv * p.page + (row & (p.page - 1));
        else
          atomicOr(p.status, FA_DEV_BAD_PAGE);
      }
    }
    s_base[tid] = base;
  }
  __syncthreads();
  const int rows = min(RD_ROWS, p.total - t0);
  const int items = rows * p.Hkv * UNITS;
  for (int x0 = tid; x0 < items; x0 += RD_FLIGHT * RD_THREADS) {
    Unit k[RD_FLIGHT], v[RD_FLIGHT];
    bool ok[RD_FLIGHT];
    int u[RD_FLIGHT], r[RD_FLIGHT], hk[RD_FLIGHT];
#pragma unroll
    for (int i = 0; i < RD_FLIGHT; ++i) {
      const int x = x0 + i * RD_THREADS;
      u[i] = x % UNITS;
      hk[i] = (x / UNITS) / rows;
      r[i] = (x / UNITS) % rows;
      const long long base = x < items ? s_base[r[i]] : -1;
      ok[i] = base >= 0;
      if (ok[i]) {
        const long long row = base + static_cast<long long>(hk[i]) * p.page;
        const long long ph = row >> p.page_shift;  // page and head
        rd_load<D, KIND>(k[i], p.k, p.k_scale, row, ph, u[i]);
        rd_load<D, KIND>(v[i], p.v, p.v_scale, row, ph, u[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < RD_FLIGHT; ++i) {
      if (!ok[i]) continue;
      const long long t = t0 + r[i];
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_out) + t * p.kst + hk[i] * p.ksh + 8 * u[i]) = rd_bf16<KIND>(k[i]);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_out) + t * p.vst + hk[i] * p.vsh + 8 * u[i]) = rd_bf16<KIND>(v[i]);
    }
  }
}

template <int D>
static cudaError_t rd_launch(int kind, const ReadPagedParams& p, cudaStream_t stream) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.total) + RD_ROWS - 1) / RD_ROWS));
  cfg.blockDim = dim3(RD_THREADS);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = cfg.gridDim.x >= RD_BESIDE ? 1 : 0;
  if (kind == PAGES_FP4) return cudaLaunchKernelEx(&cfg, fa_read_paged_kernel<D, PAGES_FP4>, p);
  return kind == PAGES_E4M3 ? cudaLaunchKernelEx(&cfg, fa_read_paged_kernel<D, PAGES_E4M3>, p)
                            : cudaLaunchKernelEx(&cfg, fa_read_paged_kernel<D, PAGES_BF16>, p);
}
cudaError_t launch_read_paged(int d, int kind, const ReadPagedParams& p, cudaStream_t stream) {
  return d == 64 ? rd_launch<64>(kind, p, stream) : rd_launch<128>(kind, p, stream);
}

}  // namespace fa
