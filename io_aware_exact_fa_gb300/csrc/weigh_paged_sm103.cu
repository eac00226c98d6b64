// Accumulated attention weights over a paged K cache for sm_103a: for every key j
// of sequence b and K/V head hk
//     weights[b, hk, j] += sum over rows r that see j of exp(scale <q_r, k_j> - lse_r),
// where the rows are the (head, token) pairs of the head's group and lse_r what a
// forward pass over the same keys returned. Rows with lse = -inf add nothing.
//
// What bounds it: HBM for a step's few rows (a key's row read once, its weight read
// and written), the warp-level products for a window of many (2 d operations for
// each of up to 128 rows and key). With the log-sum-exp given there is no running
// maximum and nothing to merge: every 16 keys are on their own. The keys are the M
// side of S^T = K Q^T, as in the paged decode, and stay in registers as fragments
// while the 8-row tiles of the queries pass by on the N side (fragments in shared
// memory, laid out once a block); a row's sum over the queries is then four lanes'
// partial sums, so no atomics, and results do not depend on any order.
//
// A block takes `chunk` keys of one sequence and K/V head; its warps take tiles of
// them in turn and load the next tile's rows, and the page entries of the one after,
// before they work on the current one.
#include <climits>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

constexpr int WG_WARPS = 4;
constexpr int WG_THREADS = 32 * WG_WARPS;

template <int D, int KIND>
struct WgCfg {
  static constexpr bool F16 = KIND != PAGES_BF16;
  static constexpr int RB = paged_row_bytes(KIND, D);
  static constexpr int KST = D / 16;                 // k-steps
  static constexpr int LB = RB / 4;                  // bytes of a row that one lane holds: 8, 16, 32 or 64
  static constexpr int LW = LB / 4;                  // as words
  static constexpr int KG = KIND == PAGES_FP4 ? 4 : 64 / LB;  // 16-key groups of a warp's tile
  static constexpr int TILE = 16 * KG;
};

// Rows gid and gid + 8 of a group: the lane's share of each.
template <int D, int KIND>
struct WgRaw {
  uint32_t w[2][WgCfg<D, KIND>::LW];
  uint32_t f[2];  // 4-bit rows: the lane's one or two scale bytes
};

// Lane tig and k-step j of the four elements 4 x .. 4 x + 3 of a row, in the order that the lanes hold keys: 16-byte
// pieces tig, tig + 4, ..., or a quarter of a 4-bit row.
template <int D, int KIND>
__device__ __forceinline__ void wg_place(int x, int& tig, int& j) {
  if constexpr (KIND == PAGES_FP4) {
    tig = x / (D / 16);
    j = x % (D / 16);
  } else {
    constexpr int Q = KIND == PAGES_E4M3 ? 4 : 2;  // fours of elements in a piece
    tig = (x / Q) % 4;
    j = x / Q / 4 * Q + x % Q;
  }
}

}  // namespace

template <int D, int KIND>
__global__ void __launch_bounds__(WG_THREADS, 3) fa_weigh_paged_kernel(const WeighPagedParams p) {
  using C = WgCfg<D, KIND>;
  constexpr unsigned ALL = 0xffffffffu;
  extern __shared__ __align__(16) uint8_t wg_smem[];
  uint2* s_q = reinterpret_cast<uint2*>(wg_smem);                                   // [row tile][k-step][lane]
  float4* s_row = reinterpret_cast<float4*>(wg_smem + p.row_tiles * C::KST * 256);  // of rows 2i, 2i + 1: factors, lse
  int2* s_lim = reinterpret_cast<int2*>(s_row + p.row_tiles * 4);                   // and the last key they see
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int part = static_cast<int>(blockIdx.x) % p.chunks, pair = static_cast<int>(blockIdx.x) / p.chunks;
  const int b = pair / p.Hkv, hk = pair % p.Hkv;
  const int raw_len = __ldg(p.seqlens + b), L = paged_clip_len(raw_len, p.max_len);
  if (raw_len != L && part == 0 && hk == 0 && threadIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const int first = part * p.chunk;
  if (first >= L) return;
  const int end = min(L, first + p.chunk);

  // ---- the warp's tiles: first + (warp + WG_WARPS i) TILE
  int key0 = first + warp * C::TILE;
  auto page_of = [&](int k0) -> int {
    const int key = k0 + 16 * lane;
    return (lane < C::KG && key < end) ? __ldg(p.table + b * p.table_stride + (key >> p.page_shift)) : -1;
  };
  WgRaw<D, KIND> raw[C::KG];
  float ka[C::KG];
  uint32_t live = 0u;  // groups that have keys, in a page of the pool
  auto load = [&](int k0, int id) {
    const int gkey = k0 + 16 * lane;
    const bool want = lane < C::KG && gkey < end;
    const long long off = want ? paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, gkey & (p.page - 1), 1) : -1;
    if (__any_sync(ALL, want && off < 0) && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
    live = __ballot_sync(ALL, off >= 0);
    float scale = 1.f;
    if constexpr (KIND == PAGES_E4M3)
      if (off >= 0) scale = __ldg(static_cast<const float*>(p.k_scale) + static_cast<long long>(id) * p.Hkv + hk);
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      const long long row0 = __shfl_sync(ALL, off, g);
      ka[g] = KIND == PAGES_E4M3 ? __shfl_sync(ALL, scale, g) : 1.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = gid + 8 * h;
        const bool in = row0 >= 0 && k0 + 16 * g + r < end;
        const uint8_t* src = static_cast<const uint8_t*>(p.k) + (in ? row0 + r : 0) * C::RB;
        if constexpr (KIND == PAGES_FP4) {
          const uint8_t* sp = static_cast<const uint8_t*>(p.k_scale) + (in ? row0 + r : 0) * (D / 16);
          if constexpr (D == 128) {
            const uint4 y = in ? __ldg(reinterpret_cast<const uint4*>(src) + tig) : make_uint4(0, 0, 0, 0);
            raw[g].w[h][0] = y.x, raw[g].w[h][1] = y.y, raw[g].w[h][2] = y.z, raw[g].w[h][3] = y.w;
            raw[g].f[h] = in ? __ldg(reinterpret_cast<const uint16_t*>(sp) + tig) : 0u;
          } else {
            const uint2 y = in ? __ldg(reinterpret_cast<const uint2*>(src) + tig) : make_uint2(0, 0);
            raw[g].w[h][0] = y.x, raw[g].w[h][1] = y.y;
            raw[g].f[h] = in ? __ldg(sp + tig) : 0u;
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::LW / 4; ++i) {
            const uint4 y = in ? __ldg(reinterpret_cast<const uint4*>(src) + tig + 4 * i) : make_uint4(0, 0, 0, 0);
            raw[g].w[h][4 * i] = y.x, raw[g].w[h][4 * i + 1] = y.y, raw[g].w[h][4 * i + 2] = y.z, raw[g].w[h][4 * i + 3] = y.w;
          }
        }
      }
    }
  };
  load(key0, page_of(key0));
  constexpr int STEP = WG_WARPS * C::TILE;
  int id = page_of(key0 + STEP);

  // ---- the queries: a warp a row, a lane four of its elements
  for (int r = warp; r < 8 * p.row_tiles; r += WG_WARPS) {
    const bool in = r < p.R;
    const int h = hk * p.G + (in ? r / p.Nq : 0), tok = in ? r % p.Nq : 0;
    uint2 x = make_uint2(0u, 0u);
    if (in && lane < D / 4)
      x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + b * p.qsb + h * p.qsh + tok * p.qst) + lane);
    float factor = p.scale_log2;
    if constexpr (C::F16) {
      // as in the paged decode: the row's power of two brings its largest element to [1, 2), so that all but elements
      // below 2^-14 of it are exact in f16
      const float e[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                          __uint_as_float(x.y & 0xffff0000u)};
      float amax = fmaxf(fmaxf(fabsf(e[0]), fabsf(e[1])), fmaxf(fabsf(e[2]), fabsf(e[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, o));
      const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -120), 120);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      factor *= __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      x = make_uint2(pack_f16x2(e[0] * down, e[1] * down), pack_f16x2(e[2] * down, e[3] * down));
    }
    if (lane < D / 4) {
      int qt, j;
      wg_place<D, KIND>(lane, qt, j);
      s_q[((r / 8) * C::KST + j) * 32 + (r % 8) * 4 + qt] = x;
    }
    if (lane == 0) {
      const float lse = in ? __ldg(p.lse + (static_cast<long long>(b) * p.H + h) * p.Nq + tok) : -INFINITY;
      const bool none = lse == -INFINITY;
      float* f = reinterpret_cast<float*>(s_row + r / 2) + (r & 1);
      f[0] = factor;
      f[2] = none ? 0.f : lse * 1.4426950408889634f;
      reinterpret_cast<int*>(s_lim + r / 2)[r & 1] = none ? -1 : min(L - 1, L - p.Nq + tok);
    }
  }
  __syncthreads();

  float* wrow = p.weights + (static_cast<long long>(b) * p.Hkv + hk) * p.wstride;
  for (; key0 < end; key0 += STEP) {
    // this tile's rows become fragments group by group; the next tile's loads follow the last group
    const uint32_t now = live;
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      uint32_t a[C::KST][4];
      const float kf = ka[g];
      if constexpr (KIND == PAGES_FP4) {
        const uint32_t fa[2] = {fp4_scale2<0>(raw[g].f[0]), fp4_scale2<1>(raw[g].f[0])};
        const uint32_t fb[2] = {fp4_scale2<0>(raw[g].f[1]), fp4_scale2<1>(raw[g].f[1])};
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          uint32_t y[4], z[4];
          e2m1x8_to_f16x2x4(raw[g].w[0][x], y);
          e2m1x8_to_f16x2x4(raw[g].w[1][x], z);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[2 * x + e / 2][2 * (e & 1)] = hmul2_bits(y[e], fa[x >> 1]);
            a[2 * x + e / 2][2 * (e & 1) + 1] = hmul2_bits(z[e], fb[x >> 1]);
          }
        }
      } else if constexpr (KIND == PAGES_E4M3) {
#pragma unroll
        for (int x = 0; x < C::LW; ++x) {
          e4m3x4_to_f16x2x2(raw[g].w[0][x], a[x][0], a[x][2]);
          e4m3x4_to_f16x2x2(raw[g].w[1][x], a[x][1], a[x][3]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < C::KST; ++x) {
          a[x][0] = raw[g].w[0][2 * x], a[x][2] = raw[g].w[0][2 * x + 1];
          a[x][1] = raw[g].w[1][2 * x], a[x][3] = raw[g].w[1][2 * x + 1];
        }
      }
      if (g == C::KG - 1 && key0 + STEP < end) {
        load(key0 + STEP, id);
        id = page_of(key0 + 2 * STEP);
      }
      if (!((now >> g) & 1u)) continue;  // (the same in every lane)
      const int key = key0 + 16 * g + gid;
      const int mine = key + 8 * tig;    // the key whose weight this lane writes (tig 0 and 1)
      const bool writes = tig < 2 && mine < end;
      const float old = writes ? wrow[mine] : 0.f;
      float sum0 = 0.f, sum1 = 0.f;      // keys gid and gid + 8, rows 2 tig and 2 tig + 1 of each tile
#pragma unroll 1
      for (int n = 0; n < p.row_tiles; ++n) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const uint2* qn = s_q + n * C::KST * 32 + lane;
#pragma unroll
        for (int j = 0; j < C::KST; ++j) {
          const uint2 q = qn[j * 32];
          mma_16816<C::F16>(s, a[j][0], a[j][1], a[j][2], a[j][3], q.x, q.y);
        }
        const float4 f = s_row[n * 4 + tig];
        const int2 lim = s_lim[n * 4 + tig];
        const float c0 = KIND == PAGES_E4M3 ? f.x * kf : f.x, c1 = KIND == PAGES_E4M3 ? f.y * kf : f.y;
        const float p0 = ex2_approx(fmaf(s[0], c0, -f.z)), p1 = ex2_approx(fmaf(s[1], c1, -f.w));
        const float p2 = ex2_approx(fmaf(s[2], c0, -f.z)), p3 = ex2_approx(fmaf(s[3], c1, -f.w));
        sum0 += (key <= lim.x ? p0 : 0.f) + (key <= lim.y ? p1 : 0.f);
        sum1 += (key + 8 <= lim.x ? p2 : 0.f) + (key + 8 <= lim.y ? p3 : 0.f);
      }
      sum0 += __shfl_xor_sync(ALL, sum0, 1);
      sum1 += __shfl_xor_sync(ALL, sum1, 1);
      sum0 += __shfl_xor_sync(ALL, sum0, 2);
      sum1 += __shfl_xor_sync(ALL, sum1, 2);
      if (writes) wrow[mine] = old + (tig == 0 ? sum0 : sum1);
    }
  }
}

template <int D, int KIND>
static int wg_smem(int row_tiles) {
  return row_tiles * (WgCfg<D, KIND>::KST * 256 + 4 * 16 + 4 * 8);
}
template <int KIND>
static cudaError_t wg_attrs() {
  const cudaError_t a = cudaFuncSetAttribute(fa_weigh_paged_kernel<64, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             wg_smem<64, KIND>(16));
  const cudaError_t b = cudaFuncSetAttribute(fa_weigh_paged_kernel<128, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             wg_smem<128, KIND>(16));
  return a != cudaSuccess ? a : b;
}
cudaError_t weigh_paged_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {wg_attrs<PAGES_BF16>(), wg_attrs<PAGES_E4M3>(), wg_attrs<PAGES_FP4>()})
    if (x != cudaSuccess) e = x;
  return e;
}

template <int D, int KIND>
static cudaError_t wg_launch(WeighPagedParams p, int num_sms, cudaStream_t stream) {
  // Keys of a block: from two tiles a warp up to 64, as many as leave the GPU six blocks an SM.
  constexpr int STEP = WG_WARPS * WgCfg<D, KIND>::TILE;
  const long long pairs = static_cast<long long>(p.B) * p.Hkv;
  long long chunk = 2LL * STEP;
  auto blocks = [&](long long c) { return (p.max_len + c - 1) / c * pairs; };
  while (chunk < p.max_len && ((chunk < 64LL * STEP && blocks(2 * chunk) >= 6LL * num_sms) || blocks(chunk) > INT_MAX)) chunk *= 2;
  p.chunk = static_cast<int>(chunk);
  p.chunks = static_cast<int>((p.max_len + chunk - 1) / chunk);
  if (p.chunks == 0) return cudaSuccess;  // no keys
  fa_weigh_paged_kernel<D, KIND><<<static_cast<unsigned>(blocks(chunk)), WG_THREADS, wg_smem<D, KIND>(p.row_tiles), stream>>>(p);
  return cudaGetLastError();
}
template <int D>
static cudaError_t wg_launch_kind(int kind, const WeighPagedParams& p, int num_sms, cudaStream_t stream) {
  if (kind == PAGES_FP4) return wg_launch<D, PAGES_FP4>(p, num_sms, stream);
  return kind == PAGES_E4M3 ? wg_launch<D, PAGES_E4M3>(p, num_sms, stream) : wg_launch<D, PAGES_BF16>(p, num_sms, stream);
}
cudaError_t launch_weigh_paged(int d, int kind, WeighPagedParams p, int num_sms, cudaStream_t stream) {
  return d == 64 ? wg_launch_kind<64>(kind, p, num_sms, stream) : wg_launch_kind<128>(kind, p, num_sms, stream);
}

}  // namespace fa
