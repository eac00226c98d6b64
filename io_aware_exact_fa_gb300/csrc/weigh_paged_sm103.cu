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
// The batch's keys are shared out in equal contiguous ranges, as in the paged decode:
// one for each warp that the GPU holds where a K/V head has up to 16 query rows
// (whose fragments then stay in registers), one for each block above that. The
// next tile's rows, and the page entries of the one after, are loaded before a
// warp works on the current one.
#include <type_traits>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged_walk.cuh"

namespace fa {

namespace {

constexpr int WG_WARPS = 4;
constexpr int WG_THREADS = 32 * WG_WARPS;
constexpr int WG_FEW_CTAS = 4;   // blocks of the kernel for few rows that an SM holds
constexpr unsigned ALL = 0xffffffffu;

template <int D, int KIND>
struct WgCfg {
  static constexpr bool F16 = KIND != PAGES_BF16;
  static constexpr int RB = paged_row_bytes(KIND, D);
  static constexpr int KST = D / 16;                 // k-steps
  static constexpr int LB = RB / 4;                  // bytes of a row that one lane holds: 8, 16, 32 or 64
  static constexpr int LW = LB / 4;                  // as words
  static constexpr int KG = KIND == PAGES_FP4 ? 4 : 64 / LB;  // 16-key groups of a warp's tile: 4, 2 or 1
  static constexpr int TILE = 16 * KG;
};

// Rows gid and gid + 8 of a group: the lane's share of each.
template <int D, int KIND>
struct WgRaw {
  uint32_t w[2][WgCfg<D, KIND>::LW];
  uint32_t f[2];  // 4-bit rows: the lane's one or two scale bytes
};

// The lane's share of the rows gid, gid + 8 of a group whose first row is `row0` of the pool. Past its `rows` rows the last
// one is read again, and of a group that is not there (row0 < 0) the pool's first: every key's sum is its own, and those are
// not written, so no load needs a branch.
template <int D, int KIND>
__device__ __forceinline__ void wg_load(WgRaw<D, KIND>& x, const WeighPagedParams& p, long long row0, int rows, int gid, int tig) {
  using C = WgCfg<D, KIND>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long row = row0 < 0 ? 0 : row0 + max(min(gid + 8 * h, rows - 1), 0);
    const uint8_t* src = static_cast<const uint8_t*>(p.k) + row * C::RB;
    if constexpr (KIND == PAGES_FP4) {
      const uint8_t* sp = static_cast<const uint8_t*>(p.k_scale) + row * (D / 16);
      if constexpr (D == 128) {
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(src) + tig);
        x.w[h][0] = y.x, x.w[h][1] = y.y, x.w[h][2] = y.z, x.w[h][3] = y.w;
        x.f[h] = __ldg(reinterpret_cast<const uint16_t*>(sp) + tig);
      } else {
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(src) + tig);
        x.w[h][0] = y.x, x.w[h][1] = y.y;
        x.f[h] = __ldg(sp + tig);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C::LW / 4; ++i) {
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(src) + tig + 4 * i);
        x.w[h][4 * i] = y.x, x.w[h][4 * i + 1] = y.y, x.w[h][4 * i + 2] = y.z, x.w[h][4 * i + 3] = y.w;
      }
    }
  }
}

// The two rows' A fragments of every k-step, handed on as soon as they are made: f(k-step, a0, a1, a2, a3).
template <int D, int KIND, class F>
__device__ __forceinline__ void wg_fragments(const WgRaw<D, KIND>& x, F&& f) {
  using C = WgCfg<D, KIND>;
  if constexpr (KIND == PAGES_FP4) {
    const uint32_t fa[2] = {fp4_scale2<0>(x.f[0]), fp4_scale2<1>(x.f[0])};
    const uint32_t fb[2] = {fp4_scale2<0>(x.f[1]), fp4_scale2<1>(x.f[1])};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t y[4], z[4];
      e2m1x8_to_f16x2x4(x.w[0][i], y);
      e2m1x8_to_f16x2x4(x.w[1][i], z);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        f(2 * i + e, hmul2_bits(y[2 * e], fa[i >> 1]), hmul2_bits(z[2 * e], fb[i >> 1]), hmul2_bits(y[2 * e + 1], fa[i >> 1]),
          hmul2_bits(z[2 * e + 1], fb[i >> 1]));
    }
  } else if constexpr (KIND == PAGES_E4M3) {
#pragma unroll
    for (int i = 0; i < C::LW; ++i) {
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_f16x2x2(x.w[0][i], a0, a2);
      e4m3x4_to_f16x2x2(x.w[1][i], a1, a3);
      f(i, a0, a1, a2, a3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C::KST; ++i) f(i, x.w[0][2 * i], x.w[1][2 * i], x.w[0][2 * i + 1], x.w[1][2 * i + 1]);
  }
}

// First of the four elements that lane tig holds in k-step j: its keys are 16-byte pieces tig, tig + 4, ..., or a quarter of
// a 4-bit row.
template <int D, int KIND>
__device__ __forceinline__ int wg_elem(int tig, int j) {
  if constexpr (KIND == PAGES_FP4) return 4 * (tig * (D / 16) + j);
  constexpr int Q = KIND == PAGES_E4M3 ? 4 : 2;
  return 4 * ((j / Q * 4 + tig) * Q + j % Q);
}

// Largest magnitude of four bf16 values.
__device__ __forceinline__ float wg_amax(uint2 x) {
  return fmaxf(fmaxf(fabsf(__uint_as_float(x.x << 16)), fabsf(__uint_as_float(x.x & 0xffff0000u))),
               fmaxf(fabsf(__uint_as_float(x.y << 16)), fabsf(__uint_as_float(x.y & 0xffff0000u))));
}
// As in the paged decode, codes meet queries in f16: the row's power of two brings its largest element to [1, 2), so that all
// but elements below 2^-14 of it are exact. `up` is the power.
__device__ __forceinline__ float wg_powers(float amax, float& up) {
  const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -120), 120);
  up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
}
__device__ __forceinline__ uint2 wg_to_f16(uint2 x, float down) {
  return make_uint2(pack_f16x2(__uint_as_float(x.x << 16) * down, __uint_as_float(x.x & 0xffff0000u) * down),
                    pack_f16x2(__uint_as_float(x.y << 16) * down, __uint_as_float(x.y & 0xffff0000u) * down));
}

// Sums v[g][h] (group g, key gid + 8 h) over the four lanes tig: afterwards v[x][0] of lane tig is that of group
// g(x) = x + (tig / 2) KG / 2 and key gid + 8 (tig % 2); with one group lanes 2 and 3 hold what 0 and 1 do.
template <int KG>
__device__ __forceinline__ void wg_sum_lanes(float (&v)[KG][2], int tig) {
#pragma unroll
  for (int g = 0; g < KG; ++g) {
    const float mine = (tig & 1) ? v[g][1] : v[g][0], other = (tig & 1) ? v[g][0] : v[g][1];
    v[g][0] = mine + __shfl_xor_sync(ALL, other, 1);
  }
  if constexpr (KG == 1) {
    v[0][0] += __shfl_xor_sync(ALL, v[0][0], 2);
  } else {
#pragma unroll
    for (int x = 0; x < KG / 2; ++x) {
      const float mine = (tig & 2) ? v[x + KG / 2][0] : v[x][0], other = (tig & 2) ? v[x][0] : v[x + KG / 2][0];
      v[x][0] = mine + __shfl_xor_sync(ALL, other, 2);
    }
  }
}

}  // namespace

// ---- up to 8 or 16 rows a K/V head: the queries' fragments stay in registers
template <int D, int KIND, int NR>
__global__ void __launch_bounds__(WG_THREADS, NR == 1 ? WG_FEW_CTAS : 3) fa_weigh_paged_few_kernel(const WeighPagedParams p) {
  using C = WgCfg<D, KIND>;
  constexpr int KG = C::KG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int range = static_cast<int>(blockIdx.x) * WG_WARPS + warp;
  bool clipped = false;
  const long long sum = paged_count_tiles<C::TILE>(p.seqlens, p.B, p.max_len, lane, clipped);
  if (range == 0 && __any_sync(ALL, clipped) && lane == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const PagedRanges ranges(sum * p.Hkv, p.n_ranges);
  if (range >= ranges.n) return;
  const long long t0 = ranges.begin(range);
  int todo = static_cast<int>(ranges.begin(range + 1) - t0);
  PagedTile at = paged_seek<C::TILE>(p.seqlens, p.B, p.Hkv, p.max_len, t0, lane);

  // ---- loads run a tile ahead (each group's as soon as the one before is used), page entries two
  PagedTile ahead = at;
  int to_load = todo;
  auto page_of = [&]() -> int {
    const int key = ahead.i * C::TILE + 16 * lane;
    return (lane < KG && to_load > 0 && key < ahead.L) ? __ldg(p.table + ahead.b * p.table_stride + (key >> p.page_shift)) : -1;
  };
  int id = page_of();
  WgRaw<D, KIND> raw[KG];
  float ka[KG];
  // of the tile that is loaded next: row of the lane's group, its rows, the groups to work on, e4m3 scale
  long long off = -1;
  int rows = 0;
  unsigned next_live = 0u;
  float scale = 1.f;
  auto locate = [&]() {
    const int key = ahead.i * C::TILE + 16 * lane;
    const bool want = lane < KG && to_load > 0 && key < ahead.L;
    off = want ? paged_row_offset(id, p.num_pages, p.Hkv, ahead.hk, p.page, key & (p.page - 1), 1) : -1;
    if (__any_sync(ALL, want && off < 0) && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
    rows = ahead.L - ahead.i * C::TILE;
    next_live = __ballot_sync(ALL, off >= 0);
    if constexpr (KIND == PAGES_E4M3)
      scale = off >= 0 ? __ldg(static_cast<const float*>(p.k_scale) + static_cast<long long>(id) * p.Hkv + ahead.hk) : 0.f;
    if (to_load > 0) {
      --to_load;
      if (to_load > 0) paged_next<C::TILE>(ahead, p.seqlens, p.B, p.Hkv, p.max_len);
      id = page_of();
    }
  };
  locate();
#pragma unroll
  for (int g = 0; g < KG; ++g) {
    wg_load<D, KIND>(raw[g], p, __shfl_sync(ALL, off, g), rows - 16 * g, gid, tig);
    ka[g] = __shfl_sync(ALL, scale, g);
  }
  unsigned live = next_live;

  while (todo > 0) {
    // ================================================================ one segment: keys of (b, hk) from tile i on
    const int b = at.b, hk = at.hk, L = at.L, i1 = todo < at.nt - at.i ? at.i + todo : at.nt;
    uint2 qf[NR][C::KST];
    float c1[NR][2], ls[NR][2];  // factors of the scores of rows 2 tig and 2 tig + 1, their log-sum-exp (log2 units)
    int lim[NR][2];              // the last key they see; -1: the row adds nothing
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = n * 8 + gid;
      const bool in = r < p.R;
      const uint16_t* qr = static_cast<const uint16_t*>(p.q) + b * p.qsb + (hk * p.G + (in ? r / p.Nq : 0)) * p.qsh +
                           (in ? r % p.Nq : 0) * p.qst;
      float amax = 0.f, up = 1.f;
#pragma unroll
      for (int j = 0; j < C::KST; ++j) {
        qf[n][j] = in ? __ldg(reinterpret_cast<const uint2*>(qr + wg_elem<D, KIND>(tig, j))) : make_uint2(0u, 0u);
        if (C::F16) amax = fmaxf(amax, wg_amax(qf[n][j]));
      }
      if constexpr (C::F16) {
        amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, 2));
        const float down = wg_powers(amax, up);
#pragma unroll
        for (int j = 0; j < C::KST; ++j) qf[n][j] = wg_to_f16(qf[n][j], down);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c1[n][e] = p.scale_log2 * (C::F16 ? __shfl_sync(ALL, up, (2 * tig + e) * 4) : 1.f);
        const int r2 = n * 8 + 2 * tig + e;
        const bool real = r2 < p.R;
        const int h2 = hk * p.G + (real ? r2 / p.Nq : 0), tok = real ? r2 % p.Nq : 0;
        const float lse = real ? __ldg(p.lse + (static_cast<long long>(b) * p.H + h2) * p.Nq + tok) : -INFINITY;
        const bool none = lse == -INFINITY;
        ls[n][e] = none ? 0.f : lse * 1.4426950408889634f;
        lim[n][e] = none ? -1 : min(L - 1, L - p.Nq + tok);
      }
    }
    float* wrow = p.weights + (static_cast<long long>(b) * p.Hkv + hk) * p.wstride;

    for (; at.i < i1; ++at.i) {
      const int key0 = at.i * C::TILE;
      // the weights of this lane's keys
      constexpr int OWN = KG > 1 ? KG / 2 : 1;
      float old[OWN];
      int mine[OWN];
      bool writes[OWN];
#pragma unroll
      for (int x = 0; x < OWN; ++x) {
        const int g = x + (tig >> 1) * (KG / 2);
        mine[x] = key0 + 16 * g + gid + 8 * (tig & 1);
        writes[x] = ((live >> g) & 1u) && mine[x] < L && (KG > 1 || tig < 2);
        old[x] = writes[x] ? wrow[mine[x]] : 0.f;
      }
      locate();
      float v[KG][2];
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        float s[NR][4];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
        wg_fragments<D, KIND>(raw[g], [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int n = 0; n < NR; ++n) mma_16816<C::F16>(s[n], a0, a1, a2, a3, qf[n][j].x, qf[n][j].y);
        });
        const float kf = ka[g];
        wg_load<D, KIND>(raw[g], p, __shfl_sync(ALL, off, g), rows - 16 * g, gid, tig);
        ka[g] = __shfl_sync(ALL, scale, g);
        v[g][0] = v[g][1] = 0.f;
        const int key = key0 + 16 * g + gid;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const float c0 = KIND == PAGES_E4M3 ? c1[n][0] * kf : c1[n][0], c2 = KIND == PAGES_E4M3 ? c1[n][1] * kf : c1[n][1];
          float pr[4] = {ex2_approx(fmaf(s[n][0], c0, -ls[n][0])), ex2_approx(fmaf(s[n][1], c2, -ls[n][1])),
                         ex2_approx(fmaf(s[n][2], c0, -ls[n][0])), ex2_approx(fmaf(s[n][3], c2, -ls[n][1]))};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pr[e] = key + 8 * (e >> 1) > lim[n][e & 1] ? 0.f : pr[e];
          v[g][0] += pr[0] + pr[1];
          v[g][1] += pr[2] + pr[3];
        }
      }
      wg_sum_lanes<KG>(v, tig);
#pragma unroll
      for (int x = 0; x < OWN; ++x)
        if (writes[x]) wrow[mine[x]] = old[x] + v[x][0];
      live = next_live;
      --todo;
    }
    if (todo > 0) {
      --at.i;  // the last tile of (b, hk) is done
      paged_next<C::TILE>(at, p.seqlens, p.B, p.Hkv, p.max_len);
    }
  }
}

// ---- more rows: tensor-memory products, a tile of 128 keys on the lanes
constexpr int WM_THREADS = 128;
constexpr int WM_TILE = 128;

template <int D, int KIND>
struct WmCfg {
  static constexpr int RB = paged_row_bytes(KIND, D);
  static constexpr int PPR = RB / 16;               // 16-byte pieces of a row, and of the tile that one thread takes
  static constexpr int CP = D / PPR / 8;            // 8-element chunks of a piece: 1, 2 or 4
  static constexpr int BOX = WM_TILE * 128;         // 64 elements of every key, rows of 128 swizzled bytes
  static constexpr int K_BYTES = BOX * (D / 64);
  static constexpr int LPR = 8 / CP;                // lanes side by side on a row: a box's pieces
  static constexpr int RW = 32 / LPR;               // rows of one load of a warp: 4, 8 or 16
  static constexpr int SETS = WM_TILE / (4 * RW);   // of them, a warp's
  static constexpr int CTAS = KIND == PAGES_BF16 && D == 128 ? 3 : 4;  // by registers
};
__host__ __device__ constexpr int wm_cols(int rows) { return (rows + 31) / 32 * 32; }       // query rows, padded
__host__ __device__ constexpr int wm_tmem(int cols) { return 2 * cols <= 64 ? 64 : 2 * cols <= 128 ? 128 : 256; }

// Byte of element e of row r in an operand of `rows` rows.
__device__ __forceinline__ uint32_t wm_at(int rows, int r, int e) {
  return (e >> 6) * (rows * 128) + (r >> 3) * 1024 + (r & 7) * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + (e & 7) * 2;
}

template <int D, int KIND>
__global__ void __launch_bounds__(WM_THREADS, WmCfg<D, KIND>::CTAS) fa_weigh_paged_many_kernel(const WeighPagedParams p) {
  using C = WmCfg<D, KIND>;
  constexpr bool F16 = KIND != PAGES_BF16;
  extern __shared__ uint8_t wm_raw[];
  uint8_t* smem = wm_raw + ((1024u - (smem_u32(wm_raw) & 1023u)) & 1023u);
  const int N = wm_cols(p.R);
  uint8_t* s_k = smem;
  uint8_t* s_q = smem + C::K_BYTES;
  float4* s_row = reinterpret_cast<float4*>(s_q + N * D * 2);  // of rows 2i, 2i + 1: factors, and the log-sum-exp's negatives
  int2* s_lim = reinterpret_cast<int2*>(s_row + N / 2);        // and the last key they see
  uint64_t* done = reinterpret_cast<uint64_t*>(s_lim + N / 2); // a tile's products are in tensor memory
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(done + 1) + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int range = static_cast<int>(blockIdx.x);
  bool clipped = false;
  const long long sum = paged_count_tiles<WM_TILE>(p.seqlens, p.B, p.max_len, lane, clipped);
  if (range == 0 && __any_sync(ALL, clipped) && tid == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const PagedRanges ranges(sum * p.Hkv, p.n_ranges);
  if (range >= ranges.n) return;
  const long long t0 = ranges.begin(range);
  int todo = static_cast<int>(ranges.begin(range + 1) - t0);
  PagedTile at = paged_seek<WM_TILE>(p.seqlens, p.B, p.Hkv, p.max_len, t0, lane);

  const uint32_t tmem_columns = wm_tmem(N);
  if (tid == 0) {
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(slot, tmem_columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t my_lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  constexpr uint32_t DHI = sdesc_sw128_hi(1024);
  const uint32_t k_lo = sdesc_sw128_lo(smem_u32(s_k), 16), q_lo = sdesc_sw128_lo(smem_u32(s_q), 16);
  const uint32_t idesc = idesc_bf16_f32(WM_TILE, N, false) & (F16 ? ~((1u << 7) | (1u << 10)) : ~0u);
  // This thread's place in a load: row (of the warp's RW) and piece of a box. Eight lanes read 128 bytes of one to four
  // neighbouring rows, and their chunks of one e lie in different banks: the rows' chunk numbers differ by the swizzle.
  const int lr = lane / C::LPR, lc = lane % C::LPR, to = C::RW * warp + lr;
  auto chunk_at = [&](int s, int y, int e) {  // element wm_at(row, 64 y + 8 (CP lc + e)), taken apart
    return s_k + s * (C::RW * 4 * 128) + y * C::BOX + (to * 128 + (((lc * C::CP + e) ^ (to & 7)) << 4));
  };
  uint32_t issued = 0u;  // tiles whose products were started; the last of them is waited for before anything is reused
  bool ok = true;

  while (todo > 0 && ok) {
    // ================================================================ one segment: tiles of (b, hk)
    const int b = at.b, hk = at.hk, L = at.L, i0 = at.i, n = todo < at.nt - at.i ? todo : at.nt - at.i;
    auto page_of = [&](int t) -> int {  // of 16-key group `lane` of the segment's tile t
      const int key = (i0 + t) * WM_TILE + 16 * lane;
      return (lane < 8 && t < n && key < L) ? __ldg(p.table + b * p.table_stride + (key >> p.page_shift)) : -1;
    };
    uint4 raw[C::PPR];
    uint32_t f[KIND == PAGES_FP4 ? C::PPR : 1];  // 4-bit rows: a piece's two scale bytes
    // of the tile loaded last, the one before, and the one before that: groups in pages of the pool; e4m3: lane g holds the
    // scale of group g (asked for with the rows, and handed out a tile later), then of this thread's key
    unsigned live = 0u, live1 = 0u, live2 = 0u;
    float scale = 1.f, ka1 = 1.f, ka2 = 1.f;
    auto load = [&](int t, int id) {
      const int key = (i0 + t) * WM_TILE + 16 * lane;
      const bool want = lane < 8 && t < n && key < L;
      const long long off = want ? paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, key & (p.page - 1), 1) : -1;
      if (__any_sync(ALL, want && off < 0) && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      live = __ballot_sync(ALL, off >= 0);
      if constexpr (KIND == PAGES_E4M3)
        scale = off >= 0 ? __ldg(static_cast<const float*>(p.k_scale) + static_cast<long long>(id) * p.Hkv + hk) : 0.f;
      // (rows that are not there: the last one of the group, or the pool's first, whose sums are not written)
      const int rows = L - (i0 + t) * WM_TILE;
#pragma unroll
      for (int s = 0; s < C::SETS; ++s) {
        const int r0 = C::RW * (4 * s + warp), r = r0 + lr, g = r0 / 16;
        const long long base = __shfl_sync(ALL, off, g);
        const long long row = base < 0 ? 0 : base + max(min(r, rows - 1) - 16 * g, 0);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k) + row * C::RB);
#pragma unroll
        for (int y = 0; y < C::PPR / C::LPR; ++y) {
          const int x = s * (C::PPR / C::LPR) + y;
          raw[x] = __ldg(src + lc + C::LPR * y);
          if constexpr (KIND == PAGES_FP4)
            f[x] = __ldg(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.k_scale) + row * (D / 16)) + lc + C::LPR * y);
        }
      }
    };
    load(0, page_of(0));
    int id = page_of(1);
    __syncthreads();  // the segment before is done with the queries' memory

    // ---- the queries: a warp a row, a lane four of its elements, eight rows at a time
    constexpr int QB = 8;
    bool dead = false;  // a row adds nothing
    for (int r0 = warp; r0 < N; r0 += 4 * QB) {  // (N is a multiple of 32)
      uint2 x[QB];
      float lse[QB];
      int tok[QB];
#pragma unroll
      for (int i = 0; i < QB; ++i) {
        const int r = r0 + 4 * i;
        const bool in = r < p.R;
        const int h = hk * p.G + (in ? r / p.Nq : 0);
        tok[i] = in ? r % p.Nq : 0;
        x[i] = in && lane < D / 4
                   ? __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + b * p.qsb + h * p.qsh + tok[i] * p.qst) + lane)
                   : make_uint2(0u, 0u);
        lse[i] = in ? __ldg(p.lse + (static_cast<long long>(b) * p.H + h) * p.Nq + tok[i]) : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < QB; ++i) {
        const int r = r0 + 4 * i;
        float up = 1.f;
        if constexpr (F16) {
          float amax = wg_amax(x[i]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, o));
          x[i] = wg_to_f16(x[i], wg_powers(amax, up));
        }
        if (lane < D / 4) *reinterpret_cast<uint2*>(s_q + wm_at(N, r, 4 * lane)) = x[i];
        if (lane == 0) {
          const bool none = lse[i] == -INFINITY;
          float* at2 = reinterpret_cast<float*>(s_row + r / 2) + (r & 1);
          at2[0] = p.scale_log2 * up;
          at2[2] = none ? 0.f : lse[i] * -1.4426950408889634f;
          const int lim = none ? -1 : min(L - 1, L - p.Nq + tok[i]);
          reinterpret_cast<int*>(s_lim + r / 2)[r & 1] = lim;
          dead = dead || (lim < 0 && r < p.R);
        }
      }
    }

    dead = __syncthreads_or(dead);

    float* wrow = p.weights + (static_cast<long long>(b) * p.Hkv + hk) * p.wstride;
    for (int t = 0; t <= n; ++t) {
      // tile t - 1: this thread's key and what its weight was
      const int tile = (i0 + t - 1) * WM_TILE, key = tile + tid;
      live2 = live1, live1 = live, ka2 = ka1;
      if constexpr (KIND == PAGES_E4M3) ka1 = __shfl_sync(ALL, scale, tid >> 4);
      const bool writes = t > 0 && key < L && ((live2 >> (tid >> 4)) & 1u);
      const float old = writes ? wrow[key] : 0.f;
      if (t > 0) {
        ok = mbar_wait(done, (issued - 1u) & 1u, p.wait_limit_ns, p.status, abort_flag);
        tc_fence_after();
      }
      if (t < n) {  // tile t becomes the products' operand (quarter warps write eight rows: every bank once)
#pragma unroll
        for (int s = 0; s < C::SETS; ++s) {
#pragma unroll
          for (int y = 0; y < C::PPR / C::LPR; ++y) {
            const int x = s * (C::PPR / C::LPR) + y;
            const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
            if constexpr (KIND == PAGES_FP4) {
              const uint32_t f0 = fp4_scale2<0>(f[x]), f1 = fp4_scale2<1>(f[x]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t h[4];
                e2m1x8_to_f16x2x4(w[e], h);
                const uint32_t fe = e < 2 ? f0 : f1;
                *reinterpret_cast<uint4*>(chunk_at(s, y, e)) =
                    make_uint4(hmul2_bits(h[0], fe), hmul2_bits(h[1], fe), hmul2_bits(h[2], fe), hmul2_bits(h[3], fe));
              }
            } else if constexpr (KIND == PAGES_E4M3) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint4 h;
                e4m3x4_to_f16x2x2(w[2 * e], h.x, h.y);
                e4m3x4_to_f16x2x2(w[2 * e + 1], h.z, h.w);
                *reinterpret_cast<uint4*>(chunk_at(s, y, e)) = h;
              }
            } else {
              *reinterpret_cast<uint4*>(chunk_at(s, y, 0)) = raw[x];
            }
          }
        }
        fence_proxy_async_smem();  // the tensor core reads the operands through the async proxy
      }
      tc_fence_before();
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (t < n) {
        if (warp == 0) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = static_cast<uint32_t>((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4;
            const uint32_t qo = static_cast<uint32_t>((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4;
            if (elect_one()) mma_ss_w(tmem + (t & 1) * N, k_lo + ko, DHI, q_lo + qo, DHI, idesc, kk > 0 ? 1u : 0u);
          }
          if (elect_one()) mma_commit(done);
          __syncwarp();
        }
        ++issued;
      }
      if (t + 1 < n) {
        load(t + 1, id);
        id = page_of(t + 2);
      }
      if (t == 0) continue;
      // ---- tile t - 1: this lane's key against every row, two at a time
      const bool plain = tile + WM_TILE <= L - p.Nq && !dead;  // every row sees every key
      const uint64_t ka_2 = f2pack(ka2, ka2);
      uint64_t acc = 0ull;
      for (int c0 = 0; c0 < p.R; c0 += 32) {
        uint32_t sv[32];
        tmem_ld32(my_lanes + ((t - 1) & 1) * N + c0, sv);
        tmem_ld_wait32(sv);
        auto pairs = [&](auto masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = c0 + 2 * i;
            const float4 cl = s_row[c / 2];
            uint64_t y = f2pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
            if constexpr (KIND == PAGES_E4M3) y = fmul2(y, ka_2);
            float y0, y1;
            f2unpack(ffma2(y, f2pack(cl.x, cl.y), f2pack(cl.z, cl.w)), y0, y1);
            y0 = ex2_approx(y0), y1 = ex2_approx(y1);
            if constexpr (decltype(masked)::value) {
              const int2 lim = s_lim[c / 2];
              y0 = key <= lim.x ? y0 : 0.f;
              y1 = key <= lim.y ? y1 : 0.f;
            }
            acc = fadd2(acc, f2pack(y0, y1));
          }
        };
        if (plain && c0 + 32 <= p.R) pairs(std::false_type{});
        else pairs(std::true_type{});  // (padding rows see no key)
      }
      float a0, a1;
      f2unpack(acc, a0, a1);
      if (writes) wrow[key] = old + (a0 + a1);
    }
    todo -= n;
    if (todo > 0) {
      at.i = at.nt - 1;
      paged_next<WM_TILE>(at, p.seqlens, p.B, p.Hkv, p.max_len);
    }
  }
  // (a wait that gave up: the products in flight end before their memory is given back)
  if (!ok && issued > 0u) {
    const uint64_t t1 = globaltimer_ns();
    for (uint32_t i = 0; !mbar_try_wait(smem_u32(done), (issued - 1u) & 1u); ++i)
      if ((i & 31u) == 31u && globaltimer_ns() - t1 > p.wait_limit_ns) break;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_columns);
  }
}

template <int D, int KIND>
static int wm_smem(int cols) {
  // operands, row arrays, barrier and flags, alignment; and no more blocks on an SM than its tensor memory holds
  const int need = WmCfg<D, KIND>::K_BYTES + cols * D * 2 + cols * 12 + 32 + 1024;
  const int ctas = 512 / wm_tmem(cols);
  const int most = ctas >= WmCfg<D, KIND>::CTAS ? 0 : 228 * 1024 / (ctas + 1);
  return need > most ? need : most;
}
template <int KIND>
static cudaError_t wg_attrs() {
  const cudaError_t a = cudaFuncSetAttribute(fa_weigh_paged_many_kernel<64, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             wm_smem<64, KIND>(128));
  const cudaError_t b = cudaFuncSetAttribute(fa_weigh_paged_many_kernel<128, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             wm_smem<128, KIND>(128));
  return a != cudaSuccess ? a : b;
}
cudaError_t weigh_paged_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {wg_attrs<PAGES_BF16>(), wg_attrs<PAGES_E4M3>(), wg_attrs<PAGES_FP4>()})
    if (x != cudaSuccess) e = x;
  return e;
}

template <int D, int KIND, int NR>
static cudaError_t wg_launch_few(WeighPagedParams p, int num_sms, cudaStream_t stream) {
  p.n_ranges = num_sms * (NR == 1 ? WG_FEW_CTAS : 3) * WG_WARPS;
  fa_weigh_paged_few_kernel<D, KIND, NR><<<p.n_ranges / WG_WARPS, WG_THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}
template <int D, int KIND>
static cudaError_t wg_launch(WeighPagedParams p, int num_sms, cudaStream_t stream) {
  if (p.R <= 8) return wg_launch_few<D, KIND, 1>(p, num_sms, stream);
  if (p.R <= 16) return wg_launch_few<D, KIND, 2>(p, num_sms, stream);
  const int cols = wm_cols(p.R), ctas = 512 / wm_tmem(cols);
  p.n_ranges = num_sms * (ctas < WmCfg<D, KIND>::CTAS ? ctas : WmCfg<D, KIND>::CTAS);
  fa_weigh_paged_many_kernel<D, KIND><<<p.n_ranges, WM_THREADS, wm_smem<D, KIND>(cols), stream>>>(p);
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
