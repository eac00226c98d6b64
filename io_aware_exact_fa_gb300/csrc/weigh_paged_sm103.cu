// Accumulated attention weights over a paged K cache for sm_103a: for every key j
// of sequence b and K/V head hk
//     weights[b, hk, j] += sum over rows r that see j of exp(scale <q_r, k_j> - lse_r),
// where the rows are the (head, token) pairs of the head's group and lse_r what a
// forward pass over the same keys returned. Rows with lse = -inf add nothing.
//
// With the log-sum-exp given there is no running maximum and nothing to merge: every
// key's sum is its own. The keys are the M side of S^T = K Q^T; a lane then holds whole
// sums, so no atomics, and results do not depend on any order. The batch's keys are
// shared out in equal contiguous ranges, as in the paged decode.
//
// Up to 16 query rows a K/V head (a decode step): HBM bounds it (a key's row read once,
// its weight read and written). A warp has a range of its own, the queries' fragments
// stay in registers, the keys go from global memory to fragments of warp-level products,
// and the loads of the next tile, and the page entries of the one after, are on their way
// while a warp works on the current one. 64 sequences of 4-8k keys, 4-bit, 8 rows: 52 us,
// 0.68 of the bytes' time; tiles of 32 keys 60 us, 3 blocks an SM for 4 56 us.
//
// Up to 128 rows (a window of tokens): the exponentials and what carries the operands
// (2 d operations and one exponential for each row and key) bound it. A block has a range:
// one warp copies rows to shared memory in bulk and issues tcgen05 products, four warps
// turn codes into f16 operands and scores into weights. The keys' operand stands in tensor
// memory: 16 tokens of 32/8 heads over 16 sequences of 1-16k keys, e4m3, take 39 us (0.53
// of the bytes' time; a new (sequence, head)'s queries 6,500 cycles, then 3,100 a tile).
// The operand in shared memory, at once the products' and the conversions' traffic, 59 us
// with bulk copies and 67 with each warp's own loads; products at warp level 80; loads
// that touched 32 rows at once 81. The ranges count a head's start as tiles: 41 without.
//
// The rule's 16 rows: over 16 sequences of 1-16k keys, 8 heads, 4-bit / e4m3 / bf16, d = 128,
// 16 rows a head take 25 / 38 / 74 us from registers and 29 / 40 / 71 in tensor memory;
// 8 rows 25 / 31 / 50 against 35 / 37 / 53. (From registers more rows do not fit.) bf16 of d = 128 with 9 to 16 rows
// is 2 to 5 % faster in tensor memory where keys are many (143 against 138 us for 64 sequences of 4-8k), but a third slower
// where they are few (6.4 against 8.4 us for one of 700 keys, 22.6 against 28.9 for 200 of up to 300), and the host does not
// see the lengths: it stays with the registers. bf16 of d = 128 in tensor memory, 64 rows 57 us, 128 rows 86: a row's 256 bytes
// leave one stage at four blocks an SM, and 64 bytes of registers are spilled.
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
//   warps 0-3  put a tile into tensor memory as the products' operand (f16 where it is codes) and turn the scores of the one
//              before into weights: a lane has one key and sums over the rows
//   warp 4     copies the tiles' rows to shared memory and issues the products
constexpr int WM_ROLE = 128;  // threads of the first four warps
constexpr int WM_THREADS = WM_ROLE + 32;
constexpr int WM_TILE = 128;

template <int D, int KIND>
struct WmCfg {
  static constexpr int RB = paged_row_bytes(KIND, D);
  static constexpr int ROWS = WM_TILE * RB;         // bytes of a tile's rows
  static constexpr int SCALES = KIND == PAGES_FP4 ? WM_TILE * (D / 16) : 0;
  static constexpr int STAGES = ROWS > 16384 ? 1 : 2;  // tiles in shared memory
  static constexpr int CTAS = 4;                    // by registers, shared and tensor memory
  // Tiles' time that a new (sequence, head)'s queries take, by which its range is shorter. 16 sequences of 1-16k, e4m3, 64 / 128
  // rows: d = 128 with 2 45 / 63 us, with 0 50 / 73; d = 64 (half the queries) with 2 35 / 55, with 1 37 / 55, with 0 35 / 57, but
  // bf16 38 / 66, 38 / 66 and 36 / 62.
  static constexpr int START = D == 128 ? 2 : 0;
};
__host__ __device__ constexpr int wm_cols(int rows) { return (rows + 31) / 32 * 32; }       // query rows, padded
__host__ __device__ constexpr int wm_tmem(int d, int cols) {                                 // scores and operand
  return d / 2 + cols <= 64 ? 64 : d / 2 + cols <= 128 ? 128 : 256;
}

// Byte of element e of row r in an operand of `rows` rows.
__device__ __forceinline__ uint32_t wm_at(int rows, int r, int e) {
  return (e >> 6) * (rows * 128) + (r >> 3) * 1024 + (r & 7) * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + (e & 7) * 2;
}
// Where elements 4 u .. 4 u + 3 of a row stand in the products: wg_elem's inverse, 16 j + 4 tig.
template <int D, int KIND>
__device__ __forceinline__ int wm_place(int u) {
  if constexpr (KIND == PAGES_FP4) return 16 * (u % (D / 16)) + 4 * (u / (D / 16));
  constexpr int Q = KIND == PAGES_E4M3 ? 4 : 2;
  return 16 * (u / (4 * Q) * Q + u % Q) + 4 * (u / Q % 4);
}
// Rows gid and gid + 8 of a 16-key group in shared memory: the lane's share of each. (Of rows of 128 bytes and more the odd ones
// are read in another order, so that the eight lanes of two neighbours meet every bank once.)
template <int D, int KIND>
__device__ __forceinline__ void wm_read(WgRaw<D, KIND>& x, const uint8_t* rows, const uint8_t* scales, int gid, int tig) {
  using C = WgCfg<D, KIND>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* src = rows + (gid + 8 * h) * C::RB;
    if constexpr (KIND == PAGES_FP4) {
      const uint8_t* sp = scales + (gid + 8 * h) * (D / 16);
      if constexpr (D == 128) {
        const uint4 y = reinterpret_cast<const uint4*>(src)[tig];
        x.w[h][0] = y.x, x.w[h][1] = y.y, x.w[h][2] = y.z, x.w[h][3] = y.w;
        x.f[h] = reinterpret_cast<const uint16_t*>(sp)[tig];
      } else {
        const uint2 y = reinterpret_cast<const uint2*>(src)[tig];
        x.w[h][0] = y.x, x.w[h][1] = y.y;
        x.f[h] = sp[tig];
      }
    } else if constexpr (C::RB < 128) {
      const uint4 y = reinterpret_cast<const uint4*>(src)[tig];
      x.w[h][0] = y.x, x.w[h][1] = y.y, x.w[h][2] = y.z, x.w[h][3] = y.w;
    } else {
      const int flip = gid & 1;
#pragma unroll
      for (int i = 0; i < C::LW / 4; i += 2) {
        const uint4 y = reinterpret_cast<const uint4*>(src)[tig + 4 * (i + flip)], z = reinterpret_cast<const uint4*>(src)[tig + 4 * (i + 1 - flip)];
        const uint4 a = flip ? z : y, b = flip ? y : z;
        x.w[h][4 * i] = a.x, x.w[h][4 * i + 1] = a.y, x.w[h][4 * i + 2] = a.z, x.w[h][4 * i + 3] = a.w;
        x.w[h][4 * i + 4] = b.x, x.w[h][4 * i + 5] = b.y, x.w[h][4 * i + 6] = b.z, x.w[h][4 * i + 7] = b.w;
      }
    }
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(WM_THREADS, WmCfg<D, KIND>::CTAS) fa_weigh_paged_many_kernel(const WeighPagedParams p) {
  using C = WmCfg<D, KIND>;
  constexpr bool F16 = KIND != PAGES_BF16;
  extern __shared__ uint8_t wm_raw[];
  uint8_t* smem = wm_raw + ((1024u - (smem_u32(wm_raw) & 1023u)) & 1023u);
  const int N = wm_cols(p.R);
  uint8_t* s_q = smem;
  uint8_t* s_rows = s_q + N * D * 2;                           // [stage] a tile's rows as they are in the pool
  uint8_t* s_scale = s_rows + C::STAGES * C::ROWS;             // [stage] 4-bit rows: their scales
  float4* s_row = reinterpret_cast<float4*>(s_scale + C::STAGES * C::SCALES);  // of rows 2i, 2i + 1: factors, and the log-sum-exp's negatives
  int2* s_lim = reinterpret_cast<int2*>(s_row + N / 2);        // and the last key they see
  float* s_ka = reinterpret_cast<float*>(s_lim + N / 2);       // [4][8]: e4m3 scales of a tile's 16-key groups
  unsigned* s_live = reinterpret_cast<unsigned*>(s_ka + 32);   // [4]: which of them are in pages of the pool
  uint64_t* full = reinterpret_cast<uint64_t*>(s_live + 4);    // [stage] a tile's rows are there
  uint64_t* empty = full + C::STAGES;                          // [stage] and taken
  uint64_t* ready = empty + C::STAGES;                         // its operand is written, and the scores before it read
  uint64_t* done = ready + 1;                                  // its products are in tensor memory
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int range = static_cast<int>(blockIdx.x);
  bool clipped = false;
  const long long sum = paged_count_tiles<WM_TILE, C::START>(p.seqlens, p.B, p.max_len, lane, clipped);
  if (range == 0 && __any_sync(ALL, clipped) && tid == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const PagedRanges ranges(sum * p.Hkv, p.n_ranges);
  if (range >= ranges.n) return;
  const long long t0 = ranges.begin(range);
  int todo = static_cast<int>(ranges.begin(range + 1) - t0);
  PagedTile at = paged_seek<WM_TILE, C::START>(p.seqlens, p.B, p.Hkv, p.max_len, t0, lane);

  const uint32_t tmem_columns = wm_tmem(D, N);
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, WM_ROLE);
    }
    mbar_init(ready, WM_ROLE);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(slot, tmem_columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot, operand = tmem + N;
  uint32_t c0 = 0u;                    // tiles before the segment: the barriers' phases run on
  uint32_t copied = 0u, issued = 0u;   // (warp 4) tiles whose copies, and whose products, were started
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t turn) {  // one answer for the warp
    ok = ok && __all_sync(ALL, mbar_wait(bar, turn & 1u, p.wait_limit_ns, p.status, abort_flag));
    return ok;
  };

  while (todo > 0) {
    // ================================================================ one segment: tiles of (b, hk)
    const int counted = todo < at.nt - at.i ? todo : at.nt - at.i;  // (the first C::START of a head's are none)
    const int b = at.b, hk = at.hk, L = at.L, i0 = max(at.i - C::START, 0), n = at.i + counted - C::START - i0;
    if (n <= 0) {
      // (the range ends, or the head's tiles begin in the next one)
    } else if (warp == 4) {
      // ------------------------------------------------------------ copies and products: lane g has 16-key group g of a tile
      auto page_of = [&](int t) -> int {
        const int key = (i0 + t) * WM_TILE + 16 * lane;
        return (lane < 8 && t < n && key < L) ? __ldg(p.table + b * p.table_stride + (key >> p.page_shift)) : -1;
      };
      auto scale_of = [&](int id) {
        return KIND == PAGES_E4M3 && static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages)
                   ? __ldg(static_cast<const float*>(p.k_scale) + static_cast<long long>(id) * p.Hkv + hk)
                   : 0.f;
      };
      int id = page_of(0), id1 = page_of(1);
      float scale = scale_of(id);
      auto copy = [&](int t) {
        const uint32_t c = c0 + t;
        const uint32_t stage = c % C::STAGES;
        if (c >= C::STAGES && !wait(empty + stage, c / C::STAGES - 1u)) return;
        const int key = (i0 + t) * WM_TILE + 16 * lane;
        const bool want = lane < 8 && key < L;
        const long long off = want ? paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, key & (p.page - 1), 1) : -1;
        const unsigned live = __ballot_sync(ALL, off >= 0);
        if (__any_sync(ALL, want && off < 0) && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
        if (KIND == PAGES_E4M3 && lane < 8) s_ka[(c & 3u) * 8 + lane] = scale;
        __syncwarp();
        if (lane == 0) {
          s_live[c & 3u] = live;
          mbar_arrive_expect_tx(full + stage, __popc(live) * (16 * C::RB + C::SCALES / 8));
        }
        __syncwarp();
        // A page's groups side by side are one copy, by the lane of its first. (Whole groups: rows past the sequence's last are
        // the page's own, and their sums are not written.)
        const int first = key & (p.page - 1);
        if (off >= 0 && first == 0) {
          const int rows = 16 * __popc(live & ((p.page >= WM_TILE ? 0xffu : (1u << (p.page / 16)) - 1u) << lane));
          bulk_load_1d(s_rows + stage * C::ROWS + lane * 16 * C::RB, static_cast<const uint8_t*>(p.k) + off * C::RB, rows * C::RB, full + stage);
          if constexpr (KIND == PAGES_FP4)
            bulk_load_1d(s_scale + stage * C::SCALES + lane * D, static_cast<const uint8_t*>(p.k_scale) + off * (D / 16), rows * (D / 16), full + stage);
        }
        copied = c + 1u;
        id = id1;
        scale = scale_of(id);
        id1 = page_of(t + 2);
      };
      copy(0);
      __syncthreads_or(0);  // the queries are there
      if (C::STAGES > 1 && n > 1) copy(1);
      constexpr uint32_t DHI = sdesc_sw128_hi(1024);
      const uint32_t q_lo = sdesc_sw128_lo(smem_u32(s_q), 16);
      const uint32_t idesc = idesc_bf16_f32(WM_TILE, N, false) & (F16 ? ~((1u << 7) | (1u << 10)) : ~0u);
      for (int t = 0; t < n && ok; ++t) {
        if (!wait(ready, c0 + t)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qo = static_cast<uint32_t>((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4;
            mma_ts_w(tmem, operand + 8 * kk, q_lo + qo, DHI, idesc, kk > 0 ? 1u : 0u);
          }
          mma_commit(done);
        }
        __syncwarp();
        issued = c0 + t + 1u;
        if (t + C::STAGES < n) copy(t + C::STAGES);
      }
    } else {
      // ------------------------------------------------------------ the queries: a warp N / 4 rows, a lane eight elements of one
      constexpr int QL = D / 8, QR = 32 / QL, QB = 8;  // lanes of a row, rows of a warp's load, loads at a time
      const int rows = N / 4, r_of = warp * rows + lane;  // lane m finds row m's place
      const bool in = lane < rows && r_of < p.R;
      const int h = hk * p.G + (in ? r_of / p.Nq : 0), tok = in ? r_of % p.Nq : 0;
      const long long off = b * p.qsb + h * p.qsh + tok * p.qst;
      const float lse = in ? __ldg(p.lse + (static_cast<long long>(b) * p.H + h) * p.Nq + tok) : -INFINITY;
      const unsigned real = __ballot_sync(ALL, in);
      for (int m0 = 0; m0 < rows; m0 += QR * QB) {
        uint4 x[QB];
#pragma unroll
        for (int i = 0; i < QB; ++i) {
          const int m = (m0 + QR * i + lane / QL) & 31;
          const long long at_row = __shfl_sync(ALL, off, m);
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if ((real >> m) & 1u) x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at_row) + lane % QL);
        }
#pragma unroll
        for (int i = 0; i < QB; ++i) {
          const int m = m0 + QR * i + lane / QL, r = warp * rows + m;
          float up = 1.f;
          if constexpr (F16) {
            uint2 lo = make_uint2(x[i].x, x[i].y), hi = make_uint2(x[i].z, x[i].w);
            float amax = fmaxf(wg_amax(lo), wg_amax(hi));
#pragma unroll
            for (int o = QL / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, o));
            const float down = wg_powers(amax, up);
            lo = wg_to_f16(lo, down), hi = wg_to_f16(hi, down);
            x[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
          if (m < rows) {
            *reinterpret_cast<uint2*>(s_q + wm_at(N, r, wm_place<D, KIND>(2 * (lane % QL)))) = make_uint2(x[i].x, x[i].y);
            *reinterpret_cast<uint2*>(s_q + wm_at(N, r, wm_place<D, KIND>(2 * (lane % QL) + 1))) = make_uint2(x[i].z, x[i].w);
            if (lane % QL == 0) reinterpret_cast<float*>(s_row + r / 2)[r & 1] = p.scale_log2 * up;
          }
        }
      }
      bool dead = false;  // a row adds nothing
      if (lane < rows) {
        const bool none = lse == -INFINITY;
        const int lim = none ? -1 : min(L - 1, L - p.Nq + tok);
        reinterpret_cast<float*>(s_row + r_of / 2)[2 + (r_of & 1)] = none ? 0.f : lse * -1.4426950408889634f;
        reinterpret_cast<int*>(s_lim + r_of / 2)[r_of & 1] = lim;
        dead = lim < 0 && in;
      }
      fence_proxy_async_smem();  // the tensor core reads the queries through the async proxy
      dead = __syncthreads_or(dead);

      // ------------------------------------------------------------ tiles
      const uint32_t my_lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      float* wrow = p.weights + (static_cast<long long>(b) * p.Hkv + hk) * p.wstride;
      bool writes_next = false;
      float old_next = 0.f, ka_next = 1.f;
      for (int t = 0; t <= n; ++t) {
        if (t > 0) {
          if (!wait(done, c0 + t - 1u)) break;
          tc_fence_after();
        }
        const bool writes = writes_next;
        const float old = old_next, ka = ka_next;
        if (t < n) {  // tile t becomes the products' operand
          const uint32_t c = c0 + t, stage = c % C::STAGES;
          if (!wait(full + stage, c / C::STAGES)) break;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            WgRaw<D, KIND> x;
            wm_read<D, KIND>(x, s_rows + stage * C::ROWS + (2 * warp + g) * 16 * C::RB, s_scale + stage * C::SCALES + (2 * warp + g) * D,
                             lane >> 2, lane & 3);
            uint32_t a[D / 4];
            wg_fragments<D, KIND>(x, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
              a[4 * j] = a0, a[4 * j + 1] = a2, a[4 * j + 2] = a1, a[4 * j + 3] = a3;
            });
            tmem_st_rows<D / 16>(operand + (static_cast<uint32_t>(32 * warp + 16 * g) << 16), a);
          }
          mbar_arrive(empty + stage);
          tmem_st_wait();
          // this thread's key, for the next turn: whether it is there, what its weight was, its scale
          const uint32_t at4 = c & 3u;
          const int next = (i0 + t) * WM_TILE + tid;
          writes_next = next < L && ((s_live[at4] >> (tid >> 4)) & 1u);
          old_next = writes_next ? wrow[next] : 0.f;
          if constexpr (KIND == PAGES_E4M3) ka_next = s_ka[at4 * 8 + (tid >> 4)];
          if (t == 0) {
            tc_fence_before();
            mbar_arrive(ready);
            continue;
          }
        }
        const int tile = (i0 + t - 1) * WM_TILE, key = tile + tid;
        // ---- tile t - 1: this lane's key against every row, two at a time
        const bool plain = tile + WM_TILE <= L - p.Nq && !dead;  // every row sees every key
        const uint64_t ka_2 = f2pack(ka, ka);
        uint64_t acc = 0ull;
        for (int col = 0; col < p.R; col += 32) {
          uint32_t sv[32];
          tmem_ld32(my_lanes + col, sv);
          tmem_ld_wait32(sv);
          if (t < n && col + 32 >= p.R) {  // the last of them: the next products may begin
            tc_fence_before();
            mbar_arrive(ready);
          }
          auto pairs = [&](auto masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 cl = s_row[col / 2 + i];
              uint64_t y = f2pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
              if constexpr (KIND == PAGES_E4M3) y = fmul2(y, ka_2);
              float y0, y1;
              f2unpack(ffma2(y, f2pack(cl.x, cl.y), f2pack(cl.z, cl.w)), y0, y1);
              y0 = ex2_approx(y0), y1 = ex2_approx(y1);
              if constexpr (decltype(masked)::value) {
                const int2 lim = s_lim[col / 2 + i];
                y0 = key <= lim.x ? y0 : 0.f;
                y1 = key <= lim.y ? y1 : 0.f;
              }
              acc = fadd2(acc, f2pack(y0, y1));
            }
          };
          if (plain && col + 32 <= p.R) pairs(std::false_type{});
          else pairs(std::true_type{});  // (padding rows see no key)
        }
        float a0, a1;
        f2unpack(acc, a0, a1);
        if (writes) wrow[key] = old + (a0 + a1);
      }
      tc_fence_before();
    }
    c0 += max(n, 0);
    todo -= counted;
    ok = __syncthreads_and(ok);  // the segment is done with the queries' memory
    if (!ok) break;
    if (todo > 0) {
      at.i = at.nt - 1;
      paged_next<WM_TILE, C::START>(at, p.seqlens, p.B, p.Hkv, p.max_len);
    }
  }
  if (warp == 4) {
    // (a wait that gave up: copies and products in flight get the limit's time, or a second, before their memory is given back)
    if (!ok) {
      const uint64_t t1 = globaltimer_ns();
      auto ended = [&](uint64_t* bar, uint32_t turns) { return turns == 0u || mbar_try_wait(smem_u32(bar), (turns - 1u) & 1u); };
      for (uint32_t i = 0; !(ended(full, (copied + C::STAGES - 1) / C::STAGES) && ended(full + C::STAGES - 1, copied / C::STAGES) &&
                             ended(done, issued)); ++i)
        if ((i & 31u) == 31u && globaltimer_ns() - t1 > (p.wait_limit_ns > 1000000000ull ? p.wait_limit_ns : 1000000000ull)) break;
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, tmem_columns);
  }
}

template <int D, int KIND>
static int wm_smem(int cols) {
  // queries, rows and scales, row arrays, barriers and flags, alignment; and no more blocks on an SM than its tensor memory holds
  using C = WmCfg<D, KIND>;
  const int need = cols * D * 2 + C::STAGES * (C::ROWS + C::SCALES) + cols * 12 + 128 + 16 + (2 * C::STAGES + 2) * 8 + 16 + 1024;
  const int ctas = 512 / wm_tmem(D, cols);
  const int most = ctas >= C::CTAS ? 0 : 228 * 1024 / (ctas + 1);
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
  const int cols = wm_cols(p.R), ctas = 512 / wm_tmem(D, cols);
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
