// Attention of a few new tokens over a paged K/V cache (bf16 or e4m3 pages)
// for sm_103a.
//
// For sequence b with L_b keys, query head h (K/V head hk = h / G) and token t
// of its last Nq positions:
//     y_j = scale * log2(e) * <q, k_j>              keys j < L_b, j <= L_b - Nq + t
//     O   = sum_j 2^(y_j) v_j / sum_j 2^(y_j),  lse = ln sum_j exp(scale <q, k_j>)
// An e4m3 page holds codes with one scale a for its keys and one scale c for its
// values (per K/V head): k = a K~, v = c V~. The key scale joins the softmax
// scale. The value scale joins the exponent: with z_j = y_j + log2 c and the
// running base M = max z_j,
//     W_j = 2^(z_j - M),  O = sum_j W_j V~_j / sum_j (W_j / c_j),
//     lse = ln 2 (M + log2 sum_j (W_j / c_j)),
// (M may lag behind, see DpBase) so the value products run on the codes themselves
// (append writes powers of two, for which W_j / c_j and the shift by log2 c are
// exact). W is rounded to f16 for the product, which would cost pages of small
// values their weights' bits beside a page of large ones: groups of keys whose scale
// lies far below the largest count their weights from a base of their own (`far`).
//
// What bounds it: HBM. Each key and value is read once per K/V head; at 6.8 TB/s
// an SM takes about 24 bytes a clock, 24 e4m3 codes. The work per code has to
// stay well below the SM's issue rate, which rules out CUDA-core products for
// more than a few rows; a 128-row tensor-memory tile would be nearly empty and
// cannot convert codes. So warp-level products on registers: the keys are the
// M side of S^T = K Q^T and the head dimension the M side of O^T = V^T P^T, the
// 8 (or 16) query rows the N side, and neither product pads the rows past 8.
//
// Work split: all keys of the batch, as tiles of KS keys laid end to end (sequence
// by sequence, K/V head by K/V head), are shared out in equal contiguous ranges,
// one for each warp that the GPU holds, so ragged lengths leave no SM idle and no
// warp starts anew for every chunk (blocks of one chunk each spent a third of
// their time filling and draining: 97 in place of 74 us for two sequences of 110k
// tokens, 137 in place of 125 us for 64 of 4-8k; e4m3, d = 128, 8 K/V heads:
// 6.1 and 6.4 TB/s, 0.89 and 0.95 of the copy rate). A warp walks its range
// through a private ring of asynchronous 16-byte copies that runs on across
// sequences; it meets no other warp, so there is no barrier at all. Where a
// sequence's keys of one head lie in several ranges, each warp leaves its base,
// sum and output, and the first and the last of them their number, and the merge
// kernel joins the parts. About 8 us of a call are fixed: launches, the chain
// lengths -> page -> first tile, the merge.
//
// A tile's 16-key groups may lie in different pages; one lane per group looks the
// page up, a tile ahead. The fragments are read straight from the copied rows: the
// order of the contraction over d (for S) and of the output rows (for O^T) is
// free, so each lane takes whole 16-byte pieces of its rows, and the shared-memory
// positions of the pieces are XORed with the row so that those reads touch every
// bank once.
#include <cuda_bf16.h>

#include <type_traits>

#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

constexpr int DP_WARPS = 4;
constexpr int DP_THREADS = 32 * DP_WARPS;

// Where the weights 2^(z - M) lie: the base M is set so that a row's largest z is TOP above it, and moves when one passes
// it by more than LIMIT. bf16 weights have fp32's exponents; f16 ends at 2^16, and its weights lie as high as that allows,
// to leave room below for pages whose scales are smaller, up to 2^-GAP times (see `far`).
template <bool F8>
struct DpBase {
  static constexpr float TOP = F8 ? 7.f : 0.f, LIMIT = F8 ? 15.f : 8.f, GAP = TOP;
};

template <int D, bool F8, int NR>
struct DpCfg {
  static constexpr int ROWS = 8 * NR;            // query rows of a warp
  static constexpr int ESZ = F8 ? 1 : 2;
  static constexpr int RB = D * ESZ;             // bytes of a key's row: 64, 128 or 256
  static constexpr int CR = RB / 16;             // 16-byte pieces of a row
  static constexpr int HALF = 4096;              // K (or V) bytes of a tile
  static constexpr int KS = HALF / RB;           // its keys
  static constexpr int KG = KS / 16;             // its 16-key groups
  static constexpr int EPC = 16 / ESZ;           // elements of a piece
  static constexpr int DL = D / 4;               // elements of a K row that one lane holds
  static constexpr int NPK = DL / EPC;           // as pieces
  static constexpr int KST = D / 16;             // k-steps of S^T, and M tiles of O^T
  static constexpr int META = KG * 2 * 4;        // e4m3 scales of a tile
  static constexpr int STAGE = 2 * HALF;
  // Tiles in each warp's ring: what fits beside the warps an SM holds. (Three tiles for eight warps against two for
  // twelve: 136 against 130 us at 8 rows, e4m3, d = 128. Tiles of half the size, four to a ring: 134. Sixteen warps
  // of those: 133.)
  static constexpr int DP_STAGES = decode_paged_ctas(D, ROWS) == 3 ? 2 : 3;
  static constexpr int RING = DP_WARPS * DP_STAGES * STAGE;
  static constexpr int META_OFF = RING;
  static constexpr int SMEM = RING + DP_WARPS * DP_STAGES * META;
};

// Byte offset of 16-byte piece c of row r in a tile of RB-byte rows.
template <int RB>
__device__ __forceinline__ uint32_t dp_swz(uint32_t r, uint32_t c) {
  if constexpr (RB == 64)
    return (r >> 1) * 128u + (((((r & 1u) << 2) | c) ^ (((r >> 1) & 3u) << 1)) << 4);
  else
    return r * RB + (((c & ~7u) | ((c ^ r) & 7u)) << 4);
}

// The piece of a K row that lane tig holds i-th.
template <int D, bool F8>
__device__ __forceinline__ int dp_k_piece(int tig, int i) {
  if constexpr (F8 && D == 64) return tig;
  else return 2 * tig + (i & 1) + 8 * (i >> 1);
}
// First of the four output elements 4 jj .. 4 jj + 3 (of its D / 8) that lane group gid holds: M tile j has 2j, 2j + 1.
template <int D, bool F8>
__device__ __forceinline__ int dp_o_elem(int gid, int jj) {
  if constexpr (!F8 && D == 128) return (gid + 8 * (jj >> 1)) * 8 + (jj & 1) * 4;
  else return gid * (D / 8) + 4 * jj;
}

// How the batch's tiles are shared out: tile t of the whole (sequence by
// sequence, K/V head by K/V head) belongs to range t's; range r has tiles
// begin(r) .. begin(r + 1) - 1, none of them empty.
struct DpRanges {
  long long tiles, n;  // all tiles; ranges
  __device__ __forceinline__ DpRanges(long long tiles_, int most) : tiles(tiles_), n(most < tiles_ ? most : tiles_) {}
  __device__ __forceinline__ long long begin(long long r) const { return r * tiles / n; }
};

// What a row's scores count from.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ int dp_len(const DecodePagedParams& p, int b) {
  return paged_clip_len(__ldg(p.seqlens + b), p.max_len);
}

}  // namespace

template <int D, bool F8, int NR>
__global__ void __launch_bounds__(DP_THREADS, decode_paged_ctas(D, 8 * NR)) fa_decode_paged_kernel(const DecodePagedParams p) {
  using C = DpCfg<D, F8, NR>;
  extern __shared__ __align__(128) uint8_t dp_smem[];
  const uint32_t sbase = smem_u32(dp_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  constexpr unsigned ALL = 0xffffffffu;

  pdl_launch_dependents();
  // ---- this warp's range of tiles, and where it starts. The row tiles of the same keys are neighbouring warps.
  const int worker = static_cast<int>(blockIdx.x) * DP_WARPS + warp;
  const int rt = worker % p.row_tiles;
  const int range = worker / p.row_tiles;
  long long sum = 0;
  bool clipped = false;
#pragma unroll 4
  for (int b = lane; b < p.B; b += 32) {
    const int raw = __ldg(p.seqlens + b), L = paged_clip_len(raw, p.max_len);
    clipped = clipped || L != raw;
    sum += (L + C::KS - 1) / C::KS;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
  if (worker == 0 && __any_sync(ALL, clipped) && lane == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const DpRanges ranges(sum * p.Hkv, p.n_ranges);
  if (range >= ranges.n) return;
  const long long t0 = ranges.begin(range);
  int todo = static_cast<int>(ranges.begin(range + 1) - t0);  // tiles to compute (the host keeps a range below 2^31)
  int b = 0, hk = 0, i = 0, L = 0, nt = 0;        // position: sequence, K/V head, tile; its length and tiles
  {
    long long base = 0;  // tiles of one K/V head of the sequences before
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int mine = b0 + lane < p.B ? dp_len(p, b0 + lane) : 0;
      const int n = (mine + C::KS - 1) / C::KS;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(ALL, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned past = __ballot_sync(ALL, (base + inc) * p.Hkv > t0);
      if (past != 0u) {
        const int at = __ffs(past) - 1;
        b = b0 + at;
        L = __shfl_sync(ALL, mine, at);
        nt = __shfl_sync(ALL, n, at);
        const long long rest = t0 - (base + __shfl_sync(ALL, inc, at) - nt) * p.Hkv;
        hk = static_cast<int>(rest / nt);
        i = static_cast<int>(rest % nt);
        break;
      }
      base += __shfl_sync(ALL, inc, 31);
    }
  }
  // the next tile after (b, hk, i)
  auto advance = [&](int& b_, int& hk_, int& i_, int& L_, int& nt_) {
    if (++i_ < nt_) return;
    i_ = 0;
    if (++hk_ < p.Hkv) return;
    hk_ = 0;
    do {
      if (++b_ >= p.B) return;  // past the last tile
      L_ = dp_len(p, b_);
      nt_ = (L_ + C::KS - 1) / C::KS;
    } while (nt_ == 0);
  };

  // ---- the copies, which run ahead of the computation: position of the next tile to copy, and its pages
  const uint32_t ring = sbase + warp * (C::DP_STAGES * C::STAGE);
  const uint32_t meta = sbase + C::META_OFF + warp * (C::DP_STAGES * C::META);
  const uint8_t* my_ring = dp_smem + warp * (C::DP_STAGES * C::STAGE);
  const uint8_t* my_meta = dp_smem + C::META_OFF + warp * (C::DP_STAGES * C::META);
  int cb = b, chk = hk, ci = i, cL = L, cnt = nt;
  int to_copy = todo;
  uint32_t copied = 0u;          // tiles copied so far
  uint32_t hidden = 0u;          // 4 bits for each of 8 tiles: groups whose page is not in the pool
  // page of 16-key group `lane` of the next tile; -1 past the keys or for other lanes
  auto page_of = [&]() -> int {
    const int key = ci * C::KS + 16 * lane;
    return (lane < C::KG && to_copy > 0 && key < cL) ? __ldg(p.table + cb * p.table_stride + (key >> p.page_shift)) : -1;
  };
  int id = page_of();
  constexpr int RPI = 32 / C::CR;                                        // rows of one copy instruction of the warp
  constexpr int PERIOD = C::RB == 64 ? 1 : (8 / RPI > 1 ? 8 / RPI : 1);  // after which the swizzle repeats
  const int piece = lane % C::CR, rin = lane / C::CR;
  uint32_t dst[PERIOD];
#pragma unroll
  for (int u = 0; u < PERIOD; ++u) dst[u] = dp_swz<C::RB>(u * RPI + rin, piece) - u * RPI * C::RB;
  const uint32_t src_lane = rin * C::RB + piece * 16;
  auto issue = [&]() {
    if (to_copy > 0) {
      const int key0 = ci * C::KS;
      const int gkey = key0 + 16 * lane;
      const bool want = lane < C::KG && gkey < cL;
      const long long off = want ? paged_row_offset(id, p.num_pages, p.Hkv, chk, p.page, gkey & (p.page - 1), D) : -1;
      const unsigned bad = __ballot_sync(ALL, want && off < 0);
      if (bad != 0u && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      const uint32_t sh = 4u * (copied & 7u);
      hidden = (hidden & ~(0xfu << sh)) | ((bad & 0xfu) << sh);
      const uint32_t slot = copied % C::DP_STAGES;
      const uint32_t kdst = ring + slot * C::STAGE;
      if constexpr (F8) {
        if (lane < C::KG) {
          const uint32_t m = meta + slot * C::META + lane * 8u;
          if (off >= 0) {
            const long long sc = static_cast<long long>(id) * p.Hkv + chk;
            cp_async4(m, p.k_scale + sc);
            cp_async4(m + 4u, p.v_scale + sc);
          } else {
            st_shared_f32(m, 0.f);
            st_shared_f32(m + 4u, 1.f);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < C::KG; ++g) {
        const long long goff = __shfl_sync(ALL, off, g);
        const int left = goff < 0 ? 0 : cL - (key0 + 16 * g);  // rows of the group to read
        const uint8_t* kg = static_cast<const uint8_t*>(p.k) + (goff < 0 ? 0 : goff) * C::ESZ;
        const uint8_t* vg = static_cast<const uint8_t*>(p.v) + (goff < 0 ? 0 : goff) * C::ESZ;
        if (left >= 16) {
          kg += src_lane;
          vg += src_lane;
#pragma unroll
          for (int u = 0; u < 16 / RPI; ++u) {
            const uint32_t to = kdst + dst[u % PERIOD] + (16 * g + u * RPI) * C::RB;
            cp_async16(to, kg + u * RPI * C::RB, 16u);
            cp_async16(to + C::HALF, vg + u * RPI * C::RB, 16u);
          }
        } else {  // the rows past the sequence's end become zeros
#pragma unroll
          for (int u = 0; u < 16 / RPI; ++u) {
            const int row = u * RPI + rin;
            const uint32_t to = kdst + dst[u % PERIOD] + (16 * g + u * RPI) * C::RB;
            const uint32_t n = row < left ? 16u : 0u, so = n ? row * C::RB + piece * 16 : 0;
            cp_async16(to, kg + so, n);
            cp_async16(to + C::HALF, vg + so, n);
          }
        }
      }
      ++copied;
      --to_copy;
      advance(cb, chk, ci, cL, cnt);
      id = page_of();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < C::DP_STAGES - 1; ++k) issue();

  uint32_t done = 0u;  // tiles computed
  while (todo > 0) {
    // ================================================================ one segment: keys of (b, hk) from tile i on
    const int i0 = i;
    const int i1 = todo < nt - i ? i + todo : nt;
    // ---- Q: lane (gid, tig) holds its elements of query row gid of every 8-row tile
    uint32_t qf[NR][C::KST][2];
    float c1[NR][2];   // factor of the scores of rows 2tig and 2tig + 1 (log2 units)
    int lim[NR][2];    // last key those rows see
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = rt * C::ROWS + n * 8 + gid;
      const bool in = r < p.R;
      const uint16_t* qr = static_cast<const uint16_t*>(p.q) + b * p.qsb + (hk * p.G + (in ? r / p.Nq : 0)) * p.qsh +
                           (in ? r % p.Nq : 0) * p.qst;
      uint2 raw[C::KST];
#pragma unroll
      for (int j = 0; j < C::KST; ++j) {  // elements 4j .. 4j + 3 of the lane's
        const int d0 = dp_k_piece<D, F8>(tig, 4 * j / C::EPC) * C::EPC + (4 * j) % C::EPC;
        raw[j] = in ? __ldg(reinterpret_cast<const uint2*>(qr + d0)) : make_uint2(0u, 0u);
      }
      float row_factor = 1.f;
      if constexpr (F8) {
        // The products with the codes run in f16 (every e4m3 code is an f16
        // value). The row's power of two 2^x brings its largest element to [1, 2):
        // elements down to 2^-14 of it keep all their 8 bits, smaller ones are
        // off by at most 2^-25 of 2^x: a score by d 2^-25 max|q| max|k| at most.
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < C::KST; ++j) {
          const uint32_t w[2] = {raw[j].x, raw[j].y};
#pragma unroll
          for (int e = 0; e < 2; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(ALL, amax, 2));
        const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -120), 120);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        row_factor = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int j = 0; j < C::KST; ++j) {
          qf[n][j][0] = pack_f16x2(__uint_as_float(raw[j].x << 16) * down, __uint_as_float(raw[j].x & 0xffff0000u) * down);
          qf[n][j][1] = pack_f16x2(__uint_as_float(raw[j].y << 16) * down, __uint_as_float(raw[j].y & 0xffff0000u) * down);
        }
      } else {
#pragma unroll
        for (int j = 0; j < C::KST; ++j) {
          qf[n][j][0] = raw[j].x;
          qf[n][j][1] = raw[j].y;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c1[n][e] = p.scale_log2 * (F8 ? __shfl_sync(ALL, row_factor, (2 * tig + e) * 4) : 1.f);
        const int r2 = rt * C::ROWS + n * 8 + 2 * tig + e;
        lim[n][e] = min(L - 1, r2 < p.R ? L - p.Nq + r2 % p.Nq : L - 1);
      }
    }
    const int full_lim = min(L - 1, L - p.Nq);  // every row sees the keys up to here

    float M[NR][2], l[NR][2];
    [[maybe_unused]] float ev_most = -INFINITY;  // largest log2 c of the segment's pages so far
    float oacc[NR][C::KST][4];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      M[n][0] = M[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < C::KST; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[n][j][e] = 0.f;
    }

    for (; i < i1; ++i, ++done) {
      cp_async_wait<C::DP_STAGES - 2>();
      __syncwarp();  // the tile landed for every lane, and every lane is done with the one before's slot
      issue();
      const uint32_t slot = done % C::DP_STAGES;
      const uint8_t* kt = my_ring + slot * C::STAGE;
      const uint8_t* vt = kt + C::HALF;
      const int key0 = i * C::KS;
      // ---- S^T: 16 keys x 8 rows for each group and row tile
      auto scores = [&](int g, float (&s)[NR][4]) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int i2 = 0; i2 < C::NPK; ++i2) {
          const int piece = dp_k_piece<D, F8>(tig, i2);
          const uint4 ra = *reinterpret_cast<const uint4*>(kt + dp_swz<C::RB>(16 * g + gid, piece));
          const uint4 rb = *reinterpret_cast<const uint4*>(kt + dp_swz<C::RB>(16 * g + gid + 8, piece));
          const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
          if constexpr (F8) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2x2(wa[w], a0, a2);
              e4m3x4_to_f16x2x2(wb[w], a1, a3);
#pragma unroll
              for (int n = 0; n < NR; ++n)
                mma_16816<true>(s[n], a0, a1, a2, a3, qf[n][i2 * 4 + w][0], qf[n][i2 * 4 + w][1]);
            }
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int n = 0; n < NR; ++n)
                mma_16816<false>(s[n], wa[2 * w], wb[2 * w], wa[2 * w + 1], wb[2 * w + 1], qf[n][i2 * 2 + w][0],
                                 qf[n][i2 * 2 + w][1]);
          }
        }
      };
      float sc[C::KG][NR][4];
#pragma unroll
      for (int g = 0; g < C::KG; ++g) scores(g, sc[g]);

      // ---- z - M for z = y + log2 c, in packed fp32 pairs (rows 2tig and 2tig + 1). The base M moves only when a row
      // passes it by more than LIMIT; a row without one yet (M = -inf) counts from 0 and takes its first.
      float ka[C::KG], ev[C::KG], rv[C::KG];
      [[maybe_unused]] uint32_t far = 0u;
      if constexpr (F8) {
#pragma unroll
        for (int g = 0; g < C::KG; ++g) {
          const float2 ac = *reinterpret_cast<const float2*>(my_meta + slot * C::META + g * 8);
          ka[g] = ac.x;
          ev[g] = lg2_approx(ac.y);
          rv[g] = __fdividef(1.f, ac.y);
          if (ac.x > 0.f) ev_most = fmaxf(ev_most, ev[g]);  // (a group without keys has a = 0)
        }
        // A page's scale is in its keys' exponents, so pages of small values have small weights, and f16 keeps a weight's
        // bits down to 2^-14. With E = ev_most the base is at most max_j (y_j + log2 c_j) - TOP <= max y + E - TOP, hence
        // z_j - M >= (y_j - max y) - (E - log2 c_j) + TOP: up to GAP = TOP below E a page's scale costs its weights nothing.
        // A group further below (rare: values of two pages that differ more than 100-fold) is left out here and has its
        // turn after the others, with weights that count from its own largest. (64 sequences of 4-8k, d = 128: 125 us, 129
        // with every other page's values 2^10 larger, 149 with the first page's alone.)
#pragma unroll
        for (int g = 0; g < C::KG; ++g)
          if (ka[g] > 0.f && ev[g] < ev_most - DpBase<F8>::GAP) far |= 1u << g;  // (the same in every lane)
      }
      float mx[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n) mx[n][0] = mx[n][1] = -INFINITY;
      const uint32_t hid = ((hidden >> (4u * (done & 7u))) & 0xfu) | far;
      const bool need_mask = key0 + C::KS - 1 > full_lim || hid != 0u;
#pragma unroll
      for (int g = 0; g < C::KG; ++g) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint64_t c2 = F8 ? f2pack(c1[n][0] * ka[g], c1[n][1] * ka[g]) : f2pack(c1[n][0], c1[n][1]);
          const float e0 = F8 ? ev[g] : 0.f;
          const uint64_t b2 = f2pack(e0 - base_of(M[n][0]), e0 - base_of(M[n][1]));
          float(&z)[4] = sc[g][n];
          f2unpack(ffma2(f2pack(z[0], z[1]), c2, b2), z[0], z[1]);
          f2unpack(ffma2(f2pack(z[2], z[3]), c2, b2), z[2], z[3]);
          if (need_mask) {
            const int key = key0 + 16 * g + gid;
            const bool gone = (hid >> g) & 1u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + (e >> 1) * 8 > lim[n][e & 1] || gone) z[e] = -INFINITY;
          }
          mx[n][0] = fmax3(mx[n][0], z[0], z[2]);
          mx[n][1] = fmax3(mx[n][1], z[1], z[3]);
        }
      }
      bool over = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          over = over || mx[n][e] > (M[n][e] == -INFINITY ? -INFINITY : DpBase<F8>::LIMIT);
      if (__any_sync(ALL, over)) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float up = mx[n][e];
            up = fmaxf(up, __shfl_xor_sync(ALL, up, 4));
            up = fmaxf(up, __shfl_xor_sync(ALL, up, 8));
            up = fmaxf(up, __shfl_xor_sync(ALL, up, 16));
            const bool none = M[n][e] == -INFINITY;
            up -= DpBase<F8>::TOP;
            if (none) M[n][e] = up;                 // (still -inf when this tile shows the row nothing)
            else M[n][e] += up = fmaxf(up, 0.f);    // the base only rises
            up = up == -INFINITY ? 0.f : up;
            const float alpha = none ? 1.f : ex2_approx(-up);  // (without a base nothing was summed)
            l[n][e] *= alpha;
#pragma unroll
            for (int j = 0; j < C::KST; ++j) {
              oacc[n][j][e] *= alpha;
              oacc[n][j][e + 2] *= alpha;
            }
#pragma unroll
            for (int g = 0; g < C::KG; ++g) {
              sc[g][n][e] -= up;
              sc[g][n][e + 2] -= up;
            }
          }
      }
      // ---- W = 2^(z - M), its sums, and W as the B operand (rows on the columns): 8x8 transposes
      uint32_t pf[C::KG][NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int g = 0; g < C::KG; ++g) {
          const float w0 = ex2_approx(sc[g][n][0]), w1 = ex2_approx(sc[g][n][1]);
          const float w2 = ex2_approx(sc[g][n][2]), w3 = ex2_approx(sc[g][n][3]);
          const uint64_t ws = fadd2(f2pack(w0, w1), f2pack(w2, w3));
          const uint64_t l2 = f2pack(l[n][0], l[n][1]);
          f2unpack(F8 ? ffma2(ws, f2pack(rv[g], rv[g]), l2) : fadd2(l2, ws), l[n][0], l[n][1]);
          pf[g][n][0] = movmatrix_trans(F8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1));
          pf[g][n][1] = movmatrix_trans(F8 ? pack_f16x2(w2, w3) : pack_bf16x2(w2, w3));
        }
      // ---- O^T += V^T W^T
      // (FAR: times f for each row)
      auto product = [&](int g, const uint32_t (&w)[NR][2], auto far_group, const float (&f)[NR][2]) {
        constexpr bool FAR = decltype(far_group)::value;
        const uint32_t r0 = 16 * g + 2 * tig;
        if constexpr (F8) {
          constexpr int NW32 = D / 32;  // 32-bit words of the lane's codes: 4 or 2
          uint32_t v[4][NW32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t row = r0 + (q & 1) + 8 * (q >> 1);
            if constexpr (D == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(vt + dp_swz<C::RB>(row, gid));
              v[q][0] = y.x;
              v[q][1] = y.y;
              v[q][2] = y.z;
              v[q][3] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(vt + dp_swz<C::RB>(row, gid >> 1) + (gid & 1) * 8u);
              v[q][0] = y.x;
              v[q][1] = y.y;
            }
          }
#pragma unroll
          for (int x = 0; x < NW32; ++x) {
            const uint32_t x0 = __byte_perm(v[0][x], v[1][x], 0x5140), x1 = __byte_perm(v[0][x], v[1][x], 0x7362);
            const uint32_t y0 = __byte_perm(v[2][x], v[3][x], 0x5140), y1 = __byte_perm(v[2][x], v[3][x], 0x7362);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t xa = h ? x1 : x0, ya = h ? y1 : y0;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2x2(xa, a0, a1);
              e4m3x4_to_f16x2x2(ya, a2, a3);
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                float(&o)[4] = oacc[n][2 * x + h];
                if constexpr (FAR) {
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_16816<true>(t, a0, a1, a2, a3, w[n][0], w[n][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] = fmaf(t[e], f[n][e & 1], o[e]);
                } else {
                  mma_16816<true>(o, a0, a1, a2, a3, w[n][0], w[n][1]);
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int hp = 0; hp < D / 64; ++hp) {  // pieces gid and (d = 128) gid + 8
            uint32_t v[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 y = *reinterpret_cast<const uint4*>(vt + dp_swz<C::RB>(r0 + (q & 1) + 8 * (q >> 1), gid + 8 * hp));
              v[q][0] = y.x;
              v[q][1] = y.y;
              v[q][2] = y.z;
              v[q][3] = y.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a0 = __byte_perm(v[0][x], v[1][x], 0x5410), a1 = __byte_perm(v[0][x], v[1][x], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][x], v[3][x], 0x5410), a3 = __byte_perm(v[2][x], v[3][x], 0x7632);
#pragma unroll
              for (int n = 0; n < NR; ++n)
                mma_16816<false>(oacc[n][4 * hp + x], a0, a1, a2, a3, w[n][0], w[n][1]);
            }
          }
        }
      };
#pragma unroll
      for (int g = 0; g < C::KG; ++g) product(g, pf[g], std::false_type{}, M);
      // ---- the groups left out: with u a row's largest z in the group, W = 2^(u - M) W', W' = 2^(z - u)
      if constexpr (F8) {
        // (told to be rare: d = 64 spills otherwise)
        if (__builtin_expect(far != 0u, 0)) for (uint32_t rest = far; rest != 0u; rest &= rest - 1u) {
          const int g = __ffs(rest) - 1;
          const float2 ac = *reinterpret_cast<const float2*>(my_meta + slot * C::META + g * 8);
          const float lc = lg2_approx(ac.y);
          float z[NR][4], f[NR][2];
          uint32_t w[NR][2];
          scores(g, z);
#pragma unroll
          for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + 16 * g + gid;
              z[n][e] = key > lim[n][e] ? -INFINITY : fmaf(z[n][e], c1[n][e] * ac.x, lc);
              z[n][e + 2] = key + 8 > lim[n][e] ? -INFINITY : fmaf(z[n][e + 2], c1[n][e] * ac.x, lc);
              float u = fmaxf(z[n][e], z[n][e + 2]);
              u = fmaxf(u, __shfl_xor_sync(ALL, u, 4));
              u = fmaxf(u, __shfl_xor_sync(ALL, u, 8));
              u = fmaxf(u, __shfl_xor_sync(ALL, u, 16));
              const float m = fmaxf(M[n][e], u - DpBase<F8>::TOP), ub = base_of(u);
              const float alpha = m == M[n][e] ? 1.f : ex2_approx(M[n][e] - m);  // (0 for a row without a base)
              M[n][e] = m;
              f[n][e] = ex2_approx(ub - base_of(m));
              z[n][e] = ex2_approx(z[n][e] - ub);
              z[n][e + 2] = ex2_approx(z[n][e + 2] - ub);
              l[n][e] = fmaf(z[n][e] + z[n][e + 2], ex2_approx(ub - lc - base_of(m)), l[n][e] * alpha);
#pragma unroll
              for (int j = 0; j < C::KST; ++j) {
                oacc[n][j][e] *= alpha;
                oacc[n][j][e + 2] *= alpha;
              }
            }
            w[n][0] = movmatrix_trans(pack_f16x2(z[n][0], z[n][1]));
            w[n][1] = movmatrix_trans(pack_f16x2(z[n][2], z[n][3]));
          }
          product(g, w, std::true_type{}, f);
        }
      }
    }

    // ---- the segment's end: sums over the lanes, then the result, or this range's part of it
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[n][e];
        t += __shfl_xor_sync(ALL, t, 4);
        t += __shfl_xor_sync(ALL, t, 8);
        t += __shfl_xor_sync(ALL, t, 16);
        const int rl = n * 8 + 2 * tig + e, rr = rt * C::ROWS + rl;
        if (rr >= p.R) continue;
        // (scores that were all NaN leave the base where it was: their sum is NaN, and so is the row)
        const float m = M[n][e] == -INFINITY && t != 0.f ? 0.f : M[n][e];
        if (i0 == 0 && i1 == nt) {
          // the whole sequence; a row that sees no key has m = -inf, t = 0 (its O may be 0 times a NaN or infinity in v)
          const bool none = m == -INFINITY;
          const float inv = 1.f / t;
          auto out = [&](float y) { return none ? 0.f : y * inv; };
          const int h = hk * p.G + rr / p.Nq, tok = rr % p.Nq;
          uint16_t* op = static_cast<uint16_t*>(p.o) + b * p.osb + h * p.osh + tok * p.ost;
#pragma unroll
          for (int jj = 0; jj < C::KST / 2; ++jj)
            *reinterpret_cast<uint2*>(op + dp_o_elem<D, F8>(gid, jj)) =
                make_uint2(pack_bf16x2(out(oacc[n][2 * jj][e]), out(oacc[n][2 * jj][e + 2])),
                           pack_bf16x2(out(oacc[n][2 * jj + 1][e]), out(oacc[n][2 * jj + 1][e + 2])));
          if (p.lse != nullptr && gid == 0)
            p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + tok] =
                none ? -INFINITY : (m + lg2_approx(t)) * 0.69314718055994530942f;
        } else {
          // ranges and (sequence, head) pairs both only grow along the tiles, so their sum numbers the parts
          const long long part =
              ((static_cast<long long>(range) + static_cast<long long>(b) * p.Hkv + hk) * p.row_tiles + rt) * C::ROWS + rl;
          float* op = p.ws_o + part * D;
#pragma unroll
          for (int jj = 0; jj < C::KST / 2; ++jj)
            *reinterpret_cast<float4*>(op + dp_o_elem<D, F8>(gid, jj)) = make_float4(
                oacc[n][2 * jj][e], oacc[n][2 * jj][e + 2], oacc[n][2 * jj + 1][e], oacc[n][2 * jj + 1][e + 2]);
          if (gid == 0) *reinterpret_cast<float2*>(p.ws_ml + part * 2) = make_float2(m, t);
        }
      }
    // where the merge finds the parts of (b, hk)
    if (lane == 0 && rt == 0) {
      int* ends = p.ws_ends + 2 * (static_cast<long long>(b) * p.Hkv + hk);
      if (i0 == 0) ends[0] = range;
      if (i1 == nt) ends[1] = range;
    }
    todo -= i1 - i0;
    if (todo > 0) {
      i = nt - 1;  // the last tile of (b, hk) is done
      advance(b, hk, i, L, nt);
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of the query rows whose keys lie in several ranges: M = max m_r,
// O = sum 2^(m_r - M) o_r / sum 2^(m_r - M) l_r. WPR warps a row (one where a row
// has a few parts, eight where long sequences have many); a warp has up to eight
// parts in flight. Rows of one range were written by the decode kernel itself;
// rows of an empty sequence, which no range holds, are written here.
constexpr int DP_MERGE_WARPS = 8;
template <int D, int WPR>
__global__ void __launch_bounds__(32 * DP_MERGE_WARPS) fa_decode_paged_merge_kernel(const DecodePagedParams p, int rows) {
  __shared__ float sm[DP_MERGE_WARPS], sl[DP_MERGE_WARPS];
  __shared__ float so[WPR > 1 ? DP_MERGE_WARPS : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = warp % WPR;  // of the row's warps
  const int row = static_cast<int>(blockIdx.x) * (DP_MERGE_WARPS / WPR) + warp / WPR;
  const bool in = row < p.B * p.H * p.Nq;
  const int t = in ? row % p.Nq : 0, bh = in ? row / p.Nq : 0;
  const int h = bh % p.H, b = bh / p.H;
  const int hk = h / p.G, rr = (h - hk * p.G) * p.Nq + t;
  const int L = dp_len(p, b);
  // (every warp waits, also those with nothing to join: what follows this launch may not pass the decode kernel)
  pdl_wait();
  const int2 ends = L > 0 ? __ldcg(reinterpret_cast<const int2*>(p.ws_ends) + static_cast<long long>(b) * p.Hkv + hk)
                          : make_int2(0, -1);
  if (!in || ends.x == ends.y) return;  // (with WPR > 1 the same for the block: it is one row)
  const int ns = ends.y - ends.x + 1;
  const long long step = static_cast<long long>(p.row_tiles) * rows;  // parts from one range to the next
  const long long part0 = (ends.x + static_cast<long long>(b) * p.Hkv + hk) * step + (rr / rows) * rows + rr % rows;
  constexpr int EL = D / 32, FLIGHT = 8;
  float acc[EL], lt = 0.f, m = -INFINITY;
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  for (int s0 = w; s0 < ns; s0 += FLIGHT * WPR) {
    float2 ml[FLIGHT];
    float y[FLIGHT][EL];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
      const int s = s0 + j * WPR;
      ml[j] = make_float2(-INFINITY, 0.f);
      if (s < ns) {
        const long long part = part0 + s * step;
        ml[j] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + part);
        if constexpr (EL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_o + part * D) + lane);
          y[j][0] = v.x, y[j][1] = v.y, y[j][2] = v.z, y[j][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(p.ws_o + part * D) + lane);
          y[j][0] = v.x, y[j][1] = v.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) mn = fmaxf(mn, ml[j].x);
    if (mn == -INFINITY) continue;  // nothing seen so far
    const float a = ex2_approx(m - mn);
    lt *= a;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] *= a;
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
      if (ml[j].x == -INFINITY) continue;  // no part, or one that saw no key
      const float wgt = ex2_approx(ml[j].x - mn);
      lt = fmaf(wgt, ml[j].y, lt);
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[e] = fmaf(wgt, y[j][e], acc[e]);
    }
    m = mn;
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      sm[w] = m;
      sl[w] = lt;
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) so[w][lane * EL + e] = acc[e];
    __syncthreads();
    if (w > 0) return;
    m = sm[0];
#pragma unroll
    for (int x = 1; x < WPR; ++x) m = fmaxf(m, sm[x]);
    lt = 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = 0.f;
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
      const float f = sm[x] == -INFINITY ? 0.f : ex2_approx(sm[x] - m);
      lt = fmaf(f, sl[x], lt);
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[e] = fmaf(f, so[x][lane * EL + e], acc[e]);
    }
  }
  const float inv = m == -INFINITY ? 0.f : 1.f / lt;
  uint16_t* op = static_cast<uint16_t*>(p.o) + b * p.osb + h * p.osh + t * p.ost + lane * EL;
  if constexpr (EL == 4)
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = m == -INFINITY ? -INFINITY : (m + lg2_approx(lt)) * 0.69314718055994530942f;
}

template <int D, bool F8, int NR>
static cudaError_t dp_attr() {
  return cudaFuncSetAttribute(fa_decode_paged_kernel<D, F8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DpCfg<D, F8, NR>::SMEM);
}
cudaError_t decode_paged_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {dp_attr<64, false, 1>(), dp_attr<64, false, 2>(), dp_attr<64, true, 1>(), dp_attr<64, true, 2>(),
                        dp_attr<128, false, 1>(), dp_attr<128, false, 2>(), dp_attr<128, true, 1>(),
                        dp_attr<128, true, 2>()})
    if (x != cudaSuccess) e = x;
  return e;
}

template <int D, bool F8, int NR>
static cudaError_t dp_launch(const DecodePagedParams& p, cudaStream_t stream) {
  using C = DpCfg<D, F8, NR>;
  const long long workers = static_cast<long long>(p.n_ranges) * p.row_tiles;
  fa_decode_paged_kernel<D, F8, NR><<<static_cast<unsigned>((workers + DP_WARPS - 1) / DP_WARPS), DP_THREADS, C::SMEM, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the merge's CTAs may be set up while the last ranges run; those that read parts wait for them
  cudaLaunchConfig_t cfg{};
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nq;
  // Eight warps a row where it has more than eight parts on average (two sequences of 110k tokens: 74 us a call, one
  // warp a row 85), else one (64 of 4-8k: 124 against 132 us; 48 with 4 tokens, 6144 rows: 62 against 77).
  const bool many = p.n_ranges / (static_cast<long long>(p.B) * p.Hkv) > 8;
  cfg.gridDim = dim3(static_cast<unsigned>(many ? rows : (rows + DP_MERGE_WARPS - 1) / DP_MERGE_WARPS));
  cfg.blockDim = dim3(32 * DP_MERGE_WARPS);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, fa_decode_paged_merge_kernel<D, DP_MERGE_WARPS>, p, C::ROWS)
              : cudaLaunchKernelEx(&cfg, fa_decode_paged_merge_kernel<D, 1>, p, C::ROWS);
}

template <int D, bool F8>
static cudaError_t dp_launch_rows(const DecodePagedParams& p, cudaStream_t stream) {
  return decode_paged_rows(p.R) == 8 ? dp_launch<D, F8, 1>(p, stream) : dp_launch<D, F8, 2>(p, stream);
}
cudaError_t launch_decode_paged(int d, bool f8, const DecodePagedParams& p, cudaStream_t stream) {
  if (d == 64) return f8 ? dp_launch_rows<64, true>(p, stream) : dp_launch_rows<64, false>(p, stream);
  return f8 ? dp_launch_rows<128, true>(p, stream) : dp_launch_rows<128, false>(p, stream);
}

}  // namespace fa
