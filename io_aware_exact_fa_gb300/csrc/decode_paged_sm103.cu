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
//     W_j = 2^(z_j - M) <= 1,  O = sum_j W_j V~_j / sum_j (W_j / c_j),
//     lse = ln 2 (M + log2 sum_j (W_j / c_j)),
// so the value products run on the codes themselves, whatever the pages' scales
// are to one another, and neither sum can overflow (append writes powers of two,
// for which W_j / c_j and the shift by log2 c are exact).
//
// What bounds it: HBM. Each key and value is read once per K/V head; at 6.8 TB/s
// an SM takes about 24 bytes a clock, 24 e4m3 codes. The work per code has to
// stay well below the SM's issue rate, which rules out CUDA-core products for
// more than a few rows; a 128-row tensor-memory tile would be nearly empty and
// cannot convert codes. So warp-level products on registers: the keys are the
// M side of S^T = K Q^T and the head dimension the M side of O^T = V^T P^T, the
// 8 (or 16) query rows the N side, and neither product pads the rows past 8.
//
// Split-KV: CTA (row tile, split, K/V head, sequence); its 4 warps take tiles of
// KS keys in turn, each with a private ring of asynchronous 16-byte copies, so
// there is no barrier inside the loop. A tile's 16-key groups may lie in
// different pages; one lane per group looks the page up. The fragments are read
// straight from the copied rows: the order of the contraction over d (for S) and
// of the output rows (for O^T) is free, so each lane takes whole 16-byte pieces
// of its rows, and the shared-memory positions of the pieces are XORed with the
// row so that those reads touch every bank once.
#include <cuda_bf16.h>

#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

constexpr int DP_WARPS = 4;
constexpr int DP_THREADS = 32 * DP_WARPS;
constexpr int DP_STAGES = 3;           // tiles in each warp's ring
constexpr int DP_HALF_BYTES = 4096;    // K (or V) bytes of a tile
constexpr float DP_RESCALE_LOG2 = 8.f; // the base moves when a score passes it by more than this

template <int D, bool F8, int NR>
struct DpCfg {
  static constexpr int ESZ = F8 ? 1 : 2;
  static constexpr int RB = D * ESZ;             // bytes of a key's row: 64, 128 or 256
  static constexpr int CR = RB / 16;             // 16-byte pieces of a row
  static constexpr int KS = DP_HALF_BYTES / RB;  // keys of a tile: 64, 32 or 16
  static constexpr int KG = KS / 16;             // its 16-key groups
  static constexpr int EPC = 16 / ESZ;           // elements of a piece
  static constexpr int DL = D / 4;               // elements of a K row that one lane holds
  static constexpr int NPK = DL / EPC;           // as pieces
  static constexpr int KST = D / 16;             // k-steps of S^T, and M tiles of O^T
  static constexpr int ROWS = 8 * NR;
  static constexpr int META = KG * 2 * 4;        // e4m3 scales of a tile
  static constexpr int STAGE = 2 * DP_HALF_BYTES;
  static constexpr int RING = DP_WARPS * DP_STAGES * STAGE;
  static constexpr int META_OFF = RING;
  static constexpr int SMEM = RING + DP_WARPS * DP_STAGES * META;
  // after the loop the ring holds the warps' outputs and their (base, sum)
  static constexpr int OROW = D + 4;             // floats of a row: 8-byte stores of a half-warp hit every bank once
  static constexpr int ML_OFF = DP_WARPS * ROWS * OROW * 4;
  static_assert(ML_OFF + DP_WARPS * ROWS * 8 <= RING, "the merge area fits the ring");
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
// Position (j * 8 + gid) * 2 + e of element d of an output row: lane group gid
// holds it in M tile j, fragment row gid + 8 e.
template <int D, bool F8>
__device__ __forceinline__ int dp_o_pos(int d) {
  int gid, j2;
  if constexpr (!F8 && D == 128) {
    gid = (d >> 3) & 7;
    j2 = (d & 7) + ((d >> 6) << 3);
  } else {
    gid = d / (D / 8);
    j2 = d % (D / 8);
  }
  return ((j2 >> 1) * 8 + gid) * 2 + (j2 & 1);
}

}  // namespace

template <int D, bool F8, int NR>
__global__ void __launch_bounds__(DP_THREADS, 2) fa_decode_paged_kernel(const DecodePagedParams p) {
  using C = DpCfg<D, F8, NR>;
  extern __shared__ __align__(128) uint8_t dp_smem[];
  const uint32_t sbase = smem_u32(dp_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;

  // block -> (row tile, K/V head, split, sequence); row tiles of the same keys are neighbours
  int x = static_cast<int>(blockIdx.x);
  const int rt = x % p.row_tiles;
  x /= p.row_tiles;
  const int hk = x % p.Hkv;
  x /= p.Hkv;
  const int s = x % p.S;
  const int b = x / p.S;

  pdl_launch_dependents();
  const int raw_len = __ldg(p.seqlens + b);
  const int L = paged_clip_len(raw_len, p.max_len);
  if (L != raw_len && s == 0 && rt == 0 && hk == 0 && threadIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
  const int k0 = s * p.chunk;
  if (k0 >= L && s > 0) return;  // this split has no key: the merge does not read it
  const int kend = min(L, k0 + p.chunk);

  // ---- Q: lane (gid, tig) holds its elements of query row gid of every 8-row tile
  uint32_t qf[NR][C::KST][2];
  float c1[NR][2];   // factor of the scores of rows 2tig and 2tig + 1 (log2 units)
  int lim[NR][2];    // last key those rows see
  const uint16_t* qp = static_cast<const uint16_t*>(p.q) + b * p.qsb;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = rt * C::ROWS + n * 8 + gid;
    const bool in = r < p.R;
    const uint16_t* qr = qp + (hk * p.G + (in ? r / p.Nq : 0)) * p.qsh + (in ? r % p.Nq : 0) * p.qst;
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
      // off by at most 2^-25 of the largest, below fp32 accumulation's own error.
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < C::KST; ++j) {
        const uint32_t w[2] = {raw[j].x, raw[j].y};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
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
      c1[n][e] = p.scale_log2 * (F8 ? __shfl_sync(0xffffffffu, row_factor, (2 * tig + e) * 4) : 1.f);
      const int r2 = rt * C::ROWS + n * 8 + 2 * tig + e;
      lim[n][e] = min(kend - 1, r2 < p.R ? L - p.Nq + r2 % p.Nq : kend - 1);
    }
  }

  // ---- the warp's tiles: base key k0 + (warp + 4 i) KS
  const int ntiles_cta = (kend - k0 + C::KS - 1) / C::KS;  // (negative spans give no tile)
  const int ntiles = ntiles_cta > warp ? (ntiles_cta - warp + DP_WARPS - 1) / DP_WARPS : 0;
  const uint32_t ring = sbase + warp * (DP_STAGES * C::STAGE);
  const uint32_t meta = sbase + C::META_OFF + warp * (DP_STAGES * C::META);
  const int* trow = p.table + b * p.table_stride;
  const int full_lim = min(kend - 1, L - p.Nq);  // every row sees the keys up to here
  uint32_t hidden = 0u;                          // 4 bits for each of 8 tiles: groups whose page is not in the pool

  auto tile_key = [&](int i) { return k0 + (warp + DP_WARPS * i) * C::KS; };
  // page of 16-key group `lane` of tile i; -1 past the keys or for other lanes
  auto page_of = [&](int i) -> int {
    const int key = tile_key(i) + 16 * lane;
    return (lane < C::KG && i < ntiles && key < kend) ? __ldg(trow + (key >> p.page_shift)) : -1;
  };
  auto issue = [&](int i, int id) {
    if (i < ntiles) {
      const int key0 = tile_key(i);
      const int gkey = key0 + 16 * lane;
      const bool want = lane < C::KG && gkey < kend;
      long long off = want ? paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, gkey & (p.page - 1), D) : -1;
      const unsigned bad = __ballot_sync(0xffffffffu, want && off < 0);
      if (bad != 0u && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      const uint32_t sh = 4u * (static_cast<uint32_t>(i) & 7u);
      hidden = (hidden & ~(0xfu << sh)) | ((bad & 0xfu) << sh);
      const uint32_t slot = static_cast<uint32_t>(i % DP_STAGES);
      const uint32_t kdst = ring + slot * C::STAGE, vdst = kdst + DP_HALF_BYTES;
      if constexpr (F8) {
        if (lane < C::KG) {
          const uint32_t m = meta + slot * C::META + lane * 8u;
          if (off >= 0) {
            const long long sc = static_cast<long long>(id) * p.Hkv + hk;
            cp_async4(m, p.k_scale + sc);
            cp_async4(m + 4u, p.v_scale + sc);
          } else {
            st_shared_f32(m, 0.f);
            st_shared_f32(m + 4u, 1.f);
          }
        }
      }
      constexpr int RPI = 32 / C::CR;        // rows of one copy instruction of the warp
      const int piece = lane % C::CR, rin = lane / C::CR;
#pragma unroll
      for (int g = 0; g < C::KG; ++g) {
        const long long goff = __shfl_sync(0xffffffffu, off, g);
        const int left = goff < 0 ? 0 : kend - (key0 + 16 * g);  // rows of the group to read
        const uint8_t* kg = static_cast<const uint8_t*>(p.k) + (goff < 0 ? 0 : goff) * C::ESZ;
        const uint8_t* vg = static_cast<const uint8_t*>(p.v) + (goff < 0 ? 0 : goff) * C::ESZ;
#pragma unroll
        for (int u = 0; u < 16 / RPI; ++u) {
          const int row = u * RPI + rin;
          const uint32_t dst = dp_swz<C::RB>(16 * g + row, piece);
          const uint32_t n = row < left ? 16u : 0u;
          const size_t so = n ? static_cast<size_t>(row) * C::RB + piece * 16 : 0;
          cp_async16(kdst + dst, kg + so, n);
          cp_async16(vdst + dst, vg + so, n);
        }
      }
    }
    cp_async_commit();
  };

  float M[NR][2], l[NR][2];
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

  int id_next = page_of(0);
#pragma unroll
  for (int i = 0; i < DP_STAGES - 1; ++i) {
    const int id = id_next;
    id_next = page_of(i + 1);
    issue(i, id);
  }
  for (int i = 0; i < ntiles; ++i) {
    cp_async_wait<DP_STAGES - 2>();
    __syncwarp();  // tile i landed for every lane, and every lane is done with tile i - 1's slot
    {
      const int id = id_next;
      id_next = page_of(i + DP_STAGES);
      issue(i + DP_STAGES - 1, id);
    }
    const uint32_t slot = static_cast<uint32_t>(i % DP_STAGES);
    const uint32_t kt = ring + slot * C::STAGE, vt = kt + DP_HALF_BYTES;
    const int key0 = tile_key(i);

    // ---- S^T: 16 keys x 8 rows for each group and row tile
    float sc[C::KG][NR][4];
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[g][n][e] = 0.f;
#pragma unroll
      for (int i2 = 0; i2 < C::NPK; ++i2) {
        const int piece = dp_k_piece<D, F8>(tig, i2);
        const uint4 ra = ld_shared_v4(kt + dp_swz<C::RB>(16 * g + gid, piece));
        const uint4 rb = ld_shared_v4(kt + dp_swz<C::RB>(16 * g + gid + 8, piece));
        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
        if constexpr (F8) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(wa[w]), a2 = e4m3x2_to_f16x2(wa[w] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(wb[w]), a3 = e4m3x2_to_f16x2(wb[w] >> 16);
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma_16816<true>(sc[g][n], a0, a1, a2, a3, qf[n][i2 * 4 + w][0], qf[n][i2 * 4 + w][1]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma_16816<false>(sc[g][n], wa[2 * w], wb[2 * w], wa[2 * w + 1], wb[2 * w + 1], qf[n][i2 * 2 + w][0],
                               qf[n][i2 * 2 + w][1]);
        }
      }
    }

    // ---- z = y + log2 c, masked; the base moves only when a row passes it by 2^8
    float rv[C::KG];
    float mx[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) mx[n][0] = mx[n][1] = -INFINITY;
    const uint32_t hid = (hidden >> (4u * (static_cast<uint32_t>(i) & 7u))) & 0xfu;
    const bool need_mask = key0 + C::KS - 1 > full_lim || hid != 0u;
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      float ka = 1.f, ev = 0.f;
      rv[g] = 1.f;
      if constexpr (F8) {
        const float c = ld_shared_f32(meta + slot * C::META + g * 8u + 4u);
        ka = ld_shared_f32(meta + slot * C::META + g * 8u);
        ev = lg2_approx(c);
        rv[g] = __fdividef(1.f, c);
      }
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = F8 ? fmaf(sc[g][n][e], c1[n][e & 1] * ka, ev) : sc[g][n][e] * c1[n][e & 1];
          if (need_mask) {
            const int key = key0 + 16 * g + gid + (e >> 1) * 8;
            if (key > lim[n][e & 1] || ((hid >> g) & 1u)) z = -INFINITY;
          }
          sc[g][n][e] = z;
          mx[n][e & 1] = fmaxf(mx[n][e & 1], z);
        }
    }
    bool over = false;
#pragma unroll
    for (int n = 0; n < NR; ++n)
      over = over || mx[n][0] > M[n][0] + DP_RESCALE_LOG2 || mx[n][1] > M[n][1] + DP_RESCALE_LOG2;
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(mx[n][e], M[n][e]);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const float alpha = m == -INFINITY ? 1.f : ex2_approx(M[n][e] - m);
          M[n][e] = m;
          l[n][e] *= alpha;
#pragma unroll
          for (int j = 0; j < C::KST; ++j) {
            oacc[n][j][e] *= alpha;
            oacc[n][j][e + 2] *= alpha;
          }
        }
    }
    // ---- W = 2^(z - M), its sums, and W as the B operand (rows on the columns): 8x8 transposes
    uint32_t pf[C::KG][NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const float m0 = M[n][0] == -INFINITY ? 0.f : M[n][0], m1 = M[n][1] == -INFINITY ? 0.f : M[n][1];
#pragma unroll
      for (int g = 0; g < C::KG; ++g) {
        const float w0 = ex2_approx(sc[g][n][0] - m0), w1 = ex2_approx(sc[g][n][1] - m1);
        const float w2 = ex2_approx(sc[g][n][2] - m0), w3 = ex2_approx(sc[g][n][3] - m1);
        l[n][0] = F8 ? fmaf(w0 + w2, rv[g], l[n][0]) : l[n][0] + (w0 + w2);
        l[n][1] = F8 ? fmaf(w1 + w3, rv[g], l[n][1]) : l[n][1] + (w1 + w3);
        pf[g][n][0] = movmatrix_trans(F8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1));
        pf[g][n][1] = movmatrix_trans(F8 ? pack_f16x2(w2, w3) : pack_bf16x2(w2, w3));
      }
    }
    // ---- O^T += V^T W^T
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      const uint32_t r0 = 16 * g + 2 * tig;
      if constexpr (F8) {
        constexpr int NW32 = D / 32;  // 32-bit words of the lane's codes: 4 or 2
        uint32_t v[4][NW32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t row = r0 + (q & 1) + 8 * (q >> 1);
          if constexpr (D == 128) {
            const uint4 y = ld_shared_v4(vt + dp_swz<C::RB>(row, gid));
            v[q][0] = y.x;
            v[q][1] = y.y;
            v[q][2] = y.z;
            v[q][3] = y.w;
          } else {
            const uint2 y = ld_shared_v2(vt + dp_swz<C::RB>(row, gid >> 1) + (gid & 1) * 8u);
            v[q][0] = y.x;
            v[q][1] = y.y;
          }
        }
#pragma unroll
        for (int w = 0; w < NW32; ++w) {
          const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t xa = h ? x1 : x0, ya = h ? y1 : y0;
            const uint32_t a0 = e4m3x2_to_f16x2(xa), a1 = e4m3x2_to_f16x2(xa >> 16);
            const uint32_t a2 = e4m3x2_to_f16x2(ya), a3 = e4m3x2_to_f16x2(ya >> 16);
#pragma unroll
            for (int n = 0; n < NR; ++n) mma_16816<true>(oacc[n][2 * w + h], a0, a1, a2, a3, pf[g][n][0], pf[g][n][1]);
          }
        }
      } else {
#pragma unroll
        for (int hp = 0; hp < D / 64; ++hp) {  // pieces gid and (d = 128) gid + 8
          uint32_t v[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 y = ld_shared_v4(vt + dp_swz<C::RB>(r0 + (q & 1) + 8 * (q >> 1), gid + 8 * hp));
            v[q][0] = y.x;
            v[q][1] = y.y;
            v[q][2] = y.z;
            v[q][3] = y.w;
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma_16816<false>(oacc[n][4 * hp + w], a0, a1, a2, a3, pf[g][n][0], pf[g][n][1]);
          }
        }
      }
    }
  }

  // ---- join the warps: bases and sums, then the rescaled outputs, in shared memory
  cp_async_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(dp_smem);
  float2* sml = reinterpret_cast<float2*>(dp_smem + C::ML_OFF);
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[n][e];
      t += __shfl_xor_sync(0xffffffffu, t, 4);
      t += __shfl_xor_sync(0xffffffffu, t, 8);
      t += __shfl_xor_sync(0xffffffffu, t, 16);
      if (gid == 0) sml[warp * C::ROWS + n * 8 + 2 * tig + e] = make_float2(M[n][e], t);
    }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = n * 8 + 2 * tig + e;
      float m = sml[r].x;
#pragma unroll
      for (int w = 1; w < DP_WARPS; ++w) m = fmaxf(m, sml[w * C::ROWS + r].x);
      f[e] = M[n][e] == -INFINITY ? 0.f : ex2_approx(M[n][e] - m);
    }
#pragma unroll
    for (int j = 0; j < C::KST; ++j) {
      float* dst = so + (warp * C::ROWS + n * 8 + 2 * tig) * C::OROW + (j * 8 + gid) * 2;
      *reinterpret_cast<float2*>(dst) = make_float2(oacc[n][j][0] * f[0], oacc[n][j][2] * f[0]);
      *reinterpret_cast<float2*>(dst + C::OROW) = make_float2(oacc[n][j][1] * f[1], oacc[n][j][3] * f[1]);
    }
  }
  __syncthreads();
  const bool last = p.S == 1;  // no merge follows
  for (int i = threadIdx.x; i < C::ROWS * (D / 2); i += DP_THREADS) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2));
    const int rr = rt * C::ROWS + r;
    if (rr >= p.R) break;  // rows are in order
    float m = sml[r].x;
#pragma unroll
    for (int w = 1; w < DP_WARPS; ++w) m = fmaxf(m, sml[w * C::ROWS + r].x);
    float lt = 0.f, o0 = 0.f, o1 = 0.f;
    const int pos = dp_o_pos<D, F8>(d);
#pragma unroll
    for (int w = 0; w < DP_WARPS; ++w) {
      const float2 ml = sml[w * C::ROWS + r];
      lt += ml.x == -INFINITY ? 0.f : ml.y * ex2_approx(ml.x - m);
      const float2 y = *reinterpret_cast<const float2*>(so + (w * C::ROWS + r) * C::OROW + pos);
      o0 += y.x;
      o1 += y.y;
    }
    const int h = hk * p.G + rr / p.Nq, t = rr % p.Nq;
    const long long row = (static_cast<long long>(b) * p.H + h) * p.Nq + t;
    if (last) {
      // a row that sees no key: m = -inf, lt = 0
      const float inv = m == -INFINITY ? 0.f : 1.f / lt;
      uint16_t* op = static_cast<uint16_t*>(p.o) + b * p.osb + h * p.osh + t * p.ost + d;
      *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(o0 * inv, o1 * inv);
      if (p.lse != nullptr && d == 0) p.lse[row] = m == -INFINITY ? -INFINITY : (m + lg2_approx(lt)) * 0.69314718055994530942f;
    } else {
      const long long part = row * p.S + s;
      *reinterpret_cast<float2*>(p.ws_o + part * D + d) = make_float2(o0, o1);
      if (d == 0) *reinterpret_cast<float2*>(p.ws_ml + part * 2) = make_float2(m, lt);
    }
  }
}

// Joins the splits of one query row: M = max m_s, O = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s over
// the splits that hold keys. One CTA a row; warp w takes splits w, w + 4, ..
template <int D>
__global__ void __launch_bounds__(128) fa_decode_paged_merge_kernel(const DecodePagedParams p) {
  __shared__ float sm[4], sl[4];
  __shared__ float so[4][D];
  const int row = static_cast<int>(blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = row % p.Nq, bh = row / p.Nq;
  const int h = bh % p.H, b = bh / p.H;
  const int L = paged_clip_len(__ldg(p.seqlens + b), p.max_len);
  const int ns = max(1, (L + p.chunk - 1) / p.chunk);
  pdl_wait();
  const float* ml = p.ws_ml + static_cast<long long>(row) * p.S * 2;
  float m = -INFINITY;
  for (int s = threadIdx.x; s < ns; s += 128) m = fmaxf(m, __ldcg(ml + 2 * s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  constexpr int EL = D / 32;
  float acc[EL], lt = 0.f;
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  const float* po = p.ws_o + static_cast<long long>(row) * p.S * D + lane * EL;
#pragma unroll 4
  for (int s = warp; s < ns; s += 4) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(ml) + s);
    const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - m);
    lt = fmaf(w, x.y, lt);
    float y[EL];
    if constexpr (EL == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(po + static_cast<long long>(s) * D));
      y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(po + static_cast<long long>(s) * D));
      y[0] = v.x, y[1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = fmaf(w, y[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < EL; ++e) so[warp][lane * EL + e] = acc[e];
  if (lane == 0) sl[warp] = lt;
  __syncthreads();
  if (threadIdx.x < D / 2) {
    const int d = 2 * threadIdx.x;
    const float tot = (sl[0] + sl[1]) + (sl[2] + sl[3]);
    const float inv = m == -INFINITY ? 0.f : 1.f / tot;
    const float o0 = (so[0][d] + so[1][d]) + (so[2][d] + so[3][d]);
    const float o1 = (so[0][d + 1] + so[1][d + 1]) + (so[2][d + 1] + so[3][d + 1]);
    uint16_t* op = static_cast<uint16_t*>(p.o) + b * p.osb + h * p.osh + t * p.ost + d;
    *reinterpret_cast<uint32_t*>(op) = pack_bf16x2(o0 * inv, o1 * inv);
    if (p.lse != nullptr && d == 0)
      p.lse[row] = m == -INFINITY ? -INFINITY : (m + lg2_approx(tot)) * 0.69314718055994530942f;
  }
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
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(p.row_tiles) * p.Hkv * p.S * p.B);
  fa_decode_paged_kernel<D, F8, NR><<<grid, DP_THREADS, DpCfg<D, F8, NR>::SMEM, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.S == 1) return e;
  // the merge's CTAs may be set up while the last splits run; it waits for them before it reads
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.H * p.Nq));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_decode_paged_merge_kernel<D>, p);
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
