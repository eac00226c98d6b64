// Eviction from a paged K/V cache by accumulated attention weight, for sm_103a.
//
// Of the L rows of a sequence every K/V head keeps its first `first` and last
// `recent`, and of those between the keep - first - recent with the largest weights
// (ties to the lowest index; NaN counts as -inf); a sequence of at most `keep` rows
// keeps all. The rows that stay are moved, in order, to the pages of a new table.
//
// Two launches. (1) Selection. A weight's bits, flipped so that they order as
// unsigned integers, are compared through digits: the rows between are counted by
// their top 11 bits, then those that share the border's digit by the next 11, then
// by the last 10; after that the border value and how many of its ties stay are
// known, exactly. A cluster of blocks shares one (sequence, K/V head): each holds a
// contiguous part of its keys in shared memory (so the weights are read once), and
// the counts are summed over the cluster's shared memories. Then every warp counts
// its contiguous run, and with the runs' sums before it writes indices and weights
// in order. (2) The move: a block takes 128 new rows of one head and copies their
// keys and values, 16 bytes (4-bit rows: also the scale bytes) a thread. A new e4m3
// page's scale is the largest of its rows' old ones, and codes whose scale grew are
// rounded again.
// What bounds it: HBM, the weights read and the kept rows read and written; for one
// or two sequences the selection's chain of passes.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace cg = cooperative_groups;

namespace fa {

namespace {

constexpr int EV_THREADS = 512;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048;
constexpr int EV_MAX_CLUSTER = 8;
constexpr int EV_HELD = 40960;    // keys that a block holds in shared memory, at most
constexpr int EV_ROWS = 128;      // new rows of a moving block
constexpr int EV_MOVE_THREADS = 256;

// Order-preserving bits: larger weights have larger keys, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

static_assert(EV_BINS == 4 * EV_THREADS, "a thread sums four bins");

struct EvShared {
  uint32_t hist[EV_BINS];   // this block's counts
  uint32_t part[EV_WARPS];  // scans
  uint32_t above[EV_WARPS], ties[EV_WARPS];
  uint32_t digit, left;     // the border's digit and how many of its rows stay
  uint32_t totals[2];       // kept and tied rows of this block
};

}  // namespace

// HELD: a block's keys fit its shared memory; else they are read again for every pass.
template <bool HELD>
__global__ void __launch_bounds__(EV_THREADS) fa_evict_select_kernel(const EvictPagedParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  extern __shared__ uint32_t ev_keys[];
  __shared__ EvShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = static_cast<int>(blockIdx.x) / ranks;
  const int b = pair / p.Hkv, hk = pair % p.Hkv;
  pdl_launch_dependents();
  const int raw = __ldg(p.seqlens + b), L = paged_clip_len(raw, p.max_len);
  const int keep = p.keep, n_new = min(L, keep);
  if (hk == 0 && rank == 0 && tid == 0) {
    if (raw != L) atomicOr(p.status, FA_DEV_BAD_LENS);
    p.new_seqlens[b] = n_new;
    p.new_offsets[b] = static_cast<int>((p.offsets == nullptr ? 0u : static_cast<unsigned>(p.offsets[b])) +
                                        static_cast<unsigned>(L - n_new));
  }
  const float* w = p.weights + pair * p.wstride;
  int* kept = p.kept + static_cast<long long>(pair) * keep;
  float* nw = p.new_weights + pair * p.new_wstride;
  // past the rows that stay
  for (int i = n_new + rank * EV_THREADS + tid; i < p.new_width; i += ranks * EV_THREADS) {
    if (i < keep) kept[i] = -1;
    nw[i] = 0.f;
  }
  if (L <= keep) {  // (the same for the whole cluster)
    for (int i = rank * EV_THREADS + tid; i < L; i += ranks * EV_THREADS) {
      kept[i] = i;
      nw[i] = w[i];
    }
    return;
  }
  // ---- this block's part of the rows, a multiple of 32 of them a warp
  const int per_warp = ((L + ranks * EV_WARPS - 1) / (ranks * EV_WARPS) + 31) / 32 * 32;
  const int part0 = min(static_cast<long long>(L), static_cast<long long>(rank) * per_warp * EV_WARPS);
  const int part1 = min(static_cast<long long>(L), static_cast<long long>(rank + 1) * per_warp * EV_WARPS);
  const int lo = p.first, hi = L - p.recent;            // rows between
  uint32_t want = static_cast<uint32_t>(keep - p.first - p.recent);  // of them stay
  uint32_t border = 0u, known = 0u;                     // the border's upper digits and their mask
  bool exact = want == 0u;                              // border found: rows with key > border (and `want` ties) stay
  if (want == 0u) border = 0xffffffffu;                 // (no weight has this key: it would be a NaN's)
  auto key_at = [&](int j) { return HELD ? ev_keys[j - part0] : order_key(__ldg(w + j)); };
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : EV_BINS;
    for (int i = tid; i < EV_BINS; i += EV_THREADS) sh.hist[i] = 0u;
    __syncthreads();
    if (pass == 0) {
      for (int j = part0 + tid; j < part1; j += EV_THREADS) {
        const uint32_t k = order_key(__ldg(w + j));
        if (HELD) ev_keys[j - part0] = k;
        if (!exact && j >= lo && j < hi) atomicAdd(&sh.hist[k >> 21], 1u);
      }
    } else if (!exact) {
      for (int j = part0 + tid; j < part1; j += EV_THREADS) {
        const uint32_t k = key_at(j);
        if (j >= lo && j < hi && ((k ^ border) & known) == 0u) atomicAdd(&sh.hist[(k >> shift) & (bins - 1)], 1u);
      }
    }
    cluster.sync();
    if (!exact) {
      // every block sums the cluster's counts for itself; a thread has four bins, the highest first
      uint32_t c[4], sum = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int bin = EV_BINS - 1 - (4 * tid + i);
        c[i] = 0u;
        for (int r = 0; r < ranks; ++r) c[i] += cluster.map_shared_rank(sh.hist, r)[bin];
        sum += c[i];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sh.part[warp] = inc;
      __syncthreads();
      uint32_t before = inc - sum;
      for (int x = 0; x < warp; ++x) before += sh.part[x];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < want && want <= before + c[i]) {
          sh.digit = EV_BINS - 1 - (4 * tid + i);
          sh.left = want - before;
        }
        before += c[i];
      }
      __syncthreads();
      border |= sh.digit << shift;
      known |= static_cast<uint32_t>(bins - 1) << shift;
      want = sh.left;
    }
    cluster.sync();  // nobody reads the counts any more
    if (exact) break;
  }
  // ---- each warp counts its run, then writes
  const int run0 = min(part1, part0 + warp * per_warp), run1 = min(part1, run0 + per_warp);
  uint32_t above = 0u, ties = 0u;
  for (int j0 = run0; j0 < run1; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < run1, sure = in && (j < lo || j >= hi);
    const uint32_t k = in ? key_at(j) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, sure || (in && k > border)));
    ties += __popc(__ballot_sync(0xffffffffu, in && !sure && k == border));
  }
  if (lane == 0) sh.above[warp] = above, sh.ties[warp] = ties;
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0u, t = 0u;
    for (int x = 0; x < EV_WARPS; ++x) {
      const uint32_t a1 = sh.above[x], t1 = sh.ties[x];
      sh.above[x] = a, sh.ties[x] = t;
      a += a1, t += t1;
    }
    sh.totals[0] = a, sh.totals[1] = t;
  }
  cluster.sync();
  uint32_t at = sh.above[warp], tie = sh.ties[warp];
  for (int r = 0; r < rank; ++r) {
    const uint32_t* t = cluster.map_shared_rank(sh.totals, r);
    at += t[0], tie += t[1];
  }
  for (int j0 = run0; j0 < run1; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < run1, sure = in && (j < lo || j >= hi);
    const uint32_t k = in ? key_at(j) : 0u;
    const unsigned a = __ballot_sync(0xffffffffu, sure || (in && k > border));
    const unsigned t = __ballot_sync(0xffffffffu, in && !sure && k == border);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t my_ties = tie + __popc(t & below);
    const bool stays = ((a >> lane) & 1u) || (((t >> lane) & 1u) && my_ties < want);
    if (stays) {
      const uint32_t i = at + __popc(a & below) + min(my_ties, want);
      kept[i] = j;
      nw[i] = __ldg(w + j);
    }
    at += __popc(a);
    tie += __popc(t);
  }
  cluster.sync();  // the totals are read before a block leaves
}

// ---- the move
template <int D, int KIND>
__global__ void __launch_bounds__(EV_MOVE_THREADS) fa_evict_move_kernel(const EvictPagedParams p) {
  constexpr int RB = paged_row_bytes(KIND, D), CR = RB / 16, SB = D / 16;
  __shared__ long long s_src[EV_ROWS], s_dst[EV_ROWS];  // rows in the pool, or -1
  __shared__ float s_scale[2][EV_ROWS];                  // e4m3: old scales of the rows
  __shared__ unsigned int s_most[2][EV_ROWS / 16];       // and the largest of each new page
  const int tid = threadIdx.x;
  const int parts = (p.keep + EV_ROWS - 1) / EV_ROWS;
  const int part = static_cast<int>(blockIdx.x % parts), pair = static_cast<int>(blockIdx.x / parts);
  const int b = pair / p.Hkv, hk = pair % p.Hkv;
  const int row0 = part * EV_ROWS;
  const int n_new = min(paged_clip_len(__ldg(p.seqlens + b), p.max_len), p.keep);
  const int rows = min(EV_ROWS, n_new - row0);
  if (KIND == PAGES_E4M3 && tid < 2 * (EV_ROWS / 16)) s_most[tid / (EV_ROWS / 16)][tid % (EV_ROWS / 16)] = 0u;
  if (rows > 0 && tid < rows) {  // where the row goes does not depend on the selection
    const int i = row0 + tid;
    const int id = __ldg(p.new_table + b * p.new_table_stride + (i >> p.page_shift));
    s_dst[tid] = paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, i & (p.page - 1), 1);
  }
  __syncthreads();
  pdl_wait();
  if (rows <= 0) return;
  bool bad = false;
  if (tid < rows) {
    const int j = __ldcg(p.kept + static_cast<long long>(pair) * p.keep + row0 + tid);
    const int id = __ldg(p.table + b * p.table_stride + (j >> p.page_shift));
    const long long src = paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, j & (p.page - 1), 1);
    bad = src < 0 || s_dst[tid] < 0;
    s_src[tid] = bad ? -1 : src;
    if constexpr (KIND == PAGES_E4M3) {
      if (!bad) {
        const int at = ((row0 + tid) >> p.page_shift) - (row0 >> p.page_shift);
        const long long ph = static_cast<long long>(id) * p.Hkv + hk;
        const float ks = static_cast<const float*>(p.k_scale)[ph], vs = static_cast<const float*>(p.v_scale)[ph];
        s_scale[0][tid] = ks, s_scale[1][tid] = vs;
        // positive factors order as integers
        if (ks > 0.f) atomicMax(&s_most[0][at], __float_as_uint(ks));
        if (vs > 0.f) atomicMax(&s_most[1][at], __float_as_uint(vs));
      }
    }
  }
  if (bad) atomicOr(p.status, FA_DEV_BAD_PAGE);
  __syncthreads();
  uint8_t* kp = static_cast<uint8_t*>(const_cast<void*>(p.k));
  uint8_t* vp = static_cast<uint8_t*>(const_cast<void*>(p.v));
  if constexpr (KIND == PAGES_E4M3) {
    // (a page's first new row writes its scales; rows of a page are all in this block)
    if (tid < rows && s_src[tid] >= 0) {
      const int at = ((row0 + tid) >> p.page_shift) - (row0 >> p.page_shift);
      const long long ph = s_dst[tid] >> p.page_shift;
      static_cast<float*>(const_cast<void*>(p.k_scale))[ph] = __uint_as_float(s_most[0][at]);
      static_cast<float*>(const_cast<void*>(p.v_scale))[ph] = __uint_as_float(s_most[1][at]);
    }
  }
  constexpr int FLIGHT = 4;
  const int items = rows * CR * 2;  // pieces of K, then of V
  for (int x0 = tid; x0 < items; x0 += FLIGHT * EV_MOVE_THREADS) {
    uint4 y[FLIGHT];
    long long to[FLIGHT];
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
      const int x = x0 + i * EV_MOVE_THREADS;
      const bool is_v = x >= items / 2;
      const int r = (is_v ? x - items / 2 : x) / CR, c = x % CR;
      to[i] = -1;
      if (x < items && s_src[r] >= 0) {
        y[i] = *reinterpret_cast<const uint4*>((is_v ? vp : kp) + s_src[r] * RB + c * 16);
        to[i] = s_dst[r] * RB + c * 16;
      }
    }
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
      if (to[i] < 0) continue;
      const int x = x0 + i * EV_MOVE_THREADS;
      const bool is_v = x >= items / 2;
      if constexpr (KIND == PAGES_E4M3) {
        const int r = (is_v ? x - items / 2 : x) / CR;
        const float old = s_scale[is_v][r];
        const float now = __uint_as_float(s_most[is_v][((row0 + r) >> p.page_shift) - (row0 >> p.page_shift)]);
        if (old != now) {  // (a ratio of powers of two is exact; NaN codes stay NaN)
          const float f = old / now;
          uint32_t* w[4] = {&y[i].x, &y[i].y, &y[i].z, &y[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h0, h1;
            e4m3x4_to_f16x2x2(*w[e], h0, h1);
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
            const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h1));
            *w[e] = pack_e4m3x4(a.x * f, a.y * f, c.x * f, c.y * f);
          }
        }
      }
      *reinterpret_cast<uint4*>((is_v ? vp : kp) + to[i]) = y[i];
    }
  }
  if constexpr (KIND == PAGES_FP4) {  // the rows' scale bytes: 8 or 4, a word at a time
    const int words = SB / 4;
    for (int x = tid; x < rows * words * 2; x += EV_MOVE_THREADS) {
      const bool is_v = x >= rows * words;
      const int y = is_v ? x - rows * words : x, r = y / words, c = y % words;
      if (s_src[r] < 0) continue;
      uint8_t* s = static_cast<uint8_t*>(const_cast<void*>(is_v ? p.v_scale : p.k_scale));
      *reinterpret_cast<uint32_t*>(s + s_dst[r] * SB + 4 * c) = *reinterpret_cast<const uint32_t*>(s + s_src[r] * SB + 4 * c);
    }
  }
}

cudaError_t evict_paged_set_attributes() {
  return cudaFuncSetAttribute(fa_evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_HELD * 4);
}

template <int D>
static cudaError_t ev_move(int kind, const cudaLaunchConfig_t& cfg, const EvictPagedParams& p) {
  if (kind == PAGES_FP4) return cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_FP4>, p);
  return kind == PAGES_E4M3 ? cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_E4M3>, p)
                            : cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_BF16>, p);
}

cudaError_t launch_evict_paged(int d, int kind, const EvictPagedParams& p, int num_sms, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(p.B) * p.Hkv;
  // Blocks of a cluster: more while a block would have over 4096 rows and the GPU has SMs left.
  int ranks = 1;
  while (ranks < EV_MAX_CLUSTER && p.max_len > 4096LL * ranks && pairs * ranks * 2 <= 2LL * num_sms) ranks *= 2;
  const int per_warp = ((p.max_len + ranks * EV_WARPS - 1) / (ranks * EV_WARPS) + 31) / 32 * 32;
  const bool held = per_warp * EV_WARPS <= EV_HELD;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * ranks));
  cfg.blockDim = dim3(EV_THREADS);
  cfg.dynamicSmemBytes = held ? per_warp * EV_WARPS * 4 : 0;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = held ? cudaLaunchKernelEx(&cfg, fa_evict_select_kernel<true>, p)
                             : cudaLaunchKernelEx(&cfg, fa_evict_select_kernel<false>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mv{};
  mv.gridDim = dim3(static_cast<unsigned>(pairs * ((p.keep + EV_ROWS - 1) / EV_ROWS)));
  mv.blockDim = dim3(EV_MOVE_THREADS);
  mv.stream = stream;
  cudaLaunchAttribute pd{};
  pd.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pd.val.programmaticStreamSerializationAllowed = 1;
  mv.attrs = &pd;
  mv.numAttrs = 1;
  return d == 64 ? ev_move<64>(kind, mv, p) : ev_move<128>(kind, mv, p);
}

}  // namespace fa
