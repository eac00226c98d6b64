// Eviction from a paged K/V cache by accumulated attention weight, for sm_103a.
//
// Of the L rows of a sequence every K/V head keeps its first `first` and last
// `recent`, and of those between the keep - first - recent with the largest weights
// (ties to the lowest index; NaN counts as -inf); a sequence of at most `keep` rows
// keeps all. The rows that stay are moved, in order, to the pages of a new table.
//
// Two launches. (1) Selection. A weight's bits, flipped so that they order as
// unsigned integers, are compared digit by digit: the rows between are counted by
// their top 11 bits; those that share the border's digit, a few in a hundred, go on
// a list, which the next 11 and the last 10 bits are counted on; after that the
// border value and how many of its ties stay are known, exactly. (With four digits of
// 8 bits counted over all rows the instructions for each weight were the bound: 42 us
// in place of 21 for 32 sequences of 8-16k and 8 K/V heads.) A cluster of blocks shares
// one (sequence, K/V head): each holds a contiguous part of its weights in shared memory
// (so they are read once), and the counts are summed over the cluster's shared memories.
// Then every warp counts its contiguous run, and with the runs' sums before it writes
// indices and weights in order. (2) The move: a warp takes 16 new rows of one
// head, which lie in one page, and copies their keys and values, 16 bytes (4-bit
// rows: also the scale bytes) a lane; no warp waits for another. A new e4m3 page's
// scale is the largest of its rows' old ones, which each warp of the page finds for
// itself, and codes whose scale grew are rounded again. (Those 32 sequences, 4001 rows
// kept, e4m3, take 110 us in all; 2 of 90-131k, 32768 rows kept and read back, 4-bit, 119.
// While launched beside the selection's tail 135 and 123; then, with 32 rows a warp, 106
// registers, 162 and 126; with blocks of 128 rows that meet at barriers 130 and 127.)
// What bounds it: HBM, the weights read and the kept rows read and written; for one
// or two sequences the selection's chain of passes.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace cg = cooperative_groups;

namespace fa {

namespace {

constexpr int EV_MAX_WARPS = 32;
constexpr int EV_BINS = 2048;     // of a digit of eleven bits
constexpr int EV_COPIES = 4;      // of the first digit's counters
constexpr int EV_LIST = 4096;     // rows of the border's first digit that a block's warps list, at most
constexpr int EV_MAX_CLUSTER = 8;
constexpr int EV_HELD = 40960;    // keys that a block holds in shared memory, at most
constexpr int EV_FLIGHT = 8;      // weights that a thread asks for at once
constexpr int EV_MOVE_WARPS = 8;
constexpr size_t EV_BESIDE = 96 * 1024;  // shared memory of the selection on an SM up to which the move is set up beside it
constexpr unsigned ALL = 0xffffffffu;

// Bits that order weights downwards: larger ones have smaller keys, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(fmaxf(w + 0.f, -INFINITY));
  return u ^ (~static_cast<uint32_t>(static_cast<int>(u) >> 31) & 0x7fffffffu);
}
__device__ __forceinline__ float weight_of(uint32_t key) {
  return __uint_as_float(key ^ (~static_cast<uint32_t>(static_cast<int>(key) >> 31) & 0x7fffffffu));
}

struct alignas(16) EvShared {  // (the keys that a block holds lie behind it, and are read four at a time)
  union {
    uint32_t hist[EV_BINS][EV_COPIES];  // counts of the first digit
    struct {
      uint32_t digit2[EV_BINS], digit3[EV_BINS / 2];  // of the other two
      uint32_t list[EV_LIST];                         // keys that share the border's first digit, of each warp's run
    };
  };
  uint32_t digit1[EV_BINS];            // the first digit's counts, summed
  uint32_t all[EV_BINS];               // a digit's counts of the whole cluster
  uint32_t part[EV_MAX_WARPS];         // scans
  uint32_t above[EV_MAX_WARPS], ties[EV_MAX_WARPS], listed[EV_MAX_WARPS];  // of each warp's run
  uint32_t digit, left;                // the border's digit, and how many of its rows stay
  uint2 totals;                        // kept and tied rows of this block
};
static_assert(sizeof(EvShared) % 16 == 0, "the keys behind it are 16-byte aligned");

// Sum over the lanes before this one.
__device__ __forceinline__ uint32_t before_in_warp(uint32_t x, int lane) {
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(ALL, inc, o);
    if (lane >= o) inc += y;
  }
  return inc - x;
}

}  // namespace

// HELD: the keys of a block's rows fit its shared memory; else they are read again for every pass.
template <bool HELD, int EV_THREADS>
__global__ void __launch_bounds__(EV_THREADS, 1024 / EV_THREADS) fa_evict_select_kernel(const EvictPagedParams p) {
  constexpr int EV_WARPS = EV_THREADS / 32, LIST = EV_LIST / EV_WARPS;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  extern __shared__ __align__(16) uint8_t ev_smem[];
  EvShared& sh = *reinterpret_cast<EvShared*>(ev_smem);
  uint32_t* held = reinterpret_cast<uint32_t*>(ev_smem + sizeof(EvShared));
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
  const int step = ranks * EV_THREADS, own = rank * EV_THREADS + tid;
  // rows that are kept without a look: all, or the first and the most recent; and what lies past the rows that stay
  const int lo = L <= keep ? L : p.first, hi = L - p.recent;
  auto edges = [&]() {
    for (int i = own; i < lo; i += step) {
      kept[i] = i;
      nw[i] = __ldg(w + i);
    }
    if (L > keep)
      for (int i = own; i < p.recent; i += step) {
        kept[keep - p.recent + i] = hi + i;
        nw[keep - p.recent + i] = __ldg(w + hi + i);
      }
    for (int i = n_new + own; i < p.new_width; i += step) {
      if (i < keep) kept[i] = -1;
      nw[i] = 0.f;
    }
  };
  uint32_t want = static_cast<uint32_t>(keep - p.first - p.recent);  // of the rows between stay
  if (L <= keep || want == 0u) {  // (the same for the whole cluster)
    edges();
    return;
  }
  // ---- this block's part of the rows between, in runs of a multiple of 32 for each warp, counted from row lo
  const float* between = w + lo;
  const int n = hi - lo;
  const int per_warp = ((n + ranks * EV_WARPS - 1) / (ranks * EV_WARPS) + 31) / 32 * 32;
  const int part0 = min(static_cast<long long>(n), static_cast<long long>(rank) * per_warp * EV_WARPS);
  const int part1 = min(static_cast<long long>(n), static_cast<long long>(rank + 1) * per_warp * EV_WARPS);
  uint32_t border = 0u;                                 // the key of the last row that stays, and how many of its ties do
  auto key_at = [&](int j) { return HELD ? held[j - part0] : order_key(__ldg(between + j)); };
  auto sync_all = [&]() {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  // the digit of the border among counts that all blocks of the cluster made (in BINS bins; the counts stay as they are)
  auto find = [&](const uint32_t* counts, auto bins) {
    constexpr int BINS = decltype(bins)::value, PER = BINS / EV_THREADS;  // neighbouring bins of a thread: 4, 2 or 1
    sync_all();
    if (ranks > 1) {  // every block sums its share of the bins over the cluster, and gives all blocks the sums
      const int share = BINS / ranks;
      for (int i = rank * share + tid; i < (rank + 1) * share; i += EV_THREADS) {
        uint32_t x[EV_MAX_CLUSTER], y = 0u;
#pragma unroll
        for (int r = 0; r < EV_MAX_CLUSTER; ++r) x[r] = cluster.map_shared_rank(counts, r & (ranks - 1))[i];
#pragma unroll
        for (int r = 0; r < EV_MAX_CLUSTER; ++r) y += r < ranks ? x[r] : 0u;
#pragma unroll
        for (int r = 0; r < EV_MAX_CLUSTER; ++r)
          if (r < ranks) cluster.map_shared_rank(sh.all, r)[i] = y;
      }
      cluster.sync();
      counts = sh.all;
    }
    uint32_t n[PER], sum = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) n[i] = counts[tid * PER + i];
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += n[i];
    const uint32_t mine = __reduce_add_sync(ALL, sum);
    if (lane == 0) sh.part[warp] = mine;
    __syncthreads();
    uint32_t before = __reduce_add_sync(ALL, lane < warp ? sh.part[lane] : 0u);
    if (before < want && want <= before + mine) {  // the border is one of this warp's bins
      before += before_in_warp(sum, lane);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < want && want <= before + n[i]) {
          sh.digit = PER * tid + i;
          sh.left = want - before;
        }
        before += n[i];
      }
    }
    __syncthreads();
    want = sh.left;
    return sh.digit;
  };
  // ---- the first digit; the weights are read
  for (int i = tid; i < EV_BINS * EV_COPIES / 4; i += EV_THREADS)
    reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  {
    uint32_t* mine = &sh.hist[0][lane % EV_COPIES];
    int j = part0 + tid;
    for (; j + (EV_FLIGHT - 1) * EV_THREADS < part1; j += EV_FLIGHT * EV_THREADS) {
      float x[EV_FLIGHT];
#pragma unroll
      for (int f = 0; f < EV_FLIGHT; ++f) x[f] = __ldg(between + j + f * EV_THREADS);
#pragma unroll
      for (int f = 0; f < EV_FLIGHT; ++f) {
        const uint32_t k = order_key(x[f]);
        if (HELD) held[j + f * EV_THREADS - part0] = k;
        atomicAdd(mine + (k >> 21) * EV_COPIES, 1u);
      }
    }
#pragma unroll 4
    for (; j < part1; j += EV_THREADS) {
      const uint32_t k = order_key(__ldg(between + j));
      if (HELD) held[j - part0] = k;
      atomicAdd(mine + (k >> 21) * EV_COPIES, 1u);
    }
  }
  __syncthreads();
  const int run0 = min(part1, part0 + warp * per_warp), run1 = min(part1, run0 + per_warp);
  // keys of rows j .. j + 3 of the warp's run (j - run0 a multiple of four); past its end the key of no weight
  auto four = [&](int j, uint32_t (&k)[4]) {
    if (HELD) {  // (the memory does not end inside a four)
      const uint4 y = *reinterpret_cast<const uint4*>(held + (j - part0));
      k[0] = y.x, k[1] = y.y, k[2] = y.z, k[3] = y.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e >= run1) k[e] = 0xffffffffu;
      else if (!HELD) k[e] = order_key(__ldg(between + j + e));
  };
  if (lane == 0) sh.listed[warp] = 0u;
  for (int i = tid; i < EV_BINS; i += EV_THREADS) {
    const uint4 c = *reinterpret_cast<const uint4*>(sh.hist[i]);
    sh.digit1[i] = c.x + c.y + c.z + c.w;
  }
  __syncthreads();
  for (int i = tid; i < EV_BINS; i += EV_THREADS) sh.digit2[i] = 0u;
  for (int i = tid; i < EV_BINS / 2; i += EV_THREADS) sh.digit3[i] = 0u;
  const uint32_t top = find(sh.digit1, std::integral_constant<int, EV_BINS>{});
  border = top << 21;
  // ---- the keys of that digit go on the warp's list; those above are counted
  uint32_t above = 0u, ties = 0u;
#pragma unroll 2
  for (int j = run0 + 4 * lane; j < run1; j += 128) {
    uint32_t k[4], here = 0u;
    four(j, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      above += k[e] < border;
      here += k[e] >> 21 == top;
    }
    if (here != 0u) {
      uint32_t i = atomicAdd(&sh.listed[warp], here);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k[e] >> 21 == top) {
          if (i < LIST) sh.list[warp * LIST + i] = k[e];
          ++i;
        }
    }
  }
  __syncwarp();
  const uint32_t listed = sh.listed[warp];
  // Every key of that digit in the warp's run. The digit has four bins an octave and a list 128 or 256 keys, so weights within
  // an octave or so overflow it, and the run is looked through again in each of the three steps left: 7 us more (2
  // sequences of 110k, 32768 kept, all weights in one bin: 66 in place of 59 us; 32 of 12k 86 in place of 81).
  auto each = [&](auto&& f) {
    if (listed <= LIST) {
      for (uint32_t i = lane; i < listed; i += 32) f(sh.list[warp * LIST + i]);
    } else {
      for (int j = run0 + lane; j < run1; j += 32) {
        const uint32_t k = key_at(j);
        if (k >> 21 == top) f(k);
      }
    }
  };
  each([&](uint32_t k) { atomicAdd(&sh.digit2[(k >> 10) & 2047u], 1u); });
  border |= find(sh.digit2, std::integral_constant<int, EV_BINS>{}) << 10;
  each([&](uint32_t k) {
    if (k >> 10 == border >> 10) atomicAdd(&sh.digit3[k & 1023u], 1u);
  });
  border |= find(sh.digit3, std::integral_constant<int, EV_BINS / 2>{});
  each([&](uint32_t k) {
    above += k < border;
    ties += k == border;
  });
  above = __reduce_add_sync(ALL, above);
  ties = __reduce_add_sync(ALL, ties);
  if (lane == 0) sh.above[warp] = above, sh.ties[warp] = ties;
  __syncthreads();
  const uint32_t a_of = lane < EV_WARPS ? sh.above[lane] : 0u, t_of = lane < EV_WARPS ? sh.ties[lane] : 0u;
  uint32_t at = lo + __reduce_add_sync(ALL, lane < warp ? a_of : 0u);
  uint32_t tie = __reduce_add_sync(ALL, lane < warp ? t_of : 0u);
  if (ranks > 1) {
    if (warp == 0) {
      const uint32_t all_above = __reduce_add_sync(ALL, a_of), all_ties = __reduce_add_sync(ALL, t_of);
      if (lane == 0) sh.totals = make_uint2(all_above, all_ties);
    }
    cluster.sync();
    const uint2 t = lane < rank ? *cluster.map_shared_rank(&sh.totals, lane) : make_uint2(0u, 0u);
    at += __reduce_add_sync(ALL, t.x);
    tie += __reduce_add_sync(ALL, t.y);
    __syncthreads();
    cluster.barrier_arrive();  // (waited for at the end: the totals are read before a block leaves)
  }
  // ---- indices and weights of the warp's run, in order: 32 rows side by side, those before a lane's own counted by ballots
  const unsigned before_me = (1u << lane) - 1u;
  auto write = [&](uint32_t i, int j, uint32_t k) {
    kept[i] = lo + j;
    nw[i] = weight_of(k);
    // (0 may have been -0, and -inf NaN: rare among the rows that stay)
    if (k == 0x7fffffffu || k == 0xff800000u) nw[i] = __ldg(between + j);
  };
  if (ties == 0u) {  // no row of the run has the border's key (as in most runs; 7,000 cycles of a block in place of 9,500 for 14k rows)
    constexpr int AT_ONCE = 4;
    at += min(tie, want);
    for (int j0 = run0; j0 < run1; j0 += 32 * AT_ONCE) {
      uint32_t k[AT_ONCE], i[AT_ONCE];
#pragma unroll
      for (int e = 0; e < AT_ONCE; ++e) {
        const int j = j0 + 32 * e + lane;
        k[e] = j < run1 ? key_at(j) : 0xffffffffu;  // (the key of no weight)
      }
#pragma unroll
      for (int e = 0; e < AT_ONCE; ++e) {
        const unsigned over = __ballot_sync(ALL, k[e] < border);
        i[e] = at + __popc(over & before_me);
        at += __popc(over);
      }
#pragma unroll
      for (int e = 0; e < AT_ONCE; ++e)
        if (k[e] < border) write(i[e], j0 + 32 * e + lane, k[e]);
    }
  } else {
    for (int j0 = run0; j0 < run1; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t k = j < run1 ? key_at(j) : 0xffffffffu;
      const unsigned over = __ballot_sync(ALL, k < border), tied = __ballot_sync(ALL, k == border);
      const uint32_t my_tie = tie + __popc(tied & before_me);
      if (k < border || (k == border && my_tie < want)) write(at + __popc(over & before_me) + min(my_tie, want), j, k);
      at += __popc(over);
      tie += __popc(tied);
    }
  }
  edges();
  if (ranks > 1) cluster.barrier_wait();
}

// ---- the move: sixteen new rows of one K/V head a warp
template <int D, int KIND>
__global__ void __launch_bounds__(32 * EV_MOVE_WARPS) fa_evict_move_kernel(const EvictPagedParams p) {
  constexpr int RB = paged_row_bytes(KIND, D), CR = RB / 16, SB = D / 16;
  constexpr int RPL = 32 / CR;       // rows of one load of the warp
  constexpr int N = 16 / RPL;        // loads of K, and of V
  const int lane = threadIdx.x & 31;
  const int groups = (p.keep + 15) / 16;
  const long long unit = static_cast<long long>(blockIdx.x) * EV_MOVE_WARPS + (threadIdx.x >> 5);
  const int pair = static_cast<int>(unit / groups), row0 = static_cast<int>(unit % groups) * 16;
  const bool in = pair < p.B * p.Hkv;
  const int b = in ? pair / p.Hkv : 0, hk = pair - b * p.Hkv;
  const int n_new = in ? min(paged_clip_len(__ldg(p.seqlens + b), p.max_len), p.keep) : 0;
  const int rows = min(16, n_new - row0);
  // where the rows go does not depend on the selection: they lie in one page
  long long dst = -1;
  if (rows > 0) {
    const int id = __ldg(p.new_table + b * p.new_table_stride + (row0 >> p.page_shift));
    dst = paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, row0 & (p.page - 1), 1);
  }
  pdl_wait();
  pdl_launch_dependents();  // (as in the append)
  if (rows <= 0) return;
  // (page of the pool, and row there, of new row i: -1 where a table names none)
  auto from = [&](int i, int& id) -> long long {
    const int j = __ldcg(p.kept + static_cast<long long>(pair) * p.keep + i);
    id = __ldg(p.table + b * p.table_stride + (j >> p.page_shift));
    return paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, j & (p.page - 1), 1);
  };
  int my_id = 0;
  long long src = lane < rows ? from(row0 + lane, my_id) : -1;
  if (__any_sync(ALL, lane < rows && (src < 0 || dst < 0)) && lane == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
  if (dst < 0) return;  // (uniform)
  uint8_t* kp = static_cast<uint8_t*>(const_cast<void*>(p.k));
  uint8_t* vp = static_cast<uint8_t*>(const_cast<void*>(p.v));
  // e4m3: the new page's scales are the largest over all of its rows, of which every warp of the page looks at all
  float k_most = 0.f, v_most = 0.f, k_old = 0.f, v_old = 0.f;
  if constexpr (KIND == PAGES_E4M3) {
    float* ks = static_cast<float*>(const_cast<void*>(p.k_scale));
    float* vs = static_cast<float*>(const_cast<void*>(p.v_scale));
    if (src >= 0) {
      k_old = ks[static_cast<long long>(my_id) * p.Hkv + hk];
      v_old = vs[static_cast<long long>(my_id) * p.Hkv + hk];
    }
    const int first = row0 & ~(p.page - 1), end = min(n_new, first + p.page);
    bool any = false;
#pragma unroll 4
    for (int i = first + lane; i < end; i += 32) {
      int id;
      if (from(i, id) >= 0) {
        any = true;
        k_most = fmaxf(k_most, ks[static_cast<long long>(id) * p.Hkv + hk]);
        v_most = fmaxf(v_most, vs[static_cast<long long>(id) * p.Hkv + hk]);
      }
    }
    // positive factors order as integers
    k_most = __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(k_most)));
    v_most = __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(v_most)));
    any = __any_sync(ALL, any);
    if (row0 == first && any && lane == 0) {
      ks[dst >> p.page_shift] = k_most;
      vs[dst >> p.page_shift] = v_most;
    }
    // from here on: what the row's codes are multiplied with (where all scales are 0 all values are, and codes stay)
    k_old = k_most > 0.f ? k_old / k_most : 1.f;
    v_old = v_most > 0.f ? v_old / v_most : 1.f;
  }
  const unsigned live = __ballot_sync(ALL, src >= 0);
  const int piece = lane % CR, lr = lane / CR;
  auto load = [&](const uint8_t* pages, uint4 (&y)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // (a row that is not there: the pool's first, which is not stored)
      const long long at = max(__shfl_sync(ALL, src, i * RPL + lr), 0ll);
      y[i] = *reinterpret_cast<const uint4*>(pages + at * RB + piece * 16);
    }
  };
  auto store = [&](uint8_t* pages, uint4 (&y)[N], [[maybe_unused]] float factor) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * RPL + lr;
      const bool there = (live >> r) & 1u;
      if constexpr (KIND == PAGES_E4M3) {
        // In fp32: exact for powers of two, so the one rounding is that to e4m3; other ratios and products are off by 2^-24 of
        // themselves before it (in f16, by 2^-11 each, 0.4 % of the codes came out as their neighbours). NaN codes stay NaN.
        const float f = __shfl_sync(ALL, factor, r);
        if (there && f != 1.f) {
          const uint64_t f2 = f2pack(f, f);
          uint32_t* w[4] = {&y[i].x, &y[i].y, &y[i].z, &y[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[2];
            e4m3x4_to_f16x2x2(*w[e], h[0], h[1]);
            float z[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[x]));
              f2unpack(fmul2(f2pack(a.x, a.y), f2), z[2 * x], z[2 * x + 1]);
            }
            *w[e] = pack_e4m3x4(z[0], z[1], z[2], z[3]);
          }
        }
      }
      if (there) *reinterpret_cast<uint4*>(pages + (dst + r) * RB + piece * 16) = y[i];
    }
  };
  uint4 yk[N], yv[N];
  load(kp, yk);
  load(vp, yv);
  if constexpr (KIND == PAGES_FP4) {  // the rows' scale bytes, a word a lane
    const int r = lane / (SB / 4), c = lane % (SB / 4);
    const long long at = __shfl_sync(ALL, src, r & 15);
    uint8_t* ks = static_cast<uint8_t*>(const_cast<void*>(p.k_scale));
    uint8_t* vs = static_cast<uint8_t*>(const_cast<void*>(p.v_scale));
    if (r < 16 && at >= 0) {
      const uint32_t x = *reinterpret_cast<const uint32_t*>(ks + at * SB + 4 * c);
      const uint32_t y = *reinterpret_cast<const uint32_t*>(vs + at * SB + 4 * c);
      *reinterpret_cast<uint32_t*>(ks + (dst + r) * SB + 4 * c) = x;
      *reinterpret_cast<uint32_t*>(vs + (dst + r) * SB + 4 * c) = y;
    }
  }
  store(kp, yk, k_old);
  store(vp, yv, v_old);
}

template <int THREADS>
static cudaError_t ev_attrs() {
  const cudaError_t e = cudaFuncSetAttribute(fa_evict_select_kernel<true, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(sizeof(EvShared)) + EV_HELD * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(fa_evict_select_kernel<false, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(EvShared)));
}
cudaError_t evict_paged_set_attributes() {
  const cudaError_t e = ev_attrs<512>();
  return e != cudaSuccess ? e : ev_attrs<1024>();
}

// `smem`: what a block takes of shared memory.
template <int THREADS>
static cudaError_t ev_select(const EvictPagedParams& p, int ranks, size_t& smem, cudaStream_t stream) {
  const int warps = ranks * (THREADS / 32);
  const long long block = ((p.max_len + static_cast<long long>(warps) - 1) / warps + 31) / 32 * THREADS;  // keys of one, at most
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.Hkv * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = smem = sizeof(EvShared);
  if (block > EV_HELD) return cudaLaunchKernelEx(&cfg, fa_evict_select_kernel<false, THREADS>, p);
  cfg.dynamicSmemBytes = smem += block * 4;
  return cudaLaunchKernelEx(&cfg, fa_evict_select_kernel<true, THREADS>, p);
}

template <int D>
static cudaError_t ev_move(int kind, const cudaLaunchConfig_t& cfg, const EvictPagedParams& p) {
  if (kind == PAGES_FP4) return cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_FP4>, p);
  return kind == PAGES_E4M3 ? cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_E4M3>, p)
                            : cudaLaunchKernelEx(&cfg, fa_evict_move_kernel<D, PAGES_BF16>, p);
}

cudaError_t launch_evict_paged(int d, int kind, const EvictPagedParams& p, int num_sms, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(p.B) * p.Hkv;
  // Blocks of a cluster: more while a block would have over 4096 rows and the GPU an SM for each. Large blocks where each
  // has an SM, but not in clusters: eight free SMs next to one another are not found for every one of them then.
  int ranks = 1;
  while (ranks < EV_MAX_CLUSTER && p.max_len > 4096LL * ranks && pairs * ranks * 2 <= num_sms) ranks *= 2;
  size_t smem = 0;
  const cudaError_t e = ranks == 1 && pairs <= num_sms ? ev_select<1024>(p, ranks, smem, stream) : ev_select<512>(p, ranks, smem, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mv{};
  const long long units = pairs * ((p.keep + 15) / 16);
  mv.gridDim = dim3(static_cast<unsigned>((units + EV_MOVE_WARPS - 1) / EV_MOVE_WARPS));
  mv.blockDim = dim3(32 * EV_MOVE_WARPS);
  mv.stream = stream;
  cudaLaunchAttribute pd{};
  pd.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pd.val.programmaticStreamSerializationAllowed = 1;
  mv.attrs = &pd;
  // Set up beside the selection's tail the move starts 1 to 4 us earlier, but keeps the split of the SM's memory that the
  // selection took, for all of its time, and its loads in flight live in what that left to L1. 32 sequences of 8-16k, two
  // blocks of 106 KB an SM: 135 us, on its own 112; 2 of 90-131k, one of 98 KB, 123 and 121 (with the read); one of 100k, 91 KB, 38 and 39; 16
  // of 4k, 57 KB, 26 and 28; 4 of 1.4k 12 and 14.
  const long long on_an_sm = std::min<long long>((pairs * ranks + num_sms - 1) / num_sms, 2);
  mv.numAttrs = on_an_sm * smem < EV_BESIDE ? 1 : 0;
  return d == 64 ? ev_move<64>(kind, mv, p) : ev_move<128>(kind, mv, p);
}

}  // namespace fa
