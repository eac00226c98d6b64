// Tiles of KS keys of a paged batch, laid end to end (sequence by sequence, K/V head
// by K/V head), and how kernels whose warps take equal contiguous ranges of them
// find their way. All lanes of a warp call together.
#pragma once

#include "paged.cuh"

namespace fa {

// How the batch's tiles are shared out: range r has tiles begin(r) .. begin(r + 1) - 1, none of them empty.
struct PagedRanges {
  long long tiles, n;  // all tiles; ranges
  __device__ __forceinline__ PagedRanges(long long tiles_, int most) : tiles(tiles_), n(most < tiles_ ? most : tiles_) {}
  __device__ __forceinline__ long long begin(long long r) const { return r * tiles / n; }
};

// A tile: sequence, K/V head, tile among theirs; the sequence's length and tiles.
struct PagedTile {
  int b, hk, i, L, nt;
};

// A sequence's tiles for one K/V head. EXTRA: what starting on them costs, in tiles, counted before the first one, so that
// ranges with many short sequences take no longer than others.
template <int KS, int EXTRA = 0>
__device__ __forceinline__ int paged_tiles_of(int L) {
  return L > 0 ? (L + KS - 1) / KS + EXTRA : 0;
}

// Tiles of one K/V head of all sequences; `clipped`: a length outside [0, most] was met.
template <int KS, int EXTRA = 0>
__device__ __forceinline__ long long paged_count_tiles(const int* seqlens, int B, int most, int lane, bool& clipped) {
  long long sum = 0;
#pragma unroll 4
  for (int b = lane; b < B; b += 32) {
    const int raw = __ldg(seqlens + b), L = paged_clip_len(raw, most);
    clipped = clipped || L != raw;
    sum += paged_tiles_of<KS, EXTRA>(L);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Tile t0 of all.
template <int KS, int EXTRA = 0>
__device__ __forceinline__ PagedTile paged_seek(const int* seqlens, int B, int Hkv, int most, long long t0, int lane) {
  constexpr unsigned ALL = 0xffffffffu;
  PagedTile t{};
  long long base = 0;  // tiles of one K/V head of the sequences before
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int mine = b0 + lane < B ? paged_clip_len(__ldg(seqlens + b0 + lane), most) : 0;
    const int n = paged_tiles_of<KS, EXTRA>(mine);
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(ALL, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned past = __ballot_sync(ALL, (base + inc) * Hkv > t0);
    if (past != 0u) {
      const int at = __ffs(past) - 1;
      t.b = b0 + at;
      t.L = __shfl_sync(ALL, mine, at);
      t.nt = __shfl_sync(ALL, n, at);
      const long long rest = t0 - (base + __shfl_sync(ALL, inc, at) - t.nt) * Hkv;
      t.hk = static_cast<int>(rest / t.nt);
      t.i = static_cast<int>(rest % t.nt);
      break;
    }
    base += __shfl_sync(ALL, inc, 31);
  }
  return t;
}

// The next tile; past the last one b is B.
template <int KS, int EXTRA = 0>
__device__ __forceinline__ void paged_next(PagedTile& t, const int* seqlens, int B, int Hkv, int most) {
  if (++t.i < t.nt) return;
  t.i = 0;
  if (++t.hk < Hkv) return;
  t.hk = 0;
  do {
    if (++t.b >= B) return;
    t.L = paged_clip_len(__ldg(seqlens + t.b), most);
    t.nt = paged_tiles_of<KS, EXTRA>(t.L);
  } while (t.nt == 0);
}

}  // namespace fa
