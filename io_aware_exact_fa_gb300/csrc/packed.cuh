// Packed prefill: what the unit list, the prefill kernel and the host share.
#pragma once

#include "fa_common.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

// Rows of one entry of the unit list: one Q tile (for a pair of heads) where the
// query heads of a K/V head pair up, else two.
__host__ __device__ constexpr int packed_block_rows(bool pair_heads) { return pair_heads ? BLOCK_M : 2 * BLOCK_M; }

struct PackedArgs {
  const int4* entries;       // two per row block: {q_off, k_off, Lq, Lk}, {first row, 0, 0, 0}
  const int* n_entries;
  int head_units;            // units of one row block: H / 2 pairs of heads, or H heads
  int pair_heads;
  int G, Hkv;                // query heads per K/V head, K/V heads
  int total_q, total_k;      // rows of q and of k, v
  long long ost, osh;        // element strides of o: row and head
};

struct PackedPlan {
  const int* cu_q;           // int32 [B + 1]
  const int* cu_k;
  int4* entries;
  int* n_entries;
  int B, total_q, total_k, block_rows, causal, max_entries;
  int shift;                 // key tiles are counted in steps of 2^shift
  unsigned int* status;
};

cudaError_t packed_set_attributes();
int packed_num_regs(int d);
cudaError_t launch_packed(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& to, const PrefillParams& p, const PackedArgs& pk, const PackedPlan& plan,
                          cudaStream_t stream);

}  // namespace fa
