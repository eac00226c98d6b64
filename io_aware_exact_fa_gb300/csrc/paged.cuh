// Paged K/V caches: the parts the append and decode kernels and the host side
// of the C ABI share.
//
// A pool holds num_pages pages of `page` rows for each K/V head, contiguous as
// [num_pages, Hkv, page, d]; row b of the block table lists the pages of
// sequence b in order, so position p of it lives in row p % page of page
// table[b][p / page]. Pages have 16, 32, 64 or 128 rows: a run of 16 positions
// that starts at a multiple of 16 lies within one page.
#pragma once

#include "fa_common.cuh"

namespace fa {

constexpr unsigned int FA_DEV_BAD_PAGE = 2u;  // status word: a block-table entry outside the pool was skipped
constexpr unsigned int FA_DEV_BAD_LENS = 4u;  // status word: lengths or offsets outside their arrays were clipped

constexpr int PAGED_SCALE_EXP_MIN = -40;      // least exponent of an e4m3 page's scale

inline bool paged_page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// A sequence's length, clipped to the `most` keys the call covers.
__host__ __device__ __forceinline__ int paged_clip_len(int len, int most) {
  return len < 0 ? 0 : (len > most ? most : len);
}

// Element offset of row `row` (0 .. page - 1) of page `id` of K/V head `hk`, or
// -1 when the table entry does not name a page of the pool. 64-bit: a pool may
// hold more than 2^31 elements.
__host__ __device__ __forceinline__ long long paged_row_offset(int id, int num_pages, int Hkv, int hk, int page,
                                                               int row, int d) {
  if (static_cast<unsigned int>(id) >= static_cast<unsigned int>(num_pages)) return -1;
  return ((static_cast<long long>(id) * Hkv + hk) * page + row) * d;
}

struct DecodePagedParams {
  const void* q;             // bf16, element strides qsb / qsh / qst of batch, head, token; d contiguous
  const void* k;             // pool of K pages: bf16 or e4m3 codes
  const void* v;             // pool of V pages
  const float* k_scale;      // e4m3: fp32 [num_pages, Hkv]
  const float* v_scale;
  const int* table;          // int32 [B, >= max_len / page], row stride table_stride
  const int* seqlens;        // int32 [B]
  void* o;                   // bf16, element strides osb / osh / ost
  float* lse;                // fp32 [B, H, Nq] or nullptr
  float* ws_o;               // fp32 [n_ranges + B * Hkv, row_tiles, rows, d] unnormalised parts of outputs
  float* ws_ml;              // fp32 [n_ranges + B * Hkv, row_tiles, rows, 2] their (base in log2 units, sum)
  int* ws_ends;              // int32 [B * Hkv, 2] first and last range that holds keys of a (sequence, K/V head)
  long long qsb, qsh, qst, osb, osh, ost, table_stride;
  int B, H, Hkv, G, Nq, R;   // R = G * Nq query rows per K/V head
  int max_len;               // lengths are clipped to this; at most width * page
  int page, page_shift, num_pages;
  int n_ranges;              // the batch's keys are shared out in at most so many ranges
  int row_tiles;             // tiles of 8 or 16 query rows per K/V head
  float scale_log2;          // scale * log2(e)
  unsigned int* status;      // device status word
};

// Query rows of one warp of the paged decode: 8 where a K/V head has that few, else 16. (Four rows in a warp of 16: 129
// against 124 us for 64 sequences of 4-8k, e4m3; sixteen rows in two warps of 8, which read the keys twice: 67 against 62
// us for 48 sequences, bf16, d = 64.)
__host__ __device__ constexpr int decode_paged_rows(int R) { return R <= 8 ? 8 : 16; }
// Blocks of four such warps that an SM holds: three, but two at 16 rows of d = 128 (48 sequences, 4 tokens of 32/8 heads:
// bf16 115 against 117 us; e4m3 76 against 97 us, where the 168 registers a thread of three blocks spill; at d = 64 two
// blocks take 53 us, three 47).
__host__ __device__ constexpr int decode_paged_ctas(int d, int rows) { return rows == 16 && d == 128 ? 2 : 3; }
__host__ __device__ constexpr int decode_paged_row_tiles(int R) { return (R + decode_paged_rows(R) - 1) / decode_paged_rows(R); }
// Ranges that the batch's keys are shared out in: one for each warp that `sms` SMs hold (and row tile), or `num_splits`
// for each sequence and K/V head on average. More ranges than warps would run as a second wave, as long as the first.
constexpr int DECODE_PAGED_SMS = 152;  // a GB300's; a larger device works with so many of its own
inline int decode_paged_ranges(int sms, int B, int Hkv, int R, int d, int num_splits) {
  if (num_splits > 0) {
    const long long n = static_cast<long long>(num_splits) * B * Hkv;
    return n < (1 << 20) ? static_cast<int>(n) : 1 << 20;
  }
  const int warps = (sms < DECODE_PAGED_SMS ? sms : DECODE_PAGED_SMS) * 4 * decode_paged_ctas(d, decode_paged_rows(R));
  const int n = warps / decode_paged_row_tiles(R);
  return n < 1 ? 1 : n;
}

struct AppendPagedParams {
  const void* q;             // bf16, element strides of token and head; d contiguous
  const void* k;
  const void* v;
  void* q_out;               // bf16, its own strides; may be q itself
  void* k_out;               // bf16 or nullptr; may be k itself
  void* k_pages;             // bf16, or e4m3 codes with the scales below
  void* v_pages;
  float* k_scale;
  float* v_scale;
  const int* table;
  const int* seqlens;        // int32 [B]: lengths with the new tokens counted
  const int* cu;             // int32 [B + 1]: first new token of each sequence, or nullptr (uniform)
  const long long* turns;    // int64 [rot / 2]: each pair's frequency in 2^-64 turns a position
  const void* q_weight;      // bf16 [d] or nullptr
  const void* k_weight;
  long long qst, qsh, kst, ksh, vst, vsh, qost, qosh, kost, kosh, table_stride;
  int B, T, H, Hkv, G, d;
  int width, page, page_shift, num_pages;
  int rot, interleaved;
  int max_new;               // most new tokens of one sequence
  int per_seq;               // > 0: K/V blocks are B x per_seq pages; 0: found through cu
  int kv_blocks;             // K/V blocks (pages x K/V heads), spread evenly among the query blocks
  int max_rows;              // most new rows of one page
  int q_blocks_wanted;       // query blocks that fill the GPU a few times over
  int q_slots;               // heads of a row that a query block takes side by side
  float rot_scale, eps;
  unsigned int* status;
};

cudaError_t append_paged_set_attributes();
cudaError_t launch_append_paged(bool f8, const AppendPagedParams& p, cudaStream_t stream);

cudaError_t decode_paged_set_attributes();
cudaError_t launch_decode_paged(int d, bool f8, const DecodePagedParams& p, cudaStream_t stream);

}  // namespace fa
