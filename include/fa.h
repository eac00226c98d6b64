/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention library libfa_gb300.so.
 *
 * The operation (all entry points): for every batch b, head h and query row i
 *
 *     s_ij  = scale * <q_i, k_j>                       (scaled scores)
 *     allowed(i, j) = (!causal || j <= i + (Nk - Nq)) && keep(b, h, i, j)
 *     O_i   = sum_j softmax_j(s_ij over allowed j) * v_j
 *     lse_i = ln sum_{allowed j} exp(s_ij)
 *
 * "Flash Attention Optimization", section "Attention is not slow because of
 * arithmetic" (S = Q K^T / sqrt(d), P = softmax(S), O = P V); "Explain
 * FlashAttention. Why is it called IO-aware, and what does it actually
 * save?", section "Keep only the state needed for the final weighted average"
 * (scores plus the intended mask or bias; the causal mask uses absolute query
 * and key positions). A row with no allowed key returns O = 0 and
 * lse = -inf (the explicit empty-row policy of the section "Executable
 * recurrence, with an empty-state policy"). lse is the per-row statistic a
 * backward pass recomputes P from ("Flash Attention Optimization", section
 * "Sizing a tile, and why the backward pass recomputes instead of storing").
 * Causal alignment for Nq != Nk is bottom-right (query i sees keys
 * j <= i + Nk - Nq), the reading the library takes where the pages are silent.
 *
 * Layout (all device pointers, row-major, contiguous):
 *   q, o      bf16 [B, H, Nq, d]        k, v   bf16 [B, H, Nk, d]
 *   lse       fp32 [B, H, Nq]           (may be NULL: not written)
 *   keep_bits uint32 words; bit (j % 32) of word (j / 32) is key j, 1 = attend;
 *             the words of row (b, h, i) start at
 *             b*mstride_b + h*mstride_h + i*mstride_q (strides in words;
 *             mstride_q = 0 broadcasts one key mask over all rows). Each row
 *             holds ceil(Nk / 32) words; bits past Nk are ignored.
 *   stream    a cudaStream_t (NULL = the legacy default stream).
 * Supported: d in {64, 128}; q, k, v, o 16-byte aligned; keep_bits 4-byte
 * aligned; 1 <= B*H, Nk < 2^31; scale any finite value (a negative scale
 * gives the largest weights to the smallest dot products, as the definition
 * says; scale 0 gives uniform weights over the visible keys).
 *
 * Ownership: the caller allocates and owns every buffer; the library keeps
 * no pointer after a call returns and allocates no device memory per call
 * (the decode workspace is the caller's). Calls are asynchronous on `stream`:
 * a return of FA_OK means the work was launched.
 *
 * Errors (checked on the host before anything is launched; nothing is
 * written on error):
 *   FA_ERR_INVALID_ARG  a required pointer is NULL, a size is negative or
 *                       zero where it must be positive, scale is NaN or
 *                       infinite, or a size overflows the supported range.
 *   FA_ERR_UNSUPPORTED  d not in {64, 128}, a misaligned pointer, or no
 *                       sm_103 device is current. There is no fallback path.
 *   FA_ERR_WORKSPACE    the decode workspace is NULL or too small.
 *   FA_ERR_CUDA         a CUDA call failed (fa_last_error_detail() says which).
 *   FA_ERR_TIMEOUT      reported later by fa_get_device_status(): a bounded
 *                       wait inside a kernel gave up; that call's outputs are
 *                       undefined, the CUDA context stays usable.
 * Inputs are not scanned for NaN/inf (that would cost bandwidth): a NaN or
 * inf in q, k or v propagates to the rows it touches.
 *
 * Device reset: the first call on a device caches that device's state (the
 * status word's address, kernel attributes, the no-alloc scratch address)
 * for its primary context. cudaDeviceReset while the library is loaded
 * invalidates that state; calls made after a reset are not supported.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,
  FA_ERR_UNSUPPORTED = 2,
  FA_ERR_CUDA = 3,
  FA_ERR_TIMEOUT = 4,
  FA_ERR_WORKSPACE = 5
} fa_status;

/* Fused, tiled forward pass (prefill). Q tiles stay on chip while K/V tiles
 * stream through; the Nq x Nk score matrix never reaches HBM ("Flash
 * Attention Optimization", section "The fix: tile the computation, never
 * materialize the full matrix"). Nq = 0 is a no-op (q and o may then be NULL). */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int H, int Nq, int Nk, int d, float scale, int causal, void* stream);

/* fa_fwd with an additional key mask (see keep_bits above), ANDed with the
 * causal mask when causal != 0. keep_bits = NULL is the same as fa_fwd. */
fa_status fa_fwd_masked(const void* q, const void* k, const void* v, void* o, float* lse,
                        int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        const uint32_t* keep_bits, int64_t mstride_b, int64_t mstride_h,
                        int64_t mstride_q, void* stream);

/* Bytes of device workspace fa_fwd_packed needs: a list of its row blocks. 0
 * for invalid arguments. */
size_t fa_fwd_packed_workspace_size(int B, int total_q, int H, int Hkv);

/* fa_fwd over packed sequences of different lengths with grouped K/V heads.
 *   q, o   bf16 [total_q, H, d]     k, v   bf16 [total_k, Hkv, d]
 *   cu_seqlens_q, cu_seqlens_k  int32 [B+1] on the device: sequence b owns rows
 *          cu[b] .. cu[b+1]-1 (cu_seqlens_k NULL: those of cu_seqlens_q).
 *          Lengths of zero are fine. Offsets are read on the device when the
 *          call runs, so a captured call follows new ones; decreasing offsets or
 *          offsets past the tensors are clipped and reported by
 *          fa_get_device_status() as FA_ERR_INVALID_ARG.
 *   strides  int64 [8], host memory: row and head strides, in elements, of q, k,
 *          v, o in that order (positive multiples of 8; no two rows of o overlap, as
 *          for fa_append_paged; the d elements of a head are contiguous), so q, k and v can be parts of one projection.
 *   lse    fp32 [H, total_q] (may be NULL)
 * Query head h reads K/V head h / (H/Hkv). Inside a sequence, with causal != 0,
 * query i sees key j iff j <= i + Lk - Lq (its queries are its last positions);
 * rows that see no key get o = 0, lse = -inf, whatever v holds. Sequences never
 * reach one another, whatever the values of their rows; inside one, an infinity or
 * NaN in v reaches every row that sees a key of its 128-key tile, also those whose
 * causal mask hides it.
 * Rows of o and columns of lse past cu_seqlens_q[B] are left as they were.
 *   workspace  device memory of fa_fwd_packed_workspace_size() bytes, 256-byte
 *              aligned, owned by the caller, overwritten; calls that may overlap
 *              on the GPU need their own.
 * total_q = 0 is a no-op. Two launches (the list, the tiles). Errors as for
 * fa_fwd, plus FA_ERR_WORKSPACE, H not a multiple of Hkv, and
 * FA_ERR_UNSUPPORTED for strides that are not positive multiples of 8. */
fa_status fa_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, const int64_t* strides,
                        const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int total_q, int total_k, int H,
                        int Hkv, int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

/* Forward pass on FP8 inputs ("FlashAttention: Attention Is Limited by
 * Memory, Not Math", section "FlashAttention 1, 2 and 3", lists FP8 support
 * among FlashAttention-3's changes; the pages give no further detail).
 *   q, k, v   e4m3 codes (one byte each: 1 sign, 4 exponent bits with bias
 *             7, 3 mantissa bits; no infinities), layouts as for fa_fwd;
 *             16-byte aligned.
 *   descale_q, descale_k, descale_v
 *             one fp32 factor per tensor: the real value of a code c of q is
 *             e4m3(c) * descale_q (likewise k, v); finite and > 0.
 *   o, lse    bf16 O and fp32 lse of exact attention on those real values,
 *             softmax(scale * Q K^T + causal mask) V, as fa_fwd defines them.
 * The score and value products run on the tensor cores in e4m3 with fp32
 * accumulation; P is rounded to e4m3 (round to nearest even) before the P V
 * product, which is this path's main error against the exact result.
 * Supported: d = 64 or 128 (FA_ERR_UNSUPPORTED otherwise); no key mask. Errors as
 * for fa_fwd, plus FA_ERR_INVALID_ARG for a descale that is not finite and
 * positive, or a product scale * descale_q * descale_k that overflows. */
fa_status fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int H, int Nq, int Nk, int d, float scale,
                     float descale_q, float descale_k, float descale_v, int causal, void* stream);

/* Bytes of device workspace fa_fwd_host needs: two buffer sets, each holding
 * q, k, v, o and lse of one chunk of heads (every region rounded up to 256
 * bytes). chunk_heads <= 0 selects the default, ceil(B*H / 2) heads. Returns 0
 * for invalid arguments. */
size_t fa_fwd_host_workspace_size(int B, int H, int Nq, int Nk, int d, int chunk_heads);

/* fa_fwd on HOST buffers: q, k, v, o and lse have the layouts above but live
 * in host memory. The B*H heads (contiguous in that layout) are processed in
 * chunks of chunk_heads. Each chunk's q, k and v are copied into one of two
 * device buffer sets in the workspace, and its forward pass runs there. Its o
 * and lse are then copied back. Upload, compute and read-back of consecutive
 * chunks overlap: they run on library-owned streams (three upload streams,
 * one compute stream per buffer set, one read-back stream), one set of
 * streams per host thread and device. The call is ordered after the work
 * already queued on `stream`, and `stream` waits for the last read-back. The
 * outputs are complete once `stream` has been synchronised; the inputs must
 * stay unchanged until then.
 *
 * Host memory should be page-locked (cudaHostAlloc / cudaHostRegister) for
 * the copies to overlap the kernels. Pageable memory gives the same results
 * with serialised copies.
 *
 * workspace: device memory, 256-byte aligned, at least
 * fa_fwd_host_workspace_size(...) bytes, not used by anything else until
 * `stream` reaches the end of the call. Errors: those of fa_fwd (host
 * pointers need no alignment), and FA_ERR_WORKSPACE for a NULL, short or
 * misaligned workspace. A CUDA failure after some chunks were queued returns
 * FA_ERR_CUDA; `stream` still waits for the queued work, and the outputs are
 * undefined. */
fa_status fa_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse,
                      int B, int H, int Nq, int Nk, int d, float scale, int causal,
                      int chunk_heads, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace fa_decode_splitkv needs: fp32 partial
 * (o[d], m, l) per (b, h, split), i.e. B*H*num_splits*(d + 2)*4 rounded up
 * to 256. Returns 0 for invalid arguments. */
size_t fa_decode_workspace_size(int B, int H, int d, int num_splits);

/* Split-KV decode: one query token per (b, h) against a KV cache of Nk keys
 * ("FlashAttention: Attention Is Limited by Memory, Not Math", section
 * "Where it helps, and where it does not": split the K/V sequence across the
 * GPU, then merge the partial results; the merge re-bases each split to the
 * global max, "Handwritten Notes on Flash Attention", section "Merging two
 * blocks"). Split s covers keys [s*c, min(Nk, (s+1)*c)) with
 * c = ceil(Nk / num_splits); empty splits contribute nothing.
 *   q, o     bf16 [B, H, 1, d]     k_cache, v_cache  bf16 [B, H, Nk, d]
 *   lse      fp32 [B, H] (may be NULL)
 *   workspace  device memory of at least fa_decode_workspace_size() bytes,
 *              256-byte aligned, owned by the caller; its contents on entry
 *              do not matter and are overwritten.
 *   1 <= num_splits <= 1024. Two launches (split, then merge) on `stream`. */
fa_status fa_decode_splitkv(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                            int B, int H, int Nk, int d, float scale, int num_splits,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the static device scratch behind fa_decode_splitkv_noalloc. */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES (20u << 20)

/* Split-KV decode for callers that cannot allocate device memory. (The pages
 * have no counterpart: this is an interface variant, not part of the method.)
 * Some callers only hold the input and output buffers: a plugin or kernel
 * interface that passes no workspace, or a serving loop that must not call
 * cudaMalloc/cudaFree because those calls can synchronise the device or
 * because another allocator owns the device memory. This entry point takes
 * the same arguments as fa_decode_splitkv without the workspace, allocates
 * nothing, and keeps the per-split partial states in one static device array
 * of FA_DECODE_NOALLOC_SCRATCH_BYTES that every GPU loading the library
 * holds until the process exits. It computes exactly what fa_decode_splitkv
 * computes, with the same kernels.
 *   - Requests needing more scratch than that (fa_decode_workspace_size() >
 *     FA_DECODE_NOALLOC_SCRATCH_BYTES) return FA_ERR_WORKSPACE and launch
 *     nothing; use fa_decode_splitkv with a caller workspace instead.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture. The address is cached for the device's
 *     primary context; after cudaDeviceReset it is stale, as is the rest of
 *     the library's per-device state (see "Device reset" above).
 *   - All calls share the one array: calls whose work overlaps on the GPU
 *     (different streams, or host threads without ordering) race and corrupt
 *     each other's results. Calls ordered on one stream are safe; the array
 *     needs no clearing between them because every partial is rewritten. */
fa_status fa_decode_splitkv_noalloc(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                                    int B, int H, int Nk, int d, float scale, int num_splits, void* stream);

/* Bytes of device workspace fa_decode_grouped needs: the split-KV partial
 * states of B*H*Nq query rows, fa_decode_workspace_size(B, H*Nq, d,
 * num_splits). Returns 0 for invalid arguments (including Nq > 128). */
size_t fa_decode_grouped_workspace_size(int B, int H, int Nq, int d, int num_splits);

/* Split-KV decode with grouped K/V heads, several new query tokens per
 * sequence and per-sequence KV lengths (the decode variants next to
 * "FlashAttention: Attention Is Limited by Memory, Not Math", section "Where
 * it helps, and where it does not"; the merge as for fa_decode_splitkv).
 * H query heads share Hkv K/V heads: query head h reads K/V head h / (H/Hkv).
 * Sequence b holds L_b = seqlens_k[b] keys (clamped to [0, Nk]; all Nk when
 * seqlens_k is NULL), and its Nq new tokens are its last Nq positions: token t
 * sees key j iff j < L_b and j <= L_b - Nq + t. A token that sees no key gets
 * o = 0 and lse = -inf. The (H/Hkv)*Nq query rows of one (b, K/V head) read
 * the K/V stream together, so each K/V byte is read once per group: up to four
 * rows on the CUDA cores (packed fp32 products), more in one tensor-core tile.
 *   q, o       bf16 [B, H, Nq, d]      k_cache, v_cache  bf16 [B, Hkv, Nk, d]
 *   seqlens_k  int32 [B] in device memory, or NULL
 *   lse        fp32 [B, H, Nq] (may be NULL)
 *   workspace  device memory of at least fa_decode_grouped_workspace_size()
 *              bytes, 256-byte aligned, owned by the caller; overwritten.
 *   Split s covers keys [s*c, min(L_b, (s+1)*c)), c = ceil(Nk / num_splits)
 *   rounded up to a multiple of 128; 1 <= num_splits <= 1024.
 * Errors: FA_ERR_INVALID_ARG for NULL tensors, sizes < 1, H not a multiple of
 * Hkv or a bad scale; FA_ERR_UNSUPPORTED for d not in {64, 128},
 * (H/Hkv)*Nq > 128 or misaligned pointers; FA_ERR_WORKSPACE. Two launches
 * (grouped split kernel, then merge) on `stream`. */
fa_status fa_decode_grouped(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k, void* o,
                            float* lse, int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int num_splits,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace fa_fwd_materialized needs: the bf16 score /
 * probability matrix [B, H, Nq, Nk], rounded up to 256 bytes. 0 for invalid
 * arguments. */
size_t fa_materialized_workspace_size(int B, int H, int Nq, int Nk);

/* The materialising baseline the IO argument compares against ("Explain
 * FlashAttention ...", section "What the byte arithmetic does and does not
 * say"): S = scale * Q K^T is written to HBM in bf16, read back by a row
 * softmax that writes P (bf16, over S), and P is read again for O = P V.
 * Four N^2-sized transfers of 2-byte values, against the fused fa_fwd's
 * none. It computes the same attention as fa_fwd (without a key mask), with
 * S and P rounded to bf16. The two products are cuBLAS GEMMs (the library
 * opens libcublas.so.13 on first use and keeps one cuBLAS handle per device;
 * calls are serialised inside the library); the softmax is this library's
 * kernel.
 *   q, o      bf16 [B, H, Nq, d]       k, v  bf16 [B, H, Nk, d]
 *   lse       fp32 [B, H, Nq] (natural log; may be NULL)
 *   workspace device memory of at least fa_materialized_workspace_size()
 *             bytes, 256-byte aligned, owned by the caller; overwritten.
 * Errors: as for fa_fwd, plus FA_ERR_UNSUPPORTED when Nk is not a multiple of
 * 8 or exceeds the row held in one CTA's shared memory (about 58k keys), or
 * when cuBLAS cannot be loaded; FA_ERR_WORKSPACE. */
fa_status fa_fwd_materialized(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                              int Nk, int d, float scale, int causal, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Bytes of device workspace fa_bwd needs: an fp32 dQ accumulator of
 * B*H*ceil(Nq/128)*128*d elements (Nq padded to whole 128-row tiles) and two
 * fp32 per-row statistics [B, H, Nq], each rounded up to 256 bytes. Returns 0
 * for invalid arguments. */
size_t fa_bwd_workspace_size(int B, int H, int Nq, int d);

/* Backward pass of fa_fwd (no key mask): given dout = dL/dO, writes
 * dq = dL/dQ, dk = dL/dK and dv = dL/dV for the same q, k, v, scale and
 * causal flag. The probability tiles are recomputed from the forward's lse
 * instead of being stored ("Flash Attention Optimization", section "Sizing a
 * tile, and why the backward pass recomputes instead of storing"; "Explain
 * FlashAttention ...", section "Exact attention, finite precision and
 * backward"): with P = exp(scale Q K^T - lse) over the visible keys and
 * D_i = sum_c dout_ic o_ic,
 *   dv = P^T dout,  dS = P * (dout V^T - D),  dq = scale dS K,  dk = scale dS^T Q.
 *   q, o, dout, dq  bf16 [B, H, Nq, d]     k, v, dk, dv  bf16 [B, H, Nk, d]
 *   lse             fp32 [B, H, Nq], as written by fa_fwd for these inputs
 *   workspace       device memory of at least fa_bwd_workspace_size() bytes,
 *                   256-byte aligned, owned by the caller; overwritten.
 * Requires B, H, Nq, Nk >= 1, d in {64, 128}, 16-byte aligned bf16 buffers,
 * a finite scale. Keys no visible query reaches get dk = dv = 0. Three
 * launches on `stream` (statistics, the fused tiles, dq conversion); errors
 * as for fa_fwd, plus FA_ERR_WORKSPACE. */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                 void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- Paged K/V caches -------------------------------------------------------
 * A pool of num_pages pages of `page` rows (16, 32, 64 or 128) holds the keys
 * (another one the values) of many sequences, of K/V head hk in
 *   k_pages, v_pages  [num_pages, Hkv, page, d]: bf16, or e4m3 codes (e4m3 != 0)
 *   k_scale, v_scale  fp32 [num_pages, Hkv], e4m3 only: the real value of a code
 *                     c of page i and head hk is e4m3(c) * scale[i, hk]
 *   block_table       int32 [B, >= width]: page of positions 0 .. page-1 of
 *                     sequence b, of the next `page` positions, and so on; rows
 *                     table_stride apart (elements). Entries past a sequence's
 *                     length are not read.
 * Both entry points leave alone what they cannot place: a table entry that is
 * not in [0, num_pages) is skipped (its keys are hidden, its rows not written),
 * lengths are clipped to the cache. Such a call is reported afterwards by
 * fa_get_device_status() as FA_ERR_INVALID_ARG. */

/* Norms of query and key heads, position rotation, and append of k and v to a
 * paged cache, in one pass over a step's projections.
 *   q  bf16 [T, H, d]   k, v  bf16 [T, Hkv, d]   T new tokens, sequence after
 *      sequence: those of sequence b are cu_seqlens[b] .. cu_seqlens[b+1]-1
 *      (int32 [B+1] on the device), or T / B each when cu_seqlens is NULL.
 *   seqlens_k  int32 [B]: lengths L_b with the new tokens counted (what
 *      fa_decode_paged takes next), so token i of n_b is at position
 *      p = L_b - n_b + i. The tokens of a sequence of length 0 are padding (of a
 *      captured batch, say): nothing is written for them.
 *   q_weight, k_weight  bf16 [d] or NULL: each head is first normalised,
 *      x / sqrt(mean(x^2) + eps) * weight.
 *   rot, turns, interleaved, rot_scale  The first `rot` elements of every q and
 *      k head (a multiple of 16, 0 for none) are turned in pairs j, elements
 *      (j, j + rot/2), or (2j, 2j + 1) when interleaved != 0, by the angle
 *      2 pi frac(p * turns[j] / 2^64), times rot_scale:
 *      (a, b) -> rot_scale * (a cos - b sin, b cos + a sin). turns: int64
 *      [rot/2] on the device, the frequency in 2^-64 turns a position (modulo
 *      2^64): the product modulo 2^64 is exact at every position.
 *   q_out  bf16 [T, H, d]; may be q.   k_out  bf16 [T, Hkv, d], the turned keys
 *      (for attention among the new tokens), or NULL; may be k.
 *   strides  int64 [10], host memory: token and head strides, in elements, of q,
 *      k, v, q_out, k_out in that order (multiples of 8; those of an output such
 *      that no two of its rows of d elements overlap, from the smallest stride to
 *      the largest each past what the ones before span; the d elements of a head
 *      are contiguous), so q, k and v can be parts of one projection.
 *   max_new  the most new tokens of one sequence when cu_seqlens is given (0:
 *      not known; of sequences with more, the tokens past it are left out, the
 *      others keep their positions, and the call is reported).
 * k and v go to the row of their position, in bf16 or as e4m3 codes. The scale
 * of an e4m3 page is a power of two, the least 2^e, e >= -40, with
 * |x| <= 448 * 2^e over the rows of this sequence that the page holds. Rows that
 * earlier calls wrote keep their scale while it suffices; when it grows their
 * codes are rounded again to the new one. Rounding is to nearest even from the
 * fp32 result; an infinity or NaN is stored as the NaN code and left out of the
 * scale. A call that starts at row 0 of a page takes nothing from the page's old
 * contents or scale.
 * Every page that a call writes must be listed once, by one sequence (pages that
 * several sequences or places share may be read, not appended to). Rows of q_out and k_out of
 * tokens past cu_seqlens[B] are left as they were. T = 0 is a no-op. d = 64 or
 * 128. One launch on `stream`. Errors: FA_ERR_INVALID_ARG for NULL tensors, bad
 * sizes, H not a multiple of Hkv, T not a multiple of B without cu_seqlens;
 * FA_ERR_UNSUPPORTED for other d, rot or page sizes, strides that are not
 * multiples of 8, or pointers that are not 16-byte (scales, table, lengths and
 * offsets 4-byte) aligned. */
fa_status fa_append_paged(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* k_pages,
                          void* v_pages, float* k_scale, float* v_scale, const int* block_table, int64_t table_stride,
                          const int* seqlens_k, const int* cu_seqlens, const int64_t* turns, const void* q_weight,
                          const void* k_weight, const int64_t* strides, int B, int T, int H, int Hkv, int d,
                          int num_pages, int page, int table_width, int e4m3, int rot, int interleaved,
                          float rot_scale, float eps, int max_new, void* stream);

/* Bytes of device workspace fa_decode_paged needs: the partial states of the
 * ranges it shares the keys out in. Returns 0 for invalid arguments. */
size_t fa_decode_paged_workspace_size(int B, int H, int Hkv, int Nq, int d, int max_len, int num_splits);

/* fa_decode_grouped over a paged cache: the last Nq tokens of every sequence
 * attend to its keys in the pool. Sequence b holds L_b = seqlens_k[b] keys, its
 * new ones among them; token t sees key j iff j <= L_b - Nq + t; query head h
 * reads K/V head h / (H/Hkv). A token that sees no key gets o = 0, lse = -inf.
 *   q, o       bf16 [B, H, Nq, d] with element strides q_strides, o_strides
 *              (int64 [3], host memory: batch, head, token; multiples of 8; no two
 *              rows of o overlap, as for fa_append_paged; d contiguous). Token-major tensors, as fa_append_paged returns them,
 *              are passed by their strides.
 *   lse        fp32 [B, H, Nq] (may be NULL)
 *   max_len    no sequence is longer (at most the positions a block-table row
 *              covers, and at most 2^30; longer ones are clipped and reported).
 *   num_splits 0: the keys of the whole batch are shared out in equal ranges, one
 *              for each warp that the GPU holds, whatever the lengths;
 *              1 .. 1024: in so many ranges a sequence and K/V head on average.
 *   scales of e4m3 pages: positive factors, powers of two (as fa_append_paged
 *              writes them) or not; those of v between 2^-80 and 2^120. Pages of one
 *              sequence may differ by 2^80: each keeps its own values' precision.
 *   workspace  device memory of fa_decode_paged_workspace_size() bytes, 256-byte
 *              aligned, owned by the caller, overwritten; calls that may overlap
 *              on the GPU need their own.
 * Products with e4m3 pages run in f16 on the codes, with fp32 accumulation, the
 * weights rounded to f16 (below 2^-14 of a row's largest to 2^-25 of it) and q held
 * in f16 (elements below 2^-14 of a row's largest to 2^-25 of it); with bf16 pages
 * in bf16. A NaN or infinity in v reaches the rows of its sequence's last Nq tokens
 * that see a key. Errors as for fa_decode_grouped. Two launches (the ranges, their merge). */
fa_status fa_decode_paged(const void* q, const int64_t* q_strides, const void* k_pages, const void* v_pages,
                          const float* k_scale, const float* v_scale, const int* block_table, int64_t table_stride,
                          const int* seqlens_k, void* o, const int64_t* o_strides, float* lse, int B, int H, int Hkv,
                          int Nq, int d, int num_pages, int page, int max_len, int e4m3, float scale, int num_splits,
                          void* workspace, size_t workspace_bytes, void* stream);

/* fa_append_paged on a cache that lost rows (fa_evict_paged).
 *   offsets  int32 [B], position of row 0 of each sequence: token i of n_b is still
 *            stored in row r = L_b - n_b + i, and turned for position
 *            r + offsets[b], which lies in [0, 2^31). NULL: 0. */
fa_status fa_append_paged_at(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* k_pages,
                             void* v_pages, float* k_scale, float* v_scale, const int* block_table,
                             int64_t table_stride, const int* seqlens_k, const int* cu_seqlens, const int* offsets,
                             const int64_t* turns, const void* q_weight, const void* k_weight, const int64_t* strides,
                             int B, int T, int H, int Hkv, int d, int num_pages, int page, int table_width, int e4m3,
                             int rot, int interleaved, float rot_scale, float eps, int max_new, void* stream);

/* ---- 4-bit pages -------------------------------------------------------------
 * k_pages, v_pages  [num_pages, Hkv, page, d/2] bytes: e2m1 codes (values 0, 0.5, 1,
 *     1.5, 2, 3, 4, 6, bit 3 the sign), element 2i in the lower half of byte i;
 *     16-byte aligned.
 * k_scale, v_scale  [num_pages, Hkv, page, d/16] bytes, 16-byte aligned: the scale of
 *     each 16 neighbouring elements, unsigned with 5 exponent bits (bias 15) and 3
 *     mantissa bits (an f16's upper byte without its sign). A value is code * scale,
 *     exact in f16 and in bf16.
 * A row takes 9/32 of its bf16 bytes. Append sets a group's scale to its largest
 * magnitude / 6, rounded to nearest even, within [2^-17, 10240] (0 for a group of
 * zeros; larger magnitudes saturate at 61440), and its codes to the nearest of
 * x / scale (ties to the even code). An infinity or NaN makes its group of 16 NaN.
 *
 * Codes are steps of the key, so the way to the bf16 key is fixed in every operation, each
 * rounded to nearest in fp32: x * rsqrt(mean + eps) * weight from the left, where the mean's
 * sum takes squares 32 elements apart in order, then neighbouring sums in pairs; the two
 * products of a rotation, then their sum; cosines and sines within 2^-30 of the exact ones
 * before their rounding. q is computed as for the other kinds. */

/* fa_append_paged_at into 4-bit pages. k is quantised as k_out holds it, in bf16;
 * every row is on its own, so nothing written earlier changes. */
fa_status fa_append_paged_fp4(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* k_pages,
                              void* v_pages, uint8_t* k_scale, uint8_t* v_scale, const int* block_table,
                              int64_t table_stride, const int* seqlens_k, const int* cu_seqlens, const int* offsets,
                              const int64_t* turns, const void* q_weight, const void* k_weight, const int64_t* strides,
                              int B, int T, int H, int Hkv, int d, int num_pages, int page, int table_width, int rot,
                              int interleaved, float rot_scale, float eps, int max_new, void* stream);

/* fa_decode_paged over 4-bit pages, and its workspace. Products run in f16 on
 * code * scale, with the bounds that fa_decode_paged gives for q and the weights. */
size_t fa_decode_paged_fp4_workspace_size(int B, int H, int Hkv, int Nq, int d, int max_len, int num_splits);
fa_status fa_decode_paged_fp4(const void* q, const int64_t* q_strides, const void* k_pages, const void* v_pages,
                              const uint8_t* k_scale, const uint8_t* v_scale, const int* block_table,
                              int64_t table_stride, const int* seqlens_k, void* o, const int64_t* o_strides, float* lse,
                              int B, int H, int Hkv, int Nq, int d, int num_pages, int page, int max_len, float scale,
                              int num_splits, void* workspace, size_t workspace_bytes, void* stream);

/* What the pages of the calls below hold (`kind`), with their scales: none (NULL),
 * fp32 [num_pages, Hkv], or the bytes of 4-bit pages. */
#define FA_PAGES_BF16 0
#define FA_PAGES_E4M3 1
#define FA_PAGES_FP4 2

/* Rows of a paged cache as packed bf16 k and v, as fa_fwd_packed takes them (the
 * chunks of a prompt after its first attend to what the cache holds).
 *   cu_seqlens  int32 [B+1] on the device: the last n_b = cu[b+1] - cu[b] rows of
 *           sequence b go to rows cu[b] .. cu[b+1]-1 of k_out and v_out.
 *   k_out, v_out  bf16 [total, Hkv, d]; strides  int64 [4], host memory: token and
 *           head strides of k_out and v_out, as fa_append_paged's outputs have them.
 * A sequence of length 0 is padding; output rows that no row of the cache belongs to
 * are left as they were (rows asked for past a sequence's beginning, pages outside
 * the pool, offsets that decrease or pass `total`: also reported). e4m3 values are
 * rounded once to bf16. total = 0 is a no-op. One launch. Errors as for
 * fa_append_paged, plus FA_ERR_INVALID_ARG for an unknown kind. */
fa_status fa_read_paged(const void* k_pages, const void* v_pages, const void* k_scale, const void* v_scale, int kind,
                        const int* block_table, int64_t table_stride, const int* seqlens_k, const int* cu_seqlens,
                        void* k_out, void* v_out, const int64_t* strides, int B, int total, int Hkv, int d,
                        int num_pages, int page, int table_width, void* stream);

/* Adds the attention weights that the last Nq tokens of every sequence give its keys:
 *   weights[b, hk, j] += sum over the group's heads h and tokens t that see key j of
 *                        exp(scale <q, k_j> - lse[b, h, t])
 *   q, q_strides, scale  as for fa_decode_paged; lse  fp32 [B, H, Nq], what
 *           fa_decode_paged (or a prefill over the same keys) returned; rows with
 *           lse = -inf add nothing.
 *   weights fp32, the row of (b, hk) at (b * Hkv + hk) * weights_stride, at least
 *           max_len long; only keys that a sequence holds are written.
 *   max_len as for fa_decode_paged: longer sequences are clipped and reported.
 * Sums run in fp32 in a fixed order. Keys of pages outside the pool get nothing, and
 * the call is reported. One launch, no workspace. Errors as for fa_decode_paged,
 * plus FA_ERR_INVALID_ARG for an unknown kind or a weights_stride below max_len. */
fa_status fa_weigh_paged(const void* q, const int64_t* q_strides, const float* lse, const void* k_pages,
                         const void* k_scale, int kind, const int* block_table, int64_t table_stride,
                         const int* seqlens_k, float* weights, int64_t weights_stride, int B, int H, int Hkv, int Nq,
                         int d, int num_pages, int page, int max_len, float scale, void* stream);

/* Cuts sequences to `keep` rows. Of the L_b rows of a longer one every K/V head keeps
 * its first `first` and last `recent`, and of the others the keep - first - recent
 * with the largest weights (ties to the lowest index, NaN below all others); a
 * sequence of at most `keep` rows keeps all. Row i of those that stay is copied to
 * position i of the pages that new_table lists.
 *   weights, weights_stride  as fa_weigh_paged leaves them.
 *   block_table, new_table  int32 [B, ..] over the same pool. Pages of new_table are
 *           listed once, and none of them is read by the call (block_table's pages may
 *           be shared between sequences; the caller frees them afterwards).
 *   kept         int32 [B, Hkv, keep]: old row of each new one, -1 past them.
 *   new_seqlens  int32 [B]: min(L_b, keep).
 *   new_offsets  int32 [B]: offsets[b] (NULL: 0) + L_b - new_seqlens[b], the position
 *                of row 0 for the appends to come (the rows before the new ones keep
 *                the rotation of their old positions). May be offsets.
 *   new_weights  fp32 [B, Hkv, new_width] with rows new_weights_stride apart,
 *                new_width >= keep: the kept rows' weights, then zeros.
 * Rows of 4-bit and bf16 pages are copied as they are. The scale of a new e4m3 page is
 * the largest of its rows' old ones (factors >= 0, none NaN), and codes of smaller scales
 * are rounded to it: code * (old / new), ratio and product in fp32, to the nearest code. Rows past the new length keep what the pages held. Pages outside
 * the pool are skipped, lengths over max_len clipped, and reported. Two launches.
 * Errors: FA_ERR_INVALID_ARG for NULL arrays, sizes, first + recent > keep, an unknown
 * kind, strides that do not hold the rows, new_weights that share an element with the
 * weights read, or new_seqlens or new_table that are the arrays read; FA_ERR_UNSUPPORTED as for fa_append_paged. */
fa_status fa_evict_paged(const float* weights, int64_t weights_stride, void* k_pages, void* v_pages, void* k_scale,
                         void* v_scale, int kind, const int* block_table, int64_t table_stride, const int* seqlens_k,
                         const int* offsets, const int* new_table, int64_t new_table_stride, int* kept,
                         int* new_seqlens, int* new_offsets, float* new_weights, int64_t new_weights_stride,
                         int new_width, int B, int Hkv, int d, int num_pages, int page, int max_len, int keep,
                         int first, int recent, void* stream);

/* Synchronises `stream`, then returns and clears the device status word of
 * the current device: FA_ERR_TIMEOUT if a bounded wait gave up since the
 * last call, FA_ERR_CUDA if the stream reported an error, FA_ERR_INVALID_ARG if
 * a paged or packed call met a page, length or offset outside its arrays, else
 * FA_OK. */
fa_status fa_get_device_status(void* stream);

/* Limit, in nanoseconds, on every wait inside the library's kernels
 * (default 2e9). Applies to calls launched afterwards. */
void fa_set_wait_limit_ns(uint64_t ns);
uint64_t fa_get_wait_limit_ns(void);

/* Self-test of the failure path: launches one warp that waits on a barrier
 * nothing ever arrives on, with the given limit; returns what
 * fa_get_device_status() then reports (FA_ERR_TIMEOUT when the bounded wait
 * works). The context stays usable afterwards. */
fa_status fa_selftest_wait_timeout(uint64_t limit_ns, void* stream);

/* Self-test of the device exponential the prefill softmax runs on the FMA
 * pipe for part of each score tile: y[i] = 2^x[i] for x[i] in [-126, 127]
 * (device pointers, fp32, asynchronous on `stream`). Its maximum relative
 * error is 7.5e-5, far below the bf16 rounding applied to P. */
fa_status fa_selftest_exp2(const float* x, float* y, int n, void* stream);

/* Human-readable name of a status code. */
const char* fa_status_string(fa_status s);

/* Detail of the most recent error returned on the calling host thread
 * (empty string if none). */
const char* fa_last_error_detail(void);

/* Number of kernel launches this library issued on the calling host thread
 * since the process started (for accounting in benchmarks). */
uint64_t fa_launch_count(void);

/* Debug build (the pages have no counterpart: this checks the implementation).
 * libfa_gb300_debug.so is the same library compiled with FA_DEBUG=1: its
 * prefill kernels check, before each access, the coordinates of every TMA
 * copy (x on a 16-byte boundary and inside the row, the tile starting inside
 * the tensor, the batch-head index in range), the TMEM lanes and columns of
 * every tensor-memory load, store and product, and at the end of a launch that
 * every barrier completed as many phases as its users counted. A failed check
 * skips the access and records the failure; nothing traps. The release
 * library compiles the checks out.
 *   fa_debug_enabled()   1 in the debug build, 0 in the release build.
 *   fa_debug_record(out) waits for `stream`, copies the current device's
 *                        8-word record to host `out` and clears it: word 0
 *                        bits (1 = TMA coordinate, 2 = TMEM range, 4 =
 *                        barrier phase count), then the first failure's site,
 *                        block, thread and three values, then the number of
 *                        failed checks.
 *   fa_debug_selftest()  launches one warp that runs every check on values it
 *                        must reject, with no access; afterwards the debug
 *                        build's record holds bits 1, 2 and 4. */
int fa_debug_enabled(void);
fa_status fa_debug_record(uint32_t* out, void* stream);
fa_status fa_debug_selftest(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
