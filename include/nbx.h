/*
 * libnbx: paged KV-cache append and split-KV ("flash-decoding") decode attention
 * for one NVIDIA GB300 GPU (sm_103a).
 *
 * C ABI. Every buffer argument is a plain pointer to memory the caller owns; the
 * library allocates and frees nothing and never synchronises the stream. Device
 * pointers are marked [device], host values are passed by value. Streams are
 * passed as `void*` holding a cudaStream_t (NULL = the legacy default stream).
 *
 * Layouts are row-major with the last dimension contiguous:
 *   pool         [num_pages, h_kv, page_tokens, d]   one pool per K and per V
 *   new_k/new_v  [n_tok, h_kv, d]
 *   slot_mapping [n_tok]            int32, slot = page * page_tokens + position in page
 *   q            [batch, rows, h_q, d]
 *   block_table  [batch, max_pages] int32 page ids, -1 past each sequence
 *   seq_lens     [batch]            int32 positions each sequence holds
 *   out          [batch, rows, h_q, d] fp32
 *
 * Sources (pages the method is described on):
 *   nbxtensor 0.0.1 wheel, nbxtensor/ops/attention_wrappers.py: paged_kv_append,
 *     paged_decode_attention, decode_reduce (the boundary and its checks);
 *   nbxtensor 0.0.1 wheel, nbxtensor/ops/paged_decode_attn.py: module docstring (pool
 *     layout, slot mapping, block table), paged_kv_append_kernel, paged_decode_splits,
 *     paged_decode_attn_split_kernel (the split partial);
 *   TensorFold PR #1219: the rows-first grid (all rows of a split share its K/V from
 *     L2), the fp8 cache, the merge's skip rule.
 *
 * Errors. Host-detectable problems return a negative nbx_status before anything is
 * launched. Problems only the device can see (a slot or a page id outside the pool,
 * a length outside its bounds, a wait that ran out of time) set bits in the optional
 * [device] int32 status word with an atomic OR and skip the offending work; kernels
 * never trap. The caller reads the word after synchronising; it is never cleared by
 * the library.
 */
#ifndef NBX_H
#define NBX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define NBX_API __attribute__((visibility("default")))

typedef enum {
    NBX_F32 = 0,   /* IEEE binary32 */
    NBX_BF16 = 1,  /* bfloat16 */
    NBX_E4M3 = 2   /* OCP FP8 E4M3 (FN: no infinities, max 448), with one fp32 scale per pool */
} nbx_dtype;

typedef enum {
    NBX_OK = 0,
    NBX_ERR_NULL = -1,        /* a required pointer is NULL */
    NBX_ERR_SHAPE = -2,       /* sizes that do not fit together, or outside the supported set */
    NBX_ERR_DTYPE = -3,       /* a dtype code this call does not take */
    NBX_ERR_PAGE_ALIGN = -4,  /* page_tokens is not a multiple of NBX_TILE_POSITIONS */
    NBX_ERR_WORKSPACE = -5,   /* workspace smaller than nbx_paged_decode_workspace_bytes() */
    NBX_ERR_CUDA = -6,        /* a CUDA runtime call or launch failed */
    NBX_ERR_ALIGN = -7,       /* a buffer is not 16-byte aligned */
    NBX_ERR_VALUE = -8        /* a scalar argument is not finite or a scale is not positive */
} nbx_status;

/* Bits of the device status word. */
#define NBX_DEV_BAD_SLOT 0x1   /* an append slot outside [0, num_pages * page_tokens): token skipped */
#define NBX_DEV_BAD_PAGE 0x2   /* a block-table entry inside a sequence is -1 or >= num_pages: tile skipped */
#define NBX_DEV_BAD_LEN 0x4    /* seq_lens[b] < 0, > max_seq_len or > max_pages * page_tokens: sequence read as empty */
#define NBX_DEV_TIMEOUT 0x8    /* a bounded wait inside a kernel gave up: the output is incomplete */
#define NBX_DEV_BAD_SCALE 0x10 /* a block's scale is not a number in [2^-48, 2^48]: its positions are skipped */
#define NBX_DEV_BAD_ROW 0x20   /* a fork names a row outside the table, or a destination a second time: skipped */
#define NBX_DEV_NO_PAGE 0x40   /* a fork found no free page for its partial page: its row is left empty */

/* Positions per staged tile: every page must hold a whole number of tiles, so no
 * tile straddles two pages (paged_decode_attention's "ZERO FALLBACK" check). */
#define NBX_TILE_POSITIONS 16
/* The pages' split rule (nbxtensor/ops/paged_decode_attn.py, paged_decode_splits): it bounds the
 * splits a workspace holds; the decode itself cuts splits of two of these (see nbx_paged_decode_attn). */
#define NBX_SPLIT_POSITIONS 256
#define NBX_MAX_SPLITS 64

/*
 * nbx_paged_kv_append -- write new positions into the pools through the slot mapping.
 * (nbxtensor/ops/attention_wrappers.py, paged_kv_append; nbxtensor/ops/paged_decode_attn.py,
 * paged_kv_append_kernel.)
 *
 * For token t and KV head h: page = slot_mapping[t] / page_tokens, pos = slot_mapping[t] %
 * page_tokens, k_pool[page, h, pos, :] = cast(new_k[t, h, :] * (1 / k_scale)), the same for V.
 * The reciprocal is taken once in fp32 on the host; the cast rounds to nearest even (bf16,
 * E4M3 with saturation to +-448) or copies (fp32).
 *
 *   new_k, new_v  [device] [n_tok, h_kv, d] in new_dtype (NBX_F32 or NBX_BF16)
 *   n_tok         tokens to write; 0 returns NBX_OK without a launch
 *   k_pool, v_pool [device] [num_pages, h_kv, page_tokens, d] in pool_dtype (any nbx_dtype)
 *   slot_mapping  [device] int32 [n_tok]; entries must be distinct. A slot outside
 *                 [0, num_pages*page_tokens) sets NBX_DEV_BAD_SLOT and the token is skipped.
 *   k_scale, v_scale  dequantisation scales of the pools (finite, > 0; use 1 unless E4M3)
 *   status        [device] int32 or NULL
 *   stream        cudaStream_t
 * Requirements: d a multiple of 16 and <= 1024; all buffers 16-byte aligned.
 */
NBX_API int nbx_paged_kv_append(const void* new_k, const void* new_v, int new_dtype, int n_tok, int h_kv, int d,
                                void* k_pool, void* v_pool, int pool_dtype, int num_pages, int page_tokens,
                                const int32_t* slot_mapping, float k_scale, float v_scale, int32_t* status,
                                void* stream);

/*
 * nbx_paged_kv_append_rotated -- the append with the position rotation applied on the way.
 *
 * Token t's query and key heads are turned by its position, x' of x with the pair (a, b) at i < turned / 2:
 *   a' = a * cos[positions[t], i] - b * sin[positions[t], i],  b' = b * cos[...] + a * sin[...],
 * a and b being elements i and turned / 2 + i of the head, or with `interleaved` 2i and 2i + 1; elements from `turned`
 * on stay as they are. The turned queries go to q_out in their own type; the turned keys and the values go to the
 * pools as nbx_paged_kv_append writes them (cast(x * (1 / scale))). Arithmetic is fp32, rounded once. This call is an
 * addition of this library; the pages it was written from have no counterpart.
 *
 *   q, new_k, new_v [device] token t at element t * stride, heads [h, d] contiguous there, all in new_dtype
 *                (NBX_F32 or NBX_BF16): strides allow for the pieces of one projection
 *   h_q          query heads; 0: keys and values only (q and q_out are not read then)
 *   cos_table, sin_table [device] fp32 [n_pos, turned / 2]
 *   positions    [device] int32 [n_tok]; a position outside [0, n_pos) sets NBX_DEV_BAD_LEN and the token is
 *                skipped (in q_out and k_out too)
 *   q_out        [device] as q with q_out_stride; may be q itself (with q's stride), but not overlap an input otherwise
 *   k_out        [device] the turned keys once more, in new_dtype and unscaled, as new_k with k_out_stride (for the
 *                attention of the prompt that they belong to); may be new_k itself (with its stride), but not overlap
 *                an input otherwise; or NULL
 *   slot_mapping [device] int32 [n_tok]; a slot outside the pool sets NBX_DEV_BAD_SLOT, the pools are left alone and
 *                q_out and k_out written all the same
 *   the other arguments as for nbx_paged_kv_append
 * Requirements: d and turned multiples of 16, turned <= d <= 1024; buffers and rows 16-byte aligned (strides of whole
 * 16 bytes). n_tok == 0 returns NBX_OK without a launch.
 */
NBX_API int nbx_paged_kv_append_rotated(const void* q, int64_t q_stride, int h_q, const void* new_k, int64_t k_stride,
                                        const void* new_v, int64_t v_stride, int new_dtype, int n_tok, int h_kv, int d,
                                        const float* cos_table, const float* sin_table, int n_pos, int turned,
                                        int interleaved, const int32_t* positions, void* q_out, int64_t q_out_stride,
                                        void* k_out, int64_t k_out_stride, void* k_pool, void* v_pool, int pool_dtype,
                                        int num_pages, int page_tokens, const int32_t* slot_mapping, float k_scale,
                                        float v_scale, int32_t* status, void* stream);

/*
 * nbx_prompt_attn -- causal attention over whole prompts, packed one behind the other.
 *
 * Sequence b's tokens are rows seq_start[b] .. seq_start[b + 1] - 1 of q, k and v. Token i of a sequence (from 0) and
 * query head h attend keys 0 .. i of the sequence and KV head h / (h_q / h_kv):
 *   z_j = scale * (q . k_j),  out = sum_j e^(z_j - max z) v_j / sum_j e^(z_j - max z),
 * 0 where every z_j is -infinity. Scores, sums and statistics are fp32; weights enter the product with the values
 * rounded to bf16 (2^-8), the output is rounded once. Values at keys that a row does not see never reach it, not even a
 * NaN. Results do not depend on what else is packed into the call. This call is an addition of this library; the
 * pages it was written from have no counterpart.
 *
 *   q [n_tok, h_q, d], k, v [n_tok, h_kv, d] [device] NBX_BF16 (dtype), token t at element t * stride, its heads
 *                contiguous there: strides allow for the pieces of one projection
 *   seq_start    [device] int32 [batch + 1], ascending, seq_start[0] >= 0, seq_start[batch] <= n_tok. A sequence whose
 *                bounds make no sense sets NBX_DEV_BAD_LEN and is skipped.
 *   scale        softmax scale (finite)
 *   out          [device] bf16 [n_tok, h_q, d], contiguous; rows of no sequence are left as they were. May not overlap q, k
 *                or v (NBX_ERR_VALUE).
 *   status       [device] int32 or NULL;  stream  cudaStream_t
 * Requirements: h_q % h_kv == 0; d in {64, 128, 256}; buffers and rows 16-byte aligned (strides of whole 16 bytes), out
 * 32-byte aligned. n_tok == 0 or batch == 0 returns NBX_OK without a launch.
 */
NBX_API int nbx_prompt_attn(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int dtype, int n_tok, int h_q, int h_kv, int d, const int32_t* seq_start,
                            int batch, float scale, void* out, int32_t* status, void* stream);

/*
 * nbx_paged_decode_workspace_bytes -- bytes of workspace nbx_paged_decode_attn needs for
 * these sizes (the split plan, the work list and the fp32 split partials).
 * Returns 0 if the sizes are invalid. max_seq_len is the host-known bound on seq_lens.
 */
NBX_API size_t nbx_paged_decode_workspace_bytes(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len);

/*
 * nbx_paged_decode_workspace_bytes_for -- the workspace for these sizes and formats. Every format
 * and page size needs the same today (the tensor-core kernel reads an fp8 pool's codes as they are
 * stored), so it equals nbx_paged_decode_workspace_bytes; the formats are taken so that a caller
 * sizing per call keeps working if that changes. Returns 0 if the sizes are invalid.
 */
NBX_API size_t nbx_paged_decode_workspace_bytes_for(int q_dtype, int pool_dtype, int batch, int rows, int h_q,
                                                    int h_kv, int d, int max_seq_len, int page_tokens);

/*
 * nbx_paged_decode_attn -- split-KV decode attention read through the block table.
 * (nbxtensor/ops/attention_wrappers.py, paged_decode_attention; nbxtensor/ops/paged_decode_attn.py,
 * paged_decode_splits and paged_decode_attn_split_kernel; TensorFold PR #1219, rows-first grid.)
 *
 * For sequence b, query row r and query head h: the row sits at position
 * p = seq_lens[b] - rows + r and attends keys 0..p of KV head h / (h_q / h_kv):
 *   s_j = scale * k_scale * (q . k_j),  out = v_scale * sum_j e^(s_j - max s) v_j / sum_j e^(s_j - max s).
 * A row with no visible key (p < 0, or seq_lens[b] == 0) gets 0. Each sequence is cut into
 * min(ceil(len/512), 64) splits of whole pages, two of the pages' 256-position splits each (a window
 * on tensor cores, see nbx_paged_decode_partial_kernel: about one work unit per SM in all, splits in
 * proportion to the lengths, at most min(ceil(max_seq_len/256), 64)); each split's unnormalised
 * partial (m, l, acc) is computed with an fp32 online softmax and the partials are merged in
 * ascending split order (a split with m = -inf is skipped, so NaN inputs reach the output). The
 * result does not depend on the physical page ids or on the order the work runs in.
 *
 *   q            [device] [batch, rows, h_q, d], q_dtype NBX_F32 or NBX_BF16
 *   k_pool, v_pool [device] [num_pages, h_kv, page_tokens, d] in pool_dtype
 *   block_table  [device] int32 [batch, max_pages]
 *   seq_lens     [device] int32 [batch]
 *   max_seq_len  host bound on seq_lens (sizes the splits and the workspace);
 *                must be <= max_pages * page_tokens
 *   scale        softmax scale (finite); k_scale, v_scale: pool scales (finite, > 0)
 *   out          [device] fp32 [batch, rows, h_q, d]
 *   workspace    [device] at least nbx_paged_decode_workspace_bytes(...) bytes, 256-byte aligned;
 *                its contents need no initialisation and are overwritten
 *   status       [device] int32 or NULL
 *   stream       cudaStream_t
 * Requirements: h_q % h_kv == 0; d in {64, 128, 256}; page_tokens a multiple of
 * NBX_TILE_POSITIONS; q, pools and out 16-byte aligned. batch == 0 returns NBX_OK without a launch.
 * Calls on one workspace must not overlap on the GPU.
 */
NBX_API int nbx_paged_decode_attn(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                  const void* k_pool, const void* v_pool, int pool_dtype, int num_pages, int h_kv,
                                  int page_tokens, const int32_t* block_table, int max_pages,
                                  const int32_t* seq_lens, int max_seq_len, float scale, float k_scale,
                                  float v_scale, float* out, void* workspace, size_t workspace_bytes,
                                  int32_t* status, void* stream);

/*
 * nbx_paged_decode_step -- one decode step with no host-side positions: append, then attend.
 * (nbxtensor/ops/paged_decode_attn.py, paged_kv_append_step_kernel and paged_lens_advance_kernel:
 * the step writes at the layer's device length and the length then advances, so a recorded launch
 * replays unchanged; nbxtensor/ops/attention_wrappers.py, paged_decode_attention for the decode.)
 *
 * For each sequence b, with n = lens[b] on entry: the step's new keys and values are written at
 * positions n .. n + rows - 1 (page block_table[b, pos / page_tokens], slot pos % page_tokens,
 * cast on store exactly as nbx_paged_kv_append does), then the rows attend exactly as
 * nbx_paged_decode_attn with seq_lens[b] = n + rows, and lens[b] becomes n + rows. Everything
 * happens on the stream in that order; the call's arguments are the same at every step, so it
 * can be captured once in a CUDA graph and replayed.
 *
 *   new_k, new_v [device] [batch, rows, h_kv, d] in new_dtype (NBX_F32 or NBX_BF16): row r of
 *                sequence b is the key/value of query row r (position n + r)
 *   lens         [device] int32 [batch], read and then advanced by rows (in stream order)
 *   max_seq_len  host bound on every lens[b] + rows (sizes the splits and the workspace)
 *   every other argument as for nbx_paged_decode_attn; the workspace is sized by
 *   nbx_paged_decode_workspace_bytes(_for) with the same sizes.
 * Device-detected problems set status bits: a position at or past max_seq_len (NBX_DEV_BAD_LEN,
 * not written), a page id outside the pool (NBX_DEV_BAD_PAGE, not written). The host checks are
 * those of nbx_paged_decode_attn plus new_dtype; on any failure nothing is launched.
 * This library addition fuses what the pages run as separate launches.
 */
NBX_API int nbx_paged_decode_step(const void* q, int q_dtype, int batch, int rows, int h_q, int d, const void* new_k,
                                  const void* new_v, int new_dtype, void* k_pool, void* v_pool, int pool_dtype,
                                  int num_pages, int h_kv, int page_tokens, const int32_t* block_table, int max_pages,
                                  int32_t* lens, int max_seq_len, float scale, float k_scale, float v_scale,
                                  float* out, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * nbx_decode_attn_contiguous -- split-KV decode over a contiguous (non-paged) cache.
 * (nbxtensor/ops/attention_wrappers.py, _decode_attn_vec: the same split read and fixed-order
 * merge without a page table.)
 *
 * The caches k_cache, v_cache [device] [batch, h_kv, capacity, d] in cache_dtype hold sequence b's
 * positions 0 .. capacity - 1. That is the pool layout with one page of capacity positions per
 * sequence, so the call is nbx_paged_decode_attn with num_pages = batch, page_tokens = capacity,
 * max_pages = 1 and the identity block table (page b for sequence b), which the library writes
 * into the workspace itself. Same results, rules and errors as nbx_paged_decode_attn;
 * capacity must be a multiple of NBX_TILE_POSITIONS and >= max_seq_len; the workspace is sized by
 * nbx_paged_decode_workspace_bytes_for(..., page_tokens = capacity).
 */
NBX_API int nbx_decode_attn_contiguous(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                       const void* k_cache, const void* v_cache, int cache_dtype, int h_kv,
                                       int capacity, const int32_t* seq_lens, int max_seq_len, float scale,
                                       float k_scale, float v_scale, float* out, void* workspace,
                                       size_t workspace_bytes, int32_t* status, void* stream);

/*
 * nbx_paged_decode_merge -- the fixed-order merge of split partials on its own.
 * (nbxtensor/ops/attention_wrappers.py, decode_reduce; TensorFold PR #1219, the merge's skip rule.)
 *
 * For each row i: M = max_s m[i,s], L = sum_s l[i,s] e^(m[i,s]-M),
 * out[i,:] = sum_s acc[i,s,:] e^(m[i,s]-M) / L, s ascending, skipping splits with m = -inf.
 * A row with no live split gets 0. m is in natural-log units (the running max of the scores).
 *
 *   acc_part [device] fp32 [n_rows, splits, d];  m_part, l_part [device] fp32 [n_rows, splits]
 *   out      [device] fp32 [n_rows, d]
 * Requirements: 1 <= splits <= 4096, 1 <= d <= 1024. n_rows == 0 returns NBX_OK without a launch.
 */
NBX_API int nbx_paged_decode_merge(const float* acc_part, const float* m_part, const float* l_part, int n_rows,
                                   int splits, int d, float* out, void* stream);

/*
 * nbx_paged_decode_bounds -- the score bounds the fixed-shift softmax gates on.
 * (maxdiffusion PR #477, "fixed-m": the per-head metadata computed before the kernel, here per query
 * vector and per (sequence, KV head).)
 *
 * q_norm [device] fp32 [batch, rows, h_q]: |q| of every query vector.
 * kv_max [device] fp32 [batch, h_kv, 2]: {max_j |k_j| * k_scale, max_{j,d} |v_jd| * v_scale} over the
 * positions 0 .. seq_lens[b] - 1 of the sequence, read through the block table. A NaN input gives a
 * NaN bound (which no gate passes). One pass over the sequences' K and V. Other arguments, rules and
 * status bits as for nbx_paged_decode_attn (no workspace).
 */
NBX_API int nbx_paged_decode_bounds(const void* q, int q_dtype, int batch, int rows, int h_q, int d, const void* k_pool,
                                    const void* v_pool, int pool_dtype, int num_pages, int h_kv, int page_tokens,
                                    const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                                    int max_seq_len, float k_scale, float v_scale, float* q_norm, float* kv_max,
                                    int32_t* status, void* stream);

/*
 * nbx_paged_decode_attn_fixed_shift -- nbx_paged_decode_attn with the fixed-shift softmax of
 * maxdiffusion PR #477 ("fixed-m") on the tensor-core kernel, as an ablation of the online max.
 *
 * For a query row of a split of n keys, U = |q| * max|k| * scale * log2(e) bounds every score in
 * log2 units (Cauchy-Schwarz). With C(n) = 127 - ceil(log2 n) - ceil(log2 256) and the gate
 * floor((C(n) + 125) / 2): a row with U <= gate and max |v| <= 256 takes its weights as 2^(z - m),
 * m = ceil(U) - C(n), fixed before the split is read (no running max, no rescale; no weight above 2^C
 * or below 2^-125). A row that fails the gate, and every row of a window whose P enters the product
 * as E4M3 terms (an fp8 pool on tensor cores: E4M3 cannot hold 2^C), keeps the online max. Calls that
 * run the SIMT kernel are the same as nbx_paged_decode_attn. Results are within the decode's tolerance
 * of nbx_paged_decode_attn's.
 *
 *   q_norm, kv_max  [device] the bounds, as nbx_paged_decode_bounds writes them
 *   every other argument as for nbx_paged_decode_attn.
 */
NBX_API int nbx_paged_decode_attn_fixed_shift(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                              const void* k_pool, const void* v_pool, int pool_dtype, int num_pages,
                                              int h_kv, int page_tokens, const int32_t* block_table, int max_pages,
                                              const int32_t* seq_lens, int max_seq_len, float scale, float k_scale,
                                              float v_scale, float* out, void* workspace, size_t workspace_bytes,
                                              const float* q_norm, const float* kv_max, int32_t* status,
                                              void* stream);

/*
 * nbx_decode_fixed_shift_gate -- the fixed-shift constants for n_keys keys and a value bound
 * (maxdiffusion PR #477, get_fixed_m_constants): C = 127 - ceil(log2 n_keys) - ceil(log2 v_max_bound)
 * and gate = floor((C + 125) / 2). Host-only. NBX_ERR_VALUE for n_keys < 1 or v_max_bound < 1.
 */
NBX_API int nbx_decode_fixed_shift_gate(int n_keys, double v_max_bound, int* c_out, int* gate_out);

/* ------------------------------------------------------------------------------------------------
 * The block-scaled cache: E4M3 pools with one fp32 scale per block of tokens and KV head.
 *
 *   k_pool, v_pool      [num_pages, h_kv, page_tokens, d] E4M3 codes
 *   k_scales, v_scales  [num_pages, h_kv, page_tokens / scale_tokens] fp32, each in [2^-48, 2^48]:
 *                       position j of a page stands for code * scale[j / scale_tokens]
 *   scale_tokens        16, 32, 64 or 128, dividing page_tokens (NBX_ERR_PAGE_ALIGN otherwise)
 * These calls and the score modifications and page calls below are additions of this library; the
 * pages it was written from have no counterpart.
 */

/*
 * nbx_paged_kv_append_block_scaled -- write new positions into a block-scaled cache.
 *
 * Sequence b's new tokens are rows tok_start[b] .. tok_start[b + 1] - 1 of new_k / new_v; they go to
 * positions lens[b], lens[b] + 1, ... through the block table. For every block of scale_tokens
 * positions that gets new tokens, per KV head, K and V apart:
 *   need = the smallest power of two in [2^-48, 2^48] with max |x| <= 448 * need over the finite values
 *          of the block's new tokens;
 *   S    = need when the block's first position is new, else max(the block's scale, need);
 *   new codes are e4m3(x / S) (nearest even, saturating at +-448; NaN stays NaN); if S grew, the codes
 *   of the positions held before become e4m3(code * old S / S), which is exact but for results under 2^-6
 *   where the old S was written here too. Quotient and product are fp32 (exact with powers of two).
 * Positions past the new ones are left as they are. lens is not advanced. Appending the same tokens
 * again at the same lens gives the same cache.
 *
 *   new_k, new_v [device] [n_tok, h_kv, d], new_dtype NBX_F32 or NBX_BF16
 *   block_table  [device] int32 [batch, max_pages];  lens [device] int32 [batch]
 *   tok_start    [device] int32 [batch + 1], ascending, tok_start[batch] <= n_tok
 * A sequence whose tok_start or lens make no sense, or a block past max_pages, is skipped with
 * NBX_DEV_BAD_LEN (where tok_start does not ascend, parts of others may be skipped too), a page outside the pool with NBX_DEV_BAD_PAGE; a held block whose scale is not in
 * [2^-48, 2^48] gets need and NBX_DEV_BAD_SCALE. No two sequences may append to one page.
 * Requirements: d in {64, 128, 256}; buffers 16-byte aligned. n_tok == 0 or batch == 0 returns NBX_OK
 * without a launch.
 */
NBX_API int nbx_paged_kv_append_block_scaled(const void* new_k, const void* new_v, int new_dtype, int n_tok, int h_kv,
                                             int d, void* k_pool, void* v_pool, float* k_scales, float* v_scales,
                                             int scale_tokens, int num_pages, int page_tokens,
                                             const int32_t* block_table, int max_pages, int batch,
                                             const int32_t* lens, const int32_t* tok_start, int32_t* status,
                                             void* stream);

/*
 * nbx_paged_decode_attn_block_scaled -- split-KV decode attention over a block-scaled cache.
 * nbx_paged_decode_attn_modified     -- nbx_paged_decode_attn with the score modifications below.
 *
 * For sequence b of n = seq_lens[b] positions, query row r at position p = n - rows + r and query head h,
 * with key j standing for its value (code * block scale, or element * k_scale / v_scale):
 *   the visible keys are j in [begin, end), cut to [0, n): begin = key_begin[b, r] (0 if NULL),
 *     end = key_end[b, r] (p + 1 if NULL);
 *   z_j = scale * (q . k_j);  with softcap > 0: z_j = softcap * tanh(z_j / softcap);
 *     with slopes: z_j -= slopes[h] * |p - j|;
 *   out = sum_j e^(z_j - max z) v_j / sum_j e^(z_j - max z), 0 for a row that sees no key.
 * A document mask is key_begin = the start of the row's document, a prefix mask key_end =
 * max(p + 1, prefix length), a window key_begin = p + 1 - window. Keys before the first and behind the last that
 * some row of a sequence sees are not read: their pages may be gone from the table (-1). One between them may be
 * read without being seen, where ranges leave a gap: its page and scale count as read for the status word.
 *
 *   softcap      0 (none), or such that softcap * log2 e and its reciprocal are finite floats
 *   slopes       [device] fp32 [h_q] or NULL
 *   key_begin, key_end  [device] int32 [batch, rows] or NULL each
 *   out          [device] [batch, rows, h_q, d] in out_dtype: NBX_F32, or NBX_BF16 (rounded once)
 *   workspace    [device] nbx_paged_decode_modified_workspace_bytes(...) bytes, 256-byte aligned
 *   k_scales, v_scales, scale_tokens  as for nbx_paged_kv_append_block_scaled; scales need not be powers of
 *                two here. A block that is read whose scale is not in [2^-48, 2^48] sets NBX_DEV_BAD_SCALE and
 *                its positions are skipped.
 *   every other argument, rule and status bit as for nbx_paged_decode_attn; results likewise do not depend
 *   on page ids or on the order the work runs in.
 */
NBX_API size_t nbx_paged_decode_modified_workspace_bytes(int batch, int rows, int h_q, int h_kv, int d,
                                                         int max_seq_len);

/*
 * nbx_paged_decode_modified_partial_kernel -- which split-partial kernel these two calls run (block-scaled
 * pools: pool_dtype NBX_E4M3). Host-only. A window that nbx_paged_decode_partial_kernel gives to the tensor
 * cores runs there, but an fp8 one only with a bf16 output (its weights are held to 2^-8, a bf16 window's to
 * 2^-17, a capped score to 2^-20 of itself); with a bf16 output so do windows of 40 query vectors of a KV head,
 * 32 at d = 256. Other E4M3 pools, and bf16 pools under bf16 queries, run NBX_PARTIAL_WARP, the rest
 * NBX_PARTIAL_SIMT; both are as exact as fp32 sums.
 * Over an fp32 or bf16 pool, nbx_paged_decode_attn_modified without a modification and with an fp32 output is
 * nbx_paged_decode_attn, bit for bit, and runs that call's kernel. (Over an E4M3 pool it is not: that call's windows
 * hold weights to 2^-8 whatever the output, and are three to four times as fast as this one's fp32.)
 */
NBX_API int nbx_paged_decode_modified_partial_kernel(int q_dtype, int pool_dtype, int out_dtype, int rows, int h_q,
                                                     int h_kv, int d, int num_pages, int page_tokens);
NBX_API int nbx_paged_decode_attn_block_scaled(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                               const void* k_pool, const void* v_pool, const float* k_scales,
                                               const float* v_scales, int scale_tokens, int num_pages, int h_kv,
                                               int page_tokens, const int32_t* block_table, int max_pages,
                                               const int32_t* seq_lens, int max_seq_len, float scale, float softcap,
                                               const float* slopes, const int32_t* key_begin, const int32_t* key_end,
                                               void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                               int32_t* status, void* stream);
NBX_API int nbx_paged_decode_attn_modified(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                           const void* k_pool, const void* v_pool, int pool_dtype, int num_pages,
                                           int h_kv, int page_tokens, const int32_t* block_table, int max_pages,
                                           const int32_t* seq_lens, int max_seq_len, float scale, float k_scale,
                                           float v_scale, float softcap, const float* slopes,
                                           const int32_t* key_begin, const int32_t* key_end, void* out, int out_dtype,
                                           void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * nbx_paged_decode_attn_shared -- decode attention for sequences that share a prefix of the cache, read once a group.
 *
 * The results are nbx_paged_decode_attn's (out in out_dtype, fp32 or bf16, rounded once), to fp32 rounding. Group g is the
 * sequences group_start[g] .. group_start[g + 1] - 1, and says that the rows of the block table that belong to them name
 * the same pages for positions 0 .. shared_lens[g] - 1, as nbx_paged_kv_fork leaves them. That many positions, cut to
 * whole pages and to what every query row of the group sees, are read through the group's first row that is not empty,
 * for all of its query vectors at once; each sequence's other positions are its own. What shared_lens may say: anything up to the
 * common prefix (a row that holds other pages there is read as if it held the first row's). Sequences of no group, groups
 * of one and short prefixes are read sequence by sequence; empty sequences may lie in a group.
 * Prefixes are read apart for bf16 and E4M3 pools under bf16 queries, on the tensor cores, and so are the sequences' own
 * positions from 8 query vectors to a KV head on (rows * h_q / h_kv). There a bf16 output takes the weights
 * rounded to 2^-8 and each split's share to 2^-8, an fp32 one the weights to 2^-22 of the largest. Elsewhere the groups
 * are ignored. A call of one row a sequence that spares less than some 16,000 positions (the prefix, times the members
 * less one) is up to 5 us faster without groups (n_groups 0).
 *
 *   group_start  [device] int32 [n_groups + 1], ascending, within [0, batch]
 *   shared_lens  [device] int32 [n_groups], >= 0. Groups that make no sense set NBX_DEV_BAD_ROW and none counts.
 *   workspace    [device] nbx_paged_decode_shared_workspace_bytes(...) bytes, 256-byte aligned
 *   every other argument, rule and status bit as for nbx_paged_decode_attn_modified without a modification, but that out
 *                is 32-byte aligned
 */
NBX_API size_t nbx_paged_decode_shared_workspace_bytes(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len,
                                                       int n_groups);
NBX_API int nbx_paged_decode_attn_shared(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                         const void* k_pool, const void* v_pool, int pool_dtype, int num_pages, int h_kv,
                                         int page_tokens, const int32_t* block_table, int max_pages,
                                         const int32_t* seq_lens, int max_seq_len, const int32_t* group_start,
                                         const int32_t* shared_lens, int n_groups, float scale, float k_scale,
                                         float v_scale, void* out, int out_dtype, void* workspace,
                                         size_t workspace_bytes, int32_t* status, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Pages. A page is in use while an entry of the block table names it, within its row's length or past
 * it (a page reserved for growth). There are no reference counts: filling a row with -1 frees the pages
 * that no other row names. Rows may share pages.
 */

/*
 * nbx_paged_kv_copy_pages -- copy the held positions of pages to other pages.
 *
 * moves [device] int32 [max_moves, 3]: {source page, destination page, positions}, the first *n_moves
 * of them used ([device] int32; clamped to [0, max_moves]): positions 0 .. positions - 1 of every KV
 * head of both pools, and with k_scales / v_scales (an E4M3 pool; otherwise NULL) the scales of the
 * blocks that hold them. The moves of a fork or a compaction of one layer's table are applied to the
 * other layers' pools with this call.
 * No page may be a destination twice, or a destination and a source. A page outside the pool is skipped
 * with NBX_DEV_BAD_PAGE, a count outside [0, page_tokens] with NBX_DEV_BAD_LEN.
 * Requirements: d a multiple of 16 and <= 1024; a page of all heads under 2 GB; pools 16-byte aligned.
 */
NBX_API int nbx_paged_kv_copy_pages(const int32_t* moves, const int32_t* n_moves, int max_moves, void* k_pool,
                                    void* v_pool, int pool_dtype, int num_pages, int h_kv, int page_tokens, int d,
                                    float* k_scales, float* v_scales, int scale_tokens, int32_t* status,
                                    void* stream);

/*
 * nbx_paged_kv_fork -- rows of the block table become copies of other rows.
 *
 * For i = 0 .. n_fork - 1, row fork_dst[i] becomes row fork_src[i] as it was before the call, in length
 * and content. Full pages are shared; a last page that is partly filled is copied to the lowest free
 * page, in order of i, so that both can go on appending. Where the source row is itself a destination
 * (a beam that is replaced), its first reader takes the partial page over without a copy. The rest of
 * the destination row is -1; what it held before is free, unless another row names it.
 *
 *   block_table  [device] int32 [batch, max_pages], updated;  seq_lens [device] int32 [batch], updated
 *   fork_src, fork_dst [device] int32 [n_fork]; destinations distinct
 *   k_pool, v_pool and the arguments after them as for nbx_paged_kv_copy_pages; both NULL (the sizes
 *                num_pages and page_tokens still count): the table only, nothing is copied
 *   moves        [device] int32 [n_fork, 3], written: the copies {source, fresh page, positions} in
 *                order of i, then -1;  n_moves [device] int32, written
 *   workspace    [device] nbx_paged_kv_fork_workspace_bytes(batch, max_pages, n_fork, num_pages) bytes,
 *                256-byte aligned
 * A row outside the table, or a destination named a second time, sets NBX_DEV_BAD_ROW and that fork is
 * skipped; a source length outside its bounds sets NBX_DEV_BAD_LEN and a missing free page
 * NBX_DEV_NO_PAGE, and the destination is left empty (length 0, all -1). n_fork == 0 or batch == 0
 * returns NBX_OK without a launch.
 */
NBX_API size_t nbx_paged_kv_fork_workspace_bytes(int batch, int max_pages, int n_fork, int num_pages);
NBX_API int nbx_paged_kv_fork(int32_t* block_table, int max_pages, int32_t* seq_lens, int batch,
                              const int32_t* fork_src, const int32_t* fork_dst, int n_fork, void* k_pool, void* v_pool,
                              int pool_dtype, int num_pages, int h_kv, int page_tokens, int d, float* k_scales,
                              float* v_scales, int scale_tokens, int32_t* moves, int32_t* n_moves, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream);

/*
 * nbx_paged_kv_compact -- move the pages in use to the lowest ids.
 *
 * With n_live pages in use, the k-th page in use at an id >= n_live (ascending) moves to the k-th free
 * id < n_live; new_block_table is the table with the new ids. Ids from n_live on are then free, and the
 * pool can be cut there. The held positions of a page are copied (the most that any row holds of it).
 *
 *   block_table  [device] int32 [batch, max_pages];  new_block_table the same shape, may be block_table
 *   moves        [device] int32 [max_moves, 3], written as by nbx_paged_kv_fork; max_moves >= num_pages / 2
 *   counts       [device] int32 [2], written: {moves, pages in use}
 *   workspace    [device] nbx_paged_kv_compact_workspace_bytes(num_pages) bytes, 256-byte aligned
 *   pools        as for nbx_paged_kv_fork (both NULL: nothing is copied)
 * Entries that name no page of the pool are kept (NBX_DEV_BAD_PAGE if >= num_pages); a length outside its bounds
 * sets NBX_DEV_BAD_LEN and is cut to them. num_pages <= 2^30.
 * batch == 0 returns NBX_OK without a launch.
 */
NBX_API size_t nbx_paged_kv_compact_workspace_bytes(int num_pages);
NBX_API int nbx_paged_kv_compact(const int32_t* block_table, int32_t* new_block_table, int max_pages,
                                 const int32_t* seq_lens, int batch, void* k_pool, void* v_pool, int pool_dtype,
                                 int num_pages, int h_kv, int page_tokens, int d, float* k_scales, float* v_scales,
                                 int scale_tokens, int32_t* moves, int max_moves, int32_t* counts, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream);

/*
 * nbx_call -- one of the calls above from an array of its arguments, for bindings to which every argument of a
 * call costs (from Python it saves a call of twenty arguments 1 us of 10). args[i] is argument i: a pointer or an
 * integer as it is, a float as the bits of a double. An unknown call returns NBX_ERR_VALUE.
 */
enum nbx_callable {
  NBX_CALL_APPEND_BLOCK_SCALED = 0,
  NBX_CALL_DECODE_BLOCK_SCALED = 1,
  NBX_CALL_DECODE_MODIFIED = 2,
  NBX_CALL_COPY_PAGES = 3,
  NBX_CALL_FORK = 4,
  NBX_CALL_COMPACT = 5,
  NBX_CALL_APPEND_ROTATED = 6,
  NBX_CALL_PROMPT = 7,
  NBX_CALL_DECODE_SHARED = 8
};
NBX_API int nbx_call(int call, const int64_t* args);

/* Bytes of device scratch that libnbx keeps for nbx_paged_decode_attn_noalloc (32 MiB). */
#define NBX_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * nbx_paged_decode_attn_noalloc -- nbx_paged_decode_attn without a caller workspace.
 * The pages have no counterpart of this call: it exists for callers that cannot allocate device
 * memory (code running where cudaMalloc is not allowed, such as an allocator's own callbacks, a
 * process whose memory budget is fixed before the library loads, or a plug-in without access to
 * the host application's allocator).
 *
 * Same arguments, layouts and results as nbx_paged_decode_attn, minus workspace and
 * workspace_bytes. The scratch is a fixed array of NBX_NOALLOC_SCRATCH_BYTES in the library's
 * own device memory, held by every GPU that loads the library until the process exits. Sizes
 * whose workspace (nbx_paged_decode_workspace_bytes) exceeds it return NBX_ERR_WORKSPACE without
 * a launch. Nothing is allocated or freed.
 * The first call on a device looks up the array's device address with that device current; make
 * that first call before any stream capture. All calls share the one array and it keeps the last
 * call's contents (every call rewrites what it reads), so calls that overlap on the GPU race.
 */
NBX_API int nbx_paged_decode_attn_noalloc(const void* q, int q_dtype, int batch, int rows, int h_q, int d,
                                          const void* k_pool, const void* v_pool, int pool_dtype, int num_pages,
                                          int h_kv, int page_tokens, const int32_t* block_table, int max_pages,
                                          const int32_t* seq_lens, int max_seq_len, float scale, float k_scale,
                                          float v_scale, float* out, int32_t* status, void* stream);

/* The split-partial kernel a decode call runs (see nbx_paged_decode_partial_kernel). */
typedef enum {
    NBX_PARTIAL_SIMT = 0,            /* CUDA cores: work units of 4 query vectors, any supported shape */
    NBX_PARTIAL_TCGEN05 = 1,         /* tensor cores (tcgen05.mma): work units of 128 query vectors */
    NBX_PARTIAL_TCGEN05_FP8 = 2,     /* fp8 (E4M3) pool: the tensor-core kernel on the codes as stored
                                        (tcgen05.mma kind::f8f6f4), Q and P as two E4M3 terms each */
    NBX_PARTIAL_WARP = 3             /* modified decodes: work units of 8 query vectors, one warp each, on mma.sync */
} nbx_partial_kernel;

/*
 * nbx_paged_decode_partial_kernel -- which split-partial kernel nbx_paged_decode_attn (and
 * nbx_paged_decode_attn_noalloc) runs for these sizes and formats. Host-only; launches nothing.
 * (TensorFold PR #1219: the rows of one KV head read each K/V tile once; when rows x group
 * reaches a dense tile the QK^T and PV products become matrix products.)
 *
 * Returns NBX_PARTIAL_TCGEN05 when rows * (h_q / h_kv) >= 64, h_q / h_kv <= 128, q_dtype and
 * pool_dtype are both NBX_BF16, d is 128 or 256, page_tokens is a multiple of 64 and the pool has
 * fewer than 2^31 - 64 rows of d elements per K or V (the call itself also needs scale > 0; a
 * decode with scale <= 0 runs the SIMT kernel); NBX_PARTIAL_TCGEN05_FP8 under the same conditions
 * with an NBX_E4M3 pool; NBX_PARTIAL_SIMT for every other supported case; a negative nbx_status for
 * arguments nbx_paged_decode_attn rejects (shape, page alignment, dtype). The kernels compute the
 * same partials to within the decode's tolerance; none depends on page ids or on the grid size.
 */
NBX_API int nbx_paged_decode_partial_kernel(int q_dtype, int pool_dtype, int rows, int h_q, int h_kv, int d,
                                            int num_pages, int page_tokens);

/*
 * nbx_set_decode_grid_limit -- cap the number of CTAs nbx_paged_decode_attn launches for its split
 * partial (0 = each kernel's default: two or three CTAs per SM for the SIMT kernel, one per SM for
 * the tensor-core kernel). Process-wide; the output is bit-identical for every value.
 */
NBX_API void nbx_set_decode_grid_limit(int max_ctas);

/*
 * nbx_set_decode_wait_test -- for tests of the timeout path only; the pages have no counterpart.
 * Every wait inside the split-partial kernels, and inside those of prompts and of shared prefixes, is
 * bounded (2 s by default; in prompts and shared prefixes the bound begins anew while rows are computed
 * again, because of values that are not finite in their tile but unseen by them): a wait that runs out
 * sets NBX_DEV_TIMEOUT, the kernel lets its copies in flight land (and, on tensor cores, its MMAs
 * complete and its TMEM go back) and returns, and the output of the call is incomplete. This sets
 * that bound (wait_limit_ns; 0 restores 2 s) and holds each CTA's producer warps back for
 * producer_delay_ns before they start (0 = no delay; capped at 50 ms), so a test can make the other
 * warps' waits run out without any invalid input. Process-wide; applies to calls launched after it.
 */
NBX_API void nbx_set_decode_wait_test(unsigned long long wait_limit_ns, unsigned long long producer_delay_ns);

/* A static, human-readable name for an nbx_status value. */
NBX_API const char* nbx_status_string(int status);

/* ABI version of this header (major * 100 + minor). */
NBX_API int nbx_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NBX_H */
