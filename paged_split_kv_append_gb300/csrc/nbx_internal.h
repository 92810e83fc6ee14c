// Host-side internals of libnbx: launch parameter blocks, the workspace layout and the
// per-device launch facts. Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "nbx.h"

namespace nbx {

constexpr float kLog2eHost = 1.4426950408889634f;

struct DeviceInfo {
  int device;
  int sm_count;
  int max_smem_optin;
};

// Facts of the current device, queried once per device.
const DeviceInfo& device_info();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---------------------------------------------------------------- block-scaled pools
// Scales of an E4M3 pool's blocks lie in [2^-48, 2^48]. With every ratio of two scales inside 2^96, the
// weights p * v_scale of one row's softmax keep their order in fp32 with 2^30 to spare.
constexpr int kMaxScaleLog2 = 48;
constexpr float kMaxScale = 281474976710656.f;   // 2^48
constexpr float kMinScale = 1.f / 281474976710656.f;

// Positions a scale covers: 16, 32, 64 or 128, and a page holds a whole number of such blocks.
inline bool scale_tokens_ok(int t, int page_tokens) {
  return (t == 16 || t == 32 || t == 64 || t == 128) && page_tokens % t == 0;
}

struct AppendBlockParams {
  const void* new_k;
  const void* new_v;
  void* k_pool;
  void* v_pool;
  float* k_scales;
  float* v_scales;
  const int32_t* block_table;
  const int32_t* lens;
  const int32_t* tok_start;
  int32_t* status;
  int n_tok, h_kv, d, num_pages, page_tokens, max_pages, batch, scale_tokens;
  int scale_shift;  // log2 of scale_tokens
  int64_t n_flat;   // flat block indices: n_tok / T + 2 batch
};

// ---------------------------------------------------------------- pages
struct CopyPagesParams {
  void* k_pool;
  void* v_pool;
  float* k_scales;
  float* v_scales;
  const int32_t* moves;
  const int32_t* n_moves;
  int32_t* status;
  int max_moves, num_pages, h_kv, page_tokens;
  int row_bytes;      // bytes of one position of one KV head
  int scale_tokens;
  int chunks;         // 4 KB pieces of one KV head's page
};

enum { kForkNone = 0, kForkShare = 1, kForkCopy = 2, kForkEmpty = 3 };

struct ForkParams {
  int32_t* block_table;
  int32_t* seq_lens;
  const int32_t* fork_src;
  const int32_t* fork_dst;
  int32_t* moves;
  int32_t* n_moves;
  int32_t* status;
  uint32_t* bitmap;     // [num_pages] bits: pages in use
  int4* row_info;       // [batch] {fork that overwrites the row, first fork that reads it, length, -}; n_fork: none
  int4* outcome;        // [n_fork] {kFork..., rank among the copies, length, fresh page}
  int32_t* fresh;       // [n_fork] free pages in ascending order
  int32_t* row_keep;    // [batch, max_pages] rows that are both read and overwritten, as they were
  int max_pages, batch, n_fork, num_pages, page_tokens;
  bool copies;          // the moves are copied by the kernel launched next
};

struct CompactParams {
  const int32_t* block_table;
  int32_t* new_block_table;
  const int32_t* seq_lens;
  int32_t* moves;
  int32_t* counts;
  int32_t* status;
  int32_t* fill;        // [num_pages] 1 + positions held, 0 for a free page
  int32_t* chunk_live;  // [n_chunks] pages in use per chunk
  int32_t* rank;        // [num_pages] move number of a page that moves
  int batch, max_pages, num_pages, page_tokens, max_moves, n_chunks;
};

struct AppendParams {
  const void* new_k;
  const void* new_v;
  void* k_pool;
  void* v_pool;
  const int32_t* slot_mapping;
  int32_t* status;
  int n_tok, h_kv, d, num_pages, page_tokens;
  float k_inv, v_inv;
  // decode-step mode (lens != null): token t = b * rows + r goes to position lens[b] + r of
  // sequence b, its page read from the block table; positions at or past max_pos are refused
  const int32_t* lens;
  const int32_t* block_table;
  int max_pages, rows, max_pos;
};

cudaError_t append_dispatch(const AppendParams& p, int new_dtype, int pool_dtype, cudaStream_t stream);

// The append with the position rotation; strides in elements between tokens.
struct RotateParams {
  const void* q;
  const void* new_k;
  const void* new_v;
  const float* cos_table;   // [n_pos, turned / 2]
  const float* sin_table;
  const int32_t* positions;
  const int32_t* slot_mapping;
  void* q_out;
  void* k_out;              // or null
  void* k_pool;
  void* v_pool;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int n_tok, h_q, h_kv, d, n_pos, turned, interleaved, num_pages, page_tokens;
  int slots;          // rows of a token: h_q + 2 h_kv
  int groups, block_groups, toks;   // set by the launch: groups of slots, of a CTA, tokens of a CTA at a time
  float k_inv, v_inv;
};

cudaError_t append_rotated_dispatch(const RotateParams& p, int new_dtype, int pool_dtype, cudaStream_t stream);

// Attention over packed prompts; strides in elements between tokens.
struct PromptParams {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* seq_start;   // [batch + 1]
  void* out;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride;
  int n_tok, h_q, h_kv, d, batch;
  float scale_log2;           // scale * log2(e)
  uint64_t wait_limit_ns;     // as DecodeParams'
  uint64_t producer_delay_ns;
};

cudaError_t prompt_dispatch(const PromptParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- decode
constexpr int kTileN = NBX_TILE_POSITIONS;  // positions per staged tile
constexpr int kQB = 4;                      // query vectors (rows x heads of one KV head) per work unit
constexpr int kConsumerWarps = 4;
constexpr int kDecodeThreads = (kConsumerWarps + 1) * 32;

// One sequence of the split plan.
struct SeqPlan {
  int32_t len;       // positions read (0 if the length was out of bounds)
  int32_t seg;       // positions per split (a whole number of pages)
  int32_t n_splits;  // non-empty splits: ceil(len / seg)
  int32_t first;     // first position of the first split (0 but with key ranges)
};

// One (sequence, split) of the work list; a work unit is (entry, KV head, row block). The
// sequence's length and split count ride along, so a unit is described by one 32-byte load.
struct Entry {
  int32_t b, s, start, end;
  int32_t len, n_splits, pad0, pad1;
};
static_assert(sizeof(Entry) == 32, "Entry is one 32-byte load");

// Byte offsets of the workspace sections (each 256-byte aligned).
struct WorkspaceLayout {
  // int32[64]: [0] entries in the list, [1] work counter; modified decodes: [2] what the merge has to do,
  // kMergeSplits if some sequence has more than one split and kMergeRedo if a partial is to be recomputed,
  // [3] (entry, M tile) pairs in `order` (0: none)
  size_t header;
  size_t ident_bt;  // int32[batch]: the identity block table of a contiguous cache (row b = page b)
  size_t plan;      // SeqPlan[batch]
  size_t entries;   // Entry[batch * max_splits]
  size_t m_part;    // f32[batch * rows * h_q * max_splits]   (log2 units)
  size_t l_part;    // f32[batch * rows * h_q * max_splits]
  size_t acc_part;  // f32[batch * rows * h_q * max_splits * d]
  size_t ranges;    // int2[batch * M tiles of 128 vectors]: modified decodes only
  size_t order;     // int32[kOrderMax]: modified decodes only
  size_t total;
  int max_splits;
  int row_blocks;
};

// Returns false if the sizes overflow. modified: for the modified decodes, whose splits may be as short as 64
// positions (the kernels on the tensor cores size them by the whole call's work).
bool workspace_layout(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len, WorkspaceLayout* out,
                      bool modified = false);

int splits_for(int length);

struct DecodeParams {
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  float* out;
  int32_t* status;
  // workspace sections
  int32_t* header;
  SeqPlan* plan;
  Entry* entries;
  float* m_part;
  float* l_part;
  float* acc_part;
  int batch, rows, h_q, h_kv, group, d, num_pages, page_tokens, max_pages, max_seq_len;
  int max_splits, row_blocks;
  float qk_scale_log2;  // scale * k_scale * log2(e): scores in log2 units
  float v_scale;
  // the plan kernel writes ident_bt[b] = b (a contiguous cache read as one page per sequence;
  // block_table then points at it), and, for a decode step, attends with seq_lens[b] + len_add
  // and writes that length to lens_out[b] (null: neither)
  int32_t* ident_bt;
  int32_t* lens_out;
  int len_add;
  // fraction of the split partials' lines written with an L2 evict-last policy: about 64 MB of them
  // stay resident for the merge (1 when they all fit)
  float keep_frac;
  // the SIMT partial kernel's wait bound, and a delay before its producer warp starts (0 in normal
  // use); set only through nbx_set_decode_wait_test, to make a bounded wait run out on purpose
  uint64_t wait_limit_ns;
  uint64_t producer_delay_ns;
  // fixed-shift softmax on the tensor-core kernel (null: the online max everywhere): per query vector
  // |q| [batch * rows * h_q], per (sequence, KV head) {max |k| * k_scale, max |v| * v_scale}, and
  // scale * log2(e)
  const float* fs_q_norm;
  const float* fs_kv_max;
  float fs_scale_log2;
  float k_scale_host;   // the pool's k scale (the bounds kernel reports |k| dequantised)
  // split partials as f16 acc / l (the partial normalised by its own sum) instead of fp32 acc: set
  // for fp8 pools on tensor cores, where acc / l is a convex combination of E4M3 codes (|code|
  // <= 448, the v scale is applied by the merge), so f16 neither overflows nor loses more than
  // 2^-11 relative; each (row, split) slot holds d halves in the first half of its d floats
  int part_f16;
  // split plan for a tensor-core window or the one-warp kernel (0: the pages' rule, ceil(len / 256) splits of at most 64):
  // about tc_units work units in all, each of the tc_pairs (KV head, M tile) pairs of a sequence
  // taking floor(tc_units * len / (tc_pairs * sum of lens)) splits, clamped to [1, min(max_splits,
  // len / 64)]
  int tc_units;
  int tc_pairs;
  int tc_warps;      // warps that take units, of the one-warp kernel
  int tc_round_up;   // splits rounded up instead of down (units taken from the counter by single warps)
  // ---- read only by the kernels of the modified and block-scaled decodes (kScoreMod, kBlockScaled)
  int out_bf16;            // the output is bf16, rounded once from the fp32 result
  float cap_log2;          // softcap * log2(e), and its reciprocal; 0: no cap
  float cap_inv;
  int cap_folds;           // qk_scale_log2 * cap_inv and the cap are near enough to 1 for a product with the ninth power
  const float* slopes;     // [h_q] bias per position of distance, or null
  const int32_t* key_begin;   // [batch, rows] first visible key and one past the last, or null (0, p + 1)
  const int32_t* key_end;
  const float* k_scales;   // [num_pages, h_kv, page_tokens / scale_tokens]
  const float* v_scales;
  int scale_shift;         // log2 of the positions per scale
  int2* ranges;            // [batch, range_tiles] keys the rows of a sequence's M tile see (SIMT: of the sequence)
  int range_tiles;
  int32_t* order;          // header[3] > 0: that many (entry, M tile) = entry * range_tiles + tile, most keys first
  int pool_e4m3;           // the pools are E4M3 (else bf16): what a recomputed partial of a window reads
};

// What a decode adds to the plain one, as a template argument of its kernels: score modifications (a cap,
// a bias by distance, per-row key ranges), pools with a scale per block. Plain calls run instantiations
// without any of it.
constexpr int kScoreMod = 1;
constexpr int kBlockScaled = 2;
// Of the tensor-core kernel's score modifications, beside the key ranges of kScoreMod: a cap, a bias by distance.
constexpr int kCapped = 4;
constexpr int kSloped = 8;

// The visible keys of query row r of a sequence of len positions: [lo, hi), empty as lo = hi = 0.
struct KeyRange {
  int lo, hi;
};
#ifdef __CUDACC__
__device__ __forceinline__ KeyRange key_range(const DecodeParams& p, int b, int r, int len) {
  const int64_t i = static_cast<int64_t>(b) * p.rows + r;
  const int lo = p.key_begin ? max(0, p.key_begin[i]) : 0;
  const int hi = min(len, p.key_end ? p.key_end[i] : len - p.rows + r + 1);
  return hi > lo ? KeyRange{lo, hi} : KeyRange{0, 0};
}
#endif

cudaError_t bounds_dispatch(const DecodeParams& p, int q_dtype, int pool_dtype, float* q_norm, float* kv_max,
                            cudaStream_t stream);

// x: 0, or kScoreMod and kBlockScaled bits of a modified decode
cudaError_t decode_dispatch(const DecodeParams& p, int q_dtype, int pool_dtype, int x, int grid_limit,
                            cudaStream_t stream);

// The tensor-core partial kernel: used when the query vectors of one KV head fill an MMA tile
// (rows x group >= 64), q is bf16, the pools bf16 (kind::f16) or E4M3 (kind::f8f6f4 on the codes),
// d is 128 or 256 and pages hold a multiple of 64 positions.
bool mma_path_applies(const DecodeParams& p, int q_dtype, int pool_dtype);
constexpr int kMmaRowsPerTile = 128;   // query vectors of one M tile of the tensor-core kernel
constexpr int kOrderMax = 512;         // (entry, M tile) pairs that the plan kernel sorts by their keys
cudaError_t decode_dispatch_mma(const DecodeParams& p, int pool_dtype, int grid_limit, cudaStream_t stream);
// The same for modified decodes. An E4M3 window holds P to 2^-8, which only a bf16 output may take.
bool mma_path_applies_modified(const DecodeParams& p, int q_dtype, int pool_dtype);
cudaError_t decode_dispatch_mma_mod(const DecodeParams& p, int pool_dtype, int grid_limit, cudaStream_t stream);
cudaError_t decode_dispatch_mma_block(const DecodeParams& p, bool mod, int grid_limit, cudaStream_t stream);
// The one-warp partial kernel of modified decodes with few query vectors: E4M3 pools, bf16 pools under bf16
// queries. Its work units cover kWarpUnitVectors query vectors of a KV head; warps resident on an SM for the
// sizes of a call (what its splits are sized by).
constexpr int kWarpUnitVectors = 8;
inline bool warp_path_applies(int q_dtype, int pool_dtype) {
  return pool_dtype == NBX_E4M3 || (pool_dtype == NBX_BF16 && q_dtype == NBX_BF16);
}
constexpr int warp_path_warps(int pool_dtype, int d) {
  return d == 64 ? 16 : (d == 128 ? 12 : (pool_dtype == NBX_E4M3 ? 8 : 6));
}
cudaError_t decode_dispatch_warp_bf16(const DecodeParams& p, int grid_limit, cudaStream_t stream);
cudaError_t decode_dispatch_warp_e4m3(const DecodeParams& p, int q_dtype, int grid_limit, cudaStream_t stream);
cudaError_t decode_dispatch_warp_block(const DecodeParams& p, int q_dtype, bool mod, int grid_limit, cudaStream_t stream);
constexpr int kMergeSplits = 1, kMergeRedo = 2;   // header[2]
// m of a partial that the merge has to recompute: a NaN no computation gives
constexpr uint32_t kRedoBits = 0x7fffbad0u;

// Launch with programmatic dependent launch: the grid may start while the previous kernel in the
// stream finishes; the kernel orders itself after it with griddepcontrol.wait.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- shared prefixes
// What the plan says of a group: its first sequence, their number, positions shared (whole pages), positions of a split
// of them and their number, M tile pairs of its query vectors, its first work unit, the row of the block table that
// names the pages.
struct PrefixGroup {
  int32_t b0, n, eff, seg, splits, pairs, unit, row;
};

struct SharedParams {
  const int32_t* group_start;   // [n_groups + 1]
  const int32_t* shared_lens;   // [n_groups]
  int n_groups;
  // workspace
  int2* seqs;                   // [batch] positions read with the group, splits of them (the plan's scratch)
  PrefixGroup* groups;          // [n_groups]
};

struct SharedLayout {
  size_t header, plan, entries, m_part, l_part, acc_part, seqs, groups, total;
  int max_splits;
};
bool shared_layout(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len, int n_groups, SharedLayout* out);
// Whether prefixes are read apart for these formats; elsewhere a call is a decode that ignores its groups.
bool prefix_path_applies(int q_dtype, int pool_dtype);
cudaError_t shared_dispatch(const SharedParams& s, const DecodeParams& p, int q_dtype, int pool_dtype, int grid_limit,
                            cudaStream_t stream);

struct MergeParams {
  const float* acc_part;
  const float* m_part;
  const float* l_part;
  float* out;
  int n_rows, splits, d;
};

cudaError_t merge_dispatch(const MergeParams& p, cudaStream_t stream);

}  // namespace nbx
