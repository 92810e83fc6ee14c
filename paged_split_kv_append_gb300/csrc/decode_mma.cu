// Instantiations of the tensor-core partial kernel for plain decodes, and when a decode runs it.
#include "decode_mma.cuh"

namespace nbx {

// least: the fewest query vectors of a KV head
static bool window_applies(const DecodeParams& p, int q_dtype, int pool_dtype, int least) {
  const int64_t pool_rows = static_cast<int64_t>(p.num_pages) * p.h_kv * p.page_tokens;
  return q_dtype == NBX_BF16 && (pool_dtype == NBX_BF16 || pool_dtype == NBX_E4M3) && (p.d == 128 || p.d == 256) &&
         (p.page_tokens % kMmaN) == 0 && p.group <= kMmaM && p.rows * p.group >= least &&
         pool_rows < (int64_t{1} << 31) - kMmaN && p.qk_scale_log2 > 0.f;
}

bool mma_path_applies(const DecodeParams& p, int q_dtype, int pool_dtype) {
  return window_applies(p, q_dtype, pool_dtype, 64);
}

// A window costs the same whatever part of its 128 vectors is filled, the one-warp kernel reads the cache once for every
// 8 of them. Four sequences of 8192 positions, bf16: at d = 128 and 8 KV heads 32, 48 and 60 vectors take 59, 81 and 100
// us one-warp and 61 to 66 as windows; at d = 256 and 4 heads 24, 36 and 48 take 51, 76 and 93 and 49. (E4M3: 55, 75
// and 91, and 60 to 66; 44, 57 and 94, and 44.) An fp32 output keeps the one-warp kernel's exactness up to the plain
// decode's own limit.
bool mma_path_applies_modified(const DecodeParams& p, int q_dtype, int pool_dtype) {
  const int least = !p.out_bf16 ? 64 : (p.d == 256 ? 32 : 40);
  return window_applies(p, q_dtype, pool_dtype, least) && (pool_dtype == NBX_BF16 || p.out_bf16);
}

cudaError_t decode_dispatch_mma(const DecodeParams& p, int pool_dtype, int grid_limit, cudaStream_t stream) {
  if (pool_dtype == NBX_E4M3) {
    if (p.d == 128) return launch_mma<128, true>(p, grid_limit, stream);
    return launch_mma<256, true>(p, grid_limit, stream);
  }
  if (p.d == 128) return launch_mma<128, false>(p, grid_limit, stream);
  return launch_mma<256, false>(p, grid_limit, stream);
}

}  // namespace nbx
