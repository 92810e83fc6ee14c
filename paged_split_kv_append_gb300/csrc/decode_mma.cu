// Instantiations of the tensor-core partial kernel for plain decodes, and when a decode runs it.
#include "decode_mma.cuh"

namespace nbx {

bool mma_path_applies(const DecodeParams& p, int q_dtype, int pool_dtype) {
  const int64_t pool_rows = static_cast<int64_t>(p.num_pages) * p.h_kv * p.page_tokens;
  return q_dtype == NBX_BF16 && (pool_dtype == NBX_BF16 || pool_dtype == NBX_E4M3) && (p.d == 128 || p.d == 256) &&
         (p.page_tokens % kMmaN) == 0 && p.group <= kMmaM && p.rows * p.group >= 64 &&
         pool_rows < (int64_t{1} << 31) - kMmaN && p.qk_scale_log2 > 0.f;
}

bool mma_path_applies_modified(const DecodeParams& p, int q_dtype, int pool_dtype) {
  return mma_path_applies(p, q_dtype, pool_dtype) && (pool_dtype == NBX_BF16 || p.out_bf16);
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
