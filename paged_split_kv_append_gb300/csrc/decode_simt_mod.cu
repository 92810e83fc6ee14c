// Instantiations of the split-KV partial kernel for decodes with score modifications: fp32 pools, and bf16 pools
// under fp32 queries (neither has exact operands for the tensor cores).
#include "decode_kernels.cuh"

namespace nbx {

cudaError_t decode_dispatch_simt_mod(const DecodeParams& p, int q_dtype, int pool_dtype, int grid_limit,
                                     cudaStream_t stream) {
  if (pool_dtype == NBX_BF16) return decode_dispatch_d<BF16, F32, kScoreMod>(p, grid_limit, stream);
  return q_dtype == NBX_F32 ? decode_dispatch_d<F32, F32, kScoreMod>(p, grid_limit, stream)
                            : decode_dispatch_d<F32, BF16, kScoreMod>(p, grid_limit, stream);
}

}  // namespace nbx
