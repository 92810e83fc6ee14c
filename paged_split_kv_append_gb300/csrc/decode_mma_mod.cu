// Instantiations of the tensor-core partial kernel for decodes with score modifications.
#include "decode_mma.cuh"

namespace nbx {

cudaError_t decode_dispatch_mma_mod(const DecodeParams& p, int pool_dtype, int grid_limit, cudaStream_t stream) {
  if (pool_dtype == NBX_E4M3) {
    if (p.d == 128) return launch_mma_mod<128, true, kScoreMod>(p, grid_limit, stream);
    return launch_mma_mod<256, true, kScoreMod>(p, grid_limit, stream);
  }
  if (p.d == 128) return launch_mma_mod<128, false, kScoreMod>(p, grid_limit, stream);
  return launch_mma_mod<256, false, kScoreMod>(p, grid_limit, stream);
}

}  // namespace nbx
