// Instantiations of the tensor-core partial kernel for block-scaled pools.
#include "decode_mma.cuh"

namespace nbx {

cudaError_t decode_dispatch_mma_block(const DecodeParams& p, bool mod, int grid_limit, cudaStream_t stream) {
  if (p.d == 128)
    return mod ? launch_mma_mod<128, true, kScoreMod | kBlockScaled>(p, grid_limit, stream)
               : launch_mma_mod<128, true, kBlockScaled>(p, grid_limit, stream);
  return mod ? launch_mma_mod<256, true, kScoreMod | kBlockScaled>(p, grid_limit, stream)
             : launch_mma_mod<256, true, kBlockScaled>(p, grid_limit, stream);
}

}  // namespace nbx
