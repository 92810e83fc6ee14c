// Instantiations of the one-warp partial kernel for block-scaled pools.
#include "decode_warp.cuh"

namespace nbx {

cudaError_t decode_dispatch_warp_block(const DecodeParams& p, int q_dtype, bool mod, int grid_limit, cudaStream_t stream) {
  constexpr int kBoth = kScoreMod | kBlockScaled;
  if (q_dtype == NBX_F32)
    return mod ? launch_warp_d<E4M3, F32, kBoth>(p, grid_limit, stream)
               : launch_warp_d<E4M3, F32, kBlockScaled>(p, grid_limit, stream);
  return mod ? launch_warp_d<E4M3, BF16, kBoth>(p, grid_limit, stream)
             : launch_warp_d<E4M3, BF16, kBlockScaled>(p, grid_limit, stream);
}

}  // namespace nbx
