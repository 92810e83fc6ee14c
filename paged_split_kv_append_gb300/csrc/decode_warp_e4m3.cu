// Instantiations of the one-warp partial kernel for E4M3 pools with score modifications.
#include "decode_warp.cuh"

namespace nbx {

cudaError_t decode_dispatch_warp_e4m3(const DecodeParams& p, int q_dtype, int grid_limit, cudaStream_t stream) {
  return q_dtype == NBX_F32 ? launch_warp_d<E4M3, F32, kScoreMod>(p, grid_limit, stream)
                            : launch_warp_d<E4M3, BF16, kScoreMod>(p, grid_limit, stream);
}

}  // namespace nbx
