// Instantiations of the one-warp partial kernel for bf16 pools under bf16 queries.
#include "decode_warp.cuh"

namespace nbx {

cudaError_t decode_dispatch_warp_bf16(const DecodeParams& p, int grid_limit, cudaStream_t stream) {
  return launch_warp_d<BF16, BF16, kScoreMod>(p, grid_limit, stream);
}

}  // namespace nbx
