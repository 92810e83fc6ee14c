// Instantiations of the split-KV partial kernel for F32 pools, with score modifications (query fp32 / bf16, head dim 64 / 128 / 256).
#include "decode_kernels.cuh"

namespace nbx {
NBX_DECODE_FOR_POOL(F32_mod, F32, kScoreMod)
}  // namespace nbx
