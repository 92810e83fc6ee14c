// Causal attention over packed prompts with grouped heads.
#include "nbx_internal.h"
#include "prompt_row.cuh"

namespace nbx {
namespace {

constexpr int kRowThreads = 128;

// One warp per (token, query head).
template <int D>
__global__ void __launch_bounds__(kRowThreads) prompt_rows_kernel(PromptParams p) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / p.h_q;
  const int h = static_cast<int>(w - t * p.h_q);
  if (w == 0 && (threadIdx.x & 31) == 0)
    for (int b = 0; b < p.batch; ++b)
      if (p.seq_start[b] < 0 || p.seq_start[b + 1] < p.seq_start[b] || p.seq_start[b + 1] > p.n_tok)
        raise_status(p.status, NBX_DEV_BAD_LEN);
  if (t >= p.n_tok) return;
  int b = 0;
  while (b < p.batch && !(p.seq_start[b] >= 0 && p.seq_start[b + 1] <= p.n_tok && p.seq_start[b] <= t && t < p.seq_start[b + 1])) ++b;
  if (b == p.batch) return;
  const int64_t first = p.seq_start[b];
  const int hk = h / (p.h_q / p.h_kv);
  prompt_row<D>(static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + static_cast<int64_t>(h) * D,
                static_cast<const __nv_bfloat16*>(p.k) + first * p.k_stride + static_cast<int64_t>(hk) * D,
                static_cast<const __nv_bfloat16*>(p.v) + first * p.v_stride + static_cast<int64_t>(hk) * D, p.k_stride,
                p.v_stride, static_cast<int>(t - first) + 1, p.scale_log2,
                static_cast<__nv_bfloat16*>(p.out) + (t * p.h_q + h) * D);
}

}  // namespace

cudaError_t prompt_dispatch(const PromptParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.n_tok) * p.h_q + kRowThreads / 32 - 1) / (kRowThreads / 32));
  if (p.d == 64) prompt_rows_kernel<64><<<grid, kRowThreads, 0, stream>>>(p);
  else if (p.d == 128) prompt_rows_kernel<128><<<grid, kRowThreads, 0, stream>>>(p);
  else prompt_rows_kernel<256><<<grid, kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nbx
