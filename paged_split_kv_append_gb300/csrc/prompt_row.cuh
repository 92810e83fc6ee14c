// Causal attention of one query vector, key by key in fp32, by one warp; and which rows need it.
#pragma once

#include "nbx_device.cuh"

namespace nbx {

// out = sum_j e^(z_j - max z) v_j / sum_j e^(z_j - max z), z_j = scale (q . k_j), over keys 0 .. n - 1 (0 where no z_j
// is above -inf), rounded once to bf16. Keys 32 at a time: lane l scores key l of the block, then every lane gathers its
// D / 32 columns. k, v: key 0 of the head, rows `k_stride` and `v_stride` elements apart. c = scale * log2(e). Columns
// [col0, col1) are written.
template <int D>
__device__ __noinline__ void prompt_row(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                        int64_t k_stride, int64_t v_stride, int n, float c, __nv_bfloat16* out, int col0,
                                        int col1) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, acc[kCols];
#pragma unroll
  for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
  for (int n0 = 0; n0 < n; n0 += 32) {
    float z = -INFINITY;
    if (n0 + lane < n) {
      const uint4* kr = reinterpret_cast<const uint4*>(k + (n0 + lane) * k_stride);
      const uint4* qr = reinterpret_cast<const uint4*>(q);
      f32x2 s = pack2(0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        f32x2 a[4], b[4];
        unpack16x2<BF16>(__ldg(kr + i), a);
        unpack16x2<BF16>(__ldg(qr + i), b);
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma2(a[j], b[j], s);
      }
      const float2 t = unpack2(s);
      z = (t.x + t.y) * c;
    }
    float top = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m2 = max_nan(m, top);
    // No score yet: weights of 0, under which a NaN value still is one. (A loop of its own: weights against a reference of 0
    // instead cost the kernel of d = 256 a register that it spilled, and three prompts of 2000 to 4500 355 us for 346.)
    if (m2 == -INFINITY) {
      for (int j = n0; j < min(n0 + 32, n); ++j)
#pragma unroll
        for (int e = 0; e < kCols; e += 2) {
          const float2 x = bf16x2_to_float2(__ldg(reinterpret_cast<const uint32_t*>(v + j * v_stride + lane * kCols + e)));
          acc[e] = fmaf(0.f, x.x, acc[e]);
          acc[e + 1] = fmaf(0.f, x.y, acc[e + 1]);
        }
      continue;
    }
    const float f = fast_exp2(m - m2);
    const float w = n0 + lane < n ? fast_exp2(z - m2) : 0.f;
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = fmaf(l, f, sum);
    m = m2;
#pragma unroll
    for (int e = 0; e < kCols; ++e) acc[e] *= f;
    const int keys = min(32, n - n0);
    for (int j = 0; j < keys; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const __nv_bfloat16* vr = v + (n0 + j) * v_stride + lane * kCols;
#pragma unroll
      for (int e = 0; e < kCols; e += 2) {
        const float2 x = bf16x2_to_float2(__ldg(reinterpret_cast<const uint32_t*>(vr + e)));
        acc[e] = fmaf(wj, x.x, acc[e]);
        acc[e + 1] = fmaf(wj, x.y, acc[e + 1]);
      }
    }
  }
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < kCols; e += 2) {
    if (lane * kCols < col0 || lane * kCols >= col1) break;
    const __nv_bfloat162 h = m == -INFINITY ? __floats2bfloat162_rn(0.f, 0.f)
                                            : __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
    *reinterpret_cast<__nv_bfloat162*>(out + lane * kCols + e) = h;
  }
}

// The last of keys [lo, hi) whose value has an element among columns [col0, col1) that is not finite, or -1. A warp's work.
__device__ __noinline__ int last_not_finite(const __nv_bfloat16* v, int64_t v_stride, int lo, int hi, int col0, int col1) {
  const int chunks = (col1 - col0) / 8;
  int last = -1;
  for (int i = threadIdx.x & 31; i < (hi - lo) * chunks; i += 32) {
    const int key = lo + i / chunks, chunk = i % chunks;
    if (not_finite<false>(__ldg(reinterpret_cast<const uint4*>(v + key * v_stride + col0) + chunk))) last = key;
  }
  return __reduce_max_sync(0xffffffffu, last);
}

}  // namespace nbx
