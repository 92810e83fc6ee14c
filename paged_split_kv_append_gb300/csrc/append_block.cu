// Block-scaled append: new tokens into an E4M3 pool that holds one scale per T positions of a page
// and KV head (nbx_paged_kv_append_block_scaled).
//
// For a block with new tokens: amax = max |x| over the finite values of its new tokens, need = the
// smallest power of two with amax <= 448 need, S = need if the block begins with this call, else
// max(S_old, need). New codes are e4m3(x / S); codes already held are requantised to
// e4m3(c * S_old / S) when S grows. With a power of two both the division and that ratio are exact, so
// a held code changes only if it falls under 2^-6, E4M3's subnormals. (amax / 448 itself would round
// every held code again at each growth, and keeps no more bits: E4M3's spacing is relative.)
//
// The work is bytes only: each value is read once and held in registers between the amax and the
// conversion, so the floor is the new values in and their codes out. One group of T / 16 warps takes one
// (block, KV head, K or V): a warp holds 16 positions, D / 8 lanes to a position, 8 elements a lane (one
// 16-byte load of bf16, two of fp32; one 8-byte store of codes). Items are ordered KV head fastest, as
// the new tokens lie in memory, so the groups running side by side read whole lines.
//
// Which block an item is: sequence b owns the flat indices from tok_start[b] / T + 2 b on. Its n new
// tokens touch at most n / T + 2 blocks, so the ranges do not meet, the grid needs no device-side
// count, and a warp finds its sequence with a 32-way search over the batch.
#include "nbx_device.cuh"
#include "nbx_internal.h"

namespace nbx {
namespace {

constexpr int kBlockWarps = 8;       // warps per CTA
constexpr int kWarpRows = 16;        // positions a warp holds

// 8 elements of the new tokens: bf16 pairs as they are, or floats
template <class In>
struct Eight;
template <>
struct Eight<BF16> {
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Eight<F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const char* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// Eight floats to E4M3 codes: round to nearest even, saturating, NaN stays NaN.
__device__ __forceinline__ uint2 to_codes(const float* x, float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * mul, x[2 * i + 1] * mul), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The smallest power of two S in [2^-48, 2^48] with amax <= 448 S, from amax's bits (finite, >= 0):
// 448 = 1.75 * 2^8, so S = 2^(e - 8) for a significand up to 1.75, else 2^(e - 7).
__device__ __forceinline__ float need_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;   // a subnormal amax gives -127: clamped below
  int k = e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = min(kMaxScaleLog2, max(-kMaxScaleLog2, k));
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

template <class In, int D>
__global__ void __launch_bounds__(kBlockWarps * 32) append_block_kernel(AppendBlockParams p) {
  constexpr int kLpr = D / 8;                     // lanes to a position
  constexpr int kRpp = 32 / kLpr;                 // positions a warp takes at a time
  constexpr int kPasses = kWarpRows / kRpp;
  __shared__ uint32_t s_amax[kBlockWarps];
  pdl_launch_dependents();   // the kernels of this library wait for this grid before they read the pools
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.scale_tokens;
  const int gw = T / kWarpRows;                   // warps of a group: 1, 2, 4 or 8
  const int group = warp / gw, wg = warp - group * gw;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kBlockWarps / gw) + group;
  const int64_t fw = item / p.h_kv;
  const int h = static_cast<int>(item - fw * p.h_kv);
  const int which = static_cast<int>(fw & 1);     // 0: K, 1: V
  const int64_t flat = fw >> 1;

  // ---- the sequence: the last b with tok_start[b] / T + 2 b <= flat
  bool on = flat < p.n_flat;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const bool below = b < hi && static_cast<int64_t>(p.tok_start[b]) / T + 2 * static_cast<int64_t>(b) <= flat;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    const int k = m == 0 ? 0 : 31 - __clz(m);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int t0 = p.tok_start[b], t1 = p.tok_start[b + 1];
  const int64_t held = p.lens[b];                 // positions the sequence held before
  const int64_t end = held + (static_cast<int64_t>(t1) - t0);
  const int64_t k_blk = flat - (static_cast<int64_t>(t0) / T + 2 * static_cast<int64_t>(b));
  const bool sane = t0 >= 0 && t1 >= t0 && t1 <= p.n_tok && held >= 0;
  if (on && !sane && lane == 0 && h == 0 && which == 0) raise_status(p.status, NBX_DEV_BAD_LEN);
  const int64_t start = sane && k_blk >= 0 ? (held / T + k_blk) * T : 0;   // the block's first position
  on = on && sane && k_blk >= 0 && t1 > t0 && start < end;
  int page = 0;
  if (on) {
    const int64_t pi = start / p.page_tokens;
    if (pi >= p.max_pages) {
      if (lane == 0 && h == 0 && which == 0) raise_status(p.status, NBX_DEV_BAD_LEN);
      on = false;
    } else {
      page = p.block_table[static_cast<int64_t>(b) * p.max_pages + pi];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0 && h == 0 && which == 0) raise_status(p.status, NBX_DEV_BAD_PAGE);
        on = false;
      }
    }
  }
  const int64_t head = static_cast<int64_t>(page) * p.h_kv + h;
  const int in_page = static_cast<int>(start % p.page_tokens);
  uint8_t* const pool = static_cast<uint8_t*>(which ? p.v_pool : p.k_pool);
  float* const scale = (which ? p.v_scales : p.k_scales) + head * (p.page_tokens / T) + in_page / T;
  const bool begins = held <= start;              // no position of the block is held already
  const float was = on && !begins ? *scale : 1.f;

  // ---- the new values, in registers, and their largest finite magnitude
  const int sub = lane / kLpr, col = (lane - sub * kLpr) * 8;
  const char* src = static_cast<const char*>(which ? p.new_v : p.new_k);
  Eight<In> x[kPasses];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t pos = start + wg * kWarpRows + i * kRpp + sub;
    if (on && pos >= held && pos < end)
      x[i].load(src + ((t0 + (pos - held)) * p.h_kv + h) * D * In::kBytes + col * In::kBytes);
    else
      x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    float f[8];
    x[i].get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = __float_as_uint(f[e]) & 0x7fffffffu;
      amax = max(amax, a < 0x7f800000u ? a : 0u);   // infinities and NaN do not set the scale
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (gw > 1) {   // the same for the whole CTA
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();
    for (int w = 0; w < gw; ++w) amax = max(amax, s_amax[group * gw + w]);
  }
  if (!on) return;

  // ---- the block's scale
  const float need = need_scale(amax);
  const bool was_ok = was >= kMinScale && was <= kMaxScale;   // false for NaN
  if (!was_ok && lane == 0 && wg == 0) raise_status(p.status, NBX_DEV_BAD_SCALE);
  const float s = begins || !was_ok ? need : fmaxf(was, need);
  const float inv = 1.f / s;                      // exact for the powers of two written here
  const bool again = !begins && was_ok && s > was;
  const float ratio = was / s;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = wg * kWarpRows + i * kRpp + sub;
    const int64_t pos = start + row;
    uint2* dst = reinterpret_cast<uint2*>(pool + (head * p.page_tokens + in_page + row) * D + col);
    if (pos >= held && pos < end) {
      float f[8];
      x[i].get(f);
      *dst = to_codes(f, inv);
    } else if (again && pos < held) {
      const uint2 c = *dst;
      float f[8];
      const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 g = e4m3x2_to_float2(w[e]);
        f[2 * e] = g.x;
        f[2 * e + 1] = g.y;
      }
      *dst = to_codes(f, ratio);
    }
  }
  if (wg == 0 && lane == 0) *scale = s;
}

template <class In>
cudaError_t launch(const AppendBlockParams& p, cudaStream_t stream) {
  const int64_t items = p.n_flat * 2 * p.h_kv;
  const int per = kBlockWarps / (p.scale_tokens / kWarpRows);
  const int64_t grid = (items + per - 1) / per;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(grid);
  if (p.d == 64) append_block_kernel<In, 64><<<g, kBlockWarps * 32, 0, stream>>>(p);
  else if (p.d == 128) append_block_kernel<In, 128><<<g, kBlockWarps * 32, 0, stream>>>(p);
  else append_block_kernel<In, 256><<<g, kBlockWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace nbx

using namespace nbx;

extern "C" NBX_API int nbx_paged_kv_append_block_scaled(const void* new_k, const void* new_v, int new_dtype, int n_tok,
                                                        int h_kv, int d, void* k_pool, void* v_pool, float* k_scales,
                                                        float* v_scales, int scale_tokens, int num_pages,
                                                        int page_tokens, const int32_t* block_table, int max_pages,
                                                        int batch, const int32_t* lens, const int32_t* tok_start,
                                                        int32_t* status, void* stream) {
  if (n_tok < 0 || batch < 0 || h_kv < 1 || (d != 64 && d != 128 && d != 256) || num_pages < 1 || page_tokens < 1 ||
      max_pages < 1)
    return NBX_ERR_SHAPE;
  if (!scale_tokens_ok(scale_tokens, page_tokens)) return NBX_ERR_PAGE_ALIGN;
  if (new_dtype != NBX_F32 && new_dtype != NBX_BF16) return NBX_ERR_DTYPE;
  if (n_tok == 0 || batch == 0) return NBX_OK;
  if (!new_k || !new_v || !k_pool || !v_pool || !k_scales || !v_scales || !block_table || !lens || !tok_start)
    return NBX_ERR_NULL;
  if (!aligned16(new_k) || !aligned16(new_v) || !aligned16(k_pool) || !aligned16(v_pool)) return NBX_ERR_ALIGN;
  AppendBlockParams p = {};
  p.new_k = new_k;
  p.new_v = new_v;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_table = block_table;
  p.lens = lens;
  p.tok_start = tok_start;
  p.status = status;
  p.n_tok = n_tok;
  p.h_kv = h_kv;
  p.d = d;
  p.num_pages = num_pages;
  p.page_tokens = page_tokens;
  p.max_pages = max_pages;
  p.batch = batch;
  p.scale_tokens = scale_tokens;
  p.n_flat = static_cast<int64_t>(n_tok) / scale_tokens + 2 * static_cast<int64_t>(batch);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = new_dtype == NBX_F32 ? launch<F32>(p, st) : launch<BF16>(p, st);
  return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
}
