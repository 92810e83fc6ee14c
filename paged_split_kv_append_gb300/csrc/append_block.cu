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
// conversion, so the floor is the new values in and their codes out. One group of warps takes one
// (block, KV head, K or V): D / 8 lanes to a position, 8 elements a lane (one 16-byte load of bf16, two of
// fp32; one 8-byte store of codes). Items are ordered KV head fastest, as
// the new tokens lie in memory, so the groups running side by side read whole lines. The grid is what the
// GPU holds at once, one CTA of it without items; a group looks its next item up while the values of the
// current one are on their way (one item a group and as many CTAs as items took 51 us for 30 thousand bf16
// tokens of 4 heads of 256, two thirds of it the chain of lookups before the first value).
//
// Which block an item is: sequence b owns the flat indices from tok_start[b] / T + 2 b on. Its n new
// tokens touch at most n / T + 2 blocks, so the ranges do not meet, the grid needs no device-side
// count, and a warp finds its sequence with a 32-way search over the batch.
#include <atomic>
#include <climits>

#include "nbx_device.cuh"
#include "nbx_internal.h"

namespace nbx {
namespace {

// Positions a warp holds: 16 of up to 128 elements, or 8 of 256 (32 registers of bf16 values, 64 of fp32).
constexpr int warp_rows(int d) { return d <= 128 ? 16 : 8; }
constexpr int kMostWarps = 16;   // warps of a CTA: 8, or as many as a block needs (128 positions of 256: 16)

// 8 elements of the new tokens: bf16 pairs as they are, or floats
template <class In>
struct Eight;
template <>
struct Eight<BF16> {
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  // The largest magnitude, as the bits of a float (an infinity or NaN: their bits), two elements at a time.
  __device__ __forceinline__ uint32_t amax() const {
    constexpr uint32_t kMag = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag));
    return max(m & 0xffff0000u, m << 16);
  }
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
  __device__ __forceinline__ uint32_t amax() const {
    float x[8];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

template <class E>
__device__ __forceinline__ uint32_t finite_amax(const E& x) {
  float f[8];
  x.get(f);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = __float_as_uint(f[e]) & 0x7fffffffu;
    m = max(m, a < 0x7f800000u ? a : 0u);
  }
  return m;
}

// Eight floats to E4M3 codes: round to nearest even, saturating, NaN stays NaN.
__device__ __forceinline__ uint2 to_codes(const float* x, float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(unpack2(mul2(pack2(x[2 * i], x[2 * i + 1]), pack2(mul, mul))), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The same of x / s. With a power of two the quotient is a product, exactly; a held scale that another program wrote
// may be anything, and x * (1 / s) would round twice (codes beside a tie between two of them came out the other way).
__device__ __forceinline__ uint2 divided_codes(float* x, float s, float inv, bool power) {
  if (!power) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
    inv = 1.f;
  }
  return to_codes(x, inv);
}

// The smallest power of two S in [2^-48, 2^48] with amax <= 448 S, from amax's bits (finite, >= 0):
// 448 = 1.75 * 2^8, so S = 2^(e - 8) for a significand up to 1.75, else 2^(e - 7).
__device__ __forceinline__ float need_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;   // a subnormal amax gives -127: clamped below
  int k = e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = min(kMaxScaleLog2, max(-kMaxScaleLog2, k));
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// One item: a block of one (KV head, K or V) that gets new tokens. Everything but its values.
struct BlockItem {
  int start;          // the block's first position, and the positions the sequence held and holds
  int held, end;
  int src_row;        // row of the new tokens that position 0 would have
  int head, in_page;  // page * h_kv + KV head fits 31 bits: a page of a head is 1 KB or more
  int h, which;       // 0: K, 1: V
  bool on;
};

__device__ __forceinline__ BlockItem find_item(const AppendBlockParams& p, int64_t item) {
  const int lane = threadIdx.x & 31;
  BlockItem it;
  const int64_t fw = item / p.h_kv;
  it.h = static_cast<int>(item - fw * p.h_kv);
  it.which = static_cast<int>(fw & 1);
  const int64_t flat = fw >> 1;
  it.on = flat < p.n_flat;
  // ---- the sequence: the last b with tok_start[b] / T + 2 b <= flat
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const bool below = b < hi && static_cast<int64_t>(p.tok_start[b] >> p.scale_shift) + 2 * static_cast<int64_t>(b) <= flat;
    const uint32_t m = __ballot_sync(0xffffffffu, below);
    const int k = m == 0 ? 0 : 31 - __clz(m);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int t0 = p.tok_start[b], t1 = p.tok_start[b + 1];
  it.held = p.lens[b];
  it.src_row = t0 - it.held;
  const int64_t end = static_cast<int64_t>(it.held) + t1 - t0;
  const int64_t k_blk = flat - (static_cast<int64_t>(t0 >> p.scale_shift) + 2 * static_cast<int64_t>(b));
  const bool sane = t0 >= 0 && t1 >= t0 && t1 <= p.n_tok && it.held >= 0 && end <= INT_MAX - 128;
  it.end = sane ? static_cast<int>(end) : 0;
  const bool speaks = lane == 0 && it.h == 0 && it.which == 0;   // one warp of a group or more: the bits are the same
  if (it.on && !sane && speaks) raise_status(p.status, NBX_DEV_BAD_LEN);
  const int64_t start = ((it.held >> p.scale_shift) + k_blk) << p.scale_shift;
  it.on = it.on && sane && k_blk >= 0 && t1 > t0 && start < end;
  it.start = it.on ? static_cast<int>(start) : 0;
  int page = 0;
  const int pi = it.start / p.page_tokens;
  if (it.on) {
    if (pi >= p.max_pages) {
      if (speaks) raise_status(p.status, NBX_DEV_BAD_LEN);
      it.on = false;
    } else {
      page = p.block_table[static_cast<int64_t>(b) * p.max_pages + pi];
      if (page < 0 || page >= p.num_pages) {
        if (speaks) raise_status(p.status, NBX_DEV_BAD_PAGE);
        it.on = false;
        page = 0;
      }
    }
  }
  it.head = page * p.h_kv + it.h;
  it.in_page = it.start - pi * p.page_tokens;
  return it;
}

template <class In, int D>
__global__ void __launch_bounds__(D <= 128 ? 256 : 512) __maxnreg__(In::kBytes == 2 ? 80 : 128)
    append_block_kernel(AppendBlockParams p) {
  constexpr int kWarpRows = warp_rows(D);
  constexpr int kLpr = D / 8;                     // lanes to a position
  constexpr int kRpp = 32 / kLpr;                 // positions a warp takes at a time
  constexpr int kPasses = kWarpRows / kRpp;
  __shared__ uint32_t s_amax[2][kMostWarps];
  pdl_launch_dependents();   // the kernels of this library wait for this grid before they read the pools
  if (blockIdx.x == gridDim.x - 1) {
    // Ranges that do not ascend hide sequences from the search, and parts of others: said here, by a CTA without items.
    // (Beside them, before their loop or behind it, the question took 1.5 to 1.8 us of a call of 35.)
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
      if (p.tok_start[b + 1] < p.tok_start[b]) raise_status(p.status, NBX_DEV_BAD_LEN);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.scale_tokens;
  const int gw = T / kWarpRows;                   // warps of a group: 1, 2, 4, 8 or 16
  const int group = warp / gw, wg = warp - group * gw;
  const int per_cta = static_cast<int>(blockDim.x >> 5) / gw;
  const int sub = lane / kLpr, col = (lane - sub * kLpr) * 8;
  const int64_t items = p.n_flat * 2 * p.h_kv;
  const int64_t stride = static_cast<int64_t>(gridDim.x - 1) * per_cta;
  int64_t item = static_cast<int64_t>(blockIdx.x) * per_cta + group;
  BlockItem next = find_item(p, item);
  // (the loop's length is the group's own: its warps leave together, and its barrier is its own)
  for (int round = 0; item < items; ++round) {
    const BlockItem it = next;
    const int64_t slot = static_cast<int64_t>(it.head) * (p.page_tokens >> p.scale_shift) + (it.in_page >> p.scale_shift);
    uint8_t* const pool = static_cast<uint8_t*>(it.which ? p.v_pool : p.k_pool);
    float* const scale = (it.which ? p.v_scales : p.k_scales) + slot;
    const bool begins = it.held <= it.start;      // no position of the block is held already
    const float was = it.on && !begins ? *scale : 1.f;
    // ---- the new values, in registers; while they are on their way, the next item is looked up
    // (every address of a lane is one product and a step of its own: with each worked out anew, and every position
    // asked whether it is new, the kernel issued 14 instructions a value, and 30 thousand tokens took 40 us)
    const int pos0 = it.start + wg * kWarpRows + sub;   // this lane's first position
    const char* const src = static_cast<const char*>(it.which ? p.new_v : p.new_k) +
                            (static_cast<int64_t>(it.src_row + pos0) * p.h_kv + it.h) * (D * In::kBytes) + col * In::kBytes;
    const int64_t step = static_cast<int64_t>(p.h_kv) * (kRpp * D * In::kBytes);
    // every position of the warp is new (for the whole warp alike)
    const bool whole = it.on && it.start + wg * kWarpRows >= it.held && it.start + (wg + 1) * kWarpRows <= it.end;
    Eight<In> x[kPasses];
    if (whole) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) x[i].load(src + i * step);
    } else {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int pos = pos0 + i * kRpp;
        if (it.on && pos >= it.held && pos < it.end) x[i].load(src + i * step);
        else x[i].zero();
      }
    }
    item += stride;
    if (item < items) next = find_item(p, item);
    // ---- their largest finite magnitude
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) amax = max(amax, x[i].amax());
    if (amax >= 0x7f800000u) {   // infinities and NaN do not set the scale: look at the others alone
      amax = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) amax = max(amax, finite_amax(x[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (gw > 1) {
      uint32_t* const s = s_amax[round & 1];   // two in turn: the last round's may still be read
      if (lane == 0) s[warp] = amax;
      named_bar_sync(1 + group, gw * 32);   // at most 8 groups of two warps and more
      for (int w = 0; w < gw; ++w) amax = max(amax, s[group * gw + w]);
    }
    if (!it.on) continue;

    // ---- the block's scale
    const float need = need_scale(amax);
    const bool was_ok = was >= kMinScale && was <= kMaxScale;   // false for NaN
    if (!was_ok && lane == 0 && wg == 0) raise_status(p.status, NBX_DEV_BAD_SCALE);
    const float s = begins || !was_ok ? need : fmaxf(was, need);
    const float inv = 1.f / s;
    const bool power = (__float_as_uint(s) & 0x7fffffu) == 0;   // as every scale written here
    const bool again = !begins && was_ok && s > was;
    const float ratio = was / s;
    uint8_t* const to = pool + (static_cast<int64_t>(it.head) * p.page_tokens + it.in_page + wg * kWarpRows + sub) * D + col;
    if (wg == 0 && lane == 0) *scale = s;
    if (whole) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        float f[8];
        x[i].get(f);
        *reinterpret_cast<uint2*>(to + i * (kRpp * D)) = divided_codes(f, s, inv, power);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int pos = pos0 + i * kRpp;
      uint2* dst = reinterpret_cast<uint2*>(to + i * (kRpp * D));
      if (pos >= it.held && pos < it.end) {
        float f[8];
        x[i].get(f);
        *dst = divided_codes(f, s, inv, power);
      } else if (again && pos < it.held) {
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
  }
}

template <class In, int D>
cudaError_t launch_d(const AppendBlockParams& p, cudaStream_t stream) {
  const int gw = p.scale_tokens / warp_rows(D);
  const int warps = gw > 8 ? gw : 8;
  static std::atomic<int> resident[64][2];   // CTAs an SM holds, by device and size: asked once
  const DeviceInfo& di = device_info();
  std::atomic<int>& kept = resident[di.device & 63][warps > 8];
  int per_sm = kept.load();
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, append_block_kernel<In, D>, warps * 32, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    kept.store(per_sm);
  }
  const int64_t items = p.n_flat * 2 * p.h_kv;
  const int per = warps / gw;   // items of a CTA at a time
  int64_t grid = (items + per - 1) / per;
  const int64_t most = static_cast<int64_t>(di.sm_count) * per_sm - 1;
  if (grid > most) grid = most < 1 ? 1 : most;
  append_block_kernel<In, D><<<static_cast<unsigned>(grid) + 1, warps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class In>
cudaError_t launch(const AppendBlockParams& p, cudaStream_t stream) {
  if (p.d == 64) return launch_d<In, 64>(p, stream);
  if (p.d == 128) return launch_d<In, 128>(p, stream);
  return launch_d<In, 256>(p, stream);
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
  if (static_cast<int64_t>(num_pages) * h_kv > 0x7fffffffll) return NBX_ERR_SHAPE;
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
  while ((1 << p.scale_shift) < scale_tokens) ++p.scale_shift;
  p.n_flat = static_cast<int64_t>(n_tok) / scale_tokens + 2 * static_cast<int64_t>(batch);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = new_dtype == NBX_F32 ? launch<F32>(p, st) : launch<BF16>(p, st);
  return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
}
