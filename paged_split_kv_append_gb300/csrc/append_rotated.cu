// The append with the position rotation on the way: queries and keys are turned by their positions, keys and
// values go to the paged cache.
//
// With the pair (a, b) of a head's vector (elements i and turned / 2 + i, or neighbours 2i and 2i + 1) and the angle
// whose cosine c and sine s row `position` of the tables holds at i:
//   a' = a c - b s,   b' = b c + a s          (fp32: a product and an FMA each, then one rounding on the store)
// Elements from `turned` on, and values, are only cast.
//
//  * What bounds it: bytes. A token's row of the tables serves all its heads, everything else is touched once.
//  * A work item is 16 elements of a row, two vectors of 8 that hold whole pairs: for halves the vectors lie
//    turned / 2 apart, for neighbours side by side. So every access is 16 bytes or more and no lane exchanges anything.
//  * A thread keeps its 8 cosines and sines in registers for kHeads heads, and has the loads of all of them in
//    flight before it turns the first.
#include <algorithm>

#include "nbx_device.cuh"
#include "nbx_internal.h"

namespace nbx {
namespace {

constexpr int kRotThreads = 512;   // at most
constexpr int kRotBlocks = 1;      // an SM, of a call with many tokens: more tokens a thread (4: 70 us, 2: 67.6, 1: 66.9)

// Eight consecutive elements as floats (address aligned to 16 bytes).
struct F8 {
  float x[8];
};
template <class T>
struct Raw8 {   // as they are in memory
  uint4 w[T::kBytes / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load8(const char* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < T::kBytes / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <class T>
__device__ __forceinline__ F8 floats8(const Raw8<T>& r) {
  F8 f;
#pragma unroll
  for (int i = 0; i < T::kBytes / 2; ++i) {
    float2 o[T::kEPV / 2];
    unpack16<T>(r.w[i], o);
#pragma unroll
    for (int j = 0; j < T::kEPV / 2; ++j) {
      f.x[i * T::kEPV + 2 * j] = o[j].x;
      f.x[i * T::kEPV + 2 * j + 1] = o[j].y;
    }
  }
  return f;
}
template <class T>
__device__ __forceinline__ void store8(char* p, const F8& f);
template <>
__device__ __forceinline__ void store8<F32>(char* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.x[0], f.x[1], f.x[2], f.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.x[4], f.x[5], f.x[6], f.x[7]);
}
template <>
__device__ __forceinline__ void store8<BF16>(char* p, const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x[2 * i], f.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<E4M3>(char* p, const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f.x[2 * i], f.x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// In: the new tokens' type (and the queries'); Out: the pools'. kHeads: heads a thread takes.
// Slots are a token's rows: its query heads, then its key heads, then its value heads. A thread keeps one place of 16
// elements and the slots g, g + groups, ... for all of its tokens (blockIdx.x * toks + its own, then gridDim.x * toks
// further on), so that a token costs it no division but its page's. Found anew for every token, the places took 16384 tokens
// of 48 heads 76 to 97 us where this takes 67.
template <class In, class Out, int kHeads>
__global__ void __launch_bounds__(kRotThreads) append_rotated_kernel(RotateParams p) {
  pdl_launch_dependents();   // as the plain append: what follows waits before it reads the pools or the queries
  const int places = p.d / 16;
  const int per_tok = p.block_groups * places;
  const int tl = threadIdx.x / per_tok, rest = threadIdx.x - tl * per_tok;
  const int lg = rest / places, place = rest - lg * places;
  const int group = blockIdx.y * p.block_groups + lg;
  if (tl >= p.toks || group >= p.groups) return;
  const bool reports = group == 0 && place == 0;
  // the two vectors of the place
  const bool turns = place < p.turned / 16;
  const int a = turns && !p.interleaved ? 8 * place : 16 * place;
  const int ab = turns && !p.interleaved ? p.turned / 2 : 8;   // from the first to the second
  const int64_t table = turns ? 8 * place : 0;
  // where a token's slots lie, behind the token's own offset: from (in bytes), and to (q_out or pool)
  const char* from[kHeads];
  char* to[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    const int s = group + k * p.groups;
    const int hk = s - p.h_q, hv = hk - p.h_kv;
    const int64_t h = hk < 0 ? s : (hv < 0 ? hk : hv);
    from[k] = static_cast<const char*>(hk < 0 ? p.q : (hv < 0 ? p.new_k : p.new_v)) + (h * p.d + a) * In::kBytes;
    to[k] = hk < 0 ? static_cast<char*>(p.q_out) + (h * p.d + a) * In::kBytes
                   : static_cast<char*>(hv < 0 ? p.k_pool : p.v_pool) + (h * p.page_tokens * p.d + a) * Out::kBytes;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.toks;
  int64_t t = static_cast<int64_t>(blockIdx.x) * p.toks + tl;
  int next_pos = t < p.n_tok ? p.positions[t] : 0, next_slot = t < p.n_tok ? p.slot_mapping[t] : 0;
  for (; t < p.n_tok; t += step) {
    const int pos = next_pos, slot = next_slot;
    if (t + step < p.n_tok) {
      next_pos = p.positions[t + step];
      next_slot = p.slot_mapping[t + step];
    }
    if (pos < 0 || pos >= p.n_pos) {
      if (reports) raise_status(p.status, NBX_DEV_BAD_LEN);
      continue;
    }
    const bool held = slot >= 0 && slot < static_cast<int64_t>(p.num_pages) * p.page_tokens;
    if (reports && !held) raise_status(p.status, NBX_DEV_BAD_SLOT);
    const int wanted = held ? p.slots : (p.k_out ? p.h_q + p.h_kv : p.h_q);   // a token without a slot still turns
    const int page = held ? slot / p.page_tokens : 0;
    const int64_t in_pool = (static_cast<int64_t>(page) * p.h_kv * p.page_tokens + (slot - page * p.page_tokens)) *
                            (p.d * Out::kBytes);
    const int64_t at_q = t * p.q_stride * In::kBytes, at_k = t * p.k_stride * In::kBytes, at_v = t * p.v_stride * In::kBytes;
    Raw8<In> va[kHeads], vb[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int s = group + k * p.groups;
      if (s >= wanted) continue;
      const char* src = from[k] + (s < p.h_q ? at_q : (s < p.h_q + p.h_kv ? at_k : at_v));
      va[k] = load8<In>(src);
      vb[k] = load8<In>(src + ab * In::kBytes);
    }
    F8 c, n;
    if (turns) {
      const int64_t row = static_cast<int64_t>(pos) * (p.turned / 2) + table;
      c = floats8<F32>(load8<F32>(reinterpret_cast<const char*>(p.cos_table + row)));
      n = floats8<F32>(load8<F32>(reinterpret_cast<const char*>(p.sin_table + row)));
    }
    const int64_t at_out = t * p.q_out_stride * In::kBytes;
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int s = group + k * p.groups;
      if (s >= wanted) continue;
      F8 x = floats8<In>(va[k]), y = floats8<In>(vb[k]);
      if (turns && s < p.h_q + p.h_kv) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = x.x[2 * i], y0 = y.x[2 * i];
            x.x[2 * i] = fmaf(-x.x[2 * i + 1], n.x[i], x0 * c.x[i]);
            x.x[2 * i + 1] = fmaf(x0, n.x[i], x.x[2 * i + 1] * c.x[i]);
            y.x[2 * i] = fmaf(-y.x[2 * i + 1], n.x[4 + i], y0 * c.x[4 + i]);
            y.x[2 * i + 1] = fmaf(y0, n.x[4 + i], y.x[2 * i + 1] * c.x[4 + i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = x.x[i];
            x.x[i] = fmaf(-y.x[i], n.x[i], x0 * c.x[i]);
            y.x[i] = fmaf(x0, n.x[i], y.x[i] * c.x[i]);
          }
        }
      }
      if (s < p.h_q) {
        store8<In>(to[k] + at_out, x);
        store8<In>(to[k] + at_out + ab * In::kBytes, y);
      } else {
        if (p.k_out && s < p.h_q + p.h_kv) {
          char* const out = static_cast<char*>(p.k_out) + (t * p.k_out_stride + (s - p.h_q) * p.d + a) * In::kBytes;
          store8<In>(out, x);
          store8<In>(out + ab * In::kBytes, y);
        }
        if (!held) continue;
        const float inv = s < p.h_q + p.h_kv ? p.k_inv : p.v_inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x.x[i] *= inv;
          y.x[i] *= inv;
        }
        store8<Out>(to[k] + in_pool, x);
        store8<Out>(to[k] + in_pool + ab * Out::kBytes, y);
      }
    }
  }
}

template <class In, class Out, int kHeads>
cudaError_t launch_rotated(RotateParams p, cudaStream_t stream) {
  const int places = p.d / 16, sms = device_info().sm_count;
  p.groups = (p.slots + kHeads - 1) / kHeads;
  p.block_groups = std::min(p.groups, kRotThreads / places);
  const int per_tok = p.block_groups * places;
  p.toks = std::max(1, std::min(kRotThreads / per_tok, p.n_tok / sms));   // few tokens: one a block
  const int threads = (p.toks * per_tok + 31) / 32 * 32;
  const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(p.n_tok) + p.toks - 1) / p.toks,
                                           static_cast<int64_t>(sms) * kRotBlocks);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.groups + p.block_groups - 1) / p.block_groups));
  append_rotated_kernel<In, Out, kHeads><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class In, class Out>
cudaError_t launch_rotated(const RotateParams& p, cudaStream_t stream) {
  // few tokens: fewer heads a thread, so that their loads are on more SMs
  return static_cast<int64_t>(p.n_tok) * p.slots * (p.d / 16) < static_cast<int64_t>(device_info().sm_count) * 2048
             ? launch_rotated<In, Out, 1>(p, stream)
             : launch_rotated<In, Out, 4>(p, stream);
}

}  // namespace

cudaError_t append_rotated_dispatch(const RotateParams& p, int new_dtype, int pool_dtype, cudaStream_t stream) {
  if (new_dtype == NBX_F32) {
    if (pool_dtype == NBX_F32) return launch_rotated<F32, F32>(p, stream);
    if (pool_dtype == NBX_BF16) return launch_rotated<F32, BF16>(p, stream);
    return launch_rotated<F32, E4M3>(p, stream);
  }
  if (pool_dtype == NBX_F32) return launch_rotated<BF16, F32>(p, stream);
  if (pool_dtype == NBX_BF16) return launch_rotated<BF16, BF16>(p, stream);
  return launch_rotated<BF16, E4M3>(p, stream);
}

}  // namespace nbx
