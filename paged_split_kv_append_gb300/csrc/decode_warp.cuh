// The split partial of modified and block-scaled decodes for few query vectors: one warp per work unit, the
// two products on mma.sync.
//
// Same maths as decode_partial_kernel (per split an online softmax, an unnormalised partial (m, l, acc); plan
// and merge are shared). A single-row decode reads every key once for a handful of query vectors, so its
// floor is the cache's bytes. On the CUDA cores an E4M3 cache does not come near it: the conversions and the
// packed FMAs of 4 vectors took 125 us for 285 MB (32 sequences of 512 to 8192 positions), as much as bf16
// took for twice the bytes. tcgen05 wants 64 and more rows an operand; m16n8k16 fits 8 query vectors.
//
//  * Work unit = (split entry, KV head, 8 query vectors), taken by one warp from the list's counter. Warps
//    share nothing: no barriers, no waits but for their own copies. Splits are sized for one unit a resident
//    warp over the GPU (at least 64 positions each, at most 64 a sequence), rounded up: rounded down, some
//    sequences' units were twice the mean (ragged bf16: 246 against 220 us). Three units a warp where pairs of a
//    sequence and KV head are about as many as warps (the plan kernel says when).
//  * What bounds it: of the 62 us of that kernel the copies alone take 55 (5.4 TB/s, with the first tiles'
//    chain of loads and the tail; 44 us at the copy rate), the arithmetic alone 47.
//  * Each warp streams its unit's 16-position tiles into a ring of its own in shared memory with 16-byte
//    cp.async copies (a tile of one KV head is one contiguous block of the pool), 16-byte chunks swizzled by
//    row so that both products read them without bank conflicts.
//  * S^T = K Q^T: M = 16 keys, N = the 8 vectors, K = d. Lane (g, t) = (lane / 4, lane % 4) holds the scores of
//    keys g and g + 8 for vectors 2t and 2t + 1, whose part of O it accumulates too. (Queries as the A operand,
//    padded to 16 rows, gave P in place for the second product, but twice the MMAs and a register of zeros
//    for every two of queries: 80 against 74 us a call for the 285 MB. The first product run a tile ahead of
//    the second, to fill its latencies: no difference.)
//  * O^T += V^T P^T: M = 16 of d, N = the 8 vectors, K = 16 keys. P is transposed on the way with movmatrix. V's
//    rows are keys, so two keys' values of one dimension are paired with byte permutes.
//  * Formats. E4M3: codes convert to f16 exactly; bf16 queries times a power of two are f16 exactly but for
//    elements under 2^-29 of the vector's largest, fp32 ones are two f16 terms (22 bits); P is two f16 terms,
//    2^-22, with the running max kept so that the largest weight lies in [2^7, 2^15]. bf16: the operands as
//    they are, P as three bf16 terms, 2^-24. Sums are fp32, and results as near to 64 bits as the fp32 path's.
//  * Block scales, caps, distances and key ranges as in the other kernels (a V block's scale goes into the
//    exponent, and back out of the softmax's sum). Values at positions that only some vectors see may be NaN
//    or infinite: such a tile is added key by key. Rows that no vector sees are zeroed.
#pragma once

#include <atomic>
#include <climits>

#include "nbx_device.cuh"
#include "nbx_internal.h"

namespace nbx {
namespace {

constexpr int kWarpVecs = kWarpUnitVectors;   // 8

template <class PT, class QT, int D, int X>
struct WarpCfg {
  static constexpr bool kE4 = PT::kCode == NBX_E4M3;
  static constexpr bool kTwo = QT::kCode == NBX_F32;        // queries as two terms
  // log2 of the largest weight after a move of m, and at most: high in f16's range under E4M3 values, low under
  // bf16 ones, whose own range is fp32's
  static constexpr float kMid = kE4 ? 7.f : 0.f, kHi = kE4 ? 15.f : 8.f;
  static constexpr int kRow = D * PT::kBytes;               // bytes of a position
  static constexpr int kTile = kTileN * kRow;               // bytes of 16 positions of K (or V)
  static constexpr int kStage = 2 * kTile + ((X & kBlockScaled) ? 16 : 0);
  static constexpr int kChunks = kRow / 16;                 // 16-byte chunks of a position
  static constexpr int kKLoads = kChunks / 4;               // chunks of a key one lane reads for S
  static constexpr int kMmaPerChunk = kE4 ? 4 : 2;
  static constexpr int kQFrags = kKLoads * kMmaPerChunk;    // k16 steps of S
  static constexpr int kMTiles = D / 16;
  static constexpr int kWarpsCta = kStage <= 9000 ? 4 : 2;
  // warps an SM by their registers (accumulators and query terms): at d = 128, 16 of 128 registers spill and
  // took 80 us where 12 of 168, a stage deeper, take 74
  static constexpr int kRegWarps = D == 64 ? 16 : (D == 128 ? 12 : 8);
  static constexpr int kSmemAll = 220 * 1024;
  static constexpr int kDepthAt = kSmemAll / (kRegWarps * kStage);
  static constexpr int kDepth = kDepthAt > 6 ? 6 : (kDepthAt < 2 ? 2 : kDepthAt);   // stages of a warp's ring
  static constexpr int kWarpsBySmem = kSmemAll / (kDepth * kStage);
  static constexpr int kCtas = (kRegWarps < kWarpsBySmem ? kRegWarps : kWarpsBySmem) / kWarpsCta;
  static constexpr int kSmem = kWarpsCta * kDepth * kStage;
  static_assert(kCtas >= 1 && kSmem <= 227 * 1024, "shared memory");
  static_assert(kCtas * kWarpsCta == warp_path_warps(PT::kCode, D), "the plan's warps an SM");
};

// Physical 16-byte chunk of chunk c of a tile's row: rows 2j and 2j + 1 differ in bit 2, the even rows among
// themselves in bits 1 and 2 (S reads two rows' four chunks at a time, the second product four even or odd
// rows' two). Rows of 64 bytes are left as they are.
template <int kChunks>
__device__ __forceinline__ int swizzled(int row, int c) {
  if constexpr (kChunks < 8) return c;
  else return c ^ ((row & 6) ^ ((row & 1) << 2));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool kE4>
__device__ __forceinline__ void mma_pool(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kE4) mma_f16(c, a0, a1, a2, a3, b0, b1);
  else mma_bf16(c, a0, a1, a2, a3, b0, b1);
}
// Four E4M3 codes to two f16 pairs, exactly (the low two codes in lo).
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t h2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 h2_floats(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t b2_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The transpose of an 8 x 8 matrix of 16-bit elements, lane (g, t) holding row g's columns 2t and 2t + 1.
__device__ __forceinline__ uint32_t transposed8x8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

// Two weights as terms of the product's operand type: x = sum of the terms to 2^-22 (f16) or 2^-24 (bf16).
template <bool kE4>
__device__ __forceinline__ void split_terms(float a, float b, uint32_t (&w)[3]) {
  if constexpr (kE4) {
    w[0] = h2_bits(a, b);
    const float2 h = h2_floats(w[0]);
    w[1] = h2_bits(a - h.x, b - h.y);
    w[2] = 0u;
  } else {
    w[0] = b2_bits(a, b);
    float2 h = bf16x2_to_float2(w[0]);
    a -= h.x;
    b -= h.y;
    w[1] = b2_bits(a, b);
    h = bf16x2_to_float2(w[1]);
    w[2] = b2_bits(a - h.x, b - h.y);
  }
}

// acc += V^T P^T of one M tile and 16 keys: the terms' products from zero, the smallest first, and one rounded
// addition. The MMA's own accumulation truncates: over the tiles of a 2048-position split that took 2e-6 off
// the result, more than all other errors together.
template <bool kE4>
__device__ __forceinline__ void add_tile(float (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t (&p0)[3], const uint32_t (&p1)[3]) {
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int x = kE4 ? 1 : 2; x >= 0; --x) mma_pool<kE4>(o, a0, a1, a2, a3, p0[x], p1[x]);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += o[i];
}

// tanh for the cap: a polynomial up to 0.75 (relative error 1.2e-8); above, CUDA's.
__device__ __forceinline__ float small_tanh(float x) {
  const float u = x * x;
  float t = fmaf(u, 0.0017277069855481386f, -0.0076394579373300076f);
  t = fmaf(u, t, 0.021438755095005035f);
  t = fmaf(u, t, -0.05388793721795082f);
  t = fmaf(u, t, 0.13332609832286835f);
  t = fmaf(u, t, -0.3333330750465393f);
  return x * fmaf(u, t, 1.f);
}

template <class PT, class QT, int D, int X>
__global__ void __launch_bounds__(WarpCfg<PT, QT, D, X>::kWarpsCta * 32, WarpCfg<PT, QT, D, X>::kCtas)
    decode_partial_warp_kernel(DecodeParams p) {
  using C = WarpCfg<PT, QT, D, X>;
  constexpr bool kMod = (X & kScoreMod) != 0, kBlk = (X & kBlockScaled) != 0, kE4 = C::kE4;
  constexpr int kTerms = kE4 ? 2 : 3;
  extern __shared__ __align__(128) char smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem_raw) + warp * (C::kDepth * C::kStage);
  // Offsets within a tile, fixed for the kernel: a lane's chunk of the copies (and the same with the swizzle of
  // rows 4 further on), of its key rows g and 8 + g, and of its value rows 2t, 2t + 8 and 2t + 1, 2t + 9.
  // Chunks c + 4 of a row lie at the offset of c with bit 6 flipped, chunks c + 8 128 bytes further on.
  const int c_row = lane / C::kChunks;   // 0 with 32 chunks a row
  const uint32_t c_off = c_row * C::kRow + swizzled<C::kChunks>(c_row, lane % C::kChunks) * 16;
  const uint32_t k_off = g * C::kRow + swizzled<C::kChunks>(g, t) * 16;
  const uint32_t v_off0 = 2 * t * C::kRow + (C::kChunks >= 8 ? swizzled<C::kChunks>(2 * t, g) * 16 : g * 8);
  const uint32_t v_off1 = (2 * t + 1) * C::kRow + (C::kChunks >= 8 ? swizzled<C::kChunks>(2 * t + 1, g) * 16 : g * 8);
  pdl_wait();              // the plan kernel's work list and the append's positions are visible from here on
  pdl_launch_dependents(); // the merge kernel may be scheduled as CTAs of this grid retire
  const int RG = p.rows * p.group;
  const int blocks = (RG + kWarpVecs - 1) / kWarpVecs;   // units of 8 vectors of a KV head
  const int span = p.h_kv * blocks;
  const int n_units = p.header[0] * span;
  const int P = p.page_tokens;
  for (;;) {
    int u = 0;
    if (lane == 0) u = atomicAdd(&p.header[1], 1);
    u = __shfl_sync(0xffffffffu, u, 0);
    if (u >= n_units) break;
    const int rem = u % span;
    const int h = rem / blocks, v0 = (rem - h * blocks) * kWarpVecs;
    const Entry en = p.entries[u / span];
    // ---- vectors 2t and 2t + 1 of the unit: their rows, the keys they see, their biases
    int at[2], seen_lo[2], seen_hi[2];
    float slope[2];
    int lo = INT_MAX, hi = 0, all_lo = 0, all_hi = INT_MAX;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int v = v0 + 2 * t + y;
      const bool vq = v < RG;
      const int r = vq ? v / p.group : 0;
      at[y] = en.len - p.rows + r;
      KeyRange kr = {0, 0};
      if (vq) kr = kMod ? key_range(p, en.b, r, en.len) : (at[y] >= 0 ? KeyRange{0, at[y] + 1} : KeyRange{0, 0});
      slope[y] = kMod && vq && p.slopes ? p.slopes[h * p.group + (v - r * p.group)] * kLog2e : 0.f;
      seen_lo[y] = kr.lo;
      seen_hi[y] = kr.hi;
      if (kr.hi > kr.lo) lo = min(lo, kr.lo);
      hi = max(hi, kr.hi);
      if (vq) {
        all_lo = max(all_lo, kr.lo);
        all_hi = min(all_hi, kr.hi);
      }
    }
    // the keys that some vector sees, cut to whole tiles of the split, and those that every vector sees
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
    }
    const int start = max(en.start, lo & ~(kTileN - 1)), end = min(en.end, hi);
    const int tiles = end > start ? (end - start + kTileN - 1) / kTileN : 0;

    // ---- the tile stream: page ids 32 at a time, a chunk ahead
    const int32_t* const bt = p.block_table + static_cast<int64_t>(en.b) * p.max_pages;
    const int last_page = tiles ? (end - 1) / P : -1;
    int pc = start / P;                    // page index of the current chunk's lane 0
    int pages = pc + lane <= last_page ? bt[pc + lane] : -1;
    int pages_next = pc + 32 + lane <= last_page ? bt[pc + 32 + lane] : -1;
    int i_pi = pc, i_po = start - pc * P;  // page index and position in it of the next tile to copy
    uint32_t ok_bits = 0;                  // bit s: stage s holds a tile
    int fill = 0;                          // the stage that the next copy fills
    auto issue = [&](int i) {
      const int slot = fill;
      fill = fill + 1 == C::kDepth ? 0 : fill + 1;
      if (i < tiles) {
        if (i_pi >= pc + 32) {
          pc += 32;
          pages = pages_next;
          pages_next = pc + 32 + lane <= last_page ? bt[pc + 32 + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, pages, i_pi - pc);
        const bool ok = page >= 0 && page < p.num_pages;
        ok_bits = ok ? ok_bits | (1u << slot) : ok_bits & ~(1u << slot);
        if (ok) {
          const int64_t head = static_cast<int64_t>(page) * p.h_kv + h;
          const int64_t off = (head * P + i_po) * C::kRow;
          const char* const ks = static_cast<const char*>(p.k_pool) + off + lane * 16;
          const char* const vs = static_cast<const char*>(p.v_pool) + off + lane * 16;
          const uint32_t dst = ring + slot * C::kStage;
#pragma unroll
          for (int j = 0; j < C::kTile / 512; ++j) {
            // chunk 32 j + lane: row c_row + 32 j / kChunks
            uint32_t to;
            if constexpr (C::kChunks == 32) to = j * C::kRow + swizzled<32>(j, lane) * 16;
            else if constexpr (C::kChunks == 16) to = 2 * j * C::kRow + (c_off ^ ((2 * j) & 6) * 16);
            else if constexpr (C::kChunks == 8) to = 4 * j * C::kRow + (c_off ^ ((4 * j) & 4) * 16);
            else to = 8 * j * C::kRow + c_off;
            cp_async16(dst + to, ks + j * 512);
            cp_async16(dst + to + C::kTile, vs + j * 512);
          }
          if (kBlk && lane < 2)
            cp_async4(dst + 2 * C::kTile + lane * 4,
                      (lane ? p.v_scales : p.k_scales) + head * (P >> p.scale_shift) + (i_po >> p.scale_shift));
        } else if (lane == 0) {
          raise_status(p.status, NBX_DEV_BAD_PAGE);
        }
        i_po += kTileN;
        if (i_po == P) {
          i_po = 0;
          ++i_pi;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < C::kDepth - 1; ++i) issue(i);

    // ---- the unit's queries as the B operand: lane (g, t) holds vector g's elements of the chunks that it reads
    // of the keys
    uint32_t qh[C::kQFrags][2], ql[C::kTwo ? C::kQFrags : 1][2];
    float fac[2] = {p.qk_scale_log2, p.qk_scale_log2};   // vectors 2t, 2t + 1: from a product to log2 units
    {
      const bool vq = v0 + g < RG;
      const int r = vq ? (v0 + g) / p.group : 0, gq = vq ? v0 + g - r * p.group : 0;
      constexpr int kElems = kE4 ? 16 : 8;   // elements of a 16-byte chunk
      const int64_t orow = (static_cast<int64_t>(en.b) * p.rows + r) * p.h_q + static_cast<int64_t>(h) * p.group + gq;
      const char* const q = static_cast<const char*>(p.q) + orow * D * QT::kBytes;
      if constexpr (!kE4) {
#pragma unroll
        for (int i = 0; i < C::kKLoads; ++i) {
          const uint4 x = vq ? __ldg(reinterpret_cast<const uint4*>(q + (t + 4 * i) * 16)) : make_uint4(0u, 0u, 0u, 0u);
          qh[2 * i][0] = x.x, qh[2 * i][1] = x.y, qh[2 * i + 1][0] = x.z, qh[2 * i + 1][1] = x.w;
        }
      } else {
        // its largest element brought into [2^14, 2^15): every finite element is then f16, or two f16 terms
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < C::kKLoads; ++i) {
#pragma unroll
          for (int e = 0; e < kElems; e += 2) {
            const float2 x = vq ? load_pair<QT>(q + ((t + 4 * i) * kElems + e) * QT::kBytes) : make_float2(0.f, 0.f);
            amax = max_nan(amax, max_nan(fabsf(x.x), fabsf(x.y)));
          }
        }
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e2 = 0;   // NaN or infinity in the vector: as it is
        if (amax > 0.f && amax <= 3.402823466e38f)
          e2 = min(120, max(-120, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
        fac[0] *= __shfl_sync(0xffffffffu, down, 8 * t);
        fac[1] *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < C::kKLoads; ++i) {
#pragma unroll
          for (int e = 0; e < kElems; e += 2) {
            float2 x = vq ? load_pair<QT>(q + ((t + 4 * i) * kElems + e) * QT::kBytes) : make_float2(0.f, 0.f);
            x.x *= up;
            x.y *= up;
            const int f = i * 4 + e / 4, w = (e / 2) & 1;
            qh[f][w] = h2_bits(x.x, x.y);
            if constexpr (C::kTwo) {
              const float2 y = h2_floats(qh[f][w]);
              ql[f][w] = h2_bits(x.x - y.x, x.y - y.y);
            }
          }
        }
      }
    }

    // vectors 2t, 2t + 1: the exponent's reference, this lane's part of the sum, D / 8 dimensions of O
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float acc[C::kMTiles][4];
#pragma unroll
    for (int i = 0; i < C::kMTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

    int slot = 0;   // the stage of tile i
#pragma unroll 1
    for (int i = 0; i < tiles; ++i, slot = slot + 1 == C::kDepth ? 0 : slot + 1) {
      issue(i + C::kDepth - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kDepth - 1) : "memory");
      __syncwarp();   // every lane's copies of tile i have landed
      const uint32_t kb = ring + slot * C::kStage, vb = kb + C::kTile;
      bool ok = (ok_bits >> slot) & 1u;
      float ks = 1.f, lv = 0.f, iv = 1.f;
      if constexpr (kBlk) {
        if (ok) {
          const uint2 w = lds64(kb + 2 * C::kTile);
          ks = __uint_as_float(w.x);
          const float vs = __uint_as_float(w.y);
          ok = ks >= kMinScale && ks <= kMaxScale && vs >= kMinScale && vs <= kMaxScale;
          if (!ok && lane == 0) raise_status(p.status, NBX_DEV_BAD_SCALE);
          lv = __log2f(vs);   // both to 2^-22
          iv = fast_rcp(vs);
        }
      }
      if (ok) {
        const int n0 = start + i * kTileN;
        // ---- scores: z[0], z[1] of key n0 + g, z[2], z[3] of key n0 + 8 + g, for vectors 2t and 2t + 1
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C::kKLoads; ++c) {
          const uint32_t a = kb + (k_off ^ ((c & 1) * 64)) + (c >> 1) * 128;   // chunk t + 4 c of row g
          const uint4 x = lds128(a), y = lds128(a + 8 * C::kRow);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < C::kMmaPerChunk; ++j) {
            uint32_t a0, a1, a2, a3;
            if constexpr (kE4) {
              e4m3x4_to_h2(xw[j], a0, a2);
              e4m3x4_to_h2(yw[j], a1, a3);
            } else {
              a0 = xw[2 * j], a2 = xw[2 * j + 1];
              a1 = yw[2 * j], a3 = yw[2 * j + 1];
            }
            const int f = c * C::kMmaPerChunk + j;
            mma_pool<kE4>(z, a0, a1, a2, a3, qh[f][0], qh[f][1]);
            if constexpr (C::kTwo) mma_pool<kE4>(z, a0, a1, a2, a3, ql[f][0], ql[f][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] *= kBlk ? fac[e & 1] * ks : fac[e & 1];
        if constexpr (kMod) {
          if (p.cap_log2 > 0.f) {
            const float x[4] = {z[0] * p.cap_inv, z[1] * p.cap_inv, z[2] * p.cap_inv, z[3] * p.cap_inv};
            const float far = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = p.cap_log2 * small_tanh(x[e]);
            // (each score by its own size, whatever the others are: a key that nobody sees changes no bit)
            if (!__all_sync(0xffffffffu, far <= 0.75f)) {   // (a NaN is passed over, and stays one either way)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (fabsf(x[e]) > 0.75f) z[e] = p.cap_log2 * tanhf(x[e]);
            }
          }
          if (p.slopes != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[e] = fmaf(-slope[e & 1], static_cast<float>(abs(at[e & 1] - (n0 + (e >> 1) * 8 + g))), z[e]);
          }
        }
        const bool full = n0 >= all_lo && n0 + kTileN <= all_hi && n0 + kTileN <= end;
        uint32_t sees = 15u;   // bit e: z[e]'s vector sees its key
        if (!full) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = n0 + (e >> 1) * 8 + g;
            if (n < seen_lo[e & 1] || n >= seen_hi[e & 1] || n >= end) {
              z[e] = -INFINITY;
              sees &= ~(1u << e);
            }
          }
        }
        // ---- the reference moves when a weight would pass 2^15; a NaN one stays NaN
        float mx[2] = {max_nan(z[0], z[2]) + lv, max_nan(z[1], z[3]) + lv};
        const bool past = (!(mx[0] <= m_run[0] + C::kHi) && m_run[0] == m_run[0]) ||
                          (!(mx[1] <= m_run[1] + C::kHi) && m_run[1] == m_run[1]);
        if (__any_sync(0xffffffffu, past)) {
          float f[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx[y] = max_nan(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], o));
            const bool move = !(mx[y] <= m_run[y] + C::kHi) && m_run[y] == m_run[y];
            const float m_new = move ? mx[y] - C::kMid : m_run[y];
            f[y] = move ? fast_exp2(m_run[y] - m_new) : 1.f;
            m_run[y] = m_new;
            l_run[y] *= f[y];
          }
#pragma unroll
          for (int j = 0; j < C::kMTiles; ++j) {
            acc[j][0] *= f[0];
            acc[j][1] *= f[1];
            acc[j][2] *= f[0];
            acc[j][3] *= f[1];
          }
        }
        float pw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // nothing seen yet: every z is -inf
          const float off = m_run[e & 1] == -INFINITY ? 0.f : lv - m_run[e & 1];
          pw[e] = fast_exp2(z[e] + off);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) l_run[y] += kBlk ? (pw[y] + pw[2 + y]) * iv : pw[y] + pw[2 + y];
        // the B operand of the second product: vector g's weights of keys 2t, 2t + 1, and of 8 + 2t, 9 + 2t
        uint32_t p0[3], p1[3];
        split_terms<kE4>(pw[0], pw[1], p0);
        split_terms<kE4>(pw[2], pw[3], p1);
#pragma unroll
        for (int x = 0; x < kTerms; ++x) {
          p0[x] = transposed8x8(p0[x]);
          p1[x] = transposed8x8(p1[x]);
        }
        // ---- O^T += V^T P^T: lane (g, t) reads its 16-byte chunks of keys 2t, 2t + 1, 2t + 8, 2t + 9
        constexpr int kVLoads = C::kChunks >= 8 ? C::kChunks / 8 : 1;
        constexpr int kWords = C::kChunks >= 8 ? 4 : 2;   // 32-bit words of a load (rows of 64 bytes: 8 bytes a lane)
        bool by_key = false;
        if (!full) {
          // Rows that no vector sees hold what a page happens to hold past its sequence: zeros, so that a NaN there
          // does not choose how the others are added.
          const int first = lo - n0, past = end - n0;
          if (first > 0 || past < kTileN) {
            char* const v = smem_raw + warp * (C::kDepth * C::kStage) + slot * C::kStage + C::kTile;
#pragma unroll
            for (int i = lane; i < kTileN * C::kChunks; i += 32) {
              const int row = i / C::kChunks;
              if (row < first || row >= past) *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
          }
          // values that are not finite at a position that some vector does not see
          bool bad = false;
#pragma unroll
          for (int c = 0; c < kVLoads; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a = vb + ((e & 1) ? v_off1 : v_off0) + (e >> 1) * 8 * C::kRow + c * 128;   // chunk g + 8 c
              if constexpr (kWords == 4) {
                bad = bad || not_finite<kE4>(lds128(a));
              } else {
                const uint2 x = lds64(a);
                bad = bad || not_finite<kE4>(make_uint4(x.x, x.y, 0u, 0u));
              }
            }
          by_key = __any_sync(0xffffffffu, bad);
        }
        if (!by_key) {
#pragma unroll
          for (int c = 0; c < kVLoads; ++c) {
            uint32_t w[4][kWords];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a = vb + ((e & 1) ? v_off1 : v_off0) + (e >> 1) * 8 * C::kRow + c * 128;
              if constexpr (kWords == 4) {
                const uint4 x = lds128(a);
                w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
              } else {
                const uint2 x = lds64(a);
                w[e][0] = x.x, w[e][1] = x.y;
              }
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              if constexpr (kE4) {   // four dimensions: two M tiles
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t sel = y ? 0x7362u : 0x5140u;
                  const uint32_t ab = __byte_perm(w[0][k], w[1][k], sel), cd = __byte_perm(w[2][k], w[3][k], sel);
                  uint32_t a0, a1, a2, a3;
                  e4m3x4_to_h2(ab, a0, a1);
                  e4m3x4_to_h2(cd, a2, a3);
                  add_tile<kE4>(acc[(c * kWords + k) * 2 + y], a0, a1, a2, a3, p0, p1);
                }
              } else {               // two dimensions: one M tile
                const uint32_t a0 = __byte_perm(w[0][k], w[1][k], 0x5410), a1 = __byte_perm(w[0][k], w[1][k], 0x7632);
                const uint32_t a2 = __byte_perm(w[2][k], w[3][k], 0x5410), a3 = __byte_perm(w[2][k], w[3][k], 0x7632);
                add_tile<kE4>(acc[c * kWords + k], a0, a1, a2, a3, p0, p1);
              }
            }
          }
        } else {
          // key by key: a vector's accumulators take only the keys it sees
#pragma unroll 1
          for (int k = 0; k < kTileN; ++k) {
            const int from = (k & 7) * 4 + t;   // the lane with key k's weights for vectors 2t, 2t + 1
            const float pa = __shfl_sync(0xffffffffu, k < 8 ? pw[0] : pw[2], from);
            const float pb = __shfl_sync(0xffffffffu, k < 8 ? pw[1] : pw[3], from);
            const uint32_t both = __shfl_sync(0xffffffffu, k < 8 ? sees : sees >> 2, from);
            const bool sa = both & 1u, sb = both & 2u;
#pragma unroll
            for (int j = 0; j < C::kMTiles; ++j) {
              // M tile j of this lane: elements 2 (j % per), + 1 of its chunk j / per
              constexpr int kPer = C::kMTiles / kVLoads;
              const int c = j / kPer, el = 2 * (j % kPer);
              const uint32_t a = vb + k * C::kRow +
                                 (kWords == 4 ? swizzled<C::kChunks>(k, g + 8 * c) * 16 : g * 8) + el * PT::kBytes;
              float2 x;
              if constexpr (kE4) x = e4m3x2_to_float2(lds16(a));
              else x = bf16x2_to_float2(lds32(a));
              if (sa) {
                acc[j][0] = fmaf(pa, x.x, acc[j][0]);
                acc[j][2] = fmaf(pa, x.y, acc[j][2]);
              }
              if (sb) {
                acc[j][1] = fmaf(pb, x.x, acc[j][1]);
                acc[j][3] = fmaf(pb, x.y, acc[j][3]);
              }
            }
          }
        }
      }
      __syncwarp();   // every lane is done with the stage before it is filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    // ---- the partial: lane (g, t) holds of vectors 2t and 2t + 1 the dimensions of its chunks
    const bool multi = en.n_splits > 1;
    const uint64_t keep = l2_keep_policy(p.keep_frac);   // the partials stay in L2 for the merge
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float lw = l_run[y];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      const float mv = m_run[y];
      const int v = v0 + 2 * t + y;
      if (v >= RG) continue;
      const int rv = v / p.group;
      const int64_t orow = (static_cast<int64_t>(en.b) * p.rows + rv) * p.h_q + static_cast<int64_t>(h) * p.group +
                           (v - rv * p.group);
      const float sc = multi ? 1.f : (mv == -INFINITY ? 0.f : p.v_scale / lw);
      if (multi && g == 0) {
        st_global_hint(p.m_part + orow * p.max_splits + en.s, mv, keep);
        st_global_hint(p.l_part + orow * p.max_splits + en.s, lw, keep);
      }
      constexpr int kVLoads = C::kChunks >= 8 ? C::kChunks / 8 : 1;
      constexpr int kPer = C::kMTiles / kVLoads;   // M tiles of a chunk: 2 kPer consecutive dimensions
#pragma unroll
      for (int c = 0; c < kVLoads; ++c) {
        const int d0 = (g + 8 * c) * 2 * kPer;
#pragma unroll
        for (int j = 0; j < kPer; j += 2) {
          const float o[4] = {acc[c * kPer + j][y] * sc, acc[c * kPer + j][2 + y] * sc, acc[c * kPer + j + 1][y] * sc,
                              acc[c * kPer + j + 1][2 + y] * sc};
          const int d = d0 + 2 * j;
          if (multi) {
            st_global_hint(reinterpret_cast<int4*>(p.acc_part + (orow * p.max_splits + en.s) * D + d),
                           make_int4(__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])),
                           keep);
          } else if (p.out_bf16) {
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + d) =
                make_uint2(b2_bits(o[0], o[1]), b2_bits(o[2], o[3]));
          } else {
            *reinterpret_cast<float4*>(p.out + orow * D + d) = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
  }
}

template <class PT, class QT, int D, int X>
cudaError_t launch_warp(const DecodeParams& p, int grid_limit, cudaStream_t stream) {
  using C = WarpCfg<PT, QT, D, X>;
  static std::atomic<uint64_t> configured{0};   // devices whose shared-memory limit is raised
  const DeviceInfo& di = device_info();
  const uint64_t bit = 1ull << (di.device & 63);
  if ((configured.load() & bit) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(decode_partial_warp_kernel<PT, QT, D, X>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const int64_t upper = static_cast<int64_t>(p.batch) * p.max_splits * p.tc_pairs;
  int64_t grid = (upper + C::kWarpsCta - 1) / C::kWarpsCta;
  const int64_t most = static_cast<int64_t>(di.sm_count) * C::kCtas;
  if (grid > most) grid = most;
  if (grid_limit > 0 && grid > grid_limit) grid = grid_limit;
  if (grid < 1) grid = 1;
  return launch_pdl(decode_partial_warp_kernel<PT, QT, D, X>, static_cast<unsigned>(grid), C::kWarpsCta * 32, C::kSmem, stream,
                    p);
}

template <class PT, class QT, int X>
cudaError_t launch_warp_d(const DecodeParams& p, int grid_limit, cudaStream_t stream) {
  if (p.d == 64) return launch_warp<PT, QT, 64, X>(p, grid_limit, stream);
  if (p.d == 128) return launch_warp<PT, QT, 128, X>(p, grid_limit, stream);
  return launch_warp<PT, QT, 256, X>(p, grid_limit, stream);
}

}  // namespace
}  // namespace nbx
