// Attention of 128-row tiles of query vectors on tcgen05: what prompt attention and the shared-prefix decode run.
//
// A work unit is one or two M tiles of 128 query vectors of one KV head (a tile holds `toks` tokens with `heads` query
// heads each) and the keys they attend, in tiles of 128. Per key tile, with scores in log2 units:
//   S = Q K^T;  m' = max(m, rowmax S) (moved only when it grows by more than 2^8);  P = 2^(c S - m');
//   l = l 2^(m - m') + rowsum P;  O = O 2^(m - m') + P V.
// S and O are fp32 accumulators in TMEM; P is written over S, in bf16 (kTerms = 1: each weight is off by up to 2^-8 of
// itself, as much as the bf16 output's own rounding) or as two bf16 terms (kTerms = 2: 2^-17, for fp32 outputs).
//
// One persistent CTA per SM, ten warps, every wait bounded:
//  * warps 0-3 and 4-7: two softmax groups. Up to d = 128 each has an M tile of its own, one row a thread, and the two
//    take turns with the tensor pipe: while one group works on its S, the MMAs of the other's tile run. At d = 256 O
//    fills half of the TMEM, so there is one M tile, S is double-buffered, and the groups share each row, 64 columns
//    each; the two threads of a row swap their maxima through shared memory.
//  * warp 8 fills the ring of K and V with TMA: slots of 32 KB (16 KB at d = 64), a whole tile, or at d = 256 half of one
//    (128 columns of K, 64 keys of V); and the unit's Q tiles.
//  * warp 9 issues the MMAs: QK^T (both operands from shared memory, M = N = 128) and PV (P from TMEM, N = d), in an
//    order in which the group whose P is awaited is never the one whose S was asked for last. Waiting for P(j) of a
//    tile is all that orders PV(j), QK(j + 1) of the same tile follows it in the pipe and may overwrite P(j).
// What bounds it: the tensor pipe. Per 128 keys and two tiles of d = 128 it is busy 2048 cycles; the softmax issues
// about 900 instructions on each scheduler and takes 1024 or 2048 cycles of the special-function units.
#pragma once

#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "nbx_device.cuh"
#include "nbx_internal.h"
#include "nbx_tcgen05.cuh"

namespace nbx {
namespace {

constexpr int kAtM = 128;         // query vectors of an M tile = TMEM lanes
constexpr int kAtN = 128;         // keys of a tile
constexpr int kAtThreads = 384;
// Registers a thread: of the 168 each is launched with (65536 over three warps a scheduler), the loader's and the MMA
// warp's group gives what a softmax thread needs to hold its 128 scores: 2 * 208 + 88 = 3 * 168.
constexpr int kAtSoftmaxRegs = 208, kAtOtherRegs = 88;
constexpr float kAtTau = 8.f;     // the running maximum moves when it would grow by more, log2 units

template <int D>
struct AttnCfg {
  static constexpr int kTiles = D <= 128 ? 2 : 1;                // M tiles of a unit
  static constexpr int kParts = D <= 128 ? 1 : 2;                // ring slots of a K or V tile
  static constexpr int kAhead = D <= 128 ? 1 : 2;                // QK^T of tile j + kAhead follows PV of tile j
  static constexpr int kCols = D <= 128 ? kAtN : kAtN / 2;       // columns of S a softmax thread takes
  static constexpr int kSlotBytes = D == 64 ? 16384 : 32768;
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr int kAtom = kAtM * 128;                       // 128 rows of 128 bytes
  static constexpr int kQTile = D / 64 * kAtom;
  static constexpr int kRingOff = kTiles * kQTile;
  static constexpr int kBarOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kXOff = kBarOff + 256;
  static constexpr int kSmem = kXOff + (D == 256 ? 2 * 256 * 4 : 0) + 768;   // slack: 256-byte alignment to 1024
  static constexpr uint32_t kOCol = 256;                         // S (and P) in columns [0, 256), O from there
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert((2 * kSlots + 14) * 8 <= 256, "barrier area");
};

// One work unit.
struct AttnUnit {
  int tok;        // first token of the first tile (rows of the query tensor)
  int toks;       // tokens of the unit, of both tiles
  int head, kvh;  // first query head, KV head
  int pos;        // causal: position of the first token in its sequence
  int kv;         // causal: first key's row; paged: first position
  int end;        // paged: one past the last position
  int b, slot;    // paged: row of the block table, slot of the partials
  int n[2];       // key tiles of each M tile
};

__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if ((i & 3u) == 0u && global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ bool at_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, at_wait(bar, parity, abort_flag));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// 32 consecutive 32-bit TMEM columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a work policy W provides (prompt.cu, shared.cu):
//   typename W::Params with c (|scale| log2 e, or the least positive number for a scale of 0), negative and status;
//   W::kPaged, W::kTerms; W(params, lane) (after the grid ahead is waited for), bool unit(round, AttnUnit&): warp-wide;
//   toks_per_tile(), heads(); load_q / load_kv by the loader warp; store(...) by a softmax thread.
template <class W, int D>
struct AttnShared {
  using C = AttnCfg<D>;
  char* q_s;
  char* ring;
  uint64_t* full;      // [kSlots] a ring slot's copies have landed
  uint64_t* empty;     // [kSlots] its MMAs are done
  uint64_t* q_full;
  uint64_t* q_empty;   // every QK^T of the unit is done
  uint64_t* s_full;    // [2] S in its buffer (of M tile t, or of key tile j & 1)
  uint64_t* p_full;    // [2] P over it
  uint64_t* pv_done;   // [2] the PV from that buffer is done: O holds it
  uint64_t* o_free;    // [2] the epilogue has read O of M tile t
  uint64_t* x_bar;     // [4] d = 256: the two warps of 32 rows have left their numbers
  uint64_t* done;
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  float* xbuf;         // [2][256]
};

// ---------------------------------------------------------------- the MMA warp
template <class W, int D>
__device__ __forceinline__ bool attn_mma(W& w, const AttnShared<W, D>& sh, uint32_t tmem) {
  using C = AttnCfg<D>;
  constexpr int T = C::kTiles, NS = C::kSlots;
  constexpr uint32_t kIdescO = mma_idesc(kAtM, D, true);
  // a negative scale: S of -Q (the descriptor's bit 13 negates A), and its magnitude
  const uint32_t idesc_s = mma_idesc(kAtM, kAtN, false) | (w.p.negative ? 1u << 13 : 0u);
  const int lane = threadIdx.x & 31;
  volatile int* ab = sh.abort_flag;
  const uint32_t q_addr = smem_u32(sh.q_s), ring = smem_u32(sh.ring);
  uint32_t r = 0;                    // ring slots consumed so far, in the loader's order
  uint32_t np[2] = {0, 0};           // P buffers consumed
  uint32_t units[2] = {0, 0};        // units with this M tile
  uint32_t xs = 0;                   // d = 256: key tiles whose QK^T was issued (buffer xs & 1)
  AttnUnit u;
  auto slot_wait = [&](uint32_t at) { return at_warp_wait(&sh.full[at % NS], (at / NS) & 1u, ab); };
  auto slot_addr = [&](uint32_t at) { return ring + (at % NS) * C::kSlotBytes; };
  // S(buffer) = Q(tile t) K^T, K in ring slots at, ...
  auto qk = [&](int t, uint32_t buf, uint32_t at) {
    if (lane == 0) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int a = kk >> 2, sub = kk & 3;   // 64-column atom, 16-column step in it
        const uint64_t ad = smem_desc(q_addr + t * C::kQTile + a * C::kAtom + sub * 32, 16, 1024);
        const uint32_t kb = C::kParts == 1 ? slot_addr(at) + a * C::kAtom : slot_addr(at + (a >> 1)) + (a & 1) * C::kAtom;
        tc_mma_ss(tmem + buf * kAtN, ad, smem_desc(kb + sub * 32, 16, 1024), idesc_s, kk > 0);
      }
      tc_commit(&sh.s_full[buf]);
    }
  };
  auto release = [&](uint32_t at) {
    if (lane == 0)
      for (int i = 0; i < C::kParts; ++i) tc_commit(&sh.empty[(at + i) % NS]);
  };
  // O(tile t) += P(buffer) V, `keys` of the tile's keys, V in ring slots at, ...
  auto pv = [&](int t, uint32_t buf, uint32_t at, int keys, bool first) {
    if (lane == 0) {
      const int steps = (keys + 15) >> 4;
#pragma unroll
      for (int term = 0; term < W::kTerms; ++term)
#pragma unroll
        for (int kk = 0; kk < kAtN / 16; ++kk)
          if (kk < steps) {
            const uint32_t vb = C::kParts == 1 ? slot_addr(at) + kk * 2048 : slot_addr(at + (kk >> 2)) + (kk & 3) * 2048;
            const uint64_t bd = smem_desc(vb, C::kParts == 1 ? C::kAtom : C::kAtom / 2, 1024);
            tc_mma_ts(tmem + C::kOCol + t * D, tmem + buf * kAtN + term * (kAtN / 2) + kk * 8, bd, kIdescO,
                      !(first && term == 0 && kk == 0));
          }
      tc_commit(&sh.pv_done[buf]);
    }
  };
  // rows of V past the last key inside its 16-key step are zeroed: 0 x NaN would reach every row
  auto clear_tail = [&](uint32_t at, int keys) {
    if ((keys & 15) == 0) return;
    const int to = (keys + 15) & ~15;
    for (int row = keys; row < to; ++row) {
      // 16-byte pieces of the row: D / 64 atoms of 8
      for (int i = lane; i < D / 8; i += 32) {
        const uint32_t off = C::kParts == 1 ? slot_addr(at) + (i >> 3) * C::kAtom + row * 128
                                            : slot_addr(at + (row >> 6)) + (i >> 3) * (C::kAtom / 2) + (row & 63) * 128;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(off + (i & 7) * 16), "r"(0) : "memory");
      }
    }
    fence_proxy_async();
    __syncwarp();
  };
  for (uint32_t k = 0; w.unit(k, u); ++k) {
    if (!at_warp_wait(sh.q_full, k & 1u, ab)) return false;
    const int n = T == 2 ? max(u.n[0], u.n[1]) : u.n[0];
    // the keys that the last tile holds (V rows behind them are not the sequence's)
    const int last_keys = w.last_keys(u, n);
    auto issue_qk = [&](int j) -> bool {   // of key tile j, T == 1
      const uint32_t at = r;
      for (int i = 0; i < C::kParts; ++i)
        if (!slot_wait(at + i)) return false;
      r += C::kParts;
      tc_fence_after();
      qk(0, xs & 1u, at);
      ++xs;
      release(at);
      if (j == n - 1 && lane == 0) tc_commit(sh.q_empty);
      return true;
    };
    if constexpr (T == 2) {
      if (!slot_wait(r)) return false;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (u.n[t] > 0) qk(t, t, r);
      release(r);
      ++r;
      if (n == 1 && lane == 0) tc_commit(sh.q_empty);
      for (int j = 0; j < n; ++j) {
        const uint32_t rv = r++;
        const bool more = j + 1 < n;
        const uint32_t rk = r;
        if (more) ++r;
        const int keys = more ? kAtN : last_keys;
        bool have_v = false, have_k = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j < u.n[t]) {
            if (!have_v) {
              if (!slot_wait(rv)) return false;
              clear_tail(rv, keys);
              have_v = true;
            }
            if (j == 0 && units[t] > 0 && !at_warp_wait(&sh.o_free[t], (units[t] - 1) & 1u, ab)) return false;
            if (!at_warp_wait(&sh.p_full[t], np[t] & 1u, ab)) return false;
            ++np[t];
            tc_fence_after();
            pv(t, t, rv, keys, j == 0);
          }
          if (j + 1 < u.n[t]) {
            if (!have_k) {
              if (!slot_wait(rk)) return false;
              tc_fence_after();
              have_k = true;
            }
            qk(t, t, rk);
          }
        }
        release(rv);
        if (more) {
          release(rk);
          if (j + 2 == n && lane == 0) tc_commit(sh.q_empty);
        }
      }
    } else {
      for (int j = 0; j < C::kAhead && j < n; ++j)
        if (!issue_qk(j)) return false;
      for (int j = 0; j < n; ++j) {
        const uint32_t rv = r;
        const int keys = j + 1 < n ? kAtN : last_keys;
        for (int i = 0; i < C::kParts; ++i)
          if (!slot_wait(rv + i)) return false;
        r += C::kParts;
        clear_tail(rv, keys);
        if (j == 0 && units[0] > 0 && !at_warp_wait(&sh.o_free[0], (units[0] - 1) & 1u, ab)) return false;
        const uint32_t buf = np[0] & 1u;
        if (!at_warp_wait(&sh.p_full[buf], (np[0] >> 1) & 1u, ab)) return false;
        ++np[0];
        tc_fence_after();
        pv(0, buf, rv, keys, j == 0);
        release(rv);
        if (j + C::kAhead < n && !issue_qk(j + C::kAhead)) return false;
      }
    }
    for (int t = 0; t < T; ++t)
      if (u.n[t] > 0) ++units[t];
  }
  return true;
}

// ---------------------------------------------------------------- a softmax warp
template <class W, int D>
__device__ __forceinline__ bool attn_softmax(W& w, const AttnShared<W, D>& sh, uint32_t tmem) {
  using C = AttnCfg<D>;
  constexpr int T = C::kTiles, NC = C::kCols;
  constexpr int kOCols = T == 2 ? D : D / 2;   // columns of O that this thread rescales and stores
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp >> 2, quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const int t = T == 2 ? group : 0;
  const uint32_t o_base = lane_base + C::kOCol + t * D + (T == 2 ? 0 : group * kOCols);
  const int c0 = T == 2 ? 0 : group * NC;      // first column of S
  const int tpt = w.toks_per_tile();
  const int tok = row / w.heads(), head = row - tok * w.heads();
  const float c = w.p.c;
  volatile int* ab = sh.abort_flag;
  uint32_t x = 0;         // key tiles of this M tile so far
  uint32_t xphase = 0;
  // d = 256: swaps a number with the other thread of the row. What each did before is visible to the other then, its
  // TMEM loads included.
  auto swap = [&](float mine, float& other) -> bool {
    float* buf = sh.xbuf + (xphase & 1u) * 256;
    buf[group * 128 + row] = mine;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.x_bar[quarter]);
    const bool ok = at_warp_wait(&sh.x_bar[quarter], xphase & 1u, ab);
    ++xphase;
    if (!ok) return false;
    tc_fence_after();
    other = buf[(group ^ 1) * 128 + row];
    return true;
  };
  // Waits for the PV of key tile x - 1. A parity wait must know the barrier's phase before that one done: with a tile to
  // each group, S(x - 1) follows PV(x - 2) in the pipe, and at d = 256, with two buffers, PV(x - 3).
  auto pv_wait = [&]() -> bool {
    const uint32_t y = x - 1;
    const bool ok = T == 2 ? at_warp_wait(&sh.pv_done[t], y & 1u, ab) : at_warp_wait(&sh.pv_done[y & 1u], (y >> 1) & 1u, ab);
    tc_fence_after();
    return ok;
  };
  AttnUnit u;
  for (uint32_t k = 0; w.unit(k, u); ++k) {
    const int n = u.n[t];
    if (n == 0) continue;
    const int my_tok = t * tpt + tok;                       // of the unit
    const bool row_ok = tok < tpt && my_tok < u.toks;
    const int last_key = w.last_key(u, my_tok, row_ok);     // of the unit's keys, from 0
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j, ++x) {
      const uint32_t buf = T == 2 ? t : (x & 1u);
      const uint32_t s_col = lane_base + buf * kAtN;
      const uint32_t bad = w.bad_keys(u, j, c0);            // paged: 16-key pieces of this thread's columns without a page
      if (!at_warp_wait(&sh.s_full[buf], (T == 2 ? x : x >> 1) & 1u, ab)) return false;
      tc_fence_after();
      uint32_t s[NC];
#pragma unroll
      for (int i = 0; i < NC; i += 32) tmem_ld32(s_col + c0 + i, s + i);
      tmem_wait_ld();
      const int limit = last_key - (j * kAtN + c0);          // this thread's columns up to here are seen
      if (!__all_sync(0xffffffffu, limit >= NC - 1)) {
#pragma unroll
        for (int i = 0; i < NC; ++i) s[i] = i <= limit ? s[i] : 0xff800000u;
      }
      if (W::kPaged && bad) {   // warp-uniform
#pragma unroll
        for (int i = 0; i < NC; ++i) s[i] = (bad >> (i >> 4)) & 1u ? 0xff800000u : s[i];
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < NC; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = max3(top[e], __uint_as_float(s[i + 2 * e]), __uint_as_float(s[i + 2 * e + 1]));
      float z = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c;
      if constexpr (T == 1) {
        float other;
        if (!swap(z, other)) return false;
        z = fmaxf(z, other);
      }
      // (a NaN score leaves m alone: its own weight is a NaN, and the row's sum)
      const bool up = z > m + kAtTau;
      const float f = up ? fast_exp2(m - z) : 1.f;
      if (up) m = z;
      const float neg = m == -INFINITY ? 0.f : -m;
      const f32x2 c2 = pack2(c, c), neg2 = pack2(neg, neg);
      f32x2 sum[2] = {pack2(l * f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < NC; h += 64) {
        uint32_t hi[32];
        uint32_t lo[W::kTerms == 2 ? 32 : 1];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 e = unpack2(fma2(pack2(__uint_as_float(s[h + 2 * i]), __uint_as_float(s[h + 2 * i + 1])), c2, neg2));
          const float a = fast_exp2(e.x), b = fast_exp2(e.y);
          sum[i & 1] = add2(sum[i & 1], pack2(a, b));
          hi[i] = bf16x2_bits(a, b);
          if constexpr (W::kTerms == 2) {
            const float2 g = bf16x2_to_float2(hi[i]);
            lo[i] = bf16x2_bits(a - g.x, b - g.y);
          }
        }
        tmem_st32(s_col + (c0 + h) / 2, hi);
        if constexpr (W::kTerms == 2) tmem_st32(s_col + kAtN / 2 + (c0 + h) / 2, lo);
      }
      const float2 s0 = unpack2(sum[0]), s1 = unpack2(sum[1]);
      l = (s0.x + s0.y) + (s1.x + s1.y);
      // O follows a maximum that moved, once the last PV into it is done
      if (j > 0 && __any_sync(0xffffffffu, up)) {
        if (!pv_wait()) return false;
        const f32x2 f2 = pack2(f, f);
#pragma unroll
        for (int i = 0; i < kOCols; i += 32) {
          uint32_t o[32];
          tmem_ld32(o_base + i, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = unpack2(mul2(pack2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), f2));
            o[e] = __float_as_uint(y.x);
            o[e + 1] = __float_as_uint(y.y);
          }
          tmem_st32(o_base + i, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[buf]);
    }
    if constexpr (T == 1) {
      float other;
      if (!swap(l, other)) return false;
      l = group == 0 ? l + other : other + l;
    }
    if (!pv_wait()) return false;
    w.template store<kOCols>(u, o_base, T == 2 ? 0 : group * kOCols, my_tok, head, row_ok, m, l, &sh.o_free[t]);
  }
  return true;
}

template <class W, int D>
__global__ void __launch_bounds__(kAtThreads, 1) attn_tiles_kernel(const __grid_constant__ typename W::Params params) {
  using C = AttnCfg<D>;
  constexpr int NS = C::kSlots;
  extern __shared__ __align__(256) char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  AttnShared<W, D> sh;
  sh.q_s = smem;
  sh.ring = smem + C::kRingOff;
  sh.full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  sh.empty = sh.full + NS;
  sh.q_full = sh.empty + NS;
  sh.q_empty = sh.q_full + 1;
  sh.s_full = sh.q_full + 2;
  sh.p_full = sh.q_full + 4;
  sh.pv_done = sh.q_full + 6;
  sh.o_free = sh.q_full + 8;
  sh.done = sh.q_full + 10;
  sh.x_bar = nullptr;
  sh.abort_flag = reinterpret_cast<int*>(sh.q_full + 11);
  sh.tmem_slot = reinterpret_cast<uint32_t*>(sh.q_full + 11) + 1;
  sh.xbuf = reinterpret_cast<float*>(smem + C::kXOff);
  if constexpr (C::kTiles == 1) sh.x_bar = sh.q_full + 12;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(sh.q_full, 1);
    mbar_init(sh.q_empty, 1);
    constexpr int kRowWarps = C::kTiles == 2 ? 4 : 8;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kRowWarps);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.o_free[i], kRowWarps);
    }
    mbar_init(sh.done, 1);
    if constexpr (C::kTiles == 1)
      for (int i = 0; i < 4; ++i) mbar_init(&sh.x_bar[i], 2);
    *sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(sh.tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot;
  // the inputs are written and visible from here on. (kWaitLate: they were before the grid ahead began, which this one
  // may run beside; the grid behind waits for both through this one)
  if constexpr (!W::kWaitLate) pdl_wait();
  pdl_launch_dependents();
  bool ok = true;
  if (warp < 8) {
    W w(params, lane);
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtSoftmaxRegs));
    ok = attn_softmax<W, D>(w, sh, tmem);
  } else {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtOtherRegs));
   if (warp == 8) {
    // ---- the loader: Q of each unit, then K and V in the order in which the MMA warp consumes them
    W w(params, lane);
    uint32_t r = 0, q_units = 0;
    AttnUnit u;
    auto load = [&](bool is_v, int j) -> bool {
      for (int part = 0; part < C::kParts; ++part, ++r) {
        if (r >= NS && !at_warp_wait(&sh.empty[r % NS], (r / NS - 1) & 1u, sh.abort_flag)) return false;
        w.template load_kv<D>(u, is_v, j, part, sh.ring + (r % NS) * C::kSlotBytes, &sh.full[r % NS]);
      }
      return true;
    };
    for (uint32_t k = 0; ok && w.unit(k, u); ++k) {
      if (k > 0) ok = at_warp_wait(sh.q_empty, (k - 1) & 1u, sh.abort_flag);
      if (!ok) break;
      w.template load_q<D>(u, sh.q_s, sh.q_full);
      ++q_units;
      const int n = C::kTiles == 2 ? max(u.n[0], u.n[1]) : u.n[0];
      for (int j = 0; j < C::kAhead && j < n && ok; ++j) ok = load(false, j);
      for (int j = 0; j < n && ok; ++j) {
        ok = load(true, j);
        if (ok && j + C::kAhead < n) ok = load(false, j + C::kAhead);
      }
    }
    if (!ok) *sh.abort_flag = 1;
    // the copies issued last have landed before the CTA can exit
    if (lane == 0) {
      for (uint32_t i = r > NS ? r - NS : 0; i < r; ++i) mbar_wait(&sh.full[i % NS], (i / NS) & 1u, 100000000ull);
      if (q_units > 0) mbar_wait(sh.q_full, (q_units - 1) & 1u, 100000000ull);
    }
    __syncwarp();
   } else if (warp == 9) {
    W w(params, lane);
    ok = attn_mma<W, D>(w, sh, tmem);
    if (!ok) *sh.abort_flag = 1;
    if (lane == 0) {   // every MMA of this CTA has completed before the TMEM is released
      tc_commit(sh.done);
      mbar_wait(sh.done, 0, 100000000ull);
    }
    __syncwarp();
   }
  }
  if (!ok) {
    *sh.abort_flag = 1;
    if (lane == 0) raise_status(params.status, NBX_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if constexpr (W::kWaitLate) pdl_wait();
}

// ---- host side
PFN_cuTensorMapEncodeTiled_v12000 at_encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// A tiled bf16 map with 128-byte swizzle; dims and box innermost first, strides in bytes for dims 1...
bool at_encode(CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = at_encode_fn();
  if (fn == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class W, int D>
cudaError_t launch_attn_tiles(const typename W::Params& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};   // devices whose shared-memory limit is raised
  const uint64_t bit = 1ull << (device_info().device & 63);
  if ((configured.load() & bit) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<W, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               AttnCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_pdl(attn_tiles_kernel<W, D>, grid, kAtThreads, AttnCfg<D>::kSmem, stream, p);
}

}  // namespace
}  // namespace nbx
