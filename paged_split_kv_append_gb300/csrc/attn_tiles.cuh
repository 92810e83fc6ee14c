// Attention of 128-row tiles of query vectors on tcgen05: what prompt attention and the shared-prefix decode run. (A
// prompt of 16384 tokens, 32 / 8 heads of 128, takes 1442 us, at 80 % of the measured matrix rate and the power limit.)
//
// A work unit is one or two M tiles of 128 query vectors of one KV head (a tile holds some tokens with `heads` query heads
// each) and the keys they attend, in tiles of kN. Per key tile, with scores in log2 units:
//   S = Q K^T;  m' = max(m, rowmax S) (moved only when it grows by more than 2^8);  P = 2^(c S - m'), 2^-8 to 1 at most;
//   l = l 2^(m - m') + rowsum P;  O = O 2^(m - m') + P V.
// S and O are fp32 accumulators in TMEM; P is written over S in kTerms terms of the values' 16-bit type: one for bf16
// outputs (each weight off by up to 2^-8 of itself in bf16, as much as the output's own rounding; 2^-11 in f16), for fp32
// outputs as many as leave 2^-22 or less (three in bf16, two in f16), on key tiles of 64, whose S leaves them room.
//
// One persistent CTA per SM, sixteen warps, every wait bounded:
//  * warps 0-3 and 4-7: two softmax groups. Up to d = 128 each has an M tile of its own, one row a thread, and the two
//    take turns with the tensor pipe: while one group works on its S, the MMAs of the other's tile run. Both tiles attend
//    the same keys, or (dual units, whose query vectors fill one tile) the same vectors attend two ranges of keys. At
//    d = 64 a P of 16-bit terms has columns of its own, the next S is computed while this one's exponentials run, and the
//    turns fall away (8 prompts of 700 to 1700 tokens, 16 heads of 64: 52.4 us in turns, 46.7 so: 1.2 us for 128 keys, of
//    which S is waited for in 0.06; one softmax warp of a scheduler alone takes 0.5 us, two 1.0, in step or out of it). At
//    d = 256 O fills half of the TMEM, so there is one M tile, S is double-buffered, and the groups share each row, half
//    of the columns each; the two threads of a row swap their maxima through shared memory.
//  * warps 9 and 10 issue the MMAs: QK^T (both operands from shared memory) and PV (P from TMEM, N = d). Up to d = 128 each
//    has an M tile: waiting for P(j) is all that orders PV(j), and QK(j + 1) of the same tile follows it in the pipe and
//    may overwrite P(j). At d = 256 warp 9 has the PVs and warp 10 the QK^Ts. A single warp's chain of waits and issues
//    took 2.4 us for 128 keys and two tiles of d = 128, whose MMAs take 1.1.
//  * warp 8 fills the ring of K and V with TMA: slots of a whole tile, or at d = 256 half of one (128 columns of K, half of
//    V's keys); and the unit's Q tiles.
//  * Paged K and V come by 16-byte cp.async of warps 12-15. (A tensor copy costs the copy engine some 135 ns whatever its
//    size, and pages of 16 positions take 16 of 2 KB for 32 KB.)
//  * warp 11 finds the units and hands them to the others through shared memory, one ahead.
//  * E4M3 pools: warps 8 and 11 copy the codes of a tile as they are stored (bulk copies or cp.async), and warps 12-15 convert them to f16
//    (exactly) into the ring. Queries enter as f16 too, times a power of two that brings the largest element of each
//    vector into [2^14, 2^15): exact but for elements under 2^-29 of it. The softmax threads write them, each its own row,
//    and take the factor back in their row's c. The running maximum sits 2^7 above P's largest weight then, so that small
//    weights keep their bits in f16's range.
// What bounds it: the tensor pipe (d = 64: the softmax). Per 128 keys and two tiles of d = 128 it is busy 2048 cycles; the
// softmax issues about 900 instructions on each scheduler and takes 1024 cycles of the special-function units (4 a warp
// measured).
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
constexpr int kAtBuf = 128;       // TMEM columns of an S/P buffer
constexpr int kAtThreads = 512;
// Registers a thread: of the 128 each is launched with, the eight warps of copies and MMAs give what a softmax thread
// needs to hold its 128 scores: 200 + 56 = 2 * 128.
constexpr int kAtSoftmaxRegs = 200, kAtOtherRegs = 56;
constexpr int kAtCopyWarps = 4;   // warps 12-15
constexpr float kAtTau = 8.f;     // the running maximum moves when it would grow by more, log2 units

template <int D, int N, bool F8>
struct AttnCfg {
  static constexpr int kTiles = D <= 128 ? 2 : 1;                // M tiles of a unit
  static constexpr int kParts = D <= 128 ? 1 : 2;                // ring slots of a K or V tile
  static constexpr int kAhead = D <= 128 ? 1 : 2;                // QK^T of tile j + kAhead follows PV of tile j
  static constexpr int kCols = D <= 128 ? N : N / 2;             // columns of S a softmax thread takes
  static constexpr int kAtoms = D / 64;                          // 64-column atoms of a row
  static constexpr int kSlotBytes = N * D * 2 / kParts;
  static constexpr int kQAtom = kAtM * 128;                      // 128 rows of 128 bytes
  static constexpr int kQTile = kAtoms * kQAtom;
  static constexpr int kRawBytes = F8 ? N * D : 0;               // a tile of codes
  static constexpr int kRaws = F8 ? 4 : 0;
  static constexpr int kRoom = 224 * 1024 - kTiles * kQTile - kRaws * kRawBytes;
  static constexpr int kMost = F8 ? (kTiles == 2 ? 6 : 5) : (kTiles == 2 ? 8 : 6);   // (what the barriers and xbuf leave)
  static constexpr int kSlots = kRoom / kSlotBytes < kMost ? kRoom / kSlotBytes : kMost;
  static constexpr int kRingOff = kTiles * kQTile;
  static constexpr int kRawOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kBarOff = kRawOff + kRaws * kRawBytes;
  static constexpr int kBarBytes = 384;
  static constexpr int kUnitOff = kBarOff + kBarBytes;
  static constexpr int kXOff = kUnitOff + 128;                   // two units
  static constexpr int kSmem = kXOff + (kTiles == 1 ? 2 * 256 * 4 : 0);
  static constexpr uint32_t kOCol = 2 * kAtBuf;                  // S (and P) in columns [0, 256), O from there
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSlots >= 3, "ring");
  static_assert((2 * kSlots + 2 * kRaws + 18) * 8 <= kBarBytes - 64, "barrier area");
};

// One work unit. (It is moved as 16-byte words: where it lies in local memory, too, it is aligned to them.)
struct alignas(16) AttnUnit {
  int tok;        // first token of the first tile (rows of the query tensor)
  int toks;       // tokens of the unit, of both tiles
  int head, kvh;  // first query head, KV head
  int pos;        // causal: position of the first token in its sequence; paged: how many positions that token sees
  int b;          // paged: row of the block table
  int dual;       // the two tiles are the same query vectors, over keys of their own
  int kv[2];      // causal: first key's row; paged: first position
  int end[2];     // paged: one past the last position
  int slot[2];    // paged: slot of the partials
  int n[2];       // key tiles of each M tile
  int own;        // paged: the positions are a sequence's own
};
static_assert(sizeof(AttnUnit) == 64, "a unit is four 16-byte words");

// What the roles of a CTA share beside barriers, in shared memory.
struct AttnControl {
  int abort;          // some role has given up
  int busy;           // warps that compute rows again: as long as there are some, no wait runs out
  uint64_t wait_ns;   // how long a wait may take
  uint32_t tmem;      // TMEM's first column
};
static_assert(sizeof(AttnControl) <= 32, "x_bar lies behind it");
__device__ __forceinline__ const volatile AttnControl* volatile_of(const AttnControl* c) { return c; }
__device__ __forceinline__ void volatile_set(AttnControl* c) { static_cast<volatile AttnControl*>(c)->abort = 1; }
// This warp begins (1) or ends (-1) to compute rows again, which takes as long as their keys are many, and ends by itself.
__device__ __forceinline__ void at_busy(AttnControl* c, int more) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) atomicAdd(&c->busy, more);
}

// Bounded wait of a whole warp, with one answer: gives up when another role of the CTA has, or after the limit (2 s, but in
// a test of this path), which begins anew while some warp computes rows again. Every branch is on a vote, so the compiler knows the warp to be together behind it (and may use
// uniform registers there).
// The loop is a function, one for all sites of the warps beside the softmax (whose registers leave no room for a call): up to
// fourteen warps wait at a time, and loops of their own pushed the others' code out of the instruction caches (stalls for
// want of an instruction were a third of a shared E4M3 prefix's cycles).
__device__ __forceinline__ bool at_wait_loop(uint32_t bar, uint32_t parity, const AttnControl* ctl) {
  uint64_t t0 = global_timer_ns();
  for (;;) {
    uint32_t ok = 0;
#pragma unroll 1
    for (int i = 0; i < 4 && !ok; ++i) {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
      ok = __all_sync(0xffffffffu, ok != 0);
    }
    if (ok) return true;
    const bool busy = volatile_of(ctl)->busy != 0;
    const uint64_t now = global_timer_ns();
    if (__any_sync(0xffffffffu, volatile_of(ctl)->abort != 0 || (!busy && now - t0 > ctl->wait_ns))) return false;
    if (busy) t0 = now;
  }
}
__device__ __noinline__ bool at_wait_call(uint32_t bar, uint32_t parity, const AttnControl* ctl) {
  return at_wait_loop(bar, parity, ctl);
}
template <bool kCall = true>
__device__ __forceinline__ bool at_warp_wait(uint64_t* bar, uint32_t parity, const AttnControl* ctl) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  if constexpr (kCall) return __all_sync(0xffffffffu, at_wait_call(smem_u32(bar), parity, ctl));
  return at_wait_loop(smem_u32(bar), parity, ctl);
}
// x, the same in every lane of the warp, as a value that the compiler knows to be
__device__ __forceinline__ int at_uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

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
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 f16x2_floats(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Four E4M3 codes to two f16 pairs, exactly (the low two codes in lo).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Calls f(is_v, t, j) for the K and V tiles of a unit in the order in which the MMA warp consumes them (t: the M tile that
// they are for, 0 where both read them). f returns false to give up.
// (One place to call it from: f is long, and inlined.)
template <class C, class F>
__device__ __forceinline__ bool at_each_tile(const AttnUnit& u, F f) {
  const bool dual = C::kTiles == 2 && u.dual;
  const int n0 = u.n[0], n1 = u.n[1], n = C::kTiles == 2 ? max(n0, n1) : n0;
#pragma unroll 1
  for (int j = -C::kAhead; j < n; ++j) {
#pragma unroll 1
    for (int i = 0; i < (dual ? 4 : 2); ++i) {   // V of tile j, K of tile j + kAhead, for each tile of a dual unit
      const int t = i >> 1, at = (i & 1) ? j + C::kAhead : j;
      if (at < 0 || at >= (dual ? (t ? n1 : n0) : n)) continue;
      if (!f((i & 1) == 0, t, at)) return false;
    }
  }
  return true;
}

// d = 64 leaves TMEM for a P of its own beside S (three terms would not fit)
template <class W, int D>
constexpr bool kAtOwnP = D == 64 && W::kN == 128 && W::kTerms == 1;
constexpr int kAtPCol = 384;      // [2][64] columns

// What a work policy W provides (prompt.cu, shared.cu):
//   typename W::Params with c (|scale| log2 e, or the least positive number for a scale of 0), negative and status;
//   W::kN, kTerms, kF8, kBulk, kPaged, kMayWaitLate and wait_late(params); begin() and bool unit(round, AttnUnit&) of the warp that
//   finds the units (toks > 0 in each); toks_per_tile(), heads(); last_keys, last_key, bad_keys; load_q / load_kv by the
//   loader warps (or q_row for the softmax threads); store(...) by a softmax warp.
template <class C>
struct AttnShared {
  char* q_s;
  char* ring;
  char* raw;
  uint64_t* full;      // [kSlots] a ring slot holds its part of a tile
  uint64_t* empty;     // [kSlots] its MMAs are done
  uint64_t* q_full;
  uint64_t* q_empty;   // every QK^T of the unit is done
  uint64_t* s_full;    // [2] S in its buffer (of M tile t, or of key tile j & 1)
  uint64_t* p_full;    // [2] P over it
  uint64_t* pv_done;   // [2] the PV from that buffer is done: O holds it
  uint64_t* o_free;    // [2] the epilogue has read O of M tile t
  uint64_t* unit_full; // [2] a unit is written, every reader has read it
  uint64_t* unit_empty;
  AttnUnit* units;     // [2]
  uint64_t* turn;      // [2] d <= 128: it is the turn of M tile t's warp to issue; own P: S of tile t is in registers
  uint64_t* done;
  uint64_t* raw_full;  // [kRaws] a tile's codes have landed
  uint64_t* raw_empty; // [kRaws] and are converted
  uint64_t* x_bar;     // [4] d = 256: the two warps of 32 rows have left their numbers
  AttnControl* ctl;
  float* xbuf;         // [2][256]
};

// ---------------------------------------------------------------- units
// The k-th unit of this CTA, to every warp that asks: false behind the last, and when the wait for it ran out (which the
// abort flag says).
template <bool kCall = true, class C>
__device__ __forceinline__ bool at_unit(const AttnShared<C>& sh, uint32_t k, AttnUnit& u) {
  if (!at_warp_wait<kCall>(&sh.unit_full[k & 1u], (k >> 1) & 1u, sh.ctl)) {
    volatile_set(sh.ctl);
    return false;
  }
  uint4* const to = reinterpret_cast<uint4*>(&u);
  const uint32_t from = smem_u32(sh.units + (k & 1u));
#pragma unroll
  for (int i = 0; i < 4; ++i) to[i] = lds128(from + 16 * i);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.unit_empty[k & 1u]);
  return u.toks > 0;
}
// Finds the units; `each` is called with every one of them.
template <class W, class C, class F>
__device__ __forceinline__ bool attn_units(W& w, const AttnShared<C>& sh, F each) {
  w.begin();
  bool more = true;
  for (uint32_t k = 0; more; ++k) {
    AttnUnit u = {};
    more = w.unit(k, u);
    if (!more) u.toks = 0;
    if (k >= 2 && !at_warp_wait(&sh.unit_empty[k & 1u], ((k >> 1) - 1) & 1u, sh.ctl)) return false;
    if ((threadIdx.x & 31) == 0) {
      const uint4* const from = reinterpret_cast<const uint4*>(&u);
      const uint32_t to = smem_u32(sh.units + (k & 1u));
#pragma unroll
      for (int i = 0; i < 4; ++i) sts128(to + 16 * i, from[i]);
      mbar_arrive(&sh.unit_full[k & 1u]);
    }
    __syncwarp();
    if (more && !each(u)) return false;
  }
  return true;
}

// ---------------------------------------------------------------- the MMA warps
// MMAs and commits of one lane, as predicated instructions: the warp stays together, so that descriptors are computed once
// a warp, in uniform registers. (In a branch of one lane every operand went there by itself, and issuing 8 MMAs took 420 ns,
// twice their time in the tensor pipe.)
// Four K steps of 16: A advances by 32 bytes of its swizzled rows, B too (K-major) or by 16 rows (MN-major), or A by 8
// TMEM columns. `left`: steps that there are.
__device__ __forceinline__ void at_mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 b2, %2, 4;\n\t"
      "add.s64 a3, %1, 6;\n\tadd.s64 b3, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void at_mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, int left) {
  asm volatile(
      "{\n\t.reg .pred p, q0, q1, q2, q3;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.gt.s32 q0, %5, 0;\n\tsetp.gt.s32 q1, %5, 1;\n\tsetp.gt.s32 q2, %5, 2;\n\tsetp.gt.s32 q3, %5, 3;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\tadd.s32 a2, %1, 16;\n\tadd.s64 b2, %2, 256;\n\t"
      "add.s32 a3, %1, 24;\n\tadd.s64 b3, %2, 384;\n\t"
      "@q0 tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q1 tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@q2 tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@q3 tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(left)
      : "memory");
}
__device__ __forceinline__ void at_commit(uint64_t* bar, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(issue)
      : "memory");
}

// which: the M tile of this warp, or at d = 256 what it issues (0: PV, 1: QK^T).
template <class W, class C, int D>
__device__ __forceinline__ bool attn_mma(W& w, const AttnShared<C>& sh, uint32_t tmem, int which) {
  constexpr int T = C::kTiles, NS = C::kSlots, N = W::kN;
  constexpr int kAtomBytes = N * 128 / C::kParts;   // of V: N (or N / 2) rows of 128 bytes
  constexpr uint32_t kIdescO = mma_idesc(kAtM, D, true, W::kF8);
  // a negative scale: S of -Q (the descriptor's bit 13 negates A), and its magnitude
  const uint32_t idesc_s = mma_idesc(kAtM, N, false, W::kF8) | (w.p.negative ? 1u << 13 : 0u);
  const int lane = threadIdx.x & 31;
  const uint32_t one = lane == 0;    // the lane that issues
  const int t = T == 2 ? which : 0;
  const bool does_pv = T == 2 || which == 0, does_qk = T == 2 || which == 1;
  const AttnControl* ab = sh.ctl;
  const uint32_t ring = smem_u32(sh.ring);
  const uint64_t q_desc = smem_desc(smem_u32(sh.q_s) + t * C::kQTile, 16, 1024);
  const uint64_t k_desc = smem_desc(ring, 16, 1024), v_desc = smem_desc(ring, kAtomBytes, 1024);
  const uint32_t o_addr = tmem + C::kOCol + t * D;
  constexpr bool kOwnP = kAtOwnP<W, D>;
  int slot = 0;                      // the ring slot next consumed, in the loader's order, and its phase
  uint32_t phase = 0;
  uint32_t p_phase = 0, s_phase = 0; // bit: phase of a P buffer; d = 256: of the PV that frees an S buffer
  uint32_t o_phase = 0;
  bool o_used = false;               // O has been used
  uint32_t x = 0;                    // d = 256: key tiles so far (the buffer is bit 0)
  uint32_t steps = 0;                // turns so far
  AttnUnit u;
  // The slots of the next tile (C::kParts of them, in a row but for the ring's end): the first, or -1. Both warps wait for
  // every slot, their own or not, and both give it back: a parity wait must know the phase before to be over, and the one
  // after not to be.
  int second = 0;
  auto acquire = [&]() -> int {
    const int first = slot;
#pragma unroll
    for (int i = 0; i < C::kParts; ++i) {
      if (!at_warp_wait(&sh.full[slot], phase, ab)) return -1;
      if (i == 1) second = slot;
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
    return first;
  };
  auto release = [&](int first, int next, bool own) {
    if (own) {   // once its MMAs are done
      at_commit(&sh.empty[first], one);
      if constexpr (C::kParts == 2) at_commit(&sh.empty[next], one);
    } else if (one) {
      mbar_arrive(&sh.empty[first]);
      if constexpr (C::kParts == 2) mbar_arrive(&sh.empty[next]);
    }
  };
  auto fences = [&]() {
    if constexpr (W::kPaged && !W::kF8) fence_proxy_async();   // written by cp.async
    tc_fence_after();
  };
  // The other M tile's warp may issue
  auto pass_turn = [&]() {
    if constexpr (T == 2) {
      if (one) mbar_arrive(&sh.turn[t ^ 1]);
    }
  };
  // S(buffer) = Q K^T
  auto qk = [&](uint32_t buf, int first, int next) {
    const uint64_t k0 = k_desc + first * (C::kSlotBytes >> 4), k1 = C::kParts == 2 ? k_desc + next * (C::kSlotBytes >> 4) : 0;
#pragma unroll
    for (int a = 0; a < C::kAtoms; ++a) {
      const uint64_t kd = C::kParts == 1 ? k0 + (a * (N * 128) >> 4) : (a < 2 ? k0 : k1) + ((a & 1) * (N * 128) >> 4);
      at_mma_ss4(tmem + buf * kAtBuf, q_desc + (a * C::kQAtom >> 4), kd, idesc_s, a > 0, one);
    }
  };
  // O += P(buffer) V, `keys` of the tile's keys
  auto pv = [&](uint32_t buf, int first, int next, int keys, bool fresh) {
    constexpr int kSteps = N / 16, kPartSteps = kSteps / C::kParts;
    const int steps = one ? (keys + 15) >> 4 : 0;
    const uint64_t v0 = v_desc + first * (C::kSlotBytes >> 4), v1 = C::kParts == 2 ? v_desc + next * (C::kSlotBytes >> 4) : 0;
    const uint32_t p = kOwnP ? tmem + kAtPCol + t * 64 : tmem + buf * kAtBuf;
    if constexpr (kPartSteps % 4 == 0) {
#pragma unroll
      for (int term = 0; term < W::kTerms; ++term)
#pragma unroll
        for (int kk = 0; kk < kSteps; kk += 4)
          at_mma_ts4(o_addr, p + term * (N / 2) + kk * 8, (kk < kPartSteps ? v0 : v1) + ((kk % kPartSteps) * 2048 >> 4),
                     kIdescO, !(term == 0 && kk == 0 && fresh), steps - kk);
    } else {   // two steps a slot (d = 256, 64 keys)
#pragma unroll
      for (int term = 0; term < W::kTerms; ++term)
#pragma unroll
        for (int kk = 0; kk < kSteps; kk += 2)
          at_mma_ts4(o_addr, p + term * (N / 2) + kk * 8, kk < kPartSteps ? v0 : v1, kIdescO,
                     !(term == 0 && kk == 0 && fresh), min(2, steps - kk));
    }
  };
  // rows of V past the last key inside its 16-key step are zeroed: 0 x NaN would reach every row. (Both warps of a slot do,
  // to the same effect.)
  auto clear_tail = [&](int first, int next, int keys) {
    if ((keys & 15) == 0) return;
    const int to = (keys + 15) & ~15;
    constexpr int kRows = N / C::kParts;
    for (int row = keys; row < to; ++row)
      for (int i = lane; i < D / 8; i += 32) {   // 16-byte pieces of the row: D / 64 atoms of 8
        const uint32_t off = ring + (row < kRows ? first : next) * C::kSlotBytes + (i >> 3) * kAtomBytes +
                             (row % kRows) * 128 + (i & 7) * 16;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(off), "r"(0) : "memory");
      }
    fence_proxy_async();
    __syncwarp();
  };
  auto q_ready = [&](uint32_t k) -> bool {
    if (!at_warp_wait(sh.q_full, k & 1u, ab)) return false;
    tc_fence_after();
    return true;
  };
  for (uint32_t k = 0; at_unit(sh, k, u); ++k) {
    if (does_qk && !q_ready(k)) return false;
    const int n0 = at_uniform(u.n[0]), n1 = T == 2 ? at_uniform(u.n[1]) : 0;
    const int n = max(n0, n1), nt = t == 0 ? n0 : n1;
    const bool dual = T == 2 && at_uniform(u.dual);
    const int last = at_uniform(w.last_keys(u, t));
    for (int j = -C::kAhead; j < n; ++j) {
      // the slots of the other tile of a dual unit, V of key tile j and K of tile j + kAhead
      auto pass = [&](int no) -> bool {
        for (int is_k = 0; is_k < 2; ++is_k)
          if (is_k ? j + C::kAhead < no : j >= 0 && j < no) {
            const int at = acquire();
            if (at < 0) return false;
            release(at, second, false);
          }
        return true;
      };
      if (dual && t == 1 && !pass(n0)) return false;
      const int no = dual ? nt : n;   // key tiles with slots that this warp has a part in
      const bool pvs = does_pv && j >= 0 && j < nt, qks = does_qk && j + C::kAhead < nt;
      const uint32_t buf = T == 2 ? t : x & 1u;
      // ---- V, P and O of key tile j
      int vs = -1, vs2 = 0;
      if (j >= 0 && j < no) {
        if ((vs = acquire()) < 0) return false;
        vs2 = second;
        if (!does_pv) release(vs, vs2, false);
      }
      // ---- K of tile j + kAhead: asked for early where it has been there for long
      int ks = -1, ks2 = 0;
      auto take_k = [&]() -> bool {
        if (j + C::kAhead >= no) return true;
        if ((ks = acquire()) < 0) return false;
        ks2 = second;
        if (!does_qk) release(ks, ks2, false);
        return true;
      };
      constexpr bool kEarlyK = T == 2 && (kOwnP || !W::kPaged);
      if constexpr (kEarlyK)
        if (!take_k()) return false;
      if constexpr (kOwnP) {
        if (qks) {
          if (steps > 0 && !at_warp_wait(&sh.turn[t], (steps - 1) & 1u, ab)) return false;
          ++steps;
          fences();
          qk(buf, ks, ks2);
          at_commit(&sh.s_full[buf], one);
        }
        if (ks >= 0) release(ks, ks2, true);
        if (j + C::kAhead == n - 1) at_commit(sh.q_empty, one);
      }
      if (pvs) {
        const int keys = j + 1 < no ? N : last;
        clear_tail(vs, vs2, keys);
        if (j == 0) {
          if (o_used) {
            if (!at_warp_wait(&sh.o_free[t], o_phase, ab)) return false;
            o_phase ^= 1u;
          }
          o_used = true;
        }
        if (!at_warp_wait(&sh.p_full[buf], (p_phase >> buf) & 1u, ab)) return false;
        p_phase ^= 1u << buf;
      }
      // ---- the two M tiles' warps issue in turns, PV and QK^T together: side by side their MMAs mix in the pipe, both S are
      // done at the same time, and then the pipe waits for two softmaxes at once (16384 tokens of 32 heads: 1872 us, 1588
      // in turns)
      if constexpr (T == 2 && !kOwnP) {
        if ((t == 1 || steps > 0) && !at_warp_wait(&sh.turn[t], (steps - (t == 0)) & 1u, ab)) return false;
        ++steps;
      }
      if (pvs) {
        fences();
        pv(buf, vs, vs2, j + 1 < no ? N : last, j == 0);
      }
      if constexpr (!kEarlyK)
        if (!take_k()) return false;
      if (qks && !kOwnP) {
        if constexpr (T == 1) {   // the buffer's last PV is done (in the pipe of another warp)
          if (x >= 2) {
            if (!at_warp_wait(&sh.pv_done[buf], (s_phase >> buf) & 1u, ab)) return false;
            s_phase ^= 1u << buf;
          }
        }
        fences();
        qk(buf, ks, ks2);
      }
      if constexpr (!kOwnP) pass_turn();
      if (pvs) at_commit(&sh.pv_done[buf], one);
      if (qks && !kOwnP) at_commit(&sh.s_full[buf], one);
      if (T == 1 && (pvs || qks)) ++x;
      if (does_pv && vs >= 0) release(vs, vs2, true);
      if (does_qk && ks >= 0 && !kOwnP) release(ks, ks2, true);
      if (dual && t == 0 && !pass(n1)) return false;
      if (j + C::kAhead == n - 1 && does_qk && !kOwnP) at_commit(sh.q_empty, one);
    }
  }
  return true;
}

// ---------------------------------------------------------------- queries of E4M3 pools
// This thread's query vector (null: zeros) times 2^e as f16 into row `row` of a Q tile's swizzled atoms, elements
// [d0, d0 + kCount) of it. Returns 2^-e. (Past L1: the grid ahead may not have been waited for yet.)
template <int D, int kCount>
__device__ __forceinline__ float q_to_f16(const __nv_bfloat16* q, char* tile, int row, int d0) {
  const uint4* src = reinterpret_cast<const uint4*>(q);
  const uint32_t to = smem_u32(tile) + row * 128;
  auto place = [&](int i) { return to + (i >> 3) * (kAtM * 128) + (((i & 7) ^ (row & 7)) << 4); };
  float amax = 0.f;
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = q != nullptr ? __ldcg(src + i) : make_uint4(0u, 0u, 0u, 0u);
    float2 x[4];
    unpack16<BF16>(v, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = max_nan(amax, max_nan(fabsf(x[e].x), fabsf(x[e].y)));
    if (kCount == D || (i >= d0 / 8 && i < (d0 + kCount) / 8)) sts128(place(i), v);   // as it is, for the second pass
  }
  int e2 = 0;   // a NaN or an infinity in the vector: as it is
  if (amax > 0.f && amax <= 3.402823466e38f)
    e2 = min(120, max(-120, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127)));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
#pragma unroll 4
  for (int i = d0 / 8; i < (d0 + kCount) / 8; ++i) {
    uint32_t w[4];
    float2 x[4];
    unpack16<BF16>(lds128(place(i)), x);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = f16x2_bits(x[e].x * up, x[e].y * up);
    sts128(place(i), make_uint4(w[0], w[1], w[2], w[3]));
  }
  return __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
}

// ---------------------------------------------------------------- a softmax warp
template <class W, class C, int D>
__device__ __forceinline__ bool attn_softmax(W& w, const AttnShared<C>& sh, uint32_t tmem) {
  constexpr int T = C::kTiles, NC = C::kCols, N = W::kN;
  constexpr int kOCols = T == 2 ? D : D / 2;   // columns of O that this thread rescales and stores
  // log2 of the largest weight when m has moved. In bf16 and fp32 as low as keeps weights at 1 or less until it moves again:
  // O then passes fp32's range no sooner than in sums of weights under a maximum that always moves (values of 2^118 and
  // weights of 2^7.5 did). In f16's range as high as it goes: E4M3's values are 448 at most.
  constexpr float kMid = W::kF8 ? 7.f : -kAtTau;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp >> 2, quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const int t = T == 2 ? group : 0;
  const uint32_t o_base = lane_base + C::kOCol + t * D + (T == 2 ? 0 : group * kOCols);
  const int c0 = T == 2 ? 0 : group * NC;      // first column of S
  const int tpt = w.toks_per_tile();
  const int tok = row / w.heads(), head = row - tok * w.heads();
  float c = w.p.c;
  constexpr bool kOwnP = kAtOwnP<W, D>;
  const AttnControl* ab = sh.ctl;
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
    const bool ok = at_warp_wait<false>(&sh.x_bar[quarter], xphase & 1u, ab);
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
    const bool ok = T == 2 ? at_warp_wait<false>(&sh.pv_done[t], y & 1u, ab) : at_warp_wait<false>(&sh.pv_done[y & 1u], (y >> 1) & 1u, ab);
    tc_fence_after();
    return ok;
  };
  AttnUnit u;
  for (uint32_t k = 0; at_unit<false>(sh, k, u); ++k) {
    const int n = u.n[t];
    const int my_tok = (u.dual ? 0 : t * tpt) + tok;        // of the unit
    const bool row_ok = tok < tpt && my_tok < u.toks;
    if constexpr (W::kF8) {
      if (k > 0 && !at_warp_wait<false>(sh.q_empty, (k - 1) & 1u, ab)) return false;
      if (n > 0) {
        const float down = q_to_f16<D, kOCols>(row_ok ? w.q_row(u, my_tok, head) : nullptr, sh.q_s + t * C::kQTile, row,
                                               T == 2 ? 0 : group * kOCols);
        c = fmaxf(w.p.c * down, 1.4012985e-45f);   // (0 x a masked score would be a NaN)
        fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.q_full);
    }
    if (n == 0) continue;
    const int last_key = w.last_key(u, t, my_tok, row_ok);  // of the unit's keys, from 0
    float m = -INFINITY, l = 0.f;                           // weights are 2^(c s - m)
    for (int j = 0; j < n; ++j, ++x) {
      const uint32_t buf = T == 2 ? t : (x & 1u);
      const uint32_t s_col = lane_base + buf * kAtBuf;
      uint32_t bad = 0;                                     // paged: 16-key pieces of this thread's columns without a page
      if constexpr (W::kPaged) bad = w.bad_keys(u, t, j, c0);
      if (!at_warp_wait<false>(&sh.s_full[buf], (T == 2 ? x : x >> 1) & 1u, ab)) return false;
      tc_fence_after();
      uint32_t s[NC];
#pragma unroll
      for (int i = 0; i < NC; i += 32) tmem_ld32(s_col + c0 + i, s + i);
      tmem_wait_ld();
      if constexpr (kOwnP) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.turn[t]);
      }
      const int limit = last_key - (j * N + c0);             // this thread's columns up to here are seen
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
      const bool up = z > m + (kMid + kAtTau);
      const float f = up ? fast_exp2(m - (z - kMid)) : 1.f;
      if (up) m = z - kMid;
      const float neg = m == -INFINITY ? 0.f : -m;
      const f32x2 c2 = pack2(c, c), neg2 = pack2(neg, neg);
      f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};   // a tile's weights by themselves: beside l's 2^24 a 1 is lost
      constexpr int kChunk = NC < 64 ? NC : 64;   // columns of S whose terms are stored at once
#pragma unroll
      for (int h = 0; h < NC; h += kChunk) {
        uint32_t term[W::kTerms][kChunk / 2];
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
          const float2 e = unpack2(fma2(pack2(__uint_as_float(s[h + 2 * i]), __uint_as_float(s[h + 2 * i + 1])), c2, neg2));
          float a = fast_exp2(e.x), b = fast_exp2(e.y);
          sum[i & 1] = add2(sum[i & 1], pack2(a, b));
#pragma unroll
          for (int y = 0; y < W::kTerms; ++y) {
            const uint32_t bits = W::kF8 ? f16x2_bits(a, b) : bf16x2_bits(a, b);
            term[y][i] = bits;
            if (y + 1 < W::kTerms) {
              const float2 g = W::kF8 ? f16x2_floats(bits) : bf16x2_to_float2(bits);
              a -= g.x;
              b -= g.y;
            }
          }
        }
        if (kOwnP && h == 0 && j > 0 && !pv_wait()) return false;   // (the last P has been read)
#pragma unroll
        for (int y = 0; y < W::kTerms; ++y) {
          const uint32_t at = kOwnP ? lane_base + kAtPCol + t * 64 + h / 2 : s_col + y * (N / 2) + (c0 + h) / 2;
          if constexpr (kChunk == 64) tmem_st32(at, term[y]);
          else tmem_st16(at, term[y]);
        }
      }
      const float2 s0 = unpack2(sum[0]), s1 = unpack2(sum[1]);
      l = fmaf(l, f, (s0.x + s0.y) + (s1.x + s1.y));
      // O follows a maximum that moved, once the last PV into it is done
      if (j > 0 && __any_sync(0xffffffffu, up)) {
        if (!pv_wait()) return false;
        const f32x2 f2 = pack2(f, f);
#pragma unroll(W::kF8 ? 1 : kOCols / 32)   // (an E4M3 prefix has more code beside it: 99.3 us unrolled, 96.9 so)
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
    w.template store<kOCols>(u, t, o_base, T == 2 ? 0 : group * kOCols, my_tok, head, row_ok, m, l, &sh.o_free[t], sh.ctl);
  }
  return true;
}

// ---------------------------------------------------------------- a converting warp (E4M3 pools)
// Codes of K and V tiles, [keys][D] as they are stored, to f16 in the ring's swizzled atoms. Warp `which` takes every fourth
// group of 8 rows of a slot. Lane (rr, i) takes 16 codes of row rr, of atom (rr & 1) ^ s in turn s: the eight lanes that
// access shared memory at a time then read 128 bytes of distinct banks, and write 16-byte chunks of distinct ones.
// kRows rows and kAtoms atoms of a slot, this warp's quarter; 4 pieces of 16 codes are loaded before the first is converted
// (one at a time, by two warps, a slot of 128 rows took 1.3 us).
template <int D, int kRows, int kAtoms>
__device__ __forceinline__ void convert_slot(const char* src, char* dst, int which, int rr, int i) {
  constexpr int kSides = kAtoms > 1 ? 2 : 1;
  constexpr int kItems = kRows / 32 * kAtoms;   // a warp's pieces of a lane: (group of 8 rows, pair of atoms, side)
  constexpr int kBatch = kItems < 4 ? kItems : 4;
  const uint32_t from = smem_u32(src) + (which * 8 + rr) * D + i * 16;
  const uint32_t to = smem_u32(dst) + (which * 8 + rr) * 128;
  const uint32_t c0 = ((2 * i) ^ rr) << 4, c1 = ((2 * i + 1) ^ rr) << 4;
#pragma unroll 1
  for (int b = 0; b < kItems; b += kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int item = b + e, g = item / kAtoms, y = item % kAtoms;
      const int atom = kSides == 2 ? (y & ~1) + ((rr & 1) ^ (y & 1)) : 0;
      v[e] = lds128(from + g * (32 * D) + atom * 64);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int item = b + e, g = item / kAtoms, y = item % kAtoms;
      const int atom = kSides == 2 ? (y & ~1) + ((rr & 1) ^ (y & 1)) : 0;
      uint4 lo, hi;
      e4m3x4_to_f16x4(v[e].x, lo.x, lo.y);
      e4m3x4_to_f16x4(v[e].y, lo.z, lo.w);
      e4m3x4_to_f16x4(v[e].z, hi.x, hi.y);
      e4m3x4_to_f16x4(v[e].w, hi.z, hi.w);
      const uint32_t at = to + atom * (kRows * 128) + g * 4096;
      sts128(at + c0, lo);
      sts128(at + c1, hi);
    }
  }
}

template <class W, class C, int D>
__device__ __forceinline__ bool attn_convert(W& w, const AttnShared<C>& sh, int which) {
  constexpr int NS = C::kSlots, N = W::kN;
  const int lane = threadIdx.x & 31;
  const int rr = lane >> 2, i = lane & 3;
  uint32_t r = 0, x = 0;   // ring slots, tiles
  AttnUnit u;
  for (uint32_t k = 0; at_unit(sh, k, u); ++k) {
    const bool ok = at_each_tile<C>(u, [&](bool is_v, int, int) -> bool {
      if (!at_warp_wait(&sh.raw_full[x % C::kRaws], (x / C::kRaws) & 1u, sh.ctl)) return false;
      const char* raw = sh.raw + (x % C::kRaws) * C::kRawBytes;
      for (int part = 0; part < C::kParts; ++part, ++r) {
        if (r >= NS && !at_warp_wait(&sh.empty[r % NS], (r / NS - 1) & 1u, sh.ctl)) return false;
        char* dst = sh.ring + (r % NS) * C::kSlotBytes;
        // the part's rows and atoms: at d = 256 two atoms of every row of K, half of V's rows
        const bool half_v = C::kParts == 2 && is_v;
        const char* src = raw + (C::kParts == 2 && part ? (is_v ? N / 2 * D : 128) : 0);
        if (half_v) convert_slot<D, N / 2, C::kAtoms>(src, dst, which, rr, i);
        else convert_slot<D, N, (C::kParts == 2 ? 2 : C::kAtoms)>(src, dst, which, rr, i);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[r % NS]);
      }
      if (lane == 0) mbar_arrive(&sh.raw_empty[x % C::kRaws]);
      ++x;
      return true;
    });
    if (!ok) return false;
  }
  return true;
}

template <class W, int D>
__global__ void __launch_bounds__(kAtThreads, 1) attn_tiles_kernel(const __grid_constant__ typename W::Params params) {
  using C = AttnCfg<D, W::kN, W::kF8>;
  constexpr int NS = C::kSlots;
  constexpr bool kCopies = W::kPaged && !W::kF8;   // warps 12-15 load K and V (else warp 8)
  extern __shared__ __align__(1024) char smem[];
  AttnShared<C> sh;
  sh.q_s = smem;
  sh.ring = smem + C::kRingOff;
  sh.raw = smem + C::kRawOff;
  sh.full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  sh.empty = sh.full + NS;
  sh.raw_full = sh.empty + NS;
  sh.raw_empty = sh.raw_full + C::kRaws;
  sh.q_full = sh.raw_empty + C::kRaws;
  sh.q_empty = sh.q_full + 1;
  sh.s_full = sh.q_full + 2;
  sh.p_full = sh.q_full + 4;
  sh.pv_done = sh.q_full + 6;
  sh.o_free = sh.q_full + 8;
  sh.done = sh.q_full + 10;
  sh.turn = sh.q_full + 12;
  sh.unit_full = sh.q_full + 14;
  sh.unit_empty = sh.q_full + 16;
  sh.units = reinterpret_cast<AttnUnit*>(smem + C::kUnitOff);
  sh.ctl = reinterpret_cast<AttnControl*>(sh.full + (C::kBarBytes - 64) / 8);   // (before x_bar)
  sh.x_bar = reinterpret_cast<uint64_t*>(smem + C::kUnitOff) - 4;   // d = 256 (whose ring is short): behind them
  sh.xbuf = reinterpret_cast<float*>(smem + C::kXOff);
  const int warp = at_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], W::kF8 ? kAtCopyWarps : (W::kPaged ? 32 * kAtCopyWarps : 1));
      mbar_init(&sh.empty[i], 2);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(&sh.raw_full[i], W::kBulk ? 2 : 64);
      mbar_init(&sh.raw_empty[i], kAtCopyWarps);
    }
    mbar_init(sh.q_full, W::kF8 ? 8 : 1);
    mbar_init(sh.q_empty, C::kTiles);
    constexpr int kRowWarps = C::kTiles == 2 ? 4 : 8;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kRowWarps);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.o_free[i], kRowWarps);
    }
    mbar_init(sh.done, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      // the softmax and MMA warps, the loader, and the warps that copy or convert
      mbar_init(&sh.unit_empty[i], 11 + (W::kPaged ? kAtCopyWarps : 0));
    }
    if constexpr (C::kTiles == 2)
      for (int i = 0; i < 2; ++i) mbar_init(&sh.turn[i], kAtOwnP<W, D> ? kRowWarps : 1);
    if constexpr (C::kTiles == 1)
      for (int i = 0; i < 4; ++i) mbar_init(&sh.x_bar[i], 2);
    sh.ctl->abort = 0;
    sh.ctl->busy = 0;
    sh.ctl->wait_ns = params.wait_ns();
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = at_uniform(volatile_of(sh.ctl)->tmem);
  // the inputs are written and visible from here on. (wait_late: they were before the grid ahead began, which this one
  // may run beside; the grid behind waits for both through this one)
  if (!W::wait_late(params)) pdl_wait();
  pdl_launch_dependents();
  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtSoftmaxRegs));
    W w(params);
    ok = attn_softmax<W, C, D>(w, sh, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtOtherRegs));
    if (warp == 8 || warp == 11 || (kCopies && warp >= 12)) {
      // ---- Q of each unit (warp 8), and K and V in the order in which the MMA warps consume them: warp 8, or for paged
      // pools warps 12-15, or for E4M3 pools, whose Q the softmax threads write, warps 8 and 11, which finds the units too
      W w(params);
      constexpr int kDepth = W::kF8 ? C::kRaws : NS, kPieces = W::kF8 ? 1 : C::kParts;
      constexpr int kBytes = W::kF8 ? C::kRawBytes : C::kSlotBytes;
      uint64_t* const full = W::kF8 ? sh.raw_full : sh.full;
      uint64_t* const empty = W::kF8 ? sh.raw_empty : sh.empty;
      char* const ring = W::kF8 ? sh.raw : sh.ring;
      const int loader = kCopies ? warp - 12 : (warp == 11);
      if (params.delay_ns() != 0) {   // a test holds the loaders back so that the other roles' waits run out
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < params.delay_ns()) __nanosleep(10000);
      }
      uint32_t r = 0, q_units = 0, phase = 1;   // (the first round finds every slot empty)
      int slot = 0;
      auto next_q = [&](const AttnUnit& u) -> bool {
        if (q_units > 0 && !at_warp_wait(sh.q_empty, (q_units - 1) & 1u, sh.ctl)) return false;
        w.template load_q<C>(u, sh.q_s, sh.q_full);
        ++q_units;
        return true;
      };
      auto tiles = [&](const AttnUnit& u) -> bool {
        bool first = !W::kF8 && !kCopies;   // Q comes behind the first key tile, which need not wait for the last unit's Q
        return at_each_tile<C>(u, [&](bool is_v, int t, int j) -> bool {
#pragma unroll 1
          for (int part = 0; part < kPieces; ++part, ++r) {
            if (r >= kDepth && !at_warp_wait(&empty[slot], phase, sh.ctl)) return false;
            w.template load_kv<C>(u, is_v, t, j, part, ring + slot * kBytes, &full[slot], loader);
            if (++slot == kDepth) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (first) {
            first = false;
            return next_q(u);
          }
          return true;
        });
      };
      if (warp == 11) {
        ok = attn_units<W, C>(w, sh, [&](const AttnUnit& u) -> bool {
          if constexpr (W::kF8) return tiles(u);
          return true;
        });
      } else {
        AttnUnit u;
        for (uint32_t k = 0; ok && at_unit(sh, k, u); ++k) ok = kCopies && warp == 8 ? next_q(u) : tiles(u);
      }
      if (!ok) volatile_set(sh.ctl);
      // the copies issued last have landed before the CTA can exit
      if constexpr (W::kPaged) cp_async_wait_all();
      if (lane == 0) {
        for (uint32_t i = r > kDepth ? r - kDepth : 0; i < r; ++i) mbar_wait(&full[i % kDepth], (i / kDepth) & 1u, 100000000ull);
        if (q_units > 0) mbar_wait(sh.q_full, (q_units - 1) & 1u, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 9 || warp == 10) {
      W w(params);
      ok = attn_mma<W, C, D>(w, sh, tmem, warp - 9);
      if (!ok) volatile_set(sh.ctl);
      // every MMA of this CTA has completed before the TMEM is released
      at_commit(sh.done, lane == 0);
      mbar_wait(sh.done, 0, 100000000ull);
      __syncwarp();
    } else if (W::kF8 && warp >= 12) {
      if constexpr (W::kF8) {
        W w(params);
        ok = attn_convert<W, C, D>(w, sh, warp - 12);
      }
    }
  }
  if (!ok) volatile_set(sh.ctl);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && volatile_of(sh.ctl)->abort != 0) raise_status(params.status, NBX_DEV_TIMEOUT);
  if (warp == 9) tmem_dealloc(tmem, 512);
  if constexpr (W::kMayWaitLate) pdl_wait();
}

// ---- host side
template <class Fn>
Fn at_driver_fn(const char* name) {
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<Fn>(f);
}

// A tiled bf16 map with 128-byte swizzle; dims and box innermost first, strides in bytes for dims 1...
bool at_encode(CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box) {
  static const auto fn = at_driver_fn<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled");
  if (fn == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same map over another address.
bool at_rebase(CUtensorMap* map, const void* base) {
  static const auto fn = at_driver_fn<PFN_cuTensorMapReplaceAddress_v12000>("cuTensorMapReplaceAddress");
  return fn != nullptr && fn(map, const_cast<void*>(base)) == CUDA_SUCCESS;
}

template <class W, int D>
cudaError_t launch_attn_tiles(const typename W::Params& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};   // devices whose shared-memory limit is raised
  const uint64_t bit = 1ull << (device_info().device & 63);
  if ((configured.load() & bit) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<W, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (AttnCfg<D, W::kN, W::kF8>::kSmem));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_pdl(attn_tiles_kernel<W, D>, grid, kAtThreads, (AttnCfg<D, W::kN, W::kF8>::kSmem), stream, p);
}

}  // namespace
}  // namespace nbx
