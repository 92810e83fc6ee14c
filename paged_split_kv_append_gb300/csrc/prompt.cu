// Causal attention over packed prompts with grouped heads, on the tiles of attn_tiles.cuh.
//
//  * A unit is (block of consecutive tokens of a sequence, `heads` query heads of one KV head): tokens and heads together
//    fill its M tiles, heads being the largest power of two that divides the group, so every tile but a sequence's last
//    is full whatever the group. K and V tiles start at the sequence's first token; key tiles past a tile's last
//    position are not read, and the scores of those on the diagonal are masked by selects.
//  * The number of tokens of each sequence is known on the device only. One warp of each CTA finds its units from
//    seq_start: units are ordered by their block's place in its sequence, the last (those with most keys) first, and
//    dealt to the CTAs there and back. With S(i) = the number of blocks at place i or later, unit u lies at the place i
//    with S(i + 1) <= u < S(i). No plan kernel, no workspace.
//  * A NaN or an infinity among the values that a tile holds but the row does not see (0 x NaN) stays out of it: a row whose
//    output is not finite, with such a value behind it in its last tile, is computed again key by key (prompt_row).
#include <algorithm>
#include <cmath>
#include <limits>

#include "attn_tiles.cuh"
#include "prompt_row.cuh"

namespace nbx {
namespace {

struct PromptTilesParams {
  CUtensorMap q;      // [n_tok][h_q][d], box {64, heads, tokens of a tile}
  CUtensorMap k, v;   // [h_kv][d / 64][n_tok][64], box {64, rows, atoms, 1}
  PromptParams a;
  float c;            // |scale| log2 e; for a scale of 0 the least positive number, which leaves every finite score 0
  int negative;       // the scale is
  int32_t* status;
  int heads, sets;    // query heads of a tile; h_q / heads
  __device__ __forceinline__ uint64_t wait_ns() const { return a.wait_limit_ns; }
  __device__ __forceinline__ uint64_t delay_ns() const { return a.producer_delay_ns; }
};

template <int D>
struct PromptWork {
  using Params = PromptTilesParams;
  using C = AttnCfg<D, 128, false>;
  static constexpr int kN = 128;   // keys of a tile
  static constexpr bool kF8 = false;
  static constexpr bool kPaged = false;
  static constexpr bool kBulk = false;
  static constexpr bool kMayWaitLate = false;
  static constexpr int kTerms = 1;
  const Params& p;
  int tpt, tpb;        // tokens of a tile, of a block
  int n_units, most;   // most blocks of a sequence
  int own_blocks;      // of sequence `lane`

  __device__ __forceinline__ static bool wait_late(const Params&) { return false; }
  __device__ __forceinline__ int toks_per_tile() const { return tpt; }
  __device__ __forceinline__ int heads() const { return p.heads; }
  __device__ __forceinline__ int blocks(int b) const {
    const int s = __ldg(p.a.seq_start + b), e = __ldg(p.a.seq_start + b + 1);
    return s >= 0 && e > s && e <= p.a.n_tok ? (e - s + tpb - 1) / tpb : 0;
  }
  __device__ __forceinline__ PromptWork(const Params& params) : p(params) { tpt = kAtM / p.heads; }
  __device__ __forceinline__ void begin() {
    const int lane = threadIdx.x & 31;
    tpb = C::kTiles * tpt;
    int sum = 0;
    most = 0;
    own_blocks = 0;
    for (int b = lane; b < p.a.batch; b += 32) {
      const int n = blocks(b);
      if (b == lane) own_blocks = n;
      sum += n;
      most = max(most, n);
    }
    n_units = __reduce_add_sync(0xffffffffu, sum) * p.sets;
    most = __reduce_max_sync(0xffffffffu, most);
    if (blockIdx.x == 0) {
      for (int b = lane; b < p.a.batch; b += 32) {
        const int s = p.a.seq_start[b], e = p.a.seq_start[b + 1];
        if (s < 0 || e < s || e > p.a.n_tok) raise_status(p.status, NBX_DEV_BAD_LEN);
      }
    }
  }
  // blocks at place i or later, of all sequences
  __device__ __forceinline__ int from_place(int i) const {
    int sum = max(0, own_blocks - i);
    for (int b = (threadIdx.x & 31) + 32; b < p.a.batch; b += 32) sum += max(0, blocks(b) - i);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  __device__ __forceinline__ bool unit(uint32_t round, AttnUnit& u) const {
    const int g = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
    const int64_t at = static_cast<int64_t>(round) * g + ((round & 1) ? g - 1 - cta : cta);
    if (at >= n_units) return false;
    const int su = static_cast<int>(at) / p.sets, set = static_cast<int>(at) - su * p.sets;
    int lo = 0, hi = most, above = 0;   // from_place(lo) > su >= from_place(hi) = above
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, n = from_place(mid);
      if (n > su) lo = mid;
      else {
        hi = mid;
        above = n;
      }
    }
    // the (su - above)-th sequence that has a block at place lo
    int left = su - above, b = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += 32) {
      const int mine = b0 + static_cast<int>(threadIdx.x & 31);
      const int n = b0 == 0 ? own_blocks : (mine < p.a.batch ? blocks(mine) : 0);
      const uint32_t has = __ballot_sync(0xffffffffu, n > lo);
      const int count = __popc(has);
      if (left < count) {
        const uint32_t below = has & ((1u << (threadIdx.x & 31)) - 1u);
        const bool here = ((has >> (threadIdx.x & 31)) & 1u) && __popc(below) == left;
        b = b0 + __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        break;
      }
      left -= count;
    }
    const int s = __ldg(p.a.seq_start + b), len = __ldg(p.a.seq_start + b + 1) - s;
    u.pos = lo * tpb;
    u.kv[0] = u.kv[1] = s;
    u.dual = 0;
    u.b = u.own = 0;
    u.end[0] = u.end[1] = u.slot[0] = u.slot[1] = 0;
    u.tok = s + u.pos;
    u.toks = min(tpb, len - u.pos);
    u.head = set * p.heads;
    u.kvh = u.head / (p.a.h_q / p.a.h_kv);
    u.n[1] = 0;
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t) {
      const int last = min(u.toks, (t + 1) * tpt) - 1;   // last token of the tile, within the unit
      u.n[t] = last >= t * tpt ? (u.pos + last) / kN + 1 : 0;
    }
    return true;
  }
  __device__ __forceinline__ int last_keys(const AttnUnit& u, int) const {
    return u.pos + u.toks - (max(u.n[0], u.n[1]) - 1) * kN;
  }
  __device__ __forceinline__ int last_key(const AttnUnit& u, int, int tok, bool ok) const { return ok ? u.pos + tok : 1 << 30; }

  template <class>
  __device__ __forceinline__ void load_q(const AttnUnit& u, char* q_s, uint64_t* bar) const {
    if ((threadIdx.x & 31) != 0) return;
    mbar_arrive_expect_tx(bar, C::kQTile * (C::kTiles == 2 && u.n[1] > 0 ? 2 : 1));
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t)
      if (u.n[t] > 0)
#pragma unroll
        for (int a = 0; a < D / 64; ++a)
          tma_load_3d(q_s + t * C::kQTile + a * C::kQAtom, &p.q, a * 64, u.head, u.tok + t * tpt, bar);
  }
  template <class>
  __device__ __forceinline__ void load_kv(const AttnUnit& u, bool is_v, int, int j, int part, char* dst, uint64_t* bar,
                                          int) const {
    if ((threadIdx.x & 31) != 0) return;
    mbar_arrive_expect_tx(bar, C::kSlotBytes);
    const int row = u.kv[0] + j * kN;
    if (is_v) tma_load_4d(dst, &p.v, 0, row + part * (kN / 2), 0, u.kvh, bar);
    else tma_load_4d(dst, &p.k, 0, row, part * 2, u.kvh, bar);
  }
  template <int kCols>
  __device__ __forceinline__ void store(const AttnUnit& u, int t, uint32_t o_base, int col0, int tok, int head, bool ok, float m,
                                        float l, uint64_t* o_free, AttnControl* ctl) const {
    const int lane = threadIdx.x & 31;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.a.out);
    const int64_t row = (static_cast<int64_t>(u.tok) + tok) * p.a.h_q + u.head + head;
    f32x2 sick = pack2(0.f, 0.f);   // 0, or a NaN if some value is not finite
#pragma unroll
    for (int i = 0; i < kCols; i += 32) {
      uint32_t o[32];
      tmem_ld32(o_base + i, o);
      tmem_wait_ld();
      if (i + 32 == kCols) {   // O is free for the next unit's first PV
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      const f32x2 inv2 = pack2(inv, inv), zero2 = pack2(0.f, 0.f);
      float w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const f32x2 x = mul2(pack2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2);
        sick = fma2(x, zero2, sick);
        const float2 y = unpack2(x);
        w[e] = __uint_as_float(bf16x2_bits(y.x, y.y));
      }
      if (ok) {
        float* dst = reinterpret_cast<float*>(out + row * D + col0 + i);
        st_global_v8(dst, *reinterpret_cast<const float(*)[8]>(w));
        st_global_v8(dst + 8, *reinterpret_cast<const float(*)[8]>(w + 8));
      }
    }
    const float2 s = unpack2(sick);
    const bool odd = ok && !(s.x + s.y == 0.f);
    if (!__any_sync(0xffffffffu, odd)) return;
    if (odd && l == 0.f) {   // every score is -inf: 0
      const float none[8] = {};
#pragma unroll 1
      for (int i = 0; i < kCols; i += 16) st_global_v8(reinterpret_cast<float*>(out + row * D + col0 + i), none);
    }
    // A score that is a NaN leaves l one, and the row its NaN. For the others: is there a value that is not finite behind the
    // row, among those that its tile's last products took?
    const __nv_bfloat16* const v = static_cast<const __nv_bfloat16*>(p.a.v) + u.kv[0] * p.a.v_stride + static_cast<int64_t>(u.kvh) * D;
    const bool may = odd && l > 0.f;
    if (!__any_sync(0xffffffffu, may)) return;
    const int pos = u.pos + tok, first = __reduce_min_sync(0xffffffffu, may ? pos + 1 : 0x7fffffff);
    const int last = last_not_finite(v, p.a.v_stride, first, min(u.n[t] * kN, u.pos + u.toks), col0, col0 + kCols);
    uint32_t again = __ballot_sync(0xffffffffu, may && pos < last);
    if (!again) return;
    at_busy(ctl, 1);
    while (again) {
      const int src = __ffs(again) - 1;
      again &= again - 1;
      const int rt = __shfl_sync(0xffffffffu, tok, src);
      const int64_t rr = __shfl_sync(0xffffffffu, row, src);
      prompt_row<D>(static_cast<const __nv_bfloat16*>(p.a.q) + (static_cast<int64_t>(u.tok) + rt) * p.a.q_stride +
                        (rr % p.a.h_q) * D,
                    static_cast<const __nv_bfloat16*>(p.a.k) + u.kv[0] * p.a.k_stride + static_cast<int64_t>(u.kvh) * D,
                    v, p.a.k_stride, p.a.v_stride, u.pos + rt + 1, p.a.scale_log2, out + rr * D, col0, col0 + kCols);
    }
    at_busy(ctl, -1);
  }
};

bool encode_maps(PromptTilesParams* m) {
  const PromptParams& a = m->a;
  const cuuint64_t d = static_cast<cuuint64_t>(a.d), n = static_cast<cuuint64_t>(a.n_tok);
  const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(a.h_q), n};
  const cuuint64_t q_str[2] = {d * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
  const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(m->heads), static_cast<cuuint32_t>(kAtM / m->heads)};
  if (!at_encode(&m->q, 3, a.q, q_dims, q_str, q_box)) return false;
  const cuuint64_t dims[4] = {64, n, d / 64, static_cast<cuuint64_t>(a.h_kv)};
  const cuuint64_t k_str[3] = {static_cast<cuuint64_t>(a.k_stride) * 2, 128, d * 2};
  const cuuint64_t v_str[3] = {static_cast<cuuint64_t>(a.v_stride) * 2, 128, d * 2};
  constexpr cuuint32_t kN = 128;   // PromptWork's
  const cuuint32_t k_box[4] = {64, kN, static_cast<cuuint32_t>(a.d == 64 ? 1 : 2), 1};
  const cuuint32_t v_box[4] = {64, static_cast<cuuint32_t>(a.d == 256 ? kN / 2 : kN),
                               static_cast<cuuint32_t>(a.d == 256 ? 4 : a.d / 64), 1};
  return at_encode(&m->k, 4, a.k, dims, k_str, k_box) && at_encode(&m->v, 4, a.v, dims, v_str, v_box);
}

// The maps of the last few shapes from this host thread, put over a call's addresses: three encodings cost a call a few
// microseconds.
struct PromptKey {
  int64_t qs, ks, vs;
  int n_tok, h_q, h_kv, d;
  bool operator==(const PromptKey& o) const {
    return qs == o.qs && ks == o.ks && vs == o.vs && n_tok == o.n_tok && h_q == o.h_q && h_kv == o.h_kv && d == o.d;
  }
};

bool prompt_maps(PromptTilesParams* p) {
  constexpr int kEntries = 8;
  thread_local PromptKey keys[kEntries];
  thread_local CUtensorMap maps[kEntries][3];
  thread_local int used = 0, next = 0;
  const PromptParams& a = p->a;
  const PromptKey key{a.q_stride, a.k_stride, a.v_stride, a.n_tok, a.h_q, a.h_kv, a.d};
  for (int i = 0; i < used; ++i) {
    if (!(keys[i] == key)) continue;
    p->q = maps[i][0];
    p->k = maps[i][1];
    p->v = maps[i][2];
    return at_rebase(&p->q, a.q) && at_rebase(&p->k, a.k) && at_rebase(&p->v, a.v);
  }
  if (!encode_maps(p)) return false;
  keys[next] = key;
  maps[next][0] = p->q;
  maps[next][1] = p->k;
  maps[next][2] = p->v;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  return true;
}

template <int D>
cudaError_t launch_prompt(const PromptParams& a, cudaStream_t stream) {
  const DeviceInfo& di = device_info();
  int heads = a.h_q / a.h_kv;
  heads = std::min(heads & -heads, kAtM);   // the largest power of two in the group
  PromptTilesParams p;
  p.a = a;
  p.status = a.status;
  p.negative = a.scale_log2 < 0.f;
  p.c = std::max(std::fabs(a.scale_log2), std::numeric_limits<float>::denorm_min());
  p.heads = heads;
  p.sets = a.h_q / heads;
  if (!prompt_maps(&p)) return cudaErrorInvalidValue;
  const int tpb = AttnCfg<D, 128, false>::kTiles * kAtM / heads;
  // a sequence has its blocks and at most one that is not full
  const int64_t most = (static_cast<int64_t>(a.n_tok) / tpb + std::min(a.batch, a.n_tok)) * p.sets;
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(di.sm_count, most)));
  return launch_attn_tiles<PromptWork<D>, D>(p, grid, stream);
}

}  // namespace

cudaError_t prompt_dispatch(const PromptParams& p, cudaStream_t stream) {
  if (p.d == 64) return launch_prompt<64>(p, stream);
  if (p.d == 128) return launch_prompt<128>(p, stream);
  return launch_prompt<256>(p, stream);
}

}  // namespace nbx
