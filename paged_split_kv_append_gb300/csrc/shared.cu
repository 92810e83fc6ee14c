// Decode attention for sequences that share a prefix of the cache: the prefix is read once for a whole group.
//
// The query vectors of all sequences of a group that belong to one KV head attend the group's prefix together, as the rows
// of the matrix products of attn_tiles.cuh; each sequence's own positions are read by the one-warp kernel of the modified
// decodes (decode_warp.cuh). Both leave partials (m, l, acc), and one merge joins them. Launches:
//   shared_plan_kernel     what each group shares, the splits of prefixes and own positions, the work lists
//   decode_partial_warp_kernel   the own positions
//   attn_tiles_kernel      the prefixes; it starts as the CTAs of the one before retire, and waits for it at its end
//   shared_merge_kernel
#include <algorithm>
#include <cmath>
#include <limits>

#include "attn_tiles.cuh"

namespace nbx {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kLeastPrefix = 128;      // positions: a shorter prefix is read with each sequence's own
constexpr int kPrefixSplits = 32;      // most splits of a prefix

struct PrefixParams {
  CUtensorMap q;      // [batch * rows][h_q][d], box {64, heads, tokens of a tile}
  CUtensorMap k, v;   // pools as rows of d, box {64, positions}
  SharedParams s;
  DecodeParams a;
  float c;            // |scale * k_scale| log2 e
  int negative;
  int32_t* status;
  int heads, sets;    // query heads of a tile; h_q / heads
  int box;            // positions of a copy: gcd(page_tokens, keys of a tile)
};

// Query heads of one tile: the whole group, if it fits, so that few sequences fill few tiles.
int prefix_heads(int group) {
  int f = std::min(group, kAtM);
  while (group % f) --f;
  return f;
}

// ---------------------------------------------------------------- plan
struct PlanArgs {
  SharedParams s;
  DecodeParams a;
  int tpt, tiles; // tokens of a tile; tiles of a prefix unit
  int sets;       // head sets
  int sms;
  // its query vectors fill one M tile of the two, which then take splits of their own
  __device__ __forceinline__ bool dual(const PrefixGroup& g) const { return tiles == 2 && g.n * a.rows <= tpt; }
};

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(PlanArgs x) {
  const SharedParams& s = x.s;
  const DecodeParams& p = x.a;
  __shared__ long long s_prefix, s_own;
  __shared__ int s_ok, s_empty, s_base, s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kPlanThreads / 32;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_tokens;
  if (tid == 0) {
    s_prefix = s_own = 0;
    s_ok = 1;
    s_empty = s_base = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  auto len_of = [&](int b, bool report) -> int {
    const int L = p.seq_lens[b];
    if (L >= 0 && L <= p.max_seq_len && L <= cap) return L;
    if (report) raise_status(p.status, NBX_DEV_BAD_LEN);
    return 0;
  };
  // ---- what each group shares
  for (int g = tid; g < s.n_groups; g += kPlanThreads) {
    const int b0 = s.group_start[g], b1 = s.group_start[g + 1];
    if (b0 < 0 || b1 < b0 || b1 > p.batch || s.shared_lens[g] < 0) s_ok = 0;   // no group counts then
  }
  for (int b = tid; b < p.batch; b += kPlanThreads) s.seqs[b] = make_int2(0, 0);
  __syncthreads();
  if (tid == 0 && !s_ok) raise_status(p.status, NBX_DEV_BAD_ROW);
  for (int g = warp; g < s.n_groups; g += kWarps) {
    const int b0 = s.group_start[g], n = s_ok ? s.group_start[g + 1] - b0 : 0;
    // every row of every member that holds something sees the prefix whole
    int least = s.shared_lens[g], live = 0, row = p.batch;
    for (int i = lane; i < n; i += 32) {
      const int L = len_of(b0 + i, false);
      if (L > 0) {
        ++live;
        row = min(row, b0 + i);
        least = min(least, L - p.rows + 1);
      }
    }
    live = __reduce_add_sync(0xffffffffu, live);
    row = __reduce_min_sync(0xffffffffu, row);
    least = __reduce_min_sync(0xffffffffu, least);
    const int eff = live >= 2 && least >= kLeastPrefix ? least / p.page_tokens * p.page_tokens : 0;
    if (lane == 0) {
      const int tpu = x.tpt * x.tiles, pairs = (n * p.rows + tpu - 1) / tpu;
      PrefixGroup pg = {b0, n, eff, 0, 0, pairs, 0, row};
      s.groups[g] = pg;
      // (a dual unit works through two splits in the time of one)
      if (eff > 0)
        atomicAdd(reinterpret_cast<unsigned long long*>(&s_prefix),
                  static_cast<unsigned long long>(eff) * pairs * x.sets * (x.dual(pg) ? 1 : 2));
    }
  }
  __syncthreads();
  // ---- its splits: about one unit an SM in all, and not below 256 positions
  for (int g = warp; g < s.n_groups; g += kWarps) {
    const PrefixGroup pg = s.groups[g];
    if (pg.eff == 0) continue;
    const long long want = (2ll * x.sms * pg.eff + s_prefix / 2) / s_prefix;
    const int least = x.dual(pg) ? 128 : 256;
    const int most = min(min(kPrefixSplits, p.max_splits / 2), (pg.eff + least - 1) / least);
    const int n = static_cast<int>(want < 1 ? 1 : (want > most ? most : want));
    const int seg = ((pg.eff + n - 1) / n + 127) / 128 * 128;
    const int splits = (pg.eff + seg - 1) / seg;
    for (int i = lane; i < pg.n; i += 32)
      if (len_of(pg.b0 + i, false) > 0) s.seqs[pg.b0 + i] = make_int2(pg.eff, splits);
    if (lane == 0) {
      s.groups[g].seg = seg;
      s.groups[g].splits = splits;
    }
  }
  __syncthreads();
  // ---- the prefixes' work list: each group's first unit
  if (warp == 0) {
    int base = 0;
    for (int g0 = 0; g0 < s.n_groups; g0 += 32) {
      const int g = g0 + lane;
      int units = 0;
      if (g < s.n_groups) {
        const PrefixGroup pg = s.groups[g];
        units = (x.dual(pg) ? (pg.splits + 1) / 2 : pg.splits) * pg.pairs * x.sets;
      }
      int sum = units;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (g < s.n_groups) s.groups[g].unit = base + sum - units;
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) p.header[4] = base;
  }
  // ---- the positions of each one's own
  long long part = 0;
  for (int b = tid; b < p.batch; b += kPlanThreads) {
    const int L = len_of(b, true);
    part += L - min(L, s.seqs[b].x);
  }
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0 && part) atomicAdd(reinterpret_cast<unsigned long long*>(&s_own), static_cast<unsigned long long>(part));
  __syncthreads();
  const int align = p.page_tokens <= NBX_SPLIT_POSITIONS ? p.page_tokens : NBX_SPLIT_POSITIONS;
  for (int b00 = 0; b00 < p.batch; b00 += kPlanThreads) {
    const int b = b00 + tid;
    int n = 0, seg = 1, L = 0;
    int2 sh = make_int2(0, 0);
    if (b < p.batch) {
      L = len_of(b, false);
      sh = s.seqs[b];
      const int own = L - sh.x;
      if (own > 0) {
        const long long num = static_cast<long long>(p.tc_units) * own, den = static_cast<long long>(p.tc_pairs) * s_own;
        const long long want = (num + den - 1) / den;
        const int most = min(p.max_splits - sh.y, max(1, own / 64));
        const int S = static_cast<int>(want < 1 ? 1 : (want > most ? most : want));
        seg = (own + S - 1) / S;
        seg = (seg + align - 1) / align * align;
        n = (own + seg - 1) / seg;
      }
      p.plan[b] = SeqPlan{L, seg, sh.y + n, sh.x};
      if (sh.y + n == 0) s_empty = 1;
    }
    int sum = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int base = s_base;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    base += sum - n;
    for (int i = 0; i < n; ++i) {
      Entry e;
      e.b = b;
      e.s = sh.y + i;
      e.start = sh.x + i * seg;
      e.end = min(L, sh.x + (i + 1) * seg);
      e.len = L;
      e.n_splits = sh.y + n;
      e.pad0 = e.pad1 = 0;
      p.entries[base + i] = e;
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) s_base = base + n;
    __syncthreads();
  }
  if (tid == 0) {
    p.header[0] = s_base;
    p.header[1] = 0;
    p.header[2] = kMergeSplits;
    p.header[3] = 0;
  }
  if (s_empty) {   // a sequence with no position to read: its rows are 0
    const int64_t vec4 = static_cast<int64_t>(p.rows) * p.h_q * p.d / (p.out_bf16 ? 8 : 4);
    for (int b = 0; b < p.batch; ++b) {
      if (p.plan[b].n_splits != 0) continue;
      float4* o = reinterpret_cast<float4*>(p.out) + b * vec4;
      for (int64_t i = tid; i < vec4; i += kPlanThreads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// ---------------------------------------------------------------- prefixes
template <int D, bool kE4, int kTermsOfP>
struct PrefixWork {
  using Params = PrefixParams;
  static constexpr int kN = kTermsOfP == 3 ? 64 : 128;   // keys of a tile
  static constexpr bool kF8 = kE4;
  static constexpr bool kPaged = true;
  static constexpr bool kWaitLate = true;
  static constexpr int kTerms = kTermsOfP;
  static constexpr bool kPairs = D <= 128;               // two M tiles a unit, or one over two ranges of keys
  // What is read before the grid ahead is waited for comes past L1 (__ldcg): the plan is complete, but an older line may
  // still lie there.
  const Params& p;
  int tpt, n_units;
  int ids_next[2], ids[2];   // loader: pages of lane's box, of the next K tile and the last (of M tile t, or the last two)
  int id_next;               // softmax: page of lane's 16-key piece of the next tile

  __device__ __forceinline__ int toks_per_tile() const { return tpt; }
  __device__ __forceinline__ int heads() const { return p.heads; }
  __device__ __forceinline__ PrefixWork(const Params& params, int) : p(params) {
    tpt = kAtM / p.heads;
    n_units = __ldcg(p.a.header + 4);
    ids_next[0] = ids_next[1] = ids[0] = ids[1] = id_next = 0;
  }
  __device__ __forceinline__ bool unit(uint32_t round, AttnUnit& u) const {
    const int64_t place = static_cast<int64_t>(round) * gridDim.x + blockIdx.x;
    if (place >= n_units) return false;
    const int un = static_cast<int>(place), lane = threadIdx.x & 31;
    // the last group whose first unit is not behind this one (groups without units share theirs with the next)
    int g = 0;
    for (int g0 = 0; g0 < p.s.n_groups; g0 += 32) {
      const bool at_or_before = g0 + lane < p.s.n_groups && __ldcg(&p.s.groups[g0 + lane].unit) <= un;
      const uint32_t has = __ballot_sync(0xffffffffu, at_or_before);
      if (has == 0) break;
      g = g0 + 31 - __clz(has);
    }
    const int4* const at_g = reinterpret_cast<const int4*>(p.s.groups + g);
    const int4 w0 = __ldcg(at_g), w1 = __ldcg(at_g + 1);
    const PrefixGroup pg = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    const int rest = un - pg.unit;
    const int pair = rest % pg.pairs, which = rest / pg.pairs;
    const int set = which % p.sets, split = which / p.sets;
    u.dual = kPairs && pg.n * p.a.rows <= tpt;
    const int tpu = (kPairs ? 2 : 1) * tpt;
    u.toks = min(tpu, pg.n * p.a.rows - pair * tpu);
    u.tok = pg.b0 * p.a.rows + pair * tpu;
    u.head = set * p.heads;
    u.kvh = u.head / p.a.group;
    u.pos = 0;
    u.b = pg.row;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u.slot[t] = u.dual ? 2 * split + t : split;
      u.kv[t] = u.slot[t] * pg.seg;
      u.end[t] = min(pg.eff, u.kv[t] + pg.seg);
      u.n[t] = max(0, u.end[t] - u.kv[t] + kN - 1) / kN;
    }
    if (!u.dual && !(kPairs && u.toks > tpt)) u.n[1] = 0;
    return true;
  }
  __device__ __forceinline__ int last_keys(const AttnUnit& u, int t) const {
    return u.end[t] - u.kv[t] - (u.n[t] - 1) * kN;
  }
  __device__ __forceinline__ int last_key(const AttnUnit& u, int t, int, bool) const { return u.end[t] - u.kv[t] - 1; }
  __device__ __forceinline__ bool in_pool(int page) const { return page >= 0 && page < p.a.num_pages; }
  // the page of the 16 (or box) positions from `at` on; 0 past the end
  __device__ __forceinline__ int page_at(const AttnUnit& u, int t, int at) const {
    return at < u.end[t] ? __ldcg(p.a.block_table + static_cast<int64_t>(u.b) * p.a.max_pages + at / p.a.page_tokens) : 0;
  }
  __device__ __forceinline__ uint32_t bad_keys(const AttnUnit& u, int t, int j, int c0) {
    constexpr int kPieces = (kPairs ? kN : kN / 2) / 16;
    const int lane = threadIdx.x & 31;
    const int at = u.kv[t] + j * kN + c0 + lane * 16;
    if (j == 0) id_next = lane < kPieces ? page_at(u, t, at) : 0;
    const int id = id_next;
    id_next = lane < kPieces ? page_at(u, t, at + kN) : 0;
    return __ballot_sync(0xffffffffu, !in_pool(id));
  }
  __device__ __forceinline__ const __nv_bfloat16* q_row(const AttnUnit& u, int tok, int head) const {
    return static_cast<const __nv_bfloat16*>(p.a.q) + ((static_cast<int64_t>(u.tok) + tok) * p.a.h_q + u.head + head) * D;
  }

  template <class C>
  __device__ __forceinline__ void load_q(const AttnUnit& u, char* q_s, uint64_t* bar) const {
    if ((threadIdx.x & 31) != 0) return;
    const uint32_t bytes = tpt * p.heads * 128;   // of an atom; the lanes behind them hold what was there
    mbar_arrive_expect_tx(bar, bytes * (D / 64) * (u.n[1] > 0 ? 2 : 1));
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t)
      if (u.n[t] > 0)
#pragma unroll
        for (int a = 0; a < D / 64; ++a)
          tma_load_3d(q_s + t * C::kQTile + a * C::kQAtom, &p.q, a * 64, u.head, u.tok + (u.dual ? 0 : t * tpt), bar);
  }
  // Lane l copies a box of positions (bf16: by 64 columns); page ids are fetched a tile ahead.
  template <class C>
  __device__ __forceinline__ void load_kv(const AttnUnit& u, bool is_v, int t, int j, int part, char* dst, uint64_t* bar) {
    const int lane = threadIdx.x & 31, box = p.box;
    const int boxes = kN / box;
    const int tile = u.kv[t] + j * kN;
    int id;
    if constexpr (kPairs) {   // V of a tile follows its K before the next K of the same M tile
      if (!is_v) {
        const int at = tile + lane * box;
        const int now = j == 0 ? (lane < boxes ? page_at(u, t, at) : 0) : ids_next[t];
        const int next = lane < boxes ? page_at(u, t, at + kN) : 0;
        if (t == 0) ids[0] = now, ids_next[0] = next;
        else ids[1] = now, ids_next[1] = next;
        if (lane < boxes && at < u.end[t] && !in_pool(now)) raise_status(p.status, NBX_DEV_BAD_PAGE);
      }
      id = t == 0 ? ids[0] : ids[1];
    } else {                  // K runs two tiles ahead of V, but for a unit's last
      if (!is_v && part == 0) {
        const int at = tile + lane * box;
        ids[1] = ids[0];
        ids[0] = j == 0 ? (lane < boxes ? page_at(u, t, at) : 0) : ids_next[0];
        ids_next[0] = lane < boxes ? page_at(u, t, at + kN) : 0;
        if (lane < boxes && at < u.end[t] && !in_pool(ids[0])) raise_status(p.status, NBX_DEV_BAD_PAGE);
      }
      id = is_v && j + 1 < u.n[0] ? ids[1] : ids[0];
    }
    if constexpr (kF8) {      // the codes as they are stored: a box of a head is one run of bytes
      const int at = tile + lane * box;
      const bool mine = lane < boxes && at < u.end[t], held = mine && in_pool(id);
      if (mine && !held) {    // 0 x whatever lay here must not be a NaN
        for (int i = 0; i < box * D; i += 16) *reinterpret_cast<uint4*>(dst + lane * box * D + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();  // a copy may fill the place next time
      }
      const uint32_t copies = __popc(__ballot_sync(0xffffffffu, held));
      if (lane == 0) mbar_arrive_expect_tx(bar, copies * box * D);
      __syncwarp();
      if (held) {
        const char* pool = static_cast<const char*>(is_v ? p.a.v_pool : p.a.k_pool);
        const int64_t row = (static_cast<int64_t>(id) * p.a.h_kv + u.kvh) * p.a.page_tokens + at % p.a.page_tokens;
        bulk_g2s(dst + lane * box * D, pool + row * D, box * D, bar);
      }
    } else {
      const bool half_v = C::kParts == 2 && is_v;                        // half of V's keys
      const int vbox = half_v && box > kN / 2 ? kN / 2 : box;            // (V has a map of its own for such boxes)
      const int atoms = C::kParts == 1 || is_v ? C::kAtoms : 2;          // columns of this slot
      const int here = (half_v ? kN / 2 : kN) / vbox;                    // boxes of this slot
      const int atom = lane / here, b = lane - atom * here;
      const int off = (half_v && part ? kN / 2 : 0) + b * vbox;          // in the tile
      const int at = tile + off;
      const int page = __shfl_sync(0xffffffffu, id, (off / box) & 31);
      const bool mine = atom < atoms && at < u.end[t];
      const uint32_t copies = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) mbar_arrive_expect_tx(bar, copies * vbox * 128);
      __syncwarp();
      if (mine) {   // a page outside the pool: rows before the tensor, which read as zeros
        const int row = in_pool(page) ? (page * p.a.h_kv + u.kvh) * p.a.page_tokens + at % p.a.page_tokens : -kN;
        const int col = (C::kParts == 2 && !is_v ? part * 2 + atom : atom) * 64;
        tma_load_2d(dst + atom * (half_v ? kN * 64 : kN * 128) + b * vbox * 128, is_v ? &p.v : &p.k, col, row, bar);
      }
    }
  }
  template <int kCols>
  __device__ __forceinline__ void store(const AttnUnit& u, int t, uint32_t o_base, int col0, int tok, int head, bool ok,
                                        float m, float l, uint64_t* o_free) const {
    const int lane = threadIdx.x & 31;
    const uint64_t keep = l2_keep_policy(p.a.keep_frac);
    const int64_t row = (static_cast<int64_t>(u.tok) + tok) * p.a.h_q + u.head + head;
    const int64_t at = row * p.a.max_splits + u.slot[t];
    if (ok && col0 == 0) {
      st_global_hint(p.a.m_part + at, m, keep);
      st_global_hint(p.a.l_part + at, l, keep);
    }
#pragma unroll
    for (int i = 0; i < kCols; i += 32) {
      uint32_t o[32];
      tmem_ld32(o_base + i, o);
      tmem_wait_ld();
      if (i + 32 == kCols) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      if (ok) {
        float* dst = p.a.acc_part + at * D + col0 + i;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) w[y] = __uint_as_float(o[e + y]);
          st_global_v8_hint(dst + e, w, keep);
        }
      }
    }
  }
};

// ---------------------------------------------------------------- merge
constexpr int kMergeWarps = 4;

// One warp per (query vector, 128 columns): M = max m_s, w_s = 2^(m_s - M) (a split with m = -inf is skipped),
// out = v_scale sum w_s acc_s / sum w_s l_s, s ascending. Sequences with one split and no prefix are written already.
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(SharedParams s, DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const int d4 = p.d / 4, pieces = (d4 + 31) / 32;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.rows * p.h_q;
  pdl_wait();
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5); it < rows * pieces;
       it += static_cast<int64_t>(gridDim.x) * kMergeWarps) {
    const int64_t row = it / pieces;
    const int j = static_cast<int>(it - row * pieces) * 32 + lane;
    const int b = static_cast<int>(row / (static_cast<int64_t>(p.rows) * p.h_q));
    const int S = p.plan[b].n_splits;
    if (S == 0 || (S == 1 && s.seqs[b].y == 0)) continue;
    const float* m = p.m_part + row * p.max_splits;
    const float* l = p.l_part + row * p.max_splits;
    const float4* acc = reinterpret_cast<const float4*>(p.acc_part + row * p.max_splits * p.d);
    constexpr int N = 16;   // splits whose accumulators are loaded at once
    float4 a[N];
    auto load = [&](int s0) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        a[k] = j < d4 && s0 + k < S ? acc[static_cast<int64_t>(s0 + k) * d4 + j] : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float mv[2], w[2], M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mv[k] = lane + 32 * k < S ? m[lane + 32 * k] : -INFINITY;
      w[k] = lane + 32 * k < S ? l[lane + 32 * k] : 0.f;
      M = max_nan(M, mv[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float e = mv[k] != -INFINITY ? fast_exp2(mv[k] - M) : -1.f;   // -1: skipped
      if (e != -1.f) L += e * w[k];
      w[k] = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float sc = p.v_scale / L;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += N) {
      if (s0 > 0) load(s0);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (s0 + k >= S) break;
        const float e = __shfl_sync(0xffffffffu, s0 + k < 32 ? w[0] : w[1], (s0 + k) & 31);
        if (e != -1.f) {
          A.x += e * a[k].x;
          A.y += e * a[k].y;
          A.z += e * a[k].z;
          A.w += e * a[k].w;
        }
      }
    }
    if (j >= d4) continue;
    const float4 o = M == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(A.x * sc, A.y * sc, A.z * sc, A.w * sc);
    if (p.out_bf16)
      reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * p.d)[j] =
          make_uint2(bf16x2_bits(o.x, o.y), bf16x2_bits(o.z, o.w));
    else
      reinterpret_cast<float4*>(p.out + row * p.d)[j] = o;
  }
}

bool encode_maps(PrefixParams* m, int pool_dtype, int tile_keys) {
  const DecodeParams& a = m->a;
  if (pool_dtype == NBX_E4M3) return true;   // queries by threads, codes by plain copies
  const cuuint64_t d = static_cast<cuuint64_t>(a.d);
  const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(a.h_q), static_cast<cuuint64_t>(a.batch) * a.rows};
  const cuuint64_t q_str[2] = {d * 2, static_cast<cuuint64_t>(a.h_q) * d * 2};
  const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(m->heads), static_cast<cuuint32_t>(kAtM / m->heads)};
  if (!at_encode(&m->q, 3, a.q, q_dims, q_str, q_box)) return false;
  const cuuint64_t dims[2] = {d, static_cast<cuuint64_t>(a.num_pages) * a.h_kv * a.page_tokens};
  const cuuint64_t str[1] = {d * 2};
  const cuuint32_t k_box[2] = {64, static_cast<cuuint32_t>(m->box)};
  const cuuint32_t v_box[2] = {64, static_cast<cuuint32_t>(a.d == 256 ? std::min(m->box, tile_keys / 2) : m->box)};
  return at_encode(&m->k, 2, a.k_pool, dims, str, k_box) && at_encode(&m->v, 2, a.v_pool, dims, str, v_box);
}

// The maps of the last few calls from this host thread, keyed by everything they encode.
struct PrefixKey {
  const void *q, *k, *v;
  int rows, h_q, h_kv, d, num_pages, page_tokens, pool_dtype, tile_keys, device;
  bool operator==(const PrefixKey& o) const {
    return q == o.q && k == o.k && v == o.v && rows == o.rows && h_q == o.h_q && h_kv == o.h_kv && d == o.d &&
           num_pages == o.num_pages && page_tokens == o.page_tokens && pool_dtype == o.pool_dtype && tile_keys == o.tile_keys &&
           device == o.device;
  }
};

const PrefixParams* prefix_maps(const DecodeParams& a, int heads, int box, int pool_dtype, int tile_keys, int device) {
  constexpr int kEntries = 8;
  thread_local PrefixKey keys[kEntries];
  thread_local PrefixParams maps[kEntries];
  thread_local int used = 0, next = 0;
  const PrefixKey key{a.q, a.k_pool, a.v_pool, a.batch * a.rows, a.h_q, a.h_kv, a.d, a.num_pages, a.page_tokens,
                      pool_dtype, tile_keys, device};
  for (int i = 0; i < used; ++i)
    if (keys[i] == key) return &maps[i];
  const int at = next;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  keys[at] = PrefixKey{};   // not valid until encoded
  maps[at].a = a;
  maps[at].heads = heads;
  maps[at].box = box;
  if (!encode_maps(&maps[at], pool_dtype, tile_keys)) return nullptr;
  keys[at] = key;
  return &maps[at];
}

template <int D, bool kE4, int kTerms>
cudaError_t launch_prefix(const SharedParams& s, const DecodeParams& a, cudaStream_t stream) {
  using W = PrefixWork<D, kE4, kTerms>;
  const DeviceInfo& di = device_info();
  const int heads = prefix_heads(a.group);
  int box = W::kN;
  while (a.page_tokens % box) box >>= 1;
  const PrefixParams* maps = prefix_maps(a, heads, box, kE4 ? NBX_E4M3 : NBX_BF16, W::kN, di.device);
  if (maps == nullptr) return cudaErrorInvalidValue;
  PrefixParams p = *maps;
  p.s = s;
  p.a = a;
  p.status = a.status;
  p.negative = a.qk_scale_log2 < 0.f;
  p.c = std::max(std::fabs(a.qk_scale_log2), std::numeric_limits<float>::denorm_min());
  p.heads = heads;
  p.sets = a.h_q / heads;
  p.box = box;
  return launch_attn_tiles<W, D>(p, static_cast<unsigned>(di.sm_count), stream);
}
template <int D>
cudaError_t launch_prefix(const SharedParams& s, const DecodeParams& a, int pool_dtype, cudaStream_t stream) {
  if (pool_dtype == NBX_E4M3)
    return a.out_bf16 ? launch_prefix<D, true, 1>(s, a, stream) : launch_prefix<D, true, 2>(s, a, stream);
  return a.out_bf16 ? launch_prefix<D, false, 1>(s, a, stream) : launch_prefix<D, false, 3>(s, a, stream);
}

}  // namespace

bool shared_layout(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len, int n_groups, SharedLayout* w) {
  WorkspaceLayout plain;   // what the decode takes where the prefixes are not read apart
  if (!workspace_layout(batch, rows, h_q, h_kv, d, max_seq_len, &plain, true)) return false;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const int64_t own = std::max(1, max_seq_len / 64);
  const int64_t pre = 2 * std::min<int64_t>(kPrefixSplits, (static_cast<int64_t>(max_seq_len) + 255) / 256);
  const size_t S = static_cast<size_t>(std::min<int64_t>(NBX_MAX_SPLITS, std::max<int64_t>(own + pre, 2)));
  const size_t prow = static_cast<size_t>(batch) * rows * h_q * S;
  if (prow > (static_cast<size_t>(1) << 40) / static_cast<size_t>(d)) return false;
  size_t off = 0;
  w->header = off;
  off += up(64 * 4);
  w->plan = off;
  off += up(static_cast<size_t>(batch) * sizeof(SeqPlan));
  w->entries = off;
  off += up(static_cast<size_t>(batch) * S * sizeof(Entry));
  w->m_part = off;
  off += up(prow * 4);
  w->l_part = off;
  off += up(prow * 4);
  w->acc_part = off;
  off += up(prow * static_cast<size_t>(d) * 4);
  w->seqs = off;
  off += up(static_cast<size_t>(batch) * sizeof(int2));
  w->groups = off;
  off += up(static_cast<size_t>(n_groups) * sizeof(PrefixGroup));
  w->total = std::max(off, plain.total);
  w->max_splits = static_cast<int>(S);
  return true;
}

bool prefix_path_applies(const DecodeParams& p, int q_dtype, int pool_dtype) {
  const int64_t pool_rows = static_cast<int64_t>(p.num_pages) * p.h_kv * p.page_tokens;
  return q_dtype == NBX_BF16 && (pool_dtype == NBX_E4M3 || (pool_dtype == NBX_BF16 && pool_rows < (int64_t{1} << 31) - 128));
}

cudaError_t shared_dispatch(const SharedParams& s, const DecodeParams& p, int q_dtype, int pool_dtype, int grid_limit,
                            cudaStream_t stream) {
  const DeviceInfo& di = device_info();
  DecodeParams q = p;
  // the one-warp kernel's units, as the modified decodes size them
  const int warps = di.sm_count * warp_path_warps(pool_dtype, p.d);
  q.tc_pairs = p.h_kv * ((p.rows * p.group + kWarpUnitVectors - 1) / kWarpUnitVectors);
  const int64_t extra = static_cast<int64_t>(q.tc_pairs) * p.batch / 2;
  q.tc_units = extra < warps / 2 ? warps - static_cast<int>(extra) : warps / 2;
  q.tc_warps = warps;
  q.tc_round_up = 1;
  PlanArgs x;
  x.s = s;
  x.a = q;
  const int heads = prefix_heads(p.group);
  x.tpt = kAtM / heads;
  x.tiles = p.d <= 128 ? 2 : 1;
  x.sets = p.h_q / heads;
  x.sms = di.sm_count;
  cudaError_t e = launch_pdl(shared_plan_kernel, 1u, kPlanThreads, 0, stream, x);
  if (e != cudaSuccess) return e;
  e = pool_dtype == NBX_E4M3 ? decode_dispatch_warp_e4m3(q, q_dtype, grid_limit, stream)
                             : decode_dispatch_warp_bf16(q, grid_limit, stream);
  if (e != cudaSuccess) return e;
  e = p.d == 64    ? launch_prefix<64>(s, q, pool_dtype, stream)
      : p.d == 128 ? launch_prefix<128>(s, q, pool_dtype, stream)
                   : launch_prefix<256>(s, q, pool_dtype, stream);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(p.batch) * p.rows * p.h_q * ((p.d / 4 + 31) / 32);
  const int64_t grid = std::min<int64_t>((items + kMergeWarps - 1) / kMergeWarps, static_cast<int64_t>(di.sm_count) * 8);
  return launch_pdl(shared_merge_kernel, static_cast<unsigned>(grid), kMergeWarps * 32, 0, stream, s, q);
}

}  // namespace nbx
