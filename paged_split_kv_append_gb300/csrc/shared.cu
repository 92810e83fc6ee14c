// Decode attention for sequences that share a prefix of the cache: the prefix is read once for a whole group.
//
// The query vectors of all sequences of a group that belong to one KV head attend the group's prefix together, as the rows
// of the matrix products of attn_tiles.cuh. Each sequence's own positions are work units of the same kernel where the
// sequence has many query vectors to a KV head (kOwnTileVectors), and read by the one-warp kernel of the modified decodes
// (decode_warp.cuh) where it has few. All leave partials (m, l, acc), and one merge joins them. Launches:
//   shared_plan_kernel     what each group shares, the splits of prefixes and own positions, the work lists
//   decode_partial_warp_kernel   own positions of few vectors
//   attn_tiles_kernel      the prefixes (behind the one-warp kernel it starts as that one's CTAs retire, and waits for it at
//                          its end), and own positions of many vectors
//   shared_merge_kernel
#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

#include "attn_tiles.cuh"

namespace nbx {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kLeastPrefix = 128;      // positions: a shorter prefix is read with each sequence's own
constexpr int kPrefixSplits = 32;      // most splits of a prefix
// From so many query vectors to a KV head of a sequence on, the tiles read its own positions too. The one-warp kernel reads
// keys once for every 8 vectors, on a tensor path that makes little of them: behind a prefix of 4096, 32 sequences' 10 to
// 1000 own positions of one KV head of 128 take a call of 32 vectors to 39.9 us, 29.7 in the tiles (E4M3 46.1 and 35.8); 128
// vectors to four KV heads 127.0 and 85.0 (140.3 and 103.4); 8 to two 35.8 and 31.7 (37.9 and 35.8); 24 to four 48.1 and
// 44.0 (but 56.3 and 58.4). Five documents of 6000 to 20000, four rows of 24 heads of 256: 119.9 and 108.9. But 64 sequences
// with 4 vectors to eight KV heads 47.3 and 59.0: a unit of few keys costs the tiles as much for 4 rows as for 128.
constexpr int kOwnTileVectors = 8;

struct PrefixParams {
  CUtensorMap q;      // [batch * rows][h_q][d], box {64, heads, tokens of a tile}
  SharedParams s;
  DecodeParams a;
  float c;            // |scale * k_scale| log2 e
  int negative;
  int32_t* status;
  int heads, sets;    // query heads of a tile; h_q / heads
  bool own_tiles;     // as PlanArgs'
  __device__ __forceinline__ uint64_t wait_ns() const { return a.wait_limit_ns; }
  __device__ __forceinline__ uint64_t delay_ns() const { return a.producer_delay_ns; }
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
  bool small;     // its arrays lie in shared memory
  int own_pairs;  // units that a range of a sequence's own positions takes for one head set
  bool own_dual;  // such a unit takes two ranges
  // its query vectors fill one M tile of the two, which then take splits of their own
  __device__ __forceinline__ bool dual(const PrefixGroup& g) const { return tiles == 2 && g.n * a.rows <= tpt; }
  __device__ __forceinline__ int units_of(const PrefixGroup& g, int splits) const { return dual(g) ? (splits + 1) / 2 : splits; }
  // `len` positions in at most `most` splits of about `want`: their number, even if a unit takes two, and positions (of
  // whole key tiles)
  __device__ __forceinline__ static void cut(int len, bool two, int most, int want, int& n, int& seg) {
    n = min(most, static_cast<int>((static_cast<uint32_t>(len) + want - 1) / static_cast<uint32_t>(want)));
    if (two) n = min(most, (n + 1) / 2 * 2);
    seg = ((len - 1) / n + 128) & ~127;
    n = (len - 1) / seg + 1;
  }
  __device__ __forceinline__ void cut(const PrefixGroup& g, int want, int& n, int& seg) const {
    cut(g.eff, dual(g), min(kPrefixSplits, a.max_splits / 2), want, n, seg);
  }
  // (there is room for a split of every 64 of a sequence's positions beside the prefix's)
  __device__ __forceinline__ void cut_own(int own, int pre, int want, int& n, int& seg) const {
    cut(own, own_dual, a.max_splits - pre, want, n, seg);
  }
  __device__ __forceinline__ int own_entries(int n) const { return own_dual ? (n + 1) / 2 : n; }
};

constexpr int kPlanBatch = 2048, kPlanGroups = 512;   // up to these the plan works in shared memory
inline bool plan_small(int batch, int n_groups) { return batch <= kPlanBatch && n_groups <= kPlanGroups; }
inline size_t plan_smem(int batch, int n_groups) {
  return plan_small(batch, n_groups) ? static_cast<size_t>(n_groups) * sizeof(PrefixGroup) + static_cast<size_t>(batch) * 12 : 0;
}

// One CTA. What it reads (lengths, groups) it reads once, all at a time: a chain of dependent reads from global memory took
// 7.5 us of a call. (Larger batches keep their arrays in the workspace, and read lengths again.)
// kOwnTiles: own positions are units of the tiles, too. (Asked at run time, that cost the other calls 3 us of 46.)
template <bool kOwnTiles>
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const __grid_constant__ PlanArgs x) {
  extern __shared__ __align__(16) char plan_sm[];
  const SharedParams& s = x.s;
  const DecodeParams& p = x.a;
  __shared__ unsigned long long s_prefix, s_own;
  __shared__ int s_ok, s_empty, s_seg, s_base, s_warp[kPlanThreads / 32], s_longest[32];
  __shared__ float s_units[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kPlanThreads / 32;
  PrefixGroup* const groups = x.small ? reinterpret_cast<PrefixGroup*>(plan_sm) : s.groups;
  int2* const seqs = x.small ? reinterpret_cast<int2*>(plan_sm + s.n_groups * sizeof(PrefixGroup)) : s.seqs;
  int* const lens = reinterpret_cast<int*>(seqs + p.batch);   // small only
  const int64_t cap = min(static_cast<int64_t>(p.max_pages) * p.page_tokens, static_cast<int64_t>(p.max_seq_len));
  if (tid == 0) {
    s_prefix = s_own = 0;
    s_ok = 1;
    s_empty = 0;
  }
  if (kOwnTiles && tid < 32) {
    s_units[tid] = 0.f;
    s_longest[tid] = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  // ---- the lengths and the groups as they are given
  bool bad_len = false;
  for (int b = tid; b < p.batch; b += kPlanThreads) {
    const int L = p.seq_lens[b];
    bad_len |= L < 0 || L > cap;
    seqs[b] = make_int2(0, 0);
    if (x.small) lens[b] = L < 0 || L > cap ? 0 : L;
  }
  for (int g = tid; g < s.n_groups; g += kPlanThreads) {
    const int b0 = s.group_start[g], b1 = s.group_start[g + 1], n = s.shared_lens[g];
    if (b0 < 0 || b1 < b0 || b1 > p.batch || n < 0) s_ok = 0;   // no group counts then
    groups[g] = PrefixGroup{b0, b1 - b0, n, 0, 0, 0, 0, 0};
  }
  if (bad_len) raise_status(p.status, NBX_DEV_BAD_LEN);
  __syncthreads();
  auto len_of = [&](int b) -> int {
    if (x.small) return lens[b];
    const int L = p.seq_lens[b];
    return L < 0 || L > cap ? 0 : L;
  };
  if (tid == 0 && !s_ok) raise_status(p.status, NBX_DEV_BAD_ROW);
  // ---- what each group shares: what every row of every member that holds something sees
  for (int g = warp; g < s.n_groups; g += kWarps) {
    PrefixGroup pg = groups[g];
    if (!s_ok) pg.n = 0;
    int least = pg.eff, live = 0, row = p.batch;
    for (int i = lane; i < pg.n; i += 32) {
      const int L = len_of(pg.b0 + i);
      if (L > 0) {
        ++live;
        row = min(row, pg.b0 + i);
        least = min(least, L - p.rows + 1);
      }
    }
    live = __reduce_add_sync(0xffffffffu, live);
    row = __reduce_min_sync(0xffffffffu, row);
    least = __reduce_min_sync(0xffffffffu, least);
    pg.eff = live >= 2 && least >= kLeastPrefix ? least / p.page_tokens * p.page_tokens : 0;
    pg.row = row;
    const int tpu = x.tpt * x.tiles;
    pg.pairs = (pg.n * p.rows + tpu - 1) / tpu;
    if (pg.eff > 0)
      for (int i = lane; i < pg.n; i += 32)
        if (len_of(pg.b0 + i) > 0) seqs[pg.b0 + i].x = pg.eff;
    if (lane == 0) {
      groups[g] = pg;
      // (a dual unit works through two splits at a time)
      if (pg.eff > 0)
        atomicAdd(&s_prefix, static_cast<unsigned long long>(x.dual(pg) ? (pg.eff + 1) / 2 : pg.eff) * pg.pairs * x.sets);
    }
  }
  __syncthreads();
  auto sum_own = [&]() {
    unsigned long long part = 0;
    for (int b = tid; b < p.batch; b += kPlanThreads) {
      const int own = len_of(b) - seqs[b].x;
      part += kOwnTiles && x.own_dual ? (own + 1) / 2 : own;
    }
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0 && part) atomicAdd(kOwnTiles ? &s_prefix : &s_own, kOwnTiles ? part * x.own_pairs * x.sets : part);
  };
  if constexpr (kOwnTiles) {
    sum_own();
    __syncthreads();
  }
  // ---- the splits: one length for all that the tiles read, of 32 candidates the one whose rounds of units over the SMs
  // are done first. (A number of splits for each group, rounded to one round of units, left the longest at twice the mean:
  // samples of five documents of 6000 to 20000 positions 150 us where this took 126.)
  if ((kOwnTiles || warp == 0) && s_prefix > 0) {   // (few groups: one warp is done with them before several have met)
    // s_prefix: positions that all units work through one at a time. Lane i: a round would take 1 / (1 + i / 6) of them.
    // (fp32: 64-bit divisions cost a call 4 us here)
    const float round = __fdividef(static_cast<float>(s_prefix) * 6.f, static_cast<float>(x.sms * (6 + lane)));
    const int seg = max((static_cast<int>(fminf(round, 1e9f)) + 127) & ~127, 128);
    float units = 0.f;
    int longest = 0;
    for (int g = warp; g < s.n_groups; g += kOwnTiles ? kWarps : 1) {
      const PrefixGroup pg = groups[g];
      if (pg.eff == 0) continue;
      int n, len;
      x.cut(pg, seg, n, len);
      units += static_cast<float>(x.units_of(pg, n) * pg.pairs) * x.sets;
      longest = max(longest, len);
    }
    if constexpr (kOwnTiles) {
      for (int b = warp; b < p.batch; b += kWarps) {
        const int own = len_of(b) - seqs[b].x;
        if (own == 0) continue;
        int n, len;
        x.cut_own(own, 0, seg, n, len);
        units += static_cast<float>(x.own_entries(n) * x.own_pairs) * x.sets;
        longest = max(longest, n == 1 ? own : len);
      }
      atomicAdd(&s_units[lane], units);   // (whole numbers: in any order the same, but above 2^24, where it is an estimate)
      atomicMax(&s_longest[lane], longest);
      __syncthreads();
      units = s_units[lane];
      longest = s_longest[lane];
    }
    if (warp == 0) {
      // a unit's own costs: about as long as 256 positions
      const float cost = ceilf(units / x.sms) * (static_cast<float>(longest) + 256.f);
      float best = cost;
      for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
      if (lane == __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1) s_seg = seg;
    }
  }
  __syncthreads();
  for (int g = warp; g < s.n_groups; g += kWarps) {
    PrefixGroup pg = groups[g];
    if (pg.eff == 0) continue;
    x.cut(pg, s_seg, pg.splits, pg.seg);
    for (int i = lane; i < pg.n; i += 32)
      if (seqs[pg.b0 + i].x > 0) seqs[pg.b0 + i].y = pg.splits;
    __syncwarp();
    if (lane == 0) groups[g] = pg;
  }
  __syncthreads();
  // ---- each group's first work unit
  if (warp == 0) {
    int base = 0;
    for (int g0 = 0; g0 < s.n_groups; g0 += 32) {
      const int g = g0 + lane;
      PrefixGroup pg = {};
      int units = 0;
      if (g < s.n_groups) {
        pg = groups[g];
        units = x.units_of(pg, pg.splits) * pg.pairs * x.sets;
      }
      int sum = units;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (g < s.n_groups) {
        pg.unit = base + sum - units;
        s.groups[g] = pg;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) s_base = base;
  }
  // ---- the splits of the positions of each one's own
  if constexpr (!kOwnTiles) {
    sum_own();
    __syncthreads();
  }
  const int align = p.page_tokens <= NBX_SPLIT_POSITIONS ? p.page_tokens : NBX_SPLIT_POSITIONS;
  int total = 0;   // entries so far
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0, items = 0, seg = 1, L = 0;   // splits, entries
    int2 sh = make_int2(0, 0);
    if (b < p.batch) {
      L = len_of(b);
      sh = seqs[b];
      const int own = L - sh.x;
      if (own > 0 && kOwnTiles) {
        x.cut_own(own, sh.y, s_seg, n, seg);
        items = x.own_entries(n);
      } else if (own > 0) {
        // (the share of the units, rounded up)
        const float want = ceilf(static_cast<float>(p.tc_units) * own / (static_cast<float>(p.tc_pairs) * s_own));
        const int most = min(p.max_splits - sh.y, max(1, own / 64));
        const int S = want < 1.f ? 1 : (want > most ? most : static_cast<int>(want));
        seg = (own - 1) / S + 1;
        seg = (seg + align - 1) / align * align;
        items = n = (own + seg - 1) / seg;
      }
      // (what the merge needs, in one read: the splits that the tiles leave stand where other plans have the split's length)
      reinterpret_cast<int4*>(p.plan)[b] = make_int4(L, kOwnTiles ? sh.y + n : sh.y, sh.y + n, sh.x);
      if (sh.y + n == 0) s_empty = 1;
    }
    int sum = items;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int base = total + sum - items;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += s_warp[w];
      total += s_warp[w];
    }
    for (int i = 0; i < items; ++i) {
      int4* const e = reinterpret_cast<int4*>(p.entries + base + i);
      const int k = kOwnTiles && x.own_dual ? 2 * i : i, lo = sh.x + k * seg;
      e[0] = make_int4(b, sh.y + k, lo, kOwnTiles ? seg : min(L, lo + seg));
      e[1] = make_int4(L, sh.y + n, 0, 0);
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.header[0] = total;
    p.header[1] = 0;
    p.header[2] = kMergeSplits;
    p.header[3] = 0;
    p.header[4] = s_base;
    p.header[5] = s_base + (kOwnTiles ? total * x.own_pairs * x.sets : 0);
  }
  if (s_empty) {   // a sequence with no position to read: its rows are 0
    const int64_t vec4 = static_cast<int64_t>(p.rows) * p.h_q * p.d / (p.out_bf16 ? 8 : 4);
    for (int b = 0; b < p.batch; ++b) {
      if (len_of(b) != 0) continue;
      float4* o = reinterpret_cast<float4*>(p.out) + b * vec4;
      for (int64_t i = tid; i < vec4; i += kPlanThreads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// ---------------------------------------------------------------- one row
// acc = sum_j 2^(z_j - m) v_j of one query vector over positions [lo, hi) of sequence b, key by key in fp32, by one warp;
// columns [col0, col1) of it, or (kHalf) of bf16(acc inv), go to the partial `at`. m is the partial's own: at d = 256 the
// other columns, and l, belong to it. (It is finite: a row with a NaN among its scores, or with none above -inf, is not
// computed again.)
template <int D, bool kE4, bool kHalf>
__device__ __noinline__ void own_row(const DecodeParams& p, const __nv_bfloat16* q, int b, int kvh, int lo, int hi, int64_t at,
                                     float m, float inv, int col0, int col1) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
  float acc[kCols];
#pragma unroll
  for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
  // element offset of position x of the head, or -1
  auto place = [&](int x) -> int64_t {
    const int idx = x / p.page_tokens, id = __ldcg(p.block_table + static_cast<int64_t>(b) * p.max_pages + idx);
    return id < 0 || id >= p.num_pages
               ? -1 : ((static_cast<int64_t>(id) * p.h_kv + kvh) * p.page_tokens + (x - idx * p.page_tokens)) * D;
  };
  for (int n0 = lo; n0 < hi; n0 += 32) {
    float w = 0.f;
    const int64_t mine = n0 + lane < hi ? place(n0 + lane) : -1;
    if (mine >= 0) {
      const uint4* const kr = reinterpret_cast<const uint4*>(static_cast<const char*>(p.k_pool) + mine * (kE4 ? 1 : 2));
      f32x2 s = pack2(0.f, 0.f);
      constexpr int kPer = kE4 ? 2 : 1;   // queries' 16-byte pieces to one of the keys
#pragma unroll 2
      for (int i = 0; i < D / 8 / kPer; ++i) {
        f32x2 x[4 * kPer], y[4];
        unpack16x2<std::conditional_t<kE4, E4M3, BF16>>(__ldg(kr + i), x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          unpack16x2<BF16>(__ldg(reinterpret_cast<const uint4*>(q) + i * kPer + e), y);
#pragma unroll
          for (int j = 0; j < 4; ++j) s = fma2(x[4 * e + j], y[j], s);
        }
      }
      const float2 t = unpack2(s);
      const float z = (t.x + t.y) * p.qk_scale_log2;
      w = fast_exp2(z - m);
    }
    for (int j = 0; j < min(32, hi - n0); ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int64_t from = __shfl_sync(0xffffffffu, mine, j);
      if (from < 0) continue;
      const char* const vr = static_cast<const char*>(p.v_pool) + (from + lane * kCols) * (kE4 ? 1 : 2);
#pragma unroll
      for (int e = 0; e < kCols; e += 2) {
        float2 x;
        if constexpr (kE4) {
          const uint32_t codes = __ldg(reinterpret_cast<const uint16_t*>(vr + e));
          uint32_t lo, hi;
          e4m3x4_to_f16x4(codes, lo, hi);
          x = f16x2_floats(lo);
        } else {
          x = bf16x2_to_float2(__ldg(reinterpret_cast<const uint32_t*>(vr + 2 * e)));
        }
        acc[e] = fmaf(wj, x.x, acc[e]);
        acc[e + 1] = fmaf(wj, x.y, acc[e + 1]);
      }
    }
  }
  if (lane * kCols < col0 || lane * kCols >= col1) return;
#pragma unroll
  for (int e = 0; e < kCols; e += 2) {
    if constexpr (kHalf)
      reinterpret_cast<uint32_t*>(p.acc_part + at * D)[(lane * kCols + e) / 2] = bf16x2_bits(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<float2*>(p.acc_part + at * D + lane * kCols + e) = make_float2(acc[e], acc[e + 1]);
  }
}

// The last of positions [lo, hi) of sequence b whose value has an element among columns [col0, col1) that is not finite, or
// -1. A warp's work.
template <int D, bool kE4>
__device__ __noinline__ int own_not_finite(const DecodeParams& p, int b, int kvh, int lo, int hi, int col0, int col1) {
  constexpr int kElt = kE4 ? 1 : 2;
  const int chunks = (col1 - col0) * kElt / 16;
  int last = -1;
  for (int i = threadIdx.x & 31; i < (hi - lo) * chunks; i += 32) {
    const int x = lo + i / chunks, idx = x / p.page_tokens;
    const int id = __ldcg(p.block_table + static_cast<int64_t>(b) * p.max_pages + idx);
    if (id < 0 || id >= p.num_pages) continue;
    const int64_t at = ((static_cast<int64_t>(id) * p.h_kv + kvh) * p.page_tokens + (x - idx * p.page_tokens)) * D + col0;
    if (not_finite<kE4>(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.v_pool) + at * kElt) + i % chunks))) last = x;
  }
  return __reduce_max_sync(0xffffffffu, last);
}

// Computes those of a warp's rows again (may: this thread's is one that is not finite) that have a value that is not finite
// behind them: among positions [lo, end) of the sequence, of which the row sees those before `seen`. (A function, out of the
// way of the kernel's code: inside it, 36 sequences of two heads of 256 in four groups took 25.4 us, 25.1 so.)
template <int D, bool kE4, bool kHalf, int kCols>
__device__ __noinline__ void mend_own(const DecodeParams& p, int b, int kvh, int lo, int end, int seen, const __nv_bfloat16* q,
                                      int64_t at, bool may, float m, float inv, int col0, AttnControl* ctl) {
  const int past = max(lo, seen);
  const int first = __reduce_min_sync(0xffffffffu, may ? past : 0x7fffffff);
  const int last = own_not_finite<D, kE4>(p, b, kvh, first, end, col0, col0 + kCols);
  uint32_t again = __ballot_sync(0xffffffffu, may && past <= last);
  if (!again) return;
  at_busy(ctl, 1);
  while (again) {
    const int src = __ffs(again) - 1;
    again &= again - 1;
    own_row<D, kE4, kHalf>(p, reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(q), src)), b, kvh,
                           lo, min(end, __shfl_sync(0xffffffffu, seen, src)), __shfl_sync(0xffffffffu, at, src),
                           __shfl_sync(0xffffffffu, m, src), __shfl_sync(0xffffffffu, inv, src), col0, col0 + kCols);
  }
  at_busy(ctl, -1);
}

// ---------------------------------------------------------------- prefixes
// kOwn: it may have units of sequences' own positions. (E4M3 pools: without their code, a shared prefix of 65536 positions
// takes 3 us less.)
template <int D, bool kE4, int kTermsOfP, bool kOwn>
struct PrefixWork {
  using Params = PrefixParams;
  static constexpr int kN = kTermsOfP == 3 || (kE4 && D == 256) ? 64 : 128;   // keys of a tile
  static constexpr bool kF8 = kE4;
  static constexpr bool kPaged = true;
  // E4M3 codes come by bulk copies up to d = 128 (32 sequences behind 65536, pages of 64: 95.3 us by cp.async, 91.0 so; behind
  // 32768, pages of 16: 70.7 and 66.6), by cp.async at d = 256 (85.0, by bulk copies 91.1).
  static constexpr bool kBulk = kE4 && D <= 128;
  static constexpr bool kMayWaitLate = true;
  static constexpr int kTerms = kTermsOfP;
  // A bf16 output takes the partials as bf16(acc / l), in the first half of their slots: half the bytes both ways,
  // for up to 2^-8 of a split's share, less than the weights' own rounding leaves.
  static constexpr bool kHalfParts = kTermsOfP == 1;
  static constexpr bool kPairs = D <= 128;               // two M tiles a unit, or one over two ranges of keys
  // What is read before the grid ahead is waited for comes past L1 (__ldcg): the plan is complete, but an older line may
  // still lie there.
  const Params& p;
  int tpt, n_prefix, n_units;
  int step_idx, step_off;    // a key tile further on: pages and positions
  // Pieces of 16 positions, which no page splits: lane l < kN / 16 keeps track of piece l of a tile. The cursor is a tile
  // ahead, its page id on the way; loaders keep the places of the last K tile (of M tile t; at d = 256 of the last two).
  struct Cursor {
    int idx, off, id;        // page of the row, position in it, page id
  };
  Cursor cur[2];
  int64_t place[2];          // byte offset of the piece in a pool, or -1

  // (beside the one-warp kernel)
  __device__ __forceinline__ static bool wait_late(const Params& p) { return !kOwn || !p.own_tiles; }
  __device__ __forceinline__ int toks_per_tile() const { return tpt; }
  __device__ __forceinline__ int heads() const { return p.heads; }
  __device__ __forceinline__ PrefixWork(const Params& params) : p(params) {
    tpt = kAtM / p.heads;
    step_idx = kN / p.a.page_tokens;
    step_off = kN - step_idx * p.a.page_tokens;
    cur[0] = cur[1] = Cursor{0, 0, 0};
    place[0] = place[1] = -1;
  }
  __device__ __forceinline__ void begin() {
    n_prefix = __ldcg(p.a.header + 4);
    n_units = __ldcg(p.a.header + 5);
  }
  // A unit of a sequence's own positions
  __device__ __forceinline__ void own_unit(int place, AttnUnit& u) const {
    const int rows = p.a.rows, tpu = (kPairs ? 2 : 1) * tpt;
    const int pairs = (rows + tpu - 1) / tpu, per = pairs * p.sets;
    const int entry = place / per, rest = place - entry * per;
    const int set = rest / pairs, pair = rest - set * pairs;
    const int4 e = __ldcg(reinterpret_cast<const int4*>(p.a.entries + entry));   // sequence, split, begin, its positions
    const int len = __ldcg(reinterpret_cast<const int4*>(p.a.entries + entry) + 1).x;
    u.dual = kPairs && rows <= tpt;
    u.toks = min(tpu, rows - pair * tpu);
    u.tok = e.x * rows + pair * tpu;
    u.head = set * p.heads;
    u.kvh = u.head / p.a.group;
    u.pos = len - rows + pair * tpu + 1;
    u.own = 1;
    u.b = e.x;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u.slot[t] = e.y + (u.dual ? t : 0);
      u.kv[t] = e.z + (u.dual ? t * e.w : 0);
      u.end[t] = min(len, u.kv[t] + e.w);
      u.n[t] = max(0, u.end[t] - u.kv[t] + kN - 1) / kN;
    }
    if (!u.dual && !(kPairs && u.toks > tpt)) u.n[1] = 0;
  }
  __device__ __forceinline__ bool unit(uint32_t round, AttnUnit& u) const {
    const int64_t place = static_cast<int64_t>(round) * gridDim.x + blockIdx.x;
    if (place >= n_units) return false;
    const int un = static_cast<int>(place), lane = threadIdx.x & 31;
    if constexpr (kOwn) {
      if (un >= n_prefix) {
        own_unit(un - n_prefix, u);
        return true;
      }
    }
    // the last group whose first unit is not behind this one (groups without units share theirs with the next)
    PrefixGroup pg = {};
    for (int g0 = 0; g0 < p.s.n_groups; g0 += 32) {
      int4 w0 = make_int4(0, 0, 0, 0), w1 = w0;
      const bool there = g0 + lane < p.s.n_groups;
      if (there) {
        const int4* const g = reinterpret_cast<const int4*>(p.s.groups + g0 + lane);
        w0 = __ldcg(g);
        w1 = __ldcg(g + 1);
      }
      const uint32_t has = __ballot_sync(0xffffffffu, there && w1.z <= un);
      if (has == 0) break;
      const int src = 31 - __clz(has);
      pg.b0 = __shfl_sync(0xffffffffu, w0.x, src);
      pg.n = __shfl_sync(0xffffffffu, w0.y, src);
      pg.eff = __shfl_sync(0xffffffffu, w0.z, src);
      pg.seg = __shfl_sync(0xffffffffu, w0.w, src);
      pg.splits = __shfl_sync(0xffffffffu, w1.x, src);
      pg.pairs = __shfl_sync(0xffffffffu, w1.y, src);
      pg.unit = __shfl_sync(0xffffffffu, w1.z, src);
      pg.row = __shfl_sync(0xffffffffu, w1.w, src);
    }
    const int rest = un - pg.unit;
    const int pair = rest % pg.pairs, which = rest / pg.pairs;
    const int set = which % p.sets, split = which / p.sets;
    u.dual = kPairs && pg.n * p.a.rows <= tpt;
    const int tpu = (kPairs ? 2 : 1) * tpt;
    u.toks = min(tpu, pg.n * p.a.rows - pair * tpu);
    u.tok = pg.b0 * p.a.rows + pair * tpu;
    u.head = set * p.heads;
    u.kvh = u.head / p.a.group;
    u.pos = 0x7fffffff - (kPairs ? 2 : 1) * kAtM;   // (its tokens' are added to it)
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
  // (u.pos: how many positions the unit's first token sees)
  __device__ __forceinline__ int last_key(const AttnUnit& u, int t, int tok, bool) const {
    return min(u.end[t], u.pos + tok) - u.kv[t] - 1;
  }
  __device__ __forceinline__ bool in_pool(int page) const { return page >= 0 && page < p.a.num_pages; }
  __device__ __forceinline__ int page_id(const AttnUnit& u, int idx, bool there) const {
    return there ? __ldcg(p.a.block_table + static_cast<int64_t>(u.b) * p.a.max_pages + idx) : 0;
  }
  // The cursor on the piece at position `at` (there: it is one of this lane's, before the end)
  __device__ __forceinline__ void begin(Cursor& c, const AttnUnit& u, int at, bool there) const {
    c.idx = at / p.a.page_tokens;
    c.off = at - c.idx * p.a.page_tokens;
    c.id = page_id(u, c.idx, there);
  }
  __device__ __forceinline__ void advance(Cursor& c, const AttnUnit& u, bool there) const {
    c.idx += step_idx;
    c.off += step_off;
    if (c.off >= p.a.page_tokens) {
      c.off -= p.a.page_tokens;
      ++c.idx;
    }
    c.id = page_id(u, c.idx, there);
  }
  __device__ __forceinline__ uint32_t bad_keys(const AttnUnit& u, int t, int j, int c0) {
    constexpr int kPieces = (kPairs ? kN : kN / 2) / 16;
    const int lane = threadIdx.x & 31;
    const int at = u.kv[t] + j * kN + c0 + lane * 16;
    if (j == 0) begin(cur[0], u, at, lane < kPieces && at < u.end[t]);
    const int id = cur[0].id;
    advance(cur[0], u, lane < kPieces && at + kN < u.end[t]);
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
  // K tile j of M tile t is next: where its pieces lie, and the cursor a tile further on. Returns the places.
  __device__ __forceinline__ int64_t next_places(Cursor& c, const AttnUnit& u, int t, int j, bool reports) const {
    constexpr int kElt = kF8 ? 1 : 2;
    const int lane = threadIdx.x & 31;
    const int at = u.kv[t] + j * kN + lane * 16;
    const bool mine = lane < kN / 16 && at < u.end[t];
    if (j == 0) begin(c, u, at, mine);
    const bool held = in_pool(c.id);
    if (reports && mine && !held) raise_status(p.status, NBX_DEV_BAD_PAGE);
    const int64_t row = (static_cast<int64_t>(c.id) * p.a.h_kv + u.kvh) * p.a.page_tokens + c.off;
    advance(c, u, lane < kN / 16 && at + kN < u.end[t]);
    return held ? row * (D * kElt) : -1;
  }
  // This warp's part of a slot, or of a tile of codes, 16 bytes a lane: every piece is one run of bytes.
  template <class C>
  __device__ __forceinline__ void load_kv(const AttnUnit& u, bool is_v, int t, int j, int part, char* dst, uint64_t* bar,
                                          int loader) {
    constexpr int kPieces = kN / 16;
    const int lane = threadIdx.x & 31;
    int64_t at;
    if constexpr (kPairs) {   // V of a tile follows its K before the next K of the same M tile
      if (!is_v) {
        if (t == 0) place[0] = next_places(cur[0], u, t, j, loader == 0);
        else place[1] = next_places(cur[1], u, t, j, loader == 0);
      }
      at = t == 0 ? place[0] : place[1];
    } else {                  // K runs two tiles ahead of V, but for a unit's last
      if (!is_v && part == 0) {
        place[1] = place[0];
        place[0] = next_places(cur[0], u, t, j, loader == 0);
      }
      at = is_v && j + 1 < u.n[0] ? place[1] : place[0];
    }
    const char* const pool = static_cast<const char*>(is_v ? p.a.v_pool : p.a.k_pool);
    const int held = min(kPieces, (u.end[t] - u.kv[t] - j * kN + 15) >> 4);   // pieces of the tile before the end
    if constexpr (kBulk) {
      // The codes as they are stored, half a tile a warp: each run of pieces that lie together (a page, or what is left of the
      // half) is one bulk copy. What a missing page would hold is zeroed.
      constexpr int kBytes = 16 * D;
      const int first = loader * (kPieces / 2);
      const bool mine = lane >= first && lane < min(first + kPieces / 2, held);
      const bool have = mine && at >= 0;
      const int64_t before = __shfl_up_sync(0xffffffffu, at, 1);
      const bool leads = have && !(lane > first && before >= 0 && before + kBytes == at);
      const uint32_t got = __ballot_sync(0xffffffffu, have), heads = __ballot_sync(0xffffffffu, leads);
      uint32_t missing = __ballot_sync(0xffffffffu, mine && !have);
      if (missing) {
        for (; missing; missing &= missing - 1)
          for (int i = lane; i < kBytes / 16; i += 32)
            sts128(smem_u32(dst) + (__ffs(missing) - 1) * kBytes + i * 16, make_uint4(0, 0, 0, 0));
        fence_proxy_async();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(got) * kBytes);
      __syncwarp();
      if (leads) {
        const uint32_t ends = ~(got & ~heads) >> lane >> 1;   // bit 0: piece lane + 1 is not of the run
        bulk_g2s(dst + lane * kBytes, pool + at, (ends ? __ffs(ends) : 32) * kBytes, bar);
      }
      return;
    } else if constexpr (kF8) {
      const uint32_t to = smem_u32(dst) + lane * 16;
      const char* const from = pool + lane * 16;
#pragma unroll
      for (int i0 = 0; i0 < kPieces; i0 += 2) {   // two warps copy
        const int i = i0 + loader;
        const int64_t o = __shfl_sync(0xffffffffu, at, i);
        if (i >= held) break;
#pragma unroll
        for (int x = 0; x < 16 * D; x += 512) cp_async16_zfill(to + i * 16 * D + x, from + (o < 0 ? 0 : o) + x, o >= 0);
      }
    } else if constexpr (C::kParts == 2) {
      if (is_v) copy_pieces<32, kPieces / 2, kN * 64>(at, part * (kPieces / 2), held, dst, pool, loader);
      else copy_pieces<16, kPieces, kN * 128>(at, 0, held, dst, pool + part * 256, loader);
    } else {
      copy_pieces<D / 8, kPieces, kN * 128>(at, 0, held, dst, pool, loader);
    }
    cp_async_arrive_noinc(bar);
  }
  // Every fourth of kCount pieces from `first` on into a slot's swizzled atoms; kChunks 16-byte chunks of a row.
  template <int kChunks, int kCount, int kAtomBytes>
  __device__ __forceinline__ void copy_pieces(int64_t at, int first, int held, char* dst, const char* pool, int loader) const {
    constexpr int kRows = 32 / kChunks;   // rows a warp copies at a time
    const int lane = threadIdx.x & 31;
    const int lr = lane / kChunks, lc = lane % kChunks;
    const uint32_t to = smem_u32(dst) + (lc >> 3) * kAtomBytes + lr * 128 + (((lc & 7) ^ lr) << 4);
    const char* const from = pool + lr * (D * 2) + lc * 16;
#pragma unroll
    for (int i0 = 0; i0 < kCount; i0 += kAtCopyWarps) {
      const int i = i0 + loader;
      const int64_t o = __shfl_sync(0xffffffffu, at, (first + i) & 31);
      if (i >= kCount || first + i >= held) break;
      const char* const src = from + (o < 0 ? 0 : o);
      const uint32_t to_i = to + i * 2048;
      // (rows x + lr of the piece: x and lr share no bit, so the swizzle of row x + lr is that of lr, times x)
#pragma unroll
      for (int x = 0; x < 16; x += kRows) cp_async16_zfill((to_i ^ ((x & 7) << 4)) + x * 128, src + x * (D * 2), o >= 0);
    }
  }
  template <int kCols>
  __device__ __forceinline__ void store(const AttnUnit& u, int t, uint32_t o_base, int col0, int tok, int head, bool ok,
                                        float m, float l, uint64_t* o_free, AttnControl* ctl) const {
    const int lane = threadIdx.x & 31;
    const uint64_t keep = l2_keep_policy(p.a.keep_frac);
    const int64_t row = (static_cast<int64_t>(u.tok) + tok) * p.a.h_q + u.head + head;
    const int64_t at = row * p.a.max_splits + u.slot[t];
    // A NaN score leaves the running maximum alone, -inf where the row's every score here is a NaN: the merge, which skips
    // such a split, learns of it from m
    if (l != l) m = l;
    if (ok && col0 == 0) {
      st_global_hint(p.a.m_part + at, m, keep);
      st_global_hint(p.a.l_part + at, l, keep);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // (a NaN stays one)
    float sick = 0.f;   // or a NaN, if some value is not finite
    const bool parted = kOwn && u.own && p.a.rows > 1;   // own positions of several rows
    if (parted) {
#pragma unroll 1
      for (int i = 0; i < kCols; i += 32) {
        uint32_t o[32];
        tmem_ld32(o_base + i, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) sick = fmaf(__uint_as_float(o[e]), 0.f, sick);
      }
    }
#pragma unroll 1
    for (int i = 0; i < kCols; i += 32) {
      uint32_t o[32];
      tmem_ld32(o_base + i, o);
      tmem_wait_ld();
      if (i + 32 == kCols) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      if (ok && kHalfParts) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = __uint_as_float(bf16x2_bits(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv));
        float* dst = reinterpret_cast<float*>(reinterpret_cast<__nv_bfloat16*>(p.a.acc_part + at * D) + col0 + i);
        st_global_v8_hint(dst, *reinterpret_cast<const float(*)[8]>(w), keep);
        st_global_v8_hint(dst + 8, *reinterpret_cast<const float(*)[8]>(w + 8), keep);
      } else if (ok) {
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
    if constexpr (kOwn) {
      // Among the own positions, some of the keys of the later rows are not the earlier ones', but a NaN or an infinity
      // among their values reaches all rows of the product (0 x NaN): rows that are not finite, with such a value behind
      // them, are computed again. (Not those with l = 0, which the merge skips, or a NaN, which is every column's.)
      if (!parted) return;
      const bool may = ok && sick != 0.f && l > 0.f;
      if (__any_sync(0xffffffffu, may))
        mend_own<D, kE4, kHalfParts, kCols>(p.a, u.b, u.kvh, u.kv[t], u.end[t], u.pos + tok, q_row(u, tok, head), at, may, m, inv,
                                            col0, ctl);
    }
  }
};

// ---------------------------------------------------------------- merge
constexpr int kMergeWarps = 4;

// One warp per (query vector, 128 columns): M = max m_s, w_s = 2^(m_s - M) (a split with m = -inf is skipped),
// out = v_scale sum w_s acc_s / sum w_s l_s, s ascending: the prefix's splits, then the sequence's own. Sequences with one
// split from the one-warp kernel are written already. kHalves: the output is bf16, and the tiles' partials are bf16 acc / l.
// What bounds it: a chain of three reads (plan, first accumulators and statistics, the rest).
template <bool kHalves>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(DecodeParams p) {
  constexpr int N = 8;   // splits whose accumulators are loaded at once, of either kind
  const int lane = threadIdx.x & 31;
  const int d4 = p.d / 4, pieces = (d4 + 31) / 32;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.rows * p.h_q;
  pdl_wait();
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5); it < rows * pieces;
       it += static_cast<int64_t>(gridDim.x) * kMergeWarps) {
    const int64_t row = it / pieces;
    const int j = static_cast<int>(it - row * pieces) * 32 + lane;
    const int b = static_cast<int>(row / (static_cast<int64_t>(p.rows) * p.h_q));
    const int4 plan = reinterpret_cast<const int4*>(p.plan)[b];
    const int S = plan.z, pre = plan.y;
    if (S == 0 || (S == 1 && pre == 0)) continue;
    const float* m = p.m_part + row * p.max_splits;
    const float* l = p.l_part + row * p.max_splits;
    const float4* acc = reinterpret_cast<const float4*>(p.acc_part + row * p.max_splits * p.d) + (j < d4 ? j : 0);
    const uint2* half = reinterpret_cast<const uint2*>(p.acc_part + row * p.max_splits * p.d) + (j < d4 ? j : 0);
    float4 a[N];
    uint2 h[N];
    auto load_own = [&](int s0) {
#pragma unroll
      for (int k = 0; k < N; ++k) a[k] = acc[static_cast<int64_t>(min(s0 + k, S - 1)) * d4];
    };
    auto load_half = [&](int s0) {
#pragma unroll
      for (int k = 0; k < N; ++k) h[k] = half[static_cast<int64_t>(min(s0 + k, S - 1)) * (2 * d4)];
    };
    if (kHalves && pre > 0) load_half(0);
    load_own(kHalves ? pre : 0);
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
      w[k] = kHalves && e != -1.f && lane + 32 * k < pre ? e * w[k] : e;  // (bf16 partials carry no l)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float sc = p.v_scale / L;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int sp, const float4& v) {
      const float e = __shfl_sync(0xffffffffu, sp < 32 ? w[0] : w[1], sp & 31);
      if (e != -1.f) A = make_float4(fmaf(e, v.x, A.x), fmaf(e, v.y, A.y), fmaf(e, v.z, A.z), fmaf(e, v.w, A.w));
    };
    if constexpr (kHalves) {
#pragma unroll 1
      for (int s0 = 0; s0 < pre; s0 += N) {
        if (s0 > 0) load_half(s0);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (s0 + k >= pre) break;
          const float2 lo = bf16x2_to_float2(h[k].x), hi = bf16x2_to_float2(h[k].y);
          add(s0 + k, make_float4(lo.x, lo.y, hi.x, hi.y));
        }
      }
    }
#pragma unroll 1
    for (int s0 = kHalves ? pre : 0; s0 < S; s0 += N) {
      if (s0 > (kHalves ? pre : 0)) load_own(s0);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (s0 + k >= S) break;
        add(s0 + k, a[k]);
      }
    }
    if (j >= d4) continue;
    const float4 o = M == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(A.x * sc, A.y * sc, A.z * sc, A.w * sc);
    if (kHalves)
      reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * p.d)[j] =
          make_uint2(bf16x2_bits(o.x, o.y), bf16x2_bits(o.z, o.w));
    else
      reinterpret_cast<float4*>(p.out + row * p.d)[j] = o;
  }
}

// The query map of the last few shapes from this host thread, put over a call's address.
struct PrefixKey {
  int64_t tokens;
  int h_q, d, heads;
  bool operator==(const PrefixKey& o) const {
    return tokens == o.tokens && h_q == o.h_q && d == o.d && heads == o.heads;
  }
};

bool query_map(const DecodeParams& a, int heads, CUtensorMap* map) {
  constexpr int kEntries = 8;
  thread_local PrefixKey keys[kEntries];
  thread_local CUtensorMap maps[kEntries];
  thread_local int used = 0, next = 0;
  const PrefixKey key{static_cast<int64_t>(a.batch) * a.rows, a.h_q, a.d, heads};
  for (int i = 0; i < used; ++i) {
    if (!(keys[i] == key)) continue;
    *map = maps[i];
    return at_rebase(map, a.q);
  }
  const cuuint64_t d = static_cast<cuuint64_t>(a.d);
  const cuuint64_t dims[3] = {d, static_cast<cuuint64_t>(a.h_q), static_cast<cuuint64_t>(key.tokens)};
  const cuuint64_t strides[2] = {d * 2, static_cast<cuuint64_t>(a.h_q) * d * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(kAtM / heads)};
  if (!at_encode(map, 3, a.q, dims, strides, box)) return false;
  keys[next] = key;
  maps[next] = *map;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  return true;
}

template <int D, bool kE4, int kTerms, bool kOwn>
cudaError_t launch_prefix(const SharedParams& s, const DecodeParams& a, bool own_tiles, cudaStream_t stream) {
  using W = PrefixWork<D, kE4, kTerms, kOwn>;
  const DeviceInfo& di = device_info();
  const int heads = prefix_heads(a.group);
  PrefixParams p;
  if (!kE4 && !query_map(a, heads, &p.q)) return cudaErrorInvalidValue;   // (the softmax threads write an E4M3 pool's Q)
  p.s = s;
  p.a = a;
  p.status = a.status;
  p.negative = a.qk_scale_log2 < 0.f;
  p.c = std::max(std::fabs(a.qk_scale_log2), std::numeric_limits<float>::denorm_min());
  p.heads = heads;
  p.sets = a.h_q / heads;
  p.own_tiles = own_tiles;
  return launch_attn_tiles<W, D>(p, static_cast<unsigned>(di.sm_count), stream);
}
template <int D>
cudaError_t launch_prefix(const SharedParams& s, const DecodeParams& a, int pool_dtype, bool own_tiles, cudaStream_t stream) {
  if (pool_dtype == NBX_E4M3) {
    if (own_tiles)
      return a.out_bf16 ? launch_prefix<D, true, 1, true>(s, a, true, stream)
                        : launch_prefix<D, true, 2, true>(s, a, true, stream);
    return a.out_bf16 ? launch_prefix<D, true, 1, false>(s, a, false, stream)
                      : launch_prefix<D, true, 2, false>(s, a, false, stream);
  }
  return a.out_bf16 ? launch_prefix<D, false, 1, true>(s, a, own_tiles, stream)
                    : launch_prefix<D, false, 3, true>(s, a, own_tiles, stream);
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

bool prefix_path_applies(int q_dtype, int pool_dtype) {
  return q_dtype == NBX_BF16 && (pool_dtype == NBX_E4M3 || pool_dtype == NBX_BF16);
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
  x.small = plan_small(p.batch, s.n_groups);
  const bool own_tiles = p.rows * p.group >= kOwnTileVectors;
  x.own_pairs = (p.rows + x.tpt * x.tiles - 1) / (x.tpt * x.tiles);
  x.own_dual = x.tiles == 2 && p.rows <= x.tpt;
  cudaError_t e = launch_pdl(own_tiles ? shared_plan_kernel<true> : shared_plan_kernel<false>, 1u, kPlanThreads,
                             plan_smem(p.batch, s.n_groups), stream, x);
  if (e != cudaSuccess) return e;
  if (!own_tiles) {
    e = pool_dtype == NBX_E4M3 ? decode_dispatch_warp_e4m3(q, q_dtype, grid_limit, stream)
                               : decode_dispatch_warp_bf16(q, grid_limit, stream);
    if (e != cudaSuccess) return e;
  }
  e = p.d == 64    ? launch_prefix<64>(s, q, pool_dtype, own_tiles, stream)
      : p.d == 128 ? launch_prefix<128>(s, q, pool_dtype, own_tiles, stream)
                   : launch_prefix<256>(s, q, pool_dtype, own_tiles, stream);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(p.batch) * p.rows * p.h_q * ((p.d / 4 + 31) / 32);
  const int64_t grid = std::min<int64_t>((items + kMergeWarps - 1) / kMergeWarps, static_cast<int64_t>(di.sm_count) * 8);
  return p.out_bf16 ? launch_pdl(shared_merge_kernel<true>, static_cast<unsigned>(grid), kMergeWarps * 32, 0, stream, q)
                    : launch_pdl(shared_merge_kernel<false>, static_cast<unsigned>(grid), kMergeWarps * 32, 0, stream, q);
}

}  // namespace nbx
