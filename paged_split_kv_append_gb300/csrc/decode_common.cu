// The split plan kernel, the standalone merge kernel, the workspace layout and the
// decode launch sequence (plan, then the persistent partial kernel).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cuda_fp16.h>

#include "decode_kernels.cuh"

namespace nbx {

constexpr int kPlanThreads = 256;
constexpr int kSortMax = 2048;   // batches up to this size are planned in shared memory, longest split first

// Dynamic shared memory of the plan kernel: five int arrays of the batch (4 (5B + 1) bytes), none
// above kSortMax. Sized to the batch, so that the CTA leaves room on its SM for a CTA of the
// partial kernel that follows it (launched while the plan runs): a fixed 40 KB took that room from
// one tensor-core CTA, whose late start lengthened a one-wave grid by the plan's own time.
inline size_t plan_smem_bytes(int batch) {
  return batch <= kSortMax ? static_cast<size_t>(5 * batch + 1) * sizeof(int) : 0;
}
// With key ranges two arrays more, and the entries and keys of what the plan puts in order.
constexpr bool plan_orders(int batch, bool tc) { return tc && batch <= kOrderMax; }
inline size_t plan_ranges_smem_bytes(int batch, bool tc) {
  if (batch > kSortMax) return 0;
  return static_cast<size_t>((7 * batch + 4) & ~3) * sizeof(int) + (plan_orders(batch, tc) ? kOrderMax * 20 : 0);
}
constexpr int kPlanMaxSmem = 64 << 10;
static_assert((7 * kSortMax + 4) * 4 <= kPlanMaxSmem && (7 * kOrderMax + 4) * 4 + kOrderMax * 20 <= kPlanMaxSmem,
              "the plan's shared memory");

// Positions per split of the SIMT partial kernel: two of the pages' splits (NBX_SPLIT_POSITIONS).
// Each work unit of the persistent kernel pays about 2.4 us at its boundaries (the cross-warp merge
// and the partial's stores, the next unit's query staging and first stage); at 512 positions a unit
// single_row's decode call took 109.4 against 115.5 us at 256 (ragged 754.1 against 755.9 us).
constexpr int kSimtSplitPositions = 2 * NBX_SPLIT_POSITIONS;

int splits_for(int length) {
  const int l = length < 1 ? 1 : length;
  int s = (l + NBX_SPLIT_POSITIONS - 1) / NBX_SPLIT_POSITIONS;
  return s < 1 ? 1 : (s > NBX_MAX_SPLITS ? NBX_MAX_SPLITS : s);
}

bool workspace_layout(int batch, int rows, int h_q, int h_kv, int d, int max_seq_len, WorkspaceLayout* w,
                      bool modified) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  // 64-position splits of the modified decodes: a quarter of the pages' 256
  const size_t S = static_cast<size_t>(splits_for(modified && max_seq_len < (1 << 28) ? 4 * max_seq_len : max_seq_len));
  const size_t rb = (static_cast<size_t>(rows) * (h_q / h_kv) + kQB - 1) / kQB;
  const size_t prow = static_cast<size_t>(batch) * rows * h_q * S;   // partial rows
  if (prow > (static_cast<size_t>(1) << 40) / static_cast<size_t>(d)) return false;
  size_t off = 0;
  w->header = off;
  off += up(64 * 4);
  w->ident_bt = off;
  off += up(static_cast<size_t>(batch) * 4);
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
  w->ranges = off;
  const size_t m_tiles = (static_cast<size_t>(rows) * (h_q / h_kv) + kMmaRowsPerTile - 1) / kMmaRowsPerTile;
  if (modified) off += up(static_cast<size_t>(batch) * m_tiles * sizeof(int2));
  w->order = off;
  if (modified) off += up(kOrderMax * 4);
  w->total = off;
  w->max_splits = static_cast<int>(S);
  w->row_blocks = static_cast<int>(rb);
  return true;
}

// The plan kernel may run while the kernel before it (a decode step's append, which reads the
// lengths; another decode's partial, where no merge follows it) still runs. Until it has waited for that
// grid it only reads the lengths and works in shared memory: the workspace, the output and the advanced
// lengths may all be memory that the grid ahead still uses. It has waited before it completes, so the kernels
// after it see the append's positions.
__device__ __forceinline__ void plan_finish(const DecodeParams& p) {
  pdl_wait();
  if (p.lens_out)   // the step's length advance; nothing later reads seq_lens
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) p.lens_out[b] = p.seq_lens[b] + p.len_add;
}

// Reads the device lengths, cuts every sequence into splits, then (past the wait) writes every
// sequence's plan (len, positions per split, non-empty splits), zeroes the work counter, writes 0 to
// the output rows of empty sequences, and writes the work list of (sequence, split) entries: every
// sequence's last split first, then the other splits, sequences with the longest splits first (stable),
// splits ascending. Batches above kSortMax keep their own order and take a slower serial path.
// TC: a tensor-core window, whose splits are sized by the call's total work (DecodeParams::tc_units);
// otherwise splits of kSimtSplitPositions. Two instantiations keep each rule's code free of the other.
// (TC is also the rule of a modified decode's one-warp kernel.)
// X: a modified decode. With key ranges a sequence's splits cut only the positions from the first key that
// some row sees (down to a split boundary's alignment) to the last one, and a tensor-core window gets the
// range of every M tile; the ranges come from the caller's kernels, so that plan waits before it reads.
template <bool TC, bool X>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(DecodeParams p) {
  extern __shared__ int plan_sm[];   // plan_smem_bytes(batch)
  int* const s_len = plan_sm;
  int* const s_seg = s_len + p.batch;
  int* const s_n = s_seg + p.batch;
  int* const s_order = s_n + p.batch;
  int* const s_base = s_order + p.batch;   // [batch + 1]
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_empty;
  __shared__ int s_bad;   // a length out of bounds
  __shared__ int s_nb;
  const int tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int B = p.batch;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_tokens;
  const bool small = B <= kSortMax;
  const bool waited = X || !small;
  if (waited) pdl_wait();
  pdl_launch_dependents();   // the partial kernel may start its prologue now; it waits for this grid
  const bool ranges = X && (p.key_begin != nullptr || p.key_end != nullptr);
  // splits start on whole pages, or on 256-position boundaries when a page is longer (a
  // contiguous cache read as one page per sequence): tile starts either way
  const int align = p.page_tokens <= NBX_SPLIT_POSITIONS ? p.page_tokens : NBX_SPLIT_POSITIONS;
  __shared__ long long s_total;
  __shared__ int s_multi;
  // with key ranges: the first and one past the last key that a sequence's rows see; then, where the work is put in
  // order, its entries' {b, start, end} and the pairs' keys
  int* const s_lo = s_base + B + 1;
  int* const s_hi = s_lo + B;
  int4* const s_entry = reinterpret_cast<int4*>(plan_sm + ((7 * B + 4) & ~3));
  if (tid == 0) {
    s_empty = 0;
    s_bad = 0;
    s_nb = 0;
    if constexpr (TC) s_total = 0;
    if (waited) p.header[1] = 0;
    if constexpr (X) {
      p.header[3] = 0;
      s_multi = B > kSortMax;
    }
  }
  __syncthreads();
  if constexpr (X) {
    if (ranges) {
      // the keys that the rows of a (sequence, M tile), or of a sequence, see between them: `width` lanes to each (a
      // whole warp for a single row made 1024 rows 115 us)
      if (small) {
        for (int b = tid; b < B; b += kPlanThreads) {
          s_lo[b] = INT_MAX;
          s_hi[b] = 0;
        }
        __syncthreads();
      }
      const int most = p.range_tiles == 1 ? p.rows : kMmaRowsPerTile / p.group + 2;   // rows of a tile
      int width = 1;
      while (width < most && width < 32) width <<= 1;
      const int per_warp = 32 / width;
      const int64_t items = static_cast<int64_t>(B) * p.range_tiles;
      for (int64_t i0 = warp * per_warp; i0 < items; i0 += kPlanThreads / 32 * per_warp) {
        const int64_t it = i0 + lane / width;
        const int b = it < items ? static_cast<int>(it / p.range_tiles) : 0;
        const int mt = static_cast<int>(it - static_cast<int64_t>(b) * p.range_tiles);
        const int L = p.seq_lens[b];
        const bool fit = it < items && L >= 0 && L <= p.max_seq_len && static_cast<int64_t>(L) <= cap;
        const int r0 = mt * kMmaRowsPerTile / p.group;
        const int r1 = p.range_tiles == 1 ? p.rows : min(p.rows, ((mt + 1) * kMmaRowsPerTile + p.group - 1) / p.group);
        int lo = INT_MAX, hi = 0;
        if (fit) {
          for (int r = r0 + (lane & (width - 1)); r < r1; r += width) {
            const KeyRange kr = key_range(p, b, r, L);
            if (kr.hi > kr.lo) {
              lo = min(lo, kr.lo);
              hi = max(hi, kr.hi);
            }
          }
        }
        for (int o = width >> 1; o > 0; o >>= 1) {
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (it < items && (lane & (width - 1)) == 0) {
          p.ranges[it] = hi > lo ? make_int2(lo, hi) : make_int2(0, 0);
          if (small && hi > lo) {
            atomicMin(&s_lo[b], lo);
            atomicMax(&s_hi[b], hi);
          }
        }
      }
      __syncthreads();   // orders the ranges' writes before this CTA's reads
    }
  }
  // the positions of sequence b that are read: its length, or its rows' range from an aligned start
  auto reach = [&](int b, int L) -> int2 {
    if (!ranges) return make_int2(0, L);
    int lo = INT_MAX, hi = 0;
    if (small) {
      lo = s_lo[b];
      hi = s_hi[b];
    } else {
      for (int mt = 0; mt < p.range_tiles; ++mt) {
        const int2 r = p.ranges[static_cast<int64_t>(b) * p.range_tiles + mt];
        if (r.y > r.x) {
          lo = min(lo, r.x);
          hi = max(hi, r.y);
        }
      }
    }
    return hi > 0 ? make_int2(lo / align * align, min(hi, L)) : make_int2(0, 0);
  };
  // a tensor-core window sizes its splits by the whole call's work: the sum of the lengths
  long long len_sum = 0;
  if constexpr (TC) {
    long long part = 0;
    for (int b = tid; b < B; b += kPlanThreads) {
      const int L = p.seq_lens[b] + p.len_add;
      if (L > 0 && L <= p.max_seq_len && static_cast<int64_t>(L) <= cap) {
        if constexpr (X) {
          const int2 w = reach(b, L);
          part += w.y - w.x;
        } else {
          part += L;
        }
      }
    }
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0 && part) atomicAdd(reinterpret_cast<unsigned long long*>(&s_total), static_cast<unsigned long long>(part));
    __syncthreads();
    len_sum = s_total;
  }
  for (int b = tid; b < B; b += kPlanThreads) {
    int L = p.seq_lens[b] + p.len_add;   // a decode step attends to its own new positions
    if (L < 0 || L > p.max_seq_len || static_cast<int64_t>(L) > cap) {
      s_bad = 1;
      L = 0;
    }
    const int len = L;
    int first = 0;   // X: L becomes the positions read, from `first` on
    if constexpr (X) {
      const int2 w = reach(b, L);
      first = w.x;
      L = w.y - w.x;
    }
    int S;
    if (TC && len_sum > 0) {
      // about tc_units units in all, shared in proportion to the lengths (the grid's one wave); a
      // split keeps at least 64 positions (the tensor-core tile), and a sequence has at most the
      // workspace's partial slots (max_splits, the pages' rule at the longest length)
      long long aim = p.tc_units;
      if constexpr (X) {
        // A pair of a sequence has few units then, and one split more for each may be a second round for some warps:
        // three rounds, if the units stay long enough (32 sequences of 2048 positions with 32 KV heads, 2 splits or 5:
        // 204 and 159 us; 64 ragged ones of up to 2048 with 8, where they would not: 56 and 58).
        if (p.tc_round_up && 5ll * p.tc_pairs * B >= p.tc_warps && len_sum * p.tc_pairs >= 448ll * p.tc_warps)
          aim += 2ll * p.tc_warps;
      }
      long long num = aim * L;
      const long long den = static_cast<long long>(p.tc_pairs) * len_sum;
      // units taken from a counter may pass one wave by a few, but must not be long: their splits round up
      if (X && p.tc_round_up) num += den - 1;
      const long long want = num / den;
      // (a window has no more splits than the pages' rule gives: 16 sequences of 200 positions under 64 rows took
      // 23.4 us a call cut in two, 20.7 whole)
      int cap_s = min(p.max_splits, max(1, L / 64));
      if (X && !p.tc_round_up) cap_s = min(cap_s, (L - 1) / NBX_SPLIT_POSITIONS + 1);
      S = static_cast<int>(want < 1 ? 1 : (want > cap_s ? cap_s : want));
    } else {
      // two of the pages' 256-position splits a split: half the unit boundaries, at most 64 splits
      S = (max(L, 1) + kSimtSplitPositions - 1) / kSimtSplitPositions;
      S = S > NBX_MAX_SPLITS ? NBX_MAX_SPLITS : S;
    }
    int seg = (L + S - 1) / S;
    seg = ((seg + align - 1) / align) * align;
    const int n = L > 0 ? (L + seg - 1) / seg : 0;
    // kept in L2 for the merge, which reads the split counts after the K/V stream
    if (waited) {
      if (p.ident_bt) p.ident_bt[b] = b;
      st_global_hint(reinterpret_cast<int4*>(p.plan + b), make_int4(X ? len : L, seg, n, first), l2_evict_last_policy());
    }
    if constexpr (X) {
      if (n > 1) s_multi = 1;
    }
    if (n == 0) s_empty = 1;
    else if (small) atomicAdd(&s_nb, 1);
    if (small) {
      s_len[b] = X ? first + L : L;
      s_seg[b] = seg;
      s_n[b] = n;
    }
  }
  __syncthreads();
  if constexpr (X) {
    if (tid == 0) p.header[2] = s_multi ? kMergeSplits : 0;
  }
  // a sequence with no position to read gets no work unit: its rows are written here (0)
  auto zero_empty_rows = [&]() {
    if (!s_empty) return;
    // 16-byte pieces of a sequence's output (d is a multiple of 64)
    const int64_t row_vec4 = static_cast<int64_t>(p.rows) * p.h_q * p.d / (X && p.out_bf16 ? 8 : 4);
    for (int b = 0; b < B; ++b) {
      if ((small ? s_n[b] : p.plan[b].n_splits) != 0) continue;
      float4* o = reinterpret_cast<float4*>(p.out) + b * row_vec4;
      for (int64_t x = tid; x < row_vec4; x += kPlanThreads) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  if (!small) {
    // large batch: batch order, one thread writes the whole list
    zero_empty_rows();
    if (tid == 0) {
      if (s_bad) raise_status(p.status, NBX_DEV_BAD_LEN);
      int base = 0;
      for (int b = 0; b < B; ++b) {
        const SeqPlan sp = p.plan[b];
        for (int s = 0; s < sp.n_splits; ++s) {
          Entry e;
          e.b = b;
          e.s = s;
          e.start = sp.first + s * sp.seg;
          e.end = min(sp.first + (s + 1) * sp.seg, X ? reach(b, sp.len).y : sp.len);
          e.len = sp.len;
          e.n_splits = sp.n_splits;
          e.pad0 = e.pad1 = 0;
          p.entries[base + s] = e;
        }
        base += sp.n_splits;
      }
      p.header[0] = base;
    }
    plan_finish(p);
    return;
  }
  // stable rank by split length, longest first (empty sequences last). The list then holds every
  // sequence's last split first (in that order), then the other splits: the last splits are of
  // uneven length, so the persistent grid's first wave of units ends at scattered times instead of
  // every CTA reaching a unit boundary at once; the rest follow longest first.
  for (int b = tid; b < B; b += kPlanThreads) {
    const int k = s_n[b] > 0 ? s_seg[b] : -1;
    int rank = 0;
    for (int c = 0; c < B; ++c) {
      const int kc = s_n[c] > 0 ? s_seg[c] : -1;
      rank += (kc > k) || (kc == k && c < b);
    }
    s_order[rank] = b;
  }
  __syncthreads();
  // exclusive scan of the split counts in list order (a contiguous run per thread, then a block scan)
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(B, tid * per), hi = min(B, lo + per);
  int run = 0;
  for (int i = lo; i < hi; ++i) run += max(s_n[s_order[i]] - 1, 0);
  int x = run;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < kPlanThreads / 32) s_warp[lane] = w;
  }
  __syncthreads();
  int base = x - run + (warp > 0 ? s_warp[warp - 1] : 0);
  for (int i = lo; i < hi; ++i) {
    s_base[i] = base;
    base += max(s_n[s_order[i]] - 1, 0);
  }
  if (tid == kPlanThreads - 1) s_base[B] = x + (warp > 0 ? s_warp[warp - 1] : 0);
  __syncthreads();
  // ---- the wait (a modified decode's plan has waited already), then the global writes
  pdl_wait();
  if (!waited) {
    for (int b = tid; b < B; b += kPlanThreads) {
      if (p.ident_bt) p.ident_bt[b] = b;
      st_global_hint(reinterpret_cast<int4*>(p.plan + b), make_int4(s_len[b], s_seg[b], s_n[b], 0), l2_evict_last_policy());
    }
    if (tid == 0) p.header[1] = 0;
  }
  if (tid == 0 && s_bad) raise_status(p.status, NBX_DEV_BAD_LEN);
  zero_empty_rows();
  // the entries, in parallel: entry e belongs to the list position i with s_base[i] <= e < s_base[i+1]
  const int nb = s_nb;
  const int total = s_base[B] + nb;
  for (int e = tid; e < total; e += kPlanThreads) {
    int b, s;
    if (e < nb) {
      b = s_order[e];
      s = s_n[b] - 1;
    } else {
      const int e2 = e - nb;
      int l = 0, r = B - 1;
      while (l < r) {
        const int m = (l + r + 1) >> 1;
        if (s_base[m] <= e2) l = m; else r = m - 1;
      }
      b = s_order[l];
      s = e2 - s_base[l];
    }
    Entry en;
    en.b = b;
    en.s = s;
    if constexpr (X) {   // the list of splits starts at the first position read and ends at the last
      const SeqPlan sp = p.plan[b];
      en.start = sp.first + s * s_seg[b];
      en.end = min(sp.first + (s + 1) * s_seg[b], s_len[b]);
      en.len = sp.len;
    } else {
      en.start = s * s_seg[b];
      en.end = min((s + 1) * s_seg[b], s_len[b]);
      en.len = s_len[b];
    }
    en.n_splits = s_n[b];
    en.pad0 = en.pad1 = 0;
    p.entries[e] = en;
    if constexpr (X && TC) {
      if (ranges && e < kOrderMax && plan_orders(B, TC)) s_entry[e] = make_int4(en.b, en.start, en.end, 0);
    }
  }
  if (tid == 0) p.header[0] = total;
  // A window whose rows see their own keys: its M tiles differ in length, and a CTA takes one or two units of
  // them. Most keys first, dealt to the CTAs there and back, the longest CTA of 512 rows of documents of up to
  // 1500 positions (256 units) reads 31 tiles where it read 39.
  if constexpr (TC && X) {
    int4* const s_cost = s_entry + kOrderMax;
    int* const cost = reinterpret_cast<int*>(s_cost);
    const int64_t all = static_cast<int64_t>(total) * p.range_tiles;
    if (ranges && plan_orders(B, TC) && !p.tc_round_up && all <= kOrderMax && all * p.h_kv > p.tc_units) {
      const int items = static_cast<int>(all);
      __syncthreads();
      for (int i = tid; i < (items + 3) / 4 * 4; i += kPlanThreads) {
        int c = -1;
        if (i < items) {
          const int4 en = s_entry[i / p.range_tiles];
          const int2 r = p.ranges[en.x * p.range_tiles + i % p.range_tiles];
          c = max(0, min(en.z, r.y) - max(en.y, r.x));
        }
        cost[i] = c;
      }
      __syncthreads();
      for (int x = tid; x < items; x += kPlanThreads) {
        const int c = cost[x];
        int rank = 0;
        for (int i = 0; i < items; i += 4) {   // stable: ties keep their order
          const int4 o = s_cost[i / 4];
          rank += (o.x > c || (o.x == c && i < x)) + (o.y > c || (o.y == c && i + 1 < x)) +
                  (o.z > c || (o.z == c && i + 2 < x)) + (o.w > c || (o.w == c && i + 3 < x));
        }
        p.order[rank] = x;
      }
      if (tid == 0) p.header[3] = items;
    }
  }
  plan_finish(p);
}

// ------------------------------------------------------------------------------------ standalone merge
constexpr int kMergeThreads = 128;

// One CTA per row: M = max_s m_s, weights e^(m_s - M) (splits with m = -inf are skipped),
// L = sum_s l_s w_s, out = sum_s w_s acc_s / L, s ascending.
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(MergeParams p) {
  extern __shared__ float msm[];
  float* w = msm;
  int* live = reinterpret_cast<int*>(msm + p.splits);
  __shared__ float s_inv;
  __shared__ int s_dead;
  const int64_t row = blockIdx.x;
  const float* m = p.m_part + row * p.splits;
  const float* l = p.l_part + row * p.splits;
  if (threadIdx.x == 0) {
    float M = -INFINITY;
    for (int s = 0; s < p.splits; ++s) M = max_nan(M, m[s]);
    float L = 0.f;
    for (int s = 0; s < p.splits; ++s) {
      const float ms = m[s];
      const int lv = ms != -INFINITY;
      const float ws = lv ? fast_exp2((ms - M) * kLog2e) : 0.f;
      if (lv) L += ws * l[s];
      w[s] = ws;
      live[s] = lv;
    }
    s_dead = (M == -INFINITY);
    s_inv = 1.f / L;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.d; d += kMergeThreads) {
    float A = 0.f;
    for (int s = 0; s < p.splits; ++s)
      if (live[s]) A += w[s] * p.acc_part[(row * p.splits + s) * p.d + d];
    p.out[row * p.d + d] = s_dead ? 0.f : A * s_inv;
  }
}

cudaError_t merge_dispatch(const MergeParams& p, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.splits) * 8;
  merge_kernel<<<static_cast<unsigned>(p.n_rows), kMergeThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------------------ decode merge
constexpr int kDecodeMergeThreads = 32;   // one warp per CTA

// One query vector's partial over keys [start, end) of a bf16-query window, key by key: m, l (the same in
// every lane) and this lane's float4 j of acc (zeros past d). Only rows that a tensor-core window marked
// come here: a value row holds a NaN or an infinity, or O overflowed.
struct RowPartial {
  float m, l;
  float4 acc;
};
__device__ __noinline__ RowPartial recompute_partial(const DecodeParams& p, int b, int h, int r, int g, int start, int end,
                                                     int len, int j) {
  const int lane = threadIdx.x & 31;
  const int64_t orow = (static_cast<int64_t>(b) * p.rows + r) * p.h_q + static_cast<int64_t>(h) * p.group + g;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + orow * p.d;
  const KeyRange kr = key_range(p, b, r, len);
  const float slope = p.slopes ? p.slopes[h * p.group + g] * kLog2e : 0.f;
  const int at = len - p.rows + r;
  RowPartial o = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int n = max(start, kr.lo); n < min(end, kr.hi); ++n) {
    const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + n / p.page_tokens];
    if (page < 0 || page >= p.num_pages) continue;
    const int in_page = n % p.page_tokens;
    const int64_t head = static_cast<int64_t>(page) * p.h_kv + h;
    float ks = 1.f, vs = 1.f;
    if (p.k_scales) {
      const int64_t blk = head * (p.page_tokens >> p.scale_shift) + (in_page >> p.scale_shift);
      ks = p.k_scales[blk];
      vs = p.v_scales[blk];
      if (!(ks >= kMinScale && ks <= kMaxScale && vs >= kMinScale && vs <= kMaxScale)) continue;
    }
    const int64_t row = (head * p.page_tokens + in_page) * p.d;
    float s = 0.f;
    for (int e = 2 * lane; e < p.d; e += 64) {
      const float2 qq = load_pair<BF16>(q + e);
      const float2 kk = p.pool_e4m3 ? load_pair<E4M3>(static_cast<const char*>(p.k_pool) + row + e)
                                    : load_pair<BF16>(static_cast<const char*>(p.k_pool) + (row + e) * 2);
      s = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, s));
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    float z = s * p.qk_scale_log2 * ks;
    if (p.cap_log2 > 0.f) z = p.cap_log2 * tanhf(z * p.cap_inv);
    z = fmaf(-slope, static_cast<float>(abs(at - n)), z);
    const float m = max_nan(o.m, z);
    if (m == -INFINITY) continue;
    const float f = fast_exp2(o.m - m), w = fast_exp2(z - m);
    const float wv = w * vs;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < p.d / 4) {
      float2 lo, hi;
      if (p.pool_e4m3) {
        lo = load_pair<E4M3>(static_cast<const char*>(p.v_pool) + row + 4 * j);
        hi = load_pair<E4M3>(static_cast<const char*>(p.v_pool) + row + 4 * j + 2);
      } else {
        lo = load_pair<BF16>(static_cast<const char*>(p.v_pool) + (row + 4 * j) * 2);
        hi = load_pair<BF16>(static_cast<const char*>(p.v_pool) + (row + 4 * j + 2) * 2);
      }
      v = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    o.acc = make_float4(fmaf(o.acc.x, f, wv * v.x), fmaf(o.acc.y, f, wv * v.y), fmaf(o.acc.z, f, wv * v.z),
                        fmaf(o.acc.w, f, wv * v.w));
    o.l = fmaf(o.l, f, w);
    o.m = m;
  }
  return o;
}

// Four output values (columns 4 j .. 4 j + 3 of row orow); a modified decode's output may be bf16.
template <bool X>
__device__ __forceinline__ void store_out4(const DecodeParams& p, int64_t orow, int j, float4 o) {
  if (X && p.out_bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * p.d)[j] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    reinterpret_cast<float4*>(p.out + orow * p.d)[j] = o;
  }
}

// Merges the split partials of every query vector of a (sequence, KV head) with more than one
// split: M = max_s m_s, w_s = 2^(m_s - M) (m in log2 units; splits with m = -inf skipped),
// out = v_scale * sum_s w_s acc_s / sum_s w_s l_s, s ascending. One-split sequences were written
// by the partial kernel.
// One warp per query vector and 128 output columns, each its own CTA so the work spreads evenly
// over the SMs: lane k holds m and l of splits k and k + 32 (max and sums are butterfly
// reductions, a fixed order), the weights reach every lane by shuffles, and each lane owns one
// float4 of the output, with every split's accumulator load in flight and the sum in ascending
// split order.
// N: the splits whose accumulators are loaded at once.
// F16: the partials are f16 acc / l (DecodeParams::part_f16); a split then weighs 2^(m - M) * l.
// X: a modified decode, whose output may be bf16, and whose windows on tensor cores mark partials to be
// recomputed (header[2] says that there are any): such rows take the slow path above, splits ascending too.
template <bool F16, bool X, int N>
__global__ void __launch_bounds__(kDecodeMergeThreads) decode_merge_kernel(DecodeParams p) {
  const int lane = threadIdx.x;
  const int RG = p.rows * p.group;
  const int per_seq = p.h_kv * p.row_blocks;
  const int d4 = p.d / 4;
  const int n_col = (d4 + 31) / 32;   // 128-column pieces of a vector
  const int64_t n_items = static_cast<int64_t>(p.batch) * per_seq * kQB * n_col;
  // The plan kernel had completed before any CTA of the partial kernel passed its own wait, and this
  // grid is launched only after they did, so the first item's split count can be read (from L2)
  // before this grid waits for the partials.
  int s_first = 0;
  if (blockIdx.x < n_items)
    s_first = __ldcg(&p.plan[blockIdx.x / (static_cast<int64_t>(per_seq) * kQB * n_col)].n_splits);
  pdl_wait();   // every partial of the decode is written and visible from here on
  const int todo = X ? p.header[2] : kMergeSplits;
  if (X && todo == 0) return;   // the partial kernel wrote every row
  const bool redo_any = X && (todo & kMergeRedo) != 0;
  for (int64_t it = blockIdx.x; it < n_items; it += gridDim.x) {
    const int64_t vi = it / n_col;
    const int j = static_cast<int>(it - vi * n_col) * 32 + lane;   // this lane's float4 column
    const int64_t gi = vi / kQB;
    const int i = static_cast<int>(vi - gi * kQB);
    const int b = static_cast<int>(gi / per_seq);
    const int rem = static_cast<int>(gi - static_cast<int64_t>(b) * per_seq);
    const int h = rem / p.row_blocks;
    const int rb = rem - h * p.row_blocks;
    const int qi = rb * kQB + i;
    if (qi >= RG) continue;
    const int S = it == blockIdx.x ? s_first : p.plan[b].n_splits;
    if (S <= 1 && !redo_any) continue;
    const int r = qi / p.group;
    const int g = qi - r * p.group;
    const int64_t orow = (static_cast<int64_t>(b) * p.rows + r) * p.h_q + static_cast<int64_t>(h) * p.group + g;
    const float* m = p.m_part + orow * p.max_splits;
    const float* l = p.l_part + orow * p.max_splits;
    if (X && redo_any) {
      bool redo = false;
      for (int sp = lane; sp < S; sp += 32) redo = redo || __float_as_uint(m[sp]) == kRedoBits;
      if (__any_sync(0xffffffffu, redo)) {
        const SeqPlan plan = p.plan[b];
        RowPartial t = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int sp = 0; sp < S; ++sp) {
          RowPartial o;
          if (__float_as_uint(m[sp]) == kRedoBits) {
            const int start = plan.first + sp * plan.seg;
            o = recompute_partial(p, b, h, r, g, start, start + plan.seg, plan.len, j);
          } else {
            o.m = m[sp];
            o.l = l[sp];
            o.acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const float* a = p.acc_part + (orow * p.max_splits + sp) * p.d;
            if (j < d4) {
              if constexpr (F16) {
                const uint2 hv = reinterpret_cast<const uint2*>(a)[j];
                const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&hv.x));
                const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&hv.y));
                o.acc = make_float4(lo.x * o.l, lo.y * o.l, hi.x * o.l, hi.y * o.l);
              } else {
                o.acc = reinterpret_cast<const float4*>(a)[j];
              }
            }
          }
          if (o.m == -INFINITY) continue;
          const float M2 = max_nan(t.m, o.m);
          const float f = fast_exp2(t.m - M2), w = fast_exp2(o.m - M2);
          t.acc = make_float4(fmaf(t.acc.x, f, w * o.acc.x), fmaf(t.acc.y, f, w * o.acc.y),
                              fmaf(t.acc.z, f, w * o.acc.z), fmaf(t.acc.w, f, w * o.acc.w));
          t.l = fmaf(t.l, f, w * o.l);
          t.m = M2;
        }
        const float tc = t.m == -INFINITY ? 0.f : p.v_scale / t.l;
        if (j < d4) store_out4<X>(p, orow, j, make_float4(t.acc.x * tc, t.acc.y * tc, t.acc.z * tc, t.acc.w * tc));
        continue;
      }
      if (S <= 1) continue;
    }
    const float4* acc = reinterpret_cast<const float4*>(p.acc_part + orow * p.max_splits * p.d);
    // f16 partials: the d halves at the start of each split's d-float slot, 4 per lane (8 bytes)
    const uint2* acc_h = reinterpret_cast<const uint2*>(p.acc_part + orow * p.max_splits * p.d);
    auto load_batch = [&](int j, int s0, float4 (&a)[N]) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const bool in = j < d4 && s0 + k < S;
        if constexpr (F16) {
          const uint2 hv = in ? acc_h[static_cast<int64_t>(s0 + k) * (2 * d4) + j] : make_uint2(0u, 0u);
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&hv.x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&hv.y));
          a[k] = make_float4(lo.x, lo.y, hi.x, hi.y);
        } else {
          a[k] = in ? acc[static_cast<int64_t>(s0 + k) * d4 + j] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    };
    float4 a[N];
    load_batch(j, 0, a);   // in flight together with the m / l loads
    float mv[2], lv[2];
    bool live[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int sp = lane + 32 * k;
      mv[k] = sp < S ? m[sp] : -INFINITY;
      lv[k] = sp < S ? l[sp] : 0.f;
      live[k] = mv[k] != -INFINITY;
    }
    float M = max_nan(mv[0], mv[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float wv[2];   // weight of split lane + 32k, -1 for a split with no visible key
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float w = live[k] ? fast_exp2(mv[k] - M) : 0.f;
      if (live[k]) L += w * lv[k];
      // an f16 partial is acc / l: its weight carries l
      wv[k] = live[k] ? (F16 ? w * lv[k] : w) : -1.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const bool dead = M == -INFINITY;
    const float sc = p.v_scale / L;
    // every lane runs every step (the shuffles need the whole warp); lanes past the row store nothing
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += N) {
      if (s0 > 0) load_batch(j, s0, a);
      const float wsrc = s0 < 32 ? wv[0] : wv[1];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (s0 + k >= S) break;
        const float w = __shfl_sync(0xffffffffu, wsrc, (s0 + k) & 31);
        if (w != -1.f) {
          A.x += w * a[k].x;
          A.y += w * a[k].y;
          A.z += w * a[k].z;
          A.w += w * a[k].w;
        }
      }
    }
    if (j < d4)
      store_out4<X>(p, orow, j,
                    dead ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(A.x * sc, A.y * sc, A.z * sc, A.w * sc));
  }
}

// ------------------------------------------------------------------------------------ score bounds
constexpr int kBoundsThreads = 256;
constexpr int kBoundsChunk = 512;   // positions per CTA

// Score bounds for the fixed-shift softmax (maxdiffusion PR #477: the metadata computed before the
// kernel, here per query vector and per (sequence, KV head)): |q| of every query vector, and
// max_j |k_j| * k_scale and max_{j,d} |v_jd| * v_scale over the positions a sequence holds, read
// through the block table. A NaN input gives a NaN bound, which no gate passes; a length out of
// bounds is read as empty (NBX_DEV_BAD_LEN) and a page id outside the pool is skipped
// (NBX_DEV_BAD_PAGE). One CTA per (sequence, KV head, chunk of 512 positions), a warp per position;
// the chunks combine with an atomic max on the bit patterns (the bounds are >= 0, and a NaN's bits
// order above every finite value's), so kv_max must hold zeros first. The chunk-0 CTAs of KV head 0
// write the sequence's query norms.
template <class PT, class QT>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(DecodeParams p, float* q_norm, float* kv_max,
                                                                 int n_chunks) {
  __shared__ float s_k[kBoundsThreads / 32], s_v[kBoundsThreads / 32];
  const int chunk = static_cast<int>(blockIdx.x % static_cast<unsigned>(n_chunks));
  const int bh = static_cast<int>(blockIdx.x / static_cast<unsigned>(n_chunks));   // b * h_kv + h
  const int b = bh / p.h_kv;
  const int h = bh - b * p.h_kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kBoundsThreads / 32;
  int L = p.seq_lens[b];
  if (L < 0 || L > p.max_seq_len || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_pages) * p.page_tokens) {
    if (h == 0 && chunk == 0 && threadIdx.x == 0) raise_status(p.status, NBX_DEV_BAD_LEN);
    L = 0;
  }
  const int j0 = chunk * kBoundsChunk, j1 = min(L, j0 + kBoundsChunk);
  float k2 = 0.f, va = 0.f;   // max |k|^2 and max |v| (pool units) over this warp's positions
  for (int j = j0 + warp; j < j1; j += kWarps) {
    const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_tokens];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) raise_status(p.status, NBX_DEV_BAD_PAGE);
      continue;
    }
    const int64_t row = ((static_cast<int64_t>(page) * p.h_kv + h) * p.page_tokens + j % p.page_tokens) * p.d;
    const char* kr = static_cast<const char*>(p.k_pool) + row * PT::kBytes;
    const char* vr = static_cast<const char*>(p.v_pool) + row * PT::kBytes;
    float ks = 0.f, vm = 0.f;
    for (int e = 2 * lane; e < p.d; e += 64) {
      const float2 kk = load_pair<PT>(kr + e * PT::kBytes);
      const float2 vv = load_pair<PT>(vr + e * PT::kBytes);
      ks = fmaf(kk.x, kk.x, fmaf(kk.y, kk.y, ks));
      vm = max_nan(vm, max_nan(fabsf(vv.x), fabsf(vv.y)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ks += __shfl_xor_sync(0xffffffffu, ks, o);
      vm = max_nan(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
    k2 = max_nan(k2, ks);
    va = max_nan(va, vm);
  }
  if (lane == 0) {
    s_k[warp] = k2;
    s_v[warp] = va;
  }
  __syncthreads();
  if (threadIdx.x == 0 && j0 < L) {
    float kt = 0.f, vt = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      kt = max_nan(kt, s_k[w]);
      vt = max_nan(vt, s_v[w]);
    }
    atomicMax(reinterpret_cast<int*>(kv_max) + 2 * bh, __float_as_int(sqrtf(kt) * p.k_scale_host));
    atomicMax(reinterpret_cast<int*>(kv_max) + 2 * bh + 1, __float_as_int(vt * p.v_scale));
  }
  if (h != 0 || chunk != 0) return;
  const int nq = p.rows * p.h_q;   // this sequence's query vectors
  for (int v = warp; v < nq; v += kWarps) {
    const char* qr = static_cast<const char*>(p.q) + (static_cast<int64_t>(b) * nq + v) * p.d * QT::kBytes;
    float qs = 0.f;
    for (int e = 2 * lane; e < p.d; e += 64) {
      const float2 qq = load_pair<QT>(qr + e * QT::kBytes);
      qs = fmaf(qq.x, qq.x, fmaf(qq.y, qq.y, qs));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) qs += __shfl_xor_sync(0xffffffffu, qs, o);
    if (lane == 0) q_norm[static_cast<int64_t>(b) * nq + v] = sqrtf(qs);
  }
}

cudaError_t bounds_dispatch(const DecodeParams& p, int q_dtype, int pool_dtype, float* q_norm, float* kv_max,
                            cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(kv_max, 0, static_cast<size_t>(p.batch) * p.h_kv * 2 * sizeof(float), stream);
  if (e != cudaSuccess) return e;
  const int n_chunks = p.max_seq_len > 0 ? (p.max_seq_len + kBoundsChunk - 1) / kBoundsChunk : 1;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.batch) * p.h_kv * n_chunks);
#define NBX_BOUNDS(PT, QT) bounds_kernel<PT, QT><<<grid, kBoundsThreads, 0, stream>>>(p, q_norm, kv_max, n_chunks)
  if (q_dtype == NBX_F32) {
    if (pool_dtype == NBX_F32) NBX_BOUNDS(F32, F32);
    else if (pool_dtype == NBX_BF16) NBX_BOUNDS(BF16, F32);
    else NBX_BOUNDS(E4M3, F32);
  } else {
    if (pool_dtype == NBX_F32) NBX_BOUNDS(F32, BF16);
    else if (pool_dtype == NBX_BF16) NBX_BOUNDS(BF16, BF16);
    else NBX_BOUNDS(E4M3, BF16);
  }
#undef NBX_BOUNDS
  return cudaGetLastError();
}

template <bool X>
cudaError_t launch_plan(const DecodeParams& p, cudaStream_t stream) {
  const bool tc = p.tc_units > 0;
  size_t smem = plan_smem_bytes(p.batch);
  if (X && (p.key_begin != nullptr || p.key_end != nullptr)) {
    static std::atomic<uint64_t> configured{0};   // devices whose shared-memory limit is raised
    const uint64_t bit = 1ull << (device_info().device & 63);
    if ((configured.load() & bit) == 0) {
      cudaError_t e =
          cudaFuncSetAttribute(plan_kernel<true, X>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxSmem);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(plan_kernel<false, X>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxSmem);
      if (e != cudaSuccess) return e;
      configured.fetch_or(bit);
    }
    smem = plan_ranges_smem_bytes(p.batch, tc);
  }
  return tc ? launch_pdl(plan_kernel<true, X>, 1u, kPlanThreads, smem, stream, p)
            : launch_pdl(plan_kernel<false, X>, 1u, kPlanThreads, smem, stream, p);
}

template <bool X, int N>
cudaError_t launch_merge(const DecodeParams& p, unsigned grid, cudaStream_t stream) {
  return p.part_f16 ? launch_pdl(decode_merge_kernel<true, X, N>, grid, kDecodeMergeThreads, 0, stream, p)
                    : launch_pdl(decode_merge_kernel<false, X, N>, grid, kDecodeMergeThreads, 0, stream, p);
}

cudaError_t decode_dispatch(const DecodeParams& p, int q_dtype, int pool_dtype, int x, int grid_limit,
                            cudaStream_t stream) {
  DecodeParams q = p;
  const bool mma = x ? mma_path_applies_modified(p, q_dtype, pool_dtype) : mma_path_applies(p, q_dtype, pool_dtype);
  // fp8 pools on tensor cores: f16 partials (block scales may take acc / l out of f16's range)
  q.part_f16 = mma && pool_dtype == NBX_E4M3 && !(x & kBlockScaled) ? 1 : 0;
  q.pool_e4m3 = pool_dtype == NBX_E4M3;
  q.range_tiles = 1;
  if (mma) {
    // a tensor-core window: splits sized for one wave of work units over the GPU's SMs (the grid
    // limit does not enter, so the partition, and the result, is the same at any grid size)
    q.tc_units = device_info().sm_count;
    q.range_tiles = (p.rows * p.group + kMmaRowsPerTile - 1) / kMmaRowsPerTile;
    q.tc_pairs = p.h_kv * q.range_tiles;
  }
  const bool warps = x && !mma && warp_path_applies(q_dtype, pool_dtype);
  if (warps) {   // one unit a resident warp over the GPU
    // (splits round up, by half a split a sequence on average: taken off the aim)
    const int units = device_info().sm_count * warp_path_warps(pool_dtype, p.d);
    q.tc_pairs = p.h_kv * ((p.rows * p.group + kWarpUnitVectors - 1) / kWarpUnitVectors);
    const int64_t extra = static_cast<int64_t>(q.tc_pairs) * p.batch / 2;
    q.tc_units = extra < units / 2 ? units - static_cast<int>(extra) : units / 2;
    q.tc_warps = units;
    q.tc_round_up = 1;
  }
  cudaError_t e = x ? launch_plan<true>(q, stream) : launch_plan<false>(q, stream);
  if (e != cudaSuccess) return e;
  if (mma && (x & kBlockScaled)) e = decode_dispatch_mma_block(q, (x & kScoreMod) != 0, grid_limit, stream);
  else if (mma)
    e = x ? decode_dispatch_mma_mod(q, pool_dtype, grid_limit, stream) : decode_dispatch_mma(q, pool_dtype, grid_limit, stream);
  else if (warps && (x & kBlockScaled)) e = decode_dispatch_warp_block(q, q_dtype, (x & kScoreMod) != 0, grid_limit, stream);
  else if (warps)
    e = pool_dtype == NBX_E4M3 ? decode_dispatch_warp_e4m3(q, q_dtype, grid_limit, stream)
                               : decode_dispatch_warp_bf16(q, grid_limit, stream);
  else if (x) e = decode_dispatch_simt_mod(q, q_dtype, pool_dtype, grid_limit, stream);
  else if (pool_dtype == NBX_F32) e = decode_dispatch_F32(q, q_dtype, grid_limit, stream);
  else if (pool_dtype == NBX_BF16) e = decode_dispatch_BF16(q, q_dtype, grid_limit, stream);
  else e = decode_dispatch_E4M3(q, q_dtype, grid_limit, stream);
  if (e != cudaSuccess) return e;
  // every sequence has one split: the partials are the output (but for rows a modified window marked). A modified
  // decode's workspace has room for splits of 64 positions; the plan's own rules say how many there can be.
  int most = q.max_splits;
  if (x && !mma) most = std::min(most, warps ? q.max_seq_len / 64 : (q.max_seq_len - 1) / kSimtSplitPositions + 1);
  if (most <= 1 && !(x && mma)) return cudaSuccess;
  const int64_t items = static_cast<int64_t>(q.batch) * q.h_kv * q.row_blocks * kQB * ((q.d / 4 + 31) / 32);
  int64_t grid = static_cast<int64_t>(device_info().sm_count) * 24;
  if (grid > items) grid = items;
  const unsigned g = static_cast<unsigned>(grid);
  // A window has many rows of few splits: fewer loads of a row in flight, more warps (128 rows of 24 heads of 256 in
  // 6 splits: 2 of 11 us less). A single row has few rows and up to 64 splits.
  if (x && mma) return launch_merge<true, 8>(q, g, stream);
  return x ? launch_merge<true, 32>(q, g, stream) : launch_merge<false, 32>(q, g, stream);
}

}  // namespace nbx
