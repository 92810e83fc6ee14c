// Page bookkeeping of a paged cache on the device: copying pages, forking rows of the block table with
// copy of the last partial page, and compacting the pages in use.
//
// A page is in use while some entry of the block table names it. No reference counts are kept, so there
// is nothing that a graph replay, a dropped call or a freed row (its entries set to -1) could leave
// wrong; each call marks the pages named by the table first, one warp per row. That costs the table's
// bytes, a few hundred KB, against the MB to GB of positions that are then copied.
//
// The copies bound these calls: 2 bytes of traffic a byte moved. A warp moves 4 KB of one (page, KV head,
// K or V) at a time, every lane with eight 16-byte loads in flight, so small pages and partly filled ones
// spread over the SMs as whole ones do; only the positions a page holds are copied.
#include <atomic>

#include "nbx_device.cuh"
#include "nbx_internal.h"

namespace nbx {
namespace {

constexpr int kChunk = 4096;          // bytes a warp copies at a time
constexpr int kCopyThreads = 256;
constexpr int kPlanThreads = 1024;    // single-CTA steps
constexpr int kScanPages = 2048;      // pages per CTA of the compaction's scan
// Up to these sizes one CTA does all the bookkeeping of a call, where the launches of the steps of their own cost
// about 10 us on the GPU (and each costs the host 2). A fork of half of 64 rows of 250 pages: 7.5 us against 16.6, of
// 250 rows of 250: 13 against 16, of 1000 rows of 10 (a warp takes a row at a time): 30 against 17. A compaction of 128
// pages: 4.3 against 12.5, of 20000: 18 against 15.
constexpr int64_t kSmallTable = 65536;        // entries of the block table
constexpr int kForkSmallRows = 256;           // rows, and forks
constexpr int kForkSmallPages = 262144;       // pages: a bitmap of 32 KB
constexpr int kCompactSmallPages = 12288;     // pages: fill counts and destinations of 72 KB

int64_t up256(int64_t x) { return (x + 255) & ~static_cast<int64_t>(255); }

// ------------------------------------------------------------------------------------ copying pages
// moves[m] = {source page, destination page, positions}: positions 0 .. positions - 1 of every KV head.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CopyPagesParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5;
  const int64_t n_warps = (static_cast<int64_t>(gridDim.x) * kCopyThreads) >> 5;
  const int n_moves = min(max(*p.n_moves, 0), p.max_moves);
  const int per_move = 2 * p.h_kv * p.chunks;
  const int64_t items = static_cast<int64_t>(n_moves) * per_move;
  for (int64_t it = warp; it < items; it += n_warps) {
    const int m = static_cast<int>(it / per_move);
    int rem = static_cast<int>(it - static_cast<int64_t>(m) * per_move);
    const int c = rem % p.chunks;
    rem /= p.chunks;
    const int which = rem & 1, h = rem >> 1;
    const int src = p.moves[3 * static_cast<int64_t>(m)], dst = p.moves[3 * static_cast<int64_t>(m) + 1];
    const int count = p.moves[3 * static_cast<int64_t>(m) + 2];
    const bool pages_ok = src >= 0 && src < p.num_pages && dst >= 0 && dst < p.num_pages;
    if (!pages_ok || count < 0 || count > p.page_tokens) {
      if (lane == 0 && rem == 0 && c == 0) raise_status(p.status, pages_ok ? NBX_DEV_BAD_LEN : NBX_DEV_BAD_PAGE);
      continue;
    }
    if (src == dst) continue;
    const int64_t head_bytes = static_cast<int64_t>(p.page_tokens) * p.row_bytes;
    const int64_t used = static_cast<int64_t>(count) * p.row_bytes;   // a multiple of 16
    const int64_t from = static_cast<int64_t>(c) * kChunk;
    char* const pool = static_cast<char*>(which ? p.v_pool : p.k_pool);
    const char* const sp = pool + (static_cast<int64_t>(src) * p.h_kv + h) * head_bytes + from;
    char* const dp = pool + (static_cast<int64_t>(dst) * p.h_kv + h) * head_bytes + from;
    const int bytes = static_cast<int>(min(static_cast<int64_t>(kChunk), used - from));   // <= 0: nothing held here
    uint4 v[kChunk / 512];
#pragma unroll
    for (int i = 0; i < kChunk / 512; ++i)
      if (i * 512 + lane * 16 < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(sp + i * 512 + lane * 16));
#pragma unroll
    for (int i = 0; i < kChunk / 512; ++i)
      if (i * 512 + lane * 16 < bytes) __stcs(reinterpret_cast<uint4*>(dp + i * 512 + lane * 16), v[i]);
    if (c == 0 && p.k_scales != nullptr) {   // the scales of the blocks that hold positions
      float* const sc = which ? p.v_scales : p.k_scales;
      const int nb = p.page_tokens / p.scale_tokens;
      const int n = (count + p.scale_tokens - 1) / p.scale_tokens;
      for (int i = lane; i < n; i += 32)
        sc[(static_cast<int64_t>(dst) * p.h_kv + h) * nb + i] = sc[(static_cast<int64_t>(src) * p.h_kv + h) * nb + i];
    }
  }
}

cudaError_t launch_copy(const CopyPagesParams& p, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(p.max_moves) * 2 * p.h_kv * p.chunks;
  int64_t grid = (warps * 32 + kCopyThreads - 1) / kCopyThreads;
  const int64_t cap = static_cast<int64_t>(device_info().sm_count) * 8;
  if (grid > cap) grid = cap;
  if (grid < 1) grid = 1;
  return launch_pdl(copy_pages_kernel, static_cast<unsigned>(grid), kCopyThreads, 0, stream, p);
}

// ------------------------------------------------------------------------------------ block scan
// Exclusive prefix sum of one int per thread over the CTA (any multiple of 32 threads up to 1024);
// *total gets the sum. s: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int* s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the previous use of s is over
  if (lane == 31) s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? s[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s[lane] = w;
    if (lane == 31) s[32] = w;
  }
  __syncthreads();
  *total = s[32];
  return x - v + (warp > 0 ? s[warp - 1] : 0);
}

// ------------------------------------------------------------------------------------ fork
// Three steps, each a kernel of its own for a large table; for a small one a single CTA does all three in turn (a
// launch less saves more than the SMs would: 64 forks in 72 rows of 250 pages took 14.5 us on the GPU as memset and
// four launches).
//
// Step 1, one warp per row: which fork overwrites the row (the first in order that names it), which
// fork is the first to read it, and, for a row whose pages stay (not overwritten, or read), its pages
// marked in the bitmap. A row that is both read and overwritten is kept aside, as are the lengths, so
// that step 3 writes rows in any order.
__device__ __forceinline__ void fork_mark(const ForkParams& p, uint32_t* bitmap, int warp, int n_warps) {
  const int lane = threadIdx.x & 31;
  for (int row = warp; row < p.batch; row += n_warps) {
    int writer = p.n_fork, reader = p.n_fork;
    for (int i = lane; i < p.n_fork; i += 32) {
      const int s = p.fork_src[i], d = p.fork_dst[i];
      if (d == row && s >= 0 && s < p.batch) writer = min(writer, i);
      if (s == row && d >= 0 && d < p.batch) reader = min(reader, i);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      writer = min(writer, __shfl_xor_sync(0xffffffffu, writer, o));
      reader = min(reader, __shfl_xor_sync(0xffffffffu, reader, o));
    }
    const bool over = writer < p.n_fork, read = reader < p.n_fork;
    if (lane == 0) p.row_info[row] = make_int4(writer, reader, p.seq_lens[row], 0);
    if (over && !read) continue;
    const int32_t* const bt = p.block_table + static_cast<int64_t>(row) * p.max_pages;
    int32_t* const keep = p.row_keep + static_cast<int64_t>(row) * p.max_pages;
#pragma unroll 4
    for (int j = lane; j < p.max_pages; j += 32) {
      const int pg = bt[j];
      if (over) keep[j] = pg;
      if (pg >= 0 && pg < p.num_pages) atomicOr(bitmap + (pg >> 5), 1u << (pg & 31));
      else if (pg >= p.num_pages) raise_status(p.status, NBX_DEV_BAD_PAGE);
    }
  }
}

// Step 2, one CTA: every fork's outcome, the fresh pages (the lowest free ids, in order of the forks)
// and the list of moves.
__device__ __forceinline__ void fork_plan(const ForkParams& p, const uint32_t* bitmap) {
  __shared__ int s_scan[33];
  const int tid = threadIdx.x;
  // ---- forks that need a fresh page, ranked in order
  int base = 0;
  for (int i0 = 0; i0 < p.n_fork; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int what = kForkNone, need = 0, len = 0;
    if (i < p.n_fork) {
      const int s = p.fork_src[i], d = p.fork_dst[i];
      if (s < 0 || s >= p.batch || d < 0 || d >= p.batch || p.row_info[d].x != i) {
        raise_status(p.status, NBX_DEV_BAD_ROW);   // a row outside the table, or a destination named before
      } else {
        const int4 ri = p.row_info[s];
        len = ri.z;
        if (len < 0 || static_cast<int64_t>(len) > static_cast<int64_t>(p.max_pages) * p.page_tokens) {
          raise_status(p.status, NBX_DEV_BAD_LEN);
          what = kForkEmpty;
        } else {
          what = kForkShare;
          const int rest = len % p.page_tokens;
          // the source row is overwritten too: its first reader takes the partial page itself
          const bool takes = ri.x < p.n_fork && ri.y == i;
          if (rest != 0 && !takes) {
            const int32_t* const row = ri.x < p.n_fork ? p.row_keep : p.block_table;
            const int pg = row[static_cast<int64_t>(s) * p.max_pages + len / p.page_tokens];
            if (pg < 0 || pg >= p.num_pages) {
              raise_status(p.status, NBX_DEV_BAD_PAGE);   // nothing to copy: the entry is taken over as it is
            } else {
              what = kForkCopy;
              need = 1;
            }
          }
        }
      }
    }
    int total;
    const int rank = base + block_scan(need, s_scan, &total);
    base += total;
    if (i < p.n_fork) p.outcome[i] = make_int4(what, rank, len, -1);
  }
  const int n_need = base;
  // ---- the n_need lowest free pages, in ascending order
  const int words = (p.num_pages + 31) / 32;
  int found = 0;
  for (int w0 = 0; w0 < words && found < n_need; w0 += kPlanThreads) {
    const int w = w0 + tid;
    uint32_t free_bits = 0;
    if (w < words) {
      free_bits = ~bitmap[w];
      if (w == words - 1 && (p.num_pages & 31)) free_bits &= (1u << (p.num_pages & 31)) - 1u;
    }
    int total;
    int at = found + block_scan(__popc(free_bits), s_scan, &total);
    found += total;
    while (free_bits && at < n_need) {
      p.fresh[at++] = w * 32 + __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
    }
  }
  const int n_copy = min(found, n_need);   // the same in every thread
  __syncthreads();   // orders the writes of fresh and outcome before the reads below (same CTA)
  for (int i = tid; i < p.n_fork; i += kPlanThreads) {
    int4 o = p.outcome[i];
    if (o.x != kForkCopy) continue;
    if (o.y >= n_copy) {   // no page left for this one
      raise_status(p.status, NBX_DEV_NO_PAGE);
      o.x = kForkEmpty;
    } else {
      const int s = p.fork_src[i];
      const int32_t* const row = p.row_info[s].x < p.n_fork ? p.row_keep : p.block_table;
      o.w = p.fresh[o.y];
      int32_t* const mv = p.moves + 3 * static_cast<int64_t>(o.y);
      mv[0] = row[static_cast<int64_t>(s) * p.max_pages + o.z / p.page_tokens];
      mv[1] = o.w;
      mv[2] = o.z % p.page_tokens;
    }
    p.outcome[i] = o;
  }
  for (int64_t i = 3 * static_cast<int64_t>(n_copy) + tid; i < 3 * static_cast<int64_t>(p.n_fork); i += kPlanThreads)
    p.moves[i] = -1;
  if (tid == 0) *p.n_moves = n_copy;
}

// Step 3, one warp per fork: the destination's row and length.
__device__ __forceinline__ void fork_rows(const ForkParams& p, int warp, int n_warps) {
  const int lane = threadIdx.x & 31;
  for (int i = warp; i < p.n_fork; i += n_warps) {
    const int4 o = p.outcome[i];
    if (o.x == kForkNone) continue;
    const int s = p.fork_src[i], d = p.fork_dst[i];
    const int32_t* const from = (p.row_info[s].x < p.n_fork ? p.row_keep : p.block_table) +
                                static_cast<int64_t>(s) * p.max_pages;
    int32_t* const to = p.block_table + static_cast<int64_t>(d) * p.max_pages;
    const int len = o.x == kForkEmpty ? 0 : o.z;
    const int pages = (len + p.page_tokens - 1) / p.page_tokens;   // len <= max_pages * page_tokens
#pragma unroll 4
    for (int j = lane; j < p.max_pages; j += 32)
      to[j] = j >= pages ? -1 : (o.x == kForkCopy && j == pages - 1 ? o.w : from[j]);
    if (lane == 0) p.seq_lens[d] = len;
  }
}

// A kernel that writes the lengths lets its dependents start early only if they are the copies of the same
// call: the plan of a decode reads the lengths before it waits for the grid ahead of it.
__global__ void __launch_bounds__(256) fork_mark_kernel(ForkParams p) {
  pdl_wait();
  pdl_launch_dependents();
  fork_mark(p, p.bitmap, static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5),
            static_cast<int>((gridDim.x * blockDim.x) >> 5));
}
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(ForkParams p) {
  pdl_wait();
  pdl_launch_dependents();
  fork_plan(p, p.bitmap);
}
__global__ void __launch_bounds__(256) fork_rows_kernel(ForkParams p) {
  pdl_wait();
  if (p.copies) pdl_launch_dependents();
  fork_rows(p, static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5),
            static_cast<int>((gridDim.x * blockDim.x) >> 5));
}

int fork_small_bytes(int batch, int n_fork, int num_pages) {   // of shared memory
  return batch * 16 + n_fork * (16 + 4 + 4 + 4) + (num_pages + 31) / 32 * 4;
}

// The three steps in one CTA, what they hand on in shared memory (in global memory: 10.4 against 8.0 us for 64 forks in
// 72 rows of 250 pages, the copies in it).
__global__ void __launch_bounds__(kPlanThreads) fork_small_kernel(ForkParams p) {
  extern __shared__ int4 fork_sm[];
  int4* const info = fork_sm;
  ForkParams q = p;
  q.row_info = info;
  q.outcome = info + p.batch;
  q.fresh = reinterpret_cast<int32_t*>(q.outcome + p.n_fork);
  int32_t* const src = q.fresh + p.n_fork;
  int32_t* const dst = src + p.n_fork;
  uint32_t* const bitmap = reinterpret_cast<uint32_t*>(dst + p.n_fork);
  q.fork_src = src;
  q.fork_dst = dst;
  const int tid = threadIdx.x;
  for (int w = tid; w < (p.num_pages + 31) / 32; w += kPlanThreads) bitmap[w] = 0u;
  pdl_wait();
  if (p.copies) pdl_launch_dependents();
  for (int r = tid; r < p.batch; r += kPlanThreads) info[r] = make_int4(p.n_fork, p.n_fork, p.seq_lens[r], 0);
  for (int i = tid; i < p.n_fork; i += kPlanThreads) {
    src[i] = p.fork_src[i];
    dst[i] = p.fork_dst[i];
  }
  __syncthreads();
  for (int i = tid; i < p.n_fork; i += kPlanThreads) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= p.batch || d < 0 || d >= p.batch) continue;
    atomicMin(&info[d].x, i);   // the fork that overwrites the row, and the first that reads it
    atomicMin(&info[s].y, i);
  }
  __syncthreads();
  // a warp a row (the table taken as one run of entries: 10 to 14 us), kBatch loads of a lane in flight before the
  // stores, which may be to the same memory for all the compiler knows
  constexpr int kBatch = 8;
  const int warp = tid >> 5, lane = tid & 31;
  for (int row = warp; row < p.batch; row += kPlanThreads / 32) {
    const int4 ri = info[row];
    const bool over = ri.x < p.n_fork;
    if (over && ri.y >= p.n_fork) continue;
    const int32_t* const bt = p.block_table + row * p.max_pages;
    for (int j0 = lane; j0 < p.max_pages; j0 += kBatch * 32) {
      int pg[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) pg[k] = j0 + k * 32 < p.max_pages ? bt[j0 + k * 32] : -1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (over && j0 + k * 32 < p.max_pages) p.row_keep[row * p.max_pages + j0 + k * 32] = pg[k];
        if (pg[k] >= 0 && pg[k] < p.num_pages) atomicOr(bitmap + (pg[k] >> 5), 1u << (pg[k] & 31));
        else if (pg[k] >= p.num_pages) raise_status(p.status, NBX_DEV_BAD_PAGE);
      }
    }
  }
  __syncthreads();   // the bitmap, and row_keep in global memory (same CTA)
  fork_plan(q, bitmap);
  __syncthreads();   // the outcomes
  for (int i = warp; i < p.n_fork; i += kPlanThreads / 32) {
    const int4 o = q.outcome[i];
    if (o.x == kForkNone) continue;
    const int32_t* const from = (info[src[i]].x < p.n_fork ? p.row_keep : p.block_table) + src[i] * p.max_pages;
    int32_t* const to = p.block_table + dst[i] * p.max_pages;
    const int len = o.x == kForkEmpty ? 0 : o.z;
    const int pages = (len + p.page_tokens - 1) / p.page_tokens;   // len <= max_pages * page_tokens
    for (int j0 = lane; j0 < p.max_pages; j0 += kBatch * 32) {
      int pg[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int j = j0 + k * 32;
        pg[k] = j >= pages ? -1 : (o.x == kForkCopy && j == pages - 1 ? o.w : from[j]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (j0 + k * 32 < p.max_pages) to[j0 + k * 32] = pg[k];
    }
    if (lane == 0) p.seq_lens[dst[i]] = len;
  }
}

// Raises a kernel's shared-memory limit, once per device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& configured) {
  const uint64_t bit = 1ull << (device_info().device & 63);
  if (configured.load() & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured.fetch_or(bit);
  return e;
}

// ------------------------------------------------------------------------------------ compaction
// Positions row `row` holds of its page number j, or -1 if the entry names no page of the pool.
__device__ __forceinline__ int compact_fill(const CompactParams& p, int row, int j, int pg) {
  if (pg < 0) return -1;
  if (pg >= p.num_pages) {
    raise_status(p.status, NBX_DEV_BAD_PAGE);
    return -1;
  }
  const int64_t len = p.seq_lens[row];
  if (j == 0 && (len < 0 || len > static_cast<int64_t>(p.max_pages) * p.page_tokens))
    raise_status(p.status, NBX_DEV_BAD_LEN);
  const int64_t left = len - static_cast<int64_t>(j) * p.page_tokens;
  return left <= 0 ? 0 : (left >= p.page_tokens ? p.page_tokens : static_cast<int>(left));
}

// fill[page] = 1 + the most positions a row holds of the page, 0 for a free page.
__global__ void __launch_bounds__(256) compact_mark_kernel(CompactParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t n_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int per_row = (p.max_pages + 31) / 32;
  for (int64_t it = warp; it < static_cast<int64_t>(p.batch) * per_row; it += n_warps) {
    const int row = static_cast<int>(it / per_row);
    const int j = static_cast<int>(it - static_cast<int64_t>(row) * per_row) * 32 + lane;
    if (j >= p.max_pages) continue;
    const int pg = p.block_table[static_cast<int64_t>(row) * p.max_pages + j];
    const int cnt = compact_fill(p, row, j, pg);
    if (cnt >= 0) atomicMax(p.fill + pg, 1 + cnt);
  }
}

// Pages in use of every chunk of kScanPages.
__global__ void __launch_bounds__(256) compact_count_kernel(CompactParams p) {
  __shared__ int s_scan[33];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kScanPages;
  int n = 0;
  for (int i = threadIdx.x; i < kScanPages; i += 256)
    if (first + i < p.num_pages) n += p.fill[first + i] != 0;
  int total;
  block_scan(n, s_scan, &total);
  if (threadIdx.x == 0) p.chunk_live[blockIdx.x] = total;
}

// Every CTA sums the chunk counts (n_live of them in all, and those before its own chunk), then ranks
// the pages of its chunk: a page in use at or above n_live is source number (pages in use before it) -
// (pages in use below n_live), a free page below n_live is destination number (free pages before it).
// There are as many of one as of the other.
__global__ void __launch_bounds__(256) compact_rank_kernel(CompactParams p) {
  __shared__ int s_scan[33];
  constexpr int kPer = kScanPages / 256;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int all = 0, mine = 0;
  for (int c = tid; c < p.n_chunks; c += 256) {
    const int v = p.chunk_live[c];
    all += v;
    if (c < static_cast<int>(blockIdx.x)) mine += v;
  }
  int n_live, before;
  block_scan(all, s_scan, &n_live);
  block_scan(mine, s_scan, &before);
  // pages in use below n_live: whole chunks, then the part of the chunk that n_live falls into
  const int edge = n_live / kScanPages;
  int low = 0;
  for (int c = tid; c < min(edge, p.n_chunks); c += 256) low += p.chunk_live[c];
  for (int i = edge * kScanPages + tid; i < n_live; i += 256) low += p.fill[i] != 0;
  int below;
  block_scan(low, s_scan, &below);
  const int first = blockIdx.x * kScanPages + tid * kPer;
  int f[kPer], n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    f[i] = first + i < p.num_pages ? p.fill[first + i] : 0;
    n += f[i] != 0;
  }
  int total;
  int live = before + block_scan(n, s_scan, &total);   // pages in use before this thread's first
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int pg = first + i;
    if (pg >= p.num_pages) break;
    if (f[i] != 0) {
      if (pg >= n_live) {
        const int k = live - below;
        p.rank[pg] = k;
        p.moves[3 * static_cast<int64_t>(k)] = pg;
        p.moves[3 * static_cast<int64_t>(k) + 2] = f[i] - 1;
      }
      ++live;
    } else if (pg < n_live) {
      p.moves[3 * static_cast<int64_t>(pg - live) + 1] = pg;
    }
  }
  const int n_moves = n_live - below;
  for (int64_t i = 3 * static_cast<int64_t>(n_moves) + blockIdx.x * 256 + tid; i < 3 * static_cast<int64_t>(p.max_moves);
       i += static_cast<int64_t>(gridDim.x) * 256)
    p.moves[i] = -1;
  if (blockIdx.x == 0 && tid == 0) {
    p.counts[0] = n_moves;
    p.counts[1] = n_live;
  }
}

// All of it in one CTA, for a small table and pool: fill and the destinations live in shared memory, a page
// that moves holds -1 - (number of its move) once it is ranked.
__global__ void __launch_bounds__(kPlanThreads) compact_small_kernel(CompactParams p) {
  extern __shared__ int fill[];   // [num_pages], then the destinations [num_pages / 2]
  __shared__ int s_scan[33];
  int* const dst = fill + p.num_pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < p.num_pages; i += kPlanThreads) fill[i] = 0;
  pdl_wait();
  pdl_launch_dependents();   // (this kernel writes no lengths)
  __syncthreads();
  const int n = p.batch * p.max_pages;
#pragma unroll 4
  for (int i = tid; i < n; i += kPlanThreads) {
    const int row = i / p.max_pages, pg = p.block_table[i];
    const int cnt = compact_fill(p, row, i - row * p.max_pages, pg);
    if (cnt >= 0) atomicMax(fill + pg, 1 + cnt);
  }
  __syncthreads();
  // each warp takes a run of pages, 32 at a time; ranks as in compact_rank_kernel
  const int per = (p.num_pages + kPlanThreads - 1) / kPlanThreads * 32;
  const int lo = min(p.num_pages, warp * per), hi = min(p.num_pages, lo + per);
  int mine = 0;
  for (int i = lo + lane; i < hi; i += 32) mine += fill[i] != 0;
  int n_live, below;
  int live = block_scan(mine, s_scan, &n_live);
  live = __shfl_sync(0xffffffffu, live, 0);   // pages in use before the warp's run
  int low = 0;
  for (int i = lo + lane; i < min(hi, n_live); i += 32) low += fill[i] != 0;
  block_scan(low, s_scan, &below);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int pg = i0 + lane;
    const int f = pg < hi ? fill[pg] : 0;
    const uint32_t used = __ballot_sync(0xffffffffu, f != 0);
    const int before = live + __popc(used & ((1u << lane) - 1u));
    if (pg < hi) {
      if (f != 0 && pg >= n_live) {
        p.moves[3 * (before - below)] = pg;
        p.moves[3 * (before - below) + 2] = f - 1;
        fill[pg] = -1 - (before - below);
      } else if (f == 0 && pg < n_live) {
        p.moves[3 * (pg - before) + 1] = pg;
        dst[pg - before] = pg;
      }
    }
    live += __popc(used);
  }
  const int n_moves = n_live - below;
  for (int64_t i = 3 * n_moves + tid; i < 3 * static_cast<int64_t>(p.max_moves); i += kPlanThreads) p.moves[i] = -1;
  if (tid == 0) {
    p.counts[0] = n_moves;
    p.counts[1] = n_live;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < n; i += kPlanThreads) {
    const int pg = p.block_table[i];
    p.new_block_table[i] = pg >= n_live && pg < p.num_pages ? dst[-1 - fill[pg]] : pg;
  }
}

// The table with every moved page's new id.
__global__ void __launch_bounds__(256) compact_table_kernel(CompactParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int n_live = p.counts[1];
  const int64_t n = static_cast<int64_t>(p.batch) * p.max_pages;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    int pg = p.block_table[i];
    if (pg >= n_live && pg < p.num_pages) pg = p.moves[3 * static_cast<int64_t>(p.rank[pg]) + 1];
    p.new_block_table[i] = pg;
  }
}

unsigned grid_for(int64_t threads, int per_cta) {
  int64_t g = (threads + per_cta - 1) / per_cta;
  const int64_t cap = static_cast<int64_t>(device_info().sm_count) * 8;
  if (g > cap) g = cap;
  return static_cast<unsigned>(g < 1 ? 1 : g);
}

// ------------------------------------------------------------------------------------ host checks
struct PoolArgs {
  void *k_pool, *v_pool;
  int pool_dtype, num_pages, h_kv, page_tokens, d;
  float *k_scales, *v_scales;
  int scale_tokens;
};

// The checks every page call makes of its pools; *copies: there are pools to copy in.
int check_pools(const PoolArgs& a, bool pools_required, bool* copies) {
  if (a.num_pages < 1 || a.page_tokens < 1) return NBX_ERR_SHAPE;
  *copies = a.k_pool != nullptr || a.v_pool != nullptr;
  if (!*copies && !pools_required) return NBX_OK;
  if (a.h_kv < 1 || a.d < 16 || a.d > 1024 || (a.d % 16) != 0) return NBX_ERR_SHAPE;
  if (a.pool_dtype != NBX_F32 && a.pool_dtype != NBX_BF16 && a.pool_dtype != NBX_E4M3) return NBX_ERR_DTYPE;
  const bool scaled = a.k_scales != nullptr || a.v_scales != nullptr;
  if (scaled && a.pool_dtype != NBX_E4M3) return NBX_ERR_DTYPE;
  if (scaled && !scale_tokens_ok(a.scale_tokens, a.page_tokens)) return NBX_ERR_PAGE_ALIGN;
  const int64_t elt = a.pool_dtype == NBX_F32 ? 4 : (a.pool_dtype == NBX_BF16 ? 2 : 1);
  if (static_cast<int64_t>(a.page_tokens) * a.d * elt * a.h_kv > 0x7fffffffll) return NBX_ERR_SHAPE;
  if (!a.k_pool || !a.v_pool || (scaled && (!a.k_scales || !a.v_scales))) return NBX_ERR_NULL;
  if (!aligned16(a.k_pool) || !aligned16(a.v_pool)) return NBX_ERR_ALIGN;
  return NBX_OK;
}

CopyPagesParams copy_params(const PoolArgs& a, const int32_t* moves, const int32_t* n_moves, int max_moves,
                            int32_t* status) {
  const int elt = a.pool_dtype == NBX_F32 ? 4 : (a.pool_dtype == NBX_BF16 ? 2 : 1);
  CopyPagesParams c = {};
  c.k_pool = a.k_pool;
  c.v_pool = a.v_pool;
  c.k_scales = a.k_scales;
  c.v_scales = a.v_scales;
  c.moves = moves;
  c.n_moves = n_moves;
  c.status = status;
  c.max_moves = max_moves;
  c.num_pages = a.num_pages;
  c.h_kv = a.h_kv;
  c.page_tokens = a.page_tokens;
  c.row_bytes = a.d * elt;
  c.scale_tokens = a.scale_tokens;
  c.chunks = static_cast<int>((static_cast<int64_t>(a.page_tokens) * c.row_bytes + kChunk - 1) / kChunk);
  return c;
}

struct ForkLayout {
  int64_t bitmap, row_info, outcome, fresh, row_keep, total;
};
ForkLayout fork_layout(int64_t batch, int64_t max_pages, int64_t n_fork, int64_t num_pages) {
  ForkLayout w;
  int64_t off = 0;
  w.bitmap = off;
  off += up256((num_pages + 31) / 32 * 4);
  w.row_info = off;
  off += up256(batch * 16);
  w.outcome = off;
  off += up256(n_fork * 16);
  w.fresh = off;
  off += up256(n_fork * 4);
  w.row_keep = off;
  off += up256(batch * max_pages * 4);
  w.total = off;
  return w;
}
struct CompactLayout {
  int64_t fill, chunk_live, rank, total;
  int n_chunks;
};
CompactLayout compact_layout(int64_t num_pages) {
  CompactLayout w;
  w.n_chunks = static_cast<int>((num_pages + kScanPages - 1) / kScanPages);
  int64_t off = 0;
  w.fill = off;
  off += up256(num_pages * 4);
  w.chunk_live = off;
  off += up256(static_cast<int64_t>(w.n_chunks) * 4);
  w.rank = off;
  off += up256(num_pages * 4);
  w.total = off;
  return w;
}
bool table_ok(int batch, int max_pages) {
  return batch >= 0 && max_pages >= 1 && static_cast<int64_t>(batch) * max_pages <= 0x7fffffffll;
}

}  // namespace
}  // namespace nbx

using namespace nbx;

extern "C" {

NBX_API int nbx_paged_kv_copy_pages(const int32_t* moves, const int32_t* n_moves, int max_moves, void* k_pool,
                                    void* v_pool, int pool_dtype, int num_pages, int h_kv, int page_tokens, int d,
                                    float* k_scales, float* v_scales, int scale_tokens, int32_t* status,
                                    void* stream) {
  const PoolArgs a = {k_pool, v_pool, pool_dtype, num_pages, h_kv, page_tokens, d, k_scales, v_scales, scale_tokens};
  bool copies;
  if (max_moves < 0) return NBX_ERR_SHAPE;
  const int st = check_pools(a, true, &copies);
  if (st != NBX_OK) return st;
  if (max_moves == 0) return NBX_OK;
  if (!moves || !n_moves) return NBX_ERR_NULL;
  const cudaError_t e = launch_copy(copy_params(a, moves, n_moves, max_moves, status), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
}

NBX_API size_t nbx_paged_kv_fork_workspace_bytes(int batch, int max_pages, int n_fork, int num_pages) {
  if (!table_ok(batch, max_pages) || n_fork < 0 || num_pages < 1) return 0;
  return static_cast<size_t>(fork_layout(batch, max_pages, n_fork, num_pages).total);
}

NBX_API int nbx_paged_kv_fork(int32_t* block_table, int max_pages, int32_t* seq_lens, int batch,
                              const int32_t* fork_src, const int32_t* fork_dst, int n_fork, void* k_pool, void* v_pool,
                              int pool_dtype, int num_pages, int h_kv, int page_tokens, int d, float* k_scales,
                              float* v_scales, int scale_tokens, int32_t* moves, int32_t* n_moves, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream) {
  const PoolArgs a = {k_pool, v_pool, pool_dtype, num_pages, h_kv, page_tokens, d, k_scales, v_scales, scale_tokens};
  bool copies;
  if (!table_ok(batch, max_pages) || n_fork < 0) return NBX_ERR_SHAPE;
  const int ok = check_pools(a, false, &copies);
  if (ok != NBX_OK) return ok;
  if (n_fork == 0 || batch == 0) return NBX_OK;
  if (!block_table || !seq_lens || !fork_src || !fork_dst || !moves || !n_moves || !workspace) return NBX_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return NBX_ERR_ALIGN;
  const ForkLayout w = fork_layout(batch, max_pages, n_fork, num_pages);
  if (workspace_bytes < static_cast<size_t>(w.total)) return NBX_ERR_WORKSPACE;
  char* const ws = static_cast<char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ForkParams p = {};
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.fork_src = fork_src;
  p.fork_dst = fork_dst;
  p.moves = moves;
  p.n_moves = n_moves;
  p.status = status;
  p.bitmap = reinterpret_cast<uint32_t*>(ws + w.bitmap);
  p.row_info = reinterpret_cast<int4*>(ws + w.row_info);
  p.outcome = reinterpret_cast<int4*>(ws + w.outcome);
  p.fresh = reinterpret_cast<int32_t*>(ws + w.fresh);
  p.row_keep = reinterpret_cast<int32_t*>(ws + w.row_keep);
  p.max_pages = max_pages;
  p.batch = batch;
  p.n_fork = n_fork;
  p.num_pages = num_pages;
  p.page_tokens = page_tokens;
  p.copies = copies;
  cudaError_t e;
  if (static_cast<int64_t>(batch) * max_pages <= kSmallTable && batch <= kForkSmallRows && n_fork <= kForkSmallRows &&
      num_pages <= kForkSmallPages) {
    static std::atomic<uint64_t> configured{0};
    e = allow_smem(reinterpret_cast<const void*>(fork_small_kernel),
                   fork_small_bytes(kForkSmallRows, kForkSmallRows, kForkSmallPages), configured);
    if (e == cudaSuccess)
      e = launch_pdl(fork_small_kernel, 1u, kPlanThreads,
                     static_cast<size_t>(fork_small_bytes(batch, n_fork, num_pages)), st, p);
    if (e == cudaSuccess && copies) e = launch_copy(copy_params(a, moves, n_moves, n_fork, status), st);
    return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
  }
  e = cudaMemsetAsync(p.bitmap, 0, static_cast<size_t>(w.row_info - w.bitmap), st);
  if (e == cudaSuccess) e = launch_pdl(fork_mark_kernel, grid_for(static_cast<int64_t>(batch) * 32, 256), 256u, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(fork_plan_kernel, 1u, kPlanThreads, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(fork_rows_kernel, grid_for(static_cast<int64_t>(n_fork) * 32, 256), 256u, 0, st, p);
  if (e == cudaSuccess && copies) e = launch_copy(copy_params(a, moves, n_moves, n_fork, status), st);
  return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
}

NBX_API size_t nbx_paged_kv_compact_workspace_bytes(int num_pages) {
  return num_pages < 1 ? 0 : static_cast<size_t>(compact_layout(num_pages).total);
}

NBX_API int nbx_paged_kv_compact(const int32_t* block_table, int32_t* new_block_table, int max_pages,
                                 const int32_t* seq_lens, int batch, void* k_pool, void* v_pool, int pool_dtype,
                                 int num_pages, int h_kv, int page_tokens, int d, float* k_scales, float* v_scales,
                                 int scale_tokens, int32_t* moves, int max_moves, int32_t* counts, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream) {
  const PoolArgs a = {k_pool, v_pool, pool_dtype, num_pages, h_kv, page_tokens, d, k_scales, v_scales, scale_tokens};
  bool copies;
  if (!table_ok(batch, max_pages)) return NBX_ERR_SHAPE;
  const int ok = check_pools(a, false, &copies);
  if (ok != NBX_OK) return ok;
  if (num_pages > (1 << 30)) return NBX_ERR_SHAPE;       // page arithmetic is 32-bit
  if (max_moves < num_pages / 2) return NBX_ERR_SHAPE;   // the most pages that can have to move
  if (batch == 0) return NBX_OK;
  if (!block_table || !new_block_table || !seq_lens || !counts || !workspace || (!moves && max_moves > 0))
    return NBX_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return NBX_ERR_ALIGN;
  const CompactLayout w = compact_layout(num_pages);
  if (workspace_bytes < static_cast<size_t>(w.total)) return NBX_ERR_WORKSPACE;
  char* const ws = static_cast<char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CompactParams p = {};
  p.block_table = block_table;
  p.new_block_table = new_block_table;
  p.seq_lens = seq_lens;
  p.moves = moves;
  p.counts = counts;
  p.status = status;
  p.fill = reinterpret_cast<int32_t*>(ws + w.fill);
  p.chunk_live = reinterpret_cast<int32_t*>(ws + w.chunk_live);
  p.rank = reinterpret_cast<int32_t*>(ws + w.rank);
  p.batch = batch;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_tokens = page_tokens;
  p.max_moves = max_moves;
  p.n_chunks = w.n_chunks;
  const unsigned chunks = static_cast<unsigned>(w.n_chunks);
  const int64_t entries = static_cast<int64_t>(batch) * max_pages;
  cudaError_t e;
  if (entries <= kSmallTable && num_pages <= kCompactSmallPages) {
    static std::atomic<uint64_t> configured{0};
    e = allow_smem(reinterpret_cast<const void*>(compact_small_kernel), kCompactSmallPages * 6, configured);
    if (e == cudaSuccess)
      e = launch_pdl(compact_small_kernel, 1u, kPlanThreads, (static_cast<size_t>(num_pages) + num_pages / 2) * 4, st, p);
    if (e == cudaSuccess && copies && max_moves > 0)
      e = launch_copy(copy_params(a, moves, counts, max_moves, status), st);
    return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
  }
  e = cudaMemsetAsync(p.fill, 0, static_cast<size_t>(num_pages) * 4, st);
  if (e == cudaSuccess)
    e = launch_pdl(compact_mark_kernel, grid_for(static_cast<int64_t>(batch) * ((max_pages + 31) / 32) * 32, 256), 256u, 0,
                   st, p);
  if (e == cudaSuccess) e = launch_pdl(compact_count_kernel, chunks, 256u, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(compact_rank_kernel, chunks, 256u, 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(compact_table_kernel, grid_for(entries, 256), 256u, 0, st, p);
  if (e == cudaSuccess && copies && max_moves > 0)
    e = launch_copy(copy_params(a, moves, counts, max_moves, status), st);
  return e == cudaSuccess ? NBX_OK : NBX_ERR_CUDA;
}

}  // extern "C"
