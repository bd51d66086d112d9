// kvx_pages.cu -- references to the pages of a cache: rows of a block table forked,
// freed, given pages of their own, pages copied and compacted (kvx_pages_fork,
// kvx_pages_free, kvx_pages_reserve, kvx_pages_compact, kvx_cache8_copy).
//
// refs[b] is the number of table entries that hold page b.  What takes pages does so in
// an order that does not depend on timing: the i-th need of a call, in the order of rows
// and slots, gets the i-th page whose count is 0.  So needs and free pages are counted,
// their counts summed up to each warp, and both walked again in that order.  Atomics are
// integer sums, minima and maxima only.
//
// The counting kernels are one CTA, or a cluster of eight where there is more to read:
// phases of a few loads each with a barrier between, bound by the latency of those.
// Copies are bound by HBM: whole pages, 16 bytes a thread at a time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

namespace {

// --- copies --------------------------------------------------------------------

constexpr int kMaxCaches = 32;               // of a launch: their pointers are its parameters
constexpr int kCopyThreads = 256, kPiece = kCopyThreads * 16 * 4;   // bytes a CTA copies at a time

struct CacheView {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t page;              // bytes of a page's keys or values
  int heads;
};
constexpr int kMaxTables = 8;
// Tables whose entries become the pages' new numbers.
struct Tables {
  int32_t *table[kMaxTables];
  int64_t entries[kMaxTables];
  const int32_t *moved;
  int count;
};
struct CopyParams {
  CacheView cache[kMaxCaches];
  Tables tables;
  const int32_t *pairs, *count;   // count NULL: all pairs
  uint32_t *status;
  int64_t num_blocks;
  int num_caches, num_pairs, pieces;   // pieces: of the largest cache's page
};

// A CTA copies a piece of a page's keys and values at a time: eight loads a thread on
// their way before the first store.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  wait_for_kernel_before();
  let_next_kernel_start();
  for (int x = 0; x < p.tables.count; ++x) {
    int32_t *table = p.tables.table[x];
    for (int64_t i = blockIdx.x * (int64_t)kCopyThreads + threadIdx.x; i < p.tables.entries[x]; i += (int64_t)gridDim.x * kCopyThreads) {
      const int page = table[i];
      if (page >= 0 && page < p.num_blocks) {
        const int to = __ldcg(p.tables.moved + page);
        if (to != page) table[i] = to;
      } else if (page != -1) {
        raise(p.status, KVX_FLAG_BAD_BLOCK);
      }
    }
  }
  int n = p.num_pairs;
  if (p.count) {
    const int c = __ldcg(p.count);
    if (c < 0 || c > n) {
      if (blockIdx.x == 0 && threadIdx.x == 0) raise(p.status, KVX_FLAG_BAD_LENGTH);
      return;
    }
    n = c;
  }
  const int per = p.pieces * p.num_caches;
  if (per == 0) return;
  const int64_t units = (int64_t)n * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t pair = u / per;
    const int in = (int)(u - pair * per), c = in / p.pieces, piece = in - c * p.pieces;
    const int32_t from = __ldcg(p.pairs + 2 * pair), to = __ldcg(p.pairs + 2 * pair + 1);
    if (from < 0 || to < 0) continue;
    if (from >= p.num_blocks || to >= p.num_blocks) {
      if (threadIdx.x == 0) raise(p.status, KVX_FLAG_BAD_BLOCK);
      continue;
    }
    const CacheView &x = p.cache[c];
    const int64_t src = from * x.page, dst = to * x.page, at = (int64_t)piece * kPiece + threadIdx.x * 16;
    uint4 k[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * kCopyThreads * 16 < x.page) {
        k[i] = __ldcs(reinterpret_cast<const uint4 *>(x.k + src + at + i * kCopyThreads * 16));
        v[i] = __ldcs(reinterpret_cast<const uint4 *>(x.v + src + at + i * kCopyThreads * 16));
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * kCopyThreads * 16 < x.page) {
        *reinterpret_cast<uint4 *>(x.k + dst + at + i * kCopyThreads * 16) = k[i];
        *reinterpret_cast<uint4 *>(x.v + dst + at + i * kCopyThreads * 16) = v[i];
      }
    if (piece == 0)
      for (int h = threadIdx.x; h < x.heads; h += kCopyThreads) {
        x.ks[(int64_t)to * x.heads + h] = x.ks[(int64_t)from * x.heads + h];
        x.vs[(int64_t)to * x.heads + h] = x.vs[(int64_t)from * x.heads + h];
      }
  }
}

// The caches of a call: block_size 0 stands for any, if all have one.
kvx_status check_caches(const kvx_cache8 *caches, int n, int64_t num_blocks, int block_size) {
  if (n < 0 || (n > 0 && !caches)) return KVX_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    kvx_cache8 c = caches[i];
    c.block_table = reinterpret_cast<const int32_t *>(c.k_scale);   // not used
    c.max_blocks_per_req = 1;
    if (const kvx_status st = check_cache8(c)) return st;
    if (c.num_blocks != num_blocks || (block_size && c.block_size != block_size)) return KVX_ERR_INVALID_ARG;
  }
  return KVX_OK;
}
// The pages of all caches, and `tables` in the first launch.
kvx_status copy_pages(const kvx_cache8 *caches, int n, int64_t num_blocks, const int32_t *pairs, int64_t num_pairs,
                      const int32_t *count, const Tables &tables, uint32_t *status, cudaStream_t s) {
  int64_t entries = 0;
  for (int i = 0; i < tables.count; ++i) entries = tables.entries[i] > entries ? tables.entries[i] : entries;
  if (num_pairs == 0) n = 0;
  int first = 0;
  do {
    CopyParams p = {};
    p.num_caches = n - first < kMaxCaches ? n - first : kMaxCaches;
    int64_t most = 0;
    for (int i = 0; i < p.num_caches; ++i) {
      const kvx_cache8 &c = caches[first + i];
      const int64_t page = (int64_t)c.heads * c.block_size * c.head_dim;
      p.cache[i] = {(uint8_t *)c.k_codes, (uint8_t *)c.v_codes, c.k_scale, c.v_scale, page, c.heads};
      most = page > most ? page : most;
    }
    if (first == 0) p.tables = tables;
    p.pairs = pairs;
    p.count = count;
    p.status = status;
    p.num_blocks = num_blocks;
    p.num_pairs = (int)num_pairs;
    p.pieces = (int)((most + kPiece - 1) / kPiece);
    int64_t grid = num_pairs * p.num_caches * p.pieces;
    if (first == 0 && (entries + kCopyThreads - 1) / kCopyThreads > grid) grid = (entries + kCopyThreads - 1) / kCopyThreads;
    if (grid > 152 * 8) grid = 152 * 8;         // eight CTAs an SM
    if (grid > 0)
      if (const kvx_status st = launch_after(copy_kernel, dim3((unsigned)grid), kCopyThreads, 0, s, p)) return st;
    first += kMaxCaches;
  } while (first < n);
  return KVX_OK;
}

// --- rows ----------------------------------------------------------------------

struct ForkParams {
  int32_t *refs;
  int64_t num_blocks;
  const int32_t *table, *lens, *parents;
  int32_t *new_table, *new_lens;
  uint32_t *status;
  int bs, R, N, W;
};
// Pages that a row's length covers (0 where it is out of bounds).
__device__ __forceinline__ int held_of(const ForkParams &p, int r, bool tell) {
  const int len = p.lens[r];
  if (len < 0 || len > (int64_t)p.W * p.bs) {
    if (tell && threadIdx.x == 0) raise(p.status, KVX_FLAG_BAD_LENGTH);
    return 0;
  }
  return (len + (p.bs - 1)) / p.bs;
}
// CTAs 0 .. N - 1 write a new row each, the others change the counts of what an old row
// holds: a page that its length covers gains its children and loses the row itself.
__global__ void __launch_bounds__(128) fork_kernel(const __grid_constant__ ForkParams p) {
  wait_for_kernel_before();
  let_next_kernel_start();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < p.N) {
    const int n = blockIdx.x, r = p.parents[n];
    const bool has = r >= 0 && r < p.R;
    if (!has && r != -1 && tid == 0) raise(p.status, KVX_FLAG_BAD_ROW);
    const int held = has ? held_of(p, r, true) : 0;
    for (int i = tid; i < p.W; i += blockDim.x) {
      const int page = i < held ? p.table[(int64_t)r * p.W + i] : -1;
      const bool good = page >= 0 && page < p.num_blocks;
      if (i < held && !good) raise(p.status, KVX_FLAG_BAD_BLOCK);
      p.new_table[(int64_t)n * p.W + i] = good ? page : -1;
    }
    if (tid == 0) {
      const int len = has ? p.lens[r] : 0;
      p.new_lens[n] = len < 0 || len > (int64_t)p.W * p.bs ? 0 : len;
    }
    return;
  }
  const int r = blockIdx.x - p.N;
  int children = 0;
  for (int n0 = 0; n0 < p.N; n0 += blockDim.x) children += __syncthreads_count(n0 + tid < p.N && p.parents[n0 + tid] == r);
  const int held = held_of(p, r, true);
  for (int i = tid; i < p.W; i += blockDim.x) {
    const int page = p.table[(int64_t)r * p.W + i], by = i < held ? children - 1 : -1;
    if (page >= 0 && page < p.num_blocks) {
      if (by) atomicAdd(p.refs + page, by);
    } else if (page != -1) {
      raise(p.status, KVX_FLAG_BAD_BLOCK);
    }
  }
}

__global__ void __launch_bounds__(256) free_kernel(int32_t *refs, int64_t num_blocks, int32_t *table, int64_t entries, uint32_t *status) {
  wait_for_kernel_before();
  let_next_kernel_start();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < entries; i += (int64_t)gridDim.x * blockDim.x) {
    const int page = table[i];
    if (page >= 0 && page < num_blocks) atomicSub(refs + page, 1);
    else if (page != -1) raise(status, KVX_FLAG_BAD_BLOCK);
    if (page != -1) table[i] = -1;
  }
}

// --- counting ------------------------------------------------------------------

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBigCtas = 8;
// A workspace: sums of the warps, pages that are wanted, pairs that are copied; from kListAt
// on a list of num_blocks pages and one of as many pairs.
constexpr int kSums = kBigCtas * kWarps, kWantedAt = 3 * kSums, kCountAt = kWantedAt + 1, kListAt = 1024;
static_assert(kCountAt < kListAt, "workspace");
__host__ __device__ inline int64_t pairs_at(int64_t num_blocks) { return kListAt + (num_blocks + 63) / 64 * 64; }

// A barrier of all threads of the grid, which is one CTA or one cluster; what they wrote
// to global memory before it is seen behind it.
template <int CTAS>
__device__ __forceinline__ void barrier() {
  if constexpr (CTAS == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}
// The sum of the first `upto` of the warps' counts, and of all; every lane calls it.
template <int CTAS>
__device__ __forceinline__ int2 sums_of(const int32_t *counts, int upto) {
  int below = 0, all = 0;
#pragma unroll
  for (int i = 0; i < CTAS * kWarps; i += 32) {
    const int x = __ldcg(counts + i + threadIdx.x % 32);
    all += x;
    below += i + (int)(threadIdx.x % 32) < upto ? x : 0;
  }
  return make_int2(__reduce_add_sync(~0u, below), __reduce_add_sync(~0u, all));
}
// The warp's share of n: a contiguous range, in multiples of `unit`.
struct Range {
  int64_t begin, end;
};
template <int CTAS>
__device__ __forceinline__ Range share_of(int64_t n, int unit) {
  const int warp = blockIdx.x * kWarps + threadIdx.x / 32, warps = CTAS * kWarps;
  const int64_t per = ((n + warps - 1) / warps + unit - 1) / unit * unit, begin = min(warp * per, n);
  return {begin, min(begin + per, n)};
}
// f(page, count of the lane's page) for the range, 32 pages at a time, all lanes together
// (a count of -1 behind the end).
template <class F>
__device__ __forceinline__ void walk(const int32_t *refs, Range x, F f) {
  for (int64_t i = x.begin; i < x.end; i += 32 * 8) {
    int c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = i + 32 * k + threadIdx.x % 32;
      c[k] = at < x.end ? __ldcg(refs + at) : -1;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + 32 * k < x.end) f((int)(i + 32 * k + threadIdx.x % 32), c[k]);
  }
}
__device__ __forceinline__ int lanes_below(unsigned mask) {
  unsigned lt;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(lt));
  return __popc(mask & lt);
}

struct ReserveParams {
  int32_t *refs;
  int64_t num_blocks;
  int32_t *table, *copies, *work;
  const int32_t *lens, *add;
  uint32_t *status;
  int bs, R, W, add_all;
  int lanes, chunks, rows;     // of a row: lanes of a warp, times that they take; rows of a warp
};
// An entry of a row's new slots, one a lane.
struct Entry {
  int32_t *at;               // NULL: none
  int value, row, len;       // -1 no page, -(page + 2) a page that others hold too
  bool first, whole;         // of the row's entries; its page holds none of the row's slots
};
__device__ __forceinline__ Entry entry_of(const ReserveParams &p, int turn, bool tell) {
  const int lane = threadIdx.x % 32, at_once = 32 / p.lanes;
  const int r = (int)(threadIdx.x / 32) * p.rows + turn / p.chunks * at_once + lane / p.lanes;
  const int b = turn % p.chunks * 32 + lane % p.lanes;
  Entry e = {nullptr, 0, r, 0, b == 0, true};
  if (r >= p.R) {
    e.row = -1;
    return e;
  }
  const int64_t len = __ldg(p.lens + r), add = p.add ? __ldg(p.add + r) : p.add_all;
  if (len < 0 || add < 0 || add > p.add_all || len + add > (int64_t)p.W * p.bs) {
    if (tell && b == 0) raise(p.status, KVX_FLAG_BAD_LENGTH);
    return e;
  }
  const uint32_t first = (uint32_t)len / (uint32_t)p.bs, inside = (uint32_t)len - first * p.bs;
  if (add == 0 || first + b > (uint32_t)(len + add - 1) / (uint32_t)p.bs) return e;
  e.whole = b > 0 || inside == 0;
  e.at = p.table + (int64_t)r * p.W + first + b;
  e.value = *e.at;
  return e;
}
// The entries are looked after by the first CTA, rows to its warps in order, and a row's
// entries to lanes side by side: two for a token, a warp's for a prompt.  Where each
// warp takes one turn its entries stay in registers between the phases.  All CTAs
// look through the references.
//
// Which of the rows that hold a page keeps it: all that ask let go of it, and where that
// leaves none the last of them, found by a minimum over -(row + 1), takes it back.
template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) reserve_kernel(const __grid_constant__ ReserveParams p) {
  __shared__ int needs_of[kWarps];
  wait_for_kernel_before();
  let_next_kernel_start();
  const int lane = threadIdx.x % 32, in = threadIdx.x / 32, warp = blockIdx.x * kWarps + in;
  int32_t *free_of = p.work, *list = p.work + kListAt;
  const bool leads = blockIdx.x == 0;
  const int turns = in * p.rows < p.R ? p.rows / (32 / p.lanes) * p.chunks : 0;
  Entry only = {nullptr, 0, -1, 0, false, true};
  const auto entries = [&](auto f) {
    if (turns == 1) {
      f(only);
    } else {
      for (int t = 0; t < turns; ++t) {
        Entry e = entry_of(p, t, false);
        f(e);
      }
    }
  };
  bool shared = false;
  if (leads) {
    for (int t = 0; t < turns; ++t) {
      Entry e = entry_of(p, t, true);
      if (e.at && (e.value < 0 || e.value >= p.num_blocks)) {
        if (e.value != -1) raise(p.status, KVX_FLAG_BAD_BLOCK);
        if (e.value != -1) *e.at = -1;
        e.value = -1;
      } else if (e.at && __ldcg(p.refs + e.value) > 1) {
        e.value = -(e.value + 2);
        *e.at = e.value;
        shared = true;
      }
      if (turns == 1) only = e;
    }
  }
  // what is free
  const Range pages = share_of<CTAS>(p.num_blocks, 32);
  int free_here = 0;
  walk(p.refs, pages, [&](int, int c) { free_here += __popc(__ballot_sync(~0u, c == 0)); });
  if (lane == 0) free_of[warp] = free_here;
  barrier<CTAS>();
  if (leads) {
    if (__syncthreads_or(shared)) {
      entries([&](Entry &e) {
        if (e.at && e.value < -1) atomicSub(p.refs - (e.value + 2), 1);
      });
      __syncthreads();
      entries([&](Entry &e) {
        int32_t *count = p.refs - (e.value + 2);
        if (e.at && e.value < -1 && __ldcg(count) <= 0) atomicMin(count, -(e.row + 1));
      });
      __syncthreads();
    }
    int needs = 0;
    entries([&](Entry &e) {
      bool need = e.at && e.value < 0;
      if (need && e.value < -1) {
        int32_t *count = p.refs - (e.value + 2);
        if (__ldcg(count) == -(e.row + 1)) {     // others of its rows see this or the 1: not theirs
          *count = 1;
          e.value = -(e.value + 2);
          *e.at = e.value;
          need = false;
        }
      }
      needs += __popc(__ballot_sync(~0u, need));
    });
    if (lane == 0) needs_of[in] = needs;
    __syncthreads();
    const int sum = __reduce_add_sync(~0u, needs_of[lane]);
    if (threadIdx.x == 0) {
      p.work[kWantedAt] = sum;
      p.work[kCountAt] = 0;
    }
  }
  barrier<CTAS>();
  const int wanted = __ldcg(p.work + kWantedAt);
  const int2 free_sum = sums_of<CTAS>(free_of, warp);
  const bool enough = wanted <= free_sum.y;
  // the free pages that are taken, in order
  if (enough && free_here && free_sum.x < wanted) {
    int at = free_sum.x;
    walk(p.refs, pages, [&](int page, int c) {
      const unsigned mask = __ballot_sync(~0u, c == 0);
      const int to = at + lanes_below(mask);
      if (c == 0 && to < wanted) list[to] = page;
      at += __popc(mask);
    });
  }
  barrier<CTAS>();
  if (!leads) return;
  if (!enough && threadIdx.x == 0) raise(p.status, KVX_FLAG_NO_PAGES);
  int at = 0;
  for (int w = 0; w < in; ++w) at += needs_of[w];
  entries([&](Entry &e) {
    const bool need = e.at && e.value < 0;
    const unsigned mask = __ballot_sync(~0u, need);
    const int old = -(e.value + 2);            // -1: none
    int page = -1;
    if (need && enough) {
      page = __ldcg(list + at + lanes_below(mask));
      *e.at = page;
      p.refs[page] = 1;
    } else if (need && old >= 0) {             // as it was
      atomicAdd(p.refs + old, 1);
      *e.at = old;
    }
    at += __popc(mask);
    if (e.first && e.row >= 0) {
      const bool copied = page >= 0 && old >= 0 && !e.whole;
      if (copied) {          // in any order: pages are copied to once
        int32_t *to = p.work + pairs_at(p.num_blocks) + 2 * (int64_t)atomicAdd(p.work + kCountAt, 1);
        to[0] = old;
        to[1] = page;
      }
      if (p.copies) {
        p.copies[2 * (int64_t)e.row] = copied ? old : -1;
        p.copies[2 * (int64_t)e.row + 1] = copied ? page : -1;
      }
    }
  });
}

struct CompactParams {
  int32_t *refs;
  int64_t num_blocks;
  int32_t *used, *moved, *work;
};
template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ CompactParams p) {
  wait_for_kernel_before();
  let_next_kernel_start();
  const int lane = threadIdx.x % 32, warp = blockIdx.x * kWarps + threadIdx.x / 32;
  int32_t *held_of = p.work, *holes_of = p.work + kSums, *movers_of = p.work + 2 * kSums, *pairs = p.work + kListAt;
  const Range pages = share_of<CTAS>(p.num_blocks, 32);
  int held = 0;
  walk(p.refs, pages, [&](int page, int c) { held += __popc(__ballot_sync(~0u, page < pages.end && c != 0)); });
  if (lane == 0) held_of[warp] = held;
  barrier<CTAS>();
  const int used = sums_of<CTAS>(held_of, 0).y;
  int holes = 0, movers = 0;
  walk(p.refs, pages, [&](int page, int c) {
    const bool in = page < pages.end;
    holes += __popc(__ballot_sync(~0u, in && c == 0 && page < used));
    movers += __popc(__ballot_sync(~0u, in && c != 0 && page >= used));
    if (in) p.moved[page] = c != 0 ? page : -1;
  });
  if (lane == 0) {
    holes_of[warp] = holes;
    movers_of[warp] = movers;
  }
  barrier<CTAS>();
  int hole_at = sums_of<CTAS>(holes_of, warp).x;
  const int2 mover_sum = sums_of<CTAS>(movers_of, warp);
  int mover_at = mover_sum.x;
  if (holes || movers)
    walk(p.refs, pages, [&](int page, int c) {
      const bool in = page < pages.end, hole = in && c == 0 && page < used, mover = in && c != 0 && page >= used;
      const unsigned hs = __ballot_sync(~0u, hole), ms = __ballot_sync(~0u, mover);
      if (hole) pairs[2 * (hole_at + lanes_below(hs)) + 1] = page;
      if (mover) pairs[2 * (mover_at + lanes_below(ms))] = page;
      hole_at += __popc(hs);
      mover_at += __popc(ms);
    });
  barrier<CTAS>();
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < mover_sum.y; i += CTAS * kThreads) {
    const int from = __ldcg(pairs + 2 * i), to = __ldcg(pairs + 2 * i + 1);
    p.moved[from] = to;
    p.refs[to] = __ldcg(p.refs + from);
    p.refs[from] = 0;
  }
  if (warp == 0 && lane == 0) {
    p.work[kCountAt] = mover_sum.y;
    *p.used = used;
  }
}
// --- host ------------------------------------------------------------------------

// One CTA for a small pool, a cluster of eight for more.
constexpr int64_t kSmallPool = 8192;
// pages, and slots of a row, are counted in 32 bits, a little beyond the last one too
constexpr int64_t kMostPages = INT32_MAX - 1024, kMostSlots = INT32_MAX - 1024;
constexpr int64_t kMostEntries = (int64_t)1 << 60;   // of a table: their bytes are counted in 64 bits
template <class P>
kvx_status launch_counting(void (*one)(P), void (*many)(P), const P &p, cudaStream_t s) {
  if (p.num_blocks <= kSmallPool) return launch_after(one, dim3(1), kThreads, 0, s, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBigCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBigCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, many, p) == cudaSuccess ? KVX_OK : KVX_ERR_CUDA;
}
// 32-bit words: all given lie on their boundaries.
template <class... P>
bool words_ok(P... p) {
  return (aligned_to(p, 4) && ...);
}
bool pool_ok(const int32_t *refs, int64_t num_blocks) {
  return refs && aligned_to(refs, 4) && num_blocks >= 1 && num_blocks <= kMostPages;
}
bool workspace_ok(const void *ws, size_t bytes, int64_t num_blocks) {
  return ws && aligned_to(ws, 256) && bytes >= kvx_pages_workspace_bytes(num_blocks);
}

}  // namespace

extern "C" size_t kvx_pages_workspace_bytes(int64_t num_blocks) {
  if (num_blocks < 1 || num_blocks > kMostPages) return 0;
  return (size_t)(pairs_at(num_blocks) + 2 * num_blocks) * 4;
}

extern "C" kvx_status kvx_cache8_copy(const kvx_cache8_copy_args *a, void *stream) {
  if (!a || a->num_pairs < 0 || (a->num_pairs > 0 && !a->pairs) || !words_ok(a->pairs, a->count, a->status)) return KVX_ERR_INVALID_ARG;
  if (a->num_caches < 0 || (a->num_caches > 0 && !a->caches)) return KVX_ERR_INVALID_ARG;
  if (a->num_caches == 0) return KVX_OK;
  const int64_t num_blocks = a->caches[0].num_blocks;
  if (const kvx_status st = check_caches(a->caches, a->num_caches, num_blocks, 0)) return st;
  return copy_pages(a->caches, a->num_caches, num_blocks, a->pairs, a->num_pairs, a->count, Tables{}, a->status, (cudaStream_t)stream);
}

extern "C" kvx_status kvx_pages_fork(const kvx_pages_fork_args *a, void *stream) {
  if (!a || !pool_ok(a->refs, a->num_blocks) || a->block_size < 1 || a->block_size > 1024 || a->num_rows < 0 || a->width < 1 ||
      a->num_new < 0 || (a->num_rows > 0 && (!a->table || !a->lens)) ||
      (a->num_new > 0 && (!a->parents || !a->new_table || !a->new_lens)) || (int64_t)a->width * a->block_size > kMostSlots ||
      !words_ok(a->table, a->lens, a->parents, a->new_table, a->new_lens, a->status))
    return KVX_ERR_INVALID_ARG;
  // new rows are written while other CTAs still read the old ones
  const int64_t old_words = (int64_t)a->num_rows * a->width, new_words = (int64_t)a->num_new * a->width;
  if (overlap(a->table, old_words, a->new_table, new_words) || overlap(a->lens, a->num_rows, a->new_lens, a->num_new) ||
      overlap(a->parents, a->num_new, a->new_table, new_words) || overlap(a->parents, a->num_new, a->new_lens, a->num_new))
    return KVX_ERR_INVALID_ARG;
  const int64_t ctas = (int64_t)a->num_new + a->num_rows;
  if (ctas == 0) return KVX_OK;
  if (ctas > INT32_MAX) return KVX_ERR_UNSUPPORTED;
  ForkParams p = {a->refs,      a->num_blocks, a->table,      a->lens,     a->parents, a->new_table,
                  a->new_lens,  a->status,     a->block_size, a->num_rows, a->num_new, a->width};
  return launch_after(fork_kernel, dim3((unsigned)ctas), 128, 0, (cudaStream_t)stream, p);
}

extern "C" kvx_status kvx_pages_free(const kvx_pages_free_args *a, void *stream) {
  if (!a || !pool_ok(a->refs, a->num_blocks) || a->num_rows < 0 || a->width < 1 || (a->num_rows > 0 && !a->table) || !words_ok(a->table, a->status))
    return KVX_ERR_INVALID_ARG;
  const int64_t entries = (int64_t)a->num_rows * a->width;
  if (entries == 0) return KVX_OK;
  const int64_t ctas = (entries + 255) / 256;
  return launch_after(free_kernel, dim3((unsigned)(ctas < 152 * 8 ? ctas : 152 * 8)), 256, 0, (cudaStream_t)stream, a->refs,
                      a->num_blocks, a->table, entries, a->status);
}

extern "C" kvx_status kvx_pages_reserve(const kvx_pages_reserve_args *a, void *stream) {
  if (!a || !pool_ok(a->refs, a->num_blocks) || a->block_size < 1 || a->block_size > 1024 || a->num_rows < 0 || a->width < 1 ||
      a->add_all < 0 || (int64_t)a->width * a->block_size > kMostSlots || !words_ok(a->table, a->lens, a->add, a->copies, a->status))
    return KVX_ERR_INVALID_ARG;
  if (const kvx_status st = check_caches(a->caches, a->num_caches, a->num_blocks, a->block_size)) return st;
  if (a->num_rows == 0) return KVX_OK;
  if ((int64_t)a->num_rows * a->width > INT32_MAX) return KVX_ERR_UNSUPPORTED;   // needs are counted in 32 bits
  if (!a->table || !a->lens || !workspace_ok(a->workspace, a->workspace_bytes, a->num_blocks))
    return KVX_ERR_INVALID_ARG;
  ReserveParams p = {a->refs, a->num_blocks, a->table,      a->copies,   (int32_t *)a->workspace, a->lens,
                     a->add,  a->status,     a->block_size, a->num_rows, a->width,                a->add_all};
  // entries of a row at most, lanes for them, and rows for the warps
  const int64_t asked = ((int64_t)a->add_all + a->block_size - 1) / a->block_size + 1, per = asked < a->width ? asked : a->width;
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < per) p.lanes *= 2;
  p.chunks = (int)((per + 31) / 32);
  const int at_once = 32 / p.lanes;
  p.rows = (int)(((int64_t)a->num_rows + kWarps * at_once - 1) / (kWarps * at_once)) * at_once;
  cudaStream_t s = (cudaStream_t)stream;
  if (const kvx_status st = launch_counting(reserve_kernel<1>, reserve_kernel<kBigCtas>, p, s)) return st;
  if (a->num_caches == 0) return KVX_OK;
  const int64_t most = a->num_rows < a->num_blocks ? a->num_rows : a->num_blocks;
  return copy_pages(a->caches, a->num_caches, a->num_blocks, p.work + pairs_at(a->num_blocks), most, p.work + kCountAt, Tables{}, a->status, s);
}

extern "C" kvx_status kvx_pages_compact(const kvx_pages_compact_args *a, void *stream) {
  if (!a || !pool_ok(a->refs, a->num_blocks) || a->block_size < 1 || a->block_size > 1024 || a->num_tables < 0 ||
      a->num_tables > kMaxTables || (a->num_tables > 0 && (!a->tables || !a->entries)) || !a->used || !a->moved ||
      !words_ok(a->used, a->moved, a->status))
    return KVX_ERR_INVALID_ARG;
  if (const kvx_status st = check_caches(a->caches, a->num_caches, a->num_blocks, a->block_size)) return st;
  if (!workspace_ok(a->workspace, a->workspace_bytes, a->num_blocks)) return KVX_ERR_INVALID_ARG;
  Tables t = {};
  for (int i = 0; i < a->num_tables; ++i) {
    if (a->entries[i] < 0 || a->entries[i] > kMostEntries || (a->entries[i] > 0 && (!a->tables[i] || !aligned_to(a->tables[i], 4))))
      return KVX_ERR_INVALID_ARG;
    // an entry is rewritten once: its new number may be another page's old one
    for (int j = 0; j < i; ++j)
      if (overlap(a->tables[j], a->entries[j], a->tables[i], a->entries[i])) return KVX_ERR_INVALID_ARG;
    t.table[i] = a->tables[i];
    t.entries[i] = a->entries[i];
  }
  t.moved = a->moved;
  t.count = a->num_tables;
  int32_t *work = (int32_t *)a->workspace;
  const CompactParams p = {a->refs, a->num_blocks, a->used, a->moved, work};
  cudaStream_t s = (cudaStream_t)stream;
  if (const kvx_status st = launch_counting(compact_kernel<1>, compact_kernel<kBigCtas>, p, s)) return st;
  return copy_pages(a->caches, a->num_caches, a->num_blocks, work + kListAt, a->num_blocks / 2, work + kCountAt, t, a->status, s);
}
