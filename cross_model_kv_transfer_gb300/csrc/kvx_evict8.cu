// kvx_evict8.cu -- eviction from the 8-bit paged cache by accumulated attention
// weight (kvx_evict8): which slots of each request and head stay, and their
// move into fresh blocks.
//
// Selection.  The weights' bits, made monotone, are 32-bit keys; the need-th
// largest key of the slots that may go is found eleven bits at a time from
// histograms.  What is above it stays, and of its equals the first ones.  A
// cluster of CTAs works on one request and head, each on its slots, with their
// histograms added up through distributed shared memory: a chain of short steps,
// bound by their latency (16 requests of up to 16,384 slots, 8 heads: 21 us, of
// which the weights' bytes would be 0.7).  With one CTA for each the call takes 76 us
// instead of 72, and one request of 131,072 slots, 32,768 kept, 228 instead of 63.
//
// Move.  A block's tokens are read as code * scale, and the block gets the
// smallest power of two as scale that its tokens allow.  Bound by HBM: every
// kept row is read once and written once, and stays in registers between the
// maximum and its new code.  The same batch with 4096 slots kept: 47 us, 5.3 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMoveWarps = 4;
// Of a CTA, in shared memory (two CTAs an SM); more are read again from L2: the batch
// above then takes 80 us instead of 72.
constexpr int kMaxKeys = 22 * 1024;
constexpr int kBins = 2048;
constexpr int kMaxCtas = 8;         // of a cluster
constexpr int kSlotsEach = 4096;

struct EvictParams {
  uint8_t *codes[2];
  float *scale[2];
  const int32_t *table, *dst_table, *lens;
  const float *weights;
  int32_t *kept, *new_lens;
  float *kept_weights;
  uint32_t *status;
  int64_t num_blocks, wstride;
  int R, H, d, bs, max_blocks, max_dst, max_len, keep, sinks, recent, key_cap;
};

__device__ __forceinline__ int evict_len(const EvictParams &p, int r) {
  const int n = __ldg(p.lens + r);
  return n < 0 || n > p.max_len ? 0 : n;
}

// Order-preserving bits of a weight: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Its weight again; not for key 0.
__device__ __forceinline__ float weight_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ int warp_scan(int v) {   // inclusive
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The CTAs that work on one request and head are a cluster.
__device__ __forceinline__ int cluster_rank() {
  uint32_t v;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
  return (int)v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t shared_of(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 load4_of(const void *p, int rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(shared_of(p, rank)));
  return v;
}
__device__ __forceinline__ int load_of(const void *p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(shared_of(p, rank)));
  return v;
}

struct __align__(16) Shared {
  // One for each digit: no CTA clears what another still reads.  The first digit is
  // counted in all three, by lane, because its few bins (a sign, an exponent, two
  // bits) are what lanes collide in; equal bins lie in different banks.
  int hist[3][kBins + 8];
  int sums[kWarps][2];
  int sure, ties;         // the CTA's
  int bin, left, count;
};

// The least `threshold` above which at most `need` keys of the cluster's slots that
// may go lie, and how many of its equals complete them.  This CTA looks at slots
// [lo, hi), whose keys are key(j).
template <typename Key>
__device__ int select_key(Shared &sh, int lo, int hi, int need, int ctas, uint32_t &threshold, const Key &key) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  static_assert(kBins == 4 * kThreads, "four bins a thread");
  for (int i = tid; i < 3 * (kBins + 8); i += kThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
    const uint32_t digit = (1u << bits) - 1;
    int *hist = sh.hist[pass];
    if (pass == 0) {
      int *copy = sh.hist[lane % 3];
#pragma unroll 8
      for (int j = lo + tid; j < hi; j += kThreads) atomicAdd(&copy[key(j) >> shift], 1);
      __syncthreads();
      int4 *one = reinterpret_cast<int4 *>(hist) + tid;
      int4 *two = reinterpret_cast<int4 *>(sh.hist[1]) + tid, *three = reinterpret_cast<int4 *>(sh.hist[2]) + tid;
      const int4 x = *one, y = *two, z = *three;
      *one = make_int4(x.x + y.x + z.x, x.y + y.y + z.y, x.z + y.z + z.z, x.w + y.w + z.w);
      *two = *three = make_int4(0, 0, 0, 0);
    } else {
#pragma unroll 8
      for (int j = lo + tid; j < hi; j += kThreads) {
        const uint32_t k = key(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1);
      }
    }
    cluster_sync();
    // thread t: the four bins that end t fours below the highest
    const int4 *four = reinterpret_cast<const int4 *>(hist) + (kThreads - 1 - tid);
    int4 n = make_int4(0, 0, 0, 0);
    for (int c = 0; c < ctas; ++c) {
      const int4 x = load4_of(four, c);
      n = make_int4(n.x + x.x, n.y + x.y, n.z + x.z, n.w + x.w);
    }
    const int mine = n.x + n.y + n.z + n.w, upto = warp_scan(mine);
    if (lane == 31) sh.sums[warp][0] = upto;
    __syncthreads();
    int above = upto - mine;
    for (int w = 0; w < warp; ++w) above += sh.sums[w][0];
    if (above < need && above + mine >= need) {
      const int of[4] = {n.w, n.z, n.y, n.x};
      bool done = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!done && above + of[i] >= need) {
          sh.bin = kBins - 1 - 4 * tid - i;
          sh.left = need - above;
          sh.count = of[i];
          done = true;
        }
        above += of[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh.bin << shift;
    mask |= digit << shift;
    need = sh.left;
    if (need == sh.count && prefix) {   // the whole bin stays: no need to look into it
      threshold = prefix - 1;
      return 0;
    }
  }
  threshold = prefix;
  return need;
}

// Lists, from entry `out` on and in order, which of the cluster's slots that may go
// stay: those above the threshold and its first `need` equals.  A warp looks after
// consecutive slots of the CTA's [beg, end).
template <typename Key>
__device__ void list_kept(Shared &sh, int beg, int end, uint32_t threshold, int need, int out, const float *w,
                          int32_t *kept, float *kept_w, const Key &key) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int each = end > beg ? (end - beg + 32 * kWarps - 1) / (32 * kWarps) * 32 : 0;
  beg += warp * each;
  end = beg + each < end ? beg + each : end;
  const unsigned before = (1u << lane) - 1;
  int nsure = 0, nties = 0;
#pragma unroll 4
  for (int j0 = beg; j0 < end; j0 += 32) {
    const bool mine = j0 + lane < end;
    const uint32_t k = mine ? key(j0 + lane) : 0u;
    nsure += __popc(__ballot_sync(~0u, k > threshold));
    nties += __popc(__ballot_sync(~0u, mine && k == threshold));
  }
  if (lane == 0) {
    sh.sums[warp][0] = nsure;
    sh.sums[warp][1] = nties;
  }
  __syncthreads();
  int ties = 0, all_sure = 0, all_ties = 0;
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    if (v == warp) out += all_sure, ties = all_ties;
    all_sure += sh.sums[v][0];
    all_ties += sh.sums[v][1];
  }
  if (threadIdx.x == 0) sh.sure = all_sure, sh.ties = all_ties;
  cluster_sync();
  for (int c = cluster_rank() - 1; c >= 0; --c) {
    out += load_of(&sh.sure, c);
    ties += load_of(&sh.ties, c);
  }
  out += ties < need ? ties : need;
#pragma unroll 4
  for (int j0 = beg; j0 < end; j0 += 32) {
    const bool mine = j0 + lane < end;
    const uint32_t k = mine ? key(j0 + lane) : 0u;
    const unsigned tied = __ballot_sync(~0u, mine && k == threshold);
    const bool stays = k > threshold || (mine && k == threshold && ties + __popc(tied & before) < need);
    const unsigned all = __ballot_sync(~0u, stays);
    if (stays) {
      const int at = out + __popc(all & before);
      kept[at] = j0 + lane;
      if (kept_w) kept_w[at] = k ? weight_of(k) : __ldg(w + j0 + lane);
    }
    ties += __popc(tied);
    out += __popc(all);
  }
}

// A warp moves one block of one head: keys and values of up to four slots a lane stay
// in registers between the maximum and the new codes; a longer block is read again
// (with two slots a lane, which makes blocks of 16 x 128 such longer ones, a call of
// the batch above took 123 us where it took 99).
struct Moved {
  uint4 x[2];
  float scale[2];
};
__device__ __forceinline__ void fetch(const EvictParams &p, int r, int h, int part, int j, Moved &t) {
  const int b = j / p.bs;
  const int64_t from = b < p.max_blocks ? (int64_t)__ldg(p.table + (int64_t)r * p.max_blocks + b) : -1;
  if (from < 0 || from >= p.num_blocks) {
    raise(p.status, KVX_FLAG_BAD_BLOCK);
    t.x[0] = t.x[1] = make_uint4(0, 0, 0, 0);
    t.scale[0] = t.scale[1] = 0.f;
    return;
  }
  const int64_t at = from * p.H + h, code = (at * p.bs + j % p.bs) * p.d + part * 16;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    t.x[m] = __ldcs(reinterpret_cast<const uint4 *>(p.codes[m] + code));
    t.scale[m] = p.scale[m][at];
  }
}
__device__ __forceinline__ float largest(const uint4 &t, float scale) {
  const uint32_t most = __vmaxu4(__vmaxu4(t.x & 0x7f7f7f7fu, t.y & 0x7f7f7f7fu),
                                 __vmaxu4(t.z & 0x7f7f7f7fu, t.w & 0x7f7f7f7fu));
  const float2 a = floats_of(most), b = floats_of(most >> 16);
  return fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)) * scale;
}
__device__ __forceinline__ uint4 rescaled(const uint4 &t, float f) {
  // An infinite factor is that of zeros beside a large value in their old block and none
  // in the new one (a code that is none keeps it below 2^18): they stay as they are.
  if (f == 1.f || f == INFINITY) return t;
  uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = floats_of(w[e]), b = floats_of(w[e] >> 16);
    w[e] = e4m3x2(a.x * f, a.y * f) | e4m3x2(b.x * f, b.y * f) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ void move_block(const EvictParams &p, int r, int h, int64_t page, const int32_t *kept, int rows) {
  const int lane = threadIdx.x % 32, per_row = p.d / 16, side = 32 / per_row, part = lane % per_row;
  const int mine = lane < side * per_row ? lane / per_row : rows;
  constexpr int kHeld = 4;
  Moved held[kHeld];
  const bool holds = rows <= kHeld * side;   // of the whole warp
  float amax[2] = {0.f, 0.f};
  if (holds) {
    int j[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) j[k] = mine + k * side < rows ? kept[mine + k * side] : -1;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (j[k] >= 0) fetch(p, r, h, part, j[k], held[k]);
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (j[k] >= 0)
#pragma unroll
        for (int m = 0; m < 2; ++m) amax[m] = fmaxf(amax[m], largest(held[k].x[m], held[k].scale[m]));
  } else {
    for (int i = mine; i < rows; i += side) {
      Moved t;
      fetch(p, r, h, part, kept[i], t);
#pragma unroll
      for (int m = 0; m < 2; ++m) amax[m] = fmaxf(amax[m], largest(t.x[m], t.scale[m]));
    }
  }
  float f[2];
  const int64_t at = page * p.H + h;
#pragma unroll
  for (int m = 0; m < 2; ++m) {   // not negative: ordered as their bits are
    const float now = pow2_scale(__uint_as_float(__reduce_max_sync(~0u, __float_as_uint(amax[m]))));
    if (lane == 0) p.scale[m][at] = now;
    f[m] = 1.f / now;
  }
  const int64_t to = at * p.bs * p.d + part * 16;
  const auto store = [&](int i, const Moved &t) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
      __stcs(reinterpret_cast<uint4 *>(p.codes[m] + to + (int64_t)i * p.d), rescaled(t.x[m], t.scale[m] * f[m]));
  };
  if (holds) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (mine + k * side < rows) store(mine + k * side, held[k]);
  } else {
    for (int i = mine; i < rows; i += side) {
      Moved t;
      fetch(p, r, h, part, kept[i], t);
      store(i, t);
    }
  }
}

// Selects for request r's head h and lists what it keeps; returns how many slots
// that is.  Every CTA of the cluster calls it.
__device__ int select_and_list(const EvictParams &p, int r, int h, Shared &sh, uint32_t *keys) {
  const int tid = threadIdx.x, rank = cluster_rank(), ctas = gridDim.x;
  const int len = evict_len(p, r), n = len < p.keep ? len : p.keep;
  if (rank == 0 && h == 0 && tid == 0) {
    p.new_lens[r] = n;
    if (len != __ldg(p.lens + r)) raise(p.status, KVX_FLAG_BAD_LENGTH);
  }
  const int64_t row = (int64_t)r * p.H + h;
  const float *w = p.weights + row * p.wstride;
  int32_t *kept = p.kept + row * p.keep;
  float *kept_w = p.kept_weights ? p.kept_weights + row * p.keep : nullptr;
  // entry i of the list, where which slot that is needs no selection
  const auto plain = [&](int i, int slot) {
    kept[i] = slot;
    if (kept_w) kept_w[i] = slot < 0 ? 0.f : w[slot];
  };
  const int t0 = rank * kThreads + tid, threads = ctas * kThreads;
  for (int64_t i = (int64_t)n + t0; i < p.keep; i += threads) plain((int)i, -1);
  if (len <= p.keep) {
    for (int64_t i = t0; i < n; i += threads) plain((int)i, (int)i);
    return n;
  }
  const int lo = p.sinks, hi = len - p.recent;   // slots that may go
  for (int64_t i = t0; i < lo; i += threads) plain((int)i, (int)i);
  for (int64_t i = t0; i < p.recent; i += threads) plain(p.keep - p.recent + (int)i, hi + (int)i);
  int need = p.keep - p.sinks - p.recent;        // of them, how many stay
  if (need == 0) return n;
  const int each = (hi - lo + ctas - 1) / ctas;  // slots of a CTA
  const int beg = hi - lo - rank * each > 0 ? lo + rank * each : hi, end = hi - beg < each ? hi : beg + each;
  uint32_t threshold = 0;
  const auto list = [&](const auto &key) {
    need = select_key(sh, beg, end, need, ctas, threshold, key);
    __syncthreads();
    list_kept(sh, beg, end, threshold, need, lo, w, kept, kept_w, key);
  };
  if (each <= p.key_cap) {
#pragma unroll 8
    for (int j = beg + tid; j < end; j += kThreads) keys[j - beg] = key_of(w[j]);
    list([&](int j) { return keys[j - beg]; });   // a thread's own keys until the first barrier
  } else {
    list([&](int j) { return key_of(__ldg(w + j)); });
  }
  return n;
}

__device__ __forceinline__ void move_dst_block(const EvictParams &p, int r, int h, int b, int n) {
  const int64_t page = b < p.max_dst ? (int64_t)__ldg(p.dst_table + (int64_t)r * p.max_dst + b) : -1;
  if (page < 0 || page >= p.num_blocks) {
    if (threadIdx.x % 32 == 0) raise(p.status, KVX_FLAG_BAD_BLOCK);
    return;
  }
  const int rows = n - b * p.bs < p.bs ? n - b * p.bs : p.bs;
  move_block(p, r, h, page, p.kept + ((int64_t)r * p.H + h) * p.keep + b * p.bs, rows);
}

// Grid: x = the CTAs of a cluster, y = heads, z = requests.
template <bool MOVE>
__global__ void __launch_bounds__(kThreads, MOVE ? 1 : 2) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ Shared sh;
  extern __shared__ uint32_t keys[];
  const int h = blockIdx.y, r = blockIdx.z;
  const int n = select_and_list(p, r, h, sh, keys);
  cluster_sync();   // the list is whole, and no CTA's shared memory is read any more
  if constexpr (MOVE)
    for (int b = threadIdx.x / 32 * gridDim.x + blockIdx.x; (int64_t)b * p.bs < n; b += kWarps * gridDim.x)
      move_dst_block(p, r, h, b, n);
}

// Many: the moves by a kernel of their own, with a warp for each block.
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(const __grid_constant__ EvictParams p) {
  const int h = blockIdx.y, r = blockIdx.z, b = blockIdx.x * kMoveWarps + threadIdx.x / 32;
  const int len = evict_len(p, r), n = len < p.keep ? len : p.keep;
  wait_for_kernel_before();
  if ((int64_t)b * p.bs < n) move_dst_block(p, r, h, b, n);
}

kvx_status check(const kvx_evict8_args *a) {
  if (!a) return KVX_ERR_INVALID_ARG;
  if (const kvx_status st = check_cache8(a->cache)) return st;
  if (!a->dst_table || a->num_requests < 1 || a->num_requests > 65535 || !a->lens || a->max_len < 0 ||
      a->max_len > INT32_MAX - 1024 ||
      a->keep < 1 || a->sinks < 0 || a->recent < 0 || (int64_t)a->sinks + a->recent > a->keep ||
      !a->weights || a->weights_stride < a->max_len || !a->kept || !a->new_lens)
    return KVX_ERR_INVALID_ARG;
  const int64_t most = a->keep < a->max_len ? a->keep : a->max_len;
  if (a->max_dst_blocks < (most + a->cache.block_size - 1) / a->cache.block_size) return KVX_ERR_INVALID_ARG;
  return KVX_OK;
}

}  // namespace

extern "C" size_t kvx_evict8_workspace_bytes(const kvx_evict8_args *a) {
  return check(a) == KVX_OK ? 256 : 0;
}

extern "C" kvx_status kvx_evict8(const kvx_evict8_args *a, void *stream) {
  if (const kvx_status st = check(a)) return st;
  if (!a->workspace || !aligned_to(a->workspace, 256) || a->workspace_bytes < kvx_evict8_workspace_bytes(a))
    return KVX_ERR_INVALID_ARG;
  const kvx_cache8 &c = a->cache;
  // results are written while other CTAs still read lengths and weights
  const int64_t lists = (int64_t)a->num_requests * c.heads;
  if (overlap(a->lens, a->num_requests, a->new_lens, a->num_requests) ||
      (a->kept_weights && a->max_len > 0 &&
       overlap(a->weights, (lists - 1) * a->weights_stride + a->max_len, a->kept_weights, lists * a->keep)))
    return KVX_ERR_INVALID_ARG;
  EvictParams p;
  p.codes[0] = (uint8_t *)c.k_codes;
  p.codes[1] = (uint8_t *)c.v_codes;
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.table = c.block_table;
  p.dst_table = a->dst_table;
  p.lens = a->lens;
  p.weights = a->weights;
  p.kept = a->kept;
  p.new_lens = a->new_lens;
  p.kept_weights = a->kept_weights;
  p.status = a->status;
  p.num_blocks = c.num_blocks;
  p.wstride = a->weights_stride;
  p.R = a->num_requests;
  p.H = c.heads;
  p.d = c.head_dim;
  p.bs = c.block_size;
  p.max_blocks = c.max_blocks_per_req;
  p.max_dst = a->max_dst_blocks;
  p.max_len = a->max_len;
  p.keep = a->keep;
  p.sinks = a->sinks;
  p.recent = a->recent;
  const int64_t most = a->keep < a->max_len ? a->keep : a->max_len;
  const int64_t blocks = (most + c.block_size - 1) / c.block_size, rows = (int64_t)c.heads * a->num_requests;
  // One launch where no warp would move more than a block: 18.4 us for 512 of 2048
  // slots and 8 heads where two launches take 19.1, and a launch less of the host's
  // time; with 4096 slots kept of 16,384 one takes 30.7 us and two 27.5, for four
  // requests 56 and 36.
  const bool few = rows <= 152 / kMaxCtas && blocks <= kMaxCtas * kWarps;
  // CTAs of a request and head: one for 4096 slots, while all fit the GPU at once;
  // where the selection moves the slots too, one for as many blocks as it has warps
  int ctas = 1;
  while (ctas < kMaxCtas && 2 * ctas * rows <= 2 * 152 &&
         ((int64_t)ctas * kSlotsEach < a->max_len || (few && ctas * kWarps < blocks)))
    ctas *= 2;
  const int each = (a->max_len + ctas - 1) / ctas;
  p.key_cap = each < kMaxKeys ? each : kMaxKeys;
  const size_t smem = (size_t)p.key_cap * 4;
  const auto kernel = few ? select_kernel<true> : select_kernel<false>;
  // the same for every call: the attribute is the kernel's, which calls from other
  // host threads share, not this launch's
  if (sizeof(Shared) + smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4) != cudaSuccess)
    return KVX_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, c.heads, a->num_requests);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return KVX_ERR_CUDA;
  if (few || blocks == 0) return KVX_OK;
  return launch_after(move_kernel, dim3((unsigned)((blocks + kMoveWarps - 1) / kMoveWarps), c.heads, a->num_requests),
                      32 * kMoveWarps, 0, cfg.stream, p);
}
