// kvx_evict8.cu -- eviction from the 8-bit paged cache by accumulated attention
// weight (kvx_evict8): which slots of each request and head stay, and their
// move into fresh blocks.
//
// Selection.  The weights' bits, made monotone, are 32-bit keys; the need-th
// largest key of the slots that may go is found eight bits at a time from
// histograms.  What is above it stays, and of its equals the first ones.
// Move.  A block's tokens are read as code * scale, and the block gets the
// smallest power of two as scale that its tokens allow.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveWarps = 4;

struct EvictParams {
  uint8_t *codes[2];
  float *scale[2];
  const int32_t *table, *dst_table, *lens;
  const float *weights;
  int32_t *kept, *new_lens;
  float *kept_weights;
  uint32_t *status;
  int64_t num_blocks, wstride;
  int R, H, d, bs, max_blocks, max_dst, max_len, keep, sinks, recent;
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

// The CTA's exclusive sum of `v` by thread; `total` is the whole sum.
__device__ __forceinline__ int cta_scan(int v, int *warps, int &total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += y;
    }
    warps[lane] = s;
  }
  __syncthreads();
  total = warps[31];
  const int before = (warp ? warps[warp - 1] : 0) + x - v;
  __syncthreads();
  return before;
}

// One CTA for each request and head.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[256], warps[32];
  __shared__ uint32_t found;
  __shared__ int left;
  const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int len = evict_len(p, r), n = len < p.keep ? len : p.keep;
  if (h == 0 && tid == 0) {
    p.new_lens[r] = n;
    if (len != __ldg(p.lens + r)) raise(p.status, KVX_FLAG_BAD_LENGTH);
  }
  const int64_t row = (int64_t)r * p.H + h;
  const float *w = p.weights + row * p.wstride;
  int32_t *kept = p.kept + row * p.keep;
  float *kept_w = p.kept_weights ? p.kept_weights + row * p.keep : nullptr;
  for (int i = n + tid; i < p.keep; i += kSelThreads) {
    kept[i] = -1;
    if (kept_w) kept_w[i] = 0.f;
  }
  if (len <= p.keep) {
    for (int i = tid; i < n; i += kSelThreads) {
      kept[i] = i;
      if (kept_w) kept_w[i] = w[i];
    }
    return;
  }
  const int lo = p.sinks, hi = len - p.recent;   // slots that may go
  int need = p.keep - p.sinks - p.recent;        // of them, how many stay
  uint32_t prefix = 0, mask = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t k = key_of(w[j]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      // thread b: how many keys lie in bins above b
      int total;
      const int mine = tid < 256 ? hist[255 - tid] : 0, above = cta_scan(mine, warps, total);
      if (tid < 256 && above < need && above + mine >= need) {
        found = 255 - tid;
        left = need - above;
      }
      __syncthreads();
      prefix |= found << shift;
      mask |= 255u << shift;
      need = left;
      __syncthreads();
    }
  }
  // the slots in order: those above the threshold, its first `need` equals, and
  // the ones that always stay
  int out = 0, ties = 0;
  for (int j0 = 0; j0 < len; j0 += kSelThreads) {
    const int j = j0 + tid;
    const bool may = j >= lo && j < hi;
    const uint32_t k = may ? key_of(w[j]) : 0u;
    const bool tie = may && mask && k == prefix;
    int total;
    const int rank = ties + cta_scan(tie, warps, total);
    ties += total;
    const bool stays = j < len && (!may || (mask && (k > prefix || (tie && rank < need))));
    const int at = out + cta_scan(stays, warps, total);
    out += total;
    if (stays) {
      kept[at] = j;
      if (kept_w) kept_w[at] = w[j];
    }
  }
}

// A warp for each destination block, head, and K|V.
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(const __grid_constant__ EvictParams p) {
  const int hm = blockIdx.y * kMoveWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (hm >= 2 * p.H) return;
  const int m = hm / p.H, h = hm % p.H, r = blockIdx.z, block = blockIdx.x;
  const int len = evict_len(p, r), n = len < p.keep ? len : p.keep;
  const int first = block * p.bs, rows = n - first < p.bs ? n - first : p.bs;
  if (rows <= 0) return;
  const int64_t page = block < p.max_dst ? (int64_t)p.dst_table[(int64_t)r * p.max_dst + block] : -1;
  if (page < 0 || page >= p.num_blocks) {
    if (lane == 0) raise(p.status, KVX_FLAG_BAD_BLOCK);
    return;
  }
  const int per_row = p.d / 16, side = 32 / per_row, part = lane % per_row;
  const int mine = lane < side * per_row ? lane / per_row : rows;
  const int32_t *kept = p.kept + ((int64_t)r * p.H + h) * p.keep + first;
  const auto source = [&](int i, float &scale) -> const uint4 * {
    const int j = kept[i], b = j / p.bs;
    const int64_t from = b < p.max_blocks ? (int64_t)p.table[(int64_t)r * p.max_blocks + b] : -1;
    if (from < 0 || from >= p.num_blocks) {
      raise(p.status, KVX_FLAG_BAD_BLOCK);
      return nullptr;
    }
    scale = p.scale[m][from * p.H + h];
    return reinterpret_cast<const uint4 *>(p.codes[m] + ((from * p.H + h) * p.bs + j % p.bs) * (int64_t)p.d +
                                           part * 16);
  };
  float amax = 0.f;
  for (int i = mine; i < rows; i += side) {
    float scale;
    const uint4 *src = source(i, scale);
    if (!src) continue;
    const uint4 t = *src;
    const uint32_t most = __vmaxu4(__vmaxu4(t.x & 0x7f7f7f7fu, t.y & 0x7f7f7f7fu),
                                   __vmaxu4(t.z & 0x7f7f7f7fu, t.w & 0x7f7f7f7fu));
    const float2 a = floats_of(most), b = floats_of(most >> 16);
    amax = fmaxf(amax, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)) * scale);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  const float now = pow2_scale(amax), f = 1.f / now;
  if (lane == 0) p.scale[m][page * p.H + h] = now;
  uint8_t *to = p.codes[m] + (page * p.H + h) * p.bs * (int64_t)p.d + part * 16;
  for (int i = mine; i < rows; i += side) {
    float scale;
    const uint4 *src = source(i, scale);
    const uint4 t = src ? *src : make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {t.x, t.y, t.z, t.w};
    if (src && scale != now) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = floats_of(w[e]), b = floats_of(w[e] >> 16);
        w[e] = e4m3x2(a.x * scale * f, a.y * scale * f) | e4m3x2(b.x * scale * f, b.y * scale * f) << 16;
      }
    }
    *reinterpret_cast<uint4 *>(to + (int64_t)i * p.d) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

kvx_status check(const kvx_evict8_args *a) {
  if (!a) return KVX_ERR_INVALID_ARG;
  if (const kvx_status st = check_cache8(a->cache)) return st;
  if (!a->dst_table || a->num_requests < 1 || a->num_requests > 65535 || !a->lens || a->max_len < 0 ||
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
  cudaStream_t s = (cudaStream_t)stream;
  select_kernel<<<dim3(c.heads, a->num_requests), kSelThreads, 0, s>>>(p);
  if (const kvx_status st = launched()) return st;
  const int64_t most = a->keep < a->max_len ? a->keep : a->max_len;
  if (most == 0) return KVX_OK;
  const dim3 grid((unsigned)((most + c.block_size - 1) / c.block_size),
                  (unsigned)((2 * c.heads + kMoveWarps - 1) / kMoveWarps), a->num_requests);
  move_kernel<<<grid, 32 * kMoveWarps, 0, s>>>(p);
  return launched();
}
