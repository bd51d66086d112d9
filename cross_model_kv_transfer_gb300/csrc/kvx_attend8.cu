// kvx_attend8.cu -- attention of new tokens over the 8-bit paged cache
// (kvx_attend8), and the attention weight that each slot receives.
//
//   out_i = sum_j exp(x_ij - lse_i) v_j,  x_ij = scale q_i . k_j,
//   lse_i = log sum_j exp(x_ij),          j <= len - new + i.
// One pass over the slots with a running maximum and sum (fp32): when a larger
// score arrives, what was summed is scaled down to it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvx_cache8.cuh"

namespace {

constexpr int kMaxD = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendParams {
  const uint8_t *k, *v;
  const float *ks, *vs;
  const void *q;
  void *out;
  int64_t qt, qh, ot, oh;
  const int32_t *table, *lens;
  float *lse, *weights;
  uint32_t *status;
  Requests req;
  int64_t num_blocks, wstride;
  int H, Hq, G, d, bs, max_blocks, max_len, max_new, bf16;
  float c;   // scale * log2(e): scores are kept in base 2
};

// The request's length (0 where it is out of bounds).
__device__ __forceinline__ int len_of(const AttendParams &p, int r) {
  const int n = __ldg(p.lens + r);
  return n < 0 || n > p.max_len ? 0 : n;
}
// The pool's block of slot j, or -1.
__device__ __forceinline__ int64_t page_of(const AttendParams &p, int r, int64_t block) {
  const int64_t page = block < p.max_blocks ? (int64_t)__ldg(p.table + (int64_t)r * p.max_blocks + block) : -1;
  return page >= 0 && page < p.num_blocks ? page : -1;
}
__device__ __forceinline__ float q_at(const AttendParams &p, int64_t g, int h, int i) {
  const int64_t at = g * p.qt + h * p.qh + i;
  return p.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.q)[at])
                : reinterpret_cast<const float *>(p.q)[at];
}
__device__ __forceinline__ bool requests_ok(const AttendParams &p) {
  bool good = p.req.ok();
  if (p.req.cu) {
    bool few = true;
    for (int r = threadIdx.x; good && r < p.req.R; r += blockDim.x)
      few = few && p.req.cu[r + 1] - p.req.cu[r] <= p.max_new;
    good = __syncthreads_and(good && few);
  }
  return good;
}
// q . k_j of one slot.
__device__ __forceinline__ float dot_row(const uint8_t *row, const float *q, int d) {
  float s = 0.f;
  for (int i = 0; i < d; i += 16) {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(row + i));
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = floats_of(w[e]), b = floats_of(w[e] >> 16);
      s += q[i + 4 * e] * a.x + q[i + 4 * e + 1] * a.y + q[i + 4 * e + 2] * b.x + q[i + 4 * e + 3] * b.y;
    }
  }
  return s;
}

// One warp for each query and head: 32 slots at a time, a lane each, then the
// lanes share the value dimensions.
__global__ void __launch_bounds__(128) attend_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float qs[4][kMaxD];
  if (!requests_ok(p)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise(p.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp;
  if (row >= p.req.ntok * p.Hq) return;
  const int64_t g = row / p.Hq;
  const int hq = (int)(row % p.Hq), h = hq / p.G, r = p.req.of(g);
  const int len = len_of(p, r);
  if (len != __ldg(p.lens + r) && lane == 0) raise(p.status, KVX_FLAG_BAD_LENGTH);
  const int64_t n = p.req.begin(r + 1) - p.req.begin(r);
  const int64_t seen = len - n + (g - p.req.begin(r)) + 1;   // slots [0, seen)
  for (int i = lane; i < p.d; i += 32) qs[warp][i] = q_at(p, g, hq, i);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[kMaxD / 32] = {};
  for (int64_t j0 = 0; j0 < seen; j0 += 32) {
    const int64_t j = j0 + lane, page = j < seen ? page_of(p, r, j / p.bs) : -1;
    const int64_t at = page < 0 ? 0 : (page * p.H + h) * p.bs + j % p.bs;
    float x = -INFINITY, sv = 0.f;
    if (page >= 0) {
      x = dot_row(p.k + at * p.d, qs[warp], p.d) * (p.ks[page * p.H + h] * p.c);
      sv = p.vs[page * p.H + h];
    } else if (j < seen) {
      raise(p.status, KVX_FLAG_BAD_BLOCK);
    }
    float top = x;
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
    if (top == -INFINITY) continue;
    const float now = fmaxf(m, top), down = exp2f(m - now);
    const float e = exp2f(x - now);
    float sum = e;
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
    l = l * down + sum;
    m = now;
    for (int i = 0; i < kMaxD / 32; ++i) o[i] *= down;
    for (int k = 0; k < 32; ++k) {
      const int64_t a = __shfl_sync(~0u, at, k);
      const float w = __shfl_sync(~0u, e * sv, k);
      if (w == 0.f) continue;
#pragma unroll
      for (int i = 0; i < kMaxD / 32; ++i)
        if (32 * i + lane < p.d) o[i] += w * floats_of(__ldg(p.v + a * p.d + 32 * i + lane)).x;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) {
    if (32 * i + lane >= p.d) continue;
    const int64_t to = g * p.ot + hq * p.oh + 32 * i + lane;
    if (p.bf16)
      reinterpret_cast<__nv_bfloat16 *>(p.out)[to] = __float2bfloat16_rn(o[i] * inv);
    else
      reinterpret_cast<float *>(p.out)[to] = o[i] * inv;
  }
  if (lane == 0) p.lse[g * p.Hq + hq] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// weights[r][h][j] += sum of p_ij: a thread for each slot, the scores again.
__global__ void __launch_bounds__(128) weights_kernel(const __grid_constant__ AttendParams p) {
  if (!requests_ok(p)) return;
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(p, r);
  const int64_t j = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (j >= len) return;
  const int64_t page = page_of(p, r, j / p.bs);
  if (page < 0) return;
  const int64_t beg = p.req.begin(r), n = p.req.begin(r + 1) - beg;
  const uint8_t *row = p.k + ((page * p.H + h) * p.bs + j % p.bs) * p.d;
  const float ks = p.ks[page * p.H + h] * p.c;
  float sum = 0.f;
  for (int64_t i = j - (len - n) > 0 ? j - (len - n) : 0; i < n; ++i)
    for (int u = 0; u < p.G; ++u) {
      const int hq = h * p.G + u;
      float s = 0.f;
      for (int e = 0; e < p.d; e += 2) {
        const float2 a = floats_of(*reinterpret_cast<const uint16_t *>(row + e));
        s += q_at(p, beg + i, hq, e) * a.x + q_at(p, beg + i, hq, e + 1) * a.y;
      }
      sum += exp2f(s * ks - p.lse[(beg + i) * p.Hq + hq] * kLog2e);
    }
  p.weights[((int64_t)r * p.H + h) * p.wstride + j] += sum;
}

kvx_status check(const kvx_attend8_args *a) {
  if (!a) return KVX_ERR_INVALID_ARG;
  const kvx_cache8 &c = a->cache;
  if (const kvx_status st = check_cache8(c)) return st;
  if ((a->dtype != KVX_F32 && a->dtype != KVX_BF16) || a->num_requests < 1 || a->ntok < 0 ||
      a->ntok > INT32_MAX || (!a->cu_seqlens && a->ntok != a->num_requests) || a->max_new < 1 ||
      a->max_len < 0 || !a->lens || !std::isfinite(a->scale) || a->q_heads < 1 ||
      a->q_heads > 65535 || a->q_heads % c.heads)
    return KVX_ERR_INVALID_ARG;
  if (a->weights && a->weights_stride < a->max_len) return KVX_ERR_INVALID_ARG;
  return KVX_OK;
}

}  // namespace

extern "C" size_t kvx_attend8_workspace_bytes(const kvx_attend8_args *a) {
  if (check(a) != KVX_OK) return 0;
  return 256 + (size_t)a->ntok * a->q_heads * 4;
}

extern "C" kvx_status kvx_attend8(const kvx_attend8_args *a, void *stream) {
  if (const kvx_status st = check(a)) return st;
  if (a->ntok == 0) return KVX_OK;
  const kvx_cache8 &c = a->cache;
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  if (!a->q || !a->out || !aligned_to(a->q, size) || !aligned_to(a->out, size)) return KVX_ERR_INVALID_ARG;
  if (!a->workspace || !aligned_to(a->workspace, 256) || a->workspace_bytes < kvx_attend8_workspace_bytes(a))
    return KVX_ERR_INVALID_ARG;
  AttendParams p;
  p.k = (const uint8_t *)c.k_codes;
  p.v = (const uint8_t *)c.v_codes;
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.q = a->q;
  p.out = a->out;
  p.qt = a->q_token_stride;
  p.qh = a->q_head_stride;
  p.ot = a->out_token_stride;
  p.oh = a->out_head_stride;
  p.table = c.block_table;
  p.lens = a->lens;
  p.lse = a->lse ? a->lse : (float *)((char *)a->workspace + 256);
  p.weights = a->weights;
  p.status = a->status;
  p.req = {a->cu_seqlens, a->num_requests, a->ntok};
  p.num_blocks = c.num_blocks;
  p.wstride = a->weights_stride;
  p.H = c.heads;
  p.Hq = a->q_heads;
  p.G = a->q_heads / c.heads;
  p.d = c.head_dim;
  p.bs = c.block_size;
  p.max_blocks = c.max_blocks_per_req;
  p.max_len = a->max_len;
  p.max_new = a->max_new;
  p.bf16 = size == 2;
  p.c = a->scale * kLog2e;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t rows = a->ntok * a->q_heads;
  attend_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(p);
  if (const kvx_status st = launched()) return st;
  if (!a->weights || a->max_len == 0) return KVX_OK;
  weights_kernel<<<dim3((a->max_len + 127) / 128, c.heads, a->num_requests), 128, 0, s>>>(p);
  return launched();
}
