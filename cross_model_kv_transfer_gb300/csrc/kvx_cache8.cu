// kvx_cache8.cu -- the 8-bit paged cache's write (kvx_cache8_write).
//
// For each block and head, separately for keys and values: the scale is the
// smallest power of two that brings the largest new magnitude to 448 or less
// (or the block's own where it already holds tokens and that is larger), and
// code = e4m3(x / scale).  Bound by HBM: the new rows are read once (a warp
// re-reads its few rows from L1 after their maximum is known) and one byte an
// element is written.
//
// A warp quantises one run: the tokens of one request that share a block, for
// one head's keys or values.  Runs are found from the tokens: a unit of
// `per_unit` consecutive tokens looks after the runs that begin in it, so
// neither the host nor a first kernel has to count blocks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

namespace {

constexpr int kWriteWarps = 4;

struct WriteParams {
  uint8_t *codes[2];
  float *scale[2];
  const void *x[2];
  int64_t ts[2], hs[2];       // token and head strides, elements
  const int32_t *table, *start, *src_rows;
  uint32_t *status;
  Requests req;
  int64_t num_blocks, num_src_rows;
  int H, d, bs, max_blocks, per_unit, bf16;
};

// 16 consecutive elements; infinities and NaN leave `amax` alone and raise `odd`.
template <typename T>
__device__ __forceinline__ void load16(const T *p, bool vec, float (&v)[16]) {
  if constexpr (sizeof(T) == 2) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 t = reinterpret_cast<const uint4 *>(p)[i];
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __bfloat162float(p[i]);
    }
  } else {
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = reinterpret_cast<const float4 *>(p)[i];
        v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = p[i];
    }
  }
}

template <typename T>
__device__ void write_run(const WriteParams &p, int m, int h, int64_t page, int s0, int64_t g0, int n,
                          bool vec) {
  const int lane = threadIdx.x % 32, per_row = p.d / 16, rows = 32 / per_row;
  const int part = lane % per_row, mine = lane < rows * per_row ? lane / per_row : p.bs;
  const T *x = reinterpret_cast<const T *>(p.x[m]) + (int64_t)h * p.hs[m] + part * 16;
  uint8_t *to = p.codes[m] + (page * p.H + h) * p.bs * (int64_t)p.d + part * 16;
  const auto source = [&](int i) -> const T * {
    int64_t row = g0 + i;
    if (p.src_rows) {
      row = __ldg(p.src_rows + row);
      if (row < 0 || row >= p.num_src_rows) return nullptr;
    }
    return x + row * p.ts[m];
  };
  float amax = 0.f;
  bool odd = false, lost = false;
  for (int i = mine; i < n; i += rows) {
    const T *src = source(i);
    lost = lost || !src;
    if (!src) continue;
    float v[16];
    load16(src, vec, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float a = fabsf(v[e]);
      if (a < INFINITY) amax = fmaxf(amax, a); else odd = true;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  float *scale = p.scale[m] + page * p.H + h;
  float now = pow2_scale(amax);
  if (s0) {   // the block's first tokens stay: one scale for both
    const float old = *scale;
    if (old > now) now = old;
    if (old != now) {
      const float inv = now / old;   // >= 1, a power of two where the old scale is one
      for (int i = mine; i < s0; i += rows) {
        uint4 *q = reinterpret_cast<uint4 *>(to + (int64_t)i * p.d);
        uint4 t = *q;
        uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = floats_of(w[j]), b = floats_of(w[j] >> 16);
          const float f = 1.f / inv;
          w[j] = e4m3x2(a.x * f, a.y * f) | e4m3x2(b.x * f, b.y * f) << 16;
        }
        *q = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();   // every lane has read the old scale
  }
  if (lane == 0) *scale = now;
  const float f = 1.f / now;
  for (int i = mine; i < n; i += rows) {
    const T *src = source(i);
    uint32_t w[4] = {0, 0, 0, 0};
    if (src) {
      float v[16];
      load16(src, vec, v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        v[e] = v[e] != v[e] ? 0.f : v[e] * f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = e4m3x2(v[4 * j], v[4 * j + 1]) | e4m3x2(v[4 * j + 2], v[4 * j + 3]) << 16;
    }
    *reinterpret_cast<uint4 *>(to + (int64_t)(s0 + i) * p.d) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (odd) raise(p.status, KVX_FLAG_NOT_FINITE);
  if (lost) raise(p.status, KVX_FLAG_BAD_SRC_BLOCK);
}

// Grid: x = units of tokens, y = groups of kWriteWarps (head, K|V) pairs.
template <typename T>
__global__ void __launch_bounds__(32 * kWriteWarps) write_kernel(const __grid_constant__ WriteParams p,
                                                                 bool vec) {
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
  if (!p.req.ok()) {
    if (first_cta && threadIdx.x == 0) raise(p.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  const int hm = blockIdx.y * kWriteWarps + threadIdx.x / 32;
  if (hm >= 2 * p.H) return;
  const int m = hm / p.H, h = hm % p.H;
  const bool speaks = hm == 0 && threadIdx.x % 32 == 0;
  int64_t g = (int64_t)blockIdx.x * p.per_unit;
  const int64_t end = g + p.per_unit < p.req.ntok ? g + p.per_unit : p.req.ntok;
  while (g < end) {
    const int r = p.req.of(g);
    const int64_t beg = p.req.begin(r), stop = p.req.begin(r + 1);
    const int64_t start = p.start ? (int64_t)p.start[r] : 0;
    if (start < 0) {
      if (speaks) raise(p.status, KVX_FLAG_BAD_LENGTH);
      g = stop;
      continue;
    }
    const int64_t slot = start + g - beg, block = slot / p.bs;
    const int s0 = (int)(slot % p.bs);
    const int64_t left = stop - g, n = p.bs - s0 < left ? p.bs - s0 : left;
    if (g == beg || s0 == 0) {
      const int64_t page = block < p.max_blocks ? (int64_t)p.table[(int64_t)r * p.max_blocks + block] : -1;
      if (page >= 0 && page < p.num_blocks)
        write_run<T>(p, m, h, page, s0, g, (int)n, vec);
      else if (speaks)
        raise(p.status, block < p.max_blocks ? KVX_FLAG_BAD_BLOCK : KVX_FLAG_BAD_LENGTH);
    }
    g += n;
  }
}

}  // namespace

extern "C" kvx_status kvx_cache8_write(const kvx_cache8_write_args *a, void *stream) {
  if (!a) return KVX_ERR_INVALID_ARG;
  const kvx_cache8 &c = a->cache;
  if (const kvx_status st = check_cache8(c)) return st;
  if ((a->dtype != KVX_F32 && a->dtype != KVX_BF16) || a->num_requests < 1 || a->ntok < 0 ||
      a->ntok > INT32_MAX || (!a->cu_seqlens && a->ntok != a->num_requests) ||
      (a->src_rows && a->num_src_rows < 1))
    return KVX_ERR_INVALID_ARG;
  if (a->ntok == 0) return KVX_OK;
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  if (!a->k || !a->v || !aligned_to(a->k, size) || !aligned_to(a->v, size)) return KVX_ERR_INVALID_ARG;
  WriteParams p;
  p.codes[0] = (uint8_t *)c.k_codes;
  p.codes[1] = (uint8_t *)c.v_codes;
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.x[0] = a->k;
  p.x[1] = a->v;
  p.ts[0] = a->k_token_stride;
  p.ts[1] = a->v_token_stride;
  p.hs[0] = a->k_head_stride;
  p.hs[1] = a->v_head_stride;
  p.table = c.block_table;
  p.start = a->start;
  p.src_rows = a->src_rows;
  p.status = a->status;
  p.req = {a->cu_seqlens, a->num_requests, a->ntok};
  p.num_blocks = c.num_blocks;
  p.num_src_rows = a->num_src_rows;
  p.H = c.heads;
  p.d = c.head_dim;
  p.bs = c.block_size;
  p.max_blocks = c.max_blocks_per_req;
  // a unit begins about one run: a block's tokens, or a request's where those
  // are fewer
  const int64_t mean = a->ntok / a->num_requests;
  p.per_unit = (int)(mean < 1 ? 1 : mean > c.block_size ? c.block_size : mean);
  const bool vec = aligned_to(a->k, 16) && aligned_to(a->v, 16) &&
                   ((p.ts[0] | p.ts[1] | p.hs[0] | p.hs[1]) * size) % 16 == 0;
  const dim3 grid((unsigned)((a->ntok + p.per_unit - 1) / p.per_unit),
                  (unsigned)((2 * c.heads + kWriteWarps - 1) / kWriteWarps));
  cudaStream_t s = (cudaStream_t)stream;
  if (size == 2)
    write_kernel<__nv_bfloat16><<<grid, 32 * kWriteWarps, 0, s>>>(p, vec);
  else
    write_kernel<float><<<grid, 32 * kWriteWarps, 0, s>>>(p, vec);
  return launched();
}
