// kvx_cache8.cu -- the 8-bit paged cache's write (kvx_cache8_write).
//
// For each block and head, separately for keys and values: the scale is the
// smallest power of two that brings the largest new magnitude to 448 or less
// (or the block's own where it already holds tokens and that is larger), and
// code = e4m3(x / scale).  Bound by HBM: the new rows are read once and one byte an
// element is written.  139 thousand bf16 tokens of 8 heads x 128 dimensions into
// blocks of 16 take 141 us, 6.06 TB/s, where a copy reaches 6.74.  A run of up to 64
// elements a lane (those 16 x 128) stays in registers between the maximum and the
// codes, all of its loads on their way at once; a longer one is read again, from L1
// or L2 (the same call then takes 238 us).  The maximum is taken on the bits, bf16
// two at a time, and finite numbers are told from others once a run: with
// both done element by element the call was bound by its instructions (229 us).
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

// 16 consecutive elements as they lie.
template <typename T>
struct Sixteen {
  uint4 x[sizeof(T)];
  __device__ __forceinline__ void load(const T *p, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) x[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    } else {
      T v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = p[i];
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) {
        constexpr int n = 16 / sizeof(T);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (sizeof(T) == 2)
            w[k] = (uint32_t)__bfloat16_as_ushort(v[n * i + 2 * k]) | (uint32_t)__bfloat16_as_ushort(v[n * i + 2 * k + 1]) << 16;
          else
            w[k] = __float_as_uint(v[n * i + k]);
        }
        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) x[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
          v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
          v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          v[4 * i + k] = __uint_as_float(w[k]);
        }
      }
    }
  }
  // The larger of the magnitudes' bits and `most` (bf16: two at a time, in the two
  // halves): above those of every finite number where there is an infinity or a NaN.
  __device__ __forceinline__ uint32_t largest(uint32_t most) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) most = __vmaxu2(most, w[k] & 0x7fff7fffu);
        else most = max(most, w[k] & 0x7fffffffu);
      }
    }
    return most;
  }
  // The largest finite magnitude and `amax` (where there is an infinity or a NaN).
  __device__ __forceinline__ float largest_finite(float amax) const {
    float v[16];
    floats(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fabsf(v[e]) < INFINITY ? fmaxf(amax, fabsf(v[e])) : amax;
    return amax;
  }
  template <bool ODD>
  __device__ __forceinline__ uint4 codes(float f) const {
    float v[16];
    floats(v);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = ODD && v[e] != v[e] ? 0.f : v[e] * f;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = e4m3x2(v[4 * j], v[4 * j + 1]) | e4m3x2(v[4 * j + 2], v[4 * j + 3]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

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
  uint32_t most = 0;
  bool lost = false;
  constexpr int HELD = 4;
  Sixteen<T> held[HELD];
  const bool holds = n <= HELD * rows;     // of the whole warp
  if (holds) {
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int i = mine + k * rows;
      const T *src = i < n ? source(i) : nullptr;
      lost = lost || (i < n && !src);
      if (src) held[k].load(src, vec); else held[k].zero();
    }
#pragma unroll
    for (int k = 0; k < HELD; ++k) most = held[k].largest(most);
  } else {
#pragma unroll 2
    for (int i = mine; i < n; i += rows) {
      const T *src = source(i);
      lost = lost || !src;
      if (!src) continue;
      Sixteen<T> x;
      x.load(src, vec);
      most = x.largest(most);
    }
  }
  if constexpr (sizeof(T) == 2) most = max(most & 0xffffu, most >> 16) << 16;
  most = __reduce_max_sync(~0u, most);
  float amax = __uint_as_float(most);
  const bool odd = most >= 0x7f800000u;
  if (odd) {     // seldom: leave the infinities and NaN out
    amax = 0.f;
    for (int i = mine; i < n; i += rows) {
      const T *src = source(i);
      if (!src) continue;
      Sixteen<T> x;
      x.load(src, vec);
      amax = x.largest_finite(amax);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if (lane == 0) raise(p.status, KVX_FLAG_NOT_FINITE);
  }
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
  const auto store = [&](int i, const Sixteen<T> &x) {
    __stcs(reinterpret_cast<uint4 *>(to + (int64_t)(s0 + i) * p.d), odd ? x.template codes<true>(f) : x.template codes<false>(f));
  };
  if (holds) {
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (mine + k * rows < n) store(mine + k * rows, held[k]);
  } else {
#pragma unroll 2
    for (int i = mine; i < n; i += rows) {
      const T *src = source(i);
      Sixteen<T> x;
      if (src) x.load(src, vec); else x.zero();
      store(i, x);
    }
  }
  if (lost) raise(p.status, KVX_FLAG_BAD_SRC_BLOCK);
}

// The request of token g, by the whole warp: how many requests begin at or before it.
__device__ __forceinline__ int request_of(const Requests &q, int64_t g) {
  if (!q.cu) return (int)g;
  int n = 0;
  for (int r0 = 0; r0 < q.R; r0 += 32) {
    const int r = r0 + threadIdx.x % 32;
    const unsigned here = __ballot_sync(~0u, r < q.R && (int64_t)__ldg(q.cu + r) <= g);
    n += __popc(here);
    if (here != ~0u) break;
  }
  return n - 1;
}
// Requests::ok by each warp for itself.
__device__ __forceinline__ bool table_ok(const Requests &q) {
  bool good = true;
  if (q.cu)
    for (int r = threadIdx.x % 32; r < q.R; r += 32) {
      const int32_t beg = __ldg(q.cu + r), end = __ldg(q.cu + r + 1);
      good = good && end >= beg && (r > 0 || beg == 0) && (r + 1 < q.R || end == q.ntok);
    }
  return __all_sync(~0u, good);
}

// Grid: x = units of tokens, y = groups of (head, K|V) pairs.  A warp takes several
// pairs of a run in turn: finding the run costs more than one pair of it (up to four
// pairs 141 us, two 147; CTAs of eight warps 154).
template <typename T>
__global__ void __launch_bounds__(32 * kWriteWarps) write_kernel(const __grid_constant__ WriteParams p,
                                                                 bool vec) {
  const int hm0 = blockIdx.y * kWriteWarps + threadIdx.x / 32;
  const bool speaks = hm0 == 0 && threadIdx.x % 32 == 0;
  if (!table_ok(p.req)) {
    if (speaks && blockIdx.x == 0) raise(p.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  int64_t g = (int64_t)blockIdx.x * p.per_unit;
  const int64_t end = g + p.per_unit < p.req.ntok ? g + p.per_unit : p.req.ntok;
  while (g < end) {
    const int r = request_of(p.req, g);
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
      if (page >= 0 && page < p.num_blocks) {
        for (int hm = hm0; hm < 2 * p.H; hm += gridDim.y * kWriteWarps)
          write_run<T>(p, hm / p.H, hm % p.H, page, s0, g, (int)n, vec);
      } else if (speaks) {
        raise(p.status, block < p.max_blocks ? KVX_FLAG_BAD_BLOCK : KVX_FLAG_BAD_LENGTH);
      }
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
  // pairs in turn in a warp: up to four once that leaves 16 warps an SM
  const int64_t units = (a->ntok + p.per_unit - 1) / p.per_unit, want = units * 2 * c.heads / (152 * 16);
  const int turns = kWriteWarps * (int)(want < 1 ? 1 : want > 4 ? 4 : want);
  const dim3 grid((unsigned)units, (unsigned)((2 * c.heads + turns - 1) / turns));
  cudaStream_t s = (cudaStream_t)stream;
  if (size == 2)
    write_kernel<__nv_bfloat16><<<grid, 32 * kWriteWarps, 0, s>>>(p, vec);
  else
    write_kernel<float><<<grid, 32 * kWriteWarps, 0, s>>>(p, vec);
  return launched();
}
