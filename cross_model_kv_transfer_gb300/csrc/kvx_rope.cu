// kvx_rope.cu -- rotary positions of new tokens' queries and keys
// (kvx_rope_init, kvx_rope_apply).
//
// y = a R(p) x: pair i of the rotated part is turned by p w_i,
//   (x0, x1) -> a (x0 cos - x1 sin, x1 cos + x0 sin),
// and the transposed turn is the gradient.  Frequencies are kept in turns a
// position as 64-bit binary fractions (rope_cs in kvx_ptx.cuh): the phase of
// any position is an exact integer product, so long contexts lose nothing and
// no table is read.
//
// Bound by HBM: every row is read and written once (32,768 bf16 tokens of 72 heads x
// 128: 186 us, 6.5 TB/s of the 6.7 that a copy reaches).  A thread owns one piece
// of a head vector (V pairs: 16 bytes of each side of the pairs) and walks
// over several heads of one token with the same cosines and sines, because
// forming them costs about as much as moving the piece of four heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvx_internal.h"
#include "kvx_ptx.cuh"

namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const void *x[2];      // q, k
  void *y[2];
  int64_t xt[2], xh[2], yt[2], yh[2];   // token and head strides, elements
  const int32_t *positions;
  uint32_t *status;
  int64_t first, ntok;
  int heads[2];
  int d, rot, transpose, interleaved;
  int head_lanes, head_steps;   // heads side by side in a CTA, and in turn in a thread
  float amp;
  unsigned long long turns[128];
};

template <typename T> struct Piece;
template <> struct Piece<float> {
  static constexpr int V = 4;           // elements of 16 bytes
  float v[4];
  __device__ void load(const float *p) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
  __device__ void store(float *p) const {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int V = 8;
  float v[8];
  __device__ void load(const __nv_bfloat16 *p) {
    const uint4 t = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};

// cos and sin of the phase pos * turns.  bf16 outputs take the transfer's form, off by up
// to 8e-7 of the row's values (their own rounding is 2e-3); fp32 outputs one that is off by
// 1e-7: the phase is exact to 2^-32 of a turn, and what is left of it after whole quarters is
// rounded to fp32 by 2e-8 rad at most (32,768 tokens of 72 heads x 128: 364.2 us, 363.4 with
// the transfer's form).
template <typename T>
__device__ __forceinline__ void turn_of(uint32_t pos, unsigned long long turns, float &c, float &s) {
  if constexpr (sizeof(T) == 2) {
    rope_cs(pos, turns, c, s);
  } else {
    const uint32_t top = (uint32_t)((unsigned long long)pos * turns >> 32);
    const uint32_t quarters = (top + 0x20000000u) >> 30;
    float x, y;
    sincospif((float)(int32_t)(top - (quarters << 30)) * 0x1p-31f, &y, &x);
    const float u = quarters & 1 ? y : x, v = quarters & 1 ? x : y;
    c = (quarters + 1) & 2 ? -u : u;
    s = quarters & 2 ? -v : v;
  }
}

// One head row: which array, and where its piece starts.
template <typename T>
__device__ __forceinline__ bool row_of(const RopeParams &p, int64_t g, int h, const T *&src, T *&dst) {
  const int w = h >= p.heads[0];
  const int hh = w ? h - p.heads[0] : h;
  if (w && hh >= p.heads[1]) return false;
  src = reinterpret_cast<const T *>(p.x[w]) + g * p.xt[w] + hh * p.xh[w];
  dst = reinterpret_cast<T *>(p.y[w]) + g * p.yt[w] + hh * p.yh[w];
  return true;
}

// A CTA: consecutive tokens x head_lanes heads x the pieces of a head vector.
// Pieces [0, rot / 2 / V) rotate two 16-byte vectors, the rest copy one.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = Piece<T>::V;
  const int half = p.rot / 2, turning = half / V, pieces = turning + (p.d - p.rot) / V;
  const int slots = kRopeThreads / pieces, tokens = slots / p.head_lanes;
  const int slot = threadIdx.x / pieces, u = threadIdx.x % pieces;
  const int64_t g = (int64_t)blockIdx.x * tokens + slot / p.head_lanes;
  if (slot >= tokens * p.head_lanes || g >= p.ntok) return;
  int h = blockIdx.y * p.head_lanes * p.head_steps + slot % p.head_lanes;
  const int64_t pos = p.positions ? (int64_t)__ldg(p.positions + g) : p.first + g;
  if (pos < 0 || pos > INT32_MAX) {
    if (u == 0 && slot % p.head_lanes == 0 && p.status) atomicOr(p.status, KVX_FLAG_BAD_POSITION);
    return;
  }
  if (u >= turning) {
    const int at = p.rot + (u - turning) * V;
#pragma unroll 4
    for (int j = 0; j < p.head_steps; ++j, h += p.head_lanes) {
      const T *src;
      T *dst;
      if (!row_of(p, g, h, src, dst)) break;
      if (src != dst) *reinterpret_cast<uint4 *>(dst + at) = *reinterpret_cast<const uint4 *>(src + at);
    }
    return;
  }
  float c[V], s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    turn_of<T>((uint32_t)pos, p.turns[u * V + e], c[e], s[e]);
    c[e] *= p.amp;
    s[e] *= p.transpose ? -p.amp : p.amp;
  }
  const int a0 = p.interleaved ? 2 * u * V : u * V;
  const int a1 = p.interleaved ? a0 + V : a0 + half;
#pragma unroll 4
  for (int j = 0; j < p.head_steps; ++j, h += p.head_lanes) {
    const T *src;
    T *dst;
    if (!row_of(p, g, h, src, dst)) break;
    Piece<T> a, b;
    a.load(src + a0);
    b.load(src + a1);
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < V; ++e) {   // pair e: elements 2e, 2e + 1 of the two vectors
        float &x0 = e < V / 2 ? a.v[2 * e] : b.v[2 * e - V];
        float &x1 = e < V / 2 ? a.v[2 * e + 1] : b.v[2 * e + 1 - V];
        const float y0 = x0 * c[e] - x1 * s[e], y1 = x1 * c[e] + x0 * s[e];
        x0 = y0;
        x1 = y1;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y0 = a.v[e] * c[e] - b.v[e] * s[e], y1 = b.v[e] * c[e] + a.v[e] * s[e];
        a.v[e] = y0;
        b.v[e] = y1;
      }
    }
    a.store(dst + a0);
    b.store(dst + a1);
  }
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Rows that 16-byte pieces do not fit (a rotated half that is not whole
// pieces, bases or strides off 16 bytes): one pair or one copied element a
// thread.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(const __grid_constant__ RopeParams p) {
  const int half = p.rot / 2, pieces = half + p.d - p.rot, total = p.heads[0] + p.heads[1];
  const int64_t n = p.ntok * total * pieces;
  for (int64_t i = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kRopeThreads) {
    const int u = (int)(i % pieces);
    const int64_t row = i / pieces, g = row / total;
    const int64_t pos = p.positions ? (int64_t)__ldg(p.positions + g) : p.first + g;
    if (pos < 0 || pos > INT32_MAX) {
      if (u == 0 && p.status) atomicOr(p.status, KVX_FLAG_BAD_POSITION);
      continue;
    }
    const T *src;
    T *dst;
    if (!row_of(p, g, (int)(row % total), src, dst)) continue;
    if (u >= half) {
      dst[p.rot + u - half] = src[p.rot + u - half];
      continue;
    }
    float c, s;
    turn_of<T>((uint32_t)pos, p.turns[u], c, s);
    c *= p.amp;
    s *= p.transpose ? -p.amp : p.amp;
    const int a0 = p.interleaved ? 2 * u : u, a1 = p.interleaved ? a0 + 1 : a0 + half;
    const float x0 = to_f(src[a0]), x1 = to_f(src[a1]);
    put(dst + a0, x0 * c - x1 * s);
    put(dst + a1, x1 * c + x0 * s);
  }
}

// Turns a position as a 64-bit binary fraction.
unsigned long long fraction(long double turns) {
  const long double x = ldexpl(turns - floorl(turns), 32), hi = floorl(x);
  return ((unsigned long long)hi << 32) + (unsigned long long)roundl(ldexpl(x - hi, 32));
}

}  // namespace

extern "C" kvx_status kvx_rope_init(const kvx_rope_desc *d, kvx_rope *rope) {
  if (!d || !rope) return KVX_ERR_INVALID_ARG;
  const int rot = d->rot_dim;
  if (d->head_dim < 2 || d->head_dim > 256 || (d->head_dim & 1) || rot < 2 || rot > d->head_dim ||
      (rot & 1) || (d->layout != KVX_ROPE_HALF && d->layout != KVX_ROPE_INTERLEAVED) ||
      d->scaling < KVX_ROPE_UNSCALED || d->scaling > KVX_ROPE_YARN ||
      !(std::isfinite(d->theta) && d->theta > 1.0) || !std::isfinite(d->amplitude))
    return KVX_ERR_INVALID_ARG;
  if (d->scaling != KVX_ROPE_UNSCALED && !(std::isfinite(d->factor) && d->factor >= 1.0))
    return KVX_ERR_INVALID_ARG;
  if (d->scaling >= KVX_ROPE_BANDS && d->original_context < 1) return KVX_ERR_INVALID_ARG;
  if (d->scaling == KVX_ROPE_BANDS &&
      !(std::isfinite(d->high_band) && d->low_band >= 0.0 && d->low_band < d->high_band))
    return KVX_ERR_INVALID_ARG;
  if (d->scaling == KVX_ROPE_YARN &&
      !(std::isfinite(d->beta_fast) && d->beta_slow > 0.0 && d->beta_fast > d->beta_slow))
    return KVX_ERR_INVALID_ARG;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  rope->head_dim = d->head_dim;
  rope->rot_dim = rot;
  rope->layout = d->layout;
  long double lo = 0, hi = 1;
  if (d->scaling == KVX_ROPE_YARN) {
    const auto pair = [&](long double beta) {
      return rot * logl(d->original_context / (beta * two_pi)) / (2 * logl((long double)d->theta));
    };
    lo = fmaxl(floorl(pair(d->beta_fast)), 0.0L);
    hi = fmaxl(fminl(ceill(pair(d->beta_slow)), rot - 1), lo + 0.001L);
  }
  for (int i = 0; i < 128; ++i) {
    rope->turns[i] = 0;
    if (i >= rot / 2) continue;
    const long double w = powl((long double)d->theta, -2.0L * i / rot);
    const long double f = d->scaling == KVX_ROPE_UNSCALED ? 1.0L : (long double)d->factor;
    long double s = 0;   // share that is not stretched
    if (d->scaling == KVX_ROPE_BANDS)
      s = (d->original_context * w / two_pi - d->low_band) / ((long double)d->high_band - d->low_band);
    else if (d->scaling == KVX_ROPE_YARN)
      s = 1 - fminl(fmaxl((i - lo) / (hi - lo), 0.0L), 1.0L);
    s = fminl(fmaxl(s, 0.0L), 1.0L);
    rope->turns[i] = fraction(w * (s + (1 - s) / f) / two_pi);
  }
  const double own = d->scaling == KVX_ROPE_YARN ? 0.1 * std::log(d->factor) + 1.0 : 1.0;
  rope->amplitude = (float)(d->amplitude != 0.0 ? d->amplitude : own);
  return KVX_OK;
}

extern "C" kvx_status kvx_rope_apply(const kvx_rope *rope, const kvx_rope_args *a, void *stream) {
  if (!rope || !a) return KVX_ERR_INVALID_ARG;
  const int d = rope->head_dim, rot = rope->rot_dim;
  if (d < 2 || d > 256 || (d & 1) || rot < 2 || rot > d || (rot & 1)) return KVX_ERR_INVALID_ARG;
  if (a->dtype != KVX_F32 && a->dtype != KVX_BF16) return KVX_ERR_INVALID_ARG;
  if (a->ntok < 0 || (a->transpose != 0 && a->transpose != 1)) return KVX_ERR_INVALID_ARG;
  if (!a->positions && (a->first_position < 0 || a->ntok > INT64_MAX - a->first_position))
    return KVX_ERR_INVALID_ARG;
  if (a->ntok == 0) return KVX_OK;
  if (!a->q && !a->k) return KVX_ERR_INVALID_ARG;
  const int size = a->dtype == KVX_BF16 ? 2 : 4, V = 16 / size;
  RopeParams p;
  p.x[0] = a->q;
  p.x[1] = a->k;
  p.y[0] = a->q_out;
  p.y[1] = a->k_out;
  const int64_t xs[2][2] = {{a->q_token_stride, a->q_head_stride}, {a->k_token_stride, a->k_head_stride}};
  const int64_t ys[2][2] = {{a->q_out_token_stride, a->q_out_head_stride},
                            {a->k_out_token_stride, a->k_out_head_stride}};
  const int heads[2] = {a->q ? a->q_heads : 0, a->k ? a->k_heads : 0};
  bool wide = rot / 2 % V == 0 && (d - rot) % V == 0;
  for (int w = 0; w < 2; ++w) {
    p.heads[w] = heads[w];
    p.xt[w] = xs[w][0];
    p.xh[w] = xs[w][1];
    p.yt[w] = ys[w][0];
    p.yh[w] = ys[w][1];
    if (!p.x[w]) continue;
    if (heads[w] < 1 || heads[w] > 65535 || !p.y[w]) return KVX_ERR_INVALID_ARG;
    const uintptr_t both = (uintptr_t)p.x[w] | (uintptr_t)p.y[w];
    if (both % size) return KVX_ERR_INVALID_ARG;
    // a single token or head has no stride to speak of
    const int64_t steps = (a->ntok > 1 ? p.xt[w] | p.yt[w] : 0) | (heads[w] > 1 ? p.xh[w] | p.yh[w] : 0);
    wide = wide && both % 16 == 0 && steps % V == 0;
  }
  p.positions = a->positions;
  p.first = a->first_position;
  p.status = a->status;
  p.ntok = a->ntok;
  p.d = d;
  p.rot = rot;
  p.transpose = a->transpose;
  p.interleaved = rope->layout == KVX_ROPE_INTERLEAVED;
  p.amp = rope->amplitude;
  for (int i = 0; i < 128; ++i) p.turns[i] = rope->turns[i];
  const int total = heads[0] + heads[1];
  cudaStream_t s = (cudaStream_t)stream;
  if (!wide) {
    const int64_t n = a->ntok * total * (rot / 2 + d - rot);
    const int64_t blocks = (n + kRopeThreads - 1) / kRopeThreads;
    const unsigned grid = (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
    if (size == 2)
      rope_scalar_kernel<__nv_bfloat16><<<grid, kRopeThreads, 0, s>>>(p);
    else
      rope_scalar_kernel<float><<<grid, kRopeThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? KVX_OK : KVX_ERR_CUDA;
  }
  const int pieces = rot / 2 / V + (d - rot) / V, slots = kRopeThreads / pieces;
  // up to eight heads in turn in a thread, fewer where that would not leave 1024
  // threads an SM (2047 fp32 tokens of 16 + 8 heads x 128, 64 turned: 19.6 us; with
  // 512 an SM 20.3, with 2048 22.8, with 4096 26.1); the heads side by side in a
  // CTA are a power of two, to fill it
  const int64_t want = a->ntok * total * pieces / (152 * 1024);
  const int turns = (int)(want < 1 ? 1 : want > 8 ? 8 : want);
  p.head_lanes = 1;
  while (2 * p.head_lanes <= slots && 2 * p.head_lanes * turns <= total) p.head_lanes *= 2;
  const int groups = (total + p.head_lanes * turns - 1) / (p.head_lanes * turns);
  p.head_steps = (total + p.head_lanes * groups - 1) / (p.head_lanes * groups);
  const int tokens = slots / p.head_lanes;
  const int64_t gx = (a->ntok + tokens - 1) / tokens;
  if (gx > INT32_MAX) return KVX_ERR_UNSUPPORTED;
  const int per = p.head_lanes * p.head_steps;
  if ((total + per - 1) / per > 65535) return KVX_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)((total + per - 1) / per));
  if (size == 2)
    rope_kernel<__nv_bfloat16><<<grid, kRopeThreads, 0, s>>>(p);
  else
    rope_kernel<float><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KVX_OK : KVX_ERR_CUDA;
}
