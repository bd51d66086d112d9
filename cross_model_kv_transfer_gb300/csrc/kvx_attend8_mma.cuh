// kvx_attend8_mma.cuh -- what the attention kernels on 16 x 8 x 16 matrix instructions
// share (kvx_attend8_split.cu, kvx_attend8_own.cu): the instructions, sizes, the queries'
// fragments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_async.cuh"
#include "kvx_attend8.cuh"

namespace {

// D += A B of f16 operands, fp32 accumulation: 16 x 8, 16 deep.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, transposed between the lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t b) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&b));
}

template <int DP_, int NT_, int PARTS_, int MT_, int WARPS_, int STAGES_>
struct SplitCfg {
  static constexpr int RC = WARPS_ > 8 ? 2 : 4;   // columns joined at a time
  static constexpr int DP = DP_;         // head_dim, padded
  static constexpr int NT = NT_;         // column tiles of 8
  static constexpr int PARTS = PARTS_;   // f16 parts of an operand: 1 for bf16, 2 for fp32 queries
  static constexpr int MT = MT_;         // 16-slot tiles a warp takes at a time
  static constexpr int WARPS = WARPS_, STAGES = STAGES_;
  static constexpr int KW = 16 * MT, KT = KW * WARPS, COLS = 8 * NT, CH = DP / 16;
  static constexpr int ROWF = DP + 4;    // floats of a reduced row (padded against bank conflicts)
  static constexpr size_t kTile = (size_t)KW * DP;              // bytes of one K or V tile
  static constexpr size_t kStage = 2 * kTile + 2 * KW * 4 + 16; // + scales + valid bits
  static constexpr size_t kRing = kStage * STAGES * WARPS;
  static constexpr size_t kReduce = (size_t)WARPS * (RC * ROWF + 2 * COLS) * 4;
  static constexpr size_t kQ = (size_t)PARTS * COLS * DP * 2;   // query fragments (NT * PARTS > 2)
  static constexpr bool kQInSmem = NT * PARTS > 2;
  static constexpr size_t kSmem = kRing + kReduce + (kQInSmem ? kQ : 0) + COLS * 4 + 64;
  static constexpr int kSlot = COLS * (DP + 2);                 // floats of a partial result
  static constexpr size_t kAgainTile = kTile;                   // the weights' second pass: keys only
  static constexpr size_t kAgainSmem = kAgainTile * WARPS + (kQInSmem ? kQ : 0) + COLS * 4;
};

constexpr float kRoom = 24.f, kUnit = 0x1p-38f;   // 2^-kRoom over the 2^14 that probabilities carry

struct SplitParams {
  AttendParams a;
  int groups;            // column groups of max_new queries
  int *arrived;          // [grid] CTAs that have left a partial result of the item split after CTA c
  float *partial;        // [2 * grid][kSlot]
  float *scores;         // [R][H][groups][max_len][COLS], base 2, or NULL
  int vec_q, vec_out;    // rows on boundaries of whole loads and stores
};

// Where 16-byte piece c of slot row j lies in a tile: pieces move by the row,
// so that both ways of reading (one piece of eight rows, four pieces of two
// rows) meet every bank once.
template <int DP>
__device__ __forceinline__ uint32_t piece_at(int j, int c) {
  if constexpr (DP == 64) return (uint32_t)(j * 64 + ((c ^ (j >> 1 & 3)) << 4));
  const int f = (j & 1) << 2 | (j & 6) >> 1;
  return (uint32_t)(j * DP + ((c ^ f) << 4));
}

// Query fragments of a group of columns: the thread's column is g, its dimensions
// 64 q + 16 t ..; every thread of the CTA calls it where they lie in shared memory.
template <class C>
struct Queries {
  static constexpr int QD = C::DP / 64;
  uint32_t f[C::kQInSmem ? 1 : C::NT][C::PARTS][QD * 4][2];
  float cs[C::NT][2];           // factors of columns 2t, 2t + 1
  __device__ __forceinline__ void load(const SplitParams &p, int64_t beg, int h, int col0, int cols, uint2 *qs,
                                       float *col_scale) {
    constexpr int NT = C::NT, PARTS = C::PARTS;
    const AttendParams &a = p.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    if (C::kQInSmem) __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (C::kQInSmem && n % C::WARPS != warp % (NT < C::WARPS ? NT : C::WARPS)) continue;
      if (C::kQInSmem && warp >= NT) continue;
      const int col = col0 + 8 * n + g;
      float x[QD][16];
      float top = 0.f;
      const int64_t tok = beg + col / a.G;
      const int hq = h * a.G + col % a.G;
#pragma unroll
      for (int q = 0; q < QD; ++q) {
        const int d0 = 64 * q + 16 * t;
        const bool in = col < cols && d0 < a.d;
        const int64_t at = tok * a.qt + hq * a.qh + d0;
        if (PARTS == 1) {
          const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(a.q) + at;
          if (p.vec_q) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint4 y = in ? __ldg(reinterpret_cast<const uint4 *>(src) + v) : make_uint4(0, 0, 0, 0);
              const uint32_t b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[q][8 * v + 2 * e] = __uint_as_float(b[e] << 16);
                x[q][8 * v + 2 * e + 1] = __uint_as_float(b[e] & 0xffff0000u);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[q][e] = in ? __bfloat162float(src[e]) : 0.f;
          }
        } else {
          const float *src = reinterpret_cast<const float *>(a.q) + at;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[q][e] = in ? __ldg(src + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[q][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      e2 = e2 < -100 ? -100 : e2;
      // the factor stays positive, so that maxima may be taken without it
      const float up = a.c != 0.f ? copysignf(__uint_as_float((uint32_t)(14 - e2 + 127) << 23), a.c) : 0.f;
      const float factor = fmaxf(fabsf(a.c) * __uint_as_float((uint32_t)(e2 - 14 + 127) << 23), 0x1p-126f);
#pragma unroll
      for (int q = 0; q < QD; ++q)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = x[q][4 * s + e] * up;
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            const uint32_t b0 = half2_bits(y[0], y[1]), b1 = half2_bits(y[2], y[3]);
            if (C::kQInSmem) {
              qs[((part * NT + n) * QD * 4 + q * 4 + s) * 32 + lane] = make_uint2(b0, b1);
            } else {
              f[C::kQInSmem ? 0 : n][part][q * 4 + s][0] = b0;
              f[C::kQInSmem ? 0 : n][part][q * 4 + s][1] = b1;
            }
            const float2 r0 = half2_floats(b0), r1 = half2_floats(b1);
            y[0] -= r0.x; y[1] -= r0.y; y[2] -= r1.x; y[3] -= r1.y;
          }
        }
      if (C::kQInSmem) {
        if (t == 0) col_scale[8 * n + g] = factor;
      } else {
        cs[n][0] = __shfl_sync(~0u, factor, 8 * t);        // lane 4 g' holds column g'
        cs[n][1] = __shfl_sync(~0u, factor, 8 * t + 4);
      }
    }
    if (C::kQInSmem) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        cs[n][0] = col_scale[8 * n + 2 * t];
        cs[n][1] = col_scale[8 * n + 2 * t + 1];
      }
    }
  }
  // S^T = K Q^T of a warp's tile at st
  __device__ __forceinline__ void scores(const unsigned char *st, const uint2 *qs, float (&s)[C::MT][C::NT][4]) const {
    constexpr int DP = C::DP, NT = C::NT, PARTS = C::PARTS, MT = C::MT;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
    for (int q = 0; q < QD; ++q) {
      uint4 k0[MT], k1[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        k0[i] = *reinterpret_cast<const uint4 *>(st + piece_at<DP>(16 * i + g, 4 * q + t));
        k1[i] = *reinterpret_cast<const uint4 *>(st + piece_at<DP>(16 * i + g + 8, 4 * q + t));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t b[NT][PARTS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            if (C::kQInSmem) {
              const uint2 y = qs[((part * NT + n) * QD * 4 + q * 4 + u) * 32 + lane];
              b[n][part][0] = y.x;
              b[n][part][1] = y.y;
            } else {
              b[n][part][0] = f[C::kQInSmem ? 0 : n][part][q * 4 + u][0];
              b[n][part][1] = f[C::kQInSmem ? 0 : n][part][q * 4 + u][1];
            }
          }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t x0 = u == 0 ? k0[i].x : u == 1 ? k0[i].y : u == 2 ? k0[i].z : k0[i].w;
          const uint32_t x1 = u == 0 ? k1[i].x : u == 1 ? k1[i].y : u == 2 ? k1[i].z : k1[i].w;
          const uint32_t kf[4] = {f16x2_of(x0), f16x2_of(x1), f16x2_of(x0 >> 16), f16x2_of(x1 >> 16)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < PARTS; ++part) mma16816(s[i][n], kf, b[n][part][0], b[n][part][1]);
        }
      }
    }
  }
};

}  // namespace
