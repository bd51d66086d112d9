// kvx_attend8.cu -- attention of new tokens over the 8-bit paged cache
// (kvx_attend8), and the attention weight that each slot receives.
//
//   out_i = sum_j exp(x_ij - lse_i) v_j,  x_ij = scale q_i . k_j,
//   lse_i = log sum_j exp(x_ij),          j <= len - new + i.
// One pass over the slots with a running maximum and sum (fp32): when a larger
// score arrives, what was summed is scaled down to it.
//
// Here: fp32 queries, head dims above 128 and blocks that are not whole 8-slot
// groups; the rest runs on tcgen05 (kvx_attend8_tc.cu).  Products of f16 operands on
// 16 x 8 x 16 matrix instructions: codes are exact in f16, fp32 queries and
// probabilities go in two f16 parts.  Bound by those instructions, whose rate on this
// GPU is about 150 TFLOP/s: fp32, 16 requests of 1024 to 16,384 slots with 64 heads
// over 8 x 128 take 104 us, 133 with weights; one short request (4 heads over 2 x 64, 512
// slots) 13 us, the latency of its chain.  Prompts take long: every group of columns
// reads and multiplies all of its request's slots, those that none of it sees as well
// (8192 fp32 tokens of 64 heads 19.9 ms).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvx_async.cuh"
#include "kvx_attend8.cuh"

namespace {

// --- few queries: the slots split over the whole GPU -----------------------------

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
// The flattened work: for each request, each KV head, each group of columns
// (a column is a query of one head), the steps over its slots.  CTA c of n
// takes the steps [c T / n, (c + 1) T / n) of all T, so every CTA reads the same
// number of bytes whatever the lengths are, and a request's slots are split
// between as many CTAs as that takes.
struct Walk {
  int r, len, fresh, groups, h, group, steps, step;   // fresh: new tokens; groups: of columns
  int64_t beg;
};

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
  int vec_q;
};

template <class C>
__device__ __forceinline__ void enter_request(const SplitParams &p, Walk &w) {
  w.len = len_of(p.a, w.r);
  w.beg = p.a.req.begin(w.r);
  w.fresh = (int)(p.a.req.begin(w.r + 1) - w.beg);
  w.steps = w.len > 0 ? (w.len + C::KT - 1) / C::KT : 1;
  w.groups = (w.fresh * p.a.G + C::COLS - 1) / C::COLS;
}
template <class C>
__device__ __forceinline__ void advance(const SplitParams &p, Walk &w) {
  if (++w.step < w.steps) return;
  w.step = 0;
  if (++w.group < w.groups) return;
  w.group = 0;
  if (++w.h < p.a.H) return;
  w.h = 0;
  do {
    if (++w.r >= p.a.req.R) return;
    enter_request<C>(p, w);
  } while (w.groups == 0);
}
// Total steps, and (second form) the walk at step `at`.  A warp scans 32
// requests at a time.
template <class C>
__device__ __forceinline__ int64_t steps_of(const SplitParams &p, int r) {
  if (r >= p.a.req.R) return 0;
  Walk w;
  w.r = r;
  enter_request<C>(p, w);
  return (int64_t)w.steps * w.groups * p.a.H;
}
template <class C>
__device__ int64_t total_steps(const SplitParams &p) {
  int64_t sum = 0;
  for (int r = threadIdx.x % 32; r < p.a.req.R; r += 32) sum += steps_of<C>(p, r);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}
template <class C>
__device__ Walk walk_at(const SplitParams &p, int64_t at) {
  const int lane = threadIdx.x % 32;
  Walk w = {};
  int64_t before = 0;
  for (int r0 = 0; r0 < p.a.req.R; r0 += 32) {
    const int64_t mine = steps_of<C>(p, r0 + lane);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned here = __ballot_sync(~0u, at < before + upto);
    if (here) {
      const int who = __ffs(here) - 1;
      w.r = r0 + who;
      enter_request<C>(p, w);
      const int64_t in = at - before - __shfl_sync(~0u, upto - mine, who);
      const int seg = (int)(in / w.steps);
      w.step = (int)(in % w.steps);
      w.h = seg / w.groups;
      w.group = seg % w.groups;
      return w;
    }
    before += __shfl_sync(~0u, upto, 31);
  }
  return w;
}

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

// One warp: 16 MT slots at a time against COLS columns, its own ring of
// cp.async stages, its own running maximum and sum.  Scores are formed
// transposed, S^T = K Q^T with slots as the 16 rows, so the codes (converted to
// f16, exactly) are the large operand of both products and the few columns the
// small one; O^T = V^T P^T takes V by transposing 16-bit loads that carry two
// dimensions each.
//
// Ranges.  A query row is multiplied by the power of two that brings its
// largest element to [2^14, 2^15): f16 then holds a bf16 row exactly down to
// 2^-38 of that element (an fp32 row in two parts).  Probabilities carry their
// block's value scale, as a share of the largest one seen, times 2^14: f16's 11
// bits hold down to 2^-28 of the largest product, which costs an output less
// than its own rounding to bf16 (fp32 outputs take two parts here too).
template <class C>
__global__ void __launch_bounds__(32 * C::WARPS) split_kernel(const __grid_constant__ SplitParams p) {
  constexpr int DP = C::DP, NT = C::NT, PARTS = C::PARTS, MT = C::MT, KW = C::KW, CH = C::CH;
  extern __shared__ __align__(128) unsigned char smem[];
  const AttendParams &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  unsigned char *ring = smem + warp * C::STAGES * C::kStage;
  float *red = reinterpret_cast<float *>(smem + C::kRing);
  float *red_m = red + C::WARPS * C::RC * C::ROWF, *red_l = red_m + C::WARPS * C::COLS;
  uint2 *qs = reinterpret_cast<uint2 *>(smem + C::kRing + C::kReduce);
  float *col_scale = reinterpret_cast<float *>(smem + C::kRing + C::kReduce + (C::kQInSmem ? C::kQ : 0));
  int *flag = reinterpret_cast<int *>(col_scale + C::COLS);
  if (!requests_ok(a)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise(a.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < a.req.R; r += blockDim.x)
      if (len_of(a, r) != __ldg(a.lens + r)) raise(a.status, KVX_FLAG_BAD_LENGTH);
  const int64_t T = total_steps<C>(p), N = T < gridDim.x ? T : gridDim.x;   // CTAs at work
  if (blockIdx.x >= N) return;
  const int64_t first = blockIdx.x * T / N, last = (blockIdx.x + 1) * T / N;
  Walk w = walk_at<C>(p, first), pw = w;
  int64_t ahead = first;

  // Copy the warp's next tile into a stage: lane l looks up slot l, then 16-byte
  // pieces go out row by row.
  unsigned char *scales = nullptr;
  float kscale_next = 0.f, vscale_next = 0.f;
  const auto put_scales = [&]() {
    if (scales && lane < KW) {
      reinterpret_cast<float *>(scales)[lane] = kscale_next;
      reinterpret_cast<float *>(scales)[KW + lane] = vscale_next;
    }
    scales = nullptr;
  };
  const auto fetch = [&](int stage) {
    put_scales();
    unsigned char *st = ring + stage * C::kStage;
    if (ahead < last) {
      const int j = pw.step * C::KT + warp * KW + lane % KW;   // below len + KT <= 2^31
      int page = -1;
      uint32_t off = 0;
      if (j < pw.len) {
        const uint32_t block = block_of(a, j);
        off = j - block * a.bs;
        page = page_of(a, pw.r, block);
        if (page < 0) raise(a.status, KVX_FLAG_BAD_BLOCK);
      }
      const unsigned valid = __ballot_sync(~0u, page >= 0);
      const uint32_t block = page < 0 ? 0u : (uint32_t)page * a.H + pw.h;
      const uint32_t row = page < 0 ? 0u : block * a.bs + off;
      // scales by plain loads that land a step later (4-byte asynchronous copies
      // are not merged: a sector and more for each lane)
      scales = st + 2 * C::kTile;
      kscale_next = page >= 0 ? __ldg(a.ks + block) : 0.f;
      vscale_next = page >= 0 ? __ldg(a.vs + block) : 0.f;
      if (lane == 0) *reinterpret_cast<unsigned *>(st + 2 * C::kTile + 2 * KW * 4) = valid;
      const int c = lane % CH;
      if (valid == ~0u && C::DP == a.d) {
#pragma unroll
        for (int i = 0; i < KW * CH / 32; ++i) {
          const int j = i * (32 / CH) + lane / CH;
          const uint64_t at = (uint64_t)__shfl_sync(~0u, row, j) * C::DP + c * 16;
          cp_async16(st + piece_at<DP>(j, c), a.k + at, 16);
          cp_async16(st + C::kTile + piece_at<DP>(j, c), a.v + at, 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < KW * CH / 32; ++i) {
          const int j = i * (32 / CH) + lane / CH;
          const uint32_t from = __shfl_sync(~0u, row, j);
          const bool there = c * 16 < a.d && (valid >> j & 1);
          const uint64_t at = there ? (uint64_t)from * a.d + c * 16 : 0;
          cp_async16(st + piece_at<DP>(j, c), a.k + at, there ? 16 : 0);
          cp_async16(st + C::kTile + piece_at<DP>(j, c), a.v + at, there ? 16 : 0);
        }
      }
      advance<C>(p, pw);
      ++ahead;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) fetch(s);

  Queries<C> qf;
  const auto &cs = qf.cs;
  int limit[NT][2];          // last slot that they see
  // running maxima: as scores without their column's factor, and with it
  float mx[NT][2], m[NT][2], l[NT][2], o[NT][CH][4];
  bool far = false;                // one of the warp's maxima is
  float vref = 0.f, vinv = 0.f;   // largest value scale, and 2^14 over it
  int limits = 0;                 // the lowest of the limits
  int stage = 0;
  bool enter = true;
  int64_t seg_first = first;   // the CTA's first step of the segment
  for (int64_t now = first; now < last; ++now) {
    const int h = w.h, col0 = w.group * C::COLS, cols = w.fresh * a.G;
    if (enter) {
      enter = false;
      seg_first = now;
      // below 2^-112 a scale is treated as that: 2^14 over it stays finite
      vref = 0x1p-112f;
      vinv = 0x1p126f;
      far = false;
      limits = w.len - w.fresh + col0 / a.G;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = m[n][e] = -INFINITY;
          l[n][e] = 0.f;
          const int col = col0 + 8 * n + 2 * t + e;
          limit[n][e] = col < cols ? w.len - w.fresh + col / a.G : -1;
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][c][e] = 0.f;
      }
      qf.load(p, w.beg, h, col0, cols, qs, col_scale);
    }

    cp_async_wait<C::STAGES - 2>();
    put_scales();
    __syncwarp();
    fetch(stage == 0 ? C::STAGES - 1 : stage - 1);   // the tile of the step before is spent
    {
      const unsigned char *st = ring + stage * C::kStage;
      const uint32_t vaddr = (uint32_t)__cvta_generic_to_shared(st + C::kTile);
      const float *ks = reinterpret_cast<const float *>(st + 2 * C::kTile), *vs = ks + KW;
      const unsigned valid = *reinterpret_cast<const unsigned *>(st + 2 * C::kTile + 2 * KW * 4);
      const int j0 = w.step * C::KT + warp * KW;
      if (valid || (p.scores && j0 < w.len)) {
        float s[MT][NT][4];
        qf.scores(st, qs, s);
        // key scales; the mask, where the tile needs one
        float vsc[MT][2], most = 0.f;
        bool grew = false;
        // (with 16 slots a warp, lanes 16 .. 31 stand for the same ones)
        const bool masked = valid != ~0u || j0 + KW - 1 > limits || cols - col0 < C::COLS;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int j = 16 * i + 8 * half + g;
            const float kscale = ks[j];
            vsc[i][half] = vs[j];
            most = fmaxf(most, vsc[i][half]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float &x = s[i][n][2 * half + e];
                x *= kscale;
                if (masked && !((valid >> j & 1) && j0 + j <= limit[n][e])) x = -INFINITY;
                grew = grew || x > mx[n][e];
              }
          }
        if (p.scores) {
          const int64_t seg = ((int64_t)w.r * a.H + h) * p.groups + w.group;
          float *to = p.scores + seg * a.max_len * C::COLS;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int j = j0 + 16 * i + 8 * half + g;
              if (j >= w.len) continue;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2 *>(to + (int64_t)j * C::COLS + 8 * n + 2 * t) =
                    make_float2(s[i][n][2 * half] * cs[n][0], s[i][n][2 * half + 1] * cs[n][1]);
            }
        }
        if (__any_sync(~0u, grew || most > vref)) {   // seldom after the first tiles
          float top[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              top[n][e] = mx[n][e];
#pragma unroll
              for (int i = 0; i < MT; ++i) top[n][e] = fmaxf(top[n][e], fmaxf(s[i][n][e], s[i][n][2 + e]));
            }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            most = fmaxf(most, __shfl_xor_sync(~0u, most, off));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(~0u, top[n][e], off));
          }
          const float vnew = fmaxf(vref, most), vdown = vref / vnew;
          vref = vnew;
          vinv = 16384.f / vnew;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[n][e] = top[n][e];
              const float mm = finite_or_0(__fmul_rn(top[n][e], cs[n][e])), down = ex2(m[n][e] - mm);
              m[n][e] = top[n][e] > -INFINITY ? mm : -INFINITY;
              far = far || fabsf(mm) > kFar;
              l[n][e] *= down;
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                o[n][c][e] *= down * vdown;
                o[n][c][2 + e] *= down * vdown;
              }
            }
        }
        // Far scores are rounded before the maximum, which is a rounded score, is
        // subtracted: none comes out above it, however large both are.
        if (__any_sync(~0u, far)) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[i][n][e] = __fmul_rn(s[i][n][e], cs[n][e & 1]) - finite_or_0(m[n][e & 1]);
        } else {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[i][n][e] = fmaf(s[i][n][e], cs[n][e & 1], -finite_or_0(m[n][e & 1]));
        }
        // P^T: probabilities times their value scale, transposed between the lanes
        uint32_t pb[MT][NT][PARTS][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float f = vsc[i][half] * vinv;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float p0 = ex2(s[i][n][2 * half]), p1 = ex2(s[i][n][2 * half + 1]);
              l[n][0] += p0;
              l[n][1] += p1;
              float y0 = p0 * f, y1 = p1 * f;
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                const uint32_t b = half2_bits(y0, y1);
                pb[i][n][part][half] = transpose8x8(b);
                const float2 back = half2_floats(b);
                y0 -= back.x;
                y1 -= back.y;
              }
            }
          }
        // O^T += V^T P^T: rows g and g + 8 of a 16-dimension piece are its
        // dimensions 2g and 2g + 1
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int c = 0; c < CH; c += 2) {
            uint32_t v[4];
            ldmatrix_x4_trans(v, vaddr + piece_at<DP>(16 * i + lane % 16, c + lane / 16));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t y0 = __byte_perm(v[2 * k], 0, 0x3120), y1 = __byte_perm(v[2 * k + 1], 0, 0x3120);
              const uint32_t f[4] = {f16x2_of(y0), f16x2_of(y0 >> 16), f16x2_of(y1), f16x2_of(y1 >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
                  mma16816(o[n][c + k], f, pb[i][n][part][0], pb[i][n][part][1]);
            }
          }
      }
    }
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;

    const bool seg_done = w.step + 1 == w.steps;
    if (seg_done || now + 1 == last) {
      // join the warps, RC columns at a time.  From here on sums carry the values' scale,
      // which may be near the largest fp32, and 2^-kRoom: room for 2^kRoom slots
      const bool whole = seg_done && w.step + 1 <= now - seg_first + 1;
      // where it goes: the result, or a partial one (first or last of the CTA)
      float *slot = p.partial + ((int64_t)blockIdx.x * 2 + (seg_first == first ? 0 : 1)) * C::kSlot;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], off);
          if (g == 0) {
            red_m[warp * C::COLS + 8 * n + 2 * t + e] = m[n][e];
            red_l[warp * C::COLS + 8 * n + 2 * t + e] = l[n][e] * (kUnit * 16384.f);
          }
        }
#pragma unroll
      for (int round = 0; round < C::COLS / C::RC; ++round) {
        const int n = round * C::RC / 8;
        if (t / (C::RC / 2) == round % (8 / C::RC)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float *row = red + (warp * C::RC + 2 * (t % (C::RC / 2)) + e) * C::ROWF;
#pragma unroll
            for (int c = 0; c < CH; ++c)
              *reinterpret_cast<float2 *>(row + 16 * c + 2 * g) =
                  make_float2(o[n][c][e] * kUnit * vref, o[n][c][2 + e] * kUnit * vref);
          }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < C::RC * (DP / 2); x += 32 * C::WARPS) {
          const int in = x / (DP / 2), col = C::RC * round + in, d = x % (DP / 2) * 2, at = col0 + col;
          float mm = -INFINITY, ll = 0.f;
          float2 oo = make_float2(0.f, 0.f);
#pragma unroll
          for (int v = 0; v < C::WARPS; ++v) mm = fmaxf(mm, red_m[v * C::COLS + col]);
#pragma unroll
          for (int v = 0; v < C::WARPS; ++v) {
            const float f = ex2(red_m[v * C::COLS + col] - finite_or_0(mm));
            const float2 y = *reinterpret_cast<const float2 *>(red + (v * C::RC + in) * C::ROWF + d);
            ll += f * red_l[v * C::COLS + col];
            oo.x += f * y.x;
            oo.y += f * y.y;
          }
          if (whole) {
            if (at < cols && d < a.d) store_out(a, w.beg + at / a.G, h * a.G + at % a.G, d, oo, mm, kRoom, ll);
          } else {
            *reinterpret_cast<float2 *>(slot + col * DP + d) = oo;
            if (d == 0) {
              slot[C::COLS * DP + col] = mm;
              slot[C::COLS * (DP + 1) + col] = ll;
            }
          }
        }
        __syncthreads();
      }
      if (!whole) {
        // the last CTA of the segment to get here joins all of its parts
        const int64_t begin = now - w.step, end = begin + w.steps;   // the segment's steps
        const int64_t c0 = ((begin + 1) * N - 1) / T, c1 = (end * N - 1) / T;
        int *arrived = p.arrived + c0;     // of a CTA's items only the last can be split after it
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) *flag = atomicAdd(arrived, 1) == (int)(c1 - c0);
        __syncthreads();
        if (*flag) {
          __threadfence();
          if (threadIdx.x == 0) *arrived = 0;   // ready for the next call
          for (int x = threadIdx.x; x < C::COLS * (DP / 2); x += 32 * C::WARPS) {
            const int col = x / (DP / 2), d = x % (DP / 2) * 2, at = col0 + col;
            if (at >= cols || d >= a.d) continue;
            // CTA c's part is its first segment unless the segment begins inside it
            const float *p0 = p.partial + (c0 * 2 + (c0 * T / N != begin)) * C::kSlot;
            const float *p1 = p.partial + c0 * 2 * C::kSlot;
            const int parts = (int)(c1 - c0) + 1;
            float mm = -INFINITY, ll = 0.f;
            float2 oo = make_float2(0.f, 0.f);
#pragma unroll 8
            for (int c = 0; c < parts; ++c)
              mm = fmaxf(mm, __ldcg((c ? p1 + (int64_t)c * 2 * C::kSlot : p0) + C::COLS * DP + col));
            mm = finite_or_0(mm);
#pragma unroll 8
            for (int c = 0; c < parts; ++c) {
              const float *part = c ? p1 + (int64_t)c * 2 * C::kSlot : p0;
              const float f = ex2(__ldcg(part + C::COLS * DP + col) - mm);
              const float2 y = __ldcg(reinterpret_cast<const float2 *>(part + col * DP + d));
              ll += __ldcg(part + C::COLS * (DP + 1) + col) * f;
              oo.x += y.x * f;
              oo.y += y.y * f;
            }
            store_out(a, w.beg + at / a.G, h * a.G + at % a.G, d, oo, mm, kRoom, ll);
          }
        }
      }
      enter = true;
    }
    advance<C>(p, w);
  }
}

// weights[r][h][j] += sum over the columns of exp2(score - lse): the scores that
// the split kernel left, read once.
__global__ void __launch_bounds__(256) weights_of_scores_kernel(const __grid_constant__ SplitParams p,
                                                                int cols_of_group) {
  const AttendParams &a = p.a;
  constexpr int kCols = 512;     // at a time: whole groups
  __shared__ float2 lse[kCols];
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(a, r);
  if (!requests_ok(a) || (int64_t)blockIdx.x * 256 >= len) return;
  const int64_t beg = a.req.begin(r), j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cols = (int)(a.req.begin(r + 1) - beg) * a.G;
  float sum = 0.f;     // of the groups' sums: fewer roundings than of all in a row
  for (int c0 = 0; c0 < cols; c0 += cols_of_group) {
    if (c0 % kCols == 0) {
      __syncthreads();
      for (int c = threadIdx.x; c < kCols && c0 + c < cols; c += 256)
        lse[c] = a.stats[(beg + (c0 + c) / a.G) * a.Hq + h * a.G + (c0 + c) % a.G];
      __syncthreads();
    }
    if (j >= len) continue;
    float part = 0.f;
    const int64_t seg = ((int64_t)r * a.H + h) * p.groups + c0 / cols_of_group;
    const float *x = p.scores + (seg * a.max_len + j) * cols_of_group;
    for (int c = 0; c < cols_of_group && c0 + c < cols; c += 4) {
      const float4 y = *reinterpret_cast<const float4 *>(x + c);
      const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c0 + c + e < cols && z[e] > -INFINITY) part += probability(z[e], lse[c0 % kCols + c + e]);
    }
    sum += part;
  }
  if (j < len) a.weights[((int64_t)r * a.H + h) * a.wstride + j] += sum;
}

// The same where the scores were not kept: formed again from the same operands in the
// same order, so that they are the same numbers.  A CTA takes as many slots as a step of
// the split kernel and all columns that see one of them.
template <class C>
__global__ void __launch_bounds__(32 * C::WARPS) weights_again_kernel(const __grid_constant__ SplitParams p) {
  constexpr int DP = C::DP, NT = C::NT, MT = C::MT, KW = C::KW, CH = C::CH;
  extern __shared__ __align__(128) unsigned char smem[];
  const AttendParams &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  unsigned char *st = smem + warp * C::kAgainTile;
  uint2 *qs = reinterpret_cast<uint2 *>(smem + C::WARPS * C::kAgainTile);
  float *col_scale = reinterpret_cast<float *>(smem + C::WARPS * C::kAgainTile + (C::kQInSmem ? C::kQ : 0));
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(a, r);
  if (!requests_ok(a) || (int64_t)blockIdx.x * C::KT >= len) return;
  const int first = blockIdx.x * C::KT, j0 = first + warp * KW;
  const int64_t beg = a.req.begin(r);
  const int fresh = (int)(a.req.begin(r + 1) - beg), cols = fresh * a.G;
  // the warp's keys and their scales
  const int j = j0 + lane % KW;
  int page = -1;
  uint32_t row = 0;
  if (j < len) {
    const uint32_t block = block_of(a, j);
    page = page_of(a, r, block);
    if (page >= 0) row = ((uint32_t)page * a.H + h) * a.bs + (j - block * a.bs);
  }
  const float kscale = page >= 0 ? __ldg(a.ks + (uint32_t)page * a.H + h) : 0.f;
  const unsigned valid = __ballot_sync(~0u, page >= 0);
  const int c = lane % CH;
#pragma unroll
  for (int i = 0; i < KW * CH / 32; ++i) {
    const int k = i * (32 / CH) + lane / CH;
    const uint32_t from = __shfl_sync(~0u, row, k);
    const bool there = c * 16 < a.d && (valid >> k & 1);
    cp_async16(st + piece_at<DP>(k, c), a.k + (there ? (uint64_t)from * a.d + c * 16 : 0), there ? 16 : 0);
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  float sum[MT][2] = {};
  Queries<C> qf;
  // from the group of the first query that sees the CTA's first slot
  const int group0 = (int)((int64_t)max(0, first - (len - fresh)) * a.G / C::COLS);
  for (int col0 = group0 * C::COLS; col0 < cols; col0 += C::COLS) {
    qf.load(p, beg, h, col0, cols, qs, col_scale);
    float s[MT][NT][4];
    qf.scores(st, qs, s);
    float part[MT][2] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = col0 + 8 * n + 2 * t + e;
        const int limit = col < cols ? len - fresh + col / a.G : -1;
        const float2 lse = col < cols ? a.stats[(beg + col / a.G) * a.Hq + h * a.G + col % a.G] : make_float2(0.f, INFINITY);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int k = 16 * i + 8 * half + g;
            const float scale = __shfl_sync(~0u, kscale, k);
            const float z = __fmul_rn(__fmul_rn(s[i][n][2 * half + e], scale), qf.cs[n][e]);
            if ((valid >> k & 1) && j0 + k <= limit && z > -INFINITY) part[i][half] += probability(z, lse);
          }
      }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) sum[i][half] += part[i][half];
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) sum[i][half] += __shfl_xor_sync(~0u, sum[i][half], o);
      const int k = 16 * i + 8 * half + g;
      if (t == 0 && (valid >> k & 1)) a.weights[((int64_t)r * a.H + h) * a.wstride + j0 + k] += sum[i][half];
    }
}

kvx_status check(const kvx_attend8_args *a) {
  if (!a) return KVX_ERR_INVALID_ARG;
  const kvx_cache8 &c = a->cache;
  if (const kvx_status st = check_cache8(c)) return st;
  if ((a->dtype != KVX_F32 && a->dtype != KVX_BF16) || a->num_requests < 1 || a->ntok < 0 ||
      a->ntok > INT32_MAX || (!a->cu_seqlens && a->ntok != a->num_requests) || a->max_new < 1 ||
      a->max_len < 0 || a->max_len > INT32_MAX - 1024 || !a->lens || !std::isfinite(a->scale) || a->q_heads < 1 ||
      a->q_heads > 65535 || a->q_heads % c.heads)
    return KVX_ERR_INVALID_ARG;
  if (a->weights && a->weights_stride < a->max_len) return KVX_ERR_INVALID_ARG;
  if (a->weights && a->num_requests > 65535) return KVX_ERR_UNSUPPORTED;
  // the rows of one request and KV head are counted in 32 bits
  if ((int64_t)(a->q_heads / c.heads) * most_new(a) > INT32_MAX - 1024) return KVX_ERR_UNSUPPORTED;
  return KVX_OK;
}

// Sizes of a call's workspace and grid.
struct Shape {
  int cols, groups, grid;      // columns of a group, groups, CTAs
  size_t arrived, partial, stats, scores, bytes;   // offsets; what lies before the scores is needed
  bool spool;                  // the scores are kept for the weights
};
constexpr int kGrid = 152;     // one CTA an SM
static_assert(kGrid * sizeof(int) <= kWorkspaceHead, "the counters");

Shape shape_of(const kvx_attend8_args *a) {
  Shape s;
  const int64_t G = a->q_heads / a->cache.heads, most = G * most_new(a);
  s.cols = most <= 8 ? 8 : most <= 16 || a->cache.head_dim > 128 ? 16 : 32;   // registers hold 4096 sums
  s.groups = (int)((most + s.cols - 1) / s.cols);
  s.grid = kGrid;
  const int dp = a->cache.head_dim <= 64 ? 64 : a->cache.head_dim <= 128 ? 128 : 256;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.arrived = 0;
  s.partial = kWorkspaceHead;
  s.stats = s.partial + up((size_t)2 * s.grid * s.cols * (dp + 2) * 4);
  s.scores = s.stats + up((size_t)a->ntok * a->q_heads * sizeof(float2));
  // the scores of all columns, where the workspace has room for them
  const uint64_t kept = score_bytes(a, (int64_t)s.groups * s.cols, a->max_len);
  s.spool = a->weights && kept <= kMostScores && a->workspace_bytes >= s.scores + kept;
  s.bytes = s.scores + (a->weights ? up(kept < kMostScores ? kept : kMostScores) : 0);
  return s;
}

template <class C>
kvx_status launch_split(const SplitParams &p, int grid, bool again, cudaStream_t s) {
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(split_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
    return KVX_ERR_CUDA;
  split_kernel<C><<<grid, 32 * C::WARPS, C::kSmem, s>>>(p);
  if (const kvx_status st = launched()) return st;
  if (!again) return KVX_OK;
  if (cudaFuncSetAttribute(weights_again_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kAgainSmem) !=
      cudaSuccess)
    return KVX_ERR_CUDA;
  weights_again_kernel<C><<<dim3((p.a.max_len + C::KT - 1) / C::KT, p.a.H, p.a.req.R), 32 * C::WARPS, C::kAgainSmem, s>>>(p);
  return launched();
}
// tiles of 16 slots a warp works on at once, while the sums leave registers for two;
// stages: 8 slots tiles deep, or what shared memory holds
template <int DP, int NT, int PARTS>
using Cfg = SplitCfg<DP, NT, PARTS, (DP <= 128 && NT * PARTS <= 2 ? 2 : 1), 8,
                     (DP == 64 ? (NT * PARTS <= 2 ? 4 : 8) : DP == 128 ? (NT * PARTS <= 2 ? 3 : 5) : 2)>;
template <int DP, int PARTS>
kvx_status launch_cols(const SplitParams &p, int cols, int grid, bool again, cudaStream_t s) {
  if (cols == 8) return launch_split<Cfg<DP, 1, PARTS>>(p, grid, again, s);
  if (cols == 16) return launch_split<Cfg<DP, 2, PARTS>>(p, grid, again, s);
  if constexpr (DP <= 128) return launch_split<Cfg<DP, 4, PARTS>>(p, grid, again, s);
  return KVX_ERR_UNSUPPORTED;
}
// The split kernel and, with `again`, the weights from scores that were not kept.
template <int PARTS>
kvx_status launch_dim(const SplitParams &p, int cols, int grid, bool again, cudaStream_t s) {
  return p.a.d <= 64    ? launch_cols<64, PARTS>(p, cols, grid, again, s)
         : p.a.d <= 128 ? launch_cols<128, PARTS>(p, cols, grid, again, s)
                        : launch_cols<256, PARTS>(p, cols, grid, again, s);
}

}  // namespace

extern "C" size_t kvx_attend8_workspace_bytes(const kvx_attend8_args *a) {
  if (check(a) != KVX_OK) return 0;
  return kvx_attend8_tc_supports(a) ? kvx_attend8_tc_workspace_bytes(a) : shape_of(a).bytes;
}

extern "C" kvx_status kvx_attend8(const kvx_attend8_args *a, void *stream) {
  if (const kvx_status st = check(a)) return st;
  if (a->ntok == 0) return KVX_OK;
  const kvx_cache8 &c = a->cache;
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  if (!a->q || !a->out || !aligned_to(a->q, size) || !aligned_to(a->out, size)) return KVX_ERR_INVALID_ARG;
  if (a->weights && a->out == a->q) return KVX_ERR_INVALID_ARG;   // scores may be formed again
  const size_t least = kvx_attend8_tc_supports(a) ? kvx_attend8_tc_least_bytes(a) : shape_of(a).scores;
  if (!a->workspace || !aligned_to(a->workspace, 256) || a->workspace_bytes < least)
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
  p.lse = a->lse;
  p.weights = a->weights;
  p.stats = nullptr;
  p.status = a->status;
  p.req = {a->cu_seqlens, a->num_requests, a->ntok};
  p.num_blocks = (int)c.num_blocks;
  // with k = ceil(log2 bs), 2^(31 + k) / bs rounded up is off by less than 2^k / bs
  // a unit, so the quotient is exact below 2^31
  int k = 0;
  while (1 << k < c.block_size) ++k;
  p.bs_shift = 31 + k;
  p.bs_mul = (uint32_t)(((uint64_t)1 << (31 + k)) / c.block_size + 1);
  p.wstride = a->weights_stride;
  p.H = c.heads;
  p.Hq = a->q_heads;
  p.G = a->q_heads / c.heads;
  p.d = c.head_dim;
  p.bs = c.block_size;
  p.max_blocks = c.max_blocks_per_req;
  p.max_len = a->max_len;
  p.max_new = most_new(a);
  p.bf16 = size == 2;
  p.c = a->scale * kLog2e;
  cudaStream_t s = (cudaStream_t)stream;
  char *ws = (char *)a->workspace;
  if (kvx_attend8_tc_supports(a)) return kvx_attend8_tc_launch(a, p, ws, s);
  const Shape sh = shape_of(a);
  const bool weighs = a->weights && a->max_len > 0;
  if (weighs) p.stats = (float2 *)(ws + sh.stats);
  SplitParams sp;
  sp.a = p;
  sp.groups = sh.groups;
  sp.arrived = (int *)(ws + sh.arrived);
  sp.partial = (float *)(ws + sh.partial);
  sp.scores = sh.spool ? (float *)(ws + sh.scores) : nullptr;
  sp.vec_q = aligned_to(a->q, 16) && ((p.qt | p.qh) * size) % 16 == 0;
  const bool again = weighs && !sh.spool;
  const kvx_status st = size == 2 ? launch_dim<1>(sp, sh.cols, sh.grid, again, s) : launch_dim<2>(sp, sh.cols, sh.grid, again, s);
  if (st != KVX_OK || !weighs || again) return st;
  weights_of_scores_kernel<<<dim3((a->max_len + 255) / 256, c.heads, a->num_requests), 256, 0, s>>>(sp, sh.cols);
  return launched();
}
