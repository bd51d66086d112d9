// kvx_attend8.cuh -- what the attention kernels over the 8-bit cache share
// (kvx_attend8_split.cu, kvx_attend8_tc.cu, kvx_attend8_own.cu) and their calls
// (kvx_attend8.cu): parameters, lookups and checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

// Compiled twice: for kvx_attend8, and (KVX_ATTEND_SHARED) for the passes of
// kvx_attend8_shared, so that what those need costs the others nothing.
#ifndef KVX_ATTEND_SHARED
#define KVX_ATTEND_SHARED 0
#endif

namespace kvx8 {

// Requests that share prefixes, in the passes of kvx_attend8_shared.  Over the prefixes
// (`all`): a query sees every slot, and request r of the pass is the queries of the requests
// of[r] .. of[r + 1] - 1 of `inner`, or of all tokens (`whole`).  Over the requests' own
// slots: `before` and `before_stats` are what the first pass left, [ntok][Hq][d] and
// [ntok][Hq], to join with, and the `count` groups `of` are checked again, at most `most`
// tokens each, so that a bad table stops both passes.
struct Sharing {
  const int32_t *of;
  int inner, count, whole, all;
  int64_t most;
  const float *before;
  const float2 *before_stats;
};

struct AttendParams {
  const uint8_t *k, *v;
  const float *ks, *vs;
  const void *q;
  void *out;
  int64_t qt, qh, ot, oh;
  const int32_t *table, *lens;
  float *lse, *weights;      // lse may be NULL
  // with weights, [ntok][Hq]: a row's log-sum-exp in base 2 as two terms, a score and the
  // rest.  Their sum in fp32 would be off by half an ulp of large scores.
  float2 *stats;
  uint32_t *status;
  kvx8::Requests req;
  Sharing share;
  int64_t wstride;
  int num_blocks, H, Hq, G, d, bs, max_blocks, max_len, max_new;
  int bf16;                    // the type of out
  uint32_t bs_mul, bs_shift;   // j / bs = j * bs_mul >> bs_shift for j < 2^31
  float c;   // scale * log2(e): scores are kept in base 2
};

}  // namespace kvx8

namespace {

using kvx8::AttendParams;

constexpr bool kShared = KVX_ATTEND_SHARED;

// A workspace begins with the split form's counters, which are zero between calls: where
// they lie and how many there are depends on no call's sizes, and no form uses these
// bytes for anything else, so that one workspace serves calls of different sizes and forms.
constexpr size_t kWorkspaceHead = 1024;

// Scores (base 2) beyond this are far: their own half ulp, 2^-12 here, counts in exponents
// that are their differences to an unrounded number.
constexpr float kFar = 4096.f;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The request's length (0 where it is out of bounds).
__device__ __forceinline__ int len_of(const AttendParams &p, int r) {
  const int n = __ldg(p.lens + r);
  return n < 0 || n > p.max_len ? 0 : n;
}
// The request's block that holds slot j: j / bs by a multiplication.
__device__ __forceinline__ uint32_t block_of(const AttendParams &p, int j) {
  return (uint32_t)((uint64_t)(uint32_t)j * p.bs_mul >> p.bs_shift);
}
// The pool's block of a request's block, or -1.
__device__ __forceinline__ int page_of(const AttendParams &p, int r, uint32_t block) {
  const int page = block < (uint32_t)p.max_blocks ? __ldg(p.table + (int64_t)r * p.max_blocks + block) : -1;
  return page < p.num_blocks ? page : -1;
}
// A request's first token, and behind the last request the end.  An entry of the groups that
// is no request gives -1, which no good table holds.
__device__ __forceinline__ int64_t begin_of(const AttendParams &p, int r) {
  if (kShared && p.share.all) {
    if (p.share.whole) return r ? p.req.ntok : 0;
    r = p.share.of[r];
    if (r < 0 || r > p.share.inner) return -1;
  }
  return p.req.begin(r);
}
// The last slot that query i of a request sees is first_limit + i * limit_step.
__device__ __forceinline__ int first_limit(const AttendParams &p, int len, int fresh) {
  return kShared && p.share.all ? len - 1 : len - fresh;
}
__device__ __forceinline__ int limit_step(const AttendParams &p) { return kShared && p.share.all ? 0 : 1; }
// Groups of requests start at 0, never decrease, end at the last request and have at most
// `most` tokens each (without a table all tokens are one group's): this thread's share of the
// check, in the pass over own slots.
__device__ __forceinline__ bool groups_ok(const AttendParams &p, int first, int stride) {
  bool good = true;
  if (kShared && p.share.whole) good = p.req.ntok <= p.share.most;
  if (kShared && !p.share.all && p.share.of)
    for (int i = first; i < p.share.count; i += stride) {
      const int a = p.share.of[i], b = p.share.of[i + 1];
      good = good && a >= 0 && b >= a && b <= p.req.R && (i > 0 || a == 0) && (i + 1 < p.share.count || b == p.req.R);
      if (good) good = p.req.begin(b) - p.req.begin(a) <= p.share.most;
    }
  return good;
}
__device__ __forceinline__ bool requests_ok(const AttendParams &p) {
  if (kShared) {
    bool good = groups_ok(p, threadIdx.x, blockDim.x);
    for (int r = threadIdx.x; r < p.req.R; r += blockDim.x) {
      const int64_t from = begin_of(p, r), to = begin_of(p, r + 1);
      good = good && to >= from && to - from <= p.max_new && (r > 0 || from == 0) && (r + 1 < p.req.R || to == p.req.ntok);
    }
    return __syncthreads_and(good);
  }
  bool good = p.req.ok();
  if (p.req.cu) {
    bool few = true;
    for (int r = threadIdx.x; good && r < p.req.R; r += blockDim.x)
      few = few && p.req.cu[r + 1] - p.req.cu[r] <= p.max_new;
    good = __syncthreads_and(good && few);
  }
  return good;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A row's two parts, one here (sum l relative to exp2(m + shift)) and one from before: the
// factors on their outputs and the log-sum-exp of both, in base 2 as two terms.
struct Joined {
  float own, before;
  float2 lse;
};
__device__ __forceinline__ Joined join_before(const AttendParams &p, int64_t g, int hq, float m, float shift, float l) {
  const float2 b = __ldcg(p.share.before_stats + g * p.Hq + hq);
  if (l == 0.f) return {0.f, b.y < INFINITY ? 1.f : 0.f, b};
  const float rest = shift + log2f(l);
  if (b.y == INFINITY) return {1.f, 0.f, make_float2(m, rest)};
  const float more = (b.x - m) + (b.y - rest), up = ex2(more), down = ex2(-more);   // differences first: exact where they count
  return {1.f / (1.f + up), 1.f / (1.f + down),
          more > 0.f ? make_float2(b.x, b.y + log2f(1.f + down)) : make_float2(m, rest + log2f(1.f + up))};
}
// The log-sum-exp of a row whose sum l is relative to exp2(m + shift).
__device__ __forceinline__ void store_lse(const AttendParams &p, int64_t g, int hq, float m, float shift, float l) {
  if (kShared && p.share.before) {
    const float2 both = join_before(p, g, hq, m, shift, l).lse;
    if (p.lse) p.lse[g * p.Hq + hq] = both.y == INFINITY ? -INFINITY : (both.x + both.y) * kLn2;
    return;
  }
  const bool any = l != 0.f;
  const float rest = shift + log2f(l);
  if (p.lse) p.lse[g * p.Hq + hq] = any ? (m + rest) * kLn2 : -INFINITY;
  if (p.stats) p.stats[g * p.Hq + hq] = any ? make_float2(m, rest) : make_float2(0.f, INFINITY);
}
// The probability of a score, rounded as the attention kernel rounded it.
__device__ __forceinline__ float probability(float score, float2 lse) { return ex2((score - lse.x) - lse.y); }
// Two dimensions of a finished row, whose sums o and l are relative to exp2(m + shift);
// its log-sum-exp with the first.
__device__ __forceinline__ void store_out(const AttendParams &p, int64_t g, int hq, int d, float2 o, float m,
                                          float shift, float l) {
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t to = g * p.ot + hq * p.oh + d;
  float2 y = make_float2(o.x * inv, o.y * inv);
  if (kShared && p.share.before) {
    const Joined j = join_before(p, g, hq, m, shift, l);
    const float2 b = __ldcg(reinterpret_cast<const float2 *>(p.share.before + (g * p.Hq + hq) * p.d + d));
    y = make_float2(y.x * j.own + b.x * j.before, y.y * j.own + b.y * j.before);
  }
  if (p.bf16) {
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.out) + to;
    out[0] = __float2bfloat16_rn(y.x);
    out[1] = __float2bfloat16_rn(y.y);
  } else {
    float *out = reinterpret_cast<float *>(p.out) + to;
    out[0] = y.x;
    out[1] = y.y;
  }
  if (d == 0) store_lse(p, g, hq, m, shift, l);
}

// The most queries that one request of the call can have: max_new may be any bound.
inline int most_new(const kvx_attend8_args *a) {
  return (int)(a->max_new < a->ntok ? a->max_new : a->ntok > 1 ? a->ntok : 1);
}

// Bytes of the scores of `rows` columns for every slot, request and KV head that a call
// keeps for the weights: at most kMostScores, or it forms them again.
constexpr uint64_t kMostScores = (uint64_t)4 << 30;
inline uint64_t score_bytes(const kvx_attend8_args *a, int64_t rows, int64_t slots) {
  const double b = 4.0 * a->num_requests * a->cache.heads * (double)rows * (double)slots;
  return b > (double)kMostScores ? kMostScores + 1
                                 : (uint64_t)a->num_requests * a->cache.heads * rows * slots * 4;
}

// A maximum to subtract: 0 before any score (exp2(-inf - 0) is 0; a NaN score stays NaN).
__device__ __forceinline__ float finite_or_0(float m) { return m > -INFINITY ? m : 0.f; }

}  // namespace

// kvx_attend8_tc.cu: bf16 queries and head_dim up to 128 over blocks of whole 8-slot
// groups; kvx_attend8_split.cu: all others.
bool kvx_attend8_tc_supports(const kvx_attend8_args *a);
// Of a workspace: the bytes that the call needs, and with those in which calls of at most
// its sizes can keep scores.
size_t kvx_attend8_tc_least_bytes(const kvx_attend8_args *a);
size_t kvx_attend8_tc_workspace_bytes(const kvx_attend8_args *a);
size_t kvx_attend8_split_least_bytes(const kvx_attend8_args *a);
size_t kvx_attend8_split_workspace_bytes(const kvx_attend8_args *a);
// The launches, for kvx_attend8 and for the passes of kvx_attend8_shared.
typedef kvx_status kvx_attend8_launch(const kvx_attend8_args *a, const kvx8::AttendParams &p, char *workspace, cudaStream_t s);
kvx_attend8_launch kvx_attend8_tc_launch, kvx_attend8_tc_launch_shared, kvx_attend8_split_launch, kvx_attend8_split_launch_shared;

// kvx_attend8_own.cu: the own slots of requests that share prefixes, few rows and not too
// many slots; and their prefixes, where they are not much work, in a number of parts.
bool kvx_attend8_own_supports(const kvx_attend8_args *a);
int kvx_attend8_parts(const kvx_attend8_args *before);
size_t kvx_attend8_parts_bytes(const kvx_attend8_args *before);
kvx_status kvx_attend8_own_launch(const kvx_attend8_args *a, const kvx8::AttendParams &p, int parts, void *part_bytes, bool prefixes,
                                  cudaStream_t s);
