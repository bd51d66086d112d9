// kvx_beam.cu -- beam search's selection over beams and vocabulary (kvx_beam_select).
//
//   score(k, v) = scores[k] + x_kv - log sum_u exp(x_ku)
// Of a beam's candidates only its N largest logits can be chosen, so one pass over a row
// finds those and the row's sum of exponentials, and the beams' lists are ranked after.
//
// A row is read by a cluster of eight CTAs, each a contiguous share of it, in chunks
// that the threads hold in registers.  The largest logit of each thread is ranked among
// the CTA's: the N-th of them bounds the chunk's N-th largest from below, and at most N
// threads have anything above it.  What lies above goes to a list in shared memory, is
// ranked there with the N that were found before, and the first N stay.  Keys are 64 bits, the
// logit in an order-preserving form and behind it the falling position: no two are equal,
// so nothing depends on the order in which a list was filled.  Sums are fp32 over a
// thread's elements, relative to its running maximum, fp64 over threads and CTAs.
//
// Bound by HBM where there are many rows, by the latency of a chunk's ranking (a few
// barriers) where there are few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_cache8.cuh"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8, kMostBeams = 32;
constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
  const void *logits;
  int64_t stride;
  const float *scores;
  const uint8_t *done;
  int32_t *tokens, *parents;
  float *new_scores;
  uint8_t *new_done;
  uint32_t *status;
  // what the rows' clusters leave: keys, falling, 0 behind the last; log-sum-exps
  unsigned long long *keys;      // [B * K][N]
  double *lse;                   // [B * K]
  int K, N, V, eos;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A finite logit as a number of the same order; 0 is below all of them.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(unsigned long long key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float(b ^ (b >> 31 ? 0x80000000u : ~0u));
}
__device__ __forceinline__ unsigned long long key_of(float x, int v) {
  return x > -INFINITY ? (unsigned long long)ordered(x) << 32 | (uint32_t)~v : 0ull;
}
__device__ __forceinline__ int token_of(unsigned long long key) { return (int)~(uint32_t)key; }

// Does the beam have candidates from its logits?
__device__ __forceinline__ bool lives(const BeamParams &p, int row) {
  return p.scores[row] > -INFINITY && p.scores[row] < INFINITY && !(p.done && p.done[row]);
}

// E logits a thread and chunk, V a load.  Position of element j * V + k: j * 256 V + V t + k.
template <class T, int V, int E>
__device__ __forceinline__ void load_chunk(const T *row, int at, int end, float (&x)[E], bool &odd) {
#pragma unroll
  for (int j = 0; j < E / V; ++j) {
    const int v = at + (j * kThreads + threadIdx.x) * V;
    float y[V];
    if constexpr (V == 1) {
      y[0] = v < end ? (float)row[v] : -INFINITY;
    } else {
      // rows are whole loads: a load is in or out
      const uint4 w = v < end ? __ldcs(reinterpret_cast<const uint4 *>(row + v)) : make_uint4(0, 0, 0, 0);
      const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < V; ++k)
        y[k] = sizeof(T) == 4 ? __uint_as_float(b[k % 4]) : __uint_as_float(k % 2 ? b[k / 2 % 4] & 0xffff0000u : b[k / 2 % 4] << 16);
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] = v + k < end ? y[k] : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const bool bad = !(y[k] < INFINITY);
      odd = odd || bad;
      x[j * V + k] = bad ? -INFINITY : y[k] + 0.f;     // -0 and 0 are equal
    }
  }
}

struct RowShared {
  unsigned long long top[kThreads];
  unsigned long long list[kMostBeams * 32 + kMostBeams];
  unsigned long long best[2][kMostBeams];
  unsigned long long bound;
  double sum[kWarps];
  float max[kWarps];
  double total;                 // of the CTA, relative to most
  float most;
  int count;
};
// The first n of `count` keys, ranked, to `best` (0 behind the last); all threads call it.
__device__ __forceinline__ void rank_list(const unsigned long long *list, int count, unsigned long long *best, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (i >= count) best[i] = 0;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const unsigned long long key = list[i];
    int above = 0;
    for (int j = 0; j < count; ++j) above += list[j] > key;
    if (above < n) best[above] = key;
  }
}

template <class T, int V, int E>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    row_kernel(const __grid_constant__ BeamParams p) {
  static_assert(E <= 32, "the list holds 32 elements of each thread above the bound");
  __shared__ RowShared sh;
  wait_for_kernel_before();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rank = blockIdx.x % kCluster, row = blockIdx.x / kCluster;
  if (!lives(p, row)) {               // the whole cluster
    if (rank == 0 && tid == 0 && !(p.scores[row] < INFINITY)) raise(p.status, KVX_FLAG_NOT_FINITE);
    if (rank == 0 && tid < p.N) p.keys[(int64_t)row * p.N + tid] = 0;
    return;
  }
  const T *x_of = reinterpret_cast<const T *>(p.logits) + row * p.stride;
  // the CTA's share of the row, in whole loads
  const int64_t loads = (p.V + V - 1) / V;
  const int begin = (int)(loads * rank / kCluster * V), end = (int)min((int64_t)p.V, loads * (rank + 1) / kCluster * V);
  float most = -INFINITY, sum = 0.f;
  bool odd = false;
  int now = 0;
  if (tid < kMostBeams) sh.best[0][tid] = 0;
  for (int64_t at = begin; at < end; at += kThreads * E) {
    float x[E];
    load_chunk<T, V, E>(x_of, (int)at, end, x, odd);
    float top = x[0];
    int where = 0;
#pragma unroll
    for (int e = 1; e < E; ++e) {
      where = x[e] > top ? e : where;
      top = fmaxf(top, x[e]);
    }
    if (top > most) {
      sum *= ex2((most - top) * kLog2e);
      most = top;
    }
    if (most > -INFINITY) {
#pragma unroll
      for (int e = 0; e < E; ++e) sum += ex2((x[e] - most) * kLog2e);
    }
    const auto position = [&](int e) { return (int)at + (e / V * kThreads + tid) * V + e % V; };
    const unsigned long long mine = key_of(top, position(where));
    sh.top[tid] = mine;
    if (tid == 0) {
      sh.count = 0;
      sh.bound = 1;                   // fewer than N threads have anything: all of it counts
    }
    __syncthreads();
    // the bound: the N-th largest of the threads' keys, or of those found so far
    int above = 0;
    if (mine) {
#pragma unroll 8
      for (int j = 0; j < kThreads; ++j) above += sh.top[j] > mine;
      if (above == p.N - 1) sh.bound = mine;
    }
    __syncthreads();
    const unsigned long long before = sh.best[now][p.N - 1], bound = before > sh.bound ? before : sh.bound;
    if (mine >= bound) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const unsigned long long key = key_of(x[e], position(e));
        if (key >= bound) sh.list[atomicAdd(&sh.count, 1)] = key;
      }
    }
    if (tid < p.N && sh.best[now][tid]) sh.list[atomicAdd(&sh.count, 1)] = sh.best[now][tid];
    __syncthreads();
    rank_list(sh.list, sh.count, sh.best[now ^ 1], p.N);
    now ^= 1;
    __syncthreads();
  }
  if (odd) raise(p.status, KVX_FLAG_NOT_FINITE);
  // the CTA's sum
  float top = most;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  double part = most > -INFINITY ? (double)sum * exp((double)most - (double)top) : 0.0;
#pragma unroll
  for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(~0u, part, o);
  if (lane == 0) {
    sh.max[warp] = top;
    sh.sum[warp] = part;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.max[w]);
    double total = 0.0;
    for (int w = 0; w < kWarps; ++w)
      if (sh.max[w] > -INFINITY) total += sh.sum[w] * exp((double)sh.max[w] - (double)top);
    sh.total = total;
    sh.most = top;
  }
  // the cluster's: the first CTA ranks the lists of all
  const auto cluster_barrier = [] {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  const auto remote = [](const void *mine, int rank) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    return there;
  };
  const auto load64 = [](uint32_t a) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
  };
  const auto load32 = [](uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
  };
  cluster_barrier();
  if (rank == 0) {
    // which of the two lists is the last depends on the chunks of a CTA
    const auto now_of = [&](int64_t c) {
      const int64_t from = loads * c / kCluster * V, to = min((int64_t)p.V, loads * (c + 1) / kCluster * V);
      return (int)((to - from + kThreads * E - 1) / (kThreads * E) & 1);
    };
    for (int i = tid; i < kCluster * p.N; i += kThreads) {
      const int c = i / p.N;
      sh.list[i] = load64(remote(&sh.best[now_of(c)][i % p.N], c));
    }
    if (tid == 0) {
      float tops[kCluster], top = -INFINITY;
      for (int c = 0; c < kCluster; ++c) {
        tops[c] = __uint_as_float(load32(remote(&sh.most, c)));
        top = fmaxf(top, tops[c]);
      }
      double total = 0.0;
      for (int c = 0; c < kCluster; ++c)
        if (tops[c] > -INFINITY) total += __longlong_as_double(load64(remote(&sh.total, c))) * exp((double)tops[c] - (double)top);
      p.lse[row] = (double)top + log(total);
    }
    __syncthreads();
    // ranked among each other; the 0s of short lists stay behind
    unsigned long long *to = p.keys + (int64_t)row * p.N;
    const int n = kCluster * p.N;
    const unsigned long long key = tid < n ? sh.list[tid] : 0;
    int above = 0, some = 0;
    for (int j = 0; j < n; ++j) {
      above += sh.list[j] > key;
      some += sh.list[j] != 0;
    }
    if (key && above < p.N) to[above] = key;
    if (tid >= some && tid < p.N) to[tid] = 0;
  }
  cluster_barrier();                  // shared memory of the others is read until here
}

// Candidate i = k * N + j of a request: the j-th of beam k.  In that order equal scores
// go to the lower beam and token.
struct PickShared {
  double top[kThreads];
  int place[kThreads];
  double list[kMostBeams * (kMostBeams * kMostBeams / kThreads)];
  int list_place[kMostBeams * (kMostBeams * kMostBeams / kThreads)];
  double bound;
  int bound_place, count;
};
constexpr double kNone = -INFINITY;
// a before b?
__device__ __forceinline__ bool first(double a, int at, double b, int bt) { return a > b || (a == b && at < bt); }
__global__ void __launch_bounds__(kThreads) pick_kernel(const __grid_constant__ BeamParams p) {
  constexpr int kEach = kMostBeams * kMostBeams / kThreads;
  __shared__ PickShared sh;
  wait_for_kernel_before();
  const int tid = threadIdx.x, b = blockIdx.x, all = p.K * p.N;
  double x[kEach], top = kNone;
  int place = INT32_MAX;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + tid;
    x[e] = kNone;
    if (i >= all) continue;
    const int row = b * p.K + i / p.N;
    const float score = p.scores[row];
    const bool over = p.done && p.done[row];
    if (over) {
      if (i % p.N == 0 && score < INFINITY) x[e] = score;
    } else {
      const unsigned long long key = __ldcg(p.keys + (int64_t)row * p.N + i % p.N);
      if (key) x[e] = (double)score + ((double)logit_of(key) - __ldcg(p.lse + row));
    }
    if (x[e] > top) {
      top = x[e];
      place = i;
    }
  }
  sh.top[tid] = top;
  sh.place[tid] = place;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = kNone;
    sh.bound_place = INT32_MAX;
  }
  __syncthreads();
  if (top > kNone) {
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kThreads; ++j) above += first(sh.top[j], sh.place[j], top, place);
    if (above == p.N - 1) {
      sh.bound = top;
      sh.bound_place = place;
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + tid;
    if (x[e] > kNone && !first(sh.bound, sh.bound_place, x[e], i)) {
      const int at = atomicAdd(&sh.count, 1);
      sh.list[at] = x[e];
      sh.list_place[at] = i;
    }
  }
  __syncthreads();
  const int n = sh.count;
  const auto put = [&](int to, int token, int parent, float score) {
    const int64_t at = (int64_t)b * p.N + to;
    p.tokens[at] = token;
    p.parents[at] = parent;
    p.new_scores[at] = score;
    if (p.new_done) p.new_done[at] = token >= 0 && token == p.eos;
  };
  if (tid < p.N && tid >= n) put(tid, -1, -1, -INFINITY);
  if (tid < n) {
    const double s = sh.list[tid];
    const int i = sh.list_place[tid], row = b * p.K + i / p.N;
    int above = 0;
    for (int j = 0; j < n; ++j) above += first(sh.list[j], sh.list_place[j], s, i);
    if (above < p.N)
      put(above, p.done && p.done[row] ? p.eos : token_of(__ldcg(p.keys + (int64_t)row * p.N + i % p.N)), row, (float)s);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool sizes_ok(const kvx_beam_args *a) {
  return a && (a->dtype == KVX_F32 || a->dtype == KVX_BF16) && a->num_requests >= 0 && a->beams >= 1 && a->beams <= kMostBeams &&
         a->out_beams >= 1 && a->out_beams <= kMostBeams && a->vocab >= 1 && a->vocab <= INT32_MAX - 65536 &&
         (int64_t)a->num_requests * a->beams <= INT32_MAX / kCluster && a->eos >= -1 && a->eos < a->vocab;
}

}  // namespace

extern "C" size_t kvx_beam_workspace_bytes(const kvx_beam_args *a) {
  if (!sizes_ok(a)) return 0;
  const size_t rows = (size_t)a->num_requests * a->beams;
  return up256(rows * a->out_beams * 8) + up256(rows * 8) + 256;
}

extern "C" kvx_status kvx_beam_select(const kvx_beam_args *a, void *stream) {
  if (!sizes_ok(a)) return KVX_ERR_INVALID_ARG;
  if (a->done && a->eos < 0) return KVX_ERR_INVALID_ARG;
  if (a->num_requests == 0) return KVX_OK;
  const int size = a->dtype == KVX_BF16 ? 2 : 4;
  if (!a->logits || !aligned_to(a->logits, size) || !a->scores || !a->tokens || !a->parents || !a->new_scores ||
      a->new_scores == a->scores || (a->new_done && a->new_done == a->done) || !a->workspace ||
      !aligned_to(a->workspace, 256) || a->workspace_bytes < kvx_beam_workspace_bytes(a))
    return KVX_ERR_INVALID_ARG;
  const int rows = a->num_requests * a->beams;
  BeamParams p = {a->logits, a->row_stride, a->scores, a->done,   a->tokens,    a->parents, a->new_scores, a->new_done, a->status,
                  nullptr,   nullptr,       a->beams,  a->out_beams, a->vocab, a->eos};
  p.keys = (unsigned long long *)a->workspace;
  p.lse = (double *)((char *)a->workspace + up256((size_t)rows * a->out_beams * 8));
  // loads of 16 bytes where rows begin on such a boundary and the last one stays inside
  // its row's stride
  const int per = 16 / size;
  const bool vec = aligned_to(a->logits, 16) && a->row_stride % per == 0 && a->vocab % per == 0;
  cudaStream_t s = (cudaStream_t)stream;
  const dim3 grid((unsigned)rows * kCluster);
  const kvx_status st =
      size == 4 ? (vec ? launch_after(row_kernel<float, 4, 32>, grid, kThreads, 0, s, p)
                       : launch_after(row_kernel<float, 1, 16>, grid, kThreads, 0, s, p))
                : (vec ? launch_after(row_kernel<__nv_bfloat16, 8, 32>, grid, kThreads, 0, s, p)
                       : launch_after(row_kernel<__nv_bfloat16, 1, 16>, grid, kThreads, 0, s, p));
  if (st != KVX_OK) return st;
  return launch_after(pick_kernel, dim3((unsigned)a->num_requests), kThreads, 0, s, p);
}
