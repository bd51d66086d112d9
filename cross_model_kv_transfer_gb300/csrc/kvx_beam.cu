// kvx_beam.cu -- beam search's selection over beams and vocabulary (kvx_beam_select).
//
//   score(k, v) = scores[k] + x_kv - log sum_u exp(x_ku)
// Of a beam's candidates only its N largest logits can be chosen, so one pass over a row
// finds those and the row's sum of exponentials, and the beams' lists are ranked after.
//
// A row is read by a cluster of one to eight CTAs, each a contiguous share of it, in
// chunks that the threads hold in registers.  Each warp's q-th largest of its lanes' largest
// logits, q = N / 8 rounded up, is exceeded or equalled by q logits; the least of the
// eight warps' is below N of the chunk, so only what is not below it, nor below the N-th of
// what was found before, can be among the N largest.  That goes to a list in
// shared memory, is ranked there with what was found before, and the first N stay.  Where
// too many logits are equal to the bound the threads' largest are ranked as 64-bit keys
// instead: at most N threads have anything not below the N-th of them.  Keys are
// the logit in an order-preserving form and behind it the falling position: no two are
// equal, so nothing depends on the order in which a list was filled.
//
// Sums of exponentials are relative to a thread's reference, which is raised to a chunk's
// maximum where that is more than kBehind above it: so the old sum is scaled a few times at
// most while it still counts, however often the maximum moves.  They are fp32 over a warp's
// elements and fp64 above (about as many additions as there are warps: fp64 is slow here);
// a thread's sum over its chunks carries the rest of each addition along.  Their error so
// does not grow with the row: 2^-16 of the sum is a bound for 2^31 logits (two roundings of
// each argument to fp32, seven exponentials of 2^-22, twenty roundings), 2^-22.7 to 2^-24 was
// measured for normal logits.  With each maximum a reference and plain fp32 sums 2,000,001
// logits of one CTA were off by up to 2^-16.9, now 2^-21 (256 rows of 151,936 take 52.9 us, 52.2 so).
//
// Bound by HBM where there are many rows, by the latency of a chunk's ranking (a few
// barriers) where there are few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kvx_cache8.cuh"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8, kMostBeams = 32;
constexpr float kLog2e = 1.4426950408889634f, kBehind = 8.f;

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
  int K, N, V, eos, ctas;        // CTAs a row
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
// As they lie in memory first, so that the next chunk's are on their way while one is
// worked on; those behind the end are -inf.
template <class T, int V, int E>
struct Raw {
  static constexpr int LOADS = E / V;
  typename std::conditional<V == 1, float, uint4>::type w[LOADS];
  __device__ __forceinline__ void load(const T *row, int64_t at, int end) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int64_t v = at + (j * kThreads + threadIdx.x) * V;
      if constexpr (V == 1) {
        w[j] = v < end ? (float)row[v] : -INFINITY;
      } else {
        // rows are whole loads: a load is in or out
        constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
        w[j] = v < end ? __ldcs(reinterpret_cast<const uint4 *>(row + v)) : make_uint4(none, none, none, none);
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[E]) const {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      if constexpr (V == 1) {
        x[j] = w[j];
      } else {
        const uint32_t b[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int k = 0; k < V; ++k)
          x[j * V + k] = __uint_as_float(sizeof(T) == 4 ? b[k % 4] : k % 2 ? b[k / 2 % 4] & 0xffff0000u : b[k / 2 % 4] << 16);
      }
    }
  }
};
// The sum of a thread's chunk relative to exp(m).
template <int E>
__device__ __forceinline__ float sum_of(const float (&x)[E], float m) {
  float s[4] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) s[e % 4] += ex2((x[e] - m) * kLog2e);
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// A chunk's elements, those gathered before it, and the best ones before those.
constexpr int kChunk = kMostBeams * 32, kGather = 128, kList = kGather + kChunk + kMostBeams;
struct RowShared {
  unsigned long long top[kThreads];
  unsigned long long list[kList];
  unsigned long long best[2][kMostBeams];
  unsigned long long bound;
  uint32_t warp_bound[kWarps];
  double total;                 // of the CTA, relative to exp(unit)
  float sum[kWarps], max[kWarps];
  float unit;
  int count[3], many, now;      // the list's, of a chunk that overflows; which of best is the last
};
// The first n of `count` keys, ranked, to `best` (0 behind the last); all threads call it.
__device__ __forceinline__ void rank_list(const unsigned long long *list, int count, unsigned long long *best, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (i >= count) best[i] = 0;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const unsigned long long key = list[i];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < count; ++j) above += list[j] > key;
    if (above < n) best[above] = key;
  }
}

// The chunk's list from ranked keys of the threads: where it overflows.  Apart from the
// loop, from the logits read again, so that it costs that no registers.
template <class T, int V, int E>
__device__ __noinline__ int list_by_keys(RowShared &sh, int gathered, int n, unsigned long long before, const T *row, int at, int end) {
  const int tid = threadIdx.x;
  Raw<T, V, E> raw;
  raw.load(row, at, end);
  float x[E];
  raw.values(x);
  const auto key = [&](int e) {
    return x[e] < INFINITY ? key_of(x[e] + 0.f, at + (e / V * kThreads + tid) * V + e % V) : 0ull;
  };
  unsigned long long mine = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) mine = max(mine, key(e));
  sh.top[tid] = mine;
  if (tid == 0) {
    sh.many = 0;
    sh.bound = 1;                   // fewer than N threads have anything: all of it counts
  }
  __syncthreads();
  int above = 0;
  for (int j = 0; j < kThreads; ++j) above += sh.top[j] > mine;
  if (mine && above == n - 1) sh.bound = mine;
  __syncthreads();
  const unsigned long long bound = sh.bound;
  if (mine >= bound)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const unsigned long long k = key(e);
      if (k >= bound && k > before) sh.list[gathered + atomicAdd(&sh.many, 1)] = k;
    }
  __syncthreads();
  return sh.many;
}

template <class T, int V, int E>
__global__ void __launch_bounds__(kThreads, 4) row_kernel(const __grid_constant__ BeamParams p) {
  static_assert(E <= 32, "the list holds 32 elements of each thread above the bound");
  __shared__ RowShared sh;
  wait_for_kernel_before();
  let_next_kernel_start();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rank = blockIdx.x % p.ctas, row = blockIdx.x / p.ctas;
  if (!lives(p, row)) {               // the whole cluster
    if (rank == 0 && tid == 0 && !(p.scores[row] < INFINITY)) raise(p.status, KVX_FLAG_NOT_FINITE);
    if (rank == 0 && tid < p.N) p.keys[(int64_t)row * p.N + tid] = 0;
    return;
  }
  const T *x_of = reinterpret_cast<const T *>(p.logits) + row * p.stride;
  // the CTA's share of the row, in whole loads
  const int64_t loads = (p.V + V - 1) / V;
  const int begin = (int)(loads * rank / p.ctas * V), end = (int)min((int64_t)p.V, loads * (rank + 1) / p.ctas * V);
  float unit = -INFINITY, sum = 0.f, rest = 0.f;  // the thread's sum, relative to exp(unit)
  int now = 0;
  const int rounds = (p.N + kWarps - 1) / kWarps;
  if (tid < kMostBeams) sh.best[0][tid] = 0;
  if (tid == 0) sh.count[0] = 0;
  // two to a register, the next chunk's logits are on their way while one is worked on; of
  // fp32 ones other CTAs of the SM have theirs
  constexpr bool kAhead = sizeof(T) == 2 && V > 1;
  Raw<T, V, E> next;
  if (kAhead) next.load(x_of, begin, end);
  // What is not below `bound`, and whose key is above `before`, is gathered from chunk to
  // chunk and ranked when it has become many, or at the end.
  float bound = -INFINITY;
  unsigned long long before = 0;
  int turn = 0, gathered = 0;
  const auto rank_gathered = [&] {
    const unsigned long long old = tid < p.N ? sh.best[now][tid] : 0;
    if (old) sh.list[gathered + tid] = old;      // they are at the front of best
    const int held = __syncthreads_count(old != 0);
    rank_list(sh.list, gathered + held, sh.best[now ^ 1], p.N);
    now ^= 1;
    gathered = 0;
    __syncthreads();
    before = sh.best[now][p.N - 1];
    if (before) bound = fmaxf(bound, logit_of(before));
  };
  for (int64_t at = begin; at < end; at += kThreads * E, turn = turn == 2 ? 0 : turn + 1) {
    float x[E];
    if (!kAhead) next.load(x_of, at, end);
    next.values(x);
    if (kAhead) next.load(x_of, at + kThreads * E, end);
    float top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
    // 0 before any logit
    const auto reference = [&] { return top > unit + kBehind ? top : unit > -INFINITY ? unit : 0.f; };
    float more = sum_of<E>(x, reference());
    if (!(top < INFINITY) || !(more < INFINITY)) {
      // a NaN or an infinity: they become -inf
      raise(p.status, KVX_FLAG_NOT_FINITE);
      top = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] = x[e] < INFINITY ? x[e] : -INFINITY;
        top = fmaxf(top, x[e]);
      }
      more = sum_of<E>(x, reference());
    }
    if (top > unit + kBehind) {
      const float down = ex2((unit - top) * kLog2e);
      sum *= down;
      rest *= down;
      unit = top;
    }
    const float both = __fadd_rn(sum, more), part = __fsub_rn(both, sum);
    rest += __fsub_rn(sum, __fsub_rn(both, part)) + __fsub_rn(more, part);
    sum = both;
    if (at == begin) {                // what the warps agree on
      uint32_t left = top > -INFINITY ? ordered(top + 0.f) : 0u, least = 0;
      for (int i = 0; i < rounds; ++i) {
        least = __reduce_max_sync(~0u, left);
        left = left == least ? 0u : left;
      }
      if (lane == 0) sh.warp_bound[warp] = least;
      __syncthreads();
      least = ~0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) least = min(least, sh.warp_bound[w]);
      if (least) bound = logit_of((unsigned long long)least << 32);
    }
    const auto position = [&](int e) { return (int)at + (e / V * kThreads + tid) * V + e % V; };
    if (top >= bound) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x[e] >= bound) {
          const unsigned long long key = key_of(x[e] + 0.f, position(e));   // -0 and 0 are equal
          if (key > before) {
            const int to = atomicAdd(&sh.count[turn], 1);
            if (to < kChunk) sh.list[gathered + to] = key;
          }
        }
    }
    // three counts in turn: this chunk's, the next one's, and one that a thread may still read
    if (tid == 0) sh.count[turn == 2 ? 0 : turn + 1] = 0;
    __syncthreads();
    const int found = sh.count[turn];
    gathered += found <= kChunk ? found : list_by_keys<T, V, E>(sh, gathered, p.N, before, x_of, (int)at, end);
    if (gathered > kGather) rank_gathered();
  }
  if (gathered) rank_gathered();
  // the CTA's sum
  float top = unit;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  float part = unit > -INFINITY ? (sum + rest) * ex2((unit - top) * kLog2e) : 0.f;
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
    for (int w = 0; w < kWarps; ++w) total += top > -INFINITY ? (double)(sh.sum[w] * ex2((sh.max[w] - top) * kLog2e)) : 0.0;
    sh.total = total;
    sh.unit = top;
    sh.now = now;
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
    const int n = p.ctas * p.N;
    if (tid < n) {
      const int c = tid / p.N;
      sh.list[tid] = load64(remote(&sh.best[load32(remote(&sh.now, c))][tid % p.N], c));
    }
    if (tid == kThreads - 1) {        // not one of the others' warps, mostly
      float tops[kCluster], top = -INFINITY;
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        tops[c] = c < p.ctas ? __uint_as_float(load32(remote(&sh.unit, c))) : -INFINITY;
        top = fmaxf(top, tops[c]);
      }
      double total = 0.0;
#pragma unroll
      for (int c = 0; c < kCluster; ++c)
        if (c < p.ctas && tops[c] > -INFINITY) total += __longlong_as_double(load64(remote(&sh.total, c))) * (double)ex2((tops[c] - top) * kLog2e);
      p.lse[row] = (double)top + log(total);
    }
    __syncthreads();
    // ranked among each other; the 0s of short lists stay behind
    unsigned long long *to = p.keys + (int64_t)row * p.N;
    const unsigned long long key = tid < n ? sh.list[tid] : 0;
    int above = 0, some = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      above += sh.list[j] > key;
      some += sh.list[j] != 0;
    }
    if (key && above < p.N) to[above] = key;
    if (tid >= some && tid < p.N) to[tid] = 0;
  }
  cluster_barrier();                  // shared memory of the others is read until here
}

// A score as a number of the same order; 0 is below all of them.
__device__ __forceinline__ unsigned long long ordered(double x) {
  const long long b = __double_as_longlong(x + 0.0);
  return (unsigned long long)b ^ ((unsigned long long)(b >> 63) | 1ull << 63);
}
__device__ __forceinline__ double score_of(unsigned long long k) {
  return __longlong_as_double((long long)(k ^ (k >> 63 ? 1ull << 63 : ~0ull)));
}
constexpr int kEach = kMostBeams * kMostBeams / kThreads;     // candidates a thread
struct PickShared {
  unsigned long long list[kMostBeams * kMostBeams];
  int place[kMostBeams * kMostBeams], count;
  uint32_t warp_bound[kWarps];
};
// Candidate i = k * N + j of a request: the j-th of beam k.  In that order equal scores
// go to the lower beam, and in a beam to the larger logit, then the lower token.  The list is bounded as a chunk's is, by the scores'
// upper halves, and has room for all.
__global__ void __launch_bounds__(kThreads) pick_kernel(const __grid_constant__ BeamParams p) {
  __shared__ PickShared sh;
  wait_for_kernel_before();
  const int tid = threadIdx.x, b = blockIdx.x, all = p.K * p.N;
  unsigned long long x[kEach];
  uint32_t top = 0, bound = ~0u;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    // beams side by side, so that each warp has some of all
    const int c = e * kThreads + tid, k = c % p.K, j = c / p.K, row = b * p.K + k;
    x[e] = 0;
    if (c >= all) continue;
    const float score = p.scores[row];
    if (p.done && p.done[row]) {
      if (j == 0 && fabsf(score) < INFINITY) x[e] = ordered((double)score);
    } else {
      const unsigned long long key = __ldcg(p.keys + (int64_t)row * p.N + j);
      if (key) x[e] = ordered((double)score + ((double)logit_of(key) - __ldcg(p.lse + row)));
    }
    top = max(top, (uint32_t)(x[e] >> 32));
  }
  const int rounds = (p.N + kWarps - 1) / kWarps;
  uint32_t least = 0;
  for (int i = 0; i < rounds; ++i) {
    least = __reduce_max_sync(~0u, top);
    top = top == least ? 0u : top;
  }
  if (tid % 32 == 0) sh.warp_bound[tid / 32] = least;
  if (tid == 0) sh.count = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) bound = min(bound, sh.warp_bound[w]);
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (x[e] && (uint32_t)(x[e] >> 32) >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      sh.list[at] = x[e];
      const int c = e * kThreads + tid;
      sh.place[at] = c % p.K * p.N + c / p.K;
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
  for (int k = tid; k < n; k += kThreads) {
    const unsigned long long s = sh.list[k];
    const int i = sh.place[k], row = b * p.K + i / p.N;
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {     // no branches: n steps of a few instructions each
      const unsigned long long other = sh.list[j];
      above += (int)(other > s) | ((int)(other == s) & (int)(sh.place[j] < i));
    }
    if (above < p.N)
      put(above, p.done && p.done[row] ? p.eos : token_of(__ldcg(p.keys + (int64_t)row * p.N + i % p.N)), row,
          (float)score_of(s));
  }
}

// CTAs a row: as many as fill the GPU, up to four CTAs an SM, while each has a chunk.
int ctas_of(int64_t rows, int64_t vocab) {
  int c = 1;
  while (c < kCluster && rows * c * 2 <= 152 * 4 && vocab > (int64_t)c * 2048) c *= 2;
  return c;
}
template <class T, int V, int E>
kvx_status launch_rows(const BeamParams &p, int64_t rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * p.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, row_kernel<T, V, E>, p) == cudaSuccess ? KVX_OK : KVX_ERR_CUDA;
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
      !aligned_to(a->scores, 4) || !aligned_to(a->tokens, 4) || !aligned_to(a->parents, 4) || !aligned_to(a->new_scores, 4) ||
      !a->workspace ||
      !aligned_to(a->workspace, 256) || a->workspace_bytes < kvx_beam_workspace_bytes(a))
    return KVX_ERR_INVALID_ARG;
  const int rows = a->num_requests * a->beams;
  // results are written while other CTAs still read the scores
  const int64_t chosen = (int64_t)a->num_requests * a->out_beams;
  if (overlap(a->scores, rows, a->new_scores, chosen) || (a->done && a->new_done && overlap(a->done, rows, a->new_done, chosen, 1)))
    return KVX_ERR_INVALID_ARG;
  BeamParams p = {a->logits, a->row_stride, a->scores, a->done,   a->tokens,    a->parents, a->new_scores, a->new_done, a->status,
                  nullptr,   nullptr,       a->beams,  a->out_beams, a->vocab, a->eos, 1};
  p.keys = (unsigned long long *)a->workspace;
  p.lse = (double *)((char *)a->workspace + up256((size_t)rows * a->out_beams * 8));
  // loads of 16 bytes where rows begin on such a boundary and the last one stays inside
  // its row's stride
  const int per = 16 / size;
  const bool vec = aligned_to(a->logits, 16) && a->row_stride % per == 0 && a->vocab % per == 0;
  cudaStream_t s = (cudaStream_t)stream;
  p.ctas = ctas_of(rows, a->vocab);
  const kvx_status st = size == 4 ? (vec ? launch_rows<float, 4, 32>(p, rows, s) : launch_rows<float, 1, 16>(p, rows, s))
                                  : (vec ? launch_rows<__nv_bfloat16, 8, 32>(p, rows, s) : launch_rows<__nv_bfloat16, 1, 16>(p, rows, s));
  if (st != KVX_OK) return st;
  return launch_after(pick_kernel, dim3((unsigned)a->num_requests), kThreads, 0, s, p);
}
