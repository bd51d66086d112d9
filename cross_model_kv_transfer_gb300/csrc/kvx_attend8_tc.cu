// kvx_attend8_tc.cu -- attention over the 8-bit cache on tcgen05 tensor cores:
// bf16 queries, head_dim up to 128 (fewer dimensions lie in tiles of 128 whose
// others are zero), blocks of whole 8-slot groups.
//
// Rows are the (query, head of the group) pairs of one request and KV head, 128
// to a tile; slots come 128 to a tile by TMA from the paged codes.
//   S = Q K^T   kind::f8f6f4: the codes as they lie in the cache; a query row,
//               scaled by a power of two to a largest element in (224, 448], is
//               the sum of two e4m3 parts (4 + 4 bits: a bf16 element exactly,
//               down to 1/896 of the row's largest, below that to 2^-17.8 of it:
//               the second part's step is 2^-9),
//   O += P V    kind::f16: P in f16 from tensor memory (it overwrites S), V
//               converted to f16 in shared memory with its block's scale.
// Softmax statistics are fp32, a row to a thread: no exchange between threads.
// The maximum that is subtracted follows the running one lazily: P holds up to
// 2^8 times what it would with the true one before the sums are scaled down.
//
// Roles: warps 0-3 and 4-7 two softmax groups, warps 8-11 convert V, warp 12
// loads (block lookups, scales, TMA), warps 13 and 14 issue the groups' MMAs.  WIDE: the groups
// take the two 128-row halves of 256 rows, over the same slot tiles.  Narrow
// (at most 64 rows): they take the even and the odd slot tiles of the same
// rows, so that one tile's softmax overlaps the other's products.
//
// What it reaches.  Wide, one request of 8192 tokens, 64 heads: 1070 us, 1.03
// PFLOP/s of the two products counted once, 0.52 of what bf16 matrix products reach;
// counters have the tensor pipe active 0.45 of the time and the schedulers issuing
// 0.55 of it: bound by the two groups' chain of score product, softmax and value
// product.  (Score products in half tiles of 64 columns run at 0.6 of their rate at
// 128, but whole tiles leave a group nothing to do while they are formed: 1397 us
// where half tiles took 1217.)  61 tokens of 32 heads against 8192 slots, two
// requests: 45 us, 16 to join what 152 CTAs left, 26 for the weights; about a third
// of that fills and drains pipelines.
//
// Work: every CTA takes an equal share of all steps and item costs (below); what
// several CTAs did of an item is joined by a second kernel.
//
// Every wait is bounded: after 2 s without progress the CTA sets
// KVX_FLAG_TIMEOUT, all roles leave, copies and MMAs in flight are drained and
// tensor memory is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <type_traits>

#include "kvx_attend8.cuh"
#include "kvx_ptx.cuh"

namespace {

constexpr int kD = 128;             // dimensions of a tile
constexpr int kTile = 128;          // slots and rows of a tile
constexpr int kHalf = kTile / 2;   // slots whose scores and products are formed at a time
constexpr int kTileBytes = kTile * kD;
// narrow: a stage must serve one group only, whose waits on it then know that the
// phase before is over
constexpr int kMaxKStages = 4, kVStages = 2, kWStages = 2;
template <bool WIDE>
constexpr int kStagesOf = WIDE ? 3 : 4;
constexpr int kLoadWarp = 12, kMmaWarp = 13, kThreads = 16 * 32;
// registers a thread: 8 softmax warps, 4 that convert, 4 others; together the
// launch's 512 x 128
constexpr int kSoftmaxRegs = 184, kConvertRegs = 80, kOtherRegs = 64;
static_assert(256 * kSoftmaxRegs + 128 * (kConvertRegs + kOtherRegs) == kThreads * 128, "register split");
constexpr uint64_t kWaitNs = 2000000000ull;
// P carries 2^7 so that f16 keeps probabilities down to 2^-31 of the
// subtracted maximum's; with the lazy 2^8 that is at most 2^15
constexpr float kBias = 7.f, kSlack = 8.f;

struct TcWalk {
  int r, len, fresh, groups, h, group, steps, step;   // step: the CTA's first of the item
  int64_t beg, base;
};
struct Share {
  TcWalk w;                // its first item
  int64_t T, N, last;      // all places, CTAs at work, the place at which it ends
  bool good;               // the request table is
};

struct TcShared {
  uint64_t k_full[kMaxKStages], k_empty[kMaxKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t w_full[kWStages], w_empty[kWStages];
  // [group][half of the tile]; a wait on one names a phase whose predecessor is
  // known to be over, so its parity is enough
  uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2];
  uint64_t join, spent, drain[2];
  uint32_t tmem_base;
  volatile int abort;
  Share share;
  // the tile's largest value scale, as a power of two: its exponent for the
  // softmax, 2^7 over it for the conversion
  float k_ref[kMaxKStages], v_unit[kVStages];
  uint32_t k_mask[kMaxKStages], v_mask[kVStages];   // bit l: slots 4l .. 4l + 3 lie in a block of the pool
  // scales, one for four slots (which lie in one block)
  __align__(16) float ks[kMaxKStages][kTile / 4];
  __align__(16) float vs[kVStages][kTile / 4];
};
constexpr size_t kSmemQ = 4 * (size_t)kTileBytes;     // two tiles of two parts; narrow one
template <bool WIDE>
constexpr size_t smem_bytes() {
  return 1024 + (WIDE ? kSmemQ : kSmemQ / 2) + (kStagesOf<WIDE> + kVStages) * (size_t)kTileBytes +
         kWStages * 2 * (size_t)kTileBytes + sizeof(TcShared);
}
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory");

// Where CTA x begins inside an item that CTA x - 1 began: what to join.
struct Split {
  int r, h, group, c0, ctas, rows;   // ctas 0: nothing
  int64_t beg;
};
struct TcParams {
  AttendParams a;
  int grid;            // CTAs that share the work
  Split *splits;       // [grid]
  float *partial;      // [2 * grid][PARTS][part_size]: sums [rows][kD], maxima, their shifts, totals
  float *scores;       // base 2, or NULL; narrow: [R][H][rows][score_ld], columns: [R][H][score_ld][slot_rows]
  int score_ld, slot_rows, part_size;   // rows kept of a part (narrow: G * max_new), its floats
  int box;             // slots of one TMA box
  int vec_q, vec_out;
};

template <class S>
struct WaiterT {
  S *sh;
  uint32_t *status;
  __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
    const uint32_t a = smem_addr(bar);
    if (mbar_try_wait(a, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t spin = 1;; ++spin) {
      if (mbar_try_wait(a, parity)) return true;
      if (spin % 64) continue;          // the clock is slow to read
      if (sh->abort) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitNs) {
        sh->abort = 1;
        raise(status, KVX_FLAG_TIMEOUT);
        return false;
      }
    }
  }
  __device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) const {
    return __all_sync(~0u, wait(bar, parity)) != 0;
  }
};
using Waiter = WaiterT<TcShared>;
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(smem_addr(bar), parity) && globaltimer() - t0 < kWaitNs) {
  }
}

// --- the flattened work ---------------------------------------------------------
// For each request, KV head and group of rows an item: steps of one or two slot
// tiles up to the last slot that its rows see.  An item costs its steps and a fixed
// part (queries, a filling and draining pipeline, the result), so the CTAs' shares
// are of costs: an item takes SETUP + steps places from `base` on, and its step s
// is at place base + SETUP + s.  Measured, us, with SETUP as given: wide 5, 6, 7, 8, 9: a
// prompt of 8192 tokens 1133, 1082, 1070, 1079, 1089, one of 2048 158, 157, 154, 159, 147,
// 128 rows each of 16 requests of 1024 to 16,384 slots 168, 163, 161, 161, 163.  The same
// requests narrow 2, 3, 4, 5, 6: 24 rows 152, 145, 147, 152, 155, 40 rows 168, 157, 152, 153,
// 156, 64 rows 193, 180, 167, 161, 156; columns 1, 2, 3, 4: 8 rows 84, 74, 73, 72, 16 rows 136,
// 108, 101, 95.
struct Wide {
  static constexpr int ROWS = 2 * kTile, SLOTS = kTile;   // of an item, of a step
  static constexpr int PARTS = 1;                         // results that a CTA keeps for an item
  static constexpr int SETUP = 7;
};
// Few columns (kernel further down): rows are the columns of S^T.
template <int NC>
struct Columns {
  static constexpr int ROWS = NC, SLOTS = 2 * kTile, PARTS = 2, SETUP = 4;
};
struct Narrow {
  static constexpr int ROWS = kTile, SLOTS = 2 * kTile, PARTS = 2, SETUP = 4;
};
template <class G>
__device__ __forceinline__ int steps_of(const AttendParams &a, int len, int fresh, int group) {
  const int64_t end = ((int64_t)(group + 1) * G::ROWS + a.G - 1) / a.G;   // its tokens end here
  const int64_t seen = len - fresh + (end < fresh ? end : fresh);
  return seen <= 0 ? 1 : (int)((seen + G::SLOTS - 1) / G::SLOTS);
}
template <class G>
__device__ __forceinline__ int groups_of(const AttendParams &a, int fresh) {
  return (int)(((int64_t)fresh * a.G + G::ROWS - 1) / G::ROWS);
}
// To the first step of the next item.
template <class G>
__device__ __forceinline__ void next_item(const AttendParams &a, TcWalk &w) {
  w.base += G::SETUP + w.steps;
  w.step = 0;
  if (++w.group >= w.groups) {
    w.group = 0;
    if (++w.h >= a.H) {
      w.h = 0;
      do {
        if (++w.r >= a.req.R) return;
        w.len = len_of(a, w.r);
        w.beg = a.req.begin(w.r);
        w.fresh = (int)(a.req.begin(w.r + 1) - w.beg);
        w.groups = groups_of<G>(a, w.fresh);
      } while (w.groups == 0);
    }
  }
  w.steps = steps_of<G>(a, w.len, w.fresh, w.group);
}
// The CTA's steps of the item, from w.step on (the share ends at place `last`).
template <class G>
__device__ __forceinline__ int steps_here(const TcWalk &w, int64_t last) {
  return (int)min((int64_t)w.steps, last - w.base - G::SETUP) - w.step;
}
__device__ __forceinline__ int64_t scan_up(int64_t v) {   // inclusive, over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, v, o);
    if ((int)(threadIdx.x % 32) >= o) v += y;
  }
  return v;
}
// 32 requests from r0 on, one a lane: the lane's request, the places of one of its
// heads, the places up to and with it; whether the table is good there.
struct Requests32 {
  int len, fresh;
  int64_t beg, head, upto;
  bool good;
};
template <class G>
__device__ __forceinline__ Requests32 look(const AttendParams &a, int r0, bool tell) {
  const int r = r0 + threadIdx.x % 32;
  Requests32 q = {};
  bool good = true;
  if (r < a.req.R) {
    q.len = len_of(a, r);
    q.beg = a.req.begin(r);
    const int64_t end = a.req.begin(r + 1);
    q.fresh = (int)(end - q.beg);
    good = end >= q.beg && end - q.beg <= a.max_new && (r > 0 || q.beg == 0) && (r + 1 < a.req.R || end == a.req.ntok);
    if (!good) q.fresh = 0;
    if (tell && q.len != __ldg(a.lens + r)) raise(a.status, KVX_FLAG_BAD_LENGTH);
  }
  if ((int64_t)a.G * a.max_new <= G::ROWS) {
    q.head = q.fresh > 0 ? G::SETUP + steps_of<G>(a, q.len, q.fresh, 0) : 0;
  } else {
    for (int i = 0; i < 32 && r0 + i < a.req.R; ++i) {
      const int len = __shfl_sync(~0u, q.len, i), fresh = __shfl_sync(~0u, q.fresh, i), groups = groups_of<G>(a, fresh);
      int64_t sum = 0;
      for (int g = threadIdx.x % 32; g < groups; g += 32) sum += G::SETUP + steps_of<G>(a, len, fresh, g);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if ((int)(threadIdx.x % 32) == i) q.head = sum;
    }
  }
  q.upto = scan_up(q.head * a.H);
  q.good = __all_sync(~0u, good);
  return q;
}
// One warp: the share of CTA `cta` of `ctas`.
template <class G>
__device__ void find_share(const AttendParams &a, int cta, int ctas, bool tell, Share &s) {
  const int lane = threadIdx.x % 32;
  s.good = true;
  s.T = 0;
  s.N = 0;
  s.last = -1;
  s.w = {};
  Requests32 q;
  for (int r0 = 0; r0 < a.req.R; r0 += 32) {
    q = look<G>(a, r0, tell);
    s.good = s.good && q.good;
    s.T += __shfl_sync(~0u, q.upto, 31);
  }
  if (!s.good) return;
  s.N = s.T < ctas ? s.T : ctas;
  if (cta >= s.N) return;
  const int64_t at = cta * s.T / s.N;
  s.last = (cta + 1) * s.T / s.N;
  int64_t before = 0;
  for (int r0 = 0; r0 < a.req.R; r0 += 32) {
    if (a.req.R > 32) q = look<G>(a, r0, false);      // otherwise it is at hand
    const unsigned here = __ballot_sync(~0u, at < before + q.upto);
    if (!here) {
      before += __shfl_sync(~0u, q.upto, 31);
      continue;
    }
    const int who = __ffs(here) - 1;
    TcWalk &w = s.w;
    w.r = r0 + who;
    w.len = __shfl_sync(~0u, q.len, who);
    w.fresh = __shfl_sync(~0u, q.fresh, who);
    w.beg = __shfl_sync(~0u, q.beg, who);
    w.groups = groups_of<G>(a, w.fresh);
    const int64_t per = __shfl_sync(~0u, q.head, who), in = at - before - (__shfl_sync(~0u, q.upto, who) - per * a.H);
    w.h = (int)(in / per);
    int64_t rem = in % per;
    for (int g0 = 0;; g0 += 32) {
      const int64_t places = g0 + lane < w.groups ? G::SETUP + steps_of<G>(a, w.len, w.fresh, g0 + lane) : 0;
      const int64_t to = scan_up(places);
      const unsigned hit = __ballot_sync(~0u, rem < to);
      if (hit || g0 + 32 >= w.groups) {
        const int k = hit ? __ffs(hit) - 1 : 0;
        const int here_places = (int)__shfl_sync(~0u, places, k);
        const int in_item = (int)(rem - (__shfl_sync(~0u, to, k) - here_places));
        w.group = g0 + k;
        w.steps = here_places - G::SETUP;
        w.step = max(0, in_item - G::SETUP);
        w.base = at - in_item;
        return;
      }
      rem -= __shfl_sync(~0u, to, 31);
    }
  }
}

// --- tcgen05 ---------------------------------------------------------------------
// Instruction descriptors: D fp32, M = 128; e4m3 x e4m3 both K-major, N = 64, and f16
// x f16 with B as it lies in memory, [K][N] (MN-major), N = 128.
constexpr uint32_t kIdescQK = (1u << 4) | (8u << 17) | (8u << 24);
constexpr uint32_t kIdescKQ = (1u << 4) | (16u << 17) | (8u << 24);   // N = 128
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | (16u << 17) | (8u << 24);

// The whole warp calls these, with the same arguments (which stay in uniform
// registers); one elected lane issues.
// S = (Q1 + Q2) K^T for 64 slots: two parts of four 32-deep steps.
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t q, uint64_t k) {
  asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b32 r;\n.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3;\n"
      "elect.sync r|e, 0xffffffff;\n"
      "setp.ne.u32 f, 0, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u64 a1, %1, 2; add.u64 a2, %1, 4; add.u64 a3, %1, 6; add.u64 a4, %1, %4;\n"
      "add.u64 a5, a4, 2; add.u64 a6, a4, 4; add.u64 a7, a4, 6;\n"
      "add.u64 b1, %2, 2; add.u64 b2, %2, 4; add.u64 b3, %2, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a4, %2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a5, b1, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a6, b2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a7, b3, %3, t;\n}\n" ::"r"(d),
      "l"(q), "l"(k), "r"(kIdescQK), "l"((uint64_t)(kTileBytes >> 4))
      : "memory");
}
// S^T = K (Q1 + Q2)^T for 128 slots and rows.
__device__ __forceinline__ void mma_kq(uint32_t d, uint64_t k, uint64_t q) {
  asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b32 r;\n.reg .b64 a1, a2, a3, b1, b2, b3, b4, b5, b6, b7;\n"
      "elect.sync r|e, 0xffffffff;\n"
      "setp.ne.u32 f, 0, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u64 a1, %1, 2; add.u64 a2, %1, 4; add.u64 a3, %1, 6;\n"
      "add.u64 b1, %2, 2; add.u64 b2, %2, 4; add.u64 b3, %2, 6; add.u64 b4, %2, %4;\n"
      "add.u64 b5, b4, 2; add.u64 b6, b4, 4; add.u64 b7, b4, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, b4, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b5, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b6, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b7, %3, t;\n}\n" ::"r"(d),
      "l"(k), "l"(q), "r"(kIdescKQ), "l"((uint64_t)(kTileBytes >> 4))
      : "memory");
}
// O (+)= P V for 64 slots: four 16-deep steps; P 8 columns on, V 16 slots (2 KB) on.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t v, bool add) {
  asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b32 r, a1, a2, a3;\n.reg .b64 b1, b2, b3;\n"
      "elect.sync r|e, 0xffffffff;\n"
      "setp.ne.u32 f, %4, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u32 a1, %1, 8; add.u32 a2, %1, 16; add.u32 a3, %1, 24;\n"
      "add.u64 b1, %2, 128; add.u64 b2, %2, 256; add.u64 b3, %2, 384;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n}\n" ::"r"(d),
      "r"(p), "l"(v), "r"(kIdescPV), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) { tc_commit_elect<1>(smem_addr(bar)); }
// [K][N] operand of 16-bit values, 128-byte swizzle: 64-column groups 16 KB
// apart (leading offset), 8-row groups 1 KB apart (stride offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(kTileBytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]),
        "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
        "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// Wait for loads, of which v is one: what follows may not use v before.
__device__ __forceinline__ void tc_wait_ld32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The factor on a row's scores: positive, so that a masked score stays -inf, and
// NaN for a row with an infinity (NaN elements are NaN in the parts).
__device__ __forceinline__ float row_factor(const AttendParams &a, float top, float unit) {
  return top < INFINITY ? fmaxf(fabsf(a.c) * unit, 0x1p-126f) : __uint_as_float(0x7fc00000u);
}
// 32 columns of scores.  Four columns share a key scale f > 0 and a bit of `mask`;
// with MASK column e counts where e <= seen (the others become -inf, and scales
// that are missing 1).
template <bool MASK>
__device__ __forceinline__ void columns(uint32_t (&s)[32], float (&f)[8], const float4 *scale, uint32_t mask, int seen) {
  const float4 f0 = scale[0], f1 = scale[1];
  const float v[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    f[q] = v[q];
    if constexpr (MASK) {
      const bool in = mask >> q & 1;
      f[q] = in ? v[q] : 1.f;
      const int last = in ? seen - 4 * q : -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * q + e] = e <= last ? s[4 * q + e] : 0xff800000u;
    }
  }
}
// exp2(y), y = score f cs + add, in f16, two to a register, their sum and the largest y.
template <bool MASK>
__device__ __forceinline__ uint64_t probabilities(uint32_t *out, const uint32_t (&s)[32], const float (&f)[8], float cs,
                                                  uint64_t add, uint64_t sum, float &top) {
  const float *x = reinterpret_cast<const float *>(s);
  float t0 = top, t1 = top;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    // not 0, which would make NaN of -inf
    const float g = MASK ? fmaxf(f[q] * cs, 0x1p-126f) : f[q] * cs;
    const uint64_t g2 = pair(g, g);
    float y[4];
    unpair(fma2(pair(x[4 * q], x[4 * q + 1]), g2, add), y[0], y[1]);
    unpair(fma2(pair(x[4 * q + 2], x[4 * q + 3]), g2, add), y[2], y[3]);
    t0 = max3(t0, y[0], y[1]);
    t1 = max3(t1, y[2], y[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = ex2(y[e]);
    sum = add2(sum, add2(pair(y[0], y[1]), pair(y[2], y[3])));
    out[2 * q] = f16x2(y[0], y[1]);
    out[2 * q + 1] = f16x2(y[2], y[3]);
  }
  top = fmaxf(t0, t1);
  return sum;
}
__device__ __forceinline__ bool is_far(float m) { return m > -INFINITY && fabsf(m) > kFar; }
// 32 of a row's scores from tensor memory, each rounded once to fp32.
__device__ __forceinline__ void rounded_scores(uint32_t (&s)[32], uint32_t col, const float4 *scale, uint32_t mask, int seen, float cs) {
  float f[8];
  tc_ld32(col, s);
  tc_wait_ld32(s);
  columns<true>(s, f, scale, mask, seen);
#pragma unroll
  for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__fmul_rn(__uint_as_float(s[e]), fmaxf(f[e / 4] * cs, 0x1p-126f)));
}
// The largest of the 64 scores of a half tile.
__device__ __noinline__ float largest_score(uint32_t col, const float4 *scale, uint32_t mask, int seen, float cs) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t s[32];
    rounded_scores(s, col + 32 * c, scale + 2 * c, mask >> (8 * c), seen - 32 * c, cs);
#pragma unroll
    for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(s[e]));
  }
  return top;
}
// The probabilities exp2((score - m) + add) of a half tile over the scores they come
// from; returns their sum.
__device__ __noinline__ float far_probabilities(uint32_t col, const float4 *scale, uint32_t mask, int seen, float cs, float m,
                                                float add) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t s[32], out[16];
    rounded_scores(s, col + 32 * c, scale + 2 * c, mask >> (8 * c), seen - 32 * c, cs);
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float y0 = ex2((__uint_as_float(s[e]) - m) + add), y1 = ex2((__uint_as_float(s[e + 1]) - m) + add);
      part += y0 + y1;
      out[e / 2] = f16x2(y0, y1);
    }
    tc_st16(col + 16 * c, out);     // where scores were read already
    sum += part;
  }
  tc_wait_st();
  return sum;
}
// The probabilities exp2(score + add) of a half tile whose scores are near, the same way.
__device__ __noinline__ float near_probabilities(uint32_t col, const float4 *scale, uint32_t mask, int seen, float cs,
                                                 float add) {
  uint64_t sum = pair(0.f, 0.f);
  const uint64_t a2 = pair(add, add);
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t s[32], out[16];
    float f[8], top = 0.f;
    tc_ld32(col + 32 * c, s);
    tc_wait_ld32(s);
    columns<true>(s, f, scale + 2 * c, mask >> (8 * c), seen - 32 * c);
    sum = probabilities<true>(out, s, f, cs, a2, sum, top);
    tc_st16(col + 16 * c, out);
  }
  tc_wait_st();
  float s0, s1;
  unpair(sum, s0, s1);
  return s0 + s1;
}
// A half tile of a row: probabilities over the scores they come from, the row's
// running maximum (lazily) and sum.  What is subtracted from a score plus its tile's
// value scale is m + shift: the largest such sum and 0, or where it is far a score as it was
// rounded and the value scale's exponent of its tile, because the sum of those would be
// rounded: from 2^25 on by more than f16 has room for.  `raise(down)` is called by whole
// warps when a maximum has to rise: it scales down what the rows have so far.  What it
// takes then is in functions of their own, so that it costs the others no registers (in a
// loop around the code below a prompt of 8192 tokens takes 1266 us, this way 1134).
template <bool MASK, class F>
__device__ __forceinline__ bool softmax_half(uint32_t col, const float4 *scale, uint32_t mask, int seen, float cs, float ref,
                                             float &m, float &shift, float &l, F raise) {
  uint32_t a[32], b[32], out[32];
  float fa[8], fb[8];
  tc_ld32(col, a);
  tc_ld32(col + 32, b);
  tc_wait_ld32(a);
  tc_wait_ld32(b);
  columns<MASK>(a, fa, scale, mask, seen);
  columns<MASK>(b, fb, scale + 2, mask >> 8, seen - 32);
  const float add = kBias + (ref - shift) - finite_or_0(m);
  const uint64_t a2 = pair(add, add);
  float top = -INFINITY;
  uint64_t sum = probabilities<MASK>(out, a, fa, cs, a2, pair(0.f, 0.f), top);
  sum = probabilities<MASK>(out + 16, b, fb, cs, a2, sum, top);
  // -inf where nothing is seen
  const bool over = top > kBias + kSlack || (m == -INFINITY && top > -INFINITY) || fabsf(add) > kFar;
  float s0, s1;
  unpair(sum, s0, s1);
  if (!__any_sync(~0u, over)) {
    l += (s0 + s1) * ex2(-ref);    // without the value scale
    tc_st32(col, out);
    tc_wait_st();
    return true;
  }
  // seldom: the maximum rises, and the probabilities again.  Where it and the scores are
  // near they come from the same sums, which are within 2^-10 of kBias at most then.
  const uint32_t in = MASK ? mask : 0xffffu;
  const int last = MASK ? seen : kTile;
  if (!__any_sync(~0u, is_far(m) || is_far(top) || fabsf(add) > kFar)) {
    const float mm = fmaxf(m, top - kBias + finite_or_0(m)), down = ex2(m - finite_or_0(mm));
    if (!raise(down)) return false;
    m = mm;
    l = l * down + near_probabilities(col, scale, in, last, cs, kBias + (ref - shift) - finite_or_0(m)) * ex2(-ref);
    return true;
  }
  // Far: from scores rounded before the maximum, which is one of them, is subtracted.  That
  // is exact for all scores near it, so none is above kBias however large they are.
  const float most = largest_score(col, scale, in, last, cs);
  const float by = (most - finite_or_0(m)) + (ref - shift);
  const bool rises = m == -INFINITY ? most > -INFINITY : by > 0.f;
  const float down = m == -INFINITY ? 0.f : rises ? ex2(-by) : 1.f;
  if (!raise(down)) return false;
  if (rises) {
    m = most;
    shift = ref;
  }
  l = l * down + far_probabilities(col, scale, in, last, cs, finite_or_0(m), kBias + (ref - shift)) * ex2(-ref);
  return true;
}
// The factor of a lane's row, from its largest element.
__device__ __noinline__ float query_factor(const AttendParams &a, bool vec, const __nv_bfloat16 *src, bool live) {
  float top = 0.f;
  if (live && vec) {
#pragma unroll 4
    for (int e = 0; e < a.d / 8; ++e) {
      const uint4 t = __ldg(reinterpret_cast<const uint4 *>(src) + e);
      const uint32_t v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = max3(top, fabsf(__uint_as_float(v[k] << 16)), fabsf(__uint_as_float(v[k] & 0xffff0000u)));
    }
  } else if (live) {
#pragma unroll 4
    for (int e = 0; e < a.d; ++e) top = fmaxf(top, fabsf(__bfloat162float(src[e])));
  }
  return row_factor(a, top, pow2_scale(top));
}
// Up to 32 query rows of a warp (`count` of them, rounded up to 8) as two e4m3
// parts, `part` bytes apart, in the swizzled K-major tile, from row `first` of the
// tile on; `src` is the lane's own row.  Half a warp loads a row, eight rows at a
// time where a CTA does one or two items and runs this code cold, sixteen where it
// does many (wide calls).  Returns the lane's factor on its row's
// scores (its sign is in the parts).
template <int N>
__device__ __noinline__ float put_queries(const AttendParams &a, bool vec, const __nv_bfloat16 *src, bool live,
                                          unsigned char *tile, int first, int part, int count) {
  const int lane = threadIdx.x % 32, c = lane % 16;      // 8 dimensions
  float mine = 0.f;
#pragma unroll 1
  for (int i0 = 0; 2 * i0 < count; i0 += N) {
    uint4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = 2 * (i0 + i) + lane / 16;
      const uint64_t p = __shfl_sync(~0u, (uint64_t)src, row);
      const bool there = __shfl_sync(~0u, (int)live, row) && 8 * c < a.d;
      const uint4 *from = reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(p) + 8 * c);
      x[i] = there && vec ? __ldg(from) : make_uint4(0, 0, 0, 0);
      if (!vec && there) {
        const unsigned short *h = reinterpret_cast<const unsigned short *>(from);
        uint32_t v[4] = {};
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = (uint32_t)h[e] << (16 * (e & 1));
          v[0] |= e / 2 == 0 ? u : 0u;
          v[1] |= e / 2 == 1 ? u : 0u;
          v[2] |= e / 2 == 2 ? u : 0u;
          v[3] |= e / 2 == 3 ? u : 0u;
        }
        x[i] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float y[8], top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = __uint_as_float(v[e] << 16);
        y[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
        top = max3(top, fabsf(y[2 * e]), fabsf(y[2 * e + 1]));
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const float unit = pow2_scale(top);   // top <= 448 unit
      const float up = a.c != 0.f ? copysignf(1.f / unit, a.c) : 0.f;
      const float other = __shfl_xor_sync(~0u, top, 16);
      if (lane / 2 == i0 + i) mine = lane % 2 == lane / 16 ? top : other;
      uint32_t p1[2], p2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float *z = y + 4 * e;
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] *= up;
        p1[e] = e4m3x2(z[0], z[1]) | e4m3x2(z[2], z[3]) << 16;
        const float2 f0 = floats_of(p1[e]), f1 = floats_of(p1[e] >> 16);
        p2[e] = e4m3x2(z[0] - f0.x, z[1] - f0.y) | e4m3x2(z[2] - f1.x, z[3] - f1.y) << 16;
      }
      const int row = first + 2 * (i0 + i) + lane / 16;
      unsigned char *to = tile + row * kD + ((c / 2 ^ (row & 7)) << 4) + (c & 1) * 8;
      *reinterpret_cast<uint2 *>(to) = make_uint2(p1[0], p1[1]);
      *reinterpret_cast<uint2 *>(to + part) = make_uint2(p2[0], p2[1]);
    }
  }
  return row_factor(a, mine, pow2_scale(mine));
}

// O times a row's factor, in place.
__device__ __noinline__ void scale_down(uint32_t col, float down) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    tc_ld32(col + 32 * c, o);
    tc_wait_ld32(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
    tc_st32(col + 32 * c, o);
  }
}
// 64 scores, base 2, to a row (NULL: only take part).
__device__ __noinline__ void keep_scores(uint32_t col, float *to, const float4 *scale, uint32_t mask, int seen, float cs) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t s[32];
    float f[8];
    tc_ld32(col + 32 * c, s);
    tc_wait_ld32(s);
    columns<true>(s, f, scale + 2 * c, mask >> (8 * c), seen - 32 * c);
    const float *x = reinterpret_cast<const float *>(s);
    if (to)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float g = fmaxf(f[q] * cs, 0x1p-126f);
        *reinterpret_cast<float4 *>(to + 32 * c + 4 * q) =
            make_float4(x[4 * q] * g, x[4 * q + 1] * g, x[4 * q + 2] * g, x[4 * q + 3] * g);
      }
    __syncwarp();
  }
}

// A part's sums are relative to exp2 of its row's m + shift, which is left as one number
// where m is not far, as two where it is.
__device__ __forceinline__ void leave_part(float *tops, int rows, int row, float m, float shift, float l) {
  const bool far = is_far(m);
  tops[row] = far ? m : m + shift;
  tops[rows + row] = far ? shift : 0.f;
  tops[2 * rows + row] = l;
}
// Is a + sa above b + sb?
__device__ __forceinline__ bool above(float a, float sa, float b, float sb) { return (a - b) + (sa - sb) > 0.f; }
// A warp joins the parts of a row, of which some are far.
template <class G>
__device__ __forceinline__ void join_far(const TcParams &p, int c0, int parts, int row, int64_t tok, int hq) {
  const int lane = threadIdx.x % 32;
  float mm = -INFINITY, sh = 0.f, ll = 0.f;
  float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = 0; c < parts; ++c) {
    const int64_t cta = c0 + c / G::PARTS;
    const float *part = p.partial + ((cta * 2 + (c < G::PARTS)) * G::PARTS + c % G::PARTS) * (int64_t)p.part_size;
    const float *tops = part + p.slot_rows * kD + row;
    const float pm = __ldcg(tops), ps = __ldcg(tops + p.slot_rows), pl = __ldcg(tops + 2 * p.slot_rows);
    const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + row * kD) + lane);
    const bool own = above(pm, ps, mm, sh);
    const float now = finite_or_0(own ? pm : mm), by = own ? ps : sh;
    const float f0 = ex2((mm - now) + (sh - by)), f1 = ex2((pm - now) + (ps - by));
    mm = own ? pm : mm;
    sh = by;
    ll = ll * f0 + pl * f1;
    oo = make_float4(oo.x * f0 + y.x * f1, oo.y * f0 + y.y * f1, oo.z * f0 + y.z * f1, oo.w * f0 + y.w * f1);
  }
  if (lane * 4 >= p.a.d) return;
  store_out(p.a, tok, hq, lane * 4, make_float2(oo.x, oo.y), mm, sh, ll);
  store_out(p.a, tok, hq, lane * 4 + 2, make_float2(oo.z, oo.w), mm, sh, ll);
}
template <class G>
__device__ __noinline__ void join_far_rows(const TcParams &p, const TcWalk &w, int c0, int parts, int first, int stride, int rows) {
  for (int k = first; k < rows; k += stride) {
    const int64_t row = (int64_t)w.group * G::ROWS + k;
    join_far<G>(p, c0, parts, k, w.beg + row / p.a.G, w.h * p.a.G + (int)(row % p.a.G));
  }
}
// Join the parts of an item that CTAs c0 .. c0 + ctas - 1 left: rows first, first +
// stride, ... of the warp.  A CTA keeps parts of an item that others began, and of
// one that it began.  The parts' maxima and totals by the lanes, 32 parts at a time,
// then their sums, of B rows at once.
template <class G, int B>
__device__ __noinline__ void join_rows(const TcParams &p, const TcWalk &w, int c0, int ctas, int first, int stride, int rows) {
  const AttendParams &a = p.a;
  const int lane = threadIdx.x % 32, parts = ctas * G::PARTS;
  const auto part_at = [&](int c) {
    const int64_t cta = c0 + c / G::PARTS;
    return p.partial + ((cta * 2 + (c < G::PARTS)) * G::PARTS + c % G::PARTS) * (int64_t)p.part_size;
  };
  for (int r0 = first; r0 < rows; r0 += stride * B) {
    float mm[B], ll[B], f[B];
    float4 oo[B];
    int rr[B];
    bool far = false;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      rr[k] = min(r0 + k * stride, rows - 1);   // a row beyond is formed twice
      mm[k] = -INFINITY;
      ll[k] = 0.f;
      oo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int at = 0; at < parts; at += 32) {
      const float *own = part_at(min(at + lane, parts - 1)) + p.slot_rows * kD;
      float pm[B], pl[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        pm[k] = __ldcg(own + rr[k]);
        pl[k] = __ldcg(own + 2 * p.slot_rows + rr[k]);
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (at + lane >= parts) {
          pm[k] = -INFINITY;
          pl[k] = 0.f;
        }
        far = far || is_far(pm[k]);
        float top = fmaxf(mm[k], pm[k]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float down = ex2(mm[k] - finite_or_0(top));
        f[k] = ex2(pm[k] - finite_or_0(top));
        mm[k] = top;
        float sum = pl[k] * f[k];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        ll[k] = ll[k] * down + sum;
        oo[k] = make_float4(oo[k].x * down, oo[k].y * down, oo[k].z * down, oo[k].w * down);
      }
      const int here = min(32, parts - at);
#pragma unroll (8 / B)
      for (int c = 0; c < here; ++c) {
        const float *part = part_at(at + c) + lane * 4;
        float4 y[B];
#pragma unroll
        for (int k = 0; k < B; ++k) y[k] = __ldcg(reinterpret_cast<const float4 *>(part + rr[k] * kD));
#pragma unroll
        for (int k = 0; k < B; ++k) {
          const float g = __shfl_sync(~0u, f[k], c);
          oo[k].x += y[k].x * g;
          oo[k].y += y[k].y * g;
          oo[k].z += y[k].z * g;
          oo[k].w += y[k].w * g;
        }
      }
    }
    if (__any_sync(~0u, far)) {     // seldom: from the start, by both numbers of the parts
      join_far_rows<G>(p, w, c0, parts, r0, stride, rows);
      return;
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int64_t row = (int64_t)w.group * G::ROWS + rr[k], tok = w.beg + row / a.G;
      const int hq = w.h * a.G + (int)(row % a.G);
      if (lane * 4 >= a.d) continue;
      store_out(a, tok, hq, lane * 4, make_float2(oo[k].x, oo[k].y), mm[k], 0.f, ll[k]);
      store_out(a, tok, hq, lane * 4 + 2, make_float2(oo[k].z, oo[k].w), mm[k], 0.f, ll[k]);
    }
  }
}
// One lane of each CTA leaves this for the kernel that joins.
template <class G>
__device__ __forceinline__ void note_split(const TcParams &p, const Share &s) {
  Split x = {};
  const TcWalk &w = s.w;
  if (s.good && s.last >= 0 && w.step > 0) {
    const int64_t begin = w.base + G::SETUP;
    const int c0 = (int)(((begin + 1) * s.N - 1) / s.T), c1 = (int)(((begin + w.steps) * s.N - 1) / s.T);   // first, last step
    if (c0 + 1 == (int)blockIdx.x) {
      x.r = w.r;
      x.h = w.h;
      x.group = w.group;
      x.c0 = c0;
      x.ctas = c1 - c0 + 1;
      x.rows = (int)min((int64_t)G::ROWS, (int64_t)w.fresh * p.a.G - (int64_t)w.group * G::ROWS);
      x.beg = w.beg;
    }
  }
  p.splits[blockIdx.x] = x;
}
// The items that several CTAs worked on: block x looks after the one that CTA x + 1
// noted, block y after a slice of its rows.
// Three blocks an SM: its loads wait long (after a prompt of 2048 tokens 15 us, two 19).
template <class G>
__global__ void __launch_bounds__(256, 3) join_kernel(const __grid_constant__ TcParams p) {
  let_next_kernel_start();
  wait_for_kernel_before();
  const Split x = p.splits[blockIdx.x + 1];
  if (x.ctas == 0) return;
  TcWalk w;
  w.h = x.h;
  w.group = x.group;
  w.beg = x.beg;
  join_rows<G, 4>(p, w, x.c0, x.ctas, blockIdx.y * 8 + threadIdx.x / 32, gridDim.y * 8, x.rows);
}
// The same with a block for a row, whose warps share the parts: few rows, many parts.
template <class G>
__global__ void __launch_bounds__(256) join_row_kernel(const __grid_constant__ TcParams p) {
  __shared__ float top[8], sum[8];
  __shared__ float4 part_sum[8][32];
  let_next_kernel_start();
  wait_for_kernel_before();
  const Split x = p.splits[blockIdx.x + 1];
  const int row = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32, parts = x.ctas * G::PARTS;
  if (row >= x.rows || parts == 0) return;
  float mm = -INFINITY, ll = 0.f;
  float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
  bool far = false;
#pragma unroll 5
  for (int c = warp; c < parts; c += 8) {
    const int64_t cta = x.c0 + c / G::PARTS;
    const float *part = p.partial + ((cta * 2 + (c < G::PARTS)) * G::PARTS + c % G::PARTS) * (int64_t)p.part_size;
    const float pm = __ldcg(part + p.slot_rows * kD + row), pl = __ldcg(part + p.slot_rows * (kD + 2) + row);
    const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + row * kD) + lane);
    const float now = fmaxf(mm, pm), f0 = ex2(mm - finite_or_0(now)), f1 = ex2(pm - finite_or_0(now));
    far = far || is_far(pm);
    mm = now;
    ll = ll * f0 + pl * f1;
    oo = make_float4(oo.x * f0 + y.x * f1, oo.y * f0 + y.y * f1, oo.z * f0 + y.z * f1, oo.w * f0 + y.w * f1);
  }
  part_sum[warp][lane] = oo;
  if (lane == 0) {
    top[warp] = mm;
    sum[warp] = ll;
  }
  far = __syncthreads_or(far);
  if (warp > 0) return;
  const AttendParams &a = p.a;
  const int64_t at = (int64_t)x.group * G::ROWS + row, tok = x.beg + at / a.G;
  const int hq = x.h * a.G + (int)(at % a.G);
  if (far) {
    join_far<G>(p, x.c0, parts, row, tok, hq);
    return;
  }
  mm = -INFINITY;
  ll = 0.f;
  oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 8; ++k) mm = fmaxf(mm, top[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float f = ex2(top[k] - finite_or_0(mm));
    const float4 y = part_sum[k][lane];
    ll += sum[k] * f;
    oo = make_float4(oo.x + y.x * f, oo.y + y.y * f, oo.z + y.z * f, oo.w + y.w * f);
  }
  if (lane * 4 >= a.d) return;
  store_out(a, tok, hq, lane * 4, make_float2(oo.x, oo.y), mm, 0.f, ll);
  store_out(a, tok, hq, lane * 4 + 2, make_float2(oo.z, oo.w), mm, 0.f, ll);
}

// What a softmax group knows of its item when the item, or the CTA's part of it, ends.
struct Item {
  TcWalk w;
  int count, rows, row;
  bool live, warp_live;
  float m, shift, l;
  uint32_t o_col, half, joins;   // half tiles and joins of this group so far
};
// Write the result of the item, or leave this CTA's part of it for the kernel that
// joins.  Seldom, and apart from the loop so that it costs that no
// registers.
template <bool WIDE>
__device__ __noinline__ bool finish_item(const TcParams &p, TcShared *sh, const Item it, int i) {
  using G_ = std::conditional_t<WIDE, Wide, Narrow>;
  const AttendParams &a = p.a;
  const Waiter W{sh, a.status};
  const TcWalk &w = it.w;
  const uint32_t half = it.half, joins = it.joins;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rows = it.rows, row = it.row;
  const bool live = it.live, warp_live = it.warp_live, whole = it.count == w.steps;
  const float m = it.m, shift = it.shift - kBias, l = it.l;   // what the sums are relative to
  const uint32_t o_col = it.o_col;
  // the result of the item, or this CTA's part of it
  if (!W.warp_wait(&sh->pv_done[i][(half - 1) & 1], (half - 1) >> 1 & 1)) return false;
  tc_fence_after();
  // narrow: the parts of the item joined before have been read by all
  if (!WIDE && joins > 0 && !W.warp_wait(&sh->spent, (joins - 1) & 1)) return false;
  const float back = 1.f / 128.f;   // V carries 2^7
  const int64_t at = (int64_t)w.group * G_::ROWS + row;
  const int64_t tok = w.beg + at / a.G;
  const int hq = w.h * a.G + (int)(at % a.G);
  const int64_t part_size = p.part_size;
  float *slot = p.partial + (((int64_t)blockIdx.x * 2 + (w.step == 0)) * G_::PARTS + (WIDE ? 0 : i)) *
                                part_size;
  const bool direct = WIDE && whole;
  if (warp_live) {
    const float inv = direct ? (l != 0.f ? back / l : 0.f) : back;
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + tok * a.ot + hq * a.oh;
    if (WIDE && (!direct || p.vec_out)) {
      // Through shared memory, so that rows go out whole: a lane's row is written
      // there 16 bytes at a time, and half a warp stores a row's 256.  It lies where
      // the warp's own query rows were, whose products are over.
      extern __shared__ unsigned char raw[];
      unsigned char *own = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023)) +
                           i * 2 * kTileBytes + warp % 4 * 32 * kD;
      const auto cell = [&](int r, int at) {    // 16 bytes `at` of row r
        return reinterpret_cast<uint4 *>(own + (at / 8) * kTileBytes + r * 128 + ((at % 8 ^ (r & 7)) << 4));
      };
      uint64_t to = direct ? (uint64_t)out : (uint64_t)(slot + row * kD);
#pragma unroll 1
      for (int half_row = 0; half_row < (direct ? 1 : 2); ++half_row) {
#pragma unroll 1
        for (int c = 0; c < (direct ? 4 : 2); ++c) {
          uint32_t o[32];
          tc_ld32(o_col + 64 * half_row + 32 * c, o);
          tc_wait_ld32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          if (direct) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t b[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) b[k] = pack_bf16(__uint_as_float(o[8 * e + 2 * k]), __uint_as_float(o[8 * e + 2 * k + 1]));
              *cell(lane, 4 * c + e) = make_uint4(b[0], b[1], b[2], b[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) *cell(lane, 8 * c + e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += 2) {
          const int r = r0 + lane / 16;
          const uint64_t base = __shfl_sync(~0u, to, r);
          if (row - lane + r < rows && (!direct || 8 * (lane % 16) < a.d))
            reinterpret_cast<uint4 *>(base)[lane % 16] = *cell(r, lane % 16);
        }
        to += 256;
        __syncwarp();
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tc_ld32(o_col + 32 * c, o);
        tc_wait_ld32(o);
        if (live && !direct) {
          float4 *to = reinterpret_cast<float4 *>(slot + row * kD + 32 * c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            to[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e < a.d) out[32 * c + e] = __float2bfloat16_rn(__uint_as_float(o[e]) * inv);
        }
        __syncwarp();   // together to the next load
      }
    }
    if (live) {
      if (direct) {
        store_lse(a, tok, hq, m, shift, l);
      } else {
        leave_part(slot + p.slot_rows * kD, p.slot_rows, row, m, shift, l);
      }
    }
  }
  if (!direct) {
    // narrow: an item that this CTA did alone is joined from its two groups here,
    // what several CTAs worked on by the next kernel
    if (WIDE || !whole) return true;
    __threadfence_block();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh->join));
    if (!W.warp_wait(&sh->join, joins & 1)) return false;
    join_rows<G_, 1>(p, w, blockIdx.x, 1, warp, 8, rows);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh->spent));
  }
  return true;
}

// --- the kernel ------------------------------------------------------------------
template <bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
  using G_ = std::conditional_t<WIDE, Wide, Narrow>;
  constexpr int kKStages = kStagesOf<WIDE>;
  extern __shared__ unsigned char raw[];
  unsigned char *qbuf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  unsigned char *kbuf = qbuf + (WIDE ? kSmemQ : kSmemQ / 2), *vbuf = kbuf + kKStages * kTileBytes, *wbuf = vbuf + kVStages * kTileBytes;
  TcShared *sh = reinterpret_cast<TcShared *>(wbuf + kWStages * 2 * kTileBytes);
  const AttendParams &a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_addr(&sh->k_full[i]), 32);
      mbar_init(smem_addr(&sh->k_empty[i]), WIDE ? 2 + 8 : 1 + 4);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_addr(&sh->v_full[i]), 32);
      mbar_init(smem_addr(&sh->v_empty[i]), 4);
    }
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(smem_addr(&sh->w_full[i]), 4);
      mbar_init(smem_addr(&sh->w_empty[i]), WIDE ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh->q_full[i]), 4);
      mbar_init(smem_addr(&sh->drain[i]), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_addr(&sh->s_full[i][h]), 1);
        mbar_init(smem_addr(&sh->p_full[i][h]), 4);
        mbar_init(smem_addr(&sh->pv_done[i][h]), 1);
      }
    }
    mbar_init(smem_addr(&sh->join), 8);
    mbar_init(smem_addr(&sh->spent), 8);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sh->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kLoadWarp) {
    Share share;
    find_share<G_>(a, blockIdx.x, gridDim.x, blockIdx.x == 0, share);
    if (lane == 0) {
      sh->share = share;
      note_split<G_>(p, share);
      if (!share.good && blockIdx.x == 0) raise(a.status, KVX_FLAG_BAD_SEQLENS);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const Waiter W{sh, a.status};
  TcWalk w = sh->share.w;
  const int64_t last = sh->share.last;

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ----------------------------------------------------------------------
    // softmax: a row to a thread
    // ----------------------------------------------------------------------
    const int i = warp / 4;                       // group
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t s_col = tmem + lanes + i * kTile, o_col = tmem + lanes + 2 * kTile + i * kTile;
    const int row = (WIDE ? i * kTile : 0) + warp % 4 * 32 + lane;   // in the item
    uint32_t half = 0, joins = 0;                 // half tiles of this group and joins so far
    int ks = WIDE ? 0 : i;                        // the tile's K stage, and its phase
    uint32_t k_phase = 0;
    for (; w.base + G_::SETUP < last; next_item<G_>(a, w)) {
      const int count = steps_here<G_>(w, last);
      const int rows = (int)min((int64_t)G_::ROWS, (int64_t)w.fresh * a.G - (int64_t)w.group * G_::ROWS);
      const bool live = row < rows, warp_live = row - lane < rows;
      const int64_t at = (int64_t)w.group * G_::ROWS + row;         // row of the request and head
      const int64_t tok = at / a.G;
      const int limit = live ? (int)(w.len - w.fresh + tok) : -1;   // last slot seen
      const int floor_limit = (int)(w.len - w.fresh + (at - lane) / a.G);   // the lowest of the warp's live rows
      const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(a.q) + (w.beg + tok) * a.qt +
                                 (int64_t)(w.h * a.G + (int)(at % a.G)) * a.qh;
      float m = -INFINITY, shift = 0.f, l = 0.f, cs;
      if (WIDE || i == 0) {
        cs = put_queries<WIDE ? 8 : 4>(a, p.vec_q, src, live, qbuf + (WIDE ? i * 2 * kTileBytes : 0), warp % 4 * 32, kTileBytes, 32);
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->q_full[i]));
      } else {
        // the other group writes the rows; their factors are formed again
        cs = query_factor(a, p.vec_q, src, live);
      }
      float *spool = !WIDE && p.scores && live
                         ? p.scores + (((int64_t)w.r * a.H + w.h) * p.slot_rows + row) * p.score_ld
                         : nullptr;
      int j0 = w.step * G_::SLOTS + (WIDE ? 0 : i * kTile);
      for (int s = 0; s < 2 * count; ++s, ++half) {
        const int hf = s & 1;                     // half of the tile
        const uint32_t col = s_col + hf * kHalf;
        if (hf == 0 && !W.warp_wait(&sh->k_full[ks], k_phase)) goto done;
        if (!W.warp_wait(&sh->s_full[i][hf], half >> 1 & 1)) goto done;
        tc_fence_after();
        if (warp_live) {
          const uint32_t mask = sh->k_mask[ks] >> (16 * hf) & 0xffffu;
          const bool masked = mask != 0xffffu || j0 + kHalf - 1 > floor_limit;
          const float4 *scale = reinterpret_cast<const float4 *>(sh->ks[ks]) + 4 * hf;
          const float ref = sh->k_ref[ks];
          if (!WIDE && p.scores)     // the scores themselves, for the weights
            keep_scores(col, spool && j0 < p.score_ld ? spool + j0 : nullptr, scale, mask, limit - j0, cs);
          const auto raise = [&](float down) {
            if (s == 0) return true;
            if (!W.warp_wait(&sh->pv_done[i][(half - 1) & 1], (half - 1) >> 1 & 1)) return false;
            tc_fence_after();
            scale_down(o_col, down);
            return true;
          };
          if (!(masked ? softmax_half<true>(col, scale, mask, limit - j0, cs, ref, m, shift, l, raise)
                       : softmax_half<false>(col, scale, 0u, 0, cs, ref, m, shift, l, raise)))
            goto done;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->p_full[i][hf]));
        j0 += kHalf;
        if (hf) {
          if (lane == 0) mbar_arrive(smem_addr(&sh->k_empty[ks]));
          j0 += G_::SLOTS - kTile;
          ks += WIDE ? 1 : 2;
          if (ks >= kKStages) {
            ks -= kKStages;
            k_phase ^= 1;
          }
        }
      }
      // the result of the item, or this CTA's part of it
      const Item it{w, count, rows, row, live, warp_live, m, shift, cs != cs ? cs : l, o_col, half, joins};
      if (!finish_item<WIDE>(p, sh, it, i)) goto done;
      joins += !WIDE && count == w.steps;
    }
  done:;
  } else if (warp < kLoadWarp) {
    fewer_registers<kConvertRegs>();
    // ----------------------------------------------------------------------
    // V to f16, times 2^7 scale / (the tile's largest scale)
    // ----------------------------------------------------------------------
    const int t = tid - 8 * 32;
    uint32_t n = 0;
    for (; w.base + G_::SETUP < last; next_item<G_>(a, w)) {
      const int count = steps_here<G_>(w, last);
      int j0 = w.step * G_::SLOTS;
      for (int k = 0; k < count * (WIDE ? 1 : 2); ++k, ++n, j0 += kTile) {
        const int vs = n % kVStages, ws = n % kWStages;
        if (!W.warp_wait(&sh->v_full[vs], n / kVStages & 1)) goto cv_done;
        if (!W.warp_wait(&sh->w_empty[ws], (n / kWStages & 1) ^ 1)) goto cv_done;
        const unsigned char *src = vbuf + vs * kTileBytes;
        unsigned char *dst = wbuf + ws * 2 * kTileBytes;
        const uint32_t mask = sh->v_mask[vs];
        const float unit = sh->v_unit[vs];
        // 16 lanes a row, 8 dimensions each: loads and stores meet no bank twice
        const int c = t % 16;
        unsigned char *to = dst + (c / 8) * kTileBytes;
        const bool all = mask == ~0u && j0 + kTile <= w.len;
#pragma unroll 4
        for (int u = 0; u < 16; ++u) {
          const int j = u * 8 + t / 16;
          const float f = sh->vs[vs][j / 4] * unit;
          const uint32_t f2 = f16x2(f, f);
          const uint2 y = *reinterpret_cast<const uint2 *>(src + j * kD + ((c / 2 ^ (j & 7)) << 4) + (c % 2) * 8);
          uint4 h;
          h.x = mul_f16x2(f16x2_of(y.x), f2);
          h.y = mul_f16x2(f16x2_of(y.x >> 16), f2);
          h.z = mul_f16x2(f16x2_of(y.y), f2);
          h.w = mul_f16x2(f16x2_of(y.y >> 16), f2);
          if (!all && !((mask >> (j / 4) & 1) && j0 + j < w.len)) h = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(to + j * kD + ((c % 8 ^ (j & 7)) << 4)) = h;
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&sh->w_full[ws]));
          mbar_arrive(smem_addr(&sh->v_empty[vs]));
        }
      }
    }
  cv_done:;
  } else if (warp == kLoadWarp) {
    fewer_registers<kOtherRegs>();
    // ----------------------------------------------------------------------
    // block lookups, scales and TMA: lane l looks up slots 4l .. 4l + 3
    // ----------------------------------------------------------------------
    uint32_t n = 0;
    for (; w.base + G_::SETUP < last; next_item<G_>(a, w)) {
      const int count = steps_here<G_>(w, last);
      int j = w.step * G_::SLOTS + 4 * lane;
      for (int k = 0; k < count * (WIDE ? 1 : 2); ++k, ++n, j += kTile) {
        const int ks = n % kKStages, vs = n % kVStages;
        int page = -1;
        uint32_t off = 0;
        if (j < w.len) {
          const uint32_t block = block_of(a, j);
          off = j - block * a.bs;
          page = page_of(a, w.r, block);
          if (page < 0) raise(a.status, KVX_FLAG_BAD_BLOCK);
        }
        const uint32_t sb = page < 0 ? 0u : (uint32_t)page * a.H + w.h;
        const int row = (int)(sb * a.bs + off);
        const float kscale = page >= 0 ? __ldg(a.ks + sb) : 0.f, vscale = page >= 0 ? __ldg(a.vs + sb) : 0.f;
        const unsigned mask = __ballot_sync(~0u, page >= 0);
        // the tile's largest value scale, rounded up to a power of two 2^e.  Not below
        // 2^-96: such values vanish beside any other.  Not above 2^126: ex2 gives 0 for
        // 2^-127, and codes whose values are finite leave f16 room for the rest.
        const uint32_t most = __reduce_max_sync(~0u, __float_as_uint(vscale));
        const int e = min(max((int)(most >> 23) + ((most & 0x7fffff) != 0), 127 - 96), 127 + 126);
        const int per = p.box / 4, boxes = kTile / p.box;     // lanes a box, boxes
        const int from = __shfl_sync(~0u, row, lane < boxes ? lane * per : 0);
        const bool there = lane < boxes && (mask >> (lane * per) & 1);
        const uint32_t bytes = __popc(__ballot_sync(~0u, there)) * (uint32_t)p.box * kD;
        if (!W.warp_wait(&sh->k_empty[ks], (n / kKStages & 1) ^ 1)) goto ld_done;
        sh->ks[ks][lane] = kscale;
        if (lane == 0) {
          sh->k_mask[ks] = mask;
          sh->k_ref[ks] = (float)(e - 127);
          mbar_expect_tx(smem_addr(&sh->k_full[ks]), bytes);
        }
        __syncwarp();
        if (there)
          tma_load_2d(smem_addr(kbuf + ks * kTileBytes + lane * p.box * kD), &map_k, 0, from,
                      smem_addr(&sh->k_full[ks]));
        if (lane != 0) mbar_arrive(smem_addr(&sh->k_full[ks]));
        if (!W.warp_wait(&sh->v_empty[vs], (n / kVStages & 1) ^ 1)) goto ld_done;
        sh->vs[vs][lane] = vscale;
        if (lane == 0) {
          sh->v_mask[vs] = mask;
          sh->v_unit[vs] = __uint_as_float((uint32_t)(254 + 7 - e) << 23);
          mbar_expect_tx(smem_addr(&sh->v_full[vs]), bytes);
        }
        __syncwarp();
        if (there)
          tma_load_2d(smem_addr(vbuf + vs * kTileBytes + lane * p.box * kD), &map_v, 0, from,
                      smem_addr(&sh->v_full[vs]));
        if (lane != 0) mbar_arrive(smem_addr(&sh->v_full[vs]));
      }
    }
  ld_done:
    // drain: the tiles that were asked for have landed (n counts whole tiles; after
    // an abort the last keys may be one ahead of the values)
    __syncwarp();
    if (lane == 0) {
      for (uint32_t x = n > kKStages ? n - kKStages : 0; x < n; ++x) drain_wait(&sh->k_full[x % kKStages], x / kKStages & 1);
      for (uint32_t x = n > kVStages ? n - kVStages : 0; x < n; ++x) drain_wait(&sh->v_full[x % kVStages], x / kVStages & 1);
      if (sh->abort) drain_wait(&sh->k_full[n % kKStages], n / kKStages & 1);
    }
  } else if (warp < kMmaWarp + 2) {
    fewer_registers<kOtherRegs>();
    // ----------------------------------------------------------------------
    // the MMAs: a warp for each group, so that one's waits hide behind the
    // other's products
    // ----------------------------------------------------------------------
    const int i = warp - kMmaWarp;
    const uint64_t q0 = sw128_desc(smem_addr(qbuf)) + (WIDE ? (uint64_t)i * (2 * kTileBytes >> 4) : 0);
    const uint64_t k0 = sw128_desc(smem_addr(kbuf)), v0 = mn_desc(smem_addr(wbuf));
    const uint32_t s_col = tmem + i * kTile, o_col = tmem + 2 * kTile + i * kTile;
    uint32_t items = 0, u = 0;       // items, and the group's half tiles whose products were begun
    bool ok = true, issued = false;
    const auto tile_of = [&](uint32_t half) { return WIDE ? half >> 1 : (half >> 1) * 2 + i; };   // of the CTA
    const auto scores = [&](uint32_t half) {
      const uint32_t stage = tile_of(half) % kKStages, hf = half & 1;
      if (!W.warp_wait(&sh->k_full[stage], tile_of(half) / kKStages & 1)) return false;
      tc_fence_after();
      mma_qk(s_col + hf * kHalf, q0, k0 + (uint64_t)(stage * kTileBytes + hf * kHalf * kD >> 4));
      issued = true;
      commit(&sh->s_full[i][hf]);
      if (hf) commit(&sh->k_empty[stage]);
      return true;
    };
    for (; ok && w.base + G_::SETUP < last; next_item<G_>(a, w)) {
      const int count = steps_here<G_>(w, last);
      ok = W.warp_wait(&sh->q_full[WIDE ? i : 0], items & 1) && scores(u) && scores(u + 1);
      ++items;
      for (int s = 0; ok && s < 2 * count; ++s, ++u) {
        const uint32_t stage = tile_of(u) % kWStages, hf = u & 1;
        ok = W.warp_wait(&sh->w_full[stage], tile_of(u) / kWStages & 1) && W.warp_wait(&sh->p_full[i][hf], u >> 1 & 1);
        if (!ok) break;
        tc_fence_after();
        mma_pv(o_col, s_col + hf * kHalf, v0 + (uint64_t)(stage * 2 * kTileBytes + hf * kHalf * kD >> 4), s > 0);
        commit(&sh->pv_done[i][hf]);
        if (hf) commit(&sh->w_empty[stage]);
        // two halves on, over the probabilities just spent: MMAs run in order
        if (s + 2 < 2 * count) ok = scores(u + 2);
      }
    }
    if (issued) {
      commit(&sh->drain[i]);
      if (lane == 0) drain_wait(&sh->drain[i], 0);
    }
    __syncwarp();
  } else {
    fewer_registers<kOtherRegs>();   // the split counts whole warpgroups
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// weights[r][h][j] += sum over the rows of exp2(score - lse): narrow calls leave
// their scores, [rows][score_ld].
__global__ void __launch_bounds__(256) weights_of_rows_kernel(const __grid_constant__ TcParams p) {
  const AttendParams &a = p.a;
  extern __shared__ float2 lse2[];
  __shared__ float lse1[64];     // of near rows as one number
  const bool good = requests_ok(a);
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(a, r);
  const int64_t beg = a.req.begin(r);
  const int rows = (int)(a.req.begin(r + 1) - beg) * a.G;
  wait_for_kernel_before();
  if (!good) return;
  bool far = false;
  for (int c = threadIdx.x; c < rows; c += 256) {
    const float2 lse = a.stats[(beg + c / a.G) * a.Hq + h * a.G + c % a.G];
    lse2[c] = lse;
    lse1[c] = lse.x + lse.y;
    far = fabsf(lse.x) > kFar;
  }
  far = __syncthreads_or(far);
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= len || rows == 0) return;
  const float *x = p.scores + ((int64_t)r * a.H + h) * p.slot_rows * p.score_ld + j;
  float sum = 0.f;
  if (!far) {
#pragma unroll 8
    for (int c = 0; c < rows; ++c) {
      const float z = x[(int64_t)c * p.score_ld];
      sum += z > -INFINITY ? ex2(z - lse1[c]) : 0.f;
    }
  } else {
    for (int c = 0; c < rows; ++c) {
      const float z = x[(int64_t)c * p.score_ld];
      sum += z > -INFINITY ? probability(z, lse2[c]) : 0.f;
    }
  }
  a.weights[((int64_t)r * a.H + h) * a.wstride + j] += sum;
}

// --- few columns --------------------------------------------------------------------
// At most 16 (query, head of the group) pairs: one token of a group of heads, or a
// few.  128 rows of which 8 count would cost the shared memory more than HBM can
// bring, so here the slots are the rows and the pairs the columns, and neither K nor
// V is converted: both products take the codes as they lie in the cache.
//   S^T = K (Q1 + Q2)^T   the queries in two e4m3 parts, a slot to a lane,
//   O^T += V^T P^T        P in three e5m2 parts (3 + 3 + 3 bits: an f16 value to
//                         2^-10 of it), formed from the top bytes of an f16 and of
//                         what it leaves; V transposed by the descriptor.
// A slot's probabilities carry its block's value scale (as a power in the
// exponent), so that O needs none; sums without it are kept beside.  Four warps
// share a maximum for each column: they vote on a tile, and only where one of them
// exceeds it by 2^4 do they agree on a new one and scale O down.  The maximum is of score
// plus value scale; once one is beyond kFar, where that sum's rounding would count, an
// item takes the largest score and the largest value scale apart.
// Two groups of four warps take the even and the odd slot tiles.
// One query of 64 heads over 131,071 slots of 8 heads takes 57 us, 4.7 TB/s (a copy
// 6.7); 16 requests of 1024 to 16,384 slots 73 us, and with 16 columns, which read the
// same bytes, 94: the chain of a tile's softmax counts beside them.  The narrow form
// above takes 146 there, matrix instructions on registers (16 x 8 x 16) 88 with 8.
// even numbers of stages: a stage serves one group, whose waits on it then know
// that the phase before is over
constexpr int kCkStages = 4, kCvStages = 6, kScales = 16, kColThreads = 12 * 32;
constexpr int kColLoad = 8, kColMma = 10;   // keys and values; a group each
constexpr float kColBias = 11.f, kColSlack = 4.f;   // P at most 2^15, nothing lost above 2^-28 of the maximum
constexpr int kColQBytes = 32 * kD, kColPBytes = kTile * 16;   // a part of the queries, of a tile's probabilities
struct ColShared {
  uint64_t k_full[kCkStages], k_empty[kCkStages], v_full[kCvStages], v_empty[kCvStages];
  // scales[n % kScales] of tile n: the loader is never that far ahead of the softmax
  uint64_t scales[kScales], q_full[2], item_done[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], vote[2], agree[2], join, spent, drain[2];
  uint32_t tmem_base;
  volatile int abort;
  Share share;
  volatile uint32_t over[2][2];
  uint32_t mask[kScales];
  float ks[kScales][kTile / 4], vs[kScales][kTile / 4];
  float cs[2][16];             // of the item (in turn) and column
  float warp_max[2][4][16], warp_sum[2][4][16];
  float far_max[2][4][17];     // scores by column, then value scales
};
constexpr size_t kColSmem = 1024 + (kCkStages + kCvStages) * (size_t)kTileBytes + 4 * kColQBytes + 2 * 2 * 3 * kColPBytes +
                            sizeof(ColShared);
static_assert(kColSmem <= 227 * 1024, "shared memory");
// D fp32, M = 128, N = 16; e4m3 both K-major, and e4m3 x e5m2 both as they lie in
// memory (MN-major).
constexpr uint32_t kIdescColS = (1u << 4) | (2u << 17) | (8u << 24);
constexpr uint32_t kIdescColO = (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | (2u << 17) | (8u << 24);

// 32 slots deep each: four steps for each of two query parts, for each of three
// parts of P.
__device__ __forceinline__ void mma_col_s(uint32_t d, uint64_t k, uint64_t q) {
  asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b32 r;\n.reg .b64 a1, a2, a3, b1, b2, b3, b4, b5, b6, b7;\n"
      "elect.sync r|e, 0xffffffff;\n"
      "setp.ne.u32 f, 0, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u64 a1, %1, 2; add.u64 a2, %1, 4; add.u64 a3, %1, 6;\n"
      "add.u64 b1, %2, 2; add.u64 b2, %2, 4; add.u64 b3, %2, 6; add.u64 b4, %2, %4;\n"
      "add.u64 b5, b4, 2; add.u64 b6, b4, 4; add.u64 b7, b4, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, b4, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b5, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b6, %3, t;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b7, %3, t;\n}\n" ::"r"(d),
      "l"(k), "l"(q), "r"(kIdescColS), "l"((uint64_t)(kColQBytes >> 4))
      : "memory");
}
__device__ __forceinline__ void mma_col_o(uint32_t d, uint64_t v, uint64_t p, bool add) {
#pragma unroll
  for (int part = 0; part < 3; ++part)
    asm volatile(
        "{\n.reg .pred e, f, t;\n.reg .b32 r;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"
        "elect.sync r|e, 0xffffffff;\n"
        "setp.ne.u32 f, %4, 0;\nsetp.eq.u32 t, 0, 0;\n"
        "add.u64 a1, %1, 256; add.u64 a2, %1, 512; add.u64 a3, %1, 768;\n"
        "add.u64 b1, %2, 32; add.u64 b2, %2, 64; add.u64 b3, %2, 96;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(v), "l"(p + (uint64_t)part * (kColPBytes >> 4)), "r"(kIdescColO), "r"((uint32_t)(add || part > 0))
        : "memory");
}
// V as operand [slots][128 dimensions], 128-byte swizzle: one 128-dimension group,
// 8-slot groups 1 KB apart.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(1024 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// P as operand [slots][16 columns], no swizzle: 8-slot groups 128 bytes apart.
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(kColPBytes >> 4) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\ntcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld8_wait(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\ntcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(addr)
      : "memory");
}
template <int NC>
__device__ __forceinline__ void ld_columns(uint32_t addr, uint32_t (&v)[NC]) {
  if constexpr (NC == 8) tc_ld8_wait(addr, v);
  else tc_ld16(addr, v);
}
template <int NC>
__device__ __forceinline__ void st_columns(uint32_t addr, const uint32_t (&v)[NC]) {
  if constexpr (NC == 8) tc_st8(addr, v);
  else tc_st16(addr, v);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int NC>
__global__ void __launch_bounds__(kColThreads, 1)
    columns_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v) {
  using G_ = Columns<NC>;
  extern __shared__ unsigned char raw[];
  unsigned char *kbuf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  unsigned char *vbuf = kbuf + kCkStages * kTileBytes, *qbuf = vbuf + kCvStages * kTileBytes, *pbuf = qbuf + 4 * kColQBytes;
  ColShared *sh = reinterpret_cast<ColShared *>(pbuf + 2 * 2 * 3 * kColPBytes);
  const AttendParams &a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    for (int i = 0; i < kCkStages; ++i) {
      mbar_init(smem_addr(&sh->k_full[i]), 32);
      mbar_init(smem_addr(&sh->k_empty[i]), 1);
    }
    for (int i = 0; i < kScales; ++i) mbar_init(smem_addr(&sh->scales[i]), 32);
    for (int i = 0; i < kCvStages; ++i) {
      mbar_init(smem_addr(&sh->v_full[i]), 32);
      mbar_init(smem_addr(&sh->v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&sh->s_full[i][b]), 1);
        mbar_init(smem_addr(&sh->p_full[i][b]), 4);
        mbar_init(smem_addr(&sh->pv_done[i][b]), 1);
        sh->over[i][b] = 0;
      }
      mbar_init(smem_addr(&sh->q_full[i]), 1);
      mbar_init(smem_addr(&sh->item_done[i]), 8);
      mbar_init(smem_addr(&sh->vote[i]), 4);
      mbar_init(smem_addr(&sh->agree[i]), 4);
      mbar_init(smem_addr(&sh->drain[i]), 1);
    }
    mbar_init(smem_addr(&sh->join), 8);
    mbar_init(smem_addr(&sh->spent), 8);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kColMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(
                     smem_addr(&sh->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kColLoad) {
    Share share;
    find_share<G_>(a, blockIdx.x, gridDim.x, blockIdx.x == 0, share);
    if (lane == 0) {
      sh->share = share;
      note_split<G_>(p, share);
      if (!share.good && blockIdx.x == 0) raise(a.status, KVX_FLAG_BAD_SEQLENS);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const WaiterT<ColShared> W{sh, a.status};
  TcWalk w = sh->share.w;
  const int64_t last = sh->share.last;
  // scores of group i, buffer b; sums of group i
  const auto s_at = [&](int i, int b) { return tmem + (i * 2 + b) * 16; };
  const auto o_at = [&](int i) { return tmem + 64 + i * 16; };

  if (warp < 8) {
    const int i = warp / 4, in = warp % 4 * 32 + lane;      // group; slot of the tile, dimension of the sums
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    uint32_t t = 0, items = 0, joins = 0, agreed = 0;       // tiles of the group, items, joins, agreements so far
    // the queries: warp 0 brings an item's while the one before is worked on
    const auto bring = [&](const TcWalk &w, uint32_t item) {
      const int64_t row0 = (int64_t)w.group * NC, tok = (row0 + lane) / a.G;
      const int rows = (int)min((int64_t)NC, (int64_t)w.fresh * a.G - row0);
      const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(a.q) + (w.beg + tok) * a.qt +
                                 (int64_t)(w.h * a.G + (int)((row0 + lane) % a.G)) * a.qh;
      const float f = put_queries<4>(a, p.vec_q, src, lane < rows, qbuf + (item & 1) * 2 * kColQBytes, 0, kColQBytes, 16);
      if (lane < 16) sh->cs[item & 1][lane] = f;
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh->q_full[item & 1]));
    };
    if (warp == 0 && w.base + G_::SETUP < last) bring(w, 0);
    for (; w.base + G_::SETUP < last; next_item<G_>(a, w), ++items) {
      const int count = steps_here<G_>(w, last);
      const int64_t row0 = (int64_t)w.group * NC;
      const int rows = (int)min((int64_t)NC, (int64_t)w.fresh * a.G - row0);
      if (warp == 0) {
        // the next item's queries, once both groups have formed the last scores of
        // the item before this one
        TcWalk ahead = w;
        next_item<G_>(a, ahead);
        if (ahead.base + G_::SETUP < last) {
          if (items > 0 && !W.warp_wait(&sh->item_done[(items + 1) & 1], (items - 1) >> 1 & 1)) goto done;
          bring(ahead, items + 1);
        }
      }
      float cs[NC], m[NC], l[NC], shift = 0.f;   // sums are relative to exp2(m + shift - kColBias)
      bool far = false;
      if (!W.warp_wait(&sh->q_full[items & 1], items >> 1 & 1)) goto done;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        cs[c] = sh->cs[items & 1][c];
        m[c] = -FLT_MAX;     // nothing seen: any score is over it
        l[c] = 0.f;
      }
      const int low = (int)(w.len - w.fresh + row0 / a.G);   // last slot that the first column sees
      float *spool = p.scores ? p.scores + ((int64_t)w.r * a.H + w.h) * p.score_ld * (int64_t)NC : nullptr;
      int j = w.step * G_::SLOTS + i * kTile + in;
      for (int s = 0; s < count; ++s, ++t) {
        const int b = t & 1;
        const uint32_t tile = 2 * t + i;
        const int ks = tile % kScales;
        if (!W.warp_wait(&sh->scales[ks], tile / kScales & 1)) goto done;
        if (!W.warp_wait(&sh->s_full[i][b], t >> 1 & 1)) goto done;
        tc_fence_after();
        const float f = sh->ks[ks][in / 4], v = sh->vs[ks][in / 4];
        const bool there = sh->mask[ks] >> (in / 4) & 1;
        // value scales below 2^-96 count as that (their values vanish beside any other)
        const float lv = there ? fmaxf(lg2(v), -96.f) : 0.f;
        uint32_t x[NC];
        ld_columns<NC>(s_at(i, b) + lanes, x);
        float y[NC];           // scores, base 2
        const bool masked = __any_sync(~0u, !there || j > low);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          y[c] = __uint_as_float(x[c]) * f * cs[c];
          if (masked && (!there || j > (int)(w.len - w.fresh + (row0 + c) / a.G) || c >= rows)) y[c] = -INFINITY;
        }
        if (spool && j < p.score_ld) {
#pragma unroll
          for (int c = 0; c < NC; c += 4)
            *reinterpret_cast<float4 *>(spool + (int64_t)j * NC + c) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
        }
        // exponents of the probabilities times the value scale: score less maximum, which
        // are near each other where it counts, comes first
        float e[NC];
        bool over = false;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          e[c] = (y[c] - m[c]) + (lv - shift + kColBias);
          over = over || e[c] > kColBias + kColSlack;
        }
        if (__any_sync(~0u, over) && lane == 0) sh->over[i][b] = t + 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->vote[i]));
        if (!W.warp_wait(&sh->vote[i], t & 1)) goto done;
        if (sh->over[i][b] == t + 1) {
          // seldom: a new maximum for all columns, and O scaled down to it
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            float top = y[c] + lv;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            if (lane == 0) sh->warp_max[i][warp % 4][c] = top;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh->agree[i]));
          if (!W.warp_wait(&sh->agree[i], agreed++ & 1)) goto done;
          float down[NC], by = 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, sh->warp_max[i][k][c]);
            far = far || is_far(top);
            down[c] = fmaxf(m[c], top);      // the new maximum
          }
          if (__builtin_expect(far, 0)) {
            // the same of scores alone, and the largest value scale
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              float top = y[c];
#pragma unroll
              for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
              if (lane == 0) sh->far_max[i][warp % 4][c] = top;
            }
            float top = lv;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            if (lane == 0) sh->far_max[i][warp % 4][NC] = top;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh->agree[i]));
            if (!W.warp_wait(&sh->agree[i], agreed++ & 1)) goto done;
            by = -shift;
#pragma unroll
            for (int k = 0; k < 4; ++k) shift = fmaxf(shift, sh->far_max[i][k][NC]);
            by += shift;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              down[c] = m[c];
#pragma unroll
              for (int k = 0; k < 4; ++k) down[c] = fmaxf(down[c], sh->far_max[i][k][c]);
            }
          }
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float top = down[c];
            down[c] = ex2((m[c] - top) - by);
            m[c] = top;
            l[c] *= down[c];
            e[c] = (y[c] - top) + (lv - shift + kColBias);
          }
          if (s > 0) {
            if (!W.warp_wait(&sh->pv_done[i][(t - 1) & 1], (t - 1) >> 1 & 1)) goto done;
            tc_fence_after();
            uint32_t o[NC];
            ld_columns<NC>(o_at(i) + lanes, o);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * down[c]);
            st_columns<NC>(o_at(i) + lanes, o);
            tc_wait_st();
          }
        }
        // probabilities times the value scale, and sums without it
        const float root = ex2(-0.5f * lv), without = root * root;   // ex2 gives 0 for 2^-127
        uint32_t h[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float e0 = ex2(e[c]), e1 = ex2(e[c + 1]);
          l[c] = fmaf(e0, without, l[c]);
          l[c + 1] = fmaf(e1, without, l[c + 1]);
          h[c / 2] = f16x2(e0, e1);
        }
        if (__any_sync(~0u, !there || j >= w.len)) {
          // slots of no block of the pool or beyond the length: zero values, so that
          // their zero probabilities meet no NaN
          const uint32_t vstage = tile % kCvStages;
          if (!W.warp_wait(&sh->v_full[vstage], tile / kCvStages & 1)) goto done;
          if (!there || j >= w.len) {
            uint4 *row = reinterpret_cast<uint4 *>(vbuf + vstage * kTileBytes + in * kD);
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) row[k] = make_uint4(0, 0, 0, 0);
          }
        }
        // the buffer's last products are done
        if (t >= 2 && !W.warp_wait(&sh->pv_done[i][b], (t - 2) >> 1 & 1)) goto done;
        unsigned char *to = pbuf + (i * 2 + b) * 3 * kColPBytes + in * 16;
        uint32_t part[3][4] = {};
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const uint32_t a0 = h[c / 2], a1 = h[c / 2 + 1];
          const uint32_t r0 = sub_f16x2(a0, a0 & 0xff00ff00u), r1 = sub_f16x2(a1, a1 & 0xff00ff00u);
          const uint32_t q0 = sub_f16x2(r0, r0 & 0xff00ff00u), q1 = sub_f16x2(r1, r1 & 0xff00ff00u);
          part[0][c / 4] = __byte_perm(a0, a1, 0x7531);
          part[1][c / 4] = __byte_perm(r0, r1, 0x7531);
          part[2][c / 4] = e5m2x2(q0) | e5m2x2(q1) << 16;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4 *>(to + k * kColPBytes) = make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
        fence_async_proxy();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&sh->p_full[i][b]));
        }
        j += G_::SLOTS;
      }
      if (lane == 0) mbar_arrive(smem_addr(&sh->item_done[items & 1]));
      // this group's part of the item
      if (!W.warp_wait(&sh->pv_done[i][(t - 1) & 1], (t - 1) >> 1 & 1)) goto done;
      if (joins > 0 && !W.warp_wait(&sh->spent, (joins - 1) & 1)) goto done;
      tc_fence_after();
      uint32_t o[NC];
      ld_columns<NC>(o_at(i) + lanes, o);
      float *slot = p.partial + (((int64_t)blockIdx.x * 2 + (w.step == 0)) * 2 + i) * (int64_t)p.part_size;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c < rows) slot[c * kD + in] = __uint_as_float(o[c]);
        float sum = l[c];
#pragma unroll
        for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
        if (lane == 0) sh->warp_sum[i][warp % 4][c] = sum;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh->agree[i]));
      if (!W.warp_wait(&sh->agree[i], agreed++ & 1)) goto done;
      if (warp % 4 == 0 && lane < rows) {
        float mine = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) mine = lane == c ? m[c] : mine;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += sh->warp_sum[i][k][lane];
        leave_part(slot + p.slot_rows * kD, p.slot_rows, lane, mine > -FLT_MAX ? mine : -INFINITY, shift - kColBias, sum);
      }
      if (count == w.steps) {
        // an item of this CTA alone: its two parts
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->join));
        if (!W.warp_wait(&sh->join, joins & 1)) goto done;
        join_rows<G_, 1>(p, w, blockIdx.x, 1, warp, 8, rows);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->spent));
        ++joins;
      }
    }
  done:;
  } else if (warp < kColMma) {
    // A warp loads the keys and all scales, another the values.  A tile's blocks are
    // looked up two tiles ahead, their scales one: nothing waits for them.
    const bool keys = warp == kColLoad;
    struct Tile {
      int page, off;
      bool asked;
    };
    int k = 0, end = 0, j = 0;      // tile of the item, tiles of the item in this CTA, the lane's first slot
    bool more = w.base + G_::SETUP < last;
    const auto enter = [&]() {
      k = 0;
      end = 2 * steps_here<G_>(w, last);
      j = w.step * G_::SLOTS + 4 * lane;
    };
    if (more) enter();
    const auto next = [&](Tile &x, int &h) {
      x.asked = more;
      x.page = -1;
      x.off = 0;
      h = w.h;
      if (!more) return;
      if (j < w.len) {
        const uint32_t block = block_of(a, j);
        x.off = j - block * a.bs;
        x.page = page_of(a, w.r, block);
        if (x.page < 0 && keys) raise(a.status, KVX_FLAG_BAD_BLOCK);
      }
      j += kTile;
      if (++k == end) {
        next_item<G_>(a, w);
        more = w.base + G_::SETUP < last;
        if (more) enter();
      }
    };
    Tile t0, t1;
    int h0, h1;
    float f0 = 0.f, g0 = 0.f;
    const auto scales = [&](const Tile &x, int h, float &f, float &g) {
      f = g = 0.f;
      if (x.page < 0 || !keys) return;
      const uint32_t sb = (uint32_t)x.page * a.H + h;
      f = __ldg(a.ks + sb);
      g = __ldg(a.vs + sb);
    };
    next(t0, h0);
    scales(t0, h0, f0, g0);
    next(t1, h1);
    const int stages = keys ? kCkStages : kCvStages, per = p.box / 4, boxes = kTile / p.box;   // lanes a box, boxes
    uint64_t *full = keys ? sh->k_full : sh->v_full, *empty = keys ? sh->k_empty : sh->v_empty;
    unsigned char *buf = keys ? kbuf : vbuf;
    const CUtensorMap *map = keys ? &map_k : &map_v;
    uint32_t n = 0, phase = 0;
    for (int st = 0; t0.asked; ++n) {
      const int row = t0.page < 0 ? 0 : (int)(((uint32_t)t0.page * a.H + h0) * a.bs + t0.off);
      const unsigned mask = __ballot_sync(~0u, t0.page >= 0);
      const float kscale = f0, vscale = g0;
      // what the next tiles need, on its way
      t0 = t1;
      h0 = h1;
      scales(t0, h0, f0, g0);
      next(t1, h1);
      const int from = __shfl_sync(~0u, row, lane < boxes ? lane * per : 0);
      const bool there = lane < boxes && (mask >> (lane * per) & 1);
      const uint32_t bytes = __popc(__ballot_sync(~0u, there)) * (uint32_t)p.box * kD;
      if (!W.warp_wait(&empty[st], phase ^ 1)) break;
      if (keys) {
        const int sc = n % kScales;
        sh->ks[sc][lane] = kscale;
        sh->vs[sc][lane] = vscale;
        if (lane == 0) sh->mask[sc] = mask;
        __syncwarp();
        mbar_arrive(smem_addr(&sh->scales[sc]));
      }
      if (lane == 0) mbar_expect_tx(smem_addr(&full[st]), bytes);
      __syncwarp();
      if (there) tma_load_2d(smem_addr(buf + st * kTileBytes + lane * p.box * kD), map, 0, from, smem_addr(&full[st]));
      if (lane != 0) mbar_arrive(smem_addr(&full[st]));
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
    if (lane == 0)
      for (uint32_t x = n > (uint32_t)stages ? n - stages : 0; x < n; ++x) drain_wait(&full[x % stages], x / stages & 1);
  } else {
    const int i = warp - kColMma;
    const uint64_t k0 = sw128_desc(smem_addr(kbuf)), v0 = v_desc(smem_addr(vbuf));
    uint64_t q0 = 0;                 // the item's queries
    const uint64_t p0 = p_desc(smem_addr(pbuf + i * 2 * 3 * kColPBytes));
    uint32_t items = 0, t = 0;
    bool ok = true, issued = false;
    const auto scores = [&](uint32_t t) {
      const uint32_t tile = 2 * t + i, stage = tile % kCkStages;
      if (!W.warp_wait(&sh->k_full[stage], tile / kCkStages & 1)) return false;
      tc_fence_after();
      mma_col_s(s_at(i, t & 1), k0 + (uint64_t)(stage * kTileBytes >> 4), q0);
      issued = true;
      commit(&sh->s_full[i][t & 1]);
      commit(&sh->k_empty[stage]);
      return true;
    };
    for (; ok && w.base + G_::SETUP < last; next_item<G_>(a, w)) {
      const int count = steps_here<G_>(w, last);
      q0 = sw128_desc(smem_addr(qbuf + (items & 1) * 2 * kColQBytes));
      ok = W.warp_wait(&sh->q_full[items & 1], items >> 1 & 1) && scores(t) && (count == 1 || scores(t + 1));
      ++items;
      for (int s = 0; ok && s < count; ++s, ++t) {
        const uint32_t tile = 2 * t + i, stage = tile % kCvStages;
        ok = W.warp_wait(&sh->v_full[stage], tile / kCvStages & 1) && W.warp_wait(&sh->p_full[i][t & 1], t >> 1 & 1);
        if (!ok) break;
        tc_fence_after();
        mma_col_o(o_at(i), v0 + (uint64_t)(stage * kTileBytes >> 4), p0 + (uint64_t)((t & 1) * 3 * kColPBytes >> 4), s > 0);
        commit(&sh->pv_done[i][t & 1]);
        commit(&sh->v_empty[stage]);
        if (s + 2 < count) ok = scores(t + 2);   // its buffer's scores were read before P came
      }
    }
    if (issued) {
      commit(&sh->drain[i]);
      if (lane == 0) drain_wait(&sh->drain[i], 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kColMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
}

// --- accumulated weights where the scores were not kept ----------------------------
// weights[r][h][j] += sum over the rows that see slot j of exp2(score - lse).
// The scores are formed again, transposed (S^T = K Q^T, slots in the lanes), so
// that a slot's sum stays in one thread: no atomics, one order of summation.  A CTA
// takes up to `per` slot tiles of one request and head, spread over its length because
// fewer rows see the late ones, and the rows 256 at a time; two groups of four warps
// take turns with the tiles.  Bound by the exponentials' chain and, where a CTA has
// few tiles, by laying out the rows: 26 us for 244 rows and two requests of 8192.
constexpr int kWtStages = 4, kWtThreads = 10 * 32, kWtTiles = 16;   // tiles: of a CTA at most
struct WtShared {
  uint64_t k_full[kWtStages], k_empty[kWtStages], q_full, spent, s_full[2], s_empty[2], drain;
  uint32_t tmem_base;
  volatile int abort;
  uint32_t mask[kWtStages];
  float ks[kWtStages][kTile / 4];
  float sum[kWtTiles][kTile];
  __align__(16) float4 rows[kTile];   // of row pairs: two factors, two log-sum-exps (base 2, negative)
  __align__(16) float4 terms[kTile];  // the log-sum-exps' two terms: two scores, two rests (negative)
  int far[8];                         // a warp's rows with scores beyond kFar
};
constexpr size_t kWtSmem = 1024 + kSmemQ + kWtStages * (size_t)kTileBytes + sizeof(WtShared);
// A slot's sum over 256 columns, of which those below `from` do not see it, where some
// scores are beyond kFar: they are rounded as the attention kernel did, then the two terms
// of their row's log-sum-exp are subtracted.
__device__ __noinline__ float far_weights(uint32_t col, float f, int from, const WtShared *sh) {
  float sum = 0.f;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint32_t s[32];
    tc_ld32(col + 32 * q, s);
    tc_wait_ld32(s);
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float4 k = sh->rows[16 * q + e / 2];
      const float4 t = sh->far[q] ? sh->terms[16 * q + e / 2] : make_float4(k.z, k.w, 0.f, 0.f);   // of warp q
      const float z0 = __fmul_rn(__uint_as_float(s[e]), fmaxf(f * k.x, 0x1p-126f));
      const float z1 = __fmul_rn(__uint_as_float(s[e + 1]), fmaxf(f * k.y, 0x1p-126f));
      part += 32 * q + e >= from ? ex2((z0 + t.x) + t.z) : 0.f;
      part += 32 * q + e + 1 >= from ? ex2((z1 + t.y) + t.w) : 0.f;
    }
    sum += part;
  }
  return sum;
}

__global__ void __launch_bounds__(kWtThreads, 1)
    weights_tc_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap map_k, int per) {
  extern __shared__ unsigned char raw[];
  unsigned char *qbuf = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  unsigned char *kbuf = qbuf + kSmemQ;
  WtShared *sh = reinterpret_cast<WtShared *>(kbuf + kWtStages * kTileBytes);
  const AttendParams &a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(a, r);
  // the CTA's tiles, at most `per`: t0, t0 + step, ...
  const int all = (len + kTile - 1) / kTile, step = (all + per - 1) / per, t0 = blockIdx.x;
  const int tiles = t0 < step ? (all - t0 - 1) / step + 1 : 0;
  const auto tile_at = [&](int t) { return t0 + t * step; };
  for (int x = tid; x < kWtTiles * kTile; x += kWtThreads) (&sh->sum[0][0])[x] = 0.f;
  if (tid == 0) {
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(smem_addr(&sh->k_full[i]), 32);
      mbar_init(smem_addr(&sh->k_empty[i]), 1 + 4);
    }
    mbar_init(smem_addr(&sh->q_full), 8);
    mbar_init(smem_addr(&sh->spent), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh->s_full[i]), 1);
      mbar_init(smem_addr(&sh->s_empty[i]), 4);
    }
    mbar_init(smem_addr(&sh->drain), 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sh->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  const bool good = requests_ok(a);
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const WaiterT<WtShared> W{sh, a.status};
  const int64_t beg = a.req.begin(r);
  const int fresh = good ? (int)(a.req.begin(r + 1) - beg) : 0, rows = fresh * a.G;
  // rows that see the CTA's first slot: from the first query whose limit reaches it
  const int row0 = max(0, t0 * kTile - (len - fresh)) * a.G / (2 * kTile) * (2 * kTile);
  const int chunks = tiles > 0 && row0 < rows ? (rows - row0 + 2 * kTile - 1) / (2 * kTile) : 0;
  // how many of the tiles the chunk's last row sees: all of them in the last chunk
  const auto seen = [&](int c) {
    const int limit = len - fresh + (min(row0 + (c + 1) * 2 * kTile, rows) - 1) / a.G, t = limit / kTile - t0;
    return limit < 0 || t < 0 ? 0 : min(tiles, t / step + 1);
  };
  if (chunks == 0) wait_for_kernel_before();   // every CTA does, so that this kernel ends after that one

  if (warp < 8) {
    const int i = warp / 4;
    const uint32_t s_col = tmem + ((uint32_t)(warp % 4 * 32) << 16) + i * 2 * kTile;
    for (int c = 0, n = 0; c < chunks; ++c) {
      // queries: a row a thread, once all warps are through with the rows before
      if (c > 0 && !W.warp_wait(&sh->spent, (c - 1) & 1)) goto done;
      const int row = row0 + c * 2 * kTile + tid;
      const bool live = row < rows;
      const int64_t tok = beg + row / a.G;
      const int hq = h * a.G + row % a.G;
      const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(a.q) + tok * a.qt + (int64_t)hq * a.qh;
      const float cs = put_queries<4>(a, p.vec_q, src, live, qbuf + i * 2 * kTileBytes, warp % 4 * 32, kTileBytes, 32);
      float *pair_of = reinterpret_cast<float *>(&sh->rows[tid / 2]) + tid % 2;
      float *terms_of = reinterpret_cast<float *>(&sh->terms[tid / 2]) + tid % 2;
      if (c == 0) wait_for_kernel_before();   // the log-sum-exps
      // a dead row gives exp2(-inf)
      const float2 lse = live ? a.stats[tok * a.Hq + hq] : make_float2(0.f, INFINITY);
      pair_of[0] = live ? cs : 0.f;
      pair_of[2] = -(lse.x + lse.y);
      const bool beyond = __any_sync(~0u, fabsf(lse.x) > kFar);
      if (beyond) {
        terms_of[0] = -lse.x;
        terms_of[2] = -lse.y;
      }
      if (lane == 0) sh->far[warp] = beyond;
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh->q_full));
      if (!W.warp_wait(&sh->q_full, c & 1)) goto done;   // the other rows' constants
      const auto work = [&](auto far) {
        const int count = seen(c);
        for (int t = 0; t < count; ++t, ++n) {
          if ((n & 1) != i) continue;
          const int ks = n % kWtStages, j = tile_at(t) * kTile + warp % 4 * 32 + lane;
          if (!W.warp_wait(&sh->k_full[ks], n / kWtStages & 1)) return false;
          if (!W.warp_wait(&sh->s_full[i], n >> 1 & 1)) return false;
          tc_fence_after();
          const int in = warp % 4 * 32 + lane;
          const float f = sh->ks[ks][in / 4];
          const bool there = j < len && (sh->mask[ks] >> (in / 4) & 1);
          // columns below `from` do not see the slot
          const int from = (int)min((int64_t)INT32_MAX, max((int64_t)j - (len - fresh), (int64_t)0) * a.G) - (row0 + c * 2 * kTile);
          const bool masked = __any_sync(~0u, from > 0);
          const uint64_t f2 = pair(f, f);
          uint64_t sum = pair(0.f, 0.f);
          if constexpr (decltype(far)::value) sum = pair(far_weights(s_col, f, from, sh), 0.f);
#pragma unroll 1
          for (int q = decltype(far)::value ? 8 : 0; q < 8; ++q) {
            uint32_t s[32];
            tc_ld32(s_col + 32 * q, s);
            tc_wait_ld32(s);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float4 k = sh->rows[16 * q + e / 2];
              float x0, x1;
              unpair(fma2(mul2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f2), pair(k.x, k.y), pair(k.z, k.w)),
                     x0, x1);
              if (masked) {
                x0 = 32 * q + e >= from ? x0 : -INFINITY;
                x1 = 32 * q + e + 1 >= from ? x1 : -INFINITY;
              }
              sum = add2(sum, pair(ex2(x0), ex2(x1)));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&sh->s_empty[i]));
            mbar_arrive(smem_addr(&sh->k_empty[ks]));
          }
          float u0, u1;
          unpair(sum, u0, u1);
          // a slot's sum passes from group to group with the chunks
          float *total = &sh->sum[t][in];
          if (c + 1 < chunks) *total += u0 + u1;
          else if (there) a.weights[((int64_t)r * a.H + h) * a.wstride + j] += *total + (u0 + u1);
        }
        return true;
      };
      const bool far = __any_sync(~0u, sh->far[lane % 8]);
      if (!(far ? work(std::true_type()) : work(std::false_type()))) goto done;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh->spent));
    }
  done:;
  } else if (warp == 8) {
    int n = 0;
    for (int c = 0; c < chunks; ++c) {
      const int count = seen(c);
      for (int t = 0; t < count; ++t, ++n) {
        const int ks = n % kWtStages, j = tile_at(t) * kTile + 4 * lane;
        int page = -1;
        uint32_t off = 0;
        if (j < len) {
          const uint32_t block = block_of(a, j);
          off = j - block * a.bs;
          page = page_of(a, r, block);
        }
        const uint32_t sb = page < 0 ? 0u : (uint32_t)page * a.H + h;
        const int row = (int)(sb * a.bs + off);
        const float kscale = page >= 0 ? __ldg(a.ks + sb) : 0.f;
        const unsigned mask = __ballot_sync(~0u, page >= 0);
        const int step = p.box / 4, boxes = kTile / p.box;
        const int from = __shfl_sync(~0u, row, lane < boxes ? lane * step : 0);
        const bool there = lane < boxes && (mask >> (lane * step) & 1);
        const uint32_t bytes = __popc(__ballot_sync(~0u, there)) * (uint32_t)p.box * kD;
        if (!W.warp_wait(&sh->k_empty[ks], (n / kWtStages & 1) ^ 1)) goto ld_done;
        sh->ks[ks][lane] = kscale;
        if (lane == 0) {
          sh->mask[ks] = mask;
          mbar_expect_tx(smem_addr(&sh->k_full[ks]), bytes);
        }
        __syncwarp();
        if (there)
          tma_load_2d(smem_addr(kbuf + ks * kTileBytes + lane * p.box * kD), &map_k, 0, from, smem_addr(&sh->k_full[ks]));
        if (lane != 0) mbar_arrive(smem_addr(&sh->k_full[ks]));
      }
    }
  ld_done:
    __syncwarp();
    if (lane == 0)
      for (int x = n > kWtStages ? n - kWtStages : 0; x < n; ++x) drain_wait(&sh->k_full[x % kWtStages], x / kWtStages & 1);
  } else {
    const uint64_t q0 = sw128_desc(smem_addr(qbuf)), k0 = sw128_desc(smem_addr(kbuf));
    bool ok = true, issued = false;
    int n = 0;
    for (int c = 0; ok && c < chunks; ++c) {
      ok = W.warp_wait(&sh->q_full, c & 1);
      const int count = seen(c);
      for (int t = 0; ok && t < count; ++t, ++n) {
        const int ks = n % kWtStages, i = n & 1;
        ok = W.warp_wait(&sh->k_full[ks], n / kWtStages & 1) && W.warp_wait(&sh->s_empty[i], (n >> 1 & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = k0 + (uint64_t)(ks * kTileBytes >> 4);
        mma_kq(tmem + i * 2 * kTile, k, q0);
        mma_kq(tmem + i * 2 * kTile + kTile, k, q0 + (2 * kTileBytes >> 4));
        issued = true;
        commit(&sh->s_full[i]);
        commit(&sh->k_empty[ks]);
      }
    }
    if (issued) {
      commit(&sh->drain);
      if (lane == 0) drain_wait(&sh->drain, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The same from the scores of few columns, [score_ld][slot_rows].  Bound by the
// chain of its loads: a thread has four slots' on their way at once (16 requests of up
// to 16,384 slots, 8 heads: 12 us; two slots 2 more, one 4).
constexpr int kSlotsOfThread = 4;
__global__ void __launch_bounds__(256) weights_of_columns_kernel(const __grid_constant__ TcParams p) {
  const AttendParams &a = p.a;
  __shared__ float2 lse2[16];
  const int r = blockIdx.z, h = blockIdx.y, len = len_of(a, r);
  const int64_t beg = a.req.begin(r), j0 = (int64_t)blockIdx.x * (256 * kSlotsOfThread) + threadIdx.x;
  const bool good = requests_ok(a);
  const int rows = good ? (int)(a.req.begin(r + 1) - beg) * a.G : 0;
  float *to = a.weights + ((int64_t)r * a.H + h) * a.wstride + j0;
  float before[kSlotsOfThread], sum[kSlotsOfThread] = {};
#pragma unroll
  for (int k = 0; k < kSlotsOfThread; ++k) before[k] = j0 + 256 * k < len ? to[256 * k] : 0.f;
  wait_for_kernel_before();
  if ((int64_t)blockIdx.x * (256 * kSlotsOfThread) >= len || rows == 0) return;
  if (threadIdx.x < rows)
    lse2[threadIdx.x] = a.stats[(beg + threadIdx.x / a.G) * a.Hq + h * a.G + threadIdx.x % a.G];
  const float *x = p.scores + (((int64_t)r * a.H + h) * p.score_ld + j0) * p.slot_rows;
  __syncthreads();
#pragma unroll 1
  for (int c = 0; c < rows; c += 8) {
    float4 y[kSlotsOfThread][2];
#pragma unroll
    for (int k = 0; k < kSlotsOfThread; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (j0 + 256 * k < len) y[k][e] = __ldcs(reinterpret_cast<const float4 *>(x + 256 * k * p.slot_rows + c) + e);
#pragma unroll
    for (int k = 0; k < kSlotsOfThread; ++k) {
      if (j0 + 256 * k >= len) continue;
      const float z[8] = {y[k][0].x, y[k][0].y, y[k][0].z, y[k][0].w, y[k][1].x, y[k][1].y, y[k][1].z, y[k][1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < rows && z[e] > -INFINITY) sum[k] += probability(z[e], lse2[c + e]);
    }
  }
#pragma unroll
  for (int k = 0; k < kSlotsOfThread; ++k)
    if (j0 + 256 * k < len) to[256 * k] = before[k] + sum[k];
}

// --- host ------------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct TcShape {
  int slot_rows, part_size, grid, score_ld, box;
  bool wide, columns, spool;
  size_t splits, partial, stats, scores, bytes;
};
TcShape tc_shape(const kvx_attend8_args *a) {
  TcShape s;
  const int64_t G = a->q_heads / a->cache.heads, most = G * most_new(a);
  // 16 requests of 1024 to 16,384 slots, 8 KV heads, without and with weights.  16 rows:
  // columns 94 and 119 us, narrow 146 and 189.  24 rows: narrow 147 and 202, wide 151 and
  // 298; 64 rows: 167 and 274 against 159 and 308; 128 rows: 216 and 432 against 160 and
  // 309.
  s.columns = most <= 16;
  s.wide = most > 64;
  s.slot_rows = s.wide ? Wide::ROWS : s.columns ? (most <= 8 ? 8 : 16) : (int)most;
  s.part_size = (s.slot_rows * (kD + 3) + 3) / 4 * 4;
  s.grid = 152;                        // one CTA an SM
  s.score_ld = (a->max_len + 255) / 256 * 256;
  s.box = a->cache.block_size & -a->cache.block_size;
  if (s.box > kTile) s.box = kTile;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s.splits = kWorkspaceHead;
  s.partial = s.splits + up(s.grid * sizeof(Split));
  s.stats = s.partial + up((size_t)2 * s.grid * (s.wide ? 1 : 2) * s.part_size * 4);
  s.scores = s.stats + up((size_t)a->ntok * a->q_heads * sizeof(float2));
  // scores for the weights are kept where the workspace has room for them; room is made
  // for those of smaller calls too (a wide call keeps none, 64 rows of a narrow one most)
  const uint64_t kept = score_bytes(a, s.slot_rows, s.score_ld);
  s.spool = a->weights && !s.wide && kept <= kMostScores && a->workspace_bytes >= s.scores + kept;
  const uint64_t most_kept = s.wide ? score_bytes(a, 64, s.score_ld) : kept;
  s.bytes = s.scores + (a->weights ? up(most_kept < kMostScores ? most_kept : kMostScores) : 0);
  return s;
}

bool encode(CUtensorMap *map, const kvx_cache8 &c, const void *base, int box) {
  static const EncodeFn fn = reinterpret_cast<EncodeFn>(kvx_tc_encoder());
  if (!fn) return false;
  // fewer dimensions are filled with zeros
  const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.num_blocks * c.heads * c.block_size};
  const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim};
  const cuuint32_t boxes[2] = {(cuuint32_t)kD, (cuuint32_t)box}, one[2] = {1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, boxes, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class G, class K>
kvx_status launch(K kernel, int threads, size_t smem, const TcParams &p, const CUtensorMap &mk, const CUtensorMap &mv,
                  cudaStream_t s) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return KVX_ERR_CUDA;
  kernel<<<p.grid, threads, smem, s>>>(p, mk, mv);
  if (const kvx_status st = launched()) return st;
  if constexpr (G::ROWS <= 16) return launch_after(join_row_kernel<G>, dim3(p.grid - 1, p.slot_rows), 256, 0, s, p);
  return launch_after(join_kernel<G>, dim3(p.grid - 1, (p.slot_rows + 31) / 32), 256, 0, s, p);
}

}  // namespace

bool kvx_attend8_tc_supports(const kvx_attend8_args *a) {
  const kvx_cache8 &c = a->cache;
  return a->dtype == KVX_BF16 && c.head_dim <= kD && c.block_size % 8 == 0 &&
         (uint64_t)c.num_blocks * c.heads * c.block_size <= INT32_MAX;
}

size_t kvx_attend8_tc_least_bytes(const kvx_attend8_args *a) { return tc_shape(a).scores; }
size_t kvx_attend8_tc_workspace_bytes(const kvx_attend8_args *a) { return tc_shape(a).bytes; }

kvx_status kvx_attend8_tc_launch(const kvx_attend8_args *args, const kvx8::AttendParams &a, char *ws, cudaStream_t s) {
  const TcShape sh = tc_shape(args);
  CUtensorMap mk, mv;
  if (!encode(&mk, args->cache, a.k, sh.box) || !encode(&mv, args->cache, a.v, sh.box)) return KVX_ERR_CUDA;
  TcParams p;
  p.a = a;
  p.a.stats = a.weights ? (float2 *)(ws + sh.stats) : nullptr;
  p.grid = sh.grid;
  p.splits = (Split *)(ws + sh.splits);
  p.partial = (float *)(ws + sh.partial);
  p.scores = sh.spool ? (float *)(ws + sh.scores) : nullptr;
  p.score_ld = sh.score_ld;
  p.slot_rows = sh.slot_rows;
  p.part_size = sh.part_size;
  p.box = sh.box;
  p.vec_q = aligned_to(a.q, 16) && (a.qt | a.qh) % 8 == 0;
  p.vec_out = aligned_to(a.out, 16) && (a.ot | a.oh) % 8 == 0;
  const kvx_status st =
      sh.wide      ? launch<Wide>(attend_tc_kernel<true>, kThreads, smem_bytes<true>(), p, mk, mv, s)
      : !sh.columns ? launch<Narrow>(attend_tc_kernel<false>, kThreads, smem_bytes<false>(), p, mk, mv, s)
      : sh.slot_rows == 8 ? launch<Columns<8>>(columns_kernel<8>, kColThreads, kColSmem, p, mk, mv, s)
                          : launch<Columns<16>>(columns_kernel<16>, kColThreads, kColSmem, p, mk, mv, s);
  if (st != KVX_OK || !a.weights || a.max_len == 0) return st;
  if (!sh.spool) {
    // as few slot tiles a CTA as lets all run at once, within what it has room for
    const int tiles = (args->max_len + kTile - 1) / kTile, items = a.H * a.req.R;
    int per = 1;
    while (per < kWtTiles && (int64_t)items * ((tiles + per - 1) / per) > 152) ++per;
    if (cudaFuncSetAttribute(weights_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWtSmem) != cudaSuccess)
      return KVX_ERR_CUDA;
    return launch_after(weights_tc_kernel, dim3((tiles + per - 1) / per, a.H, a.req.R), kWtThreads, kWtSmem, s, p, mk, per);
  }
  const auto grid = [&](int slots) { return dim3((a.max_len + slots - 1) / slots, a.H, a.req.R); };
  if (sh.columns) return launch_after(weights_of_columns_kernel, grid(256 * kSlotsOfThread), 256, 0, s, p);
  return launch_after(weights_of_rows_kernel, grid(256), 256, sh.slot_rows * sizeof(float2), s, p);
}
