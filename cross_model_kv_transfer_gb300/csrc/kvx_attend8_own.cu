// kvx_attend8_own.cu -- kvx_attend8_shared where a request has few rows and few slots of
// its own: samples and beams that have been decoded for a while.
//
//   out = a out_before + b sum_j exp(x_j - m) v_j / sum_j exp(x_j - m)
// with a and b from the two parts' log-sum-exps.
//
// There are many such items, a (request, KV head) each, of a few tiles of slots: what the
// forms for long caches spend on an item (shares of the work, a pipeline filled and
// drained, parts joined by another kernel) is more than the item.  So here a CTA of four
// warps takes one item whole, several CTAs share an SM and hide each other's loads, and the
// result is joined with the prefix's where it is formed.  A warp takes tiles of 16 MT slots
// in turn, two on their way; the products and roundings are those of the split form
// (kvx_attend8_split.cu).
//
// The prefixes themselves go the same way while their products are few: a CTA for each
// prefix, KV head, group of eight columns and split of the slots leaves its maxima, totals and
// sums, and the items join all splits' with their own.  Two launches then, and no
// kernel that joins.  So a prefix is read (from L2, mostly) once for every eight columns of its
// group, which with eight heads to a KV head and one token is once for each request.
#define KVX_ATTEND_SHARED 1
#include "kvx_attend8_mma.cuh"

namespace {

constexpr int kMostParts = 32;      // splits of a prefix
// Multiplications of the scores up to which the prefixes go in parts.  bf16: 2.6e8 take 27 to
// 37 us, 27 to 47 otherwise, 5.2e8 37 to 43 and 41 to 44.  fp32, which counts twice: 5.4e8
// take 33 us, 66 otherwise, 8.4e9 251 and 202.
constexpr double kMostWork = 5e8, kMostWorkF32 = 2e9;

// What the splits leave: [part][token][Hq][d] sums, [part][token][Hq] maxima and totals,
// relative to exp2(maximum + kRoom).
struct Parts {
  float *sums;
  float2 *tops;
  int64_t rows;
  int count;
};
struct OwnParams {
  SplitParams s;
  Parts parts;               // count 0: `before` is one result
};

template <class C>
constexpr size_t own_smem() {
  return C::kRing + (C::kQInSmem ? C::kQ : 0) + (C::COLS * (2 * C::WARPS + 3 + 2 * kMostParts)) * 4;
}

// What a warp has of its columns.
template <class C>
struct Sums {
  static constexpr int NT = C::NT, MT = C::MT, CH = C::CH, PARTS = C::PARTS, DP = C::DP;
  float mx[NT][2], m[NT][2], l[NT][2], o[NT][CH][4];   // maxima as scores without their column's factor, and with it
  float vref, vinv;            // largest value scale, and 2^14 over it
  bool far;
  __device__ __forceinline__ void clear() {
    vref = 0x1p-112f;          // a scale below is treated as that: 2^14 over it stays finite
    vinv = 0x1p126f;
    far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[n][e] = m[n][e] = -INFINITY;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][c][e] = 0.f;
    }
  }
  // A tile of 16 MT slots from j0 on, whose codes and scales lie at st.
  __device__ __forceinline__ void add(const unsigned char *st, int j0, const Queries<C> &qf, const uint2 *qs, const int (&limit)[NT][2],
                                      int limits) {
    const int lane = threadIdx.x % 32, g = lane / 4;
    const uint32_t vaddr = (uint32_t)__cvta_generic_to_shared(st + C::kTile);
    const float *ks = reinterpret_cast<const float *>(st + 2 * C::kTile), *vs = ks + C::KW;
    const unsigned valid = *reinterpret_cast<const unsigned *>(st + 2 * C::kTile + 2 * C::KW * 4);
    if (!valid) return;
    float s[MT][NT][4];
    qf.scores(st, qs, s);
    float vsc[MT][2], most = 0.f;
    bool grew = false;
    const bool masked = valid != ~0u || j0 + C::KW - 1 > limits;
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
    if (__any_sync(~0u, grew || most > vref)) {
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
          const float mm = finite_or_0(__fmul_rn(top[n][e], qf.cs[n][e])), down = ex2(m[n][e] - mm);
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
    // far scores are rounded before the maximum, which is one of them, is subtracted
    if (__any_sync(~0u, far)) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = __fmul_rn(s[i][n][e], qf.cs[n][e & 1]) - finite_or_0(m[n][e & 1]);
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = fmaf(s[i][n][e], qf.cs[n][e & 1], -finite_or_0(m[n][e & 1]));
    }
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
    // rows g and g + 8 of a 16-dimension piece are its dimensions 2g and 2g + 1
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
            for (int part = 0; part < PARTS; ++part) mma16816(o[n][c + k], f, pb[i][n][part][0], pb[i][n][part][1]);
        }
      }
  }
};

// PART: of a prefix's slots, CTAs (prefix and KV head, group of columns, split).  Else: of a
// request's own, CTAs (request and KV head, group of columns).
template <class C, bool PART>
__global__ void __launch_bounds__(32 * C::WARPS, C::DP <= 128 ? 3 : 1) own_kernel(const __grid_constant__ OwnParams op) {
  constexpr int DP = C::DP, NT = C::NT, KW = C::KW, CH = C::CH, W = C::WARPS, COLS = C::COLS;
  extern __shared__ __align__(128) unsigned char smem[];
  const SplitParams &p = op.s;
  const AttendParams &a = p.a;
  const Parts &parts = op.parts;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  unsigned char *ring = smem + warp * 2 * C::kStage;
  uint2 *qs = reinterpret_cast<uint2 *>(smem + C::kRing);
  float *warp_m = reinterpret_cast<float *>(smem + C::kRing + (C::kQInSmem ? C::kQ : 0)), *warp_l = warp_m + W * COLS;
  float *own_of = warp_l + W * COLS, *before_of = own_of + COLS, *col_scale = before_of + COLS, *part_of = col_scale + COLS,
        *part_total = part_of + kMostParts * COLS;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, col0 = blockIdx.y * COLS;
  if (PART) {
    // the items may start beside this: what they read before they wait was there before
    wait_for_kernel_before();
    let_next_kernel_start();
  }
  // What all else waits for is asked for at once: blocks are looked up before the length is
  // known, and the whole request table is looked through while the first tiles are on their
  // way.  Nothing is written before the barrier that tells whether it is good; until then
  // the CTA's own request has to lie within bounds.
  const auto look = [&](int tile) { return tile >= 0 ? page_of(a, r, block_of(a, tile * KW + lane % KW)) : -1; };
  int page0 = -1, page1 = -1, page2 = -1;
  if (!PART) {
    page0 = look(warp);
    page1 = look(warp + W);
    page2 = look(warp + 2 * W);
  }
  const int len = len_of(a, r);
  const int64_t beg = begin_of(a, r), end = begin_of(a, r + 1);
  const int all = (len + KW - 1) / KW;
  // the CTA's tiles
  const int begin = PART ? (int)((int64_t)all * blockIdx.z / parts.count) : 0;
  const int tiles = PART ? (int)((int64_t)all * (blockIdx.z + 1) / parts.count) : all;
  if (PART) {
    page0 = look(begin + warp);
    page1 = look(begin + warp + W);
    page2 = look(begin + warp + 2 * W);
  }
  const bool inside = beg >= 0 && end >= beg && end <= a.req.ntok && end - beg <= a.max_new;
  const int fresh = inside ? (int)(end - beg) : 0, cols = fresh * a.G;
  const auto table_ok = [&]() {
    bool good = true;
    for (int i = tid; i < a.req.R; i += 32 * W) {
      const int64_t from = begin_of(a, i), to = begin_of(a, i + 1);
      good = good && to >= from && to - from <= a.max_new && (i > 0 || from == 0) && (i + 1 < a.req.R || to == a.req.ntok);
    }
    return good && groups_ok(a, tid, 32 * W);
  };
  // What follows this kernel on its stream waits for this kernel alone, which may start beside
  // the one before it.  So the first CTA never leaves before that one has ended, whatever the
  // tables hold: else no CTA might, and the next call would write where its parts still go.
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
  if (first_cta && !__syncthreads_and(table_ok())) {
    if (!PART) wait_for_kernel_before();
    if (tid == 0) raise(a.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  if (h == 0 && col0 == 0 && blockIdx.z == 0 && tid == 0 && len != __ldg(a.lens + r)) raise(a.status, KVX_FLAG_BAD_LENGTH);
  if (col0 >= cols) {
    if (!PART && first_cta) wait_for_kernel_before();
    return;
  }

  // A tile goes through three steps, so that nothing waits for one before it: its blocks are
  // looked up (lane l slot l), a turn later its codes and scales are asked for, and the
  // scales come to shared memory before it is used.
  float kscale = 0.f, vscale = 0.f;
  const auto fetch = [&](int tile, int page, int stage) {
    unsigned char *st = ring + stage * C::kStage;
    if (tile < tiles) {
      const int j = tile * KW + lane % KW;
      if (j >= len) page = -1;
      else if (page < 0) raise(a.status, KVX_FLAG_BAD_BLOCK);
      const unsigned valid = __ballot_sync(~0u, page >= 0);
      const uint32_t block = page < 0 ? 0u : (uint32_t)page * a.H + h;
      const uint32_t row = page < 0 ? 0u : block * a.bs + (j - block_of(a, j) * a.bs);
      kscale = page >= 0 ? __ldg(a.ks + block) : 0.f;
      vscale = page >= 0 ? __ldg(a.vs + block) : 0.f;
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < KW * CH / 32; ++i) {
        const int j = i * (32 / CH) + lane / CH;
        const uint32_t from = __shfl_sync(~0u, row, j);
        const bool there = c * 16 < a.d && (valid >> j & 1);
        const uint64_t at = there ? (uint64_t)from * a.d + c * 16 : 0;
        cp_async16(st + piece_at<DP>(j, c), a.k + at, there ? 16 : 0);
        cp_async16(st + C::kTile + piece_at<DP>(j, c), a.v + at, there ? 16 : 0);
      }
      if (lane == 0) *reinterpret_cast<unsigned *>(st + 2 * C::kTile + 2 * KW * 4) = valid;
    }
    cp_async_commit();
  };
  const auto put_scales = [&](int stage, float k, float v) {
    float *to = reinterpret_cast<float *>(ring + stage * C::kStage + 2 * C::kTile);
    if (lane < KW) {
      to[lane] = k;
      to[KW + lane] = v;
    }
  };
  fetch(begin + warp, page0, 0);
  float k_now = kscale, v_now = vscale;
  fetch(begin + warp + W, page1, 1);
  const int first = first_limit(a, len, fresh), more = limit_step(a);
  const int limits = cols - col0 < COLS ? -1 : first + col0 / a.G * more;
  int limit[NT][2];          // last slot that the thread's columns see
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = col0 + 8 * n + 2 * t + e;
      limit[n][e] = col < cols ? first + col / a.G * more : -1;
    }
  Queries<C> qf;
  qf.load(p, beg, h, col0, cols, qs, col_scale);
  const bool good = table_ok();
  Sums<C> x;
  x.clear();
  int stage = 0;
  for (int tile = begin + warp; tile < tiles; tile += W) {
    const int page3 = look(tile + 3 * W);
    put_scales(stage, k_now, v_now);
    k_now = kscale;
    v_now = vscale;
    cp_async_wait<1>();
    __syncwarp();
    x.add(ring + stage * C::kStage, tile * KW, qf, qs, limit, limits);
    __syncwarp();
    fetch(tile + 2 * W, page2, stage);
    page2 = page3;
    stage ^= 1;
  }
  cp_async_wait<0>();

  // the warps' columns joined, and with what came before
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x.l[n][e] += __shfl_xor_sync(~0u, x.l[n][e], off);
      if (g == 0) {
        warp_m[warp * COLS + 8 * n + 2 * t + e] = x.m[n][e];
        warp_l[warp * COLS + 8 * n + 2 * t + e] = x.l[n][e] * (kUnit * 16384.f);
      }
    }
  if (!PART) wait_for_kernel_before();
  // one result of the prefix: its rows are on their way before they are needed
  constexpr int kQuads = 8 * (DP / 4) / (32 * W);
  float4 before_row[NT][kQuads];
  if (!PART && !parts.count) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int i = tid + k * 32 * W, d = i % (DP / 4) * 4, col = col0 + 8 * n + i / (DP / 4);
        before_row[n][k] = col < cols && d < a.d ? __ldcg(reinterpret_cast<const float4 *>(
                                                       a.share.before + ((beg + col / a.G) * a.Hq + h * a.G + col % a.G) * a.d + d))
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
      }
  }
  if (!__syncthreads_and(good)) return;      // and the ring is free
  float *red = reinterpret_cast<float *>(smem);
  constexpr int ROWF = DP + 4;
  const auto put_sums = [&](int n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float *row = red + (warp * 8 + 2 * t + e) * ROWF;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        *reinterpret_cast<float2 *>(row + 16 * c + 2 * g) = make_float2(x.o[n][c][e] * kUnit * x.vref, x.o[n][c][2 + e] * kUnit * x.vref);
    }
  };
  put_sums(0);
  if (!PART && parts.count) {
    for (int i = tid; i < parts.count * COLS; i += 32 * W) {
      const int q = i / COLS, col = col0 + i % COLS;
      const float2 y = col < cols ? __ldcg(parts.tops + q * parts.rows + (beg + col / a.G) * a.Hq + h * a.G + col % a.G)
                                  : make_float2(-INFINITY, 0.f);
      part_of[i] = y.x;
      part_total[i] = y.y;
    }
    __syncthreads();
  }
  if (tid < COLS && col0 + tid < cols) {
    const int col = col0 + tid;
    float mm = -INFINITY, l = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) mm = fmaxf(mm, warp_m[v * COLS + tid]);
    if (!PART)
      for (int q = 0; q < parts.count; ++q) mm = fmaxf(mm, part_of[q * COLS + tid]);
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float f = ex2(warp_m[v * COLS + tid] - finite_or_0(mm));
      l += f * warp_l[v * COLS + tid];
      warp_m[v * COLS + tid] = f;      // from here on the warps' factors
    }
    const int64_t tok = beg + col / a.G;
    const int hq = h * a.G + col % a.G;
    if (PART) {
      own_of[tid] = 1.f;
      parts.tops[(int64_t)blockIdx.z * parts.rows + tok * a.Hq + hq] = make_float2(mm, l);
    } else if (parts.count) {
      for (int q = 0; q < parts.count; ++q) {
        const float f = ex2(part_of[q * COLS + tid] - finite_or_0(mm));
        l += f * part_total[q * COLS + tid];
        part_of[q * COLS + tid] = f;
      }
      own_of[tid] = before_of[tid] = l != 0.f ? 1.f / l : 0.f;
      if (a.lse) a.lse[tok * a.Hq + hq] = l != 0.f ? (mm + (kRoom + log2f(l))) * kLn2 : -INFINITY;
    } else {
      const Joined j = join_before(a, tok, hq, mm, kRoom, l);
      own_of[tid] = l != 0.f ? j.own / l : 0.f;
      before_of[tid] = j.before;
      if (a.lse) a.lse[tok * a.Hq + hq] = j.lse.y == INFINITY ? -INFINITY : (j.lse.x + j.lse.y) * kLn2;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n > 0) {
      __syncthreads();
      put_sums(n);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int i = tid + k * 32 * W, in = i / (DP / 4), d = i % (DP / 4) * 4, c = 8 * n + in, col = col0 + c;
      if (col >= cols || d >= a.d) continue;
      const int64_t tok = beg + col / a.G;
      const int hq = h * a.G + col % a.G;
      const int64_t row = tok * a.Hq + hq;
      float4 b = before_row[n][k], y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!PART && parts.count) {
        b = y;
#pragma unroll 16
        for (int q = 0; q < parts.count; ++q) {
          const float f = part_of[q * COLS + c];
          const float4 z = __ldcg(reinterpret_cast<const float4 *>(parts.sums + (q * parts.rows + row) * a.d + d));
          // a split without slots that count left no sums
          if (f != 0.f) b = make_float4(fmaf(f, z.x, b.x), fmaf(f, z.y, b.y), fmaf(f, z.z, b.z), fmaf(f, z.w, b.w));
        }
      }
#pragma unroll
      for (int v = 0; v < W; ++v) {
        const float f = warp_m[v * COLS + c];
        const float4 z = *reinterpret_cast<const float4 *>(red + (v * 8 + in) * ROWF + d);
        y = make_float4(fmaf(f, z.x, y.x), fmaf(f, z.y, y.y), fmaf(f, z.z, y.z), fmaf(f, z.w, y.w));
      }
      if (PART) {
        *reinterpret_cast<float4 *>(parts.sums + ((int64_t)blockIdx.z * parts.rows + row) * a.d + d) = y;
        continue;
      }
      const float own = own_of[c], before = before_of[c];
      y = make_float4(y.x * own + b.x * before, y.y * own + b.y * before, y.z * own + b.z * before, y.w * own + b.w * before);
      const int64_t to = tok * a.ot + hq * a.oh + d;
      if (a.bf16) {
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + to;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
        if (p.vec_out) {
          *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
          out[0] = lo.x;
          out[1] = lo.y;
          out[2] = hi.x;
          out[3] = hi.y;
        }
      } else {
        float *out = reinterpret_cast<float *>(a.out) + to;
        if (p.vec_out) {
          *reinterpret_cast<float4 *>(out) = y;
        } else {
          out[0] = y.x;
          out[1] = y.y;
          out[2] = y.z;
          out[3] = y.w;
        }
      }
    }
  }
}

// Eight columns a CTA: with bf16 queries more of them (two to four tiles) took the same time or
// longer in all of 8 beams, 64 samples and 192 rows of three tokens, as four or eight warps and one
// or two 16-slot tiles did; this takes the fewest registers.  With fp32 queries, whose products
// cost twice, long prefixes in parts of up to 32 columns took less: 8 requests over
// 65,000 slots 152 us (254 with eight columns, 223 in the split form, which they take now), 4 x
// 32 over 8000 316 us (428, 361).  That is not built.
template <int DP, int PARTS>
kvx_status launch_own(const OwnParams &p, int groups, bool part, cudaStream_t s) {
  using C = SplitCfg<DP, 1, PARTS, DP <= 128 ? 2 : 1, 4, 2>;
  static_assert(C::kStage % 16 == 0 && C::WARPS * 8 * (DP + 4) * 4 <= C::kRing, "shared memory");
  constexpr int smem = (int)own_smem<C>();
  const auto kernel = part ? own_kernel<C, true> : own_kernel<C, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return KVX_ERR_CUDA;
  return launch_after(kernel, dim3((unsigned)(p.s.a.req.R * p.s.a.H), (unsigned)groups, part ? (unsigned)p.parts.count : 1u),
                      32 * C::WARPS, smem, s, p);
}
template <int PARTS>
kvx_status launch_dim(const OwnParams &p, int most, bool part, cudaStream_t s) {
  const int groups = (most + 7) / 8;
  return p.s.a.d <= 64    ? launch_own<64, PARTS>(p, groups, part, s)
         : p.s.a.d <= 128 ? launch_own<128, PARTS>(p, groups, part, s)
                          : launch_own<256, PARTS>(p, groups, part, s);
}
int64_t rows_of(const kvx_attend8_args *a) { return (int64_t)(a->q_heads / a->cache.heads) * most_new(a); }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// Bytes of the parts' sums, maxima and totals: at most kPartRoom, or there is one result.
constexpr size_t kPartRoom = (size_t)32 << 20;
size_t bytes_of(int64_t parts, int64_t rows, int64_t d) {
  const double b = (double)parts * rows * (4 * d + 8) + 512;
  return b > 2 * (double)kPartRoom ? 2 * kPartRoom : up256((size_t)(parts * rows * d * 4)) + up256((size_t)(parts * rows * 8));
}

}  // namespace

// Few rows, and few enough slots that a CTA alone with an item is not the longest.  With 2048
// own slots behind a prefix of 20,000 this form takes 33 to 160 us (8 to 512 items, 8 rows;
// the forms for long caches 37 to 180), with 64 rows 36 to 208 (68 to 201), with 4096 slots
// 51 to 226 (38 to 222).
bool kvx_attend8_own_supports(const kvx_attend8_args *a) {
  return rows_of(a) <= 64 && a->max_len <= 2048 && (int64_t)a->num_requests * a->cache.heads <= INT32_MAX;
}

// Splits of the prefixes' slots that let about two CTAs an SM work, each on at least four
// tiles of its warps; 0 where the products are too many for 16 x 8 x 16 instructions.
int kvx_attend8_parts(const kvx_attend8_args *before) {
  const int64_t most = rows_of(before), rows = before->ntok * before->q_heads, d = before->cache.head_dim;
  const double work = (double)rows * before->max_len * (double)d * (before->dtype == KVX_BF16 ? 1 : 2);
  const int64_t groups = (most + 7) / 8, items = (int64_t)before->num_requests * before->cache.heads * groups;
  if (work > (before->dtype == KVX_BF16 ? kMostWork : kMostWorkF32) || groups > 65535 || items > INT32_MAX || before->max_len == 0) return 0;
  const int64_t fill = (2 * 152 + items - 1) / items, tiles = ((int64_t)before->max_len + 255) / 256;
  int64_t parts = fill < tiles ? fill : tiles;
  if (parts > kMostParts) parts = kMostParts;
  return bytes_of(parts, rows, d) <= kPartRoom ? (int)parts : 0;
}
// What calls of at most these sizes leave in parts.
size_t kvx_attend8_parts_bytes(const kvx_attend8_args *before) {
  const size_t most = bytes_of(kMostParts, before->ntok * before->q_heads, before->cache.head_dim);
  return most < kPartRoom ? most : kPartRoom;
}

kvx_status kvx_attend8_own_launch(const kvx_attend8_args *a, const kvx8::AttendParams &params, int parts, void *part_bytes, bool prefixes,
                                  cudaStream_t s) {
  OwnParams p = {};
  p.s.a = params;
  const int size = a->dtype == KVX_BF16 ? 2 : 4, most = params.G * params.max_new;
  p.s.vec_q = aligned_to(a->q, 16) && ((params.qt | params.qh) * size) % 16 == 0;
  p.s.vec_out = aligned_to(a->out, 4 * size) && (params.ot | params.oh) % 4 == 0;
  p.parts.count = parts;
  p.parts.rows = a->ntok * a->q_heads;
  p.parts.sums = (float *)part_bytes;
  p.parts.tops = (float2 *)((char *)part_bytes + up256((size_t)parts * p.parts.rows * params.d * sizeof(float)));
  return size == 2 ? launch_dim<1>(p, most, prefixes, s) : launch_dim<2>(p, most, prefixes, s);
}
