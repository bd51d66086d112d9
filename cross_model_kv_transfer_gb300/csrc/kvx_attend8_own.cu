// kvx_attend8_own.cu -- the second pass of kvx_attend8_shared where a request has few rows
// and few slots of its own: samples and beams that have been decoded for a while.
//
//   out = a out_before + b sum_j exp(x_j - m) v_j / sum_j exp(x_j - m)
// with a and b from the two parts' log-sum-exps (join_before).
//
// There are many such items, a (request, KV head) each, of a few tiles of slots: what the
// forms for long caches spend on an item (shares of the work, a pipeline filled and
// drained, parts joined by another kernel) is more than the item.  So here a CTA of four
// warps takes one item whole, several CTAs share an SM and hide each other's loads, and the
// result is joined with the prefix's where it is formed.  A warp takes tiles of 16 MT slots
// in turn, two on their way; the products and roundings are those of the split form
// (kvx_attend8.cu).
#include "kvx_attend8_mma.cuh"

namespace {

template <class C>
constexpr size_t own_smem() {
  return C::kRing + (C::kQInSmem ? C::kQ : 0) + (C::COLS * (2 * C::WARPS + 4)) * 4;
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
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
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

template <class C>
__global__ void __launch_bounds__(32 * C::WARPS) own_kernel(const __grid_constant__ SplitParams p) {
  constexpr int DP = C::DP, NT = C::NT, KW = C::KW, CH = C::CH, W = C::WARPS, COLS = C::COLS;
  extern __shared__ __align__(128) unsigned char smem[];
  const AttendParams &a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  unsigned char *ring = smem + warp * 2 * C::kStage;
  uint2 *qs = reinterpret_cast<uint2 *>(smem + C::kRing);
  float *warp_m = reinterpret_cast<float *>(smem + C::kRing + (C::kQInSmem ? C::kQ : 0)), *warp_l = warp_m + W * COLS;
  float *own_of = warp_l + W * COLS, *before_of = own_of + COLS, *col_scale = before_of + COLS;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, col0 = blockIdx.y * COLS;
  if (!requests_ok(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) raise(a.status, KVX_FLAG_BAD_SEQLENS);
    return;
  }
  const int len = len_of(a, r);
  if (h == 0 && col0 == 0 && tid == 0 && len != __ldg(a.lens + r)) raise(a.status, KVX_FLAG_BAD_LENGTH);
  const int64_t beg = a.req.begin(r);
  const int fresh = (int)(a.req.begin(r + 1) - beg), cols = fresh * a.G;
  if (col0 >= cols) return;
  const int tiles = (len + KW - 1) / KW;

  // a tile's codes into one of the warp's two stages: lane l looks up slot l
  const auto fetch = [&](int tile, int stage) {
    unsigned char *st = ring + stage * C::kStage;
    if (tile < tiles) {
      const int j = tile * KW + lane % KW;
      int page = -1;
      uint32_t off = 0;
      if (j < len) {
        const uint32_t block = block_of(a, j);
        off = j - block * a.bs;
        page = page_of(a, r, block);
        if (page < 0) raise(a.status, KVX_FLAG_BAD_BLOCK);
      }
      const unsigned valid = __ballot_sync(~0u, page >= 0);
      const uint32_t block = page < 0 ? 0u : (uint32_t)page * a.H + h;
      const uint32_t row = page < 0 ? 0u : block * a.bs + off;
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
      // scales by plain loads, which are waited for with the codes' lookups
      if (lane < KW) {
        reinterpret_cast<float *>(st + 2 * C::kTile)[lane] = page >= 0 ? __ldg(a.ks + block) : 0.f;
        reinterpret_cast<float *>(st + 2 * C::kTile)[KW + lane] = page >= 0 ? __ldg(a.vs + block) : 0.f;
      }
      if (lane == 0) *reinterpret_cast<unsigned *>(st + 2 * C::kTile + 2 * KW * 4) = valid;
    }
    cp_async_commit();
  };
  fetch(warp, 0);
  fetch(warp + W, 1);
  const int first = first_limit(a, len, fresh), limits = cols - col0 < COLS ? -1 : first + col0 / a.G;
  int limit[NT][2];          // last slot that the thread's columns see
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = col0 + 8 * n + 2 * t + e;
      limit[n][e] = col < cols ? first + col / a.G : -1;
    }
  Queries<C> qf;
  qf.load(p, beg, h, col0, cols, qs, col_scale);
  Sums<C> x;
  x.clear();
  int stage = 0;
  for (int tile = warp; tile < tiles; tile += W) {
    cp_async_wait<1>();
    __syncwarp();
    x.add(ring + stage * C::kStage, tile * KW, qf, qs, limit, limits);
    __syncwarp();
    fetch(tile + 2 * W, stage);
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
  wait_for_kernel_before();
  __syncthreads();             // and the ring is free
  if (tid < COLS && col0 + tid < cols) {
    const int col = col0 + tid;
    float mm = -INFINITY, l = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) mm = fmaxf(mm, warp_m[v * COLS + tid]);
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float f = ex2(warp_m[v * COLS + tid] - finite_or_0(mm));
      l += f * warp_l[v * COLS + tid];
      warp_m[v * COLS + tid] = f;      // from here on the warps' factors
    }
    const int64_t tok = beg + col / a.G;
    const int hq = h * a.G + col % a.G;
    const Joined j = join_before(a, tok, hq, mm, kRoom, l);
    own_of[tid] = l != 0.f ? j.own / l : 0.f;
    before_of[tid] = j.before;
    if (a.lse) a.lse[tok * a.Hq + hq] = j.lse.y == INFINITY ? -INFINITY : (j.lse.x + j.lse.y) * kLn2;
  }
  float *red = reinterpret_cast<float *>(smem);
  constexpr int ROWF = DP + 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n > 0) __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float *row = red + (warp * 8 + 2 * t + e) * ROWF;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        *reinterpret_cast<float2 *>(row + 16 * c + 2 * g) = make_float2(x.o[n][c][e] * kUnit * x.vref, x.o[n][c][2 + e] * kUnit * x.vref);
    }
    __syncthreads();
    for (int i = tid; i < 8 * (DP / 4); i += 32 * W) {
      const int in = i / (DP / 4), d = i % (DP / 4) * 4, c = 8 * n + in, col = col0 + c;
      if (col >= cols || d >= a.d) continue;
      const int64_t tok = beg + col / a.G;
      const int hq = h * a.G + col % a.G;
      const float4 b = __ldcg(reinterpret_cast<const float4 *>(a.before + (tok * a.Hq + hq) * a.d + d));
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < W; ++v) {
        const float f = warp_m[v * COLS + c];
        const float4 z = *reinterpret_cast<const float4 *>(red + (v * 8 + in) * ROWF + d);
        y = make_float4(fmaf(f, z.x, y.x), fmaf(f, z.y, y.y), fmaf(f, z.z, y.z), fmaf(f, z.w, y.w));
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

template <int DP, int NT, int PARTS>
kvx_status launch_own(const SplitParams &p, int groups, cudaStream_t s) {
  using C = SplitCfg<DP, NT, PARTS, (DP <= 128 && NT * PARTS <= 2 ? 2 : 1), 4, 2>;
  static_assert(C::kStage % 16 == 0 && 4 * 8 * (DP + 4) * 4 <= C::kRing, "shared memory");
  constexpr int smem = (int)own_smem<C>();
  if (cudaFuncSetAttribute(own_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return KVX_ERR_CUDA;
  return launch_after(own_kernel<C>, dim3((unsigned)(p.a.req.R * p.a.H), (unsigned)groups), 128, smem, s, p);
}
template <int PARTS>
kvx_status launch_dim(const SplitParams &p, int most, cudaStream_t s) {
  // columns of a CTA: registers hold 4096 sums a warp
  const int cols = most <= 8 ? 8 : most <= 16 || p.a.d > 128 ? 16 : 32, groups = (most + cols - 1) / cols;
  if (p.a.d > 128) return cols == 8 ? launch_own<256, 1, PARTS>(p, groups, s) : launch_own<256, 2, PARTS>(p, groups, s);
  if (p.a.d > 64)
    return cols == 8    ? launch_own<128, 1, PARTS>(p, groups, s)
           : cols == 16 ? launch_own<128, 2, PARTS>(p, groups, s)
                        : launch_own<128, 4, PARTS>(p, groups, s);
  return cols == 8    ? launch_own<64, 1, PARTS>(p, groups, s)
         : cols == 16 ? launch_own<64, 2, PARTS>(p, groups, s)
                      : launch_own<64, 4, PARTS>(p, groups, s);
}

}  // namespace

bool kvx_attend8_own_supports(const kvx_attend8_args *a) {
  const int64_t most = (int64_t)(a->q_heads / a->cache.heads) * most_new(a);
  return most <= 64 && a->max_len <= 2048 && (int64_t)a->num_requests * a->cache.heads <= INT32_MAX;
}

kvx_status kvx_attend8_own_launch(const kvx_attend8_args *a, const kvx8::AttendParams &params, cudaStream_t s) {
  SplitParams p = {};
  p.a = params;
  const int size = a->dtype == KVX_BF16 ? 2 : 4, most = params.G * params.max_new;
  p.vec_q = aligned_to(a->q, 16) && ((params.qt | params.qh) * size) % 16 == 0;
  p.vec_out = aligned_to(a->out, 4 * size) && (params.ot | params.oh) % 4 == 0;
  return size == 2 ? launch_dim<1>(p, most, s) : launch_dim<2>(p, most, s);
}
