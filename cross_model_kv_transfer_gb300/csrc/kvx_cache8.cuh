// kvx_cache8.cuh -- the 8-bit paged cache as the kernels see it (kvx_cache8.cu,
// kvx_attend8*.cu, kvx_pages.cu, kvx_evict8.cu): e4m3 conversions, power-of-two scales, block
// lookup, request tables and the host's checks of a kvx_cache8.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvx_internal.h"

namespace kvx8 {

// Requests of a packed batch: cu[0 .. R] (or one token each without it).
struct Requests {
  const int32_t *cu;
  int R;
  int64_t ntok;
  __device__ int64_t begin(int r) const { return cu ? (int64_t)cu[r] : r; }
  // Starts at 0, never decreases, ends at ntok; every thread of the CTA calls it.
  __device__ bool ok() const {
    bool good = true;
    if (cu) {
      for (int r = threadIdx.x; r < R; r += blockDim.x) good = good && cu[r + 1] >= cu[r];
      if (threadIdx.x == 0) good = good && cu[0] == 0 && (int64_t)cu[R] == ntok;
      good = __syncthreads_and(good);
    }
    return good;
  }
};

}  // namespace kvx8

namespace {

using kvx8::Requests;

// Two fp32 to two e4m3 codes, nearest even, clamped to +-448 (low byte = lo).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (the low half of `codes`) to f16x2, exact.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t codes) {
  const uint32_t h = f16x2_of(codes);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The smallest power of two, at least 2^-126, with amax <= 448 * scale
// (448 = 1.75 * 2^8; amax finite and not negative).  From amax's bits: its
// exponent less 8, one more where its significand is above 1.75.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ void raise(uint32_t *status, uint32_t bits) {
  if (status) atomicOr(status, bits);
}

inline bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// Do arrays of 32-bit words (or elements of another size) share memory?
inline bool overlap(const void *a, int64_t a_words, const void *b, int64_t b_words, int size = 4) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a_words > 0 && b_words > 0 && x < y + size * (uintptr_t)b_words && y < x + size * (uintptr_t)a_words;
}

// The kernel is launched while the one before on its stream still runs: what that
// one writes may be read after this.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may start once all CTAs have come here; it calls the above.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Host checks of a cache.
inline kvx_status check_cache8(const kvx_cache8 &c) {
  if (!c.k_codes || !c.v_codes || !c.k_scale || !c.v_scale || !c.block_table)
    return KVX_ERR_INVALID_ARG;
  if (c.num_blocks < 1 || c.num_blocks > INT32_MAX || c.heads < 1 || c.heads > 65535 ||
      c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16 || c.block_size < 1 ||
      c.block_size > 1024 || c.max_blocks_per_req < 1)
    return KVX_ERR_INVALID_ARG;
  // rows are counted in 32 bits
  if ((uint64_t)c.num_blocks * c.heads > UINT32_MAX / (uint64_t)c.block_size) return KVX_ERR_UNSUPPORTED;
  if (!aligned_to(c.k_codes, 16) || !aligned_to(c.v_codes, 16) || !aligned_to(c.k_scale, 4) ||
      !aligned_to(c.v_scale, 4) || !aligned_to(c.block_table, 4))
    return KVX_ERR_INVALID_ARG;
  return KVX_OK;
}

// Launch beside the end of the kernel before (which the kernel waits for itself).
template <class... P, class... A>
kvx_status launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? KVX_OK : KVX_ERR_CUDA;
}

inline kvx_status launched() { return cudaGetLastError() == cudaSuccess ? KVX_OK : KVX_ERR_CUDA; }

}  // namespace
