// Helpers of layer norm's and the distillation loss's kernels (train_ops.h).  Not part
// of the public interface.
#pragma once

#include <cfloat>

#include "train_internal.h"

namespace traingb {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d /= 2) x += __shfl_xor_sync(kAll, x, d);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d /= 2) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}

// Sum (largest) over a CTA's threads, the same bits in each.  `part` holds one
// value a warp; a place may be used again when a second call, with another
// place, has been passed.
template <int THREADS>
__device__ __forceinline__ float cta_sum(float x, float* part) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / kWarp; ++w) x += part[w];
  return x;
}
template <int THREADS>
__device__ __forceinline__ float cta_max(float x, float* part) {
  x = warp_max(x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWarp; ++w) x = fmaxf(x, part[w]);
  return x;
}

// The threads that share a row: part of a warp (a power of two), a warp, or several
// warps with a named barrier and, for each of kSlots sums, a place a warp in shared
// memory.  A place may be used again when another sum has been taken in between.
enum class Span { kPart, kWarp, kWarps };
constexpr int kSlots = 5;

struct Group {
  int lanes;
  int lane;     // of this thread
  int barrier;  // kWarps
  float* part;  // kWarps: [kSlots][32 a CTA], at this group's first warp

  template <Span S, class F>
  __device__ __forceinline__ float join(float x, int slot, float none, F&& f) const {
    if constexpr (S == Span::kPart) {
      for (int d = 1; d < lanes; d *= 2) x = f(x, __shfl_xor_sync(kAll, x, d));
      return x;
    }
#pragma unroll
    for (int d = 1; d < traingb::kWarp; d *= 2) x = f(x, __shfl_xor_sync(kAll, x, d));
    if constexpr (S == Span::kWarps) {
      float* p = part + slot * traingb::kWarp;
      if ((lane & 31) == 0) p[lane >> 5] = x;
      asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(lanes) : "memory");
      x = (lane & 31) < lanes / traingb::kWarp ? p[lane & 31] : none;
#pragma unroll
      for (int d = 1; d < traingb::kWarp; d *= 2) x = f(x, __shfl_xor_sync(kAll, x, d));
    }
    return x;
  }
  template <Span S>
  __device__ __forceinline__ float sum(float x, int slot) const {
    return join<S>(x, slot, 0.f, [](float a, float b) { return a + b; });
  }
  // N sums at once (2 or 4), of at most 24 warps.  In the first steps the lanes split
  // the sums up among themselves: 32 / N lanes end with one each.
  template <Span S, int N>
  __device__ __forceinline__ void sums(float (&x)[N], int slot) const {
    static_assert(N == 2 || N == 4, "");
    if constexpr (S == Span::kPart) {
      for (int d = 1; d < lanes; d *= 2)
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(kAll, x[n], d);
      return;
    }
    constexpr int kShare = traingb::kWarp / N;  // lanes a sum
    const bool upper = lane & 16;
    float v = upper ? x[1] : x[0];
    v += __shfl_xor_sync(kAll, upper ? x[0] : x[1], 16);
    if constexpr (N == 4) {
      float w = upper ? x[3] : x[2];
      w += __shfl_xor_sync(kAll, upper ? x[2] : x[3], 16);
      const bool odd = lane & 8;
      const float keep = odd ? w : v;
      v = keep + __shfl_xor_sync(kAll, odd ? v : w, 8);
    }
#pragma unroll
    for (int d = kShare / 2; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    if constexpr (S == Span::kWarps) {
      float* p = part + (slot * N + (lane & 31) / kShare) * traingb::kWarp;
      if ((lane & (kShare - 1)) == 0) p[lane >> 5] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(lanes) : "memory");
      const int warps = lanes / traingb::kWarp, k = lane & (kShare - 1);
      v = k < warps ? p[k] : 0.f;
#pragma unroll
      for (int o = kShare; o < 24; o += kShare)
        if (k + o < warps) v += p[k + o];
#pragma unroll
      for (int d = kShare / 2; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    }
    // Lanes 0 and 16 hold sums 0 and 1; of four, 8 and 24 hold 2 and 3.
    x[0] = __shfl_sync(kAll, v, 0), x[1] = __shfl_sync(kAll, v, 16);
    if constexpr (N == 4) x[2] = __shfl_sync(kAll, v, 8), x[3] = __shfl_sync(kAll, v, 24);
  }
  template <Span S>
  __device__ __forceinline__ float largest(float x, int slot) const {
    return join<S>(x, slot, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
  }
};

__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return uint32_t(__cvta_generic_to_shared(p));
}
// BYTES from global to shared memory, both aligned to them.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  static_assert(BYTES == 8 || BYTES == 16, "");
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
template <int DT, int VEC>
__device__ __forceinline__ void load_shared(Pack<DT, VEC>& p, uint32_t from) {
  constexpr int B = Pack<DT, VEC>::kBytes;
  static_assert(B == 8 || B == 16, "");
  if constexpr (B == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(p.w[0]), "=r"(p.w[1]), "=r"(p.w[2]), "=r"(p.w[3])
                 : "r"(from)
                 : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(p.w[0]), "=r"(p.w[1])
                 : "r"(from)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Whether the squares that gave a variance kept their bits: none left fp32's
// range at the top, and those that did at the bottom are nothing beside eps.
__device__ __forceinline__ bool in_range(float var, float eps) {
  return var <= FLT_MAX && var + eps > 0x1p-80f;
}
// 1 / sqrt(var + eps), by a step of Newton's method on the instruction's result.
__device__ __forceinline__ float rstd_of(float var, float eps) {
  const float v = var + eps, r = rsqrtf(v);
  return fmaf(r * 0.5f, fmaf(-v * r, r, 1.f), r);
}
// A power of two that brings a row with this largest magnitude near 1.
__device__ __forceinline__ float scale_of(float top) {
  if (!(top > 0.f && top <= FLT_MAX)) return 1.f;
  const int e = max(-126, min(126, 127 - int(__float_as_uint(top) >> 23)));
  return __uint_as_float(uint32_t(e + 127) << 23);
}
// 1 / sqrt(var / scale^2 + eps), in fp64 where the quotient may leave fp32.
static __device__ __noinline__ float rstd_of_scaled(float var, float scale, float eps) {
  const double v = double(var) / (double(scale) * double(scale)) + double(eps);
  return float(1.0 / sqrt(v));
}

// ------------------------------------------------------------------- host
inline int check_vector(const char* name, const void* p, int32_t dtype) {
  if (dtype != TRAIN_BF16 && dtype != TRAIN_FP16 && dtype != TRAIN_FP32)
    return fail(LAMB_ERR_INVALID, std::string(name) + ": unknown element type");
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(size_of(dtype)))
    return fail(LAMB_ERR_ALIGN, std::string(name) + " is not aligned to its element type");
  return LAMB_OK;
}

// A matrix, or one row of consecutive elements.
inline Rows rows_of(const char* name, const void* p, int32_t type, int64_t n, int64_t dim,
                    int64_t stride = 0) {
  return {name, p, n, dim, stride, size_of(type), type};
}

inline int launched(const char* what, cudaError_t ce) {
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(ce));
}

}  // namespace traingb
