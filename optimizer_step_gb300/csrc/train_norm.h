// Helpers of layer norm's kernels (train_ops.h).  Not part of the public
// interface.
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

// Whether the squares that gave a variance kept their bits: none left fp32's
// range at the top, and those that did at the bottom are nothing beside eps.
__device__ __forceinline__ bool in_range(float var, float eps) {
  return var <= FLT_MAX && var + eps > 0x1p-80f;
}
__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.f / sqrtf(var + eps); }
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

inline int launched(const char* what, cudaError_t ce) {
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(ce));
}

}  // namespace traingb
