// Device helpers shared by the operators of train_ops.h.  Not part of the
// public interface.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "train_ops.h"

namespace traingb {

template <int DT>
struct TypeOf;
template <>
struct TypeOf<TRAIN_BF16> {
  using T = uint16_t;
};
template <>
struct TypeOf<TRAIN_FP16> {
  using T = uint16_t;
};
template <>
struct TypeOf<TRAIN_FP32> {
  using T = float;
};

__host__ __device__ constexpr int size_of(int dt) { return dt == TRAIN_FP32 ? 4 : 2; }

template <int DT>
__device__ __forceinline__ float to_float(typename TypeOf<DT>::T x) {
  if constexpr (DT == TRAIN_BF16) return __uint_as_float(uint32_t(x) << 16);
  if constexpr (DT == TRAIN_FP16) return __half2float(__ushort_as_half(x));
  if constexpr (DT == TRAIN_FP32) return x;
}

// Rounds to nearest even, once.
template <int DT>
__device__ __forceinline__ typename TypeOf<DT>::T from_float(float x) {
  if constexpr (DT == TRAIN_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  if constexpr (DT == TRAIN_FP16) return __half_as_ushort(__float2half_rn(x));
  if constexpr (DT == TRAIN_FP32) return x;
}

}  // namespace traingb
