// Device helpers shared by the operators of train_ops.h.  Not part of the
// public interface.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "lamb_internal.h"
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

// Two values rounded to 16 bits, the first in the low half: one instruction.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  static_assert(DT != TRAIN_FP32, "16-bit types");
  if constexpr (DT == TRAIN_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

template <int DT>
struct Type {
  static constexpr int value = DT;
};

// Calls f with a type known at run time as a compile-time value, so that loops
// inside f do not ask again.
template <class F>
__device__ __forceinline__ void by_type(int type, F&& f) {
  if (type == TRAIN_BF16) f(Type<TRAIN_BF16>{});
  else if (type == TRAIN_FP32) f(Type<TRAIN_FP32>{});
  else f(Type<TRAIN_FP16>{});
}

// VEC neighbouring elements, aligned to their size together or to 16 bytes.
template <int DT, int VEC>
struct Pack {
  using T = typename TypeOf<DT>::T;
  static constexpr int kBytes = VEC * int(sizeof(T));
  uint32_t w[(kBytes + 3) / 4];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
    }
  }
  // The same of what is read once, by a plain load: what a kernel also writes.
  __device__ __forceinline__ void load_once(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = uint16_t(w[0]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (kBytes + 3) / 4; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == TRAIN_FP32) {
      return __uint_as_float(w[i]);
    } else {
      return to_float<DT>(uint16_t((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xffffu));
    }
  }
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
    if constexpr (DT == TRAIN_FP32) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(x[i]);
    } else if constexpr (VEC == 1) {
      w[0] = from_float<DT>(x[0]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) w[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
    }
  }
};

// Two fp32 values in one register pair, for the instructions that work on both.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 pair(float x) { return pair(x, x); }
__device__ __forceinline__ void split(F2 p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(F2 p) {
  float lo, hi;
  split(p, lo, hi);
  return lo + hi;
}

// Elements 2 i and 2 i + 1 of a pack.
template <int DT, int VEC>
__device__ __forceinline__ F2 get2(const Pack<DT, VEC>& p, int i) {
  static_assert(VEC % 2 == 0, "pairs");
  if constexpr (DT == TRAIN_FP32) {
    return pair(__uint_as_float(p.w[2 * i]), __uint_as_float(p.w[2 * i + 1]));
  } else if constexpr (DT == TRAIN_BF16) {
    // Byte permutation: a shift may become a multiplication, in the pipe of the sums.
    return pair(__uint_as_float(__byte_perm(p.w[i], 0u, 0x1044)),
                __uint_as_float(p.w[i] & 0xffff0000u));
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p.w[i]));
    return pair(f.x, f.y);
  }
}
template <int DT, int VEC>
__device__ __forceinline__ void set2(Pack<DT, VEC>& p, int i, F2 x) {
  float lo, hi;
  split(x, lo, hi);
  if constexpr (DT == TRAIN_FP32) {
    p.w[2 * i] = __float_as_uint(lo), p.w[2 * i + 1] = __float_as_uint(hi);
  } else {
    p.w[i] = pack2<DT>(lo, hi);
  }
}

// Lets the kernel behind this one start (its CTAs wait for this one to end
// before they touch what it writes), and waits for the kernel in front.
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kWarp = 32;
constexpr unsigned kAll = 0xffffffffu;

// Row of the table (or of its gradient) that a token names, or -1.
template <class ID>
__device__ __forceinline__ int64_t row_of(ID id, int64_t first_row, int64_t n_rows) {
  const uint64_t r = uint64_t(int64_t(id)) - uint64_t(first_row);
  return r < uint64_t(n_rows) ? int64_t(r) : -1;
}

// ------------------------------------------------------------------- host
inline int fail(int code, const std::string& msg) {
  lambgb::set_last_error(msg);
  return code;
}

constexpr int64_t kMaxCount = 0x7fffffff;

// Checks one matrix; LAMB_OK or the error.
inline int check_matrix(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t dim,
                 int64_t stride) {
  if (dtype != TRAIN_BF16 && dtype != TRAIN_FP16 && dtype != TRAIN_FP32)
    return fail(LAMB_ERR_INVALID, std::string(name) + ": unknown element type");
  if (rows < 0 || dim < 0 || rows > kMaxCount || dim > kMaxCount)
    return fail(LAMB_ERR_INVALID, std::string(name) + ": sizes must be in [0, 2^31 - 1]");
  if (stride < dim)
    return fail(LAMB_ERR_INVALID, std::string(name) + ": stride is less than dim");
  if (rows == 0 || dim == 0) return LAMB_OK;
  if (!p) return fail(LAMB_ERR_INVALID, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(size_of(dtype)))
    return fail(LAMB_ERR_ALIGN, std::string(name) + " is not aligned to its element type");
  return LAMB_OK;
}

inline int check_ids(const void* ids, int32_t ids_dtype, int64_t n_ids, int64_t first_row,
                     int64_t n_rows) {
  if (ids_dtype != TRAIN_INT32 && ids_dtype != TRAIN_INT64)
    return fail(LAMB_ERR_INVALID, "ids: unknown type");
  if (n_ids < 0 || n_ids > kMaxCount)
    return fail(LAMB_ERR_INVALID, "n_ids must be in [0, 2^31 - 1]");
  if (first_row < 0) return fail(LAMB_ERR_INVALID, "first_row must be >= 0");
  // Rows behind the last number would be named by negative ids.
  if (n_rows > 0 && first_row > INT64_MAX - (n_rows - 1))
    return fail(LAMB_ERR_INVALID, "first_row + n_rows - 1 must be at most 2^63 - 1");
  if (n_ids == 0) return LAMB_OK;
  if (!ids) return fail(LAMB_ERR_INVALID, "ids is NULL");
  if (reinterpret_cast<uintptr_t>(ids) % (ids_dtype == TRAIN_INT64 ? 8u : 4u))
    return fail(LAMB_ERR_ALIGN, "ids is not aligned to its type");
  return LAMB_OK;
}

// What a call reads or writes: rows of `dim` elements, `stride` elements apart.
struct Rows {
  const char* name;
  const void* p;
  int64_t n, dim, stride;
  int size;  // bytes an element
  int32_t type;
  __int128 end;  // behind the last byte; 0 if there is none

  Rows(const char* name, const void* p, int64_t n, int64_t dim, int64_t stride, int size,
       int32_t type)
      : name(name), p(p), n(n), dim(dim), stride(stride), size(size), type(type), end(0) {
    if (p && n > 0 && dim > 0) end = begin() + (__int128(n - 1) * stride + dim) * size;
  }
  __int128 begin() const { return __int128(reinterpret_cast<uintptr_t>(p)); }
};

// Whether two of them have a byte in common.  Exact where the strides are alike or no two
// rows can meet at any distance; at two strides whose rows could meet, the ranges decide.
inline bool meet(const Rows& a, const Rows& b) {
  using I = __int128;
  const I at = a.begin(), bt = b.begin();
  if (a.end <= bt || b.end <= at) return false;
  const I wa = I(a.dim) * a.size, wb = I(b.dim) * b.size;
  const I sa = a.n > 1 ? I(a.stride) * a.size : 0, sb = b.n > 1 ? I(b.stride) * b.size : 0;
  // Row i of a and row j of b meet where i sa - j sb, a multiple of g, lies between
  // bt - at - wa and bt - at + wb.
  I g = sa, r = sb;
  while (r) {
    const I rest = g % r;
    g = r, r = rest;
  }
  if (g == 0) return true;
  const I last = bt - at + wb - 1;
  const I most = last - ((last % g) + g) % g;  // the largest multiple that is not above
  return most > bt - at - wa;
}

// Refuses an output that lies partly over something else of its call; `same`: it may be
// that very matrix.
inline int check_apart(const Rows& out, const Rows& other, bool same = false) {
  if (!meet(out, other)) return LAMB_OK;
  if (same && out.p == other.p && out.type == other.type &&
      (out.stride == other.stride || out.n == 1))
    return LAMB_OK;
  return fail(LAMB_ERR_INVALID, std::string(out.name) + " overlaps " + other.name);
}

// Launches a kernel, if asked as a programmatic dependent of the one before
// it in the stream, in clusters of `cluster` CTAs.
template <class... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   bool dependent, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int k = 0;
  if (dependent) {
    attr[k].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[k++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[k].id = cudaLaunchAttributeClusterDimension;
    attr[k].val.clusterDim.x = unsigned(cluster);
    attr[k].val.clusterDim.y = 1;
    attr[k++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(k);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace traingb
