// Global gradient norm over many tensors and clipping (train_ops.h).
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "train_internal.h"

using namespace traingb;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Bytes of grads in one piece of work: eight 16-byte loads a thread.
constexpr int kLoads = 8;
constexpr int64_t kItemBytes = kThreads * kLoads * 16;
// Half as many as long as the norm's CTAs (3 an SM) take all of those in one round:
// fp32 clipped into bf16, halves against whole ones, 6 MB 9.7 us and 10.4, 6.5 MB 9.5
// and 9.7, 7.6 MB 12.2 and 10.1, 13 MB 16.3 and 11.3, 43 MB 26.5 and 22.8.
constexpr int64_t kHalfBytes = 7 << 20;
// What fits into L2.
constexpr int64_t kSmallTotal = 128 << 20;
constexpr int64_t kEarlyBytes = 5 << 20;
// Items of at most so many bytes are packed, one a warp of a CTA: 1204 tensors of 4 KB
// are clipped in 8.8 us, with a CTA each in 14.4; 4000 of 2 KB in 12.4 and 24.6.
constexpr int64_t kPackedBytes = 4096;
// CTAs of the norm kernel an SM, from 128 MB on and below.  With 3 the norm of 2.4 GB
// takes 360 us, with 5 330; 600 MB 96 and 90.  Below, 5 are as good or a little better
// (20 MB 8.8 and 8.8 us, 43 MB 12.5 and 12.4, 130 MB 25.6 and 24.6; clipped, 20 MB 16.5
// and 13.7): 3 were chosen when the sums of the CTAs cost more.
constexpr int kNormCtas = 5, kNormCtasSmall = 3;

// One piece of work: count elements from src, written to dst; or, where `in`
// is kPack, count items at src, a warp for each of them in turn.
constexpr int8_t kPack = -1;
struct __align__(32) Item {
  const void* src;
  void* dst;
  int32_t count;
  int8_t in, out;  // element types
  // Elements before the first 16-byte boundary of src, and whether dst is
  // aligned too there (to the 16 bytes or less that a thread writes at a time).
  int8_t head;
  int8_t aligned;
  int64_t unused;
};

// What clipping multiplies by, first by one and then by the other.  A factor below
// 2^-100, of grads that have exploded but are finite, is lifted by a power of two
// that `after` takes off the products, or it would be a number of few bits (below
// 2^-126) or zero.  Lifted it is at least 2^-126 wherever a product can be, and
// below 1, so no product overflows.
struct Factor {
  float lifted, after;
};

// What the kernels of one call leave for one another.
struct Scalars {
  Factor factor;    // c / S
  uint32_t bad;     // a grad is inf or NaN
  uint32_t ticket;  // CTAs of the norm kernel that have finished
};

struct Tables {
  const Item* items;
  double* partial;  // per CTA of the norm kernel
  Scalars* sc;
  int64_t n_items;
  int32_t poison;  // outputs become NaN when a grad is inf or NaN
};

// 16 bytes, in order with the other loads of its kind: as many of a thread's are on
// their way together as it has registers for, all eight in the clipping (62
// registers), fewer in the norm (32 registers, so that more warps run).
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 q;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// Fixed-shape block sum; the result is valid in the first warp.  An fp64 instruction
// of a warp takes 16 cycles of its SM, so one warp adds the threads' values (13 such
// instructions, where shuffles in every warp are 64).
__device__ __forceinline__ double block_sum(double x, double* red) {
  red[threadIdx.x] = x;
  __syncthreads();
  if (threadIdx.x >= kWarp) return 0.0;
  double y = red[threadIdx.x];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) y += red[w * kWarp + threadIdx.x];
#pragma unroll
  for (int o = kWarp / 2; o > 0; o >>= 1) y += __shfl_xor_sync(kAll, y, o);
  return y;
}

template <int DT>
__device__ __forceinline__ float2 decode2(uint32_t w) {
  if constexpr (DT == TRAIN_BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return make_float2(to_float<TRAIN_FP16>(uint16_t(w & 0xffffu)),
                     to_float<TRAIN_FP16>(uint16_t(w >> 16)));
}

struct Squares {
  double sum;
  uint32_t bad;
};

// The squares of one value, exactly enough for any finite one.
__device__ __forceinline__ void add_square(Squares& s, float x) {
  if (isfinite(x)) s.sum = fma(double(x), double(x), s.sum);
  else s.bad = 1u;
}

// The squares of a thread's vectors (v, v + threads, ... below end) in fp64,
// and whether one is inf or NaN.  The rare path: not inlined, and the values
// are read again, so that the fast path carries neither fp64 code nor words
// kept for it.  Where every vector comes here, it is slow: the norm of 2.4 GB takes
// 4.6 ms if they are bf16 of 1e-16, 2.4 ms if they are fp32, instead of 0.33.
template <int DT>
__device__ __noinline__ Squares squares_fp64(const char* base, int v, int end, int threads) {
  Squares s{0.0, 0u};
  for (int u = 0; u < kLoads; ++u, v += threads) {
    if (v >= end) break;
    for (int i = 0; i < 16 / size_of(DT); ++i)
      add_square(s, to_float<DT>(reinterpret_cast<const typename TypeOf<DT>::T*>(
                        base + int64_t(v) * 16)[i]));
  }
  return s;
}

// A thread's share of the squares of one item that `threads` threads take, this
// one the `tid`-th.  They are summed in fp32, at
// most 64 of them, and from there in fp64.  bf16 and fp32 grads span fp32's
// exponents, so their squares may leave its range: a sum outside [2^-90,
// 2^120] (some value not zero) is taken again in fp64.  Inside that range
// nothing overflowed, and what underflowed weighs at most 2^-30 of the sum.
// An inf or NaN makes its sum inf or NaN, which is never inside the range, so
// the fast path does not test for them.  fp16 squares never leave it.
template <int DT>
__device__ __forceinline__ void item_squares(const Item& it, int tid, int threads, double& acc,
                                             uint32_t& bad) {
  using T = typename TypeOf<DT>::T;
  constexpr int kPer = 16 / size_of(DT);
  const int head = it.head;
  const int vecs = (it.count - head) / kPer;
  const char* base = static_cast<const char*>(it.src) + head * size_of(DT);
  const int v = tid;
  uint4 q[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    q[u] = make_uint4(0u, 0u, 0u, 0u);
    if (v + u * threads < vecs) q[u] = load16(base + int64_t(v + u * threads) * 16);
  }
  // What the 16-byte loads leave: up to 7 elements in front and behind.
  const int rest = it.count - vecs * kPer;
  if (tid < rest) {
    const int i = tid < head ? tid : vecs * kPer + tid;
    Squares s{0.0, 0u};
    add_square(s, to_float<DT>(static_cast<const T*>(it.src)[i]));
    acc += s.sum;
    bad |= s.bad;
  }
  float a = 0.0f, b = 0.0f;
  uint32_t any = 0u;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TRAIN_FP32) {
        const float x = __uint_as_float(w[i]);
        if (i & 1) a = fmaf(x, x, a);
        else b = fmaf(x, x, b);
      } else {
        const float2 x = decode2<DT>(w[i]);
        a = fmaf(x.x, x.x, a);
        b = fmaf(x.y, x.y, b);
      }
      if constexpr (DT != TRAIN_FP16) any |= w[i];
    }
  }
  a += b;
  any &= DT == TRAIN_FP32 ? 0x7fffffffu : 0x7fff7fffu;
  if constexpr (DT == TRAIN_FP16) {
    if (a <= 0x1p120f) acc += double(a);
    else bad = 1u;
  } else {
    if (a <= 0x1p120f && (a >= 0x1p-90f || any == 0u)) {
      acc += double(a);
    } else {
      const Squares s = squares_fp64<DT>(base, v, vecs, threads);
      acc += s.sum;
      bad |= s.bad;
    }
  }
}

__device__ __forceinline__ void any_squares(const Item& it, int tid, int threads, double& acc,
                                            uint32_t& bad) {
  if (it.in == TRAIN_BF16) item_squares<TRAIN_BF16>(it, tid, threads, acc, bad);
  else if (it.in == TRAIN_FP32) item_squares<TRAIN_FP32>(it, tid, threads, acc, bad);
  else item_squares<TRAIN_FP16>(it, tid, threads, acc, bad);
}

// Forms the norm, the factor and the flag from the sum of squares (infinite if
// a grad is inf or NaN).  fp64 square roots and divisions cost about half a
// microsecond each on one thread, so there are none: with sum = m 4^k, m in
// [1, 4), one Newton step y (3 - m y^2) / 2 takes the fp32 reciprocal square
// root of m (off by 2^-22 at most) to 2^-42, and the norm m y 2^k / S and the
// factor max_norm y / 2^k are products.
struct Request {
  double inv_scale;  // 1 / S
  double max_norm;
  float* stats;
  double* exchange;  // not NULL: only the sum and the flag, here
  bool early;        // the next kernel may start at once
};

__device__ __forceinline__ void publish(Scalars* sc, const Request& r, double sum) {
  const bool bad = !(sum < __longlong_as_double(0x7ff0000000000000ll));
  double root = 0.0, inverse = 0.0;
  if (!bad && sum > 0.0) {
    // Squares of fp32 numbers, so sum is a normal number.
    const int64_t bits = __double_as_longlong(sum);
    const int k = (int(bits >> 52) - 1023) >> 1;
    const double m = __longlong_as_double(bits - (int64_t(2 * k) << 52));
    double y = double(rsqrtf(float(m)));
    y *= fma(-0.5 * m * y, y, 1.5);
    root = m * y * __longlong_as_double(int64_t(1023 + k) << 52);
    inverse = y * __longlong_as_double(int64_t(1023 - k) << 52);
  }
  const double norm = root * r.inv_scale;
  const double factor = r.max_norm > 0.0 && norm > r.max_norm ? r.max_norm * inverse : r.inv_scale;
  // By its exponent alone; the factor is a normal number.
  const int64_t word = __double_as_longlong(factor);
  const int exponent = int(word >> 52) - 1023;
  const int lift = exponent >= -100 ? 0 : exponent >= -226 ? 100 : 149;
  sc->factor.lifted = float(__longlong_as_double(word + (int64_t(lift) << 52)));
  sc->factor.after = lift == 0 ? 1.0f : lift == 100 ? 0x1p-100f : 0x1p-149f;
  sc->bad = bad;
  r.stats[0] = bad ? __int_as_float(0x7f800000) : float(norm);
  r.stats[1] = bad ? 0.0f : float(factor);
  r.stats[2] = bad ? 1.0f : 0.0f;
}

// Sum of squares: each CTA walks every gridDim.x-th item, all of them through
// memory side by side; the last one to finish adds the CTAs' sums in order and
// publishes.  It is bound by reading: 1.2e9 fp16 grads take 331 us on GB300, 7.3
// TB/s.  With a few MB it is a chain of latencies: 6 MB take 6.3 us, 43 MB (three
// items for most CTAs, two for the others) 12.5; behind the last data come the CTAs'
// sums, their tickets and the sum of those.
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Tables T,
                                                        const __grid_constant__ Request r) {
  __shared__ double red[kThreads];
  __shared__ uint32_t last;
  if (r.early) pdl_trigger();
  double acc = 0.0;
  uint32_t bad = 0;
  Item next{};
  if (blockIdx.x < T.n_items) next = T.items[blockIdx.x];
  pdl_wait();
  for (int64_t k = blockIdx.x; k < T.n_items; k += gridDim.x) {
    const Item it = next;
    if (k + gridDim.x < T.n_items) next = T.items[k + gridDim.x];
    if (it.in != kPack) {
      any_squares(it, threadIdx.x, kThreads, acc, bad);
      continue;
    }
    const Item* packed = static_cast<const Item*>(it.src);
#pragma unroll 1
    for (int i = threadIdx.x >> 5; i < it.count; i += kWarps)
      any_squares(packed[i], threadIdx.x & 31, kWarp, acc, bad);
  }
  if (!r.early) pdl_trigger();
  // An inf or NaN grad makes the sum infinite; finite grads cannot.
  if (bad) acc = __longlong_as_double(0x7ff0000000000000ll);
  const double s = block_sum(acc, red);
  if (threadIdx.x == 0) {
    __stcg(&T.partial[blockIdx.x], s);
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(&T.sc->ticket)
                 : "memory");
    last = before == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double sum = threadIdx.x < gridDim.x ? __ldcg(&T.partial[threadIdx.x]) : 0.0;
  for (int i = threadIdx.x + kThreads; i < int(gridDim.x); i += kThreads)
    sum += __ldcg(&T.partial[i]);
  sum = block_sum(sum, red);
  if (threadIdx.x != 0) return;
  T.sc->ticket = 0;
  if (r.exchange) {
    const bool any = !(sum < __longlong_as_double(0x7ff0000000000000ll));
    r.exchange[0] = any ? 0.0 : sum;
    r.exchange[1] = any ? 1.0 : 0.0;
  } else {
    publish(T.sc, r, sum);
  }
}

__global__ void finish_kernel(const __grid_constant__ Tables T,
                              const __grid_constant__ Request r) {
  pdl_trigger();
  publish(T.sc, r,
          r.exchange[1] == 0.0 ? r.exchange[0] : __longlong_as_double(0x7ff0000000000000ll));
}

template <int IN>
__device__ __forceinline__ float load_value(const Item& it, int i) {
  return to_float<IN>(static_cast<const typename TypeOf<IN>::T*>(it.src)[i]);
}
template <int OUT>
__device__ __forceinline__ void store_value(const Item& it, int i, float x) {
  static_cast<typename TypeOf<OUT>::T*>(it.dst)[i] = from_float<OUT>(x);
}

// src times the factor into dst: 16 bytes of src a thread and load, coalesced on both
// sides, or element by element where src and dst are aligned differently.
template <int IN, int OUT>
__device__ __forceinline__ void item_scale(const Item& it, int tid, int threads, Factor f) {
  using TO = typename TypeOf<OUT>::T;
  constexpr int kPer = 16 / size_of(IN);
  if (!it.aligned) {
#pragma unroll 8
    for (int i = tid; i < it.count; i += threads)
      store_value<OUT>(it, i, f.lifted * load_value<IN>(it, i) * f.after);
    return;
  }
  const int head = it.head;
  const int vecs = (it.count - head) / kPer;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(it.src) +
                                                    head * size_of(IN));
  TO* dst = static_cast<TO*>(it.dst) + head;
  uint4 q[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    q[u] = make_uint4(0u, 0u, 0u, 0u);  // or it would be live from one item to the next
    if (tid + u * threads < vecs) q[u] = load16(src + tid + u * threads);
  }
  const int rest = it.count - vecs * kPer;
  if (tid < rest) {
    const int i = tid < head ? tid : vecs * kPer + tid;
    store_value<OUT>(it, i, f.lifted * load_value<IN>(it, i) * f.after);
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int v = tid + u * threads;
    if (v >= vecs) continue;
    const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
    float x[kPer];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (IN == TRAIN_FP32) {
        x[i] = f.lifted * __uint_as_float(w[i]) * f.after;
      } else {
        const float2 d = decode2<IN>(w[i]);
        x[2 * i] = f.lifted * d.x * f.after;
        x[2 * i + 1] = f.lifted * d.y * f.after;
      }
    }
    if constexpr (OUT == TRAIN_FP32) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4)
        reinterpret_cast<float4*>(dst + int64_t(v) * kPer)[i / 4] =
            make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
      uint32_t y[kPer / 2];
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i)
        y[i] = pack2<OUT>(x[2 * i], x[2 * i + 1]);
      if constexpr (kPer == 8)
        *reinterpret_cast<uint4*>(dst + int64_t(v) * kPer) = make_uint4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2*>(dst + int64_t(v) * kPer) = make_uint2(y[0], y[1]);
    }
  }
}

template <int IN>
__device__ __forceinline__ void item_scale_to(const Item& it, int tid, int threads,
                                              Factor f) {
  if (it.out == TRAIN_BF16) item_scale<IN, TRAIN_BF16>(it, tid, threads, f);
  else if (it.out == TRAIN_FP32) item_scale<IN, TRAIN_FP32>(it, tid, threads, f);
  else item_scale<IN, TRAIN_FP16>(it, tid, threads, f);
}

__device__ __forceinline__ void any_scale(const Item& it, int tid, int threads, Factor f) {
  if (it.src == it.dst && f.lifted == 1.0f) return;
  if (it.in == TRAIN_BF16) item_scale_to<TRAIN_BF16>(it, tid, threads, f);
  else if (it.in == TRAIN_FP32) item_scale_to<TRAIN_FP32>(it, tid, threads, f);
  else item_scale_to<TRAIN_FP16>(it, tid, threads, f);
}

// One item a CTA, so that the CTAs go through memory in the order they are
// launched: on GB300 a copy runs at 7.1 TB/s this way and at 6.5 with a
// persistent grid.  The last items come first: the norm kernel read them last,
// and they may still be in L2.  1.8e9 fp32 grads clipped into bf16 take 2.48 ms in
// all: 18.1 GB with the second reading, 7.3 TB/s.
__global__ void __launch_bounds__(kThreads) scale_kernel(Tables T) {
  const Item it = T.items[T.n_items - 1 - blockIdx.x];
  pdl_trigger();
  pdl_wait();
  Factor f = T.sc->factor;
  if (T.sc->bad) {
    if (!T.poison) return;
    f.lifted = __int_as_float(0x7fffffff);  // NaN times anything
  }
  const bool pack = it.in == kPack;
  const Item* packed = static_cast<const Item*>(it.src);
  const int count = pack ? it.count : 1, tid = pack ? threadIdx.x & 31 : threadIdx.x;
#pragma unroll 1
  for (int i = pack ? threadIdx.x >> 5 : 0; i < count; i += kWarps)
    any_scale(pack ? packed[i] : it, tid, pack ? kWarp : kThreads, f);
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(e == cudaErrorMemoryAllocation ? LAMB_ERR_NOMEM : LAMB_ERR_CUDA,
              std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) +
                  ")");
}

// Makes the handle's device current for a call and restores the caller's.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

}  // namespace

struct train_clip_handle {
  int device = 0;
  cudaStream_t stream = nullptr;
  void* block = nullptr;
  Tables T{};
  int grid = 1;
  int64_t bytes = 0;  // of grads, or kSmallTotal if there are more
};

namespace {

int check_scale(float loss_scale, float max_norm) {
  if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale))
    return fail(LAMB_ERR_INVALID, "loss_scale must be finite and > 0");
  // The factor 1 / S would be inf, and zeros times it NaN.
  if (!std::isfinite(float(1.0 / double(loss_scale))))
    return fail(LAMB_ERR_INVALID, "loss_scale is so small that 1 / loss_scale is not finite");
  if (std::isnan(max_norm)) return fail(LAMB_ERR_INVALID, "max_norm is NaN");
  return LAMB_OK;
}

int check_device(const void* p, size_t align, const char* name) {
  if (!p) return fail(LAMB_ERR_INVALID, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(LAMB_ERR_ALIGN, std::string(name) + " is not aligned to its element type");
  return LAMB_OK;
}

bool known(int32_t dt) { return dt == TRAIN_BF16 || dt == TRAIN_FP16 || dt == TRAIN_FP32; }

// Launches, if asked as a programmatic dependent of the kernel before it, so
// that its CTAs have their items when that one ends.
template <class... A>
int launch(train_clip_handle* h, const char* what, void (*kernel)(A...), int64_t grid,
           bool dependent, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = h->stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  const cudaError_t ce = cudaLaunchKernelEx(&cfg, kernel, args...);
  return ce == cudaSuccess ? LAMB_OK : cuda_fail(ce, what);
}

// Which kernel starts beside which, measured on GB300:
// - The clipping's CTAs may start at once, beside the norm: 6 MB 9.7 us instead of
//   10.0, 6.5 MB 9.5 instead of 10.3; 8 to 17 MB cost up to 8% so, and 20 MB and more
//   are the same either way.  Below 5 MB they wait until the squares are added: 9.3 us instead
//   of 9.9 at 4.5 MB, 6.4 instead of 6.9 at 0.7.
// - So does whatever follows the norm alone.
// - The norm itself starts before the kernel in front has ended (4.6 us instead of 6.2
//   at 0.7 MB, 12.5 instead of 14.4 at 43 MB), unless it walks over many items in front
//   of a clipping: CTAs that are spread over the SMs unevenly cost 4% at 600 MB (234 us
//   instead of 224), though 20 and 43 MB would gain (14.3 instead of 16.5, 20.7 instead
//   of 22.8).  Alone from 128 MB on it would gain 3% (600 MB: 87 us instead of 90).
int launch_norm(train_clip_handle* h, bool alone, Request r) {
  r.early = !alone && h->bytes >= kEarlyBytes;
  const bool dependent = h->T.n_items <= h->grid || (alone && h->bytes < kSmallTotal);
  return launch(h, "norm kernel", norm_kernel, h->grid, dependent, h->T, r);
}

int launch_scale(train_clip_handle* h) {
  if (h->T.n_items == 0) return LAMB_OK;
  return launch(h, "scale kernel", scale_kernel, h->T.n_items, true, h->T);
}

// A run of neighbouring elements: a tensor, or several that lie one behind the
// other on both sides.
struct Span {
  const char* src;
  char* dst;
  int64_t n;
  int32_t in, out;
};

// The memory of one tensor.
struct Range {
  uintptr_t begin, end;
  int32_t index;
  bool out;
};

// Every tensor but an output that is its own grad has memory of its own.
int check_disjoint(std::vector<Range>& ranges) {
  std::sort(ranges.begin(), ranges.end(),
            [](const Range& a, const Range& b) { return a.begin < b.begin; });
  const auto name = [](const Range& r) {
    return (r.out ? "outs[" : "grads[") + std::to_string(r.index) + "]";
  };
  for (size_t i = 1; i < ranges.size(); ++i)
    if (ranges[i].begin < ranges[i - 1].end)
      return fail(LAMB_ERR_INVALID, name(ranges[i - 1]) + " and " + name(ranges[i]) + " overlap");
  return LAMB_OK;
}

// Cuts a span into items whose first 16-byte loads are aligned: only its first
// item has elements in front of them.  Small ones go to `small`.
void add_items(std::vector<Item>* items, std::vector<Item>* small, const Span& span,
               int64_t item_bytes) {
  const int si = size_of(span.in), so = size_of(span.out);
  const int64_t per = item_bytes / si;
  const int head = int((16 - reinterpret_cast<uintptr_t>(span.src) % 16) % 16) / si;
  const int wide = 16 / si * so < 16 ? 16 / si * so : 16;  // bytes of dst written at a time
  const bool aligned = reinterpret_cast<uintptr_t>(span.dst + head * so) % unsigned(wide) == 0;
  for (int64_t b = 0; b < span.n;) {
    const int64_t left = span.n - b;
    Item it{};
    it.src = span.src + b * si;
    it.dst = span.dst + b * so;
    it.head = int8_t(b == 0 ? (head < left ? head : left) : 0);
    it.count = int32_t(left < per + it.head ? left : per + it.head);
    it.in = int8_t(span.in);
    it.out = int8_t(span.out);
    it.aligned = aligned;
    (it.count * si <= kPackedBytes ? small : items)->push_back(it);
    b += it.count;
  }
}

int create(train_clip_handle** out, int32_t n, const int64_t* sizes, const int32_t* dtypes,
           void* const* grads, void* const* outs, const int32_t* out_dtypes, void* stream) {
  std::vector<Span> spans;
  std::vector<Range> ranges;
  spans.reserve(size_t(n));
  ranges.reserve(outs ? 2 * size_t(n) : size_t(n));
  int64_t total = 0;  // bytes, or kSmallTotal if there are more
  for (int32_t i = 0; i < n; ++i) {
    const auto at = [i](const char* what) { return what + ("[" + std::to_string(i) + "]"); };
    if (sizes[i] < 0) return fail(LAMB_ERR_INVALID, at("sizes") + " < 0");
    if (!known(dtypes[i])) return fail(LAMB_ERR_INVALID, at("dtypes") + ": unknown type");
    const int32_t to = outs ? out_dtypes[i] : dtypes[i];
    if (!known(to)) return fail(LAMB_ERR_INVALID, at("out_dtypes") + ": unknown type");
    if (sizes[i] == 0) continue;
    void* dst = outs ? outs[i] : grads[i];
    const int si = size_of(dtypes[i]), so = size_of(to);
    if (!grads[i]) return fail(LAMB_ERR_INVALID, at("grads") + " is NULL");
    if (!dst) return fail(LAMB_ERR_INVALID, at("outs") + " is NULL");
    if (reinterpret_cast<uintptr_t>(grads[i]) % unsigned(si))
      return fail(LAMB_ERR_ALIGN, at("grads") + " is not aligned to its element type");
    if (reinterpret_cast<uintptr_t>(dst) % unsigned(so))
      return fail(LAMB_ERR_ALIGN, at("outs") + " is not aligned to its element type");
    if (dst == grads[i] && to != dtypes[i])
      return fail(LAMB_ERR_INVALID, at("outs") + " is " + at("grads") + ", of another type");
    if (sizes[i] > INT64_MAX / 8) return fail(LAMB_ERR_INVALID, at("sizes") + " is too large");
    spans.push_back(Span{static_cast<const char*>(grads[i]), static_cast<char*>(dst), sizes[i],
                         dtypes[i], to});
    const auto range = [&](const void* p, int size, bool out) {
      const uintptr_t begin = reinterpret_cast<uintptr_t>(p);
      ranges.push_back(Range{begin, begin + uintptr_t(sizes[i]) * unsigned(size), i, out});
    };
    range(grads[i], si, false);
    if (dst != grads[i]) range(dst, so, true);
    total = sizes[i] * si < kSmallTotal - total ? total + sizes[i] * si : kSmallTotal;
  }
  const int rc = check_disjoint(ranges);
  if (rc != LAMB_OK) return rc;
  // In the order of memory, neighbours joined.
  std::stable_sort(spans.begin(), spans.end(),
                   [](const Span& a, const Span& b) { return a.src < b.src; });
  const int64_t item_bytes = total < kHalfBytes ? kItemBytes / 2 : kItemBytes;
  std::vector<Item> items, small;
  for (size_t i = 0; i < spans.size();) {
    Span s = spans[i];
    for (++i; i < spans.size(); ++i) {
      const Span& next = spans[i];
      if (next.in != s.in || next.out != s.out || next.src != s.src + s.n * size_of(s.in) ||
          next.dst != s.dst + s.n * size_of(s.out))
        break;
      s.n += next.n;
    }
    // Refused before they are cut, which would fill the host's memory first.
    if (int64_t(items.size() + small.size()) + s.n / (item_bytes / size_of(s.in)) > kMaxCount / 2)
      return fail(LAMB_ERR_INVALID, "too many elements");
    add_items(&items, &small, s, item_bytes);
  }
  const size_t packs = (small.size() + kWarps - 1) / kWarps;
  const size_t n_items = items.size() + packs;  // followed by the packed ones
  for (size_t k = 0; k < packs; ++k) {
    const size_t left = small.size() - k * kWarps;
    Item it{};
    it.count = int32_t(left < kWarps ? left : kWarps);
    it.in = kPack;
    items.push_back(it);
  }
  items.insert(items.end(), small.begin(), small.end());
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess)
    ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess) return cuda_fail(ce, "querying the device");
  int64_t grid = int64_t(sms) * (total < kSmallTotal ? kNormCtasSmall : kNormCtas);
  if (grid > int64_t(n_items)) grid = n_items ? int64_t(n_items) : 1;
  const size_t table_bytes = (items.size() * sizeof(Item) + 255) / 256 * 256;
  const size_t part_bytes = (size_t(grid) * sizeof(double) + 255) / 256 * 256;
  void* block = nullptr;
  ce = cudaMalloc(&block, table_bytes + part_bytes + sizeof(Scalars));
  if (ce != cudaSuccess) return cuda_fail(ce, "allocating the work table");
  char* p = static_cast<char*>(block);
  for (size_t k = 0; k < packs; ++k)
    items[n_items - packs + k].src = p + (n_items + k * kWarps) * sizeof(Item);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!items.empty())
    ce = cudaMemcpyAsync(p, items.data(), items.size() * sizeof(Item), cudaMemcpyHostToDevice, s);
  if (ce == cudaSuccess)
    ce = cudaMemsetAsync(p + table_bytes, 0, part_bytes + sizeof(Scalars), s);
  if (ce == cudaSuccess) ce = cudaStreamSynchronize(s);
  train_clip_handle* h = ce == cudaSuccess ? new (std::nothrow) train_clip_handle : nullptr;
  if (!h) {
    cudaFree(block);
    return ce == cudaSuccess ? fail(LAMB_ERR_NOMEM, "out of host memory")
                             : cuda_fail(ce, "uploading the work table");
  }
  h->device = dev;
  h->stream = s;
  h->block = block;
  h->grid = int(grid);
  h->bytes = total;
  h->T.items = reinterpret_cast<const Item*>(p);
  h->T.partial = reinterpret_cast<double*>(p + table_bytes);
  h->T.sc = reinterpret_cast<Scalars*>(p + table_bytes + part_bytes);
  h->T.n_items = int64_t(n_items);
  *out = h;
  return LAMB_OK;
}

}  // namespace

extern "C" {

LAMB_API int train_clip_create(train_clip_handle** out, int32_t n_tensors, const int64_t* sizes,
                               const int32_t* dtypes, void* const* grads, void* const* outs,
                               const int32_t* out_dtypes, void* stream) {
  lambgb::set_last_error("");
  if (!out) return fail(LAMB_ERR_INVALID, "out is NULL");
  *out = nullptr;
  if (n_tensors < 0) return fail(LAMB_ERR_INVALID, "n_tensors must be >= 0");
  if (n_tensors > 0 && (!sizes || !dtypes || !grads))
    return fail(LAMB_ERR_INVALID, "sizes, dtypes and grads must be non-NULL");
  if (n_tensors > 0 && outs && !out_dtypes)
    return fail(LAMB_ERR_INVALID, "out_dtypes must be given with outs");
  try {
    return create(out, n_tensors, sizes, dtypes, grads, outs, out_dtypes, stream);
  } catch (const std::bad_alloc&) {
    return fail(LAMB_ERR_NOMEM, "out of host memory");
  }
}

LAMB_API int train_clip_set_poison(train_clip_handle* h, int32_t poison) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  if (poison != 0 && poison != 1) return fail(LAMB_ERR_INVALID, "poison must be 0 or 1");
  h->T.poison = poison;
  return LAMB_OK;
}

LAMB_API int train_clip_norm(train_clip_handle* h, float loss_scale, float* stats) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  int rc = check_scale(loss_scale, 0.0f);
  if (rc == LAMB_OK) rc = check_device(stats, 4, "stats");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  return launch_norm(h, true, Request{1.0 / double(loss_scale), 0.0, stats, nullptr, false});
}

LAMB_API int train_clip_grads(train_clip_handle* h, float max_norm, float loss_scale,
                              float* stats) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  int rc = check_scale(loss_scale, max_norm);
  if (rc == LAMB_OK) rc = check_device(stats, 4, "stats");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  rc = launch_norm(
      h, false, Request{1.0 / double(loss_scale), double(max_norm), stats, nullptr, false});
  return rc == LAMB_OK ? launch_scale(h) : rc;
}

LAMB_API int train_clip_partial(train_clip_handle* h, double* exchange) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  const int rc = check_device(exchange, 8, "exchange");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  return launch_norm(h, true, Request{1.0, 0.0, nullptr, exchange, false});
}

LAMB_API int train_clip_finish(train_clip_handle* h, const double* exchange, float max_norm,
                               float loss_scale, float* stats) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  int rc = check_scale(loss_scale, max_norm);
  if (rc == LAMB_OK) rc = check_device(exchange, 8, "exchange");
  if (rc == LAMB_OK) rc = check_device(stats, 4, "stats");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  finish_kernel<<<1, 1, 0, h->stream>>>(
      h->T, Request{1.0 / double(loss_scale), double(max_norm), stats,
                    const_cast<double*>(exchange), false});
  const cudaError_t ce = cudaGetLastError();
  if (ce != cudaSuccess) return cuda_fail(ce, "finish kernel");
  return launch_scale(h);
}

LAMB_API int train_clip_destroy(train_clip_handle* h) {
  lambgb::set_last_error("");
  if (!h) return LAMB_OK;
  DeviceGuard dg(h->device);
  cudaError_t ce = dg.ok ? cudaStreamSynchronize(h->stream) : cudaErrorInvalidDevice;
  const cudaError_t fe = cudaFree(h->block);
  if (ce == cudaSuccess) ce = fe;
  delete h;
  return ce == cudaSuccess ? LAMB_OK : cuda_fail(ce, "train_clip_destroy");
}

}  // extern "C"
