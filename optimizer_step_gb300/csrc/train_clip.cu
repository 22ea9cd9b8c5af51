// Global gradient norm over many tensors and clipping (train_ops.h).
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "lamb_internal.h"
#include "train_internal.h"

using namespace traingb;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kMaxItem = 16384;

// One piece of a tensor: count elements from src, written to dst.
struct Item {
  const void* src;
  void* dst;
  int32_t count;
  int16_t in, out;  // element types
};

// What the kernels of one call leave for one another.
struct Scalars {
  double sum;        // sum of g^2
  float factor;      // c / S, 0 when a grad is not finite
  uint32_t bad;      // a grad is inf or NaN
  uint32_t ticket;   // CTAs of the norm kernel that have finished
  uint32_t flag;     // OR of the CTAs' inf/NaN flags
};

struct Tables {
  const Item* items;
  double* partial;  // per CTA of the norm kernel
  Scalars* sc;
  int64_t n_items;
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Fixed-shape block sum; the result is valid in every thread.
__device__ __forceinline__ double block_sum(double x, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_sum(x);
  if (lane == 0) red[warp] = x;
  __syncthreads();
  double y = lane < kWarps ? red[lane] : 0.0;
  y = warp_sum(y);
  __syncthreads();
  return y;
}

__device__ __forceinline__ float load_any(const Item& it, int64_t i) {
  if (it.in == TRAIN_FP32) return static_cast<const float*>(it.src)[i];
  const uint16_t x = static_cast<const uint16_t*>(it.src)[i];
  return it.in == TRAIN_BF16 ? to_float<TRAIN_BF16>(x) : to_float<TRAIN_FP16>(x);
}

__device__ __forceinline__ void store_any(const Item& it, int64_t i, float x) {
  if (it.out == TRAIN_FP32) static_cast<float*>(it.dst)[i] = x;
  else if (it.out == TRAIN_BF16) static_cast<uint16_t*>(it.dst)[i] = from_float<TRAIN_BF16>(x);
  else static_cast<uint16_t*>(it.dst)[i] = from_float<TRAIN_FP16>(x);
}

// Forms the norm, the factor and the flag from the sum (one thread).
__device__ void publish(Scalars* sc, float* stats, double sum, bool bad, float max_norm,
                        float loss_scale) {
  const double root = sqrt(sum);
  const double norm = root / double(loss_scale);
  double factor = 1.0 / double(loss_scale);
  if (max_norm > 0.0f && norm > double(max_norm)) factor = double(max_norm) / root;
  sc->factor = bad ? 0.0f : float(factor);
  sc->bad = bad;
  stats[0] = bad ? __int_as_float(0x7f800000) : float(norm);
  stats[1] = sc->factor;
  stats[2] = bad ? 1.0f : 0.0f;
}

// Sum of squares: each CTA walks its items; the last one to finish adds the
// CTAs' sums in order and publishes.
__global__ void __launch_bounds__(kThreads) norm_kernel(Tables T, float max_norm,
                                                        float loss_scale, float* stats,
                                                        double* exchange) {
  __shared__ double red[kWarps];
  __shared__ uint32_t last;
  double acc = 0.0;
  int bad = 0;
  for (int64_t k = blockIdx.x; k < T.n_items; k += gridDim.x) {
    const Item it = T.items[k];
    for (int i = threadIdx.x; i < it.count; i += kThreads) {
      const float x = load_any(it, i);
      bad |= !isfinite(x);
      acc += double(x) * double(x);
    }
  }
  const double s = block_sum(acc, red);
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    T.partial[blockIdx.x] = s;
    if (bad) atomicOr(&T.sc->flag, 1u);
    __threadfence();
    last = atomicAdd(&T.sc->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
  for (int i = threadIdx.x; i < int(gridDim.x); i += kThreads) sum += __ldcg(&T.partial[i]);
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) {
    const bool any = atomicExch(&T.sc->flag, 0u) != 0;
    T.sc->ticket = 0;
    if (exchange) {
      exchange[0] = any ? 0.0 : sum;
      exchange[1] = any ? 1.0 : 0.0;
    } else {
      publish(T.sc, stats, sum, any, max_norm, loss_scale);
    }
  }
}

__global__ void finish_kernel(Tables T, const double* exchange, float max_norm, float loss_scale,
                              float* stats) {
  publish(T.sc, stats, exchange[0], !(exchange[1] == 0.0), max_norm, loss_scale);
}

__global__ void __launch_bounds__(kThreads) scale_kernel(Tables T) {
  const float factor = T.sc->factor;
  if (T.sc->bad) return;
  for (int64_t k = blockIdx.x; k < T.n_items; k += gridDim.x) {
    const Item it = T.items[k];
    if (it.src == it.dst && factor == 1.0f) continue;
    for (int i = threadIdx.x; i < it.count; i += kThreads)
      store_any(it, i, factor * load_any(it, i));
  }
}

int fail(int code, const std::string& msg) {
  lambgb::set_last_error(msg);
  return code;
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
};

namespace {

int check_scale(float loss_scale, float max_norm) {
  if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale))
    return fail(LAMB_ERR_INVALID, "loss_scale must be finite and > 0");
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

int launch_norm(train_clip_handle* h, float max_norm, float loss_scale, float* stats,
                double* exchange) {
  norm_kernel<<<h->grid, kThreads, 0, h->stream>>>(h->T, max_norm, loss_scale, stats, exchange);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? LAMB_OK : cuda_fail(ce, "norm kernel");
}

int launch_scale(train_clip_handle* h) {
  if (h->T.n_items == 0) return LAMB_OK;
  scale_kernel<<<h->grid, kThreads, 0, h->stream>>>(h->T);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? LAMB_OK : cuda_fail(ce, "scale kernel");
}

int create(train_clip_handle** out, int32_t n, const int64_t* sizes, const int32_t* dtypes,
           void* const* grads, void* const* outs, const int32_t* out_dtypes, void* stream) {
  std::vector<Item> items;
  for (int32_t i = 0; i < n; ++i) {
    const std::string at = "[" + std::to_string(i) + "]";
    if (sizes[i] < 0) return fail(LAMB_ERR_INVALID, "sizes" + at + " < 0");
    if (!known(dtypes[i])) return fail(LAMB_ERR_INVALID, "dtypes" + at + ": unknown type");
    const int32_t to = outs ? out_dtypes[i] : dtypes[i];
    if (!known(to)) return fail(LAMB_ERR_INVALID, "out_dtypes" + at + ": unknown type");
    if (sizes[i] == 0) continue;
    void* dst = outs ? outs[i] : grads[i];
    int rc = check_device(grads[i], size_t(size_of(dtypes[i])), ("grads" + at).c_str());
    if (rc == LAMB_OK) rc = check_device(dst, size_t(size_of(to)), ("outs" + at).c_str());
    if (rc != LAMB_OK) return rc;
    if (dst == grads[i] && to != dtypes[i])
      return fail(LAMB_ERR_INVALID, "outs" + at + " is grads" + at + ", of another type");
    for (int64_t b = 0; b < sizes[i]; b += kMaxItem) {
      const int64_t c = sizes[i] - b < kMaxItem ? sizes[i] - b : kMaxItem;
      items.push_back(Item{static_cast<const char*>(grads[i]) + b * size_of(dtypes[i]),
                           static_cast<char*>(dst) + b * size_of(to), int32_t(c),
                           int16_t(dtypes[i]), int16_t(to)});
    }
  }
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess)
    ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess) return cuda_fail(ce, "querying the device");
  const int grid = sms * 4;
  const size_t item_bytes = (items.size() * sizeof(Item) + 255) / 256 * 256;
  const size_t part_bytes = (size_t(grid) * sizeof(double) + 255) / 256 * 256;
  void* block = nullptr;
  ce = cudaMalloc(&block, item_bytes + part_bytes + sizeof(Scalars));
  if (ce != cudaSuccess) return cuda_fail(ce, "allocating the work table");
  char* p = static_cast<char*>(block);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!items.empty())
    ce = cudaMemcpyAsync(p, items.data(), items.size() * sizeof(Item), cudaMemcpyHostToDevice, s);
  if (ce == cudaSuccess)
    ce = cudaMemsetAsync(p + item_bytes, 0, part_bytes + sizeof(Scalars), s);
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
  h->grid = grid;
  h->T.items = reinterpret_cast<const Item*>(p);
  h->T.partial = reinterpret_cast<double*>(p + item_bytes);
  h->T.sc = reinterpret_cast<Scalars*>(p + item_bytes + part_bytes);
  h->T.n_items = int64_t(items.size());
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

LAMB_API int train_clip_norm(train_clip_handle* h, float loss_scale, float* stats) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  int rc = check_scale(loss_scale, 0.0f);
  if (rc == LAMB_OK) rc = check_device(stats, 4, "stats");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  return launch_norm(h, 0.0f, loss_scale, stats, nullptr);
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
  rc = launch_norm(h, max_norm, loss_scale, stats, nullptr);
  return rc == LAMB_OK ? launch_scale(h) : rc;
}

LAMB_API int train_clip_partial(train_clip_handle* h, double* exchange) {
  lambgb::set_last_error("");
  if (!h) return fail(LAMB_ERR_INVALID, "handle is NULL");
  const int rc = check_device(exchange, 8, "exchange");
  if (rc != LAMB_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(LAMB_ERR_CUDA, "cannot make the handle's device current");
  return launch_norm(h, 0.0f, 1.0f, nullptr, exchange);
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
  finish_kernel<<<1, 1, 0, h->stream>>>(h->T, exchange, max_norm, loss_scale, stats);
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
