// Layer norm and its backward pass (train_ops.h).
#include "train_norm_rows.h"

using namespace traingb;

namespace {

// ------------------------------------------------------------ rows of any width
// One CTA a row, which it reads three times (from L1 or L2 after the first): rows that fit
// neither the ring (some 18,900 elements of 16 bits, 14,300 of fp32) nor a CTA's registers
// (16,384).  8192 x 4096 bf16 took 61 us this way, 8192 x 19000 takes 220, where 18000 takes
// 118 in the ring.
struct WideArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* stats;
  int64_t n_rows, dim, x_stride, y_stride;
  float eps;
  int32_t x_type, y_type, param_type;
};

constexpr int kWideThreads = 512;

__global__ void __launch_bounds__(kWideThreads) wide_norm_kernel(const WideArgs a) {
  __shared__ float part[2][kWideThreads / kWarp];
  pdl_wait();
  const int64_t row = blockIdx.x;
  by_type(a.x_type, [&](auto X) {
    constexpr int XT = decltype(X)::value;
    using TX = typename TypeOf<XT>::T;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
    const float n = float(a.dim);
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) s += to_float<XT>(x[i]);
    float mean = cta_sum<kWideThreads>(s, part[0]) / n;
    s = 0.f;
    for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) {
      const float d = to_float<XT>(x[i]) - mean;
      s += d * d;
    }
    const float var = cta_sum<kWideThreads>(s, part[1]) / n;
    float rstd;
    if (in_range(var, a.eps)) {
      rstd = rstd_of(var, a.eps);
    } else {
      // The squares leave fp32's range: once more with the row scaled by a power of two.
      float top = 0.f;
      for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads)
        top = fmaxf(top, fabsf(to_float<XT>(x[i])));
      const float scale = scale_of(cta_max<kWideThreads>(top, part[0]));
      s = 0.f;
      for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) s += to_float<XT>(x[i]) * scale;
      const float mean2 = cta_sum<kWideThreads>(s, part[1]) / n;
      s = 0.f;
      for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) {
        const float d = to_float<XT>(x[i]) * scale - mean2;
        s += d * d;
      }
      const float var2 = cta_sum<kWideThreads>(s, part[0]) / n;
      mean = mean2 / scale;
      rstd = rstd_of_scaled(var2, scale, a.eps);
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[row] = mean;
      a.stats[a.n_rows + row] = rstd;
    }
    by_type(a.y_type, [&](auto Y) {
      constexpr int YT = decltype(Y)::value;
      using TY = typename TypeOf<YT>::T;
      TY* y = static_cast<TY*>(a.y) + row * a.y_stride;
      by_type(a.param_type, [&](auto P) {
        constexpr int PT = decltype(P)::value;
        using TP = typename TypeOf<PT>::T;
        const TP* weight = static_cast<const TP*>(a.weight);
        const TP* bias = static_cast<const TP*>(a.bias);
        for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) {
          float v = (to_float<XT>(x[i]) - mean) * rstd;
          if (weight) v *= to_float<PT>(weight[i]);
          if (bias) v += to_float<PT>(bias[i]);
          y[i] = from_float<YT>(v);
        }
      });
    });
  });
}


constexpr int kSms = 152;
constexpr int64_t kMostShared = 224 * 1024;  // a CTA's dynamic shared memory

// Launches the kernel for rows that stay on chip, if there is one; sets `done`.
cudaError_t launch_rows(NormArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream,
                        bool* done) {
  *done = false;
  const int64_t dim = a.dim;
  if (dim > 32768) return cudaSuccess;
  const NormKernels& k = x_dtype == TRAIN_BF16   ? norm_kernels_bf16(y_dtype)
                         : x_dtype == TRAIN_FP16 ? norm_kernels_fp16(y_dtype)
                                                 : norm_kernels_fp32(y_dtype);
  const auto phase = [](const void* p, int32_t type, int64_t e) {
    return int64_t(reinterpret_cast<uintptr_t>(p) / uintptr_t(size_of(type))) % e;
  };
  const auto go = [&](NormKernel kernel, int64_t ctas, int threads, int64_t smem) {
    *done = true;
    if (smem > 40 * 1024) {
      const cudaError_t ce =
          cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
      if (ce != cudaSuccess) return ce;
    }
    return launch(kernel, dim3(unsigned(ctas)), threads, size_t(smem), stream, true, 1, a);
  };
  // Short rows of whole units.
  int64_t e = x_dtype == TRAIN_FP32 || y_dtype == TRAIN_FP32 ? 4 : 8;
  if (dim <= kWarp * e && dim % e == 0 && a.x_stride % e == 0 && a.y_stride % e == 0 &&
      phase(a.x, x_dtype, e) == 0 && phase(a.y, y_dtype, e) == 0) {
    a.lanes = 1;
    while (a.lanes * e < dim) a.lanes *= 2;
    const int64_t rows = kNormThreads / a.lanes * 4;  // a CTA
    return go(k.whole, (a.n_rows + rows - 1) / rows, kNormThreads, 0);
  }
  const int64_t params = 2 * int64_t(staged_width(a.dim)) * 4;
  e = x_dtype == TRAIN_FP32 ? 4 : 8;
  const int64_t px = phase(a.x, x_dtype, e), row = a.x_stride % e;
  if (dim >= 256 && px == phase(a.y, y_dtype, e) && row == a.y_stride % e) {
    a.phase = int32_t(px), a.row_phase = int32_t(row);
    a.period = 1;
    while (a.period * row % e != 0) a.period *= 2;
    const int64_t units = dim / e;
    const int m = (units <= 16 / e * kWarp ? 16 : 32) / int(e);  // units a thread
    a.lanes = int32_t((units + m * kWarp - 1) / (m * kWarp)) * kWarp;
    const int64_t stage = int64_t(m) * a.lanes * 16;  // of a group
    if (params + 2 * stage <= kMostShared && a.lanes <= 768) {
      // As many rows at once as a CTA holds and there are for each SM.
      int64_t groups = std::min<int64_t>(768 / a.lanes, a.lanes == kWarp ? 24 : 15);
      groups = std::min(groups, (a.n_rows + kSms - 1) / kSms);
      groups = std::max<int64_t>(1, std::min(groups, (kMostShared - params) / (2 * stage)));
      a.stages = params + 3 * groups * stage <= kMostShared ? 3 : 2;
      int64_t ctas = std::min<int64_t>(kSms, (a.n_rows + groups - 1) / groups);
      ctas = (ctas + a.period - 1) / a.period * a.period;
      return go(k.ring[a.lanes > kWarp ? 2 : m * e / 32], ctas, int(groups * a.lanes),
                params + a.stages * groups * stage);
    }
  }
  // Element by element.
  int s = 0;
  while (s < 3 && dim > kScalars[s] * kWarp) ++s;
  a.lanes = int32_t((dim + kScalars[s] * kWarp - 1) / (kScalars[s] * kWarp)) * kWarp;
  // Threads without elements read behind the staged vectors' ends.
  const int64_t smem = params + int64_t(kScalars[s]) * kWarp * 4;
  if (a.lanes > 512 || smem > kMostShared) return cudaSuccess;
  const int64_t rows = (a.n_rows + kScalarRows[s] - 1) / kScalarRows[s];
  int64_t groups = std::max<int64_t>(1, std::min<int64_t>(256 / a.lanes, rows));
  const int64_t resident =
      std::max<int64_t>(1, std::min<int64_t>(1024 / (groups * a.lanes), kMostShared / smem));
  return go(k.scalar[a.lanes > kWarp ? 4 : s],
            std::min(resident * kSms, (rows + groups - 1) / groups),
            int(groups * a.lanes), smem);
}

}  // namespace

extern "C" {

LAMB_API int train_layer_norm(const void* x, int32_t x_dtype, int64_t x_stride, int64_t n_rows,
                              int64_t dim, const void* weight, const void* bias,
                              int32_t param_dtype, float eps, void* y, int32_t y_dtype,
                              int64_t y_stride, float* stats, void* stream) {
  lambgb::set_last_error("");
  int rc = check_matrix("x", x, x_dtype, n_rows, dim, x_stride);
  if (rc == LAMB_OK) rc = check_matrix("y", y, y_dtype, n_rows, dim, y_stride);
  if (rc == LAMB_OK) rc = check_vector("weight", weight, param_dtype);
  if (rc == LAMB_OK) rc = check_vector("bias", bias, param_dtype);
  if (rc == LAMB_OK) rc = check_vector("stats", stats, TRAIN_FP32);
  if (rc != LAMB_OK) return rc;
  if (dim == 0) return fail(LAMB_ERR_INVALID, "dim must be at least 1");
  if (!(eps >= 0.f && eps <= FLT_MAX)) return fail(LAMB_ERR_INVALID, "eps must be finite and >= 0");
  if (n_rows == 0) return LAMB_OK;
  const Rows in = rows_of("x", x, x_dtype, n_rows, dim, x_stride);
  const Rows out = rows_of("y", y, y_dtype, n_rows, dim, y_stride);
  const Rows kept = rows_of("stats", stats, TRAIN_FP32, 1, 2 * n_rows);
  const Rows params[] = {rows_of("weight", weight, param_dtype, 1, dim),
                         rows_of("bias", bias, param_dtype, 1, dim)};
  rc = check_apart(out, in, true);
  if (rc == LAMB_OK) rc = check_apart(out, kept);
  if (rc == LAMB_OK) rc = check_apart(kept, in);
  for (const Rows& p : params) {
    if (rc == LAMB_OK) rc = check_apart(out, p);
    if (rc == LAMB_OK) rc = check_apart(kept, p);
  }
  if (rc != LAMB_OK) return rc;
  NormArgs f{};
  f.x = x, f.weight = weight, f.bias = bias, f.y = y, f.stats = stats;
  f.n_rows = n_rows, f.x_stride = x_stride, f.y_stride = y_stride;
  f.eps = eps, f.dim = int32_t(dim), f.param_type = param_dtype;
  bool done = false;
  const cudaError_t ce =
      launch_rows(f, x_dtype, y_dtype, static_cast<cudaStream_t>(stream), &done);
  if (done || ce != cudaSuccess) return launched("layer_norm", ce);
  WideArgs a{};
  a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.stats = stats;
  a.n_rows = n_rows, a.dim = dim, a.x_stride = x_stride, a.y_stride = y_stride;
  a.eps = eps;
  a.x_type = x_dtype, a.y_type = y_dtype, a.param_type = param_dtype;
  return launched("layer_norm",
                  launch(wide_norm_kernel, dim3(unsigned(n_rows)), kWideThreads, 0,
                         static_cast<cudaStream_t>(stream), true, 1, a));
}

}  // extern "C"
