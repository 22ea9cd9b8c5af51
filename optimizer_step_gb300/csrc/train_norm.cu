// Layer norm and its backward pass (train_ops.h).
#include "train_norm.h"

using namespace traingb;

namespace {

// ------------------------------------------------------------ rows of any width
// One CTA a row, which it reads three times (from L1 or L2 after the first).
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
