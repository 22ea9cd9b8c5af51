// The loss against a teacher's top logits and the true labels, and its gradient
// (train_ops.h).
#include <mutex>

#include "train_distill_rows.h"

using namespace traingb;

namespace {

constexpr int kThreads = 512;

// The gradient of rows that no cluster holds (above 1.6 MB), and vocabularies of less than
// a unit.  One CTA a row, which it reads three times (from L1 or L2 after the first): 8192
// x 32000 bf16 took 572 us this way.
__global__ void __launch_bounds__(kThreads) row_kernel(const DistillArgs a) {
  // The row's entries: the teacher's tokens and behind them the label.
  __shared__ int32_t id[kMaxTop + 1];
  __shared__ float coef[kMaxTop + 1];  // what the entry takes off its gradient
  __shared__ float zed[kMaxTop + 1];   // the student's logit there
  __shared__ float part[4][kThreads / kWarp];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const bool soft = a.top_k > 0 && a.soft_weight != 0.f;
  int64_t label = -1;
  bool live = true;
  if (a.labels) {
    label = read_id(a.labels, row, a.labels64);
    live = label != a.ignore_id && label >= 0 && label < a.vocab;
  }
  const bool hard = a.labels && a.hard_weight != 0.f;
  float up = a.scale;
  if (a.grad && a.row_grad) up *= a.row_grad[row];
  by_type(a.type, [&](auto Z) {
    constexpr int ZT = decltype(Z)::value;
    using TZ = typename TypeOf<ZT>::T;
    const TZ* z = static_cast<const TZ*>(a.logits) + row * a.stride;
    // The teacher's distribution.
    const int top_k = soft && live ? a.top_k : 0;
    float best = -INFINITY;
    for (int k = tid; k < top_k; k += kThreads) {
      const int64_t i = read_id(a.top_ids, row * a.ids_stride + k, a.ids64);
      float t = 0.f;
      by_type(a.top_type, [&](auto T) {
        constexpr int TT = decltype(T)::value;
        t = to_float<TT>(static_cast<const typename TypeOf<TT>::T*>(
            a.top_logits)[row * a.top_stride + k]);
      });
      const bool valid = i >= 0 && i < a.vocab && t != -INFINITY;
      id[k] = valid ? int32_t(i) : -1;
      coef[k] = t;
      if (valid) {
        zed[k] = to_float<ZT>(z[i]);
        best = t != t ? t : fmaxf(best, t);
      }
    }
    best = cta_max<kThreads>(best, part[0]);
    float size = 0.f;
    for (int k = tid; k < top_k; k += kThreads)
      if (id[k] >= 0) size += exp2f((coef[k] - best) * (a.inv_temperature * kLog2e));
    size = cta_sum<kThreads>(size, part[1]);
    const bool any = size != 0.f;  // NaN too
    // The student's.
    const bool work = live && (any || hard) && (a.loss || up != 0.f);
    float top = -INFINITY, soft_sum = 0.f, hard_sum = 0.f;
    if (work) {
      for (int64_t j = tid; j < a.vocab; j += kThreads) top = fmaxf(top, to_float<ZT>(z[j]));
    }
    top = cta_max<kThreads>(top, part[2]);
    const float c = a.inv_temperature * kLog2e;
    if (work) {
      for (int64_t j = tid; j < a.vocab; j += kThreads) {
        const float d = to_float<ZT>(z[j]) - top;
        if (any) soft_sum += exp2f(d * c);
        if (hard) hard_sum += exp2f(d * kLog2e);
      }
    }
    soft_sum = cta_sum<kThreads>(soft_sum, part[0]);
    hard_sum = cta_sum<kThreads>(hard_sum, part[3]);
    // The loss, and what each entry takes off the gradient.
    float terms = 0.f;
    const float logs = logf(soft_sum) - logf(size);
    for (int k = tid; k < top_k; k += kThreads) {
      if (id[k] < 0) {
        coef[k] = 0.f;
        continue;
      }
      const float d = coef[k] - best, p = exp2f(d * c) / size;
      terms += soft_term(a, p, coef[k], best, zed[k], top, logs);
      coef[k] = a.soft_weight * a.temperature * p;
    }
    const bool hits = work && hard;
    if (tid == 0) {
      id[top_k] = hits ? int32_t(label) : -1;
      coef[top_k] = a.hard_weight;
      zed[top_k] = hits ? to_float<ZT>(z[label]) : 0.f;
    }
    terms = cta_sum<kThreads>(terms, part[1]);
    if (a.loss && tid == 0) {
      float loss = 0.f;
      // Without a distribution (soft_sum is NaN) a masked token's term means nothing.
      if (soft_sum != soft_sum) terms = soft_sum;
      if (work && any) loss = terms;
      if (hits) loss += hard_term(a, hard_sum, zed[top_k], top);
      a.loss[row] = loss;
    }
    if (!a.grad) return;
    by_type(a.grad_type, [&](auto G) {
      constexpr int GT = decltype(G)::value;
      using TG = typename TypeOf<GT>::T;
      TG* grad = static_cast<TG*>(a.grad) + row * a.grad_stride;
      const bool zero = !work || up == 0.f;
      const float qs = any ? a.soft_weight * a.temperature / soft_sum : 0.f;
      const float ss = hard ? a.hard_weight / hard_sum : 0.f;
      const auto smooth = [&](float v) {
        const float d = v - top;
        float g = 0.f;
        if (any) g += qs * exp2f(d * c);
        if (hard) g += ss * exp2f(d * kLog2e);
        return g;
      };
      for (int64_t j = tid; j < a.vocab; j += kThreads)
        grad[j] = zero ? TG(0) : from_float<GT>(up * smooth(to_float<ZT>(z[j])));
      if (zero) return;
      __syncthreads();
      // Again where the entries are: all of a token's are taken off together.
      for (int k = tid; k <= top_k; k += kThreads) {
        if (id[k] < 0) continue;
        float off = 0.f;
        for (int o = 0; o <= top_k; ++o)
          if (id[o] == id[k]) off += coef[o];
        grad[id[k]] = from_float<GT>(up * (smooth(zed[k]) - off));
      }
    });
  });
}

constexpr int kSms = 152;
constexpr int64_t kMostShared = 168 * 1024;  // a CTA's dynamic shared memory
// What a CTA holds of a row: up to 70 KB or so there are three of them an SM, up to this
// two.  Longer rows go to clusters of CTAs: 4096 x 46000 bf16 takes 146 us with one CTA a
// row and 167 with two, 4096 x 36000 129 and 148.
constexpr int64_t kSliceBytes = 104 * 1024;

// Clusters of a kernel that the device holds at once.  They lie within the device's
// groups of SMs, so there may be fewer than its SMs have room for, and one more would
// wait for the others' last row: 1021 x 131,071 fp16 took 167 us with 114 clusters and 128
// with the 110 that fit.  CUDA is asked once for each shape of a launch.
int64_t clusters_at_once(const void* kernel, int threads, int64_t smem, int ctas) {
  struct Known {
    const void* kernel;
    int device, threads, ctas, clusters;
    int64_t smem;
  };
  static std::mutex lock;
  static Known known[64];
  int device = 0;
  cudaGetDevice(&device);
  const size_t at = (reinterpret_cast<uintptr_t>(kernel) / 64 + size_t(smem) / 16 * 31 +
                     size_t(threads + ctas + device)) % 64;
  std::lock_guard<std::mutex> hold(lock);
  Known& k = known[at];
  if (k.kernel == kernel && k.device == device && k.threads == threads && k.ctas == ctas &&
      k.smem == smem)
    return k.clusters;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) clusters = 1;
  k = Known{kernel, device, threads, ctas, std::max(1, clusters), smem};
  return k.clusters;
}

// Whether rows of so many units last for the stages that are on their way.
bool ring_takes(int64_t units, int threads) {
  return units >= int64_t(kRingStages - 1) * kAtOnce * threads;
}

// Launches the kernel for rows that stay in shared memory or pass through it, if there is
// one; sets `done`.
cudaError_t launch_rows(DistillArgs& a, cudaStream_t stream, bool* done) {
  *done = false;
  const int e = 16 / size_of(a.type);
  const int64_t units = a.vocab / e;
  const auto phase = [&](const void* p, int32_t type) {
    return int32_t(reinterpret_cast<uintptr_t>(p) / uintptr_t(size_of(type)) % uintptr_t(e));
  };
  a.phase = phase(a.logits, a.type), a.row_phase = int32_t(a.stride % e);
  a.whole = !a.grad || (phase(a.grad, a.grad_type) == a.phase && a.grad_stride % e == a.row_phase);
  // Two softmaxes only where the terms are at two temperatures.
  const bool soft = a.top_k > 0 && a.soft_weight != 0.f, hard = a.labels && a.hard_weight != 0.f;
  const int terms = !soft || !hard || a.temperature == 1.f ? kOne
                    : a.temperature == 2.f                 ? kSquares
                                                           : kTwo;
  const DistillKernels& k = a.type == TRAIN_BF16   ? distill_kernels_bf16()
                            : a.type == TRAIN_FP16 ? distill_kernels_fp16()
                                                   : distill_kernels_fp32();
  // Four to eight buckets an entry, of two kinds: one entry in a hundred finds both taken.
  int64_t lists = 2 * 3 * 4 * int64_t((a.top_k + 4) / 4 * 4);
  if (a.grad) {
    a.bucket_bits = 2;
    while ((1 << a.bucket_bits) < 4 * (a.top_k + 1)) ++a.bucket_bits;
    lists += 2 * int64_t((a.top_k + 4) / 4 * 4) + 2 * 2 * (int64_t(1) << a.bucket_bits);
  }
  a.ctas = 1;
  while (units * 16 > a.ctas * kSliceBytes) a.ctas *= 2;
  int64_t clusters = 0;  // none holds a row
  if (a.ctas <= kMostCtas && units > 0) {
    a.slice = int32_t((units + a.ctas - 1) / a.ctas);
    // At least 8 units a thread (16384 x 4096 bf16 takes 72 us so, 103 with 4 and 80 with 16)
    // but at most 4 entries (6263 x 2688 fp16 with 179: 38 us so, 49 with 6 and 50 with 2).
    int threads = kDistillThreads;
    while (threads > kWarp && a.slice < threads * 8 && a.top_k <= threads * 2) threads /= 2;
    const int64_t smem = int64_t(a.slice) * 16 + lists;
    const DistillKernel kernel = a.grad ? k.grad[a.grad_type][terms] : k.loss[terms];
    const void* f = reinterpret_cast<const void*>(kernel);
    cudaError_t ce = cudaSuccess;
    if (smem > 32 * 1024)
      ce = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
    if (ce == cudaSuccess && a.ctas > 8)
      ce = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (ce != cudaSuccess) return ce;
    const int64_t resident = std::max<int64_t>(
        1, std::min<int64_t>(std::min(24, 3 * kDistillThreads / threads),
                             (227 * 1024) / (smem + 6 * 1024)));
    clusters = resident * kSms;
    if (a.ctas > 1)
      clusters = std::min(clusters / a.ctas, clusters_at_once(f, threads, smem, a.ctas));
    clusters = std::max<int64_t>(1, clusters);
    if (a.grad || a.n_rows <= clusters || !ring_takes(units, kWarp)) {
      *done = true;
      return launch(kernel, dim3(unsigned(std::min(a.n_rows, clusters) * a.ctas)), threads,
                    size_t(smem), stream, true, a.ctas, a);
    }
  }
  if (a.grad || !ring_takes(units, kWarp)) return cudaSuccess;
  // More rows than are held at once pass through the ring, as do the longest: 608 x 32000
  // bf16 takes 11.0 us so and 14.5 held, 304 rows 8.2 and 8.1, 152 rows 7.2 and 6.3; 152 x
  // 131,072 13.5 and 16.1, 64 rows 12.6 and 8.6.
  // Up to 64 units a thread (8192 x 12800 bf16 takes 47 us with 32 threads and 52 with 64, 4096
  // x 50,000 69 with 128 and 76 with 64), or more threads while all rows are there at once.
  const int64_t room = int64_t(kSms) * kRingCtas * kRingThreads;
  int threads = kWarp;
  while (threads < kRingThreads && ring_takes(units, 2 * threads) &&
         (units > 64 * threads || a.n_rows * 2 * threads <= room))
    threads *= 2;
  const int64_t smem = threads / kWarp * kRingBytes + lists;
  const int64_t resident = std::max<int64_t>(
      1, std::min<int64_t>(kRingCtas * kRingThreads / threads, (227 * 1024) / (smem + 2 * 1024)));
  const DistillKernel kernel = k.ring[terms];
  if (smem > 32 * 1024) {
    const cudaError_t ce =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
    if (ce != cudaSuccess) return ce;
  }
  a.ctas = 1, a.slice = int32_t(units);
  *done = true;
  return launch(kernel, dim3(unsigned(std::min(a.n_rows, resident * kSms))), threads,
                size_t(smem), stream, true, 1, a);
}

int check_ids(const char* name, const void* p, int32_t dtype, int64_t n) {
  if (dtype != TRAIN_INT32 && dtype != TRAIN_INT64)
    return fail(LAMB_ERR_INVALID, std::string(name) + ": unknown type");
  if (n == 0) return LAMB_OK;
  if (!p) return fail(LAMB_ERR_INVALID, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % (dtype == TRAIN_INT64 ? 8u : 4u))
    return fail(LAMB_ERR_ALIGN, std::string(name) + " is not aligned to its type");
  return LAMB_OK;
}

}  // namespace

extern "C" {

LAMB_API int train_distill(const void* logits, int32_t logits_dtype, int64_t logits_stride,
                           int64_t n_rows, int64_t vocab, const void* top_ids,
                           int32_t top_ids_dtype, int64_t top_ids_stride, const void* top_logits,
                           int32_t top_logits_dtype, int64_t top_logits_stride, int64_t top_k,
                           const void* labels, int32_t labels_dtype, int64_t ignore_id,
                           float temperature, float soft_weight, float hard_weight, float* loss,
                           const float* row_grad, float scale, void* grad, int32_t grad_dtype,
                           int64_t grad_stride, void* stream) {
  lambgb::set_last_error("");
  int rc = check_matrix("logits", logits, logits_dtype, n_rows, vocab, logits_stride);
  if (rc == LAMB_OK && grad)
    rc = check_matrix("grad", grad, grad_dtype, n_rows, vocab, grad_stride);
  if (rc != LAMB_OK) return rc;
  if (vocab == 0) return fail(LAMB_ERR_INVALID, "vocab must be at least 1");
  if (top_k < 0 || top_k > kMaxTop)
    return fail(LAMB_ERR_INVALID, "top_k must be in [0, " + std::to_string(kMaxTop) + "]");
  if (top_k > 0) {
    rc = check_matrix("top_logits", top_logits, top_logits_dtype, n_rows, top_k,
                      top_logits_stride);
    if (rc == LAMB_OK)
      rc = check_ids("top_ids", top_ids, top_ids_dtype, n_rows);
    if (rc == LAMB_OK && top_ids_stride < top_k)
      rc = fail(LAMB_ERR_INVALID, "top_ids: stride is less than top_k");
  }
  if (rc == LAMB_OK && labels) rc = check_ids("labels", labels, labels_dtype, n_rows);
  if (rc == LAMB_OK) rc = check_vector("loss", loss, TRAIN_FP32);
  if (rc == LAMB_OK) rc = check_vector("row_grad", row_grad, TRAIN_FP32);
  if (rc != LAMB_OK) return rc;
  const float inv = 1.f / temperature;
  if (!(temperature > 0.f && temperature <= FLT_MAX && inv > 0.f && inv <= FLT_MAX))
    return fail(LAMB_ERR_INVALID, "temperature and its reciprocal must be finite and > 0");
  if (!(fabsf(soft_weight) <= FLT_MAX && fabsf(hard_weight) <= FLT_MAX))
    return fail(LAMB_ERR_INVALID, "soft_weight and hard_weight must be finite");
  // What scales the exponents and the teacher's shares.
  if (top_k > 0 && soft_weight != 0.f &&
      !(inv * kLog2e <= FLT_MAX && fabsf(soft_weight * temperature) <= FLT_MAX))
    return fail(LAMB_ERR_INVALID,
                "log2(e) / temperature and soft_weight * temperature must be finite");
  if (hard_weight != 0.f && !labels && n_rows > 0)
    return fail(LAMB_ERR_INVALID, "hard_weight needs labels");
  if (n_rows == 0 || (!loss && !grad)) return LAMB_OK;
  const auto ids_of = [](const char* name, const void* p, int32_t type, int64_t n, int64_t dim,
                         int64_t stride) {
    return Rows{name, p, n, dim, stride, type == TRAIN_INT64 ? 8 : 4, -1};
  };
  const int64_t entries = soft_weight != 0.f ? top_k : 0;
  const Rows read[] = {
      rows_of("logits", logits, logits_dtype, n_rows, vocab, logits_stride),
      ids_of("top_ids", top_ids, top_ids_dtype, n_rows, entries, top_ids_stride),
      rows_of("top_logits", top_logits, top_logits_dtype, n_rows, entries, top_logits_stride),
      ids_of("labels", labels, labels_dtype, 1, n_rows, 0),
      rows_of("row_grad", row_grad, TRAIN_FP32, 1, n_rows)};
  // A row's loss is written behind the last reading of its row_grad.
  const Rows losses = rows_of("loss", loss, TRAIN_FP32, 1, n_rows);
  const Rows slopes = rows_of("grad", grad, grad_dtype, n_rows, vocab, grad_stride);
  rc = check_apart(slopes, losses);
  for (int k = 0; k < 5 && rc == LAMB_OK; ++k) {
    rc = check_apart(losses, read[k], k == 4);
    if (rc == LAMB_OK) rc = check_apart(slopes, read[k], k == 0);
  }
  if (rc != LAMB_OK) return rc;
  DistillArgs a{};
  a.logits = logits, a.top_ids = top_ids, a.top_logits = top_logits, a.labels = labels;
  a.row_grad = row_grad, a.loss = loss, a.grad = grad;
  a.stride = logits_stride, a.ids_stride = top_ids_stride, a.top_stride = top_logits_stride;
  a.grad_stride = grad_stride, a.ignore_id = ignore_id;
  a.vocab = int32_t(vocab), a.top_k = int32_t(top_k);
  a.inv_temperature = inv, a.temperature = temperature;
  a.soft_weight = soft_weight, a.hard_weight = hard_weight, a.scale = scale;
  a.type = logits_dtype, a.grad_type = grad_dtype;
  a.ids64 = top_ids_dtype == TRAIN_INT64, a.labels64 = labels_dtype == TRAIN_INT64;
  a.top_type = top_logits_dtype;
  a.n_rows = n_rows;
  bool done = false;
  const cudaError_t ce = launch_rows(a, static_cast<cudaStream_t>(stream), &done);
  if (done || ce != cudaSuccess) return launched("distill", ce);
  return launched("distill", launch(row_kernel, dim3(unsigned(n_rows)), kThreads, 0,
                                    static_cast<cudaStream_t>(stream), true, 1, a));
}

}  // extern "C"
