// The embedding lookup with scaling and its gradient (train_ops.h).
#include <cmath>
#include <string>

#include "lamb_internal.h"
#include "train_internal.h"

using namespace traingb;

namespace {

constexpr int kThreads = 256;

struct EmbedArgs {
  const void* table;
  const void* ids;
  void* out;
  int64_t n_rows, dim, table_stride, n_ids, first_row, out_stride;
  float scale;
};

// Row of the table (or of its gradient) that a token names, or -1.
template <class ID>
__device__ __forceinline__ int64_t row_of(ID id, int64_t first_row, int64_t n_rows) {
  const uint64_t r = uint64_t(int64_t(id)) - uint64_t(first_row);
  return r < uint64_t(n_rows) ? int64_t(r) : -1;
}

// One CTA per token, an element a thread.
template <int IN, int OUT, class ID>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a) {
  using TI = typename TypeOf<IN>::T;
  using TO = typename TypeOf<OUT>::T;
  for (int64_t i = blockIdx.x; i < a.n_ids; i += gridDim.x) {
    const int64_t row = row_of(static_cast<const ID*>(a.ids)[i], a.first_row, a.n_rows);
    const TI* src = static_cast<const TI*>(a.table) + row * a.table_stride;
    TO* dst = static_cast<TO*>(a.out) + i * a.out_stride;
    for (int64_t d = threadIdx.x; d < a.dim; d += kThreads)
      dst[d] = row < 0 ? from_float<OUT>(0.0f) : from_float<OUT>(a.scale * to_float<IN>(src[d]));
  }
}

struct GradArgs {
  const void* dy;
  const void* ids;
  void* grad;
  int64_t dy_stride, n_ids, first_row, padding, n_rows, dim, grad_stride;
  float scale;
  int accumulate;
};

// One CTA per row of the table and 256 columns: it walks the ids 256 at a time
// and adds the rows of its token in ascending order.
template <int IN, int OUT, class ID>
__global__ void __launch_bounds__(kThreads) embed_grad_kernel(GradArgs a) {
  using TI = typename TypeOf<IN>::T;
  using TO = typename TypeOf<OUT>::T;
  __shared__ unsigned char hit[kThreads];
  const int64_t d = int64_t(blockIdx.y) * kThreads + threadIdx.x;
  for (int64_t v = blockIdx.x; v < a.n_rows; v += gridDim.x) {
    float acc = 0.0f;
    int any = 0;
    for (int64_t i0 = 0; i0 < a.n_ids; i0 += kThreads) {
      const int64_t i = i0 + threadIdx.x;
      int mine = 0;
      if (i < a.n_ids) {
        const ID id = static_cast<const ID*>(a.ids)[i];
        mine = row_of(id, a.first_row, a.n_rows) == v && int64_t(id) != a.padding;
      }
      hit[threadIdx.x] = (unsigned char)mine;
      if (__syncthreads_or(mine)) {
        any = 1;
        for (int k = 0; k < kThreads; ++k)
          if (hit[k] && d < a.dim)
            acc += to_float<IN>(static_cast<const TI*>(a.dy)[(i0 + k) * a.dy_stride + d]);
      }
      __syncthreads();
    }
    if (d >= a.dim || (a.accumulate && !any)) continue;
    TO* g = static_cast<TO*>(a.grad) + v * a.grad_stride + d;
    const float old = a.accumulate ? to_float<OUT>(*g) : 0.0f;
    *g = from_float<OUT>(fmaf(a.scale, acc, old));
  }
}

int fail(int code, const std::string& msg) {
  lambgb::set_last_error(msg);
  return code;
}

int launched(const char* what) {
  const cudaError_t ce = cudaGetLastError();
  if (ce == cudaSuccess) return LAMB_OK;
  return fail(LAMB_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(ce));
}

constexpr int64_t kMaxCount = 0x7fffffff;

// Checks one matrix; LAMB_OK or the error.
int check_matrix(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t dim,
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

int check_ids(const void* ids, int32_t ids_dtype, int64_t n_ids, int64_t first_row) {
  if (ids_dtype != TRAIN_INT32 && ids_dtype != TRAIN_INT64)
    return fail(LAMB_ERR_INVALID, "ids: unknown type");
  if (n_ids < 0 || n_ids > kMaxCount)
    return fail(LAMB_ERR_INVALID, "n_ids must be in [0, 2^31 - 1]");
  if (first_row < 0) return fail(LAMB_ERR_INVALID, "first_row must be >= 0");
  if (n_ids == 0) return LAMB_OK;
  if (!ids) return fail(LAMB_ERR_INVALID, "ids is NULL");
  if (reinterpret_cast<uintptr_t>(ids) % (ids_dtype == TRAIN_INT64 ? 8u : 4u))
    return fail(LAMB_ERR_ALIGN, "ids is not aligned to its type");
  return LAMB_OK;
}

// KERNEL<input type, output type, id type> for types known at run time.
#define PICK_ID(KERNEL, in, out) {KERNEL<in, out, int32_t>, KERNEL<in, out, int64_t>}
#define PICK_OUT(KERNEL, in)                                           \
  {PICK_ID(KERNEL, in, TRAIN_BF16), PICK_ID(KERNEL, in, TRAIN_FP16), \
   PICK_ID(KERNEL, in, TRAIN_FP32)}
#define PICK(KERNEL) \
  {PICK_OUT(KERNEL, TRAIN_BF16), PICK_OUT(KERNEL, TRAIN_FP16), PICK_OUT(KERNEL, TRAIN_FP32)}

void (*const embed_kernels[3][3][2])(EmbedArgs) = PICK(embed_kernel);
void (*const embed_grad_kernels[3][3][2])(GradArgs) = PICK(embed_grad_kernel);

}  // namespace

extern "C" {

LAMB_API int train_embed(const void* table, int32_t table_dtype, int64_t n_rows, int64_t dim,
                         int64_t table_stride, const void* ids, int32_t ids_dtype,
                         int64_t n_ids, int64_t first_row, float scale, void* out,
                         int32_t out_dtype, int64_t out_stride, void* stream) {
  lambgb::set_last_error("");
  int rc = check_matrix("table", table, table_dtype, n_rows, dim, table_stride);
  if (rc == LAMB_OK) rc = check_ids(ids, ids_dtype, n_ids, first_row);
  if (rc == LAMB_OK) rc = check_matrix("out", out, out_dtype, n_ids, dim, out_stride);
  if (rc != LAMB_OK) return rc;
  if (n_ids == 0 || dim == 0) return LAMB_OK;
  const EmbedArgs a{table, ids, out, n_rows, dim, table_stride, n_ids, first_row, out_stride,
                    scale};
  const unsigned grid = unsigned(n_ids);
  embed_kernels[table_dtype][out_dtype][ids_dtype]<<<grid, kThreads, 0,
                                                     static_cast<cudaStream_t>(stream)>>>(a);
  return launched("embed kernel");
}

LAMB_API int train_embed_grad_workspace(int64_t n_ids, int64_t n_rows, int64_t dim,
                                        int64_t* bytes) {
  lambgb::set_last_error("");
  if (!bytes) return fail(LAMB_ERR_INVALID, "bytes is NULL");
  if (n_ids < 0 || n_rows < 0 || dim < 0 || n_ids > kMaxCount || n_rows > kMaxCount ||
      dim > kMaxCount)
    return fail(LAMB_ERR_INVALID, "sizes must be in [0, 2^31 - 1]");
  *bytes = 0;
  return LAMB_OK;
}

LAMB_API int train_embed_grad(const void* grad_out, int32_t grad_out_dtype,
                              int64_t grad_out_stride, const void* ids, int32_t ids_dtype,
                              int64_t n_ids, int64_t first_row, int64_t padding_id, float scale,
                              int32_t accumulate, void* grad, int32_t grad_dtype,
                              int64_t n_rows, int64_t dim, int64_t grad_stride, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  lambgb::set_last_error("");
  int rc = check_ids(ids, ids_dtype, n_ids, first_row);
  if (rc == LAMB_OK)
    rc = check_matrix("grad_out", grad_out, grad_out_dtype, n_ids, dim, grad_out_stride);
  if (rc == LAMB_OK) rc = check_matrix("grad", grad, grad_dtype, n_rows, dim, grad_stride);
  if (rc != LAMB_OK) return rc;
  if (accumulate != 0 && accumulate != 1)
    return fail(LAMB_ERR_INVALID, "accumulate must be 0 or 1");
  int64_t need = 0;
  rc = train_embed_grad_workspace(n_ids, n_rows, dim, &need);
  if (rc != LAMB_OK) return rc;
  if (workspace_bytes < need || (need > 0 && !workspace))
    return fail(LAMB_ERR_INVALID, "workspace: " + std::to_string(need) + " bytes are needed");
  if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 16)
    return fail(LAMB_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (n_rows == 0 || dim == 0 || (accumulate && n_ids == 0)) return LAMB_OK;
  const GradArgs a{grad_out, ids, grad, grad_out_stride, n_ids, first_row,
                   padding_id, n_rows, dim, grad_stride, scale, accumulate};
  const int64_t slabs = (dim + kThreads - 1) / kThreads;
  if (slabs > 65535) return fail(LAMB_ERR_INVALID, "dim is too large");
  const dim3 grid{unsigned(n_rows), unsigned(slabs)};
  embed_grad_kernels[grad_out_dtype][grad_dtype][ids_dtype]<<<
      grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched("embed_grad kernel");
}

}  // extern "C"
