// Layer norm's backward pass (train_ops.h).
#include "train_norm_grad_rows.h"

using namespace traingb;

namespace {

// ------------------------------------------------------------ rows of any width
constexpr int kWideThreads = 512;

// For rows wider than 12,288 (than 10,752 where x and grad_out are both fp32: two stages of
// the ring and the weight fill a CTA's shared memory there), or than 8,192 where they begin
// differently in each matrix.  dx, one CTA a row; 8192 x 4096 bf16 took 177 us with this and
// the two below, 8192 x 12288 fp32 takes 502, where 8192 x 10752 takes 179 on chip.
__global__ void __launch_bounds__(kWideThreads) wide_dx_kernel(const NormGradArgs a) {
  __shared__ float part[2][kWideThreads / kWarp];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const float mean = a.stats[row], rstd = a.stats[a.n_rows + row];
  by_type(a.x_type, [&](auto X) {
    by_type(a.dy_type, [&](auto Y) {
      by_type(a.param_type, [&](auto P) {
        constexpr int XT = decltype(X)::value, YT = decltype(Y)::value, PT = decltype(P)::value;
        using TX = typename TypeOf<XT>::T;
        using TY = typename TypeOf<YT>::T;
        using TP = typename TypeOf<PT>::T;
        const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
        const TY* dy = static_cast<const TY*>(a.dy) + row * a.dy_stride;
        const TP* weight = static_cast<const TP*>(a.weight);
        float s = 0.f, t = 0.f;
        for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) {
          float g = to_float<YT>(dy[i]);
          if (weight) g *= to_float<PT>(weight[i]);
          s += g;
          t += g * ((to_float<XT>(x[i]) - mean) * rstd);
        }
        const float along1 = cta_sum<kWideThreads>(s, part[0]) / float(a.dim);
        const float alongx = cta_sum<kWideThreads>(t, part[1]) / float(a.dim);
        TX* dx = static_cast<TX*>(a.dx) + row * a.dx_stride;
        for (int64_t i = threadIdx.x; i < a.dim; i += kWideThreads) {
          float g = to_float<YT>(dy[i]);
          if (weight) g *= to_float<PT>(weight[i]);
          const float xhat = (to_float<XT>(x[i]) - mean) * rstd;
          dx[i] = from_float<XT>(rstd * (g - along1 - xhat * alongx));
        }
      });
    });
  });
}

// Partial sums over rows_per_piece rows, a CTA for 32 columns.
constexpr int kSlabWarps = 8;
__global__ void __launch_bounds__(kSlabWarps* kWarp) wide_partial_kernel(const NormGradArgs a) {
  __shared__ float part[2][kSlabWarps][kWarp];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t column = int64_t(blockIdx.x) * kWarp + lane;
  const int64_t first = int64_t(blockIdx.y) * a.rows_per_piece;
  const int64_t end = min(a.n_rows, first + a.rows_per_piece);
  float s = 0.f, t = 0.f;
  if (column < a.dim) {
    by_type(a.x_type, [&](auto X) {
      by_type(a.dy_type, [&](auto Y) {
        constexpr int XT = decltype(X)::value, YT = decltype(Y)::value;
        const auto* x = static_cast<const typename TypeOf<XT>::T*>(a.x) + column;
        const auto* dy = static_cast<const typename TypeOf<YT>::T*>(a.dy) + column;
        for (int64_t r = first + warp; r < end; r += kSlabWarps) {
          const float g = to_float<YT>(dy[r * a.dy_stride]);
          s += g * ((to_float<XT>(x[r * a.x_stride]) - a.stats[r]) * a.stats[a.n_rows + r]);
          t += g;
        }
      });
    });
  }
  part[0][warp][lane] = s, part[1][warp][lane] = t;
  __syncthreads();
  if (warp < 2 && column < a.dim) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSlabWarps; ++w) s += part[warp][w][lane];
    a.partial[(2 * int64_t(blockIdx.y) + warp) * a.dim + column] = s;
  }
}

// --------------------------------------------------------------------- the join
struct JoinArgs {
  const float* partial;
  void* weight_grad;
  void* bias_grad;
  int64_t dim, pieces;
  int32_t type, accumulate;
};

// Adds the pieces of 32 columns in a fixed order.
constexpr int kJoinWarps = 16;
constexpr int kJoinAtOnce = 10;
__global__ void __launch_bounds__(kJoinWarps* kWarp) join_kernel(const JoinArgs a) {
  __shared__ float part[2][kJoinWarps][kWarp];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t column = int64_t(blockIdx.x) * kWarp + lane;
  float s = 0.f, t = 0.f;
  if (column < a.dim) {
    const float* p = a.partial + 2 * warp * a.dim + column;
    // As many on their way together as most sizes have (152 pieces, 16 warps).
    for (int64_t k = warp; k < a.pieces; k += kJoinAtOnce * kJoinWarps) {
      float u[kJoinAtOnce][2];
#pragma unroll
      for (int i = 0; i < kJoinAtOnce; ++i) {
        u[i][0] = u[i][1] = 0.f;
        if (k + i * kJoinWarps < a.pieces) u[i][0] = p[0], u[i][1] = p[a.dim];
        p += 2 * kJoinWarps * a.dim;
      }
#pragma unroll
      for (int i = 0; i < kJoinAtOnce; ++i) s += u[i][0], t += u[i][1];
    }
  }
  part[0][warp][lane] = s, part[1][warp][lane] = t;
  __syncthreads();
  void* out = warp == 0 ? a.weight_grad : a.bias_grad;
  if (warp < 2 && column < a.dim && out) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) s += part[warp][w][lane];
    write_grad(out, a.type, a.accumulate, column, s);
  }
}

// ------------------------------------------------------------------------- plan
constexpr int kSms = 152;
constexpr int kMostPieces = 256;
constexpr int kMostLanes = 512;  // threads a CTA
constexpr int64_t kMostShared = 224 * 1024;  // a CTA's dynamic shared memory

// Sizes whose sums one cluster takes and adds by itself, without a workspace: one launch
// and one allocation less, which from Python take 3 to 7 us.  On the GPU, in a captured
// graph, it is as quick as the pieces or quicker up to some 32,000 elements and 500 rows (64
// x 64 3.4 us and 4.0, 100 x 256 3.8 and 4.5), and loses where its 16 CTAs have more
// rounds: 512 x 256 5.9 and 4.5, 128 x 1024 7.8 and 5.7, 131 x 1000 8.9 and 6.0; 4096 x 9, 8
// rounds of two rows a warp, 7.9 and 3.9.  The limits stand where that comes to what the
// call gains: 262 x 1000 loses 3.8 us, 8192 x 9 7.7, and 26,214 x 5 took 33 us where
// pieces take 7.
bool one_cluster(int64_t n_rows, int64_t dim) {
  return dim <= 1024 && n_rows <= 4096 && n_rows * dim <= (1 << 17);
}

// Pieces that any of the kernels below may write.
int64_t most_pieces(int64_t n_rows, int64_t dim) {
  return one_cluster(n_rows, dim) ? 0 : std::min<int64_t>(kMostPieces, n_rows);
}

// Launches the kernel for rows that stay on chip, if there is one; sets `pieces`.
cudaError_t launch_rows(NormGradArgs& a, cudaStream_t stream, int64_t* pieces) {
  *pieces = 0;
  const int64_t dim = a.dim;
  if (dim > 32768) return cudaSuccess;
  const NormGradKernels& k = a.x_type == TRAIN_BF16   ? norm_grad_kernels_bf16(a.dy_type)
                             : a.x_type == TRAIN_FP16 ? norm_grad_kernels_fp16(a.dy_type)
                                                      : norm_grad_kernels_fp32(a.dy_type);
  const int64_t e = a.x_type == TRAIN_FP32 || a.dy_type == TRAIN_FP32 ? 4 : 8;
  const auto phase = [&](const void* p, int32_t type) {
    return int64_t(reinterpret_cast<uintptr_t>(p) / uintptr_t(size_of(type))) % e;
  };
  const auto go = [&](NormGradKernel kernel, int64_t ctas, int64_t groups, int64_t smem) {
    if (a.joined) {
      // All of its CTAs, those without rows too: they write their share of the sums (1 x 1024
      // takes 5.1 us so, 13.3 with one CTA).
      a.joined = kJoined;
      *pieces = 1;
      smem = std::max(smem, groups * 2 * dim * 4);
      const void* f = reinterpret_cast<const void*>(kernel);
      cudaError_t ce = cudaSuccess;
      if (smem > 40 * 1024)
        ce = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  int(kMostShared));
      if (ce == cudaSuccess)
        ce = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (ce != cudaSuccess) return ce;
      return launch(kernel, dim3(unsigned(a.joined)), int(groups * a.lanes), size_t(smem), stream,
                    true, a.joined, a);
    }
    // A CTA for each row that begins differently, but none without rows.
    ctas = std::min((ctas + a.period - 1) / a.period * a.period, a.n_rows);
    if (ctas < a.period) ctas = std::min<int64_t>(a.n_rows, a.period);
    else ctas = ctas / a.period * a.period;
    smem = std::max(smem, groups * 2 * dim * 4);
    *pieces = ctas;
    if (smem > 40 * 1024) {
      const cudaError_t ce =
          cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
      if (ce != cudaSuccess) return ce;
    }
    return launch(kernel, dim3(unsigned(ctas)), int(groups * a.lanes), size_t(smem), stream, true,
                  1, a);
  };
  a.period = 1;
  const int64_t px = phase(a.x, a.x_type), row = a.x_stride % e;
  const bool alike = px == phase(a.dy, a.dy_type) && row == a.dy_stride % e &&
                     (!a.dx || (px == phase(a.dx, a.x_type) && row == a.dx_stride % e));
  const bool whole = alike && px == 0 && row == 0 && dim % e == 0;
  if (alike && (whole || dim >= 256)) {
    a.phase = int32_t(px), a.row_phase = int32_t(row);
    while (a.period * row % e != 0) a.period *= 2;
    const int64_t units = dim / e;
    int shape = 0;
    int64_t m = 1;  // units a thread
    if (units < kWarp && whole) {
      a.lanes = 1;
      while (a.lanes < units) a.lanes *= 2;
    } else {
      m = (units * e <= 8 * kWarp ? 8 : units * e <= 16 * kMostLanes ? 16 : 24) / e;
      a.lanes = int32_t((units + m * kWarp - 1) / (m * kWarp)) * kWarp;
      shape = m * e == 24 ? 4 : a.lanes > kWarp ? 3 : int(m * e / 8);
    }
    if (a.lanes <= kMostLanes) {
      const int64_t stage = grad_rows(shape == 0 ? 8 : int(m * e)) * m * e * a.lanes *
                            (size_of(a.x_type) + size_of(a.dy_type));
      const int64_t kept = shape == 4 ? m * e * a.lanes * 4 : 0;
      int64_t groups = std::min<int64_t>(kMostLanes / a.lanes, a.lanes > kWarp ? 15 : kMostLanes);
      // Few rows: CTAs of a few rounds each rather than many pieces.
      const int64_t fill = kWarp / std::min<int64_t>(a.lanes, kWarp);  // groups a warp
      const int64_t spread = a.joined ? kJoined : kSms;
      groups = std::min(groups, ((a.n_rows + spread - 1) / spread + fill - 1) / fill * fill);
      while (groups > fill && groups * std::max(2 * stage + kept, 8 * dim) > kMostShared)
        groups -= fill;
      if (groups * std::max(2 * stage + kept, 8 * dim) <= kMostShared) {
        a.stages = int32_t(std::min<int64_t>(4, (kMostShared - groups * kept) / (groups * stage)));
        return go(k.ring[shape], std::min<int64_t>(kSms, (a.n_rows + groups - 1) / groups), groups,
                  groups * (a.stages * stage + kept));
      }
    }
    a.period = 1;
  }
  // Element by element.
  int s = 0;
  while (s < 2 && dim > kGradScalars[s] * kWarp) ++s;
  const int64_t rows = (a.n_rows + kGradScalarRows[s] - 1) / kGradScalarRows[s];
  const int64_t span = kGradScalars[s] * kWarp;
  a.lanes = int32_t((dim + span - 1) / span) * kWarp;
  if (a.lanes > 512 || dim * 8 > kMostShared) return cudaSuccess;
  int64_t groups = std::max<int64_t>(1, std::min<int64_t>(512 / a.lanes, a.lanes > kWarp ? 15 : 16));
  const int64_t spread = a.joined ? kJoined : kSms;
  groups = std::min(groups, (rows + spread - 1) / spread);
  while (groups > 1 && groups * dim * 8 > kMostShared) --groups;
  return go(k.scalar[a.lanes > kWarp ? 3 : s],
            std::min<int64_t>(kSms, (rows + groups - 1) / groups), groups, 0);
}

constexpr int64_t kMaxElements = int64_t(1) << 40;

int check_sizes(int64_t n_rows, int64_t dim) {
  if (n_rows < 0 || dim < 1 || n_rows > kMaxCount || dim > kMaxCount)
    return fail(LAMB_ERR_INVALID, "n_rows must be in [0, 2^31 - 1], dim in [1, 2^31 - 1]");
  if (n_rows > kMaxElements / dim) return fail(LAMB_ERR_INVALID, "n_rows * dim is too large");
  return LAMB_OK;
}

}  // namespace

extern "C" {

LAMB_API int train_layer_norm_grad_workspace(int64_t n_rows, int64_t dim, int64_t* bytes) {
  lambgb::set_last_error("");
  if (!bytes) return fail(LAMB_ERR_INVALID, "bytes is NULL");
  const int rc = check_sizes(n_rows, dim);
  if (rc != LAMB_OK) return rc;
  *bytes = most_pieces(n_rows, dim) * 2 * dim * 4;
  return LAMB_OK;
}

LAMB_API int train_layer_norm_grad(const void* grad_out, int32_t grad_out_dtype,
                                   int64_t grad_out_stride, const void* x, int32_t x_dtype,
                                   int64_t x_stride, int64_t n_rows, int64_t dim,
                                   const void* weight, int32_t weight_dtype, const float* stats,
                                   void* x_grad, int64_t x_grad_stride, void* weight_grad,
                                   void* bias_grad, int32_t param_grad_dtype, int32_t accumulate,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
  lambgb::set_last_error("");
  int rc = check_matrix("grad_out", grad_out, grad_out_dtype, n_rows, dim, grad_out_stride);
  if (rc == LAMB_OK) rc = check_matrix("x", x, x_dtype, n_rows, dim, x_stride);
  if (rc == LAMB_OK && x_grad)
    rc = check_matrix("x_grad", x_grad, x_dtype, n_rows, dim, x_grad_stride);
  if (rc == LAMB_OK) rc = check_sizes(n_rows, dim);
  if (rc == LAMB_OK) rc = check_vector("weight", weight, weight_dtype);
  if (rc == LAMB_OK) rc = check_vector("stats", stats, TRAIN_FP32);
  if (rc == LAMB_OK) rc = check_vector("weight_grad", weight_grad, param_grad_dtype);
  if (rc == LAMB_OK) rc = check_vector("bias_grad", bias_grad, param_grad_dtype);
  if (rc != LAMB_OK) return rc;
  if (accumulate != 0 && accumulate != 1)
    return fail(LAMB_ERR_INVALID, "accumulate must be 0 or 1");
  if (n_rows > 0 && !stats) return fail(LAMB_ERR_INVALID, "stats is NULL");
  const bool params = weight_grad || bias_grad;
  const bool joined = params && n_rows > 0 && one_cluster(n_rows, dim);
  if (params && most_pieces(n_rows, dim) > 0) {
    if (!workspace || workspace_bytes < most_pieces(n_rows, dim) * 2 * dim * 4)
      return fail(LAMB_ERR_INVALID, "workspace is missing or too small");
    if (reinterpret_cast<uintptr_t>(workspace) % 16)
      return fail(LAMB_ERR_ALIGN, "workspace is not 16-byte aligned");
  }
  if (n_rows > 0) {
    const Rows read[] = {rows_of("grad_out", grad_out, grad_out_dtype, n_rows, dim,
                                 grad_out_stride),
                         rows_of("x", x, x_dtype, n_rows, dim, x_stride),
                         rows_of("weight", weight, weight_dtype, 1, dim),
                         rows_of("stats", stats, TRAIN_FP32, 1, 2 * n_rows)};
    const int64_t held = params ? most_pieces(n_rows, dim) * 2 * dim : 0;
    const Rows written[] = {rows_of("x_grad", x_grad, x_dtype, n_rows, dim, x_grad_stride),
                            rows_of("workspace", workspace, TRAIN_FP32, 1, held),
                            rows_of("weight_grad", weight_grad, param_grad_dtype, 1, dim),
                            rows_of("bias_grad", bias_grad, param_grad_dtype, 1, dim)};
    for (int i = 0; i < 4 && rc == LAMB_OK; ++i) {
      for (int k = 0; k < i && rc == LAMB_OK; ++k) rc = check_apart(written[i], written[k]);
      // The parameters' gradients are written when everything has been read.
      if (i < 2)
        for (int k = 0; k < 4 && rc == LAMB_OK; ++k)
          rc = check_apart(written[i], read[k], i == 0 && k < 2);
    }
    if (rc != LAMB_OK) return rc;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  NormGradArgs a{};
  a.dy = grad_out, a.x = x, a.weight = weight, a.stats = stats, a.dx = x_grad;
  a.partial = params && !joined ? static_cast<float*>(workspace) : nullptr;
  a.joined = joined;
  a.weight_grad = weight_grad, a.bias_grad = bias_grad;
  a.grad_type = param_grad_dtype, a.accumulate = accumulate;
  a.n_rows = n_rows, a.dim = dim;
  a.dy_stride = grad_out_stride, a.x_stride = x_stride, a.dx_stride = x_grad_stride;
  a.dy_type = grad_out_dtype, a.x_type = x_dtype, a.param_type = weight_dtype;
  cudaError_t ce = cudaSuccess;
  int64_t pieces = 0;
  if (n_rows > 0 && (params || x_grad)) {
    ce = launch_rows(a, st, &pieces);
    if (ce == cudaSuccess && pieces == 0) {
      a.rows_per_piece = std::max<int64_t>(64, (n_rows + kMostPieces - 1) / kMostPieces);
      pieces = (n_rows + a.rows_per_piece - 1) / a.rows_per_piece;
      // The sums first: dx may take the place of grad_out.
      if (params)
        ce = launch(wide_partial_kernel,
                    dim3(unsigned((dim + kWarp - 1) / kWarp), unsigned(pieces)),
                    kSlabWarps * kWarp, 0, st, true, 1, a);
      if (ce == cudaSuccess && x_grad)
        ce = launch(wide_dx_kernel, dim3(unsigned(n_rows)), kWideThreads, 0, st, true, 1, a);
    }
  }
  if (ce == cudaSuccess && params && !joined && !(n_rows == 0 && accumulate)) {
    JoinArgs j{};
    j.partial = a.partial, j.weight_grad = weight_grad, j.bias_grad = bias_grad;
    j.dim = dim, j.pieces = pieces;
    j.type = param_grad_dtype, j.accumulate = accumulate;
    ce = launch(join_kernel, dim3(unsigned((dim + kWarp - 1) / kWarp)), kJoinWarps * kWarp, 0,
                st, true, 1, j);
  }
  return launched("layer_norm_grad", ce);
}

}  // extern "C"
