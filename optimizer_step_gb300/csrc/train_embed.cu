// The embedding lookup with scaling (train_ops.h).
#include "train_internal.h"

using namespace traingb;

namespace {

constexpr int kThreads = 256;

struct EmbedArgs {
  const void* table;
  const void* ids;
  void* out;
  int64_t n_rows, table_stride, n_ids, first_row, out_stride;
  uint32_t units;     // of VEC elements a row
  uint32_t segments;  // of 32 M units a row
  uint32_t warps;     // with work
  float scale;
  int32_t ids64;
};

// A warp takes R rows of the output and M times 32 units of VEC elements of
// each: it reads the ids, then the units, all on their way together, and
// writes them.  R is 1 where a row has more than 32 units.  A warp has one
// piece of work and the pieces follow the order of the output, so the writes
// run through memory in order; on GB300 a copy runs at 7.1 TB/s this way and at
// 6.5 with a persistent grid.
template <int IN, int OUT, int VEC, int R, int M>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedArgs a) {
  using TI = typename TypeOf<IN>::T;
  using TO = typename TypeOf<OUT>::T;
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (kThreads / kWarp) + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (warp >= a.warps) return;
  const uint32_t group = warp / a.segments;
  const uint32_t unit0 = (warp - group * a.segments) * (kWarp * M) + lane;
  const int64_t row0 = int64_t(group) * R;
  int64_t source = -1;  // row of the table
  if (lane < R && row0 + lane < a.n_ids)
    source = a.ids64
                 ? row_of(static_cast<const int64_t*>(a.ids)[row0 + lane], a.first_row, a.n_rows)
                 : row_of(static_cast<const int32_t*>(a.ids)[row0 + lane], a.first_row, a.n_rows);
  Pack<IN, VEC> x[R][M];
  bool held[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = __shfl_sync(kAll, source, r);
    held[r] = row >= 0;
    const TI* p = static_cast<const TI*>(a.table) + row * a.table_stride + int64_t(unit0) * VEC;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (held[r] && unit0 + m * kWarp < a.units) x[r][m].load(p + m * (kWarp * VEC));
      else x[r][m].clear();
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (row0 + r >= a.n_ids) break;
    TO* p = static_cast<TO*>(a.out) + (row0 + r) * a.out_stride + int64_t(unit0) * VEC;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (unit0 + m * kWarp >= a.units) break;
      Pack<OUT, VEC> y;
#pragma unroll
      for (int i = 0; i < VEC; ++i) y.set(i, held[r] ? a.scale * x[r][m].get(i) : 0.0f);
      y.store(p + m * (kWarp * VEC));
    }
  }
}

// embed_kernel by the two types, the width of a unit, and whether a row has
// more than 32 units.
using EmbedKernel = void (*)(EmbedArgs);
#define EMBED_WIDTHS(in, out)                                              \
  {{embed_kernel<in, out, 1, 8, 1>, embed_kernel<in, out, 1, 1, 8>},       \
   {embed_kernel<in, out, 2, 8, 1>, embed_kernel<in, out, 2, 1, 8>},       \
   {embed_kernel<in, out, 4, 4, 1>, embed_kernel<in, out, 4, 1, 4>},       \
   {embed_kernel<in, out, 8, 4, 1>, embed_kernel<in, out, 8, 1, 4>}}
#define EMBED_TYPES(in) \
  {EMBED_WIDTHS(in, TRAIN_BF16), EMBED_WIDTHS(in, TRAIN_FP16), EMBED_WIDTHS(in, TRAIN_FP32)}
const EmbedKernel embed_kernels[3][3][4][2] = {EMBED_TYPES(TRAIN_BF16), EMBED_TYPES(TRAIN_FP16),
                                               EMBED_TYPES(TRAIN_FP32)};
const int kUnitWidth[4] = {1, 2, 4, 8};
const int kUnitsPerLane[4] = {8, 8, 4, 4};

// The widest unit that every row of both matrices is whole pieces of, each
// aligned to its size or to 16 bytes: 0, 1, 2, 3 for 1, 2, 4, 8 elements.
int unit_width(int64_t dim, const void* p, int32_t p_type, int64_t p_stride, const void* q,
               int32_t q_type, int64_t q_stride) {
  const auto fits = [&](const void* x, int32_t type, int64_t stride, int v) {
    const int bytes = v * size_of(type) < 16 ? v * size_of(type) : 16;
    return reinterpret_cast<uintptr_t>(x) % uintptr_t(bytes) == 0 &&
           stride * size_of(type) % bytes == 0;
  };
  int w = 3;
  while (w > 0 && (dim % kUnitWidth[w] != 0 || !fits(p, p_type, p_stride, kUnitWidth[w]) ||
                   !fits(q, q_type, q_stride, kUnitWidth[w])))
    --w;
  return w;
}

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
  if (n_rows == 0) table = out;  // nothing is read
  const int w = unit_width(dim, table, table_dtype, table_stride, out, out_dtype, out_stride);
  EmbedArgs a{};
  a.table = table;
  a.ids = ids;
  a.out = out;
  a.n_rows = n_rows;
  a.table_stride = table_stride;
  a.n_ids = n_ids;
  a.first_row = first_row;
  a.out_stride = out_stride;
  a.units = uint32_t(dim / kUnitWidth[w]);
  a.scale = scale;
  a.ids64 = ids_dtype == TRAIN_INT64;
  const int per_lane = kUnitsPerLane[w];
  const bool wide = a.units > kWarp;
  a.segments = wide ? uint32_t((int64_t(a.units) + kWarp * per_lane - 1) / (kWarp * per_lane)) : 1;
  const int64_t groups = wide ? n_ids : (n_ids + per_lane - 1) / per_lane;
  if (groups > kMaxCount / int64_t(a.segments))
    return fail(LAMB_ERR_INVALID, "n_ids * dim is too large");
  a.warps = uint32_t(groups * a.segments);
  const unsigned ctas = unsigned((int64_t(a.warps) * kWarp + kThreads - 1) / kThreads);
  const cudaError_t ce =
      launch(embed_kernels[table_dtype][out_dtype][w][wide ? 1 : 0], dim3(ctas), kThreads, 0,
             static_cast<cudaStream_t>(stream), true, 1, a);
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string("embed: ") + cudaGetErrorString(ce));
}

}  // extern "C"
