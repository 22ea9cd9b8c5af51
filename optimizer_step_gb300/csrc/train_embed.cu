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
  uint32_t shift;     // NARROW: 2^shift lanes a row
  float scale;
  int32_t ids64;
};

// A warp takes some rows of the output and a part of each: it reads the ids,
// then the units of VEC elements, all on their way together, and writes them.
// NARROW (rows of at most 32 units): R times as many rows as fit into 32 lanes.
// Else R rows and M times 32 units of each.  A warp has one piece of work and
// the pieces follow the order of the output, so the writes run through memory
// in order; on GB300 a copy runs at 7.1 TB/s this way and at 6.5 with a
// persistent grid.  Memory bounds it: 8192 bf16 rows of width 4096 take 16 us, 5.8
// TB/s over the table's distinct rows and the output; 50,021 rows of width 1023
// from fp32 to bf16, element by element, 29 us, 5.3 TB/s.
template <int IN, int OUT, int VEC, int R, int M, bool NARROW>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedArgs a) {
  using TI = typename TypeOf<IN>::T;
  using TO = typename TypeOf<OUT>::T;
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (kThreads / kWarp) + (threadIdx.x >> 5);
  pdl_wait();
  if (warp >= a.warps) return;
  // This lane's first row and unit, and the rows from one to the next.
  int64_t row0;
  uint32_t unit0;
  int step = 1;
  if (NARROW) {
    step = kWarp >> a.shift;
    row0 = int64_t(warp) * (R * step) + (lane >> a.shift);
    unit0 = lane & ((1u << a.shift) - 1u);
  } else {
    const uint32_t group = warp / a.segments;
    row0 = int64_t(group) * R;
    unit0 = (warp - group * a.segments) * (kWarp * M) + lane;
  }
  int64_t source[R];  // row of the table
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = row0 + r * step;
    source[r] = -1;
    if (i < a.n_ids)
      source[r] = a.ids64
                      ? row_of(static_cast<const int64_t*>(a.ids)[i], a.first_row, a.n_rows)
                      : row_of(static_cast<const int32_t*>(a.ids)[i], a.first_row, a.n_rows);
  }
  Pack<IN, VEC> x[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (source[r] < 0) continue;
    const TI* p =
        static_cast<const TI*>(a.table) + source[r] * a.table_stride + int64_t(unit0) * VEC;
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (unit0 + m * kWarp < a.units) x[r][m].load(p + m * (kWarp * VEC));
  }
  TO* out = static_cast<TO*>(a.out) + row0 * a.out_stride + int64_t(unit0) * VEC;
#pragma unroll
  for (int r = 0; r < R; ++r, out += step * a.out_stride) {
    if (row0 + r * step >= a.n_ids) break;
    Pack<OUT, VEC> y;
    if (source[r] < 0) {
      y.clear();
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (unit0 + m * kWarp < a.units) y.store(out + m * (kWarp * VEC));
      continue;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = a.scale * x[r][m].get(i);
      y.set(v);
      if (unit0 + m * kWarp < a.units) y.store(out + m * (kWarp * VEC));
    }
  }
}

// embed_kernel by the two types, the width of a unit (1, 2, 4, and 8 where both
// types have 16 bits) and the units of a row: up to 32, up to 128, more.
// Measured on GB300: 131,072 rows of 8 units take 4.5 us with 4 of them side by side
// in a warp and 11.2 one by one; 100,000 rows of 65 units 8.5 us with 4 rows a warp
// and 20.8 with one.  Rows of 1023 scalars reach 78% of the copy rate with 16 loads
// a lane, 62% with 8 and 58% with 32.  Units of 16 bytes on the wider side, not the
// narrower, took 2048 columns of bf16 into fp32 from 33 to 25 us.
using EmbedKernel = void (*)(EmbedArgs);
#define EMBED_SHAPES(in, out)                                                                   \
  {embed_kernel<in, out, 1, 8, 1, true>, embed_kernel<in, out, 1, 4, 4, false>,                \
   embed_kernel<in, out, 1, 1, 16, false>},                                                     \
      {embed_kernel<in, out, 2, 8, 1, true>, embed_kernel<in, out, 2, 4, 4, false>,             \
       embed_kernel<in, out, 2, 1, 16, false>},                                                 \
      {embed_kernel<in, out, 4, 8, 1, true>, embed_kernel<in, out, 4, 2, 4, false>,             \
       embed_kernel<in, out, 4, 1, 8, false>}
#define EMBED_SHAPES8(in, out)                                                                  \
  {embed_kernel<in, out, 8, 4, 1, true>, embed_kernel<in, out, 8, 1, 4, false>,                \
   embed_kernel<in, out, 8, 1, 4, false>}
#define EMBED_NONE {nullptr, nullptr, nullptr}
const EmbedKernel embed_kernels[3][3][4][3] = {
    {{EMBED_SHAPES(TRAIN_BF16, TRAIN_BF16), EMBED_SHAPES8(TRAIN_BF16, TRAIN_BF16)},
     {EMBED_SHAPES(TRAIN_BF16, TRAIN_FP16), EMBED_SHAPES8(TRAIN_BF16, TRAIN_FP16)},
     {EMBED_SHAPES(TRAIN_BF16, TRAIN_FP32), EMBED_NONE}},
    {{EMBED_SHAPES(TRAIN_FP16, TRAIN_BF16), EMBED_SHAPES8(TRAIN_FP16, TRAIN_BF16)},
     {EMBED_SHAPES(TRAIN_FP16, TRAIN_FP16), EMBED_SHAPES8(TRAIN_FP16, TRAIN_FP16)},
     {EMBED_SHAPES(TRAIN_FP16, TRAIN_FP32), EMBED_NONE}},
    {{EMBED_SHAPES(TRAIN_FP32, TRAIN_BF16), EMBED_NONE},
     {EMBED_SHAPES(TRAIN_FP32, TRAIN_FP16), EMBED_NONE},
     {EMBED_SHAPES(TRAIN_FP32, TRAIN_FP32), EMBED_NONE}}};
const int kUnitWidth[4] = {1, 2, 4, 8};
const int kRows[4][3] = {{8, 4, 1}, {8, 4, 1}, {8, 2, 1}, {4, 1, 1}};
const int kSegment[4][3] = {{32, 128, 512}, {32, 128, 512}, {32, 128, 256}, {32, 128, 128}};

// The widest unit of at most 16 bytes that every row of both matrices is whole
// pieces of, each aligned to its size: 0, 1, 2, 3 for 1, 2, 4, 8 elements.
int unit_width(int64_t dim, const void* p, int32_t p_type, int64_t p_stride, const void* q,
               int32_t q_type, int64_t q_stride) {
  const auto fits = [&](const void* x, int32_t type, int64_t stride, int v) {
    const int bytes = v * size_of(type);
    return bytes <= 16 && reinterpret_cast<uintptr_t>(x) % uintptr_t(bytes) == 0 &&
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
  if (rc == LAMB_OK) rc = check_ids(ids, ids_dtype, n_ids, first_row, n_rows);
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
  const int shape = a.units <= kWarp ? 0 : a.units <= 128 ? 1 : 2;
  a.segments = (a.units + kSegment[w][shape] - 1) / kSegment[w][shape];
  int64_t rows = kRows[w][shape];  // a warp
  if (shape == 0) {
    while ((1u << a.shift) < a.units) ++a.shift;
    rows *= kWarp >> a.shift;
  }
  const int64_t groups = (n_ids + rows - 1) / rows;
  if (groups > kMaxCount / int64_t(a.segments))
    return fail(LAMB_ERR_INVALID, "n_ids * dim is too large");
  a.warps = uint32_t(groups * a.segments);
  const unsigned ctas = unsigned((int64_t(a.warps) * kWarp + kThreads - 1) / kThreads);
  const cudaError_t ce =
      launch(embed_kernels[table_dtype][out_dtype][w][shape], dim3(ctas), kThreads, 0,
             static_cast<cudaStream_t>(stream), true, 1, a);
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string("embed: ") + cudaGetErrorString(ce));
}

}  // extern "C"
