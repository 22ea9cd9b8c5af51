// Layer norm of rows that stay on chip (train_ops.h): the kernels,
// compiled once for each type of x.  Not part of the public interface.
#pragma once

#include "train_norm.h"

namespace traingb {

// ------------------------------------------------------- rows that stay on chip
struct NormArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* stats;
  int64_t n_rows, x_stride, y_stride;
  float eps;
  int32_t dim, param_type;
  int32_t lanes;              // threads a row
  int32_t period;             // rows this far apart begin equally far from a unit's boundary
  int32_t phase, row_phase;   // elements from one to the first row; from row to row
  int32_t stages;             // of the ring
};

// A row whose squares leave fp32's range, once more from memory and scaled by a
// power of two.  All threads of a group come here (of a warp, where groups are
// smaller), with `wanted` where the row is such a one.
template <int XT, int YT, Span S>
__device__ __noinline__ void scaled_row(const NormArgs& a, int64_t row, bool wanted,
                                        const Group& g) {
  const auto* x = static_cast<const typename TypeOf<XT>::T*>(a.x) + row * a.x_stride;
  auto* y = static_cast<typename TypeOf<YT>::T*>(a.y) + row * a.y_stride;
  const int end = wanted ? a.dim : 0;
  float top = 0.f, s = 0.f;
  for (int i = g.lane; i < end; i += g.lanes) top = fmaxf(top, fabsf(to_float<XT>(x[i])));
  const float scale = scale_of(g.largest<S>(top, 2)), inv = 1.f / float(a.dim);
  for (int i = g.lane; i < end; i += g.lanes) s += to_float<XT>(x[i]) * scale;
  const float centre = g.sum<S>(s, 3) * inv;
  s = 0.f;
  for (int i = g.lane; i < end; i += g.lanes) {
    const float d = to_float<XT>(x[i]) * scale - centre;
    s += d * d;
  }
  const float mean = centre / scale;
  const float rstd = rstd_of_scaled(g.sum<S>(s, 4) * inv, scale, a.eps);
  if (wanted && a.stats && g.lane == 0) a.stats[row] = mean, a.stats[a.n_rows + row] = rstd;
  by_type(a.param_type, [&](auto P) {
    constexpr int PT = decltype(P)::value;
    using TP = typename TypeOf<PT>::T;
    const TP* weight = static_cast<const TP*>(a.weight);
    const TP* bias = static_cast<const TP*>(a.bias);
    for (int i = g.lane; i < end; i += g.lanes) {
      const float v = (to_float<XT>(x[i]) - mean) * rstd;
      y[i] = from_float<YT>(v * (weight ? to_float<PT>(weight[i]) : 1.f) +
                            (bias ? to_float<PT>(bias[i]) : 0.f));
    }
  });
}

// Weight and bias as fp32 in shared memory, `width` floats each: element `column` at
// staged_at<E>(column - head).  Units of 8 elements lie in two halves apart, so that
// the threads of a warp read 16 bytes side by side from each.
constexpr int kLead = 8;
__host__ __device__ constexpr int staged_width(int dim) { return (dim + 2 * kLead + 15) / 8 * 8; }
template <int E>
__device__ __forceinline__ int staged_at(int i, int width) {
  i += kLead;
  if constexpr (E == 8) return (i & 4) * (width / 8) + (i >> 3) * 4 + (i & 3);
  return i;
}

template <int PT, int E>
__device__ __forceinline__ void stage_vector(const void* from, float none, int dim, int head,
                                             float* to) {
  using TP = typename TypeOf<PT>::T;
  constexpr int V = 16 / int(sizeof(TP));
  const int width = staged_width(dim);
  const TP* p = static_cast<const TP*>(from);
  // Elements in front of the first boundary of 16 bytes and behind the last are few.
  const int lead = min(dim, int((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(TP)));
  const int units = p ? (dim - lead) / V : 0;
#pragma unroll 4
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    Pack<PT, V> q;
    q.load(p + lead + u * V);
#pragma unroll
    for (int i = 0; i < V; ++i) to[staged_at<E>(lead + u * V + i - head, width)] = q.get(i);
  }
  for (int i = threadIdx.x; i < dim; i += blockDim.x) {
    if (p && i >= lead) i += units * V;
    if (i < dim) to[staged_at<E>(i - head, width)] = p ? to_float<PT>(p[i]) : none;
  }
}

template <int E>
__device__ __forceinline__ void stage_params(const NormArgs& a, int head, float* staged) {
  by_type(a.param_type, [&](auto P) {
    constexpr int PT = decltype(P)::value;
    stage_vector<PT, E>(a.weight, 1.f, a.dim, head, staged);
    stage_vector<PT, E>(a.bias, 0.f, a.dim, head, staged + staged_width(a.dim));
  });
  __syncthreads();
}

// ------------------------------------------------ rows that stream through a ring
// A row is shared by a warp or by a few.  Units of E elements (16 bytes) that lie
// whole and aligned in it come through a ring of asynchronous copies in shared
// memory, M units a thread; every thread reads back what it copied itself, so the
// ring needs no barriers.  What is left at the row's ends (fewer than E elements
// each) goes to single threads of the first warp, one element each.  All rows of a
// CTA begin equally far from a unit's boundary, so one layout of the parameters
// holds for all.  CTAs stay and walk through the rows.
//
// The variance comes from the differences to the mean (two joins a row), in pairs of fp32
// values.  Memory bounds it, with 15 instructions an element close behind: 8192 x 4096
// bf16 takes 25.4 us (5.3 TB/s), 8192 x 12288 71 (5.7), 50,021 x 1023 from fp32 to bf16 56
// (5.5); 3 us of each are the parameters' staging and the first rows.  Rows in registers,
// a CTA each, without a ring, took 31 to 39 us for the first; parameters read again for
// every row 57, since their loads waited for one another.
template <int XT, int YT, int M, Span S>
__global__ void __launch_bounds__(768) norm_ring_kernel(const __grid_constant__ NormArgs a) {
  using TX = typename TypeOf<XT>::T;
  using TY = typename TypeOf<YT>::T;
  constexpr int E = 16 / int(sizeof(TX));
  constexpr int C = M * E / 2;  // pairs a thread
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[kSlots * kWarp];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lanes = S == Span::kWarp ? kWarp : a.lanes;
  const int groups = threads / lanes, index = tid / lanes;
  const Group g{lanes, tid - index * lanes, index + 1, part + index * (lanes / kWarp)};
  const int dim = a.dim, width = staged_width(dim);
  float* staged = reinterpret_cast<float*>(smem);
  // A stage of the ring: each warp's M times 32 units together.
  const uint32_t stage = uint32_t(threads * M * 16);
  const uint32_t ring = shared_address(smem) + 8 * width + (tid >> 5) * (kWarp * M * 16) +
                        (tid & 31) * 16;
  const uint32_t ring_end = ring + uint32_t(a.stages) * stage;
  const int turn = int(blockIdx.x) % a.period;
  const int head = (E - (a.phase + turn * a.row_phase) % E) % E;
  const int units = (dim - head) / E;
  // This thread's units: `first` and every 32nd behind it.
  const int first = (g.lane >> 5) * (kWarp * M) + (g.lane & 31);
  const int left = units - first;
  // The column of its single element, if it has one.
  int single = -1;
  if (g.lane < head) single = g.lane;
  else if (g.lane < kWarp && kWarp - 1 - g.lane < (dim - head) % E) single = dim - kWarp + g.lane;

  pdl_wait();
  const int64_t step = int64_t(int(gridDim.x) / a.period * groups) * a.period;
  int64_t row = int64_t(int(blockIdx.x) / a.period * groups + index) * a.period + turn;
  // This thread's first unit, of the row to copy and of the row of y to write.
  const int64_t at = head + first * E;
  const TX* from = static_cast<const TX*>(a.x) + row * a.x_stride + at;
  TY* y = static_cast<TY*>(a.y) + row * a.y_stride + at;
  const int64_t step_x = step * a.x_stride, step_y = step * a.y_stride;
  const int64_t rounds = row < a.n_rows ? (a.n_rows - row + step - 1) / step : 0;
  int64_t to_copy = rounds;
  uint32_t in = ring, out = ring;
  const auto copy = [&] {
    if (to_copy > 0) {
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (m * kWarp < left) copy_async<16>(in + m * (kWarp * 16), from + m * (kWarp * E));
    }
    copy_commit();
    from += step_x, --to_copy;
    in += stage;
    if (in == ring_end) in = ring;
  };
  for (int k = 1; k < a.stages; ++k) copy();
  const TX* edge = static_cast<const TX*>(a.x) + row * a.x_stride + single;
  float coming = 0.f;
  if (single >= 0 && rounds > 0) coming = to_float<XT>(*edge);
  stage_params<E>(a, head, staged);
  const float inv = 1.f / float(dim);
  const float* w = staged + staged_at<E>(first * E, width);
  float* stats = a.stats + row;
  for (int64_t k = 1; k <= rounds; ++k, row += step, y += step_y, stats += step) {
    copy();
    float vs = coming;
    edge += step_x;
    if (single >= 0 && k < rounds) coming = to_float<XT>(*edge);
    if (a.stages == 3) copy_wait<2>();
    else copy_wait<1>();
    F2 v[C];
    F2 t = pair(vs, 0.f), u = pair(0.f);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      Pack<XT, E> x;
      x.clear();
      if (m * kWarp < left) load_shared(x, out + m * (kWarp * 16));
#pragma unroll
      for (int i = 0; i < E / 2; i += 2) {
        v[m * (E / 2) + i] = get2(x, i), v[m * (E / 2) + i + 1] = get2(x, i + 1);
        t = add2(t, v[m * (E / 2) + i]), u = add2(u, v[m * (E / 2) + i + 1]);
      }
    }
    out += stage;
    if (out == ring_end) out = ring;
    const float mean = g.sum<S>(sum2(add2(t, u)), 0) * inv;
    // From here on v is the difference to the mean.
    vs = single >= 0 ? vs - mean : 0.f;
    const F2 shift = pair(-mean);
    t = pair(vs * vs, 0.f), u = pair(0.f);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (m * kWarp >= left) continue;
#pragma unroll
      for (int i = 0; i < E / 2; i += 2) {
        F2& p = v[m * (E / 2) + i];
        F2& q = v[m * (E / 2) + i + 1];
        p = add2(p, shift), q = add2(q, shift);
        t = fma2(p, p, t), u = fma2(q, q, u);
      }
    }
    const float var = g.sum<S>(sum2(add2(t, u)), 1) * inv;
    if (!in_range(var, a.eps)) {
      scaled_row<XT, YT, S>(a, row, true, g);
      continue;
    }
    const float rstd = rstd_of(var, a.eps);
    if (a.stats && g.lane == 0) stats[0] = mean, stats[a.n_rows] = rstd;
    const F2 scale = pair(rstd);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (m * kWarp >= left) continue;
      Pack<YT, E> o;
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float* p = w + m * (kWarp * 4) + (i & 4) * (width / 8);
        const float4 f = *reinterpret_cast<const float4*>(p);
        const float4 h = *reinterpret_cast<const float4*>(p + width);
        const int c = (m * E + i) / 2;
        set2(o, i / 2, fma2(mul2(v[c], scale), pair(f.x, f.y), pair(h.x, h.y)));
        set2(o, i / 2 + 1, fma2(mul2(v[c + 1], scale), pair(f.z, f.w), pair(h.z, h.w)));
      }
      o.store(y + m * (kWarp * E));
    }
    if (single >= 0)
      y[single - at] = from_float<YT>(
          vs * rstd * staged[staged_at<E>(single - head, width)] +
          staged[width + staged_at<E>(single - head, width)]);
  }
}

// ------------------------------------------------------------------- short rows
// Less than a warp, or a warp, has R rows of one unit a thread each; a CTA has one
// piece of work.  65,536 x 256 bf16 takes 18.5 us (3.6 TB/s), 131,072 x 64 9.8.  Latency
// bounds it: 98 registers leave an SM two CTAs of 8 warps, which fill 53% of the issue slots
// with 146 instructions a row.  Of a warp's time 24% goes to waiting for its own arithmetic,
// 22% for its rows, which nothing asks for ahead, and 11% for shuffles and the root.
constexpr int kNormThreads = 256;

template <int XT, int YT, int E, int R>
__global__ void __launch_bounds__(kNormThreads)
    norm_short_kernel(const __grid_constant__ NormArgs a) {
  using TX = typename TypeOf<XT>::T;
  using TY = typename TypeOf<YT>::T;
  const int lanes = a.lanes, dim = a.dim;
  const int index = int(threadIdx.x) / lanes;
  const Group g{lanes, int(threadIdx.x) - index * lanes, 0, nullptr};
  const int64_t row0 = (int64_t(blockIdx.x) * (kNormThreads / lanes) + index) * R;
  const int rows = int(min(int64_t(R), a.n_rows - row0));  // <= 0: none
  const bool mine = g.lane < dim / E;
  const TX* from = static_cast<const TX*>(a.x) + row0 * a.x_stride + g.lane * E;
  pdl_wait();
  Pack<XT, E> x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    x[r].clear();
    if (mine && r < rows) x[r].load_once(from + r * a.x_stride);
  }
  F2 w[E / 2], b[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = pair(1.f), b[i] = pair(0.f);
  if (mine) {
    by_type(a.param_type, [&](auto P) {
      constexpr int PT = decltype(P)::value;
      const auto take = [&](const void* from, F2 (&to)[E / 2]) {
        const auto* p = static_cast<const typename TypeOf<PT>::T*>(from) + g.lane * E;
        Pack<PT, E> q;
        if (reinterpret_cast<uintptr_t>(p) % (Pack<PT, E>::kBytes < 16 ? 8 : 16) == 0) {
          q.load(p);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) to[i] = get2(q, i);
        } else {
#pragma unroll
          for (int i = 0; i < E / 2; ++i)
            to[i] = pair(to_float<PT>(p[2 * i]), to_float<PT>(p[2 * i + 1]));
        }
      };
      if (a.weight) take(a.weight, w);
      if (a.bias) take(a.bias, b);
    });
  }
  const float inv = 1.f / float(dim);
  F2 v[R][E / 2];
  float mean[R], rstd[R];
  bool odd = false, fine[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    F2 s = pair(0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[r][i] = get2(x[r], i), s = add2(s, v[r][i]);
    mean[r] = sum2(s);
  }
  for (int d = 1; d < lanes; d *= 2)
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] += __shfl_xor_sync(kAll, mean[r], d);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] *= inv;
    F2 s = pair(0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      v[r][i] = add2(v[r][i], pair(-mean[r]));
      s = fma2(v[r][i], v[r][i], s);
    }
    rstd[r] = mine ? sum2(s) : 0.f;
  }
  for (int d = 1; d < lanes; d *= 2)
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] += __shfl_xor_sync(kAll, rstd[r], d);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float var = rstd[r] * inv;
    rstd[r] = rstd_of(var, a.eps);
    fine[r] = in_range(var, a.eps);
    odd = odd || (!fine[r] && r < rows);
  }
  if (__any_sync(kAll, odd)) {
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      bool wanted = false;
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (k == r) wanted = !fine[k] && k < rows;
      scaled_row<XT, YT, Span::kPart>(a, row0 + r, wanted, g);
    }
  }
  TY* to = static_cast<TY*>(a.y) + row0 * a.y_stride + g.lane * E;
#pragma unroll
  for (int r = 0; r < R; ++r, to += a.y_stride) {
    if (!fine[r] || r >= rows) continue;
    if (a.stats && g.lane == 0)
      a.stats[row0 + r] = mean[r], a.stats[a.n_rows + row0 + r] = rstd[r];
    if (!mine) continue;
    Pack<YT, E> o;
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      set2(o, i, fma2(mul2(v[r][i], pair(rstd[r])), w[i], b[i]));
    o.store(to);
  }
}

// ------------------------------------------------------- rows element by element
// For rows of x and y that do not begin equally far from a unit's boundary, and short
// ones of odd widths: M elements a thread and R rows at once, in registers.  The loads'
// latency bounds it: 50,021 x 1023 bf16 takes 71 us (2.9 TB/s) where the ring takes 41,
// 300,000 x 33 37 us with two rows at once and 50 with one.
template <int XT, int YT, int M, int R, Span S>
__global__ void __launch_bounds__(512, M > 8 ? 0 : 2) norm_scalar_kernel(const __grid_constant__ NormArgs a) {
  using TX = typename TypeOf<XT>::T;
  using TY = typename TypeOf<YT>::T;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[kSlots * kWarp];
  const int dim = a.dim, width = staged_width(dim);
  float* staged = reinterpret_cast<float*>(smem);
  const int lanes = S == Span::kWarp ? kWarp : a.lanes;
  const int groups = int(blockDim.x) / lanes, index = int(threadIdx.x) / lanes;
  const Group g{lanes, int(threadIdx.x) - index * lanes, index + 1,
                part + index * (lanes / kWarp)};
  const int first = (g.lane >> 5) * (kWarp * M) + (g.lane & 31);
  const int left = dim - first;
  pdl_wait();
  stage_params<1>(a, 0, staged);
  const float inv = 1.f / float(dim);
  const float* w = staged + staged_at<1>(first, width);
  const int64_t step = int64_t(gridDim.x) * groups * R;
  for (int64_t row = (int64_t(blockIdx.x) * groups + index) * R; row < a.n_rows; row += step) {
    const int rows = int(min(int64_t(R), a.n_rows - row));
    const TX* from = static_cast<const TX*>(a.x) + row * a.x_stride + first;
    float v[R][M], mean[R], var[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int m = 0; m < M; ++m)
        v[r][m] = r < rows && m * kWarp < left ? to_float<XT>(from[m * kWarp]) : 0.f;
      from += a.x_stride;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int m = 0; m < M; m += 2) s += v[r][m], t += v[r][m + 1];
      mean[r] = s + t;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = g.sum<S>(mean[r], 0) * inv;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        v[r][m] = m * kWarp < left ? v[r][m] - mean[r] : 0.f;
        if (m & 1) s += v[r][m] * v[r][m];
        else t += v[r][m] * v[r][m];
      }
      var[r] = s + t;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) var[r] = g.sum<S>(var[r], 1) * inv;
    TY* y = static_cast<TY*>(a.y) + row * a.y_stride + first;
#pragma unroll
    for (int r = 0; r < R; ++r, y += a.y_stride) {
      if (r >= rows) break;
      if (!in_range(var[r], a.eps)) {
        scaled_row<XT, YT, S>(a, row + r, true, g);
        continue;
      }
      const float rstd = rstd_of(var[r], a.eps);
      if (a.stats && g.lane == 0)
        a.stats[row + r] = mean[r], a.stats[a.n_rows + row + r] = rstd;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (m * kWarp < left)
          y[m * kWarp] = from_float<YT>(v[r][m] * rstd * w[m * kWarp] + w[width + m * kWarp]);
    }
  }
}

// The kernels of two types.
using NormKernel = void (*)(NormArgs);
constexpr int kScalars[4] = {2, 4, 8, 32};     // elements a thread
constexpr int kScalarRows[4] = {2, 2, 1, 1};  // rows at once
struct NormKernels {
  NormKernel whole;       // short rows of whole units of 16 bytes of the wider type
  NormKernel ring[3];     // a warp with 16 or 32 elements a thread, several warps with 32
  NormKernel scalar[5];   // a warp with kScalars elements a thread, several with 32
};
template <int XT, int YT>
constexpr NormKernels norm_kernels() {
  constexpr int E = XT == TRAIN_FP32 || YT == TRAIN_FP32 ? 4 : 8;
  constexpr int M = XT == TRAIN_FP32 ? 4 : 2;  // units of 16 elements
  return {norm_short_kernel<XT, YT, E, 4>,
          {norm_ring_kernel<XT, YT, M, Span::kWarp>, norm_ring_kernel<XT, YT, 2 * M, Span::kWarp>,
           norm_ring_kernel<XT, YT, 2 * M, Span::kWarps>},
          {norm_scalar_kernel<XT, YT, kScalars[0], kScalarRows[0], Span::kWarp>,
           norm_scalar_kernel<XT, YT, kScalars[1], kScalarRows[1], Span::kWarp>,
           norm_scalar_kernel<XT, YT, kScalars[2], kScalarRows[2], Span::kWarp>,
           norm_scalar_kernel<XT, YT, kScalars[3], kScalarRows[3], Span::kWarp>,
           norm_scalar_kernel<XT, YT, kScalars[3], kScalarRows[3], Span::kWarps>}};
}

// Each defined in a translation unit of its own.
const NormKernels& norm_kernels_bf16(int y_type);
const NormKernels& norm_kernels_fp16(int y_type);
const NormKernels& norm_kernels_fp32(int y_type);

}  // namespace traingb
