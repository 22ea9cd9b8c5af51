// Layer norm's backward pass for rows that stay on chip (train_ops.h): the kernels,
// compiled once for each type of x.  Not part of the public interface.
#pragma once

#include <cooperative_groups.h>

#include "train_norm.h"

namespace traingb {

struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* weight;
  const float* stats;
  void* dx;        // NULL: not wanted
  float* partial;  // [pieces][2][dim]: of the weight's and the bias's gradient; NULL too
  int64_t n_rows, dim, dy_stride, x_stride, dx_stride;
  int64_t rows_per_piece;
  int32_t dy_type, x_type, param_type;
  // Of rows on chip.
  int32_t lanes;             // threads a row
  int32_t period;            // rows this far apart begin equally far from a unit's boundary
  int32_t phase, row_phase;  // elements from one to the first row; from row to row
  int32_t stages;            // of the ring
  // Where one cluster has all rows, it writes the sums itself; 0 CTAs: pieces are.
  int32_t joined;
  void* weight_grad;
  void* bias_grad;
  int32_t grad_type, accumulate;
};

constexpr int kJoined = 16;  // CTAs, at most

// One sum into a parameter's gradient.
__device__ __forceinline__ void write_grad(void* to, int type, bool accumulate, int64_t at,
                                           float s) {
  by_type(type, [&](auto P) {
    constexpr int PT = decltype(P)::value;
    auto* p = static_cast<typename TypeOf<PT>::T*>(to) + at;
    if (accumulate) s += to_float<PT>(*p);
    *p = from_float<PT>(s);
  });
}

// Rows that a group works on at once, by the elements a thread has of each.
__host__ __device__ constexpr int grad_rows(int elements) { return elements == 8 ? 2 : 1; }

// The weight's element at a column, or 1.
template <int N, class At>
__device__ __forceinline__ void load_weight(const NormGradArgs& a, float (&w)[N], At&& at) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = 1.f;
  if (!a.weight) return;
  by_type(a.param_type, [&](auto P) {
    constexpr int PT = decltype(P)::value;
    const auto* p = static_cast<const typename TypeOf<PT>::T*>(a.weight);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int column = at(i);
      if (column >= 0) w[i] = to_float<PT>(p[column]);
    }
  });
}

// Adds up the groups' sums, each at [group][2][dim] in `sums`, and writes this CTA's
// piece, or with the other CTAs of a cluster, a share of the columns each, the gradients.
__device__ __forceinline__ void write_sums(const NormGradArgs& a, float* sums, int groups) {
  const int dim = int(a.dim), n = 2 * dim;
  float* to = a.joined ? sums : a.partial + int64_t(blockIdx.x) * n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    float s = sums[i];
    for (int k = 1; k < groups; ++k) s += sums[int64_t(k) * n + i];
    to[i] = s;
  }
  if (!a.joined) return;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += a.joined * blockDim.x) {
    float s = 0.f, u[kJoined];
#pragma unroll
    for (int r = 0; r < kJoined; ++r)
      u[r] = r < a.joined ? cluster.map_shared_rank(sums, r)[i] : 0.f;
#pragma unroll
    for (int r = 0; r < kJoined; ++r) s += u[r];
    void* grad = i < dim ? a.weight_grad : a.bias_grad;
    if (grad) write_grad(grad, a.grad_type, a.accumulate, i < dim ? i : i - dim, s);
  }
  cluster.sync();  // no CTA leaves while another reads from it
}

// Rows come through a ring of asynchronous copies as in the forward pass: units of E
// elements of x and grad_out, M of each a thread.  A thread keeps the weight and the
// sums over the rows for its columns in registers, which leaves no room for the row's
// elements: they are read from the ring once for the two sums along the row and the
// sums down the columns, and again for x_grad.  Where a thread has 8 elements of a row
// there is room (32768 x 256: 16.1 us, read again 19.0; with 16 elements 47.3 and 45.1 for
// 8192 x 4096, since the compiler runs short of registers).  At the end the CTA's groups are added
// and written as one piece, and join_kernel adds the pieces; the CTAs of few rows are a
// cluster that adds its sums by itself.
//
// WS: the weight lies in shared memory instead, which the widest rows need (24 elements a
// thread: 8192 x 12288 bf16 takes 115 us so, 199 with spilled registers); with 16 elements
// registers are quicker (45.4 and 47.7 us for 8192 x 4096).  Two rows at once pay for 8
// elements a thread only (32768 x 512: 26 us and 27; with 16: 55 and 46 for 8192 x 4096).
// What bounds it is the latency of a row's steps with 16 warps an SM, as many as the
// registers allow, and instructions (24 an element, a third of them joins and addresses):
// 8192 x 4096 bf16 takes 41 us and the join 4 more (4.4 TB/s), 32768 x 12288 391 (6.2).
// Short rows are the same: at 32768 x 256 16 warps an SM fill 55% of the issue slots with 253
// instructions a row; of a warp's time 16% goes to waiting for its own arithmetic, 15% for
// rows and stats, 17% for other warps' turns, 9% for shuffles.
template <int XT, int YT, int M, int R, Span S, bool WS>
__global__ void __launch_bounds__(512) grad_ring_kernel(const __grid_constant__ NormGradArgs a) {
  using TX = typename TypeOf<XT>::T;
  using TY = typename TypeOf<YT>::T;
  constexpr int E = XT == TRAIN_FP32 || YT == TRAIN_FP32 ? 4 : 8;
  constexpr int C = M * E / 2;  // pairs a thread
  constexpr bool kKeep = M * E <= 8;  // a row's elements, in registers
  constexpr int BX = E * int(sizeof(TX)), BY = E * int(sizeof(TY));
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[4 * R * kWarp];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lanes = S == Span::kWarp ? kWarp : a.lanes;
  const int groups = threads / lanes, index = tid / lanes;
  const Group g{lanes, tid - index * lanes, index + 1, part + index * (lanes / kWarp)};
  const int dim = int(a.dim);
  // A stage of the ring: R rows, of each x's units, then grad_out's; each warp's M times
  // 32 together.
  const uint32_t half = uint32_t(threads * M * BX);
  const uint32_t line = half + uint32_t(threads * M * BY), stage = R * line;
  const uint32_t ring = shared_address(smem), ring_end = ring + uint32_t(a.stages) * stage;
  const uint32_t mine = uint32_t((tid >> 5) * (kWarp * M) + (tid & 31));
  const uint32_t mine_x = mine * BX, mine_y = half + mine * BY;
  const int turn = int(blockIdx.x) % a.period;
  const int head = S == Span::kPart ? 0 : (E - (a.phase + turn * a.row_phase) % E) % E;
  const int units = (dim - head) / E;
  // This thread's units: `first` and every 32nd behind it (one where less than a warp
  // has the row).
  const int first = S == Span::kPart ? g.lane
                                     : (g.lane >> 5) * (kWarp * M) + (g.lane & 31);
  const int left = units - first;
  // The column of its single element, if it has one.
  int single = -1;
  if (S != Span::kPart) {
    if (g.lane < head) single = g.lane;
    else if (g.lane < kWarp && kWarp - 1 - g.lane < (dim - head) % E)
      single = dim - kWarp + g.lane;
  }

  pdl_wait();
  const int64_t step = int64_t(max(1, int(gridDim.x) / a.period) * groups) * a.period;
  int64_t row = int64_t(int(blockIdx.x) / a.period * groups + index) * a.period + turn;
  const int64_t at = head + int64_t(first) * E;
  // This thread's first unit, of the row to copy and of the row of x_grad to write.
  const TX* from_x = static_cast<const TX*>(a.x) + row * a.x_stride + at;
  const TY* from_y = static_cast<const TY*>(a.dy) + row * a.dy_stride + at;
  TX* to = static_cast<TX*>(a.dx) + row * a.dx_stride + at;
  const int64_t step_x = step * a.x_stride, step_y = step * a.dy_stride;
  const int64_t step_to = step * a.dx_stride;
  const int rounds = row < a.n_rows ? int((a.n_rows - row + step - 1) / step) : 0;
  const bool ends = head > 0 || units * E < dim - head;
  int to_copy = rounds;
  uint32_t in = ring, out = ring;
  const auto copy = [&] {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (to_copy > 0) {
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (m * kWarp < left) {
            copy_async<BX>(in + r * line + mine_x + m * (kWarp * BX), from_x + m * (kWarp * E));
            copy_async<BY>(in + r * line + mine_y + m * (kWarp * BY), from_y + m * (kWarp * E));
          }
      }
      from_x += step_x, from_y += step_y, --to_copy;
    }
    copy_commit();
    in += stage;
    if (in == ring_end) in = ring;
  };
  for (int k = 1; k < a.stages; ++k) copy();
  // What a row has besides: its stats and this thread's single elements.
  const float* stats = a.stats + row;
  int64_t edge = row;
  float mean[R], rstd[R], xe[R] = {}, ye[R] = {};
  int to_look = rounds;
  const auto look = [&] {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = rstd[r] = 0.f;
      if (to_look > 0) {
        mean[r] = stats[0], rstd[r] = stats[a.n_rows];
        if (ends && single >= 0) {
          xe[r] = to_float<XT>(static_cast<const TX*>(a.x)[edge * a.x_stride + single]);
          ye[r] = to_float<YT>(static_cast<const TY*>(a.dy)[edge * a.dy_stride + single]);
        }
      }
      stats += step, --to_look;
      if (ends) edge += step;
    }
  };
  look();
  float we[1];
  load_weight(a, we, [&](int) { return single; });
  F2 w[C], dw[C], db[C];
  // In shared memory behind the ring: four elements of each thread's unit together.
  const uint32_t kept = ring_end + mine * 16;
  if constexpr (WS) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float wf[E];
      load_weight(a, wf, [&](int i) {
        return m * kWarp < left ? int(at) + m * (kWarp * E) + i : -1;
      });
#pragma unroll
      for (int i = 0; i < E; i += 4)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                         kept + uint32_t(i / 4 * threads * M + m * kWarp) * 16),
                     "f"(wf[i]), "f"(wf[i + 1]), "f"(wf[i + 2]), "f"(wf[i + 3])
                     : "memory");
    }
  } else {
    float wf[2 * C];
    load_weight(a, wf, [&](int i) {
      return i / E * kWarp < left ? int(at) + i / E * (kWarp * E) + i % E : -1;
    });
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = pair(wf[2 * c], wf[2 * c + 1]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) dw[c] = db[c] = pair(0.f);
  const auto weights = [&](int m) {
    if constexpr (WS) {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        Pack<TRAIN_FP32, 4> p;
        load_shared(p, kept + uint32_t(i / 4 * threads * M + m * kWarp) * 16);
        w[m * (E / 2) + i / 2] = get2(p, 0), w[m * (E / 2) + i / 2 + 1] = get2(p, 1);
      }
    }
  };
  float dwe = 0.f, dbe = 0.f;
  const float inv = 1.f / float(dim);
  int parity = 0;
  // Where groups share a warp, the warp's first has the most rows.
  const int turns = S == Span::kPart ? __shfl_sync(kAll, rounds, 0) : rounds;
  for (int k = 0; k < turns; k += R) {
    copy();
    F2 shift[R], scale[R];
    float rstd1[R], xs[R] = {}, ys[R] = {};
    bool held[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      held[r] = (R == 1 && S != Span::kPart) || k + r < rounds;
      shift[r] = pair(-mean[r]), scale[r] = pair(rstd[r]);
      rstd1[r] = rstd[r];
      if (ends) xs[r] = (xe[r] - mean[r]) * rstd[r], ys[r] = ye[r];
    }
    look();
    if (a.stages == 4) copy_wait<3>();
    else if (a.stages == 3) copy_wait<2>();
    else copy_wait<1>();
    const auto unit = [&](int r, int m, Pack<XT, E>& x, Pack<YT, E>& y) {
      load_shared(x, out + r * line + mine_x + m * (kWarp * BX));
      load_shared(y, out + r * line + mine_y + m * (kWarp * BY));
    };
    float along[2 * R];
    Pack<XT, E> x[R][M];
    Pack<YT, E> y[R][M];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 along1 = pair(0.f), alongx = pair(0.f);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (m * kWarp >= left || !held[r]) continue;
        unit(r, m, x[r][m], y[r][m]);
        weights(m);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const int c = m * (E / 2) + i;
          const F2 d = mul2(add2(get2(x[r][m], i), shift[r]), scale[r]);
          const F2 v = get2(y[r][m], i), gw = mul2(v, w[c]);
          along1 = add2(along1, gw);
          alongx = fma2(gw, d, alongx);
          db[c] = add2(db[c], v);
          dw[c] = fma2(v, d, dw[c]);
        }
      }
      along[2 * r] = sum2(along1), along[2 * r + 1] = sum2(alongx);
      if (ends && single >= 0 && held[r]) {
        along[2 * r] += ys[r] * we[0], along[2 * r + 1] += ys[r] * we[0] * xs[r];
        dbe += ys[r], dwe += ys[r] * xs[r];
      }
    }
    if (a.dx) {
      g.sums<S>(along, parity);
      parity ^= 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float s = along[2 * r] * inv, t = along[2 * r + 1] * inv;
        const F2 less1 = pair(-s * rstd1[r]), lessx = pair(-t);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          if (m * kWarp >= left || !held[r]) continue;
          Pack<XT, E> o;
          if (!kKeep) unit(r, m, x[r][m], y[r][m]);
          weights(m);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const F2 d = mul2(add2(get2(x[r][m], i), shift[r]), scale[r]);
            const F2 gw = mul2(get2(y[r][m], i), w[m * (E / 2) + i]);
            set2(o, i, fma2(fma2(d, lessx, gw), scale[r], less1));
          }
          o.store(to + m * (kWarp * E));
        }
        if (ends && single >= 0 && held[r])
          to[single - at] = from_float<XT>(rstd1[r] * (ys[r] * we[0] - s - xs[r] * t));
        to += step_to;
      }
    }
    out += stage;
    if (out == ring_end) out = ring;
  }
  if (!a.partial && !a.joined) return;
  pdl_trigger();
  // The ring's memory is free when all groups are through.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem) + int64_t(index) * 2 * dim;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int m = 2 * c / E;
    if (m * kWarp >= left) continue;
    const int column = int(at) + m * (kWarp * E) + 2 * c % E;
    split(dw[c], sums[column], sums[column + 1]);
    split(db[c], sums[dim + column], sums[dim + column + 1]);
  }
  if (single >= 0) sums[single] = dwe, sums[dim + single] = dbe;
  write_sums(a, reinterpret_cast<float*>(smem), groups);
}

// Element by element, M a thread and R rows at once, straight from memory: for rows of x,
// grad_out and x_grad that do not begin equally far from a unit's boundary, and short odd
// ones.  It waits for each row's loads: 50,021 x 1023 bf16 takes 132 us (2.3 TB/s).
template <int XT, int YT, int M, int R, Span S>
__global__ void __launch_bounds__(512) grad_scalar_kernel(const __grid_constant__ NormGradArgs a) {
  using TX = typename TypeOf<XT>::T;
  using TY = typename TypeOf<YT>::T;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[8 * kWarp];
  const int tid = threadIdx.x;
  const int lanes = S == Span::kWarp ? kWarp : a.lanes;
  const int groups = int(blockDim.x) / lanes, index = tid / lanes;
  const Group g{lanes, tid - index * lanes, index + 1, part + index * (lanes / kWarp)};
  const int dim = int(a.dim);
  const int first = (g.lane >> 5) * (kWarp * M) + (g.lane & 31);
  const int left = dim - first;
  pdl_wait();
  float w[M], dw[M] = {}, db[M] = {};
  load_weight(a, w, [&](int i) { return i * kWarp < left ? first + i * kWarp : -1; });
  const float inv = 1.f / float(dim);
  const int64_t step = int64_t(gridDim.x) * groups * R;
  int parity = 0;
  for (int64_t row = (int64_t(blockIdx.x) * groups + index) * R; row < a.n_rows; row += step) {
    const int rows = int(min(int64_t(R), a.n_rows - row));
    const TX* px = static_cast<const TX*>(a.x) + row * a.x_stride + first;
    const TY* py = static_cast<const TY*>(a.dy) + row * a.dy_stride + first;
    float x[R][M], y[R][M], mean[R], rstd[R], along[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = rstd[r] = 0.f;
      if (r < rows) mean[r] = a.stats[row + r], rstd[r] = a.stats[a.n_rows + row + r];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        x[r][m] = y[r][m] = 0.f;
        if (r < rows && m * kWarp < left)
          x[r][m] = to_float<XT>(px[m * kWarp]), y[r][m] = to_float<YT>(py[m * kWarp]);
      }
      px += a.x_stride, py += a.dy_stride;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        x[r][m] = r < rows && m * kWarp < left ? (x[r][m] - mean[r]) * rstd[r] : 0.f;
        db[m] += y[r][m], dw[m] += y[r][m] * x[r][m];
        y[r][m] *= w[m];
        s += y[r][m], t += y[r][m] * x[r][m];
      }
      along[2 * r] = s, along[2 * r + 1] = t;
    }
    if (a.dx) {
      g.sums<S>(along, parity);
      parity ^= 1;
      TX* to = static_cast<TX*>(a.dx) + row * a.dx_stride + first;
#pragma unroll
      for (int r = 0; r < R; ++r, to += a.dx_stride) {
        if (r >= rows) break;
        const float s = along[2 * r] * inv, t = along[2 * r + 1] * inv;
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (m * kWarp < left)
            to[m * kWarp] = from_float<XT>(rstd[r] * (y[r][m] - s - x[r][m] * t));
      }
    }
  }
  if (!a.partial && !a.joined) return;
  pdl_trigger();
  float* sums = reinterpret_cast<float*>(smem) + int64_t(index) * 2 * dim + first;
#pragma unroll
  for (int m = 0; m < M; ++m)
    if (m * kWarp < left) sums[m * kWarp] = dw[m], sums[dim + m * kWarp] = db[m];
  write_sums(a, reinterpret_cast<float*>(smem), groups);
}

// The kernels of two types.
using NormGradKernel = void (*)(NormGradArgs);
constexpr int kGradScalars[3] = {2, 8, 16};    // elements a thread
constexpr int kGradScalarRows[3] = {2, 2, 1};  // rows at once
struct NormGradKernels {
  // Part of a warp or a warp with 8 elements a thread, a warp with 16, several with 16 or 24.
  NormGradKernel ring[5];
  NormGradKernel scalar[4];  // a warp with 2, 8 or 16 elements a thread, several with 16
};
template <int XT, int YT>
constexpr NormGradKernels norm_grad_kernels() {
  constexpr int M = XT == TRAIN_FP32 || YT == TRAIN_FP32 ? 2 : 1;  // units of 8 elements
  return {{grad_ring_kernel<XT, YT, 1, grad_rows(8), Span::kPart, false>, grad_ring_kernel<XT, YT, M, grad_rows(8), Span::kWarp, false>,
           grad_ring_kernel<XT, YT, 2 * M, grad_rows(16), Span::kWarp, false>,
           grad_ring_kernel<XT, YT, 2 * M, grad_rows(16), Span::kWarps, false>,
           grad_ring_kernel<XT, YT, 3 * M, grad_rows(24), Span::kWarps, true>},
          {grad_scalar_kernel<XT, YT, kGradScalars[0], kGradScalarRows[0], Span::kWarp>,
           grad_scalar_kernel<XT, YT, kGradScalars[1], kGradScalarRows[1], Span::kWarp>,
           grad_scalar_kernel<XT, YT, kGradScalars[2], kGradScalarRows[2], Span::kWarp>,
           grad_scalar_kernel<XT, YT, kGradScalars[2], kGradScalarRows[2], Span::kWarps>}};
}

// Each defined in a translation unit of its own.
const NormGradKernels& norm_grad_kernels_bf16(int y_type);
const NormGradKernels& norm_grad_kernels_fp16(int y_type);
const NormGradKernels& norm_grad_kernels_fp32(int y_type);

}  // namespace traingb
