// The distillation loss of rows that stay in shared memory (train_ops.h): the
// kernels, compiled once for each type of the logits.  Not part of the public
// interface.
#pragma once

#include <cooperative_groups.h>

#include "train_norm.h"

namespace traingb {

constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct DistillArgs {
  const void* logits;
  const void* top_ids;
  const void* top_logits;
  const void* labels;
  const float* row_grad;
  float* loss;
  void* grad;
  int64_t n_rows, stride, ids_stride, top_stride, grad_stride, ignore_id;
  int32_t vocab, top_k;
  float inv_temperature, soft_weight, hard_weight, temperature, scale;
  int32_t type, grad_type, ids64, top_type, labels64;
  // Of the kernels below.
  int32_t ctas;              // that share a row: a cluster
  int32_t slice;             // units of a row that each of them holds
  int32_t phase, row_phase;  // elements from a unit's boundary to the first row; row to row
  int32_t whole;             // grad's units are aligned where those of the logits are
};

__device__ __forceinline__ int64_t read_id(const void* p, int64_t i, int32_t is64) {
  return is64 ? static_cast<const int64_t*>(p)[i] : int64_t(static_cast<const int32_t*>(p)[i]);
}

// 2^x, for x <= 0; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ F2 exp2_of(F2 x) {
  float lo, hi;
  split(x, lo, hi);
  return pair(exp2_of(lo), exp2_of(hi));
}

// A unit of logits: 16 bytes.
template <int ZT>
struct Unit {
  static constexpr int E = 16 / size_of(ZT);
  uint4 q;
  __device__ __forceinline__ void none() {  // -inf throughout
    const uint32_t w = ZT == TRAIN_BF16   ? 0xff80ff80u
                       : ZT == TRAIN_FP16 ? 0xfc00fc00u
                                          : 0xff800000u;
    q = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ F2 get(int i) const {
    Pack<ZT, E> p;
    p.w[0] = q.x, p.w[1] = q.y, p.w[2] = q.z, p.w[3] = q.w;
    return get2(p, i);
  }
};
template <int ZT>
__device__ __forceinline__ float largest(const Unit<ZT>& a, const Unit<ZT>& b) {
  if constexpr (ZT == TRAIN_FP32) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lo, hi;
      split(a.get(i), lo, hi);
      m = fmaxf(m, fmaxf(lo, hi));
      split(b.get(i), lo, hi);
      m = fmaxf(m, fmaxf(lo, hi));
    }
    return m;
  } else {
    const uint32_t w[8] = {a.q.x, a.q.y, a.q.z, a.q.w, b.q.x, b.q.y, b.q.z, b.q.w};
    if constexpr (ZT == TRAIN_BF16) {
      const auto* h = reinterpret_cast<const __nv_bfloat162*>(w);
      const auto m = __hmax2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])),
                             __hmax2(__hmax2(h[4], h[5]), __hmax2(h[6], h[7])));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      const auto* h = reinterpret_cast<const __half2*>(w);
      const auto m = __hmax2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])),
                             __hmax2(__hmax2(h[4], h[5]), __hmax2(h[6], h[7])));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
}

// Sums of exponentials relative to a largest value: of one temperature or of two.
// The largest value starts at the lowest finite one, so that it is never -inf.
template <int TEMPS>
struct Sums {
  float top = -FLT_MAX;
  float s[TEMPS] = {};
  __device__ __forceinline__ void raise(float to, const float (&c)[TEMPS]) {
    const float d = top - to;
#pragma unroll
    for (int k = 0; k < TEMPS; ++k) s[k] *= exp2_of(d * c[k]);
    top = to;
  }
  __device__ __forceinline__ void join_warp(const float (&c)[TEMPS]) {
    raise(warp_max(top), c);
#pragma unroll
    for (int k = 0; k < TEMPS; ++k) s[k] = warp_sum(s[k]);
  }
};

constexpr int kDistillThreads = 256;
constexpr int kDistillWarps = kDistillThreads / kWarp;
constexpr int kMostCtas = 16;
constexpr int kParts = 4;  // of a row, each waited for by itself

// A row's slice is copied into shared memory asynchronously, in units of 16 bytes, and
// read there twice: once for the running largest value and sums of exponentials, once
// for the gradient.  A thread reads back the units that it copied itself and, when it
// is through with one, asks for the next row's in its place, so copies and stores are
// under way at once.  What is left at the row's ends goes to single threads of the
// first CTA, one element each.  The teacher's entries and the label are gathered while
// the row is on its way; the tokens they name are written again, all of a token's
// shares together, when the others are done.
//   ZT, GT  types of logits and grad        TEMPS  1: one softmax serves both terms
template <int ZT, int GT, int TEMPS, bool GRAD>
__global__ void __launch_bounds__(kDistillThreads, 3)
    distill_kernel(const __grid_constant__ DistillArgs a) {
  namespace cg = cooperative_groups;
  using TZ = typename TypeOf<ZT>::T;
  using TG = typename TypeOf<GT>::T;
  constexpr int E = Unit<ZT>::E;
  extern __shared__ __align__(16) unsigned char smem[];
  struct Part {
    float top, s[2], spare;
  };
  __shared__ Part parts[2][kMostCtas * kDistillWarps];  // by the row's parity
  __shared__ float2 teacher[2][kDistillWarps];          // largest, sum
  __shared__ float terms[2][kDistillWarps];
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads / kWarp;
  const int warp = tid / kWarp, lane = tid % kWarp;
  const int vocab = a.vocab, room = a.top_k + 1;
  const int rank = a.ctas == 1 ? 0 : int(blockIdx.x) % a.ctas;
  uint4* slot = reinterpret_cast<uint4*>(smem);
  unsigned char* lists = smem + size_t(a.slice) * 16;

  const bool soft = a.top_k > 0 && a.soft_weight != 0.f;
  const bool hard = a.labels && a.hard_weight != 0.f;
  // Scales of the exponents: the soft term's and, of two, behind it the hard term's.
  float c[TEMPS];
  c[0] = soft ? a.inv_temperature * kLog2e : kLog2e;
  if constexpr (TEMPS == 2) c[1] = kLog2e;
  const float ct = a.inv_temperature * kLog2e;

  cg::cluster_group cluster = cg::this_cluster();
  if (a.ctas > 1) cluster.sync();  // all of its CTAs run now
  pdl_wait();

  const int64_t step = int64_t(gridDim.x) / a.ctas;
  const int per_thread = (a.slice + threads - 1) / threads;
  const int per_part = ((per_thread + kParts - 1) / kParts + 1) / 2 * 2;
  const auto head_of = [&](int64_t row) {
    return (E - (a.phase + int(row % E) * a.row_phase) % E) % E;
  };
  const auto row_of = [&](int64_t row) {
    return static_cast<const TZ*>(a.logits) + row * a.stride;
  };
  // What is known of a row in front of its work.
  int64_t label = -1;
  float up = a.scale;
  const auto look = [&](int64_t row, int64_t& label, float& up) {
    label = a.labels ? read_id(a.labels, row, a.labels64) : 0;
    up = GRAD && a.row_grad ? a.scale * a.row_grad[row] : a.scale;
  };
  const auto live_of = [&](int64_t label, float up) {
    return (!a.labels || (label != a.ignore_id && label >= 0 && label < vocab)) &&
           (soft || hard) && (a.loss || up != 0.f);
  };
  const auto copy = [&](const TZ* from, int units, int j) {
    const int u = rank * a.slice + j * threads + tid;
    if (j * threads + tid < a.slice && u < units)
      copy_async16(slot + j * threads + tid, from + int64_t(u) * E);
  };
  int64_t row = int64_t(blockIdx.x) / a.ctas;
  if (row < a.n_rows) {
    look(row, label, up);
    const bool live = live_of(label, up);
    const int head = head_of(row), units = (vocab - head) / E;
    for (int part = 0; part < kParts; ++part) {
      for (int j = part * per_part; live && j < min(per_thread, (part + 1) * per_part); ++j)
        copy(row_of(row) + head, units, j);
      copy_commit();
    }
  }
  int parity = 0;
  for (; row < a.n_rows; row += step, parity ^= 1) {
    int32_t* id = reinterpret_cast<int32_t*>(lists) + parity * 3 * room;
    float* coef = reinterpret_cast<float*>(id + room);
    float* zed = coef + room;
    const TZ* z = row_of(row);
    TG* grad = GRAD ? static_cast<TG*>(a.grad) + row * a.grad_stride : nullptr;
    const int head = head_of(row), units = (vocab - head) / E;
    const int mine = min(a.slice, units - rank * a.slice);  // units here; < 0: none
    const bool live = live_of(label, up);
    // The next row.
    const int64_t next = row + step;
    int64_t next_label = -1;
    float next_up = 0.f;
    bool next_live = false;
    int next_head = 0, next_units = 0;
    if (next < a.n_rows) {
      look(next, next_label, next_up);
      next_live = live_of(next_label, next_up);
      next_head = head_of(next), next_units = (vocab - next_head) / E;
    }
    const TZ* next_from = row_of(next) + next_head;
    // The column of this thread's single element, if it has one.
    int single = -1;
    if (rank == 0 && tid < kWarp) {
      if (tid < head) single = tid;
      else if (kWarp - 1 - tid < (vocab - head) % E) single = vocab - kWarp + tid;
    }
    // The teacher's entries.
    float best = -INFINITY, size = 0.f;
    if (live && soft) {
      for (int k = tid; k < a.top_k; k += threads) {
        const int64_t i = read_id(a.top_ids, row * a.ids_stride + k, a.ids64);
        float t = 0.f;
        by_type(a.top_type, [&](auto T) {
          constexpr int TT = decltype(T)::value;
          t = to_float<TT>(static_cast<const typename TypeOf<TT>::T*>(
              a.top_logits)[row * a.top_stride + k]);
        });
        const bool valid = i >= 0 && i < vocab && t != -INFINITY;
        id[k] = valid ? int32_t(i) : -1;
        coef[k] = t;
        if (!valid) continue;
        zed[k] = to_float<ZT>(z[i]);
        if (t > best) {
          size = size * exp2_of((best - t) * ct) + 1.f;
          best = t;
        } else {
          size += t == best && t < INFINITY ? 1.f : exp2_of((t - best) * ct);
        }
      }
    }
    float edge = -INFINITY;
    if (live && single >= 0) edge = to_float<ZT>(z[single]);
    if (tid == 0) {
      id[a.top_k] = live && hard ? int32_t(label) : -1;
      zed[a.top_k] = live && hard ? to_float<ZT>(z[label]) : 0.f;
    }
    // The largest value and the sums.
    Sums<TEMPS> sums;
    if (live) {
      for (int part = 0; part < kParts; ++part) {
        if constexpr (GRAD) {
          if (part == 0) copy_wait<3>();
          else if (part == 1) copy_wait<2>();
          else if (part == 2) copy_wait<1>();
          else copy_wait<0>();
        } else {
          copy_wait<3>();
        }
        const int end = min(per_thread, (part + 1) * per_part);
        for (int j = part * per_part; j < end; j += 2) {
          Unit<ZT> x, y;
          x.none(), y.none();
          const int i = j * threads + tid;
          if (i < mine) x.q = slot[i];
          if (i + threads < mine) y.q = slot[i + threads];
          sums.raise(fmaxf(sums.top, largest(x, y)), c);
          const F2 down = pair(-sums.top);
          F2 t[TEMPS];
#pragma unroll
          for (int k = 0; k < TEMPS; ++k) t[k] = pair(sums.s[k], 0.f);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const F2 d = add2(x.get(i), down), e = add2(y.get(i), down);
#pragma unroll
            for (int k = 0; k < TEMPS; ++k)
              t[k] = add2(t[k], add2(exp2_of(mul2(d, pair(c[k]))), exp2_of(mul2(e, pair(c[k])))));
          }
#pragma unroll
          for (int k = 0; k < TEMPS; ++k) sums.s[k] = sum2(t[k]);
          if constexpr (!GRAD) {
            if (next_live) {
              copy(next_from, next_units, j);
              if (j + 1 < end) copy(next_from, next_units, j + 1);
            }
          }
        }
        if constexpr (!GRAD) copy_commit();
      }
      if (single >= 0) {
        sums.raise(fmaxf(sums.top, edge), c);
#pragma unroll
        for (int k = 0; k < TEMPS; ++k) sums.s[k] += exp2_of((edge - sums.top) * c[k]);
      }
    } else if (!GRAD) {
      for (int part = 0; part < kParts; ++part) {
        for (int j = part * per_part; next_live && j < min(per_thread, (part + 1) * per_part); ++j)
          copy(next_from, next_units, j);
        copy_commit();
      }
    }
    // Over the warps of the row's CTAs; the teacher's, which each CTA has, over its own.
    const float warp_best = warp_max(best);
    size = warp_sum(size == 0.f ? 0.f : best == warp_best ? size : size * exp2_of((best - warp_best) * ct));
    if (live) sums.join_warp(c);
    if (lane == 0) teacher[parity][warp] = make_float2(warp_best, size);
    if (lane < a.ctas) {
      Part* to = &parts[parity][rank * warps + warp];
      if (a.ctas > 1) to = cluster.map_shared_rank(to, lane);
      to->top = sums.top, to->s[0] = sums.s[0], to->s[1] = sums.s[TEMPS - 1];
    }
    if (a.ctas > 1) cluster.sync();
    else __syncthreads();
    best = lane < warps ? teacher[parity][lane].x : -INFINITY;
    size = lane < warps ? teacher[parity][lane].y : 0.f;
    const float all_best = warp_max(best);
    size = warp_sum(size == 0.f ? 0.f : best == all_best ? size : size * exp2_of((best - all_best) * ct));
    best = all_best;
    const bool any = size != 0.f;  // NaN too
    const bool work = live && (any || hard);
    if (work) {
      Sums<TEMPS> all;
      for (int k = lane; k < a.ctas * warps; k += kWarp) {
        const Part p = parts[parity][k];
        const float to = fmaxf(all.top, p.top);
        all.raise(to, c);
#pragma unroll
        for (int i = 0; i < TEMPS; ++i) all.s[i] += p.s[i] * exp2_of((p.top - to) * c[i]);
      }
      all.join_warp(c);
      sums = all;
    }
    const float top = sums.top;
    // Nothing but -inf: no distribution.
    if (sums.s[0] == 0.f) sums.s[0] = sums.s[TEMPS - 1] = NAN;
    const float soft_sum = sums.s[0], hard_sum = sums.s[TEMPS - 1];
    // The terms of the loss, and what each entry takes off the gradient.
    float sum = 0.f;
    if (work && any) {
      const float log_size = logf(size), log_soft = logf(soft_sum), inv = 1.f / size;
      const float weight = a.soft_weight * a.temperature;
      for (int k = tid; k < a.top_k; k += threads) {
        if (id[k] < 0) {
          coef[k] = 0.f;
          continue;
        }
        const float d = coef[k] - best;
        const float p = exp2_of(d * ct) * inv;
        const float q = (zed[k] - top) * a.inv_temperature - log_soft;
        sum += zed[k] == -INFINITY ? INFINITY : p * (d * a.inv_temperature - log_size - q);
        coef[k] = weight * p * up;
      }
    } else if (GRAD && work) {
      for (int k = tid; k < a.top_k; k += threads) id[k] = -1;
    }
    if (GRAD && tid == 0) coef[a.top_k] = a.hard_weight * up;
    sum = warp_sum(sum);
    if (lane == 0) terms[parity][warp] = sum;
    if constexpr (GRAD) {
      const bool zero = !work || up == 0.f;
      float w[TEMPS];  // weights of the exponentials
      w[0] = soft ? (any ? up * a.soft_weight * a.temperature / soft_sum : 0.f) : 0.f;
      w[TEMPS - 1] = (TEMPS == 1 ? w[0] : 0.f) + (hard ? up * a.hard_weight / hard_sum : 0.f);
      const auto smooth = [&](F2 v) {
        const F2 d = add2(v, pair(-top));
        F2 g = mul2(exp2_of(mul2(d, pair(c[0]))), pair(w[0]));
        if constexpr (TEMPS == 2) g = fma2(exp2_of(mul2(d, pair(c[1]))), pair(w[1]), g);
        return g;
      };
      const auto smooth1 = [&](float v) {
        float lo, hi;
        split(smooth(pair(v)), lo, hi);
        return lo;
      };
      if (a.whole) {
        TG* to = grad + head + int64_t(rank) * a.slice * E;
        for (int part = 0; part < kParts; ++part) {
          for (int j = part * per_part; j < min(per_thread, (part + 1) * per_part); ++j) {
            const int i = j * threads + tid;
            if (i < mine) {
              Pack<GT, E> g;
              g.clear();
              if (!zero) {
                Unit<ZT> x;
                x.q = slot[i];
#pragma unroll
                for (int k = 0; k < E / 2; ++k) set2(g, k, smooth(x.get(k)));
              }
              g.store(to + int64_t(i) * E);
            }
            if (next_live) copy(next_from, next_units, j);
          }
          copy_commit();
        }
      } else {
        // Element by element; the next row may come when all are through.
        const TZ* from = reinterpret_cast<const TZ*>(slot);
        TG* to = grad + head + int64_t(rank) * a.slice * E;
        for (int i = tid; i < mine * E; i += threads)
          to[i] = zero ? TG(0) : from_float<GT>(smooth1(to_float<ZT>(from[i])));
        __syncthreads();
        for (int part = 0; part < kParts; ++part) {
          for (int j = part * per_part; next_live && j < min(per_thread, (part + 1) * per_part);
               ++j)
            copy(next_from, next_units, j);
          copy_commit();
        }
      }
      if (single >= 0) grad[single] = zero ? TG(0) : from_float<GT>(smooth1(edge));
      __syncthreads();
      if (!zero) {
        // All of a token's shares are taken off together, by each entry that names it.
        const int lo = rank * a.slice * E + head, hi = lo + max(mine, 0) * E;
        for (int k = tid; k <= a.top_k; k += threads) {
          const int token = id[k];
          const bool inside = token >= lo && token < hi;
          const bool end = rank == 0 && (token < head || token >= head + units * E);
          if (token < 0 || !(inside || end)) continue;
          float off = 0.f;
          for (int o = 0; o <= a.top_k; ++o) off += id[o] == token ? coef[o] : 0.f;
          grad[token] = from_float<GT>(smooth1(zed[k]) - off);
        }
      }
    } else {
      __syncthreads();
    }
    if (a.loss && rank == 0 && tid == 0) {
      float loss = 0.f;
      if (work && any) {
        for (int k = 0; k < warps; ++k) loss += terms[parity][k];
        // Without a distribution a masked token's term means nothing.
        if (soft_sum != soft_sum) loss = soft_sum;
        loss *= a.soft_weight * a.temperature * a.temperature;
      }
      if (work && hard) loss += a.hard_weight * (logf(hard_sum) - (zed[a.top_k] - top));
      a.loss[row] = loss;
    }
    label = next_label, up = next_up;
  }
  // No CTA leaves while another may store into it.
  if (a.ctas > 1) cluster.sync();
}

// The kernels of one type of logits: [type of grad][temperatures - 1], and without grad.
using DistillKernel = void (*)(DistillArgs);
struct DistillKernels {
  DistillKernel grad[3][2];
  DistillKernel loss[2];
};
template <int ZT>
constexpr DistillKernels distill_kernels() {
  return {{{distill_kernel<ZT, TRAIN_BF16, 1, true>, distill_kernel<ZT, TRAIN_BF16, 2, true>},
           {distill_kernel<ZT, TRAIN_FP16, 1, true>, distill_kernel<ZT, TRAIN_FP16, 2, true>},
           {distill_kernel<ZT, TRAIN_FP32, 1, true>, distill_kernel<ZT, TRAIN_FP32, 2, true>}},
          {distill_kernel<ZT, TRAIN_FP32, 1, false>, distill_kernel<ZT, TRAIN_FP32, 2, false>}};
}

// Each defined in a translation unit of its own.
const DistillKernels& distill_kernels_bf16();
const DistillKernels& distill_kernels_fp16();
const DistillKernels& distill_kernels_fp32();

}  // namespace traingb
