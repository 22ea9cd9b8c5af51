// The distillation loss of rows in shared memory (train_ops.h): the
// kernels, compiled once for each type of the logits.  Not part of the public
// interface.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

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
  int32_t bucket_bits;       // of a row's entries by their tokens
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

// Half the difference of two logits; logits further apart than fp32's largest number have
// one too.
__device__ __forceinline__ float half_apart(float x, float y) { return 0.5f * x - 0.5f * y; }

// An entry's term of the loss, soft_weight T^2 p (log p - log q), from the teacher's and
// the student's logit, the largest of each, and log of the student's sum less log of the
// teacher's.  The weight goes to p and T into the difference, so that a named token of the
// type's lowest value gives an infinite loss only where the loss is past fp32's range, and
// an entry with p = 0 gives 0.
__device__ __forceinline__ float soft_term(const DistillArgs& a, float p, float teacher, float best,
                                           float student, float top, float logs) {
  if (student == -INFINITY) return copysignf(INFINITY, a.soft_weight);
  const float half = half_apart(teacher, best) - half_apart(student, top);
  return a.soft_weight * a.temperature * p * (half + 0.5f * a.temperature * logs) * 2.f;
}
// The label's, hard_weight (log of the sum - (the label's logit - the largest)).
__device__ __forceinline__ float hard_term(const DistillArgs& a, float sum, float student,
                                           float top) {
  return a.hard_weight * (0.5f * logf(sum) - half_apart(student, top)) * 2.f;
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
template <int ZT, int N>
__device__ __forceinline__ float largest(const Unit<ZT> (&x)[N]) {
  if constexpr (ZT == TRAIN_FP32) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < N; ++k)
      m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(x[k].q.x), __uint_as_float(x[k].q.y))),
                fmaxf(__uint_as_float(x[k].q.z), __uint_as_float(x[k].q.w)));
    return m;
  } else {
    using H = std::conditional_t<ZT == TRAIN_BF16, __nv_bfloat162, __half2>;
    const auto as = [](const uint32_t& w) { return *reinterpret_cast<const H*>(&w); };
    H m = as(x[0].q.x);
#pragma unroll
    for (int k = 0; k < N; ++k)
      m = __hmax2(__hmax2(m, __hmax2(as(x[k].q.x), as(x[k].q.y))),
                  __hmax2(as(x[k].q.z), as(x[k].q.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

// The softmaxes that a row needs: one (one term, or both at temperature 1), two, or two
// of which the hard term's exponentials are the squares of the soft term's (at temperature
// 2: 196 us for 8192 x 32000, where two exponentials an element take 214 at temperature 3).
constexpr int kOne = 0, kTwo = 1, kSquares = 2;

// Sums of exponentials relative to a largest value.  That starts at the lowest finite
// one, so that it is never -inf.
template <int TERMS>
struct Sums {
  static constexpr int N = TERMS == kOne ? 1 : 2;
  float top = -FLT_MAX;
  float s[N] = {};
  // Factors that take sums relative to `top` to ones relative to `to`.
  static __device__ __forceinline__ void factors(float d, const float (&c)[N], float (&f)[N]) {
    f[0] = exp2_of(d * c[0]);
    if constexpr (TERMS == kTwo) f[1] = exp2_of(d * c[1]);
    if constexpr (TERMS == kSquares) f[1] = f[0] * f[0];
  }
  __device__ __forceinline__ void raise(float to, const float (&c)[N]) {
    float f[N];
    factors(top - to, c, f);
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] *= f[k];
    top = to;
  }
  // Over `lanes` neighbouring lanes.
  __device__ __forceinline__ void join(int lanes, const float (&c)[N]) {
    float to = top;
    for (int d = 1; d < lanes; d *= 2) to = fmaxf(to, __shfl_xor_sync(kAll, to, d));
    raise(to, c);
    for (int d = 1; d < lanes; d *= 2)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(kAll, s[k], d);
  }
};

constexpr int kDistillThreads = 256;
constexpr int kDistillWarps = kDistillThreads / kWarp;
constexpr int kMostCtas = 16;
constexpr int kAtOnce = 4;  // units a thread reads together
// Rows through a ring.
constexpr int kRingThreads = 128;  // a row, at most
constexpr int kRingCtas = 6;       // of as many, an SM
constexpr int kRingStages = 3;
constexpr int kChunk = kAtOnce * kWarp;  // units of a stage, a warp
constexpr int kRingBytes = kRingStages * kChunk * 16;  // a warp

// A row's slice is copied into shared memory asynchronously, in units of 16 bytes, and
// read there twice: once for the running largest value and sums of exponentials, once
// for the gradient, q = e^(z - max) / sum taken again rather than kept.  A thread reads
// back the units that it copied itself and, when it is through with its share, asks for
// the next row's in their place; that row has been on its way to L2 since the first
// barrier.  What is left at the row's ends goes to single threads of the first CTA, one
// element each.  The teacher's entries are fetched a row ahead; the tokens they name are
// written again, all of a token's shares together, when the others are done; entries that
// name the same token find one another in a table of buckets.
//
// Instructions bound it, not memory: two readings with unpacking, an exponential and four
// sums or products of pairs each take 12 an element, some 700 a row and warp come on top,
// and the warps that have entries keep the others waiting.  8192 x 32000 bf16 with 64
// entries takes 196 us at one temperature and at two (5.3 TB/s), without entries 174 (6.0
// TB/s).  Comparing all pairs of entries takes 4 us more; 4096 rows with 256 entries take 125
// us (167), with 1000 186 (620).  Without the prefetch into L2 the first was 20 us slower;
// 128 threads a CTA, or more parts of a row waited for one by one, were no quicker.
//
// RING: the loss of more rows than there is room for.  It needs a row once, so units come
// through a ring for each warp, those of the next row behind this one's without a pause; a
// row has one to four warps, which makes what a row costs besides its elements small, and
// may be of any length.  8192 x 32000 bf16 with 64 entries takes 86 us (6.1 TB/s; held whole
// 115), 16384 x 8192 50 (87), 4096 x 50,000 70 (93), 1021 x 131,071 fp16 56 (74); with
// four stages 90, 54, 71 and 54.
//   ZT, GT  types of logits and grad        TERMS  the softmaxes (kOne and so on)
template <int ZT, int GT, int TERMS, bool GRAD, bool RING>
__global__ void __launch_bounds__(RING ? kRingThreads : kDistillThreads, RING ? kRingCtas : 3)
    distill_kernel(const __grid_constant__ DistillArgs a) {
  namespace cg = cooperative_groups;
  using TZ = typename TypeOf<ZT>::T;
  using TG = typename TypeOf<GT>::T;
  constexpr int E = Unit<ZT>::E;
  extern __shared__ __align__(16) unsigned char smem[];
  struct Part {
    float top, s[2], spare;
  };
  __shared__ Part parts[2][RING ? kRingThreads / kWarp : kMostCtas * kDistillWarps];  // by the row's parity
  __shared__ float2 teacher[2][kDistillWarps];          // largest, sum
  __shared__ float terms[2][kDistillWarps];
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads / kWarp;
  const int warp = tid / kWarp, lane = tid % kWarp;
  const int vocab = a.vocab, room = (a.top_k + 4) / 4 * 4;
  const int rank = a.ctas == 1 ? 0 : int(blockIdx.x) % a.ctas;
  uint4* slot = reinterpret_cast<uint4*>(smem);
  const uint32_t slot_address = shared_address(smem);
  // Of each row's entries, twice by the row's parity: tokens, what they take off the
  // gradient, logits (`room` each), and for a gradient what is known of tokens named again;
  // then an entry for each bucket, of two kinds.
  unsigned char* lists = smem + (RING ? size_t(warps * kRingBytes) : size_t(a.slice) * 16);

  const bool soft = a.top_k > 0 && a.soft_weight != 0.f;
  const bool hard = a.labels && a.hard_weight != 0.f;
  // Scales of the exponents: the soft term's and, of two, behind it the hard term's.
  constexpr int N = Sums<TERMS>::N;
  float c[N];
  c[0] = soft ? a.inv_temperature * kLog2e : kLog2e;
  if constexpr (N == 2) c[1] = kLog2e;
  const float ct = a.inv_temperature * kLog2e;

  uint8_t* const marks = lists + 2 * 3 * 4 * room;
  uint16_t* const buckets = reinterpret_cast<uint16_t*>(marks + 2 * room);
  const auto bucket_of = [&](int token, int kind) {
    const uint32_t x = uint32_t(token) * (kind ? 2038074743u : 1000000007u);
    return (kind << a.bucket_bits) + int(x >> (32 - a.bucket_bits));
  };
  cg::cluster_group cluster = cg::this_cluster();
  if (a.ctas > 1) cluster.sync();  // all of its CTAs run now
  pdl_wait();

  const int64_t step = int64_t(gridDim.x) / a.ctas;
  // Each warp has a run of a slice's units, 32 side by side at a time.
  const int run = (a.slice + threads - 1) / threads * kWarp;
  const int first = warp * run;
  const int at0 = rank * a.slice;  // the slice's first unit
  const bool ends = a.phase != 0 || a.row_phase != 0 || vocab % E != 0;
  const auto head_of = [&](int64_t row) {
    return ends ? (E - (a.phase + int(row % E) * a.row_phase) % E) % E : 0;
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
  const auto mine_of = [&](int units) { return min(a.slice, units - at0); };
  const auto copy = [&](const TZ* from, int mine) {
    const int end = min(mine, first + run);
    uint32_t to = slot_address + (first + lane) * 16;
    from += (first + lane) * E;
    for (int i = first + lane; i < end; i += kAtOnce * kWarp) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (i + k * kWarp < end) copy_async<16>(to + k * (kWarp * 16), from + k * (kWarp * E));
      to += kAtOnce * kWarp * 16, from += kAtOnce * kWarp * E;
    }
    copy_commit();
  };
  // The ring: a warp's stages are side by side, and each thread reads back its own units.
  const uint4* stages = slot + warp * (kRingStages * kChunk) + lane;
  const int chunks = (run + kChunk - 1) / kChunk;  // a row
  const TZ* coming = nullptr;
  int coming_at = 0, coming_end = 0;  // units
  uint32_t in = 0, out = 0;           // stages
  const auto begin = [&](const TZ* from, int mine) {
    coming = from + int64_t(first + lane) * E;
    coming_at = first + lane, coming_end = min(mine, first + run);
  };
  const auto request = [&] {
    const uint32_t to = shared_address(stages + in * kChunk);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (coming_at + k * kWarp < coming_end)
        copy_async<16>(to + k * (kWarp * 16), coming + k * (kWarp * E));
    copy_commit();
    coming += kChunk * E, coming_at += kChunk;
    in = (in + 1) % kRingStages;
  };
  // The teacher's entry that this thread has of the first `threads` of a row.
  const auto entry_of = [&](int64_t row, int k, int64_t& i, float& t) {
    i = read_id(a.top_ids, row * a.ids_stride + k, a.ids64);
    by_type(a.top_type, [&](auto T) {
      constexpr int TT = decltype(T)::value;
      t = to_float<TT>(
          static_cast<const typename TypeOf<TT>::T*>(a.top_logits)[row * a.top_stride + k]);
    });
  };
  const bool has_entry = soft && tid < a.top_k;
  const int entry_warps = soft ? min(warps, (a.top_k + kWarp - 1) / kWarp) : 0;
  int64_t entry = -1;
  float entry_t = 0.f;
  int64_t row = int64_t(blockIdx.x) / a.ctas;
  bool live = false;
  if (row < a.n_rows) {
    look(row, label, up);
    live = live_of(label, up);
    if (has_entry) entry_of(row, tid, entry, entry_t);
    const int head = head_of(row);
    const int mine = live ? mine_of((vocab - head) / E) : 0;
    if constexpr (RING) begin(row_of(row) + head, mine);
    else copy(row_of(row) + head + int64_t(at0) * E, mine);
  }
  if constexpr (RING)
    for (int k = 1; k < kRingStages; ++k) request();
  int parity = 0;
  const TZ* z = row_of(row);
  TG* grad = GRAD ? static_cast<TG*>(a.grad) + row * a.grad_stride : nullptr;
  const int64_t step_z = step * a.stride, step_grad = GRAD ? step * a.grad_stride : 0;
  for (; row < a.n_rows; row += step, parity ^= 1, z += step_z, grad += step_grad) {
    int32_t* id = reinterpret_cast<int32_t*>(lists) + parity * 3 * room;
    float* coef = reinterpret_cast<float*>(id + room);
    float* zed = coef + room;
    uint8_t* mark = marks + parity * room;
    // Entries of one token meet in its buckets, where one of them stays: it stands for all,
    // and is marked if there are others.  An entry that finds another token's in both buckets
    // has to look through the list, as its token's others have.
    constexpr uint8_t kAlone = 0, kSearch = 1, kStoodFor = 2;
    const auto enter = [&](int k, int token) {
      mark[k] = kAlone;
      buckets[bucket_of(token, 0)] = buckets[bucket_of(token, 1)] = uint16_t(k);
    };
    const auto meet = [&](int k) {
      const int token = id[k];
      int held = buckets[bucket_of(token, 0)];
      if (id[held] != token) held = buckets[bucket_of(token, 1)];
      if (id[held] != token) mark[k] = kSearch;
      else if (held != k) mark[k] = kStoodFor, mark[held] = kSearch;
    };
    const int head = head_of(row), units = (vocab - head) / E;
    const int mine = mine_of(units);  // units here; < 0: none
    // The next row.
    const int64_t next = row + step;
    int64_t next_label = -1;
    float next_up = 0.f;
    const TZ* next_from = z + step_z + int64_t(at0) * E;
    bool next_live = false;
    int next_mine = 0;  // none if it is not read
    if (next < a.n_rows) {
      look(next, next_label, next_up);
      const int next_head = head_of(next);
      next_from += next_head;
      next_live = live_of(next_label, next_up);
      if (next_live) next_mine = mine_of((vocab - next_head) / E);
    }
    // The column of this thread's single element, if it has one.
    int single = -1;
    if (ends && rank == 0 && tid < kWarp) {
      if (tid < head) single = tid;
      else if (kWarp - 1 - tid < (vocab - head) % E) single = vocab - kWarp + tid;
    }
    // The teacher's entries.
    float best = -INFINITY, size = 0.f, entry_z = 0.f;
    const auto take = [&](int k, int64_t i, float t) {
      const bool valid = i >= 0 && i < vocab && t != -INFINITY;
      id[k] = valid ? int32_t(i) : -1;
      coef[k] = t;
      if (!valid) return false;
      if constexpr (GRAD) enter(k, int32_t(i));
      if (t > best) {
        size = size * exp2_of((best - t) * ct) + 1.f;
        best = t;
      } else {
        size += t == best && t < INFINITY ? 1.f : exp2_of((t - best) * ct);
      }
      return true;
    };
    if (live && has_entry) {
      if (take(tid, entry, entry_t)) entry_z = to_float<ZT>(z[entry]);
      for (int k = tid + threads; k < a.top_k; k += threads) {
        int64_t i;
        float t;
        entry_of(row, k, i, t);
        if (take(k, i, t)) zed[k] = to_float<ZT>(z[i]);
      }
    }
    // The next row's, while this one is worked on.
    if (has_entry && next < a.n_rows) entry_of(next, tid, entry, entry_t);
    float edge = -INFINITY;
    if (live && single >= 0) edge = to_float<ZT>(z[single]);
    float label_z = 0.f;
    if (tid == 0) {
      for (int k = a.top_k; k < room; ++k) id[k] = -1;
      if (live && hard) {
        id[a.top_k] = int32_t(label), label_z = to_float<ZT>(z[label]);
        if constexpr (GRAD) enter(a.top_k, int32_t(label));
      }
    }
    // The largest value and the sums.
    Sums<TERMS> sums;
    // Adds kAtOnce units, 32 apart; `i` is the first's place among the `end` of this warp.
    const auto add = [&](const uint4* from, int i, int end) {
      Unit<ZT> x[kAtOnce];
      if (i + (kAtOnce - 1) * kWarp < end) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) x[k].q = from[k * kWarp];
      } else {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          x[k].none();
          if (i + k * kWarp < end) x[k].q = from[k * kWarp];
        }
      }
      sums.raise(fmaxf(sums.top, largest(x)), c);
      const F2 down = pair(-sums.top);
      // In a ring, where a thread has more of a row, of these alone, for short chains of
      // additions.
      F2 t[N];
      if constexpr (!RING)
#pragma unroll
        for (int n = 0; n < N; ++n) t[n] = pair(sums.s[n], 0.f);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
        for (int h = 0; h < E / 2; ++h) {
          const F2 d = add2(x[k].get(h), down);
          const F2 e = exp2_of(mul2(d, pair(c[0])));
          const bool begun = !RING || k + h > 0;
          t[0] = begun ? add2(t[0], e) : e;
          if constexpr (TERMS == kTwo) {
            const F2 e1 = exp2_of(mul2(d, pair(c[1])));
            t[1] = begun ? add2(t[1], e1) : e1;
          }
          if constexpr (TERMS == kSquares) t[1] = begun ? fma2(e, e, t[1]) : mul2(e, e);
        }
#pragma unroll
      for (int n = 0; n < N; ++n) sums.s[n] = (RING ? sums.s[n] : 0.f) + sum2(t[n]);
    };
    if constexpr (RING) {
      const int end = min(mine, first + run);
      for (int k = 0, i = first + lane; k < chunks; ++k, i += kChunk) {
        if (k + kRingStages - 1 == chunks) begin(next_from, next_mine);
        request();
        copy_wait<kRingStages - 1>();
        if (live && i < end) add(stages + out * kChunk, i, end);
        out = (out + 1) % kRingStages;
      }
    }
    if (live) {
      if constexpr (!RING) {
        copy_wait<0>();
        const int end = min(mine, first + run);
        for (int i = first + lane; i < end; i += kChunk) add(slot + i, i, end);
        if constexpr (!GRAD) copy(next_from, next_mine);
      }
      if (single >= 0) {
        sums.raise(fmaxf(sums.top, edge), c);
        float f[N];
        sums.factors(edge - sums.top, c, f);
#pragma unroll
        for (int n = 0; n < N; ++n) sums.s[n] += f[n];
      }
    } else if (!GRAD && !RING) {
      copy(next_from, next_mine);
    }
    // Over the warps of the row's CTAs; the teacher's, which each CTA has, over its own.
    const auto join_teacher = [&](int lanes) {
      float to = best;
      for (int d = 1; d < lanes; d *= 2) to = fmaxf(to, __shfl_xor_sync(kAll, to, d));
      if (best != to && size != 0.f) size *= exp2_of((best - to) * ct);
      for (int d = 1; d < lanes; d *= 2) size += __shfl_xor_sync(kAll, size, d);
      best = to;
    };
    if (live) sums.join(kWarp, c);
    if (warp < entry_warps) {
      if (has_entry) zed[tid] = entry_z;
      join_teacher(kWarp);
      if (lane == 0) teacher[parity][warp] = make_float2(best, size);
    }
    if (tid == 0) zed[a.top_k] = label_z;
    if (lane < a.ctas) {
      Part* to = &parts[parity][rank * warps + warp];
      if (a.ctas > 1) to = cluster.map_shared_rank(to, lane);
      to->top = sums.top, to->s[0] = sums.s[0], to->s[1] = sums.s[N - 1];
    }
    if (a.ctas > 1) cluster.sync();
    else __syncthreads();
    // The next row is on its way to L2 from here on, and to shared memory as room is made there.
    if (!RING && tid == 0 && next_mine > 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(next_from),
                   "r"(next_mine * 16)
                   : "memory");
    if (soft) {
      best = -INFINITY, size = 0.f;
      if ((lane & (warps - 1)) < entry_warps) {
        const float2 p = teacher[parity][lane & (warps - 1)];
        best = p.x, size = p.y;
      }
      join_teacher(warps);
    }
    const bool any = size != 0.f;  // NaN too
    const bool work = live && (any || hard);
    if (work) {
      const int held = a.ctas * warps;  // a power of two
      Part p = parts[parity][lane & (held - 1)];
      sums.top = p.top, sums.s[0] = p.s[0], sums.s[N - 1] = p.s[N - 1];
      for (int k = kWarp; k < held; k += kWarp) {
        p = parts[parity][k + lane];
        const float to = fmaxf(sums.top, p.top);
        float f[N];
        sums.raise(to, c);
        sums.factors(p.top - to, c, f);
#pragma unroll
        for (int n = 0; n < N; ++n) sums.s[n] += p.s[n] * f[n];
      }
      sums.join(min(held, kWarp), c);
    }
    const float top = sums.top;
    // Nothing but -inf: no distribution.
    if (sums.s[0] == 0.f) sums.s[0] = sums.s[N - 1] = NAN;
    const float soft_sum = sums.s[0], hard_sum = sums.s[N - 1];
    // The terms of the loss, and what each entry takes off the gradient.
    if (warp < entry_warps && work && any) {
      float sum = 0.f;
      const float logs = logf(soft_sum) - logf(size), inv = 1.f / size;
      const float weight = a.soft_weight * a.temperature * up;
      for (int k = tid; k < a.top_k; k += threads) {
        if (id[k] < 0) {
          coef[k] = 0.f;
          continue;
        }
        const float d = coef[k] - best;
        const float p = exp2_of(d * ct) * inv;
        sum += soft_term(a, p, coef[k], best, zed[k], top, logs);
        coef[k] = weight * p;
        if constexpr (GRAD) meet(k);
      }
      sum = warp_sum(sum);
      if (lane == 0) terms[parity][warp] = sum;
    } else if (GRAD && work && !any) {
      for (int k = tid; k < a.top_k; k += threads) id[k] = -1;
    }
    if (GRAD && tid == 0) {
      coef[a.top_k] = a.hard_weight * up;
      if (work && any && id[a.top_k] >= 0) meet(a.top_k);
    }
    if constexpr (GRAD) {
      const bool zero = !work || up == 0.f;
      float w[N];  // weights of the exponentials
      w[0] = soft && any ? __fdividef(up * a.soft_weight * a.temperature, soft_sum) : 0.f;
      w[N - 1] = (N == 1 ? w[0] : 0.f) + (hard ? __fdividef(up * a.hard_weight, hard_sum) : 0.f);
      const auto smooth = [&](F2 v) {
        const F2 d = add2(v, pair(-top));
        const F2 e = exp2_of(mul2(d, pair(c[0])));
        if constexpr (TERMS == kSquares) return mul2(e, fma2(e, pair(w[1]), pair(w[0])));
        const F2 g = mul2(e, pair(w[0]));
        if constexpr (TERMS == kTwo)
          return fma2(exp2_of(mul2(d, pair(c[1]))), pair(w[1]), g);
        return g;
      };
      const auto smooth1 = [&](float v) {
        float lo, hi;
        split(smooth(pair(v)), lo, hi);
        return lo;
      };
      TG* to = grad + head + int64_t(at0) * E;
      if (a.whole) {
        const int end = min(mine, first + run);
        TG* out = to + (first + lane) * E;
        if (zero) {
          Pack<GT, E> g;
          g.clear();
          for (int i = first + lane; i < end; i += kWarp, out += kWarp * E) g.store(out);
        } else {
          constexpr int U = 2;
          for (int i = first + lane; i < end; i += U * kWarp, out += U * kWarp * E) {
            Unit<ZT> x[U];
#pragma unroll
            for (int k = 0; k < U; ++k) x[k].q = slot[min(i + k * kWarp, end - 1)];
#pragma unroll
            for (int k = 0; k < U; ++k) {
              Pack<GT, E> g;
#pragma unroll
              for (int h = 0; h < E / 2; ++h) set2(g, h, smooth(x[k].get(h)));
              if (i + k * kWarp < end) g.store(out + k * (kWarp * E));
            }
          }
        }
        copy(next_from, next_mine);
      } else {
        // Element by element; the next row may come when all are through.  8192 x 32000 bf16
        // takes 375 us this way and 195 by units, 1021 x 131,071 fp16 193 and 107.
        const TZ* from = reinterpret_cast<const TZ*>(slot);
        for (int i = tid; i < mine * E; i += threads)
          to[i] = zero ? TG(0) : from_float<GT>(smooth1(to_float<ZT>(from[i])));
        __syncthreads();
        copy(next_from, next_mine);
      }
      if (single >= 0) grad[single] = zero ? TG(0) : from_float<GT>(smooth1(edge));
      __syncthreads();
      if (!zero) {
        // All of a token's shares are taken off together.
        const int lo = rank * a.slice * E + head, hi = lo + max(mine, 0) * E;
        for (int k = tid; k <= a.top_k; k += threads) {
          const int token = id[k];
          const bool inside = token >= lo && token < hi;
          const bool end = rank == 0 && (token < head || token >= head + units * E);
          if (token < 0 || mark[k] == kStoodFor || !(inside || end)) continue;
          float off = coef[k];
          if (mark[k] == kSearch) {
            off = 0.f;
            for (int o = 0; o < room; o += 4) {
              const int4 i = *reinterpret_cast<const int4*>(id + o);
              if (i.x == token) off += coef[o];
              if (i.y == token) off += coef[o + 1];
              if (i.z == token) off += coef[o + 2];
              if (i.w == token) off += coef[o + 3];
            }
          }
          grad[token] = from_float<GT>(smooth1(zed[k]) - off);
        }
      }
    } else {
      __syncthreads();
    }
    if (a.loss && rank == 0 && tid == 0) {
      float loss = 0.f;
      if (work && any) {
        for (int k = 0; k < entry_warps; ++k) loss += terms[parity][k];
        // Without a distribution a masked token's term means nothing.
        if (soft_sum != soft_sum) loss = soft_sum;
      }
      if (work && hard) loss += hard_term(a, hard_sum, zed[a.top_k], top);
      a.loss[row] = loss;
    }
    label = next_label, up = next_up, live = next_live;
  }
  // No CTA leaves while another may store into it.
  if (a.ctas > 1) cluster.sync();
}

// The kernels of one type of logits: [type of grad][terms], and without grad.
using DistillKernel = void (*)(DistillArgs);
struct DistillKernels {
  DistillKernel grad[3][3];
  DistillKernel loss[3];
  DistillKernel ring[3];  // the loss of many rows
};
template <int ZT>
constexpr DistillKernels distill_kernels() {
  return {{{distill_kernel<ZT, TRAIN_BF16, kOne, true, false>, distill_kernel<ZT, TRAIN_BF16, kTwo, true, false>,
            distill_kernel<ZT, TRAIN_BF16, kSquares, true, false>},
           {distill_kernel<ZT, TRAIN_FP16, kOne, true, false>, distill_kernel<ZT, TRAIN_FP16, kTwo, true, false>,
            distill_kernel<ZT, TRAIN_FP16, kSquares, true, false>},
           {distill_kernel<ZT, TRAIN_FP32, kOne, true, false>, distill_kernel<ZT, TRAIN_FP32, kTwo, true, false>,
            distill_kernel<ZT, TRAIN_FP32, kSquares, true, false>}},
          {distill_kernel<ZT, TRAIN_FP32, kOne, false, false>, distill_kernel<ZT, TRAIN_FP32, kTwo, false, false>,
           distill_kernel<ZT, TRAIN_FP32, kSquares, false, false>},
          {distill_kernel<ZT, TRAIN_FP32, kOne, false, true>,
           distill_kernel<ZT, TRAIN_FP32, kTwo, false, true>,
           distill_kernel<ZT, TRAIN_FP32, kSquares, false, true>}};
}

// Each defined in a translation unit of its own.
const DistillKernels& distill_kernels_bf16();
const DistillKernels& distill_kernels_fp16();
const DistillKernels& distill_kernels_fp32();

}  // namespace traingb
