// The embedding lookup with scaling and its gradient (train_ops.h).
#include <cooperative_groups.h>

#include <string>

#include "lamb_internal.h"
#include "train_internal.h"

using namespace traingb;
namespace cg = cooperative_groups;

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

// --------------------------------------------------------------- gradient
// G[v, :] = scale * sum over the positions i with row(ids[i]) = v of dy[i, :].
// The positions are sorted by row (stably, so ascending within a row), and the
// sorted list is cut into blocks of C positions.  A warp takes one block and
// a slab of up to 256 columns, streams the rows of dy that its positions name
// and adds each run of equal rows in registers.  A run that ends in the next
// block at the latest is finished by the warp of the block it starts in.  A
// longer one (a frequent token) is cut at the block boundaries: each piece's
// fp32 sum goes to a slot of the workspace, and join_kernel adds the pieces in
// order.  So no warp adds more than 2 C rows whatever the tokens are, only
// long runs pay for slots, and the order of every sum depends on the ids and
// the sizes alone.

constexpr int kWarp = 32;
constexpr unsigned kAll = 0xffffffffu;

struct GradArgs {
  const void* dy;
  void* grad;
  const uint32_t* keys;  // sorted rows; n_rows for tokens that add nothing
  const uint32_t* pos;   // their positions
  float* slots;          // [2 * block + (0: run from an earlier block, 1: starts here)][slot_dim]
  int64_t dy_stride, grad_stride, n_rows, dim, slot_dim;
  int64_t n;
  int64_t n_blocks;
  int64_t sum_units, fill_units;  // warps that add, warps that write zero rows
  int32_t block, slabs;           // C, slabs of columns
  float scale;
  int32_t accumulate, out_type;
};

__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// VEC neighbouring elements, aligned to their size together (at most 16 bytes
// at a time).
template <int DT, int VEC>
struct Pack {
  using T = typename TypeOf<DT>::T;
  static constexpr int kBytes = VEC * int(sizeof(T));
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == TRAIN_FP32) return __uint_as_float(w[i]);
    const uint32_t x = (i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    return to_float<DT == TRAIN_FP32 ? TRAIN_BF16 : DT>(uint16_t(x));
  }
};

// Loads and stores of VEC neighbouring values of a type known at run time.
template <int VEC>
__device__ __forceinline__ void load_values(const void* p, int type, float (&x)[VEC]) {
  if (type == TRAIN_FP32) {
    const float* q = static_cast<const float*>(p);
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(q + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = q[i];
    }
    return;
  }
  uint16_t h[VEC];
  const uint16_t* q = static_cast<const uint16_t*>(p);
  if constexpr (VEC == 8) *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(q);
  else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(q);
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(h) = *reinterpret_cast<const uint32_t*>(q);
  else h[0] = q[0];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    x[i] = type == TRAIN_BF16 ? to_float<TRAIN_BF16>(h[i]) : to_float<TRAIN_FP16>(h[i]);
}

template <int VEC>
__device__ __forceinline__ void store_values(void* p, int type, const float (&x)[VEC]) {
  if (type == TRAIN_FP32) {
    float* q = static_cast<float*>(p);
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        *reinterpret_cast<float4*>(q + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) q[i] = x[i];
    }
    return;
  }
  alignas(16) uint16_t h[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    h[i] = type == TRAIN_BF16 ? from_float<TRAIN_BF16>(x[i]) : from_float<TRAIN_FP16>(x[i]);
  uint16_t* q = static_cast<uint16_t*>(p);
  if constexpr (VEC == 8) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(h);
  else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(h);
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(q) = *reinterpret_cast<const uint32_t*>(h);
  else q[0] = h[0];
}

__device__ __forceinline__ char* grad_at(const GradArgs& a, int64_t row, int64_t col) {
  return static_cast<char*>(a.grad) + (row * a.grad_stride + col) * size_of(a.out_type);
}

// grad[row, col ..] = round(old + scale * sum)
template <int VEC>
__device__ __forceinline__ void finish_row(const GradArgs& a, int64_t row, int64_t col,
                                           const float* acc) {
  void* p = grad_at(a, row, col);
  float x[VEC];
  if (a.accumulate) {
    load_values<VEC>(p, a.out_type, x);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = fmaf(a.scale, acc[i], x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = a.scale * acc[i];
  }
  store_values<VEC>(p, a.out_type, x);
}

// First index with keys[index] >= row.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t row) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < row) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A warp writes zeros to bytes bytes at p.
__device__ __forceinline__ void warp_zero(char* p, int64_t bytes, int lane) {
  const int64_t head = min(int64_t((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), bytes);
  for (int64_t i = 2 * lane; i < head; i += 2 * kWarp) *reinterpret_cast<uint16_t*>(p + i) = 0;
  char* q = p + head;
  const int64_t body = (bytes - head) / 16;
  for (int64_t i = lane; i < body; i += kWarp)
    reinterpret_cast<uint4*>(q)[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = 16 * body + 2 * lane; i < bytes - head; i += 2 * kWarp)
    *reinterpret_cast<uint16_t*>(q + i) = 0;
}

// Zeros the rows r0 .. r0 + 31 that no token names.
__device__ __forceinline__ void fill_rows(const GradArgs& a, int64_t r0, int lane) {
  const int64_t row = r0 + lane;
  bool idle = row < a.n_rows;
  if (idle) {
    const int64_t at = lower_bound(a.keys, a.n, uint32_t(row));
    idle = at >= a.n || a.keys[at] != uint32_t(row);
  }
  unsigned todo = __ballot_sync(kAll, idle);
  while (todo) {
    const int k = __ffs(todo) - 1;
    todo &= todo - 1;
    warp_zero(grad_at(a, r0 + k, 0), a.dim * size_of(a.out_type), lane);
  }
}

// VEC neighbouring columns a load, GROUPS loads a lane and row; a warp covers
// 32 * VEC * GROUPS columns.
template <int IN, int VEC, int GROUPS>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ GradArgs a) {
  using TI = typename TypeOf<IN>::T;
  constexpr int kCols = VEC * GROUPS;
  constexpr int kRows = 8;  // rows of dy in flight
  const int lane = threadIdx.x & 31;
  const int64_t unit = int64_t(blockIdx.x) * (kThreads / kWarp) + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (unit >= a.sum_units) {
    if (unit < a.sum_units + a.fill_units) fill_rows(a, (unit - a.sum_units) * kWarp, lane);
    return;
  }
  const int64_t b = unit / a.slabs;
  const int64_t col0 = (unit % a.slabs) * (kWarp * kCols) + lane * VEC;
  const int64_t C = a.block, n = a.n;
  const int64_t lo = b * C, hi = min(lo + C, n);
  const uint32_t none = uint32_t(a.n_rows);
  const uint32_t first = a.keys[lo], last = a.keys[hi - 1];
  if (first == none) return;
  // The run that reaches in from the block before: a piece of a long run, or
  // finished by its own block.
  const bool from_before = lo > 0 && a.keys[lo - 1] == first;
  const bool head_piece = from_before && ((hi < n && a.keys[hi] == first) ||
                                          (lo > C && a.keys[lo - C - 1] == first));
  // The run that starts here and reaches out: into the next block at most, or
  // long.
  const bool reaches_out =
      hi < n && last != none && a.keys[hi] == last && !(from_before && first == last);
  const bool tail_piece = reaches_out && hi + C < n && a.keys[hi + C] == last;
  const int64_t end = reaches_out && !tail_piece ? min(hi + C, n) : hi;
  bool skip = from_before && !head_piece;  // until the first other row
  bool head = head_piece;                  // adding the piece from before
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;

  for (int64_t x0 = lo; x0 < end; x0 += kWarp) {
    const int64_t x = x0 + lane;
    uint32_t key = none, next = none, at = 0;
    if (x < end) {
      key = a.keys[x];
      at = a.pos[x];
      if (x + 1 < n) next = a.keys[x + 1];
    }
    // Positions to add: real rows, not those of a run finished elsewhere; past
    // hi only those of the run that reaches out.
    const bool wanted = key != none && !(skip && key == first) && (x < hi || key == last);
    const unsigned use = __ballot_sync(kAll, wanted);
    const unsigned ends = __ballot_sync(kAll, wanted && key != next);
    if (skip && !__all_sync(kAll, key == first)) skip = false;
    int k = use ? __ffs(use) - 1 : kWarp;
    const int stop = use ? kWarp - __clz(use) : 0;
    while (k < stop) {
      // The wanted positions are neighbours: kRows of them at a time.
      Pack<IN, VEC> q[kRows][GROUPS];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t p = __shfl_sync(kAll, at, (k + r) & 31);
        const TI* src = static_cast<const TI*>(a.dy) + int64_t(p) * a.dy_stride + col0;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          if (k + r < stop && col0 + g * (kWarp * VEC) < a.dim)
            q[r][g].load(src + g * (kWarp * VEC));
          else
            q[r][g].clear();
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (k + r < stop) {
#pragma unroll
          for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[g * VEC + i] += q[r][g].get(i);
          if ((ends >> (k + r)) & 1u) {
            const int64_t row = __shfl_sync(kAll, key, k + r);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
              const int64_t col = col0 + g * (kWarp * VEC);
              if (col < a.dim) {
                if (head) {
                  float* s = a.slots + 2 * b * a.slot_dim + col;
#pragma unroll
                  for (int i = 0; i < VEC; ++i) s[i] = acc[g * VEC + i];
                } else {
                  finish_row<VEC>(a, row, col, acc + g * VEC);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
            head = false;
          }
        }
      }
      k += kRows;
    }
  }
  // What is left in the registers is a piece of a run that goes on.
  if (head || tail_piece) {
    float* s = a.slots + (2 * b + (head ? 0 : 1)) * a.slot_dim;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int64_t col = col0 + g * (kWarp * VEC);
      if (col < a.dim) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[col + i] = acc[g * VEC + i];
      }
    }
  }
}

// Adds the pieces of every long run, in order.  A CTA takes 32 columns (grid
// x) and every gridDim.y-th long run: its warps add neighbouring shares of the
// pieces, and the first warp adds the warps' sums.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(kJoinWarps* kWarp) join_kernel(
    const __grid_constant__ GradArgs a) {
  __shared__ float part[kJoinWarps][kWarp];
  __shared__ int64_t found[kJoinWarps * kWarp];
  __shared__ int count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = int64_t(blockIdx.x) * kWarp + lane;
  const int64_t C = a.block, n = a.n;
  const uint32_t none = uint32_t(a.n_rows);
  int64_t seen = 0;
  pdl_wait();
  for (int64_t b0 = 0; b0 < a.n_blocks; b0 += kJoinWarps * kWarp) {
    // Blocks in which a long run starts, in ascending order.
    const int64_t b = b0 + threadIdx.x;
    bool starts = false;
    if (b < a.n_blocks && (b + 2) * C < n) {
      const uint32_t last = a.keys[(b + 1) * C - 1];
      starts = last != none && a.keys[(b + 2) * C] == last &&
               (b == 0 || a.keys[b * C - 1] != last);
    }
    int at = __syncthreads_count(starts);
    if (at == 0) continue;
    // Rank of this block among them: blocks of the warps before, then lanes.
    const unsigned mask = __ballot_sync(kAll, starts);
    if (lane == 0) part[warp][0] = float(__popc(mask));
    __syncthreads();
    int before = __popc(mask & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += int(part[w][0]);
    if (starts) found[before] = b;
    if (threadIdx.x == 0) count = at;
    __syncthreads();
    const int all = count;
    for (int k = 0; k < all; ++k, ++seen) {
      if (seen % gridDim.y != blockIdx.y) continue;
      const int64_t from = found[k];
      const uint32_t row = a.keys[(from + 1) * C - 1];
      const int64_t run_end = lower_bound(a.keys, n, row + 1);
      const int64_t pieces = (run_end - 1) / C - from + 1;
      const int64_t share = (pieces + kJoinWarps - 1) / kJoinWarps;
      const int64_t p0 = warp * share, p1 = min(p0 + share, pieces);
      float acc = 0.0f;
      if (col < a.dim) {
#pragma unroll 8
        for (int64_t p = p0; p < p1; ++p)
          acc += a.slots[(2 * (from + p) + (p == 0 ? 1 : 0)) * a.slot_dim + col];
      }
      __syncthreads();
      part[warp][lane] = acc;
      __syncthreads();
      if (warp == 0 && col < a.dim) {
        float total[1] = {0.0f};
        for (int w = 0; w < kJoinWarps; ++w) total[0] += part[w][lane];
        finish_row<1>(a, row, col, total);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- sorting
// Stable radix sort of the positions by row, lowest digit first, up to 8 bits
// a pass.  Keys are rows; tokens that add nothing have the key n_rows.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / kWarp;
constexpr int kDigits = 256;

struct SortArgs {
  const void* ids;
  int64_t n, first_row, n_rows, padding;
  uint32_t* keys;
  uint32_t* pos;
  int32_t bits, passes;  // of the keys; digits of (bits + passes - 1) / passes bits
};

template <class ID>
__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i) {
  const ID id = static_cast<const ID*>(a.ids)[i];
  const int64_t row = row_of(id, a.first_row, a.n_rows);
  return row < 0 || int64_t(id) == a.padding ? uint32_t(a.n_rows) : uint32_t(row);
}

struct RankSmem {
  uint16_t warp_count[kSortWarps][kDigits];
  uint16_t part[4][kDigits];
  uint32_t total[kDigits];
  uint32_t base[kDigits];
  uint32_t scan[kDigits / kWarp];
};

// Ranks of a CTA's elements among those of equal digit.  Element j of a lane
// stands at place warp * 32 * ITEMS + 32 * j + lane of the CTA.  On return
// rank[j] counts the equal digits before it in its warp, warp_count[w][d] those
// in the warps before w, and total[d] those in the CTA.
template <int ITEMS>
__device__ __forceinline__ void rank_digits(RankSmem& s, const uint32_t (&digit)[ITEMS],
                                            uint32_t (&rank)[ITEMS]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* z = reinterpret_cast<uint32_t*>(s.warp_count[warp]);
#pragma unroll
  for (int i = 0; i < kDigits / 2 / kWarp; ++i) z[lane + kWarp * i] = 0u;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const unsigned peers = __match_any_sync(kAll, digit[j]);
    const int leader = __ffs(peers) - 1;
    uint32_t old = 0;
    if (lane == leader) {
      old = s.warp_count[warp][digit[j]];
      s.warp_count[warp][digit[j]] = uint16_t(old + __popc(peers));
    }
    __syncwarp();
    rank[j] = __shfl_sync(kAll, old, leader) + __popc(peers & ((1u << lane) - 1u));
  }
  __syncthreads();
  // Per digit, the exclusive sum over the warps: a quarter of them a thread.
  constexpr int kQuarter = kSortWarps / 4;
  const int d = threadIdx.x & (kDigits - 1), quarter = threadIdx.x / kDigits;
  uint32_t sum = 0, got[kQuarter];
#pragma unroll
  for (int w = 0; w < kQuarter; ++w) {
    got[w] = s.warp_count[quarter * kQuarter + w][d];
    sum += got[w];
  }
  s.part[quarter][d] = uint16_t(sum);
  __syncthreads();
  uint32_t before = 0;
  for (int q = 0; q < quarter; ++q) before += s.part[q][d];
  if (quarter == 3) s.total[d] = before + sum;
#pragma unroll
  for (int w = 0; w < kQuarter; ++w) {
    s.warp_count[quarter * kQuarter + w][d] = uint16_t(before);
    before += got[w];
  }
}

// base[d] = mine + sum of all[d'] over d' < d, for the first 256 threads; every
// thread of the CTA calls it.
__device__ __forceinline__ void digit_bases(RankSmem& s, uint32_t all, uint32_t mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = all;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (warp < kDigits / kWarp && lane == kWarp - 1) s.scan[warp] = x;
  __syncthreads();
  if (warp < kDigits / kWarp) {
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += s.scan[w];
    s.base[threadIdx.x] = before + x - all + mine;
  }
  __syncthreads();
}

// Up to 8 * 1024 * ITEMS positions in one cluster: every CTA holds a tile of
// 1024 * ITEMS elements in registers and shared memory, the CTAs exchange their
// digit counts, and each pass scatters through distributed shared memory; the
// last one writes to global memory.
template <int ITEMS, class ID>
__global__ void __launch_bounds__(kSortThreads) cluster_sort_kernel(
    const __grid_constant__ SortArgs a) {
  constexpr int kTile = kSortThreads * ITEMS;
  extern __shared__ __align__(16) unsigned char raw[];
  RankSmem& s = *reinterpret_cast<RankSmem*>(raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(raw + sizeof(RankSmem));
  uint32_t* pos = keys + kTile;
  cg::cluster_group cluster = cg::this_cluster();
  const int me = int(cluster.block_rank()), ctas = int(cluster.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  const int width = (a.bits + a.passes - 1) / a.passes;
  const uint32_t mask = (1u << width) - 1u;
  const int local0 = warp * (kWarp * ITEMS) + lane;
  uint32_t key[ITEMS], at[ITEMS], digit[ITEMS], rank[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int64_t i = int64_t(me) * kTile + local0 + kWarp * j;
    at[j] = uint32_t(i);
    // Behind the last token: the largest digits, so these stay behind it.
    key[j] = i < a.n ? key_of<ID>(a, i) : 0xffffffffu;
  }
  for (int p = 0; p < a.passes; ++p) {
    if (p > 0) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        key[j] = keys[local0 + kWarp * j];
        at[j] = pos[local0 + kWarp * j];
      }
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) digit[j] = (key[j] >> (p * width)) & mask;
    rank_digits<ITEMS>(s, digit, rank);
    cluster.sync();  // the counts are there, and the tiles have been read
    uint32_t all = 0, mine = 0;
    if (threadIdx.x < kDigits) {
      for (int r = 0; r < ctas; ++r) {
        const uint32_t x = cluster.map_shared_rank(s.total, r)[threadIdx.x];
        if (r < me) mine += x;
        all += x;
      }
    }
    digit_bases(s, all, mine);
    const bool out = p == a.passes - 1;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t to = s.base[digit[j]] + s.warp_count[warp][digit[j]] + rank[j];
      if (out) {
        if (to < a.n) {
          a.keys[to] = key[j];
          a.pos[to] = at[j];
        }
      } else {
        cluster.map_shared_rank(keys, int(to / kTile))[to % kTile] = key[j];
        cluster.map_shared_rank(pos, int(to / kTile))[to % kTile] = at[j];
      }
    }
    cluster.sync();  // the tiles are written, and the counts have been read
  }
}

// More positions than a cluster holds: three kernels a pass.  Counts of every
// tile's digits; their sums over the tiles, a CTA a digit; and the scatter.
constexpr int kTileItems = 4;
constexpr int kGlobalTile = kSortThreads * kTileItems;

struct PassArgs {
  SortArgs s;
  const uint32_t* keys_in;  // NULL: from the ids
  const uint32_t* pos_in;
  uint32_t* keys_out;
  uint32_t* pos_out;
  uint32_t* counts;  // [digit][tile]
  uint32_t* totals;  // [digit]
  int64_t tiles;
  int32_t shift, width;
};

template <class ID>
__device__ __forceinline__ void load_tile(const PassArgs& a, uint32_t (&key)[kTileItems],
                                          uint32_t (&at)[kTileItems],
                                          uint32_t (&digit)[kTileItems]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int64_t i = int64_t(blockIdx.x) * kGlobalTile + warp * (kWarp * kTileItems) +
                      kWarp * j + lane;
    key[j] = 0xffffffffu;
    at[j] = 0;
    if (i < a.s.n) {
      key[j] = a.keys_in ? a.keys_in[i] : key_of<ID>(a.s, i);
      at[j] = a.keys_in ? a.pos_in[i] : uint32_t(i);
    }
    digit[j] = (key[j] >> a.shift) & ((1u << a.width) - 1u);
  }
}

template <class ID>
__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ PassArgs a) {
  __shared__ RankSmem s;
  uint32_t key[kTileItems], at[kTileItems], digit[kTileItems], rank[kTileItems];
  load_tile<ID>(a, key, at, digit);
  rank_digits<kTileItems>(s, digit, rank);
  __syncthreads();
  if (threadIdx.x < kDigits) a.counts[threadIdx.x * a.tiles + blockIdx.x] = s.total[threadIdx.x];
}

__global__ void __launch_bounds__(kSortThreads) scan_kernel(const __grid_constant__ PassArgs a) {
  __shared__ uint32_t sums[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* c = a.counts + blockIdx.x * a.tiles;
  uint32_t carry = 0;
  for (int64_t t0 = 0; t0 < a.tiles; t0 += kSortThreads) {
    const int64_t t = t0 + threadIdx.x;
    const uint32_t v = t < a.tiles ? c[t] : 0u;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += y;
    }
    if (lane == kWarp - 1) sums[warp] = x;
    __syncthreads();
    uint32_t before = carry, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (t < a.tiles) c[t] = before + x - v;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.totals[blockIdx.x] = carry;
}

template <class ID>
__global__ void __launch_bounds__(kSortThreads) scatter_kernel(
    const __grid_constant__ PassArgs a) {
  __shared__ RankSmem s;
  uint32_t key[kTileItems], at[kTileItems], digit[kTileItems], rank[kTileItems];
  load_tile<ID>(a, key, at, digit);
  rank_digits<kTileItems>(s, digit, rank);
  uint32_t all = 0, mine = 0;
  if (threadIdx.x < kDigits) {
    all = a.totals[threadIdx.x];
    mine = a.counts[threadIdx.x * a.tiles + blockIdx.x];
  }
  digit_bases(s, all, mine);
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const uint32_t to = s.base[digit[j]] + s.warp_count[warp][digit[j]] + rank[j];
    if (to < a.s.n) {
      a.keys_out[to] = key[j];
      a.pos_out[to] = at[j];
    }
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

// sum_kernel by the type of dy and the shape of a lane's columns.
using SumKernel = void (*)(GradArgs);
#define SUM_SHAPES(in)                                                                     \
  {sum_kernel<in, 8, 1>, sum_kernel<in, 4, 2>, sum_kernel<in, 2, 4>, sum_kernel<in, 1, 8>, \
   sum_kernel<in, 4, 1>, sum_kernel<in, 2, 1>, sum_kernel<in, 1, 1>}
const SumKernel sum_kernels[3][7] = {SUM_SHAPES(TRAIN_BF16), SUM_SHAPES(TRAIN_FP16),
                                     SUM_SHAPES(TRAIN_FP32)};
const int kShapeVec[7] = {8, 4, 2, 1, 4, 2, 1};
const int kShapeCols[7] = {8, 8, 8, 8, 4, 2, 1};

// Where a lane's loads are as wide as the alignment lets them be, and a warp
// covers no more than twice the columns there are.
int pick_shape(int vec, int64_t dim) {
  if (vec >= 4 && dim > 64 && dim <= 128) return 4;
  if (vec >= 2 && dim > 32 && dim <= 64) return 5;
  if (dim <= 32) return 6;
  return vec == 8 ? 0 : vec == 4 ? 1 : vec == 2 ? 2 : 3;
}

// The widest of 8, 4, 2 and 1 neighbouring elements that every row can be
// cut into, each piece aligned to its size or to 16 bytes.
int vector_width(const void* p, int32_t dtype, int64_t dim, int64_t stride) {
  for (int v = 8; v > 1; v /= 2) {
    const int bytes = v * size_of(dtype) < 16 ? v * size_of(dtype) : 16;
    if (dim % v == 0 && reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes) == 0 &&
        (stride * size_of(dtype)) % bytes == 0)
      return v;
  }
  return 1;
}

constexpr int64_t kClusterCapacity = 8 * kSortThreads * 16;

// How the gradient's work is cut; depends on the sizes alone.
struct GradPlan {
  int64_t block, n_blocks, slot_dim, tiles;
  int64_t keys, pos, keys2, pos2, counts, totals, slots, bytes;  // offsets in the workspace
};

GradPlan grad_plan(int64_t n, int64_t n_rows, int64_t dim) {
  GradPlan p{};
  (void)n_rows;
  // Blocks of 64 positions where they make work for 4096 warps, else 32, else 16.
  const int64_t slabs = (dim + 255) / 256;
  p.block = 64;
  while (p.block > 16 && n / p.block * slabs < 4096) p.block /= 2;
  p.n_blocks = (n + p.block - 1) / p.block;
  p.slot_dim = (dim + 7) / 8 * 8;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.keys = take(4 * n);
  p.pos = take(4 * n);
  if (n > kClusterCapacity) {
    p.tiles = (n + kGlobalTile - 1) / kGlobalTile;
    p.keys2 = take(4 * n);
    p.pos2 = take(4 * n);
    p.counts = take(4 * kDigits * p.tiles);
    p.totals = take(4 * kDigits);
  }
  p.slots = at;
  if (n > 2 * p.block) take(2 * p.n_blocks * p.slot_dim * 4);
  p.bytes = at;
  return p;
}

// Launches a kernel, if asked as a programmatic dependent of the one before
// it in the stream, in clusters of `cluster` CTAs.
template <class... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   bool dependent, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int k = 0;
  if (dependent) {
    attr[k].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[k++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[k].id = cudaLaunchAttributeClusterDimension;
    attr[k].val.clusterDim.x = unsigned(cluster);
    attr[k].val.clusterDim.y = 1;
    attr[k++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(k);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int ITEMS, class ID>
cudaError_t launch_cluster_sort(const SortArgs& a, cudaStream_t s) {
  constexpr int kTile = kSortThreads * ITEMS;
  constexpr int kSmem = int(sizeof(RankSmem)) + 8 * kTile;
  // Above 48 KB a kernel has to be told once per device; it costs less than a
  // launch, so it is told every time.
  if (kSmem > 48 * 1024) {
    const cudaError_t ce =
        cudaFuncSetAttribute(cluster_sort_kernel<ITEMS, ID>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (ce != cudaSuccess) return ce;
  }
  int ctas = 1;
  while (int64_t(ctas) * kTile < a.n) ctas *= 2;
  return launch(cluster_sort_kernel<ITEMS, ID>, dim3(unsigned(ctas)), kSortThreads, kSmem, s,
                false, ctas, a);
}

template <class ID>
cudaError_t launch_sort(const SortArgs& a, const GradPlan& p, char* ws, cudaStream_t s) {
  if (a.n <= 8 * kSortThreads * 4) return launch_cluster_sort<4, ID>(a, s);
  if (a.n <= 8 * kSortThreads * 8) return launch_cluster_sort<8, ID>(a, s);
  if (a.n <= kClusterCapacity) return launch_cluster_sort<16, ID>(a, s);
  // The last pass writes to keys and pos.
  uint32_t* k[2] = {a.keys, reinterpret_cast<uint32_t*>(ws + p.keys2)};
  uint32_t* q[2] = {a.pos, reinterpret_cast<uint32_t*>(ws + p.pos2)};
  PassArgs b{};
  b.s = a;
  b.counts = reinterpret_cast<uint32_t*>(ws + p.counts);
  b.totals = reinterpret_cast<uint32_t*>(ws + p.totals);
  b.tiles = p.tiles;
  b.width = (a.bits + a.passes - 1) / a.passes;
  for (int i = 0; i < a.passes; ++i) {
    const int to = (a.passes - 1 - i) & 1;
    b.keys_in = i == 0 ? nullptr : k[to ^ 1];
    b.pos_in = i == 0 ? nullptr : q[to ^ 1];
    b.keys_out = k[to];
    b.pos_out = q[to];
    b.shift = i * b.width;
    const dim3 grid{unsigned(p.tiles)};
    cudaError_t ce = launch(count_kernel<ID>, grid, kSortThreads, 0, s, false, 1, b);
    if (ce == cudaSuccess) ce = launch(scan_kernel, dim3(kDigits), kSortThreads, 0, s, false, 1, b);
    if (ce == cudaSuccess)
      ce = launch(scatter_kernel<ID>, grid, kSortThreads, 0, s, false, 1, b);
    if (ce != cudaSuccess) return ce;
  }
  return cudaSuccess;
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
  *bytes = grad_plan(n_ids, n_rows, dim).bytes;
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
  const GradPlan p = grad_plan(n_ids, n_rows, dim);
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t ce = cudaSuccess;
  GradArgs a{};
  a.dy = grad_out;
  a.grad = grad;
  a.keys = reinterpret_cast<const uint32_t*>(ws + p.keys);
  a.pos = reinterpret_cast<const uint32_t*>(ws + p.pos);
  a.slots = reinterpret_cast<float*>(ws + p.slots);
  a.dy_stride = grad_out_stride;
  a.grad_stride = grad_stride;
  a.n_rows = n_rows;
  a.dim = dim;
  a.slot_dim = p.slot_dim;
  a.n = n_ids;
  a.n_blocks = p.n_blocks;
  a.block = int32_t(p.block);
  a.scale = scale;
  a.accumulate = accumulate;
  a.out_type = grad_dtype;
  if (n_ids > 0) {
    SortArgs t{};
    t.ids = ids;
    t.n = n_ids;
    t.first_row = first_row;
    t.n_rows = n_rows;
    t.padding = padding_id;
    t.keys = reinterpret_cast<uint32_t*>(ws + p.keys);
    t.pos = reinterpret_cast<uint32_t*>(ws + p.pos);
    while ((n_rows >> t.bits) != 0) ++t.bits;  // the largest key is n_rows
    t.passes = (t.bits + 7) / 8;
    ce = ids_dtype == TRAIN_INT64 ? launch_sort<int64_t>(t, p, ws, s)
                                  : launch_sort<int32_t>(t, p, ws, s);
    if (ce != cudaSuccess)
      return fail(LAMB_ERR_CUDA, std::string("sorting the tokens: ") + cudaGetErrorString(ce));
  }
  const int vec_dy = vector_width(grad_out, grad_out_dtype, dim, grad_out_stride);
  const int vec_grad = vector_width(grad, grad_dtype, dim, grad_stride);
  const int shape = pick_shape(n_ids > 0 && vec_dy < vec_grad ? vec_dy : vec_grad, dim);
  a.slabs = int32_t((dim + kWarp * kShapeCols[shape] - 1) / (kWarp * kShapeCols[shape]));
  a.sum_units = p.n_blocks * a.slabs;
  a.fill_units = accumulate ? 0 : (n_rows + kWarp - 1) / kWarp;
  const int64_t warps = kThreads / kWarp;
  const int64_t ctas = (a.sum_units + a.fill_units + warps - 1) / warps;
  if (ctas > kMaxCount) return fail(LAMB_ERR_INVALID, "n_ids * dim is too large");
  ce = launch(sum_kernels[grad_out_dtype][shape], dim3(unsigned(ctas)), kThreads, 0, s,
              n_ids > 0 && n_ids <= kClusterCapacity, 1, a);
  if (ce == cudaSuccess && n_ids > 2 * p.block) {
    // A CTA for every 32 columns, and enough in all to fill the GPU.
    const int64_t x = (dim + kWarp - 1) / kWarp;
    const int64_t y = x >= 512 ? 1 : 512 / x;
    ce = launch(join_kernel, dim3(unsigned(x), unsigned(y < p.n_blocks ? y : p.n_blocks)),
                kJoinWarps * kWarp, 0, s, true, 1, a);
  }
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string("embed_grad: ") + cudaGetErrorString(ce));
}

}  // extern "C"
