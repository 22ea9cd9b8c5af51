// The gradient of the embedding lookup by sorted tokens (train_ops.h).
#include <cooperative_groups.h>

#include "train_internal.h"

using namespace traingb;
namespace cg = cooperative_groups;

namespace {

// G[v, :] = scale * sum over the positions i with row(ids[i]) = v of dy[i, :].
//
// The positions are sorted by row (stably, so ascending within a row), and the
// sorted list is cut into blocks of C positions.  A warp takes one block and
// a slab of up to 512 columns, streams the rows of dy that its positions name
// through a ring of shared memory and adds each run of equal rows in
// registers, in fp32.  A run that ends in the next block at the latest is
// finished by the warp of the block it starts in.  A longer one (a frequent
// token) is cut at the block boundaries: each piece's fp32 sum goes to a slot
// of the workspace, and join_kernel adds the pieces in order.  So no warp adds
// more than 2 C rows whatever the tokens are, only long runs pay for slots, and
// the order of every sum depends on the ids and the sizes alone.
//
// What bounds it is memory: every row of dy is read once, and a dense gradient
// writes n_rows rows, most of them zeros.  Four launches, each started early
// behind the one before it: the sort; beside it fill_kernel, which marks the
// named rows and zeroes some of the others; sum_kernel, with CTAs behind it
// that zero more; join_kernel, and the rest of the zeros beside its few long
// chains.  On GB300 (copy rate 6.79 TB/s): 32768 bf16 tokens of width 12288 into
// a dense gradient of 32000 rows 252 us, 6.3 TB/s over the 1.59 GB that have to
// move; 8192 tokens of width 4096 60 us, 5.5 TB/s (the sort takes 9.5 of them,
// the sums 22 if nothing else is written); 50,021 tokens of which a slice of
// 15,013 rows holds half, fp16 of width 1023 added to fp32, 51 us, 4.0 TB/s (the
// sort takes 15).  Rows of 32 bits hold half as many columns a lane: 8192 fp32 tokens of
// width 4096 take 109 us dense, 6.1 TB/s, 66 added to what is there.

// One sorted position: the row that its token names (n_rows for a token that
// adds nothing) and the position.
struct __align__(8) Place {
  uint32_t key, pos;
};

// A run that is cut into pieces: the block it starts in, its row, the pieces.
struct __align__(16) LongRun {
  uint32_t block, row, pieces, unused;
};

struct GradArgs {
  const void* dy;
  void* grad;
  const void* ids;
  const Place* places;  // sorted
  float* slots;         // [2 * block + (0: run from an earlier block, 1: starts here)][slot_dim]
  uint32_t* n_long;     // long runs in the list: of few pieces, of many
  LongRun* long_runs;   // those of few pieces from the front, the others from the back
  int64_t last_run;     // of the list
  int64_t dy_stride, grad_stride, n_rows, dim, slot_dim, first_row, padding;
  int64_t n;
  int64_t n_blocks;
  int64_t units;         // blocks times slabs
  // Rows that no token names.  A CTA of fill_kernel marks the named ones among
  // rows_per_cta rows and zeroes the others of the first fill_first of them;
  // CTAs of sum_kernel and join_kernel zero the rest (fill_rest rows in all,
  // named ones among them), fill_each rows a CTA.
  uint32_t* named;  // a bit a row
  int64_t rows_per_cta, fill_first, fill_rest, fill_each;
  uint32_t fill_ctas;    // of sum_kernel
  uint32_t fill_last;    // of join_kernel
  uint32_t join_ctas;    // of join_kernel: those that join
  uint32_t join_slabs;   // of 128 columns
  int32_t block, slabs;  // C, slabs of columns
  float scale;
  int32_t accumulate, out_type;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return uint32_t(__cvta_generic_to_shared(p));
}
// 16 bytes from global to shared memory, asynchronously; the bytes from
// `bytes` on are not read and become zero.
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ char* grad_at(const GradArgs& a, int64_t row, int64_t col) {
  return static_cast<char*>(a.grad) + (row * a.grad_stride + col) * size_of(a.out_type);
}

// Eight neighbouring values, 16-byte aligned (each half, if 32 bits wide).
__device__ __forceinline__ void load8(const void* p, int type, float (&x)[8]) {
  if (type == TRAIN_FP32) {
    const float4 u = static_cast<const float4*>(p)[0], v = static_cast<const float4*>(p)[1];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    return;
  }
  const uint4 q = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == TRAIN_BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      x[2 * i] = to_float<TRAIN_FP16>(uint16_t(w[i] & 0xffffu));
      x[2 * i + 1] = to_float<TRAIN_FP16>(uint16_t(w[i] >> 16));
    }
  }
}

__device__ __forceinline__ void store8(void* p, int type, const float (&x)[8]) {
  if (type == TRAIN_FP32) {
    static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = type == TRAIN_BF16 ? pack2<TRAIN_BF16>(x[2 * i], x[2 * i + 1])
                              : pack2<TRAIN_FP16>(x[2 * i], x[2 * i + 1]);
  *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float load1(const void* p, int type) {
  if (type == TRAIN_FP32) return *static_cast<const float*>(p);
  const uint16_t h = *static_cast<const uint16_t*>(p);
  return type == TRAIN_BF16 ? to_float<TRAIN_BF16>(h) : to_float<TRAIN_FP16>(h);
}

__device__ __forceinline__ void store1(void* p, int type, float x) {
  if (type == TRAIN_FP32) *static_cast<float*>(p) = x;
  else if (type == TRAIN_BF16) *static_cast<uint16_t*>(p) = from_float<TRAIN_BF16>(x);
  else *static_cast<uint16_t*>(p) = from_float<TRAIN_FP16>(x);
}

// First index whose row is at least `row`.
__device__ __forceinline__ int64_t lower_bound(const Place* places, int64_t n, uint32_t row) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (places[mid].key < row) lo = mid + 1;
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

// Sets bit r.  A token that has stood before finds it set: 54,000 times the same
// one took 30 us of atomics.
__device__ __forceinline__ void mark(uint32_t* named, uint32_t r) {
  const uint32_t bit = 1u << (r & 31);
  if (!(*const_cast<volatile uint32_t*>(&named[r / 32]) & bit)) atomicOr(&named[r / 32], bit);
}

// Marks the rows that tokens name and zeroes some of the others, a range of
// rows a CTA.  SCAN: the CTA finds its rows by a walk over all ids, so it needs
// no sorted list and runs while the tokens are being sorted.  Else it looks
// its rows up in that list.
//
// It zeroes what fits into the time of the sort (kFillBytes); the later kernels
// zero the rest among their own work.  All of it here, before the sums, takes 71.5 us
// for 8192 tokens of width 4096 instead of 59.6, 291 for 32768 of width 12288 instead
// of 262: the sums alone leave a third of the memory rate unused.
constexpr int kFillThreads = 512;
constexpr int kFillRows = 4096;  // at most, a CTA

template <bool SCAN, class ID>
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const __grid_constant__ GradArgs a) {
  __shared__ uint32_t named[kFillRows / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = int64_t(blockIdx.x) * a.rows_per_cta;
  const int64_t count = min(a.rows_per_cta, a.n_rows - r0);
  pdl_trigger();
  for (int i = threadIdx.x; i < kFillRows / 32; i += kFillThreads) named[i] = 0u;
  __syncthreads();
  if (SCAN) {
    // 16 bytes of ids at a time, from the first 16-byte boundary; kAhead loads on
    // their way together.
    constexpr int kPer = 16 / int(sizeof(ID)), kAhead = 8;
    const ID* ids = static_cast<const ID*>(a.ids);
    const uint64_t base = uint64_t(a.first_row) + uint64_t(r0);
    const auto look = [&](ID id) {
      const uint64_t r = uint64_t(int64_t(id)) - base;
      if (r < uint64_t(count) && int64_t(id) != a.padding) mark(named, uint32_t(r));
    };
    const int64_t head =
        min(a.n, int64_t((16 - reinterpret_cast<uintptr_t>(ids) % 16) % 16 / sizeof(ID)));
    const int64_t vecs = (a.n - head) / kPer;
    const uint4* from = reinterpret_cast<const uint4*>(ids + head);
    for (int64_t v0 = threadIdx.x; v0 < vecs; v0 += kAhead * kFillThreads) {
      uint4 q[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (v0 + i * kFillThreads < vecs) q[i] = __ldg(from + v0 + i * kFillThreads);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (v0 + i * kFillThreads >= vecs) break;
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        if constexpr (sizeof(ID) == 8) {
          look(ID(int64_t(uint64_t(w[1]) << 32 | w[0])));
          look(ID(int64_t(uint64_t(w[3]) << 32 | w[2])));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) look(ID(int32_t(w[j])));
        }
      }
    }
    if (threadIdx.x < head) look(ids[threadIdx.x]);
    if (head + vecs * kPer + threadIdx.x < a.n) look(ids[head + vecs * kPer + threadIdx.x]);
  } else {
    pdl_wait();
    const int64_t lo = lower_bound(a.places, a.n, uint32_t(r0));
    const int64_t hi = lower_bound(a.places, a.n, uint32_t(r0 + count));
    for (int64_t i = lo + threadIdx.x; i < hi; i += kFillThreads) {
      mark(named, a.places[i].key - uint32_t(r0));
    }
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; 32 * i < count; i += kFillThreads)
    a.named[r0 / 32 + i] = named[i];
  const int64_t first = min(count, a.fill_first);
  for (int64_t r = warp; r < first; r += kFillThreads / kWarp)
    if (!((named[r / 32] >> (r & 31)) & 1u))
      warp_zero(grad_at(a, r0 + r, 0), a.dim * size_of(a.out_type), lane);
  // What follows waits for this kernel; it must find the sort finished too.
  if (SCAN) pdl_wait();
}

// The rows that fill_kernel has left, in a CTA of sum_kernel or join_kernel:
// fill_each of them, `index` counting the CTAs.
__device__ __forceinline__ void fill_rest(const GradArgs& a, int64_t index) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / kWarp;
  const int64_t left = a.rows_per_cta - a.fill_first;
  const int64_t q1 = min((index + 1) * a.fill_each, a.fill_rest);
  for (int64_t q0 = index * a.fill_each; q0 < q1; q0 += kWarp) {
    const int64_t q = q0 + lane;
    const int64_t row = q / left * a.rows_per_cta + a.fill_first + q % left;
    const bool idle =
        q < q1 && row < a.n_rows && !((a.named[row / 32] >> (row & 31)) & 1u);
    unsigned todo = __ballot_sync(kAll, idle);
    for (int k = 0; todo; ++k) {
      const int64_t r = __shfl_sync(kAll, row, __ffs(todo) - 1);
      todo &= todo - 1;
      if (k % warps == warp) warp_zero(grad_at(a, r, 0), a.dim * size_of(a.out_type), lane);
    }
  }
}

// The ring of one warp: kStages rows' pieces of a slab in flight.  The copies
// are asynchronous (16 bytes a lane), so they hold no registers, and the rows
// of the grad that accumulation needs come through the same ring behind the
// last row of their run: nothing waits for them when the run is finished.
// Measured on GB300 with 6 and 8 stages: 8192 tokens 59.6 and 59.5 us (added to what
// is there, 42.0 and 43.0), 32768 wide ones 262 and 256, 50,021 of width 1023 in rows
// that are not aligned 62.9 and 67.1.  (Eight rows at a time in registers
// took 276 us for that slice's sums alone, where the ring takes 31.)
constexpr int kStages = 6;
constexpr int kStageBytes = 1024 + 32;  // a piece and its ends' alignment
constexpr int kMaxBlock = 64;
constexpr uint32_t kManyPieces = 64;
constexpr int kSumWarps = 4;

struct WarpSmem {
  alignas(16) unsigned char ring[kStages][kStageBytes];
  uint32_t key[2 * kMaxBlock + 4];
  uint32_t pos[2 * kMaxBlock];
};

// COLS columns a lane: 16 where no 32-bit type comes through the ring, else 8.
// ALIGNED: rows of dy and of the grad start at multiples of 16 bytes and dim is
// a multiple of 8; a lane holds groups of 8 neighbours and copies exactly what
// it reads.  Else a lane holds every 32nd column, and the 16-byte granules
// that cover a piece are copied, its neighbours' bytes with it.
template <int IN, int COLS, bool ALIGNED>
__global__ void __launch_bounds__(kSumWarps* kWarp) sum_kernel(
    const __grid_constant__ GradArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  constexpr int kSlab = kWarp * COLS;
  const int lane = threadIdx.x & 31;
  WarpSmem& s = reinterpret_cast<WarpSmem*>(raw)[threadIdx.x >> 5];
  const int64_t unit = int64_t(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  // The CTAs behind those that add write zero rows.  (Spread among them they
  // kept some of them waiting: 65 us instead of 60 for 8192 tokens of 4096.)
  const uint32_t sum_ctas = gridDim.x - a.fill_ctas;
  if (blockIdx.x >= sum_ctas) {
    fill_rest(a, blockIdx.x - sum_ctas);
    return;
  }
  if (unit >= a.units) return;
  const int64_t b = unit / a.slabs;
  const int64_t col0 = (unit % a.slabs) * kSlab;
  const int cols = int(min(int64_t(kSlab), a.dim - col0));
  const int64_t n = a.n, lo = b * a.block;
  const int C = a.block;
  const uint32_t none = uint32_t(a.n_rows);

  // The block and the next one: rows behind the list count as `none`.
  for (int i = lane; i < 2 * C; i += kWarp) {
    Place p{none, 0u};
    if (lo + i < n) p = a.places[lo + i];
    s.key[i] = p.key;
    s.pos[i] = p.pos;
  }
  const uint32_t after = lo + 2 * C < n ? a.places[lo + 2 * C].key : none;
  const uint32_t before = lo > 0 ? a.places[lo - 1].key : none;
  const uint32_t far_before = lo > C ? a.places[lo - C - 1].key : none;
  if (lane == 0) s.key[2 * C] = after;
  __syncwarp();
  const uint32_t first = s.key[0], last = s.key[C - 1];
  if (first == none) return;
  // The run that reaches in from the block before: a piece of a long run, or
  // finished by its own block.
  const bool from_before = before == first;
  const bool head_piece = from_before && (s.key[C] == first || far_before == first);
  // The run that starts here and reaches out: into the next block at most, or
  // long.
  const bool reaches_out =
      last != none && s.key[C] == last && !(from_before && first == last);
  const bool tail_piece = reaches_out && after == last;
  const int end = reaches_out && !tail_piece ? 2 * C : C;
  // Positions [x, stop) of the window are added here.
  int x = 0, stop = 0;
  for (int i0 = 0; i0 < end; i0 += kWarp) {
    const int i = i0 + lane;
    const uint32_t key = i < end ? s.key[i] : none;
    const bool skipped = from_before && !head_piece && key == first;
    const bool wanted = key != none && !skipped && (i < C || key == last);
    const unsigned use = __ballot_sync(kAll, wanted), skip = __ballot_sync(kAll, skipped);
    x += __popc(skip);
    stop += __popc(skip | use);
  }
  if (x >= stop) return;

  const char* const dy = static_cast<const char*>(a.dy);
  char* const grad = static_cast<char*>(a.grad);
  const int out_size = size_of(a.out_type);
  // A run's last position here.  Only final sums need the old row.
  const auto ends = [&](int i) { return s.key[i] != s.key[i + 1]; };
  const auto is_head = [&](uint32_t key) { return head_piece && key == first; };

  // Starts the copy of this slab's piece of a row; src: its first byte.  [begin,
  // limit) is all that belongs to the matrix.
  const auto copy_piece = [&](unsigned char* dst, const char* src, int size, const char* begin,
                              const char* limit) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int g = 0; g < COLS / 8; ++g) {
        const int c = g * 8 * kWarp + lane * 8;
        if (c < cols) {
          copy16(dst + c * size, src + c * size, 16);
          if (size == 4) copy16(dst + c * size + 16, src + c * size + 16, 16);
        }
      }
    } else {
      const int shift = int(reinterpret_cast<uintptr_t>(src) & 15);
      const int granules = (shift + cols * size + 15) / 16;
      const char* q = src - shift + 16 * lane;
      dst += 16 * lane;
      if (src - shift >= begin && src - shift + 16 * granules <= limit) {
        // At most 65 of them.
        if (lane < granules) copy16(dst, q, 16);
        if (lane + kWarp < granules) copy16(dst + 16 * kWarp, q + 16 * kWarp, 16);
        if (lane + 2 * kWarp < granules) copy16(dst + 32 * kWarp, q + 32 * kWarp, 16);
        return;
      }
      for (int g = lane; g < granules; g += kWarp, q += 16 * kWarp, dst += 16 * kWarp) {
        if (q >= begin) {
          const int64_t left = limit - q;
          copy16(dst, q, left < 16 ? int(left) : 16);
        } else {
          // In front of the matrix: only what belongs to it.
          for (int i = int(begin - q); i < 16; i += 2)
            if (q + i < limit)
              *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(q + i);
        }
      }
    }
  };
  const int64_t dy_step = a.dy_stride * size_of(IN), grad_step = a.grad_stride * out_size;
  const char* const dy_slab = dy + col0 * size_of(IN);
  char* const grad_slab = grad + col0 * out_size;
  const char* const dy_limit = dy + (n - 1) * dy_step + a.dim * size_of(IN);
  const char* const grad_limit = grad + (a.n_rows - 1) * grad_step + a.dim * out_size;

  // The next piece to fetch: position at, or the old row behind it.
  int at = x;
  bool old_next = false;
  const auto fetch = [&](int stage) {
    if (at < stop) {
      if (!old_next) {
        copy_piece(s.ring[stage], dy_slab + s.pos[at] * dy_step, size_of(IN), dy, dy_limit);
        old_next = a.accumulate && ends(at) && !is_head(s.key[at]);
        if (!old_next) ++at;
      } else {
        copy_piece(s.ring[stage], grad_slab + s.key[at] * grad_step, out_size, grad, grad_limit);
        old_next = false;
        ++at;
      }
    }
    copy_commit();
  };
  // A lane's values of the piece in a stage.  Unaligned: it starts `low` bytes
  // (modulo 16) into its first granule.
  const auto read_piece = [&](int stage, uint32_t low, auto t, float (&v)[COLS]) {
    constexpr int type = decltype(t)::value;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int g = 0; g < COLS / 8; ++g) {
        float u[8];
        load8(s.ring[stage] + (g * 8 * kWarp + lane * 8) * size_of(type), type, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * g + i] = u[i];
      }
    } else {
      const unsigned char* p = s.ring[stage] + (low & 15u) + lane * size_of(type);
#pragma unroll
      for (int i = 0; i < COLS; ++i) v[i] = load1(p + kWarp * i * size_of(type), type);
    }
  };
  const uint32_t dy_low = uint32_t(reinterpret_cast<uintptr_t>(dy_slab));
  const uint32_t grad_low = uint32_t(reinterpret_cast<uintptr_t>(grad_slab));

  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  float acc[COLS];
#pragma unroll
  for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
  int stage = 0;
  const auto next_stage = [&] {
    // One more piece into the stage read last, then wait for the oldest.
    __syncwarp();
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    copy_wait<kStages - 1>();
    __syncwarp();
  };
  const auto done_stage = [&] { stage = stage == kStages - 1 ? 0 : stage + 1; };
  const auto write_slot = [&](int which) {
    float* slot = a.slots + (2 * b + which) * a.slot_dim + col0;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int g = 0; g < COLS / 8; ++g) {
        const int c = g * 8 * kWarp + lane * 8;
        if (c < cols) {
          float u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = acc[8 * g + i];
          store8(slot + c, TRAIN_FP32, u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < COLS; ++i)
        if (lane + kWarp * i < cols) slot[lane + kWarp * i] = acc[i];
    }
  };

  for (; x < stop; ++x) {
    next_stage();
    float v[COLS];
    read_piece(stage, dy_low + s.pos[x] * uint32_t(dy_step), Type<IN>{}, v);
    done_stage();
#pragma unroll
    for (int i = 0; i < COLS; ++i) acc[i] += v[i];
    if (!ends(x)) continue;
    const uint32_t key = s.key[x];
    if (is_head(key)) {
      write_slot(0);
    } else {
      if (a.accumulate) {
        next_stage();
        by_type(a.out_type, [&](auto t) {
          read_piece(stage, grad_low + key * uint32_t(grad_step), t, v);
        });
        done_stage();
#pragma unroll
        for (int i = 0; i < COLS; ++i) acc[i] = fmaf(a.scale, acc[i], v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < COLS; ++i) acc[i] *= a.scale;
      }
      by_type(a.out_type, [&](auto t) {
        constexpr int type = decltype(t)::value;
        char* p = grad_slab + key * grad_step;
        if constexpr (ALIGNED) {
#pragma unroll
          for (int g = 0; g < COLS / 8; ++g) {
            const int c = g * 8 * kWarp + lane * 8;
            if (c < cols) {
              float u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) u[i] = acc[8 * g + i];
              store8(p + c * size_of(type), type, u);
            }
          }
        } else {
          p += lane * size_of(type);
          if (cols == kSlab) {
#pragma unroll
            for (int i = 0; i < COLS; ++i) store1(p + kWarp * i * size_of(type), type, acc[i]);
          } else {
#pragma unroll
            for (int i = 0; i < COLS; ++i)
              if (lane + kWarp * i < cols) store1(p + kWarp * i * size_of(type), type, acc[i]);
          }
        }
      });
    }
#pragma unroll
    for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
  }
  // What is left in the registers is a piece of a run that goes on.
  if (!ends(stop - 1)) write_slot(is_head(s.key[stop - 1]) ? 0 : 1);
  if (tail_piece && col0 == 0) {
    // The run covers the start of every block it has a piece in but its first.
    uint32_t pieces = 1;
    for (int64_t q = b + 1;; q += kWarp) {
      const int64_t i = (q + lane) * C;
      const int more = __popc(__ballot_sync(kAll, i < n && a.places[i < n ? i : 0].key == last));
      pieces += more;
      if (more < kWarp) break;
    }
    if (lane == 0) {
      const int many = pieces >= kManyPieces;
      const uint32_t k = atomicAdd(&a.n_long[many], 1u);
      a.long_runs[many ? a.last_run - k : k] = LongRun{uint32_t(b), last, pieces, 0u};
    }
  }
}

// Adds the pieces of every long run, in order.  A lane takes four columns, a
// group of lanes a slab of them; the groups of a CTA add neighbouring shares of
// the pieces (8 at least), and the first group adds their sums.  A run of few
// pieces has slabs of 128 columns (a warp a group), one of many pieces slabs of
// 32, so that more CTAs and more groups share it: 847 pieces of width 4032 took 40
// us with wide slabs.
constexpr int kJoinThreads = 256;
constexpr int kJoinCols = 128, kJoinNarrow = 32;

template <int LANES>
__device__ __forceinline__ void join_run(const GradArgs& a, const LongRun& run, int64_t col0,
                                         float4* part) {
  constexpr int kGroups = kJoinThreads / LANES;
  constexpr int kAhead = 8;
  const int group = threadIdx.x / LANES;
  const int64_t col = col0 + 4 * (threadIdx.x & (LANES - 1));
  const int pieces = int(run.pieces);
  int share = (pieces + kGroups - 1) / kGroups;
  if (share < 8) share = 8;
  const int p1 = min((group + 1) * share, pieces);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < a.slot_dim) {  // whole groups of 8 columns
    // Piece 0 is in the second slot of its block, the others in the first.
    const float* slot = a.slots + 2 * int64_t(run.block) * a.slot_dim + col;
    for (int p = group * share; p < p1; p += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p + i < p1)
          v[i] = *reinterpret_cast<const float4*>(
              slot + (2 * int64_t(p + i) + (p + i == 0)) * a.slot_dim);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        acc.x += v[i].x, acc.y += v[i].y, acc.z += v[i].z, acc.w += v[i].w;
    }
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  if (group == 0) {
    for (int g = 1; g < kGroups && g * share < pieces; ++g) {
      const float4 v = part[g * LANES + threadIdx.x];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
    const float x[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (col + i < a.dim) {
        char* g = grad_at(a, run.row, col + i);
        const float old = a.accumulate ? load1(g, a.out_type) : 0.0f;
        store1(g, a.out_type, a.accumulate ? fmaf(a.scale, x[i], old) : a.scale * x[i]);
      }
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float4 part[kJoinThreads];
  pdl_wait();
  if (blockIdx.x >= a.join_ctas) {
    fill_rest(a, a.fill_ctas + (blockIdx.x - a.join_ctas));
    return;
  }
  const uint32_t few = a.n_long[0], many = a.n_long[1];
  const uint32_t narrow = uint32_t((a.dim + kJoinNarrow - 1) / kJoinNarrow);
  for (uint64_t k = blockIdx.x; k < uint64_t(many) * narrow; k += a.join_ctas)
    join_run<kJoinNarrow / 4>(a, a.long_runs[a.last_run - int64_t(k / narrow)],
                              int64_t(k % narrow) * kJoinNarrow, part);
  for (uint64_t k = blockIdx.x; k < uint64_t(few) * a.join_slabs; k += a.join_ctas)
    join_run<kJoinCols / 4>(a, a.long_runs[k / a.join_slabs],
                            int64_t(k % a.join_slabs) * kJoinCols, part);
}

// ------------------------------------------------------------- few tokens
// Without a sort, in one launch: every CTA reads all ids.  The CTA of a token
// and 256 columns leaves if the token has stood before; else it lists the
// token's positions, its warps add neighbouring shares of them, and the
// shares' sums are added in order.  The CTAs behind these zero a few rows each.
constexpr int kDirectThreads = 256;
constexpr int kDirectWarps = kDirectThreads / kWarp;
constexpr int kDirectIds = 2048;
constexpr int kDirectCols = 8 * kWarp;
constexpr int kDirectRounds = kDirectIds / kDirectThreads;
constexpr int kDirectFill = 4096;  // rows a CTA zeroes, at most

struct DirectArgs {
  GradArgs g;
  uint32_t sum_ctas;  // tokens times slabs
  int32_t ids64;
};

template <int IN, bool ALIGNED>
__global__ void __launch_bounds__(kDirectThreads, 4) direct_kernel(
    const __grid_constant__ DirectArgs d) {
  const GradArgs& a = d.g;
  __shared__ uint32_t keys[kDirectIds];
  __shared__ uint16_t list[kDirectIds];
  __shared__ int counts[kDirectRounds * kDirectWarps];
  __shared__ float part[kDirectWarps][kDirectCols];
  __shared__ uint32_t named[kDirectFill / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = int(a.n);
  pdl_wait();
  for (int j = threadIdx.x; j < n; j += kDirectThreads) {
    const int64_t id = d.ids64 ? static_cast<const int64_t*>(a.ids)[j]
                               : int64_t(static_cast<const int32_t*>(a.ids)[j]);
    const int64_t row = row_of(id, a.first_row, a.n_rows);
    keys[j] = row < 0 || id == a.padding ? uint32_t(a.n_rows) : uint32_t(row);
  }
  if (blockIdx.x >= d.sum_ctas) {
    // Rows to zero.
    const int64_t r0 = int64_t(blockIdx.x - d.sum_ctas) * a.fill_each;
    const int64_t rows = min(a.fill_each, a.n_rows - r0);
    for (int i = threadIdx.x; 32 * i < rows; i += kDirectThreads) named[i] = 0u;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kDirectThreads) {
      const uint64_t r = uint64_t(keys[j]) - uint64_t(r0);
      if (r < uint64_t(rows)) mark(named, uint32_t(r));
    }
    __syncthreads();
    for (int64_t r = warp; r < rows; r += kDirectWarps)
      if (!((named[r / 32] >> (r & 31)) & 1u))
        warp_zero(grad_at(a, r0 + r, 0), a.dim * size_of(a.out_type), lane);
    return;
  }
  __syncthreads();
  const int token = int(blockIdx.x / uint32_t(a.slabs));
  const int64_t col0 = int64_t(blockIdx.x % uint32_t(a.slabs)) * kDirectCols;
  const uint32_t key = keys[token];
  if (key == uint32_t(a.n_rows)) return;
  // The token's positions, in ascending order.
  unsigned match[kDirectRounds];
  int before = 0;
#pragma unroll
  for (int r = 0; r < kDirectRounds; ++r) {
    match[r] = 0u;
    if (r * kDirectThreads >= n) continue;
    const int j = r * kDirectThreads + threadIdx.x;
    const bool same = j < n && keys[j] == key;
    before |= same && j < token;
    match[r] = __ballot_sync(kAll, same);
    if (lane == 0) counts[r * kDirectWarps + warp] = __popc(match[r]);
  }
  if (__syncthreads_or(before)) return;
  int total = 0;
#pragma unroll
  for (int r = 0; r < kDirectRounds; ++r) {
    if (r * kDirectThreads >= n) continue;
    int at = total;
    for (int w = 0; w < kDirectWarps; ++w) {
      const int c = counts[r * kDirectWarps + w];
      if (w < warp) at += c;
      total += c;
    }
    if ((match[r] >> lane) & 1u)
      list[at + __popc(match[r] & ((1u << lane) - 1u))] =
          uint16_t(r * kDirectThreads + threadIdx.x);
  }
  __syncthreads();
  const int share = (total + kDirectWarps - 1) / kDirectWarps;
  const int l1 = min((warp + 1) * share, total);
  using T = typename TypeOf<IN>::T;
  const T* dy = static_cast<const T*>(a.dy) + col0;
  const int cols = int(min(int64_t(kDirectCols), a.dim - col0));
  // A lane's 8 columns: neighbours, or every 32nd.
  constexpr int kVec = ALIGNED ? 8 : 1, kGroups = 8 / kVec;
  constexpr int kRows = 4;  // on their way together
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int l = warp * share; l < l1; l += kRows) {
    Pack<IN, kVec> v[kRows][kGroups];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const T* row = dy + int64_t(list[min(l + q, l1 - 1)]) * a.dy_stride + kVec * lane;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        if (l + q < l1 && kVec * lane + kWarp * i < cols) v[q][i].load(row + kWarp * i);
        else v[q][i].clear();
      }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[q][i / kVec].get(i % kVec);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[warp][ALIGNED ? 8 * lane + i : lane + kWarp * i] = acc[i];
  __syncthreads();
  if (int(threadIdx.x) >= cols) return;
  float sum = part[0][threadIdx.x];
  for (int w = 1; w * share < total; ++w) sum += part[w][threadIdx.x];
  char* g = grad_at(a, key, col0 + threadIdx.x);
  store1(g, a.out_type, a.accumulate ? fmaf(a.scale, sum, load1(g, a.out_type)) : a.scale * sum);
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
  Place* places;        // the result
  uint32_t* n_long;     // the first kernel clears both
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
// Lanes of equal digits are found bit by bit: for 4 elements a lane 2.3 us, where
// __match_any_sync took 0.5 to 4, more the more digits differ.
template <int ITEMS>
__device__ __forceinline__ void rank_digits(RankSmem& s, const uint32_t (&digit)[ITEMS],
                                            uint32_t (&rank)[ITEMS], int width) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* z = reinterpret_cast<uint32_t*>(s.warp_count[warp]);
#pragma unroll
  for (int i = 0; i < kDigits / 2 / kWarp; ++i) z[lane + kWarp * i] = 0u;
  __syncwarp();
  unsigned equal[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) equal[j] = kAll;
  for (int b = 0; b < width; ++b) {
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const bool one = (digit[j] >> b) & 1u;
      const unsigned ones = __ballot_sync(kAll, one);
      equal[j] &= one ? ones : ~ones;
    }
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const unsigned peers = equal[j];
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

// A barrier of the cluster in two halves.  Shared memory of another CTA may be
// used only once that CTA runs: each arrives as it starts, and waits for the
// others in front of its first remote store, behind its own loads and ranks.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Up to 16 * 1024 * ITEMS positions in one cluster: every CTA holds a tile of
// 1024 * ITEMS elements, and the CTAs exchange their digit counts.  A CTA
// first orders its tile by digit in its own shared memory, so that a warp then
// stores neighbours to neighbours: into the tiles of the other CTAs (distributed
// shared memory), on the last pass into global memory.  (Scattered straight
// from the registers, 8 bytes at a time, two passes over 50,021 tokens took
// 28.6 us in a cluster of 8; now they take 15.)
constexpr int kSortCtas = 16;

template <int ITEMS, class ID>
__global__ void __launch_bounds__(kSortThreads) cluster_sort_kernel(
    const __grid_constant__ SortArgs a) {
  constexpr int kTile = kSortThreads * ITEMS;
  extern __shared__ __align__(16) unsigned char raw[];
  RankSmem& s = *reinterpret_cast<RankSmem*>(raw);
  uint32_t(*totals)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(raw + sizeof(RankSmem));
  Place* tile = reinterpret_cast<Place*>(totals + kSortCtas);
  Place* ordered = tile + kTile;
  cg::cluster_group cluster = cg::this_cluster();
  const int me = int(cluster.block_rank()), ctas = int(cluster.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();
  pdl_trigger();
  if (me == 0 && threadIdx.x < 2) a.n_long[threadIdx.x] = 0u;
  const int width = (a.bits + a.passes - 1) / a.passes;
  const uint32_t mask = (1u << width) - 1u;
  const int local0 = warp * (kWarp * ITEMS) + lane;
  Place x[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int64_t i = int64_t(me) * kTile + local0 + kWarp * j;
    // Behind the last token: the largest digits, so these stay behind it.
    x[j].key = i < a.n ? key_of<ID>(a, i) : 0xffffffffu;
    x[j].pos = uint32_t(i);
  }
  for (int p = 0; p < a.passes; ++p) {
    if (p > 0) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) x[j] = tile[local0 + kWarp * j];
    }
    uint32_t digit[ITEMS], rank[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) digit[j] = (x[j].key >> (p * width)) & mask;
    rank_digits<ITEMS>(s, digit, rank, width);
    __syncthreads();
    if (p == 0) cluster_wait();
    // Every CTA gets every CTA's counts.
    const int d = threadIdx.x & (kDigits - 1);
    for (int r = threadIdx.x / kDigits; r < ctas; r += kSortThreads / kDigits)
      cluster.map_shared_rank(totals[me], r)[d] = s.total[d];
    cluster.sync();  // the counts are there, and the tiles have been read
    // Thread d: where digit d starts in this CTA's ordered tile, and how far
    // from there its elements go.
    uint32_t all = 0, mine = 0, own = 0;
    if (threadIdx.x < kDigits) {
      for (int r = 0; r < ctas; ++r) {
        const uint32_t c = totals[r][threadIdx.x];
        if (r < me) mine += c;
        all += c;
      }
      own = s.total[threadIdx.x];
    }
    digit_bases(s, own, 0u);
    const uint32_t start = threadIdx.x < kDigits ? s.base[threadIdx.x] : 0u;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
      ordered[s.base[digit[j]] + s.warp_count[warp][digit[j]] + rank[j]] = x[j];
    __syncthreads();
    digit_bases(s, all, mine - start);
    const bool out = p == a.passes - 1;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int i = threadIdx.x + kSortThreads * j;
      const Place y = ordered[i];
      const uint32_t to = s.base[(y.key >> (p * width)) & mask] + uint32_t(i);
      if (!out) cluster.map_shared_rank(tile, int(to / kTile))[to % kTile] = y;
      else if (to < a.n) a.places[to] = y;
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
  const Place* in;  // NULL: from the ids
  Place* out;
  uint32_t* counts;  // [digit][tile]
  uint32_t* totals;  // [digit]
  int64_t tiles;
  int32_t shift, width;
};

template <class ID>
__device__ __forceinline__ void load_tile(const PassArgs& a, Place (&x)[kTileItems],
                                          uint32_t (&digit)[kTileItems]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int64_t i = int64_t(blockIdx.x) * kGlobalTile + warp * (kWarp * kTileItems) +
                      kWarp * j + lane;
    x[j] = Place{0xffffffffu, 0u};
    if (i < a.s.n) x[j] = a.in ? a.in[i] : Place{key_of<ID>(a.s, i), uint32_t(i)};
    digit[j] = (x[j].key >> a.shift) & ((1u << a.width) - 1u);
  }
}

template <class ID>
__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ PassArgs a) {
  __shared__ RankSmem s;
  Place x[kTileItems];
  uint32_t digit[kTileItems], rank[kTileItems];
  if (blockIdx.x == 0 && threadIdx.x < 2) a.s.n_long[threadIdx.x] = 0u;
  load_tile<ID>(a, x, digit);
  rank_digits<kTileItems>(s, digit, rank, a.width);
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
  Place x[kTileItems];
  uint32_t digit[kTileItems], rank[kTileItems];
  load_tile<ID>(a, x, digit);
  rank_digits<kTileItems>(s, digit, rank, a.width);
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
    if (to < a.s.n) a.out[to] = x[j];
  }
}

// sum_kernel by the type of dy, the columns a lane holds and the alignment.
using SumKernel = void (*)(GradArgs);
const SumKernel sum_kernels[3][2][2] = {
    {{sum_kernel<TRAIN_BF16, 8, false>, sum_kernel<TRAIN_BF16, 8, true>},
     {sum_kernel<TRAIN_BF16, 16, false>, sum_kernel<TRAIN_BF16, 16, true>}},
    {{sum_kernel<TRAIN_FP16, 8, false>, sum_kernel<TRAIN_FP16, 8, true>},
     {sum_kernel<TRAIN_FP16, 16, false>, sum_kernel<TRAIN_FP16, 16, true>}},
    {{sum_kernel<TRAIN_FP32, 8, false>, sum_kernel<TRAIN_FP32, 8, true>}, {nullptr, nullptr}}};

// Every row starts at a multiple of 16 bytes.
bool rows_aligned16(const void* p, int32_t dtype, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size_of(dtype) % 16 == 0;
}

// Zeros written while the tokens are being sorted: with 24, 48 and 80 MB 8192 tokens
// of width 4096 take 61.7, 59.6 and 60.6 us.
constexpr double kFillBytes = 48e6;

// Elements of one matrix, at most.
constexpr int64_t kMaxElements = int64_t(1) << 40;

constexpr int64_t kClusterCapacity = kSortCtas * kSortThreads * 8;

// One launch without a sort: few ids, and few enough CTAs that each of them
// reading all ids does not matter.  On GB300, summed onto a bf16 grad, frequent
// tokens as in text: 1024 ids of width 256 take 5.4 us this way and 18.5 with a
// sort, 256 of width 4096 (4096 CTAs) 11.1 and 18.1, 512 of them 23.0 and 18.5.
// A frequent token is slow this way where rows are not aligned (1024 times the same
// one, width 1023: 64 us, with a sort 18.5), so only a quarter of the ids are taken
// where the width is no multiple of 8.  The rule sees the width alone, so that the
// workspace depends on sizes only: of rows of 1024 that their address or stride puts
// off the alignment all 2048 are taken, in 18.0 us instead of 20.5 if they are 1024 as
// in text, in 64 instead of 20.4 if they are the same token throughout.
constexpr int64_t kDirectCtas = 4096;
bool use_direct(int64_t n, int64_t dim) {
  return n <= (dim % 8 == 0 ? kDirectIds : kDirectIds / 4) &&
         n * ((dim + kDirectCols - 1) / kDirectCols) <= kDirectCtas;
}

using DirectKernel = void (*)(DirectArgs);
const DirectKernel direct_kernels[3][2] = {
    {direct_kernel<TRAIN_BF16, false>, direct_kernel<TRAIN_BF16, true>},
    {direct_kernel<TRAIN_FP16, false>, direct_kernel<TRAIN_FP16, true>},
    {direct_kernel<TRAIN_FP32, false>, direct_kernel<TRAIN_FP32, true>}};

// How the gradient's work is cut; depends on the sizes alone.
struct GradPlan {
  int64_t block, n_blocks, slot_dim, tiles;
  // Offsets in the workspace, and its size.
  int64_t places, places2, counts, totals, n_long, long_runs, named, slots, bytes;
};

GradPlan grad_plan(int64_t n, int64_t n_rows, int64_t dim) {
  GradPlan p{};
  if (use_direct(n, dim)) return p;
  // Blocks of 64 positions where they make work for 4096 warps, else of 32 or 16:
  // 32768 wide tokens take 262 us with 64 and 268 with 128, 8192 of width 4096 59.6
  // with 16 and 66.5 with 32.
  const int64_t slabs = (dim + 511) / 512;
  p.block = kMaxBlock;
  while (p.block > 16 && n / p.block * slabs < 4096) p.block /= 2;
  // Where even 16 make few: 1024 tokens of width 4096 added to bf16 take 20.4 us with
  // blocks of 8, 22.7 with 16; 8192 of them (4096 warps with 16) 66.9 and 59.6.
  if (n / 16 * slabs < 2048) p.block = 8;
  p.n_blocks = (n + p.block - 1) / p.block;
  p.slot_dim = (dim + 7) / 8 * 8;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.places = take(int64_t(sizeof(Place)) * n);
  if (n > kClusterCapacity) {
    p.tiles = (n + kGlobalTile - 1) / kGlobalTile;
    p.places2 = take(int64_t(sizeof(Place)) * n);
    p.counts = take(4 * kDigits * p.tiles);
    p.totals = take(4 * kDigits);
  }
  p.n_long = take(8);
  p.long_runs = take(int64_t(sizeof(LongRun)) * (p.n_blocks / 2 + 1));
  p.named = take(4 * ((n_rows + 31) / 32));
  p.slots = at;
  if (n > 2 * p.block) take(2 * p.n_blocks * p.slot_dim * 4);
  p.bytes = at;
  return p;
}

template <int ITEMS, class ID>
cudaError_t launch_cluster_sort(const SortArgs& a, cudaStream_t s) {
  constexpr int kTile = kSortThreads * ITEMS;
  constexpr int kSmem =
      int(sizeof(RankSmem)) + 4 * kSortCtas * kDigits + 2 * int(sizeof(Place)) * kTile;
  int ctas = 1;
  while (int64_t(ctas) * kTile < a.n) ctas *= 2;
  // What a kernel has to be told once per device; it costs less than a launch,
  // so it is told every time.
  cudaError_t ce = cudaSuccess;
  if (kSmem > 48 * 1024)
    ce = cudaFuncSetAttribute(cluster_sort_kernel<ITEMS, ID>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (ce == cudaSuccess && ctas > 8)
    ce = cudaFuncSetAttribute(cluster_sort_kernel<ITEMS, ID>,
                              cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (ce != cudaSuccess) return ce;
  return launch(cluster_sort_kernel<ITEMS, ID>, dim3(unsigned(ctas)), kSortThreads, kSmem, s,
                false, ctas, a);
}

template <class ID>
cudaError_t launch_sort(const SortArgs& a, const GradPlan& p, char* ws, cudaStream_t s) {
  // As many CTAs as the cluster takes, so that each has few elements to rank
  // and to store.
  if (a.n <= kSortCtas * kSortThreads) return launch_cluster_sort<1, ID>(a, s);
  if (a.n <= kSortCtas * kSortThreads * 2) return launch_cluster_sort<2, ID>(a, s);
  if (a.n <= kSortCtas * kSortThreads * 4) return launch_cluster_sort<4, ID>(a, s);
  if (a.n <= kClusterCapacity) return launch_cluster_sort<8, ID>(a, s);
  // The last pass writes to places.
  Place* q[2] = {a.places, reinterpret_cast<Place*>(ws + p.places2)};
  PassArgs b{};
  b.s = a;
  b.counts = reinterpret_cast<uint32_t*>(ws + p.counts);
  b.totals = reinterpret_cast<uint32_t*>(ws + p.totals);
  b.tiles = p.tiles;
  b.width = (a.bits + a.passes - 1) / a.passes;
  for (int i = 0; i < a.passes; ++i) {
    const int to = (a.passes - 1 - i) & 1;
    b.in = i == 0 ? nullptr : q[to ^ 1];
    b.out = q[to];
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
  int rc = check_ids(ids, ids_dtype, n_ids, first_row, n_rows);
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
  // Beyond any memory; below it every count of CTAs and rows fits its type.
  if (n_ids > kMaxElements / dim || n_rows > kMaxElements / dim)
    return fail(LAMB_ERR_INVALID, "n_ids * dim or n_rows * dim is too large");
  const GradPlan p = grad_plan(n_ids, n_rows, dim);
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t ce = cudaSuccess;
  GradArgs a{};
  a.dy = grad_out;
  a.grad = grad;
  a.ids = ids;
  a.first_row = first_row;
  a.padding = padding_id;
  a.places = reinterpret_cast<const Place*>(ws + p.places);
  a.slots = reinterpret_cast<float*>(ws + p.slots);
  a.n_long = reinterpret_cast<uint32_t*>(ws + p.n_long);
  a.long_runs = reinterpret_cast<LongRun*>(ws + p.long_runs);
  a.named = reinterpret_cast<uint32_t*>(ws + p.named);
  a.dy_stride = grad_out_stride;
  a.grad_stride = grad_stride;
  a.n_rows = n_rows;
  a.dim = dim;
  a.slot_dim = p.slot_dim;
  a.n = n_ids;
  a.n_blocks = p.n_blocks;
  a.last_run = p.n_blocks / 2;
  a.block = int32_t(p.block);
  a.scale = scale;
  a.accumulate = accumulate;
  a.out_type = grad_dtype;
  const bool aligned = dim % 8 == 0 && rows_aligned16(grad_out, grad_out_dtype, grad_out_stride) &&
                       rows_aligned16(grad, grad_dtype, grad_stride);
  const double row_bytes = double(dim) * size_of(grad_dtype);
  if (use_direct(n_ids, dim)) {
    DirectArgs d{};
    a.slabs = int32_t((dim + kDirectCols - 1) / kDirectCols);
    d.sum_ctas = uint32_t(n_ids * a.slabs);
    d.ids64 = ids_dtype == TRAIN_INT64;
    int64_t fill = 0;
    if (!accumulate) {
      a.fill_each = int64_t(32e3 / row_bytes) + 1;
      if (a.fill_each > kDirectFill) a.fill_each = kDirectFill;
      int64_t even = (n_rows + 303) / 304;  // not fewer CTAs than 304, but 8 rows each
      if (even < 8) even = 8;
      if (a.fill_each > even) a.fill_each = even;
      fill = (n_rows + a.fill_each - 1) / a.fill_each;
    }
    d.g = a;
    ce = launch(direct_kernels[grad_out_dtype][aligned ? 1 : 0],
                dim3(unsigned(d.sum_ctas + fill)), kDirectThreads, 0, s, true, 1, d);
    return ce == cudaSuccess
               ? LAMB_OK
               : fail(LAMB_ERR_CUDA, std::string("embed_grad: ") + cudaGetErrorString(ce));
  }
  // From here on there are tokens.
  SortArgs t{};
  t.ids = ids;
  t.n = n_ids;
  t.first_row = first_row;
  t.n_rows = n_rows;
  t.padding = padding_id;
  t.places = reinterpret_cast<Place*>(ws + p.places);
  t.n_long = reinterpret_cast<uint32_t*>(ws + p.n_long);
  while ((n_rows >> t.bits) != 0) ++t.bits;  // the largest key is n_rows
  t.passes = (t.bits + 7) / 8;
  ce = ids_dtype == TRAIN_INT64 ? launch_sort<int64_t>(t, p, ws, s)
                                : launch_sort<int32_t>(t, p, ws, s);
  if (ce != cudaSuccess)
    return fail(LAMB_ERR_CUDA, std::string("sorting the tokens: ") + cudaGetErrorString(ce));
  if (!accumulate) {
    // Ids are read by every CTA, which the sort hides, unless there are too
    // many of them or of the CTAs.
    int64_t ctas = 304;
    while (n_rows > ctas * kFillRows) ctas *= 2;
    a.rows_per_cta = ((n_rows + ctas - 1) / ctas + 31) / 32 * 32;
    ctas = (n_rows + a.rows_per_cta - 1) / a.rows_per_cta;
    const bool scan = n_ids <= kClusterCapacity && ctas <= 304;
    a.fill_first = a.rows_per_cta;
    if (scan) {
      // What is written while the tokens are sorted; the rest among the sums.
      const double part = kFillBytes / (double(n_rows) * row_bytes);
      if (part < 1.0) a.fill_first = int64_t(part * double(a.rows_per_cta));
      const int64_t most = int64_t(512e3 / row_bytes) + 1;  // of one CTA
      if (a.fill_first > most) a.fill_first = most;
      if (a.fill_first > a.rows_per_cta) a.fill_first = a.rows_per_cta;
      a.fill_rest = ctas * (a.rows_per_cta - a.fill_first);
      a.fill_each = int64_t(32e3 / row_bytes) + 1;
      const uint32_t fill = uint32_t((a.fill_rest + a.fill_each - 1) / a.fill_each);
      a.fill_ctas = uint32_t(uint64_t(fill) * 3 / 4);
      a.fill_last = fill - a.fill_ctas;
    }
    const auto kernel = !scan ? fill_kernel<false, int32_t>
                        : ids_dtype == TRAIN_INT64 ? fill_kernel<true, int64_t>
                                                   : fill_kernel<true, int32_t>;
    ce = launch(kernel, dim3(unsigned(ctas)), kFillThreads, 0, s, true, 1, a);
  }
  if (ce == cudaSuccess) {
    const bool wide = grad_out_dtype == TRAIN_FP32 || (accumulate && grad_dtype == TRAIN_FP32);
    const int64_t slab = wide ? 8 * kWarp : 16 * kWarp;
    a.slabs = int32_t((dim + slab - 1) / slab);
    a.units = p.n_blocks * a.slabs;
    const int64_t ctas = (a.units + kSumWarps - 1) / kSumWarps + a.fill_ctas;
    const SumKernel kernel = sum_kernels[grad_out_dtype][wide ? 0 : 1][aligned ? 1 : 0];
    ce = launch(kernel, dim3(unsigned(ctas)), kSumWarps * kWarp, kSumWarps * sizeof(WarpSmem), s,
                true, 1, a);
  }
  if (ce == cudaSuccess && (n_ids > 2 * p.block || a.fill_last > 0)) {
    // As many CTAs as run at once, or the slabs of the runs that there can be.
    a.join_slabs = uint32_t((dim + kJoinCols - 1) / kJoinCols);
    int64_t joins = n_ids > 2 * p.block ? (p.n_blocks / 2) * 4 * int64_t(a.join_slabs) : 0;
    if (joins > 1216) joins = 1216;
    a.join_ctas = uint32_t(joins);
    ce = launch(join_kernel, dim3(a.join_ctas + a.fill_last), kJoinThreads, 0, s, true, 1, a);
  }
  return ce == cudaSuccess
             ? LAMB_OK
             : fail(LAMB_ERR_CUDA, std::string("embed_grad: ") + cudaGetErrorString(ce));
}

}  // extern "C"
