// row_ring.cuh -- rows of one to three tensors fetched ahead into a ring in
// shared memory, for the persistent row kernels of the norms.
//
// A team (a block, or some warps of one) takes `rows` consecutive rows of
// every tensor at a time (a row block); bulk copies bring its next row blocks
// into the stages of its ring while the current one is worked on.  Rows that
// are not 16-byte aligned are fetched as the 16-byte granules that hold them
// and read from shared memory value by value; the granules at a tensor's two
// ends, which may reach past it, are copied value by value instead.  Every
// wait is bounded.
#pragma once
#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8bq {

constexpr int kMostStages = 8;
constexpr int kTimeoutRows = 30;
// An SM's shared memory for the rings of its blocks, and what a block needs
// of it beside its ring (static arrays and what the system keeps).
constexpr int64_t kRingBytes = 228 * 1024;
constexpr int64_t kRingExtra = 3 * 1024;
// What every kernel with a ring is allowed: one value for all launches, since
// other host threads may be between setting it and launching.
constexpr int kMostDynamic = static_cast<int>(kRingBytes - kRingExtra);

struct RingParams {
  const void* src[3];
  int64_t ld[3];
  int64_t M;
  int n, rows, stages;
  uint32_t row_bytes, pitch;            // bytes of a row, and from one row to the next in a stage
  uint32_t tensor_bytes, stage_bytes;   // of a stage
  bool packed;                          // every tensor's rows follow one another without gaps
  int* status;
};

// ALIGNED: every row starts at a multiple of 16 bytes and is as long as one.
template <class T, int TENSORS, bool ALIGNED>
struct RowRing {
  const RingParams& p;
  uint8_t* ring;
  uint64_t* bars;   // [kMostStages], the team's own
  int* abort_flag;  // the block's
  int64_t fetch_row, step;
  int fetch_stage, stage;
  uint32_t parity;

  // The team's ring and barriers, its first row and the rows from one of its
  // row blocks to the next.  The whole block calls init, with `leader` one
  // thread of each team; then the first warp of each team calls start.
  __device__ __forceinline__ RowRing(const RingParams& params, uint8_t* smem, uint64_t* barriers, int* flag, int64_t first,
                                     int64_t stride)
      : p(params), ring(smem), bars(barriers), abort_flag(flag), fetch_row(first), step(stride) {
    fetch_stage = stage = 0;
    parity = 0;
  }
  __device__ __forceinline__ void init(bool leader) {
    if (threadIdx.x == 0) *abort_flag = 0;
    if (leader) {
      for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&bars[i]), 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ void start() {
    for (int i = 0; i < p.stages; ++i) fetch();
  }

  __device__ __forceinline__ WaitGuard guard() const { return WaitGuard{abort_flag, p.status, 2000000000ull}; }

  // The granules [from, to) of the bytes [a, e) of a tensor that bulk copies
  // may take: all that hold a value, less those that reach past the tensor.
  __device__ __forceinline__ void granules(uintptr_t a, uintptr_t e, int tensor, uintptr_t& from, uintptr_t& to) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p.src[tensor]);
    const uintptr_t hi = lo + static_cast<uintptr_t>((p.M - 1) * p.ld[tensor] * static_cast<int64_t>(sizeof(T))) + p.row_bytes;
    from = a & ~uintptr_t{15};
    if (from < lo) from += 16;
    to = (e + 15) & ~uintptr_t{15};
    if (to > hi) to -= 16;
    if (to < from) to = from;
  }

  // The team's first warp: the next row block into the next stage.
  __device__ __forceinline__ void fetch() {
    const int lane = threadIdx.x & 31;
    const int64_t row0 = fetch_row;
    if (row0 >= p.M) return;
    // one lane's reading for the warp: another team may set the flag meanwhile,
    // and lanes that left would be waited for below
    if (__shfl_sync(0xffffffffu, lane == 0 ? *static_cast<volatile int*>(abort_flag) : 0, 0) != 0) return;
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.M - row0));
    const uint32_t bar = smem_u32(&bars[fetch_stage]);
    uint8_t* base = ring + fetch_stage * p.stage_bytes;
    const int copies = p.packed ? TENSORS : TENSORS * rows;
    const uint32_t bytes = p.packed ? rows * p.row_bytes : p.row_bytes;
    if constexpr (ALIGNED) {
      if (lane == 0) mbar_arrive_expect_tx(bar, rows * TENSORS * p.row_bytes);
      __syncwarp();
      for (int i = lane; i < copies; i += 32) {
        const int r = i / TENSORS, tensor = i - r * TENSORS;
        bulk_load(smem_u32(base) + tensor * p.tensor_bytes + r * p.pitch,
                  static_cast<const T*>(p.src[tensor]) + (row0 + r) * p.ld[tensor], bytes, bar);
      }
    } else {
      uint32_t total = 0;
      for (int i = lane; i < copies; i += 32) {
        const int r = i / TENSORS, tensor = i - r * TENSORS;
        const T* src = static_cast<const T*>(p.src[tensor]) + (row0 + r) * p.ld[tensor];
        const uintptr_t a = reinterpret_cast<uintptr_t>(src), e = a + bytes;
        uintptr_t from, to;
        granules(a, e, tensor, from, to);
        total += static_cast<uint32_t>(to - from);
        T* dst = reinterpret_cast<T*>(base + tensor * p.tensor_bytes + r * p.pitch + (a & 15));
        const int count = static_cast<int>(bytes / sizeof(T));
        const int head = from > a ? static_cast<int>(min(from - a, e - a) / sizeof(T)) : 0;
        for (int k = 0; k < head; ++k) dst[k] = src[k];
        const int tail = to < e ? static_cast<int>((max(to, a) - a) / sizeof(T)) : count;
        for (int k = max(tail, head); k < count; ++k) dst[k] = src[k];
        if (head > 0 || tail < count) fence_proxy_async_smem();  // a later copy may write these bytes
      }
      total = __reduce_add_sync(0xffffffffu, total);
      __syncwarp();  // every lane's values are in the stage before lane 0 announces it (the sum orders no memory)
      if (lane == 0) mbar_arrive_expect_tx(bar, total);
      __syncwarp();
      for (int i = lane; i < copies; i += 32) {
        const int r = i / TENSORS, tensor = i - r * TENSORS;
        const uintptr_t a = reinterpret_cast<uintptr_t>(static_cast<const T*>(p.src[tensor]) + (row0 + r) * p.ld[tensor]);
        uintptr_t from, to;
        granules(a, a + bytes, tensor, from, to);
        if (to > from)
          bulk_load(smem_u32(base) + tensor * p.tensor_bytes + r * p.pitch + static_cast<uint32_t>(from - (a & ~uintptr_t{15})),
                    reinterpret_cast<const void*>(from), static_cast<uint32_t>(to - from), bar);
      }
    }
    fetch_row += step;
    fetch_stage = fetch_stage + 1 == p.stages ? 0 : fetch_stage + 1;
  }

  __device__ __forceinline__ void wait() const { mbar_wait(smem_u32(&bars[stage]), parity, guard(), kTimeoutRows); }

  // Row r of the current row block, whose first row is row0.
  __device__ __forceinline__ T* row(int tensor, int64_t row0, int r) const {
    uint8_t* at = ring + stage * p.stage_bytes + tensor * p.tensor_bytes + r * p.pitch;
    if constexpr (!ALIGNED) {
      const T* src = static_cast<const T*>(p.src[tensor]) + (row0 + (p.packed ? 0 : r)) * p.ld[tensor];
      at += reinterpret_cast<uintptr_t>(src) & 15;
    }
    return reinterpret_cast<T*>(at);
  }

  __device__ __forceinline__ void next() {
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1;
    }
  }

  // The end, by the whole block.  Where a copy never came, the ones in flight
  // get some more time before the shared memory they write is given up; true
  // then.
  __device__ __forceinline__ bool finish(bool leader) {
    __syncthreads();
    if (*static_cast<volatile int*>(abort_flag) == 0) return false;
    if (leader) {
      const uint64_t start = global_timer_ns();
      for (int i = 0; i < p.stages; ++i)
        while (!mbar_try_wait(smem_u32(&bars[i]), i < stage ? parity ^ 1 : parity) && global_timer_ns() - start < 100000000ull) {
        }
    }
    __syncthreads();
    return true;
  }
};

// W columns of a row for thread t of `stride`: a pack of W = 16 bytes
// (ALIGNED), or W values a stride apart; the j-th such group.  Pairs beyond
// the row's n columns are zeros.  FULL: there are none.  SPLIT: groups that
// lie within the row take code of their own, without the checks.
template <class T, int W, bool ALIGNED, bool FULL, bool SPLIT = true>
struct Group {
  // Column of value k.
  __device__ static __forceinline__ int column(int t, int stride, int j, int k) {
    return ALIGNED ? (t + j * stride) * W + k : t + (j * W + k) * stride;
  }

  // The same from a row padded with zeros to every thread's columns.
  __device__ static __forceinline__ void load_padded(float2 (&v)[W / 2], const T* row, int t, int stride, int j) {
    Pack<T, W> x;
    load_pack(x, row + column(t, stride, j, 0));
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = x.f2(i);
  }

  // Whether every thread's j-th group lies within the row.
  __device__ static __forceinline__ bool whole(int stride, int j, int n) { return FULL || (SPLIT && (j + 1) * W * stride <= n); }

  __device__ static __forceinline__ void load(float2 (&v)[W / 2], const T* row, int t, int stride, int j, int n) {
    if constexpr (ALIGNED) {
      const int c = column(t, stride, j, 0);
      Pack<T, W> x;
      if (FULL || c < n) load_pack(x, row + c);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) v[i] = FULL || c < n ? x.f2(i) : make_float2(0.0f, 0.0f);
    } else if (whole(stride, j, n)) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const int c = column(t, stride, j, 2 * i);
        v[i] = make_float2(to_float(row[c]), to_float(row[c + stride]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const int c = column(t, stride, j, 2 * i);
        v[i].x = c < n ? to_float(row[c]) : 0.0f;
        v[i].y = c + stride < n ? to_float(row[c + stride]) : 0.0f;
      }
    }
  }

  __device__ static __forceinline__ void store(T* row, const float2 (&v)[W / 2], int t, int stride, int j, int n) {
    if constexpr (ALIGNED) {
      const int c = column(t, stride, j, 0);
      if (!FULL && c >= n) return;
      Pack<T, W> o;
#pragma unroll
      for (int i = 0; i < W / 2; ++i) o.set2(i, v[i]);
      store_pack(row + c, o);
    } else if (whole(stride, j, n)) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const int c = column(t, stride, j, 2 * i);
        row[c] = from_float<T>(v[i].x);
        row[c + stride] = from_float<T>(v[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const int c = column(t, stride, j, 2 * i);
        if (c < n) row[c] = from_float<T>(v[i].x);
        if (c + stride < n) row[c + stride] = from_float<T>(v[i].y);
      }
    }
  }

  // Zeros in the place of values past the row.
  __device__ static __forceinline__ void clear_rest(float2 (&v)[W / 2], int t, int stride, int j, int n) {
    if constexpr (!FULL) {
      if (whole(stride, j, n)) return;
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        if (column(t, stride, j, 2 * i) >= n) v[i].x = 0.0f;
        if (column(t, stride, j, 2 * i + 1) >= n) v[i].y = 0.0f;
      }
    }
  }

  // The same columns of a parameter vector of T or FP32, `none` where it is
  // NULL, zeros past the row.
  __device__ static __forceinline__ void load_param(float2 (&v)[W / 2], const void* src, bool f32, float none, int t, int stride,
                                                    int j, int n) {
    if (src == nullptr) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        v[i].x = FULL || column(t, stride, j, 2 * i) < n ? none : 0.0f;
        v[i].y = FULL || column(t, stride, j, 2 * i + 1) < n ? none : 0.0f;
      }
    } else if (f32) {
      Group<float, W, ALIGNED, FULL, SPLIT>::load(v, static_cast<const float*>(src), t, stride, j, n);
    } else {
      load(v, static_cast<const T*>(src), t, stride, j, n);
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// K sums over the warp at once (K a power of two): halves of the values change
// places with halves of the lanes, so that K + log2(32 / K) shuffles do the
// work of 5 K.  A lane with its low bits 0 holds value `index`.
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K], int lane, int& index) {
  int o = 16;
  index = 0;
#pragma unroll
  for (int k = K; k > 1; k /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < k / 2; ++i) {
      const float give = upper ? v[i] : v[i + k / 2], keep = upper ? v[i + k / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
    if (upper) index += k / 2;
  }
  float s = v[0];
#pragma unroll
  for (; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The same within each SUB lanes; sub_sum_of gives every lane value k.
template <int K, int SUB>
__device__ __forceinline__ float sub_sums(float (&v)[K], int lane) {
  int o = SUB / 2;
#pragma unroll
  for (int k = K; k > 1; k /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < k / 2; ++i) {
      const float give = upper ? v[i] : v[i + k / 2], keep = upper ? v[i + k / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
template <int K, int SUB>
__device__ __forceinline__ float sub_sum_of(float s, int lane, int k) {
  return __shfl_sync(0xffffffffu, s, (lane & ~(SUB - 1)) + k * (SUB / K));
}

// Sums of two values over the block (every thread gets them), through
// red[warps].  The caller separates uses of one `red` by a barrier.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* red) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int w = 0; w < warps; ++w) {
    s.x += red[w].x;
    s.y += red[w].y;
  }
  return s;
}

// How a row kernel is laid out: columns a thread, threads a row, groups of
// them a block (a row each), rows a group takes between two barriers, blocks.
// cols = 0: the rows are too long for a block.
struct RowPlan {
  int cols, tpr, groups, rows;
  int64_t blocks;
  RingParams ring;
};

}  // namespace fp8bq
