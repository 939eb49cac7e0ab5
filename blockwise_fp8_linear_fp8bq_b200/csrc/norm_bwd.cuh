// norm_bwd.cuh -- the backward passes of LayerNorm and RMSNorm.
//
//   xh = (x - mean) * rstd (RMSNorm: mean = 0), g = dy * gamma
//   dx = rstd * (g - avg(g) - xh * avg(g * xh)) [+ dres]  (RMSNorm: without avg(g))
//   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
//
// FP32 arithmetic, dx rounded once.  Bound by HBM: x, dy and dres are read
// once, through a ring of rows in shared memory.  A thread keeps its columns
// for the whole launch, their dgamma and dbeta in registers; the blocks' sums
// go to the workspace and are added in a fixed order by a second kernel.
// [16384, 2048] BF16 with a residual: LayerNorm 51.2 us on the GPU (5.2 TB/s, 80%
// of the copy rate; 54.0 a call in a loop), RMSNorm 48.0 (85%; 50.0); the first
// kernel, which loaded rows straight into registers, took 94 and 86, waiting for
// them.  Few rows (small_batch) leave
// those sums to further blocks of the same launch, which read x and dy again,
// from L2: one launch instead of two, and no workspace.
//
// Included by one source for each element type (they compile side by side) and
// by norm_bwd.cu, which lays the launches out.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "row_ring.cuh"

namespace fp8bq {

struct BwdParams {
  const void* dy;
  const void* x;
  const void* dres;  // or NULL
  void* dx;
  const void* gamma;  // or NULL
  const float* mean;
  const void* rstd;
  float* partial;  // [blocks][LN ? 2 : 1][N] sums of dgamma, dbeta, or NULL
  float* dgamma;   // few rows: written by the column blocks; either may be NULL
  float* dbeta;
  int row_blocks;  // the blocks that take rows; the others take columns
  bool accumulate, in_place;  // in_place: dx overlaps x or dy
  int64_t M, N, lddy, ldx, lddres, lddx;
  float inv_n;
  bool p32, rstd64;
  int tpr;  // threads a row, a multiple of 32
};

// The launches of a planned backward pass (b.cols = 0: rows too long for a
// block, `blocks` of them for each column's sum), for one element type.
template <class T>
cudaError_t run_norm_bwd(const BwdParams& p, const RowPlan& b, bool layernorm, bool aligned, int64_t blocks,
                         cudaStream_t stream);

// Shared memory for gamma.
inline int64_t gamma_bytes(const RowPlan& b, int64_t size) { return b.cols > 16 ? static_cast<int64_t>(b.tpr) * b.cols * size : 0; }

namespace {

__device__ __forceinline__ float load_rstd(const BwdParams& p, int64_t row) {
  return p.rstd64 ? static_cast<float>(static_cast<const double*>(p.rstd)[row]) : static_cast<const float*>(p.rstd)[row];
}

__device__ __forceinline__ void write_sum(float* out, int64_t c, float s, bool accumulate) {
  if (out != nullptr) out[c] = accumulate ? out[c] + s : s;
}

// Few rows: the sums over rows of one block's slice of columns, 8 lanes of W
// columns (ALIGNED: four rows a warp at a time) or 32 lanes of one.
constexpr int kSliceFloats = 2 * 64 * 64;  // of shared memory

template <class T, bool LN, bool ALIGNED>
__device__ __forceinline__ void column_block(const BwdParams& p, float* join) {
  constexpr int W = ALIGNED ? 16 / static_cast<int>(sizeof(T)) : 1, kLanes = ALIGNED ? 8 : 32, kSlice = kLanes * W;
  constexpr int kBatch = 4;
  const int lane = threadIdx.x % kLanes, strip = threadIdx.x / kLanes, strips = blockDim.x / kLanes;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - p.row_blocks) * kSlice, c = c0 + lane * W;
  float dg[W], db[W];
#pragma unroll
  for (int i = 0; i < W; ++i) dg[i] = db[i] = 0.0f;
  if (c < p.N) {
    for (int64_t row = strip; row < p.M; row += kBatch * strips) {
      Pack<T, W> x[kBatch], y[kBatch];
      float mean[kBatch], rstd[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t r = row + k * strips;
        if (r < p.M) {
          load_pack(x[k], static_cast<const T*>(p.x) + r * p.ldx + c);
          load_pack(y[k], static_cast<const T*>(p.dy) + r * p.lddy + c);
          mean[k] = LN ? p.mean[r] : 0.0f;
          rstd[k] = load_rstd(p, r);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (row + k * strips < p.M) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            dg[i] = fmaf(y[k].f(i), (x[k].f(i) - mean[k]) * rstd[k], dg[i]);
            db[i] += y[k].f(i);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    join[strip * kSlice + lane * W + i] = dg[i];
    join[(strips + strip) * kSlice + lane * W + i] = db[i];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < (LN ? 2 : 1) * kSlice; k += blockDim.x) {
    const int which = k / kSlice, col = k - which * kSlice;
    if (c0 + col >= p.N) continue;
    float s = 0.0f;
    for (int w = 0; w < strips; ++w) s += join[(which * strips + w) * kSlice + col];
    write_sum(which == 0 ? p.dgamma : p.dbeta, c0 + col, s, p.accumulate);
  }
}

// tpr threads a row (SUB = 8: 8 lanes of a warp), COLS columns each, R rows a
// thread between two barriers; x and dy are read from shared memory twice,
// before and after the row's sums.  Aligned rows are padded there with zeros
// to the threads' columns, so that reading them needs no checks (14-40% of
// the time where N is not a multiple of the threads' columns).  RES: dres is
// given.
template <class T, int COLS, int R, int SUB, bool LN, bool RES, bool ALIGNED>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const __grid_constant__ BwdParams p,
                                                       const __grid_constant__ RingParams rp) {
  constexpr int W = ALIGNED ? 16 / static_cast<int>(sizeof(T)) : 8, G = COLS / W;
  constexpr int K = LN ? 2 * R : R;               // sums a thread takes part in
  constexpr bool kGammaRegs = COLS <= 16;         // else in shared memory, behind the ring
  using Cols = Group<T, W, ALIGNED, false, false>;
  using Sums = Group<float, W, ALIGNED, false, false>;
  extern __shared__ __align__(128) uint8_t smem[];
  cudaGridDependencySynchronize();
  if (blockIdx.x >= static_cast<unsigned>(p.row_blocks)) {
    column_block<T, LN, ALIGNED>(p, reinterpret_cast<float*>(smem));
    return;
  }
  __shared__ float red[2][16][K];
  __shared__ __align__(8) uint64_t bars[kMostStages];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tpr = SUB < 32 ? SUB : p.tpr;
  const int group = tid / tpr, t = tid - group * tpr;
  const int warps = tpr >> 5, warp0 = group * warps;  // of a row; SUB < 32: none
  const int n = rp.n;
  if constexpr (ALIGNED) {
    const int rows = rp.stages * rp.rows * (RES ? 3 : 2), tail = static_cast<int>(rp.pitch - rp.row_bytes) / 16;
    for (int i = tid; i < rows * tail; i += blockDim.x) {
      const int r = i / tail;
      *reinterpret_cast<uint4*>(smem + r * rp.pitch + rp.row_bytes + (i - r * tail) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  const auto load = [&](float2 (&v)[W / 2], const T* row, int j) {
    if constexpr (ALIGNED)
      Cols::load_padded(v, row, t, tpr, j);
    else
      Cols::load(v, row, t, tpr, j, n);
  };
  const int64_t row_step = static_cast<int64_t>(p.row_blocks) * rp.rows;
  int64_t block_row = static_cast<int64_t>(blockIdx.x) * rp.rows;
  RowRing<T, RES ? 3 : 2, ALIGNED> ring(rp, smem, bars, &abort_flag, block_row, row_step);
  ring.init(tid == 0);
  if (warp == 0) ring.start();

  // gamma: pair i of group j of thread t at [(j * W / 2 + i) * tpr + t], as FP32
  // or T pairs, whichever it came as
  uint8_t* const gamma_at = smem + rp.stages * rp.stage_bytes;
  const bool wide_gamma = p.p32 || p.gamma == nullptr;
  const auto keep_gamma = [&](int j) {
    float2 g[W / 2];
    Cols::load_param(g, p.gamma, p.p32, 1.0f, t, tpr, j, n);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const int at = (j * (W / 2) + i) * tpr + t;
      if (sizeof(T) == 4 || wide_gamma)
        reinterpret_cast<float2*>(gamma_at)[at] = g[i];
      else
        from_float2(reinterpret_cast<T*>(gamma_at) + 2 * at, g[i]);
    }
  };
  const auto kept_gamma = [&](float2 (&g)[W / 2], int j) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const int at = (j * (W / 2) + i) * tpr + t;
      g[i] = sizeof(T) == 4 || wide_gamma ? reinterpret_cast<const float2*>(gamma_at)[at]
                                          : to_float2(reinterpret_cast<const T*>(gamma_at) + 2 * at);
    }
  };
  float2 gam[kGammaRegs ? G : 1][W / 2];
  float2 dg[G][W / 2], db[G][W / 2];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if constexpr (kGammaRegs)
      Cols::load_param(gam[j], p.gamma, p.p32, 1.0f, t, tpr, j, n);
    else
      keep_gamma(j);  // each thread reads only what it wrote itself
#pragma unroll
    for (int i = 0; i < W / 2; ++i) dg[j][i] = db[j][i] = make_float2(0.0f, 0.0f);
  }
  // The rows' statistics, fetched one row block ahead: lane r (of SUB) holds
  // row r's rstd, lane R + r its mean; zeros for rows past the last.
  const int sub = lane % SUB, sub0 = lane - sub;
  const float* stat = LN && sub >= R ? p.mean : static_cast<const float*>(p.rstd);
  const int stat_row = LN && sub >= R ? sub - R : sub;
  const bool stat_lane = sub < K && !(p.rstd64 && sub < R);
  float next = 0.0f;
  double next64 = 0.0;
  auto statistics = [&](int64_t row) {
    next = 0.0f;
    if (stat_lane && row + stat_row < rp.M) next = stat[row + stat_row];
    if (p.rstd64) {
      next64 = 0.0;
      if (sub < R && row + sub < rp.M) next64 = static_cast<const double*>(p.rstd)[row + sub];
    }
  };
  statistics(block_row + group * R);

  int buf = 0;
  for (bool begun = false; block_row < rp.M; block_row += row_step, buf ^= 1, begun = true) {
    const int64_t row0 = block_row + group * R;
    float2 mean[R];  // negated
    float rstd[R];
    if (p.rstd64 && sub < R) next = static_cast<float>(next64);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = __shfl_sync(0xffffffffu, next, sub0 + r);
      const float a = LN ? -__shfl_sync(0xffffffffu, next, sub0 + R + r) : 0.0f;
      mean[r] = make_float2(a, a);
    }
    statistics(row0 + row_step);
    const int live = static_cast<int>(min(static_cast<int64_t>(R), rp.M - row0));  // rows of this group, or less than 1
    ring.wait();
    if (live < R) {  // rows past the last add nothing: each thread clears the values it reads
      const float2 zeros[W / 2] = {};
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (r >= live) {
            Cols::store(ring.row(0, block_row, group * R + r), zeros, t, tpr, j, n);
            Cols::store(ring.row(1, block_row, group * R + r), zeros, t, tpr, j, n);
          }
    }
    float v[K];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T* sx = ring.row(0, block_row, group * R + r);
      const T* sy = ring.row(1, block_row, group * R + r);
      float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
      const float2 rs = make_float2(rstd[r], rstd[r]);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float2 x[W / 2], y[W / 2], gj[W / 2];
        load(x, sx, j);
        load(y, sy, j);
        if constexpr (!kGammaRegs) kept_gamma(gj, j);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          const float2 g = __fmul2_rn(y[i], kGammaRegs ? gam[kGammaRegs ? j : 0][i] : gj[i]);
          const float2 xh = __fmul2_rn(LN ? __fadd2_rn(x[i], mean[r]) : x[i], rs);
          if (LN) s1 = __fadd2_rn(s1, g);
          s2 = __ffma2_rn(g, xh, s2);
          dg[j][i] = __ffma2_rn(y[i], xh, dg[j][i]);
          if (LN) db[j][i] = __fadd2_rn(db[j][i], y[i]);
        }
      }
      v[r] = s2.x + s2.y;
      if constexpr (LN) v[R + r] = s1.x + s1.y;
    }
    float sum = 0.0f;
    if constexpr (SUB < 32) {
      sum = sub_sums<K, SUB>(v, lane);
      __syncthreads();  // the last use of the previous stage is over
      if (warp == 0 && begun) ring.fetch();
    } else {
      int index;
      const float part = warp_sums<K>(v, lane, index);
      if ((lane & (32 / K - 1)) == 0) red[buf][warp][index] = part;
      __syncthreads();  // the last use of red[buf] and of the previous stage is over
      if (warp == 0 && begun) ring.fetch();
      // lane w * K + k adds value k of every (32 / K)-th warp from w on
      for (int w = lane / K; w < warps; w += 32 / K) sum += red[buf][warp0 + w][lane % K];
#pragma unroll
      for (int o = K; o < 32; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const auto value = [&](int k) {
      if constexpr (SUB < 32) return sub_sum_of<K, SUB>(sum, lane, k);
      return __shfl_sync(0xffffffffu, sum, k % 32);
    };
    sum *= -p.inv_n;
    // dx = rstd * (g - c1 - xh * c2): rstd stays a factor of its own on either
    // side, since rstd^2 leaves FP32's range long before x, rstd and dx do
    T* dx = static_cast<T*>(p.dx) + row0 * p.lddx;
#pragma unroll
    for (int r = 0; r < R; ++r, dx += p.lddx) {
      const float k2 = value(r), k1 = LN ? value(R + r) : 0.0f;
      if (SUB == 32 && r >= live) break;  // (SUB < 32: the warp's other rows may live)
      const float2 c1 = make_float2(k1, k1), c2 = make_float2(k2, k2), rs = make_float2(rstd[r], rstd[r]);
      const T* sx = ring.row(0, block_row, group * R + r);
      const T* sy = ring.row(1, block_row, group * R + r);
      const T* sr = ring.row(RES ? 2 : 0, block_row, group * R + r);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float2 x[W / 2], y[W / 2], z[W / 2], gj[W / 2];
        load(x, sx, j);
        load(y, sy, j);
        if (RES) load(z, sr, j);
        if constexpr (!kGammaRegs) kept_gamma(gj, j);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          const float2 gi = kGammaRegs ? gam[kGammaRegs ? j : 0][i] : gj[i];
          const float2 xh = __fmul2_rn(LN ? __fadd2_rn(x[i], mean[r]) : x[i], rs);
          float2 d = LN ? __ffma2_rn(xh, c2, c1) : __fmul2_rn(xh, c2);
          d = __ffma2_rn(y[i], gi, d);
          x[i] = RES ? __ffma2_rn(d, rs, z[i]) : __fmul2_rn(d, rs);
        }
        if (SUB == 32 || r < live) Cols::store(dx, x, t, tpr, j, n);
      }
    }
    ring.next();
  }
  if (ring.finish(tid == 0) || p.partial == nullptr) return;
  // A warp's rows, then the block's groups (SUB < 32: its warps) in order,
  // through the ring's memory (no copy is in flight any more), then one row of
  // sums.
  if constexpr (SUB < 32) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < W / 2; ++i)
#pragma unroll
        for (int o = SUB; o < 32; o *= 2) {
          dg[j][i].x += __shfl_xor_sync(0xffffffffu, dg[j][i].x, o);
          dg[j][i].y += __shfl_xor_sync(0xffffffffu, dg[j][i].y, o);
          if (LN) db[j][i].x += __shfl_xor_sync(0xffffffffu, db[j][i].x, o);
          if (LN) db[j][i].y += __shfl_xor_sync(0xffffffffu, db[j][i].y, o);
        }
  }
  const int joins = SUB < 32 ? blockDim.x / 32 : blockDim.x / tpr, mine = SUB < 32 ? warp : group;
  const bool holds = SUB == 32 || lane < SUB;
  float* join = reinterpret_cast<float*>(smem);  // [LN ? 2 : 1][N]
  for (int k = 1; k < joins; ++k) {
    __syncthreads();
    if (mine == k && holds) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        Sums::store(join, dg[j], t, tpr, j, n);
        if (LN) Sums::store(join + n, db[j], t, tpr, j, n);
      }
    }
    __syncthreads();
    if (mine == 0 && holds) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float2 a[W / 2], b[W / 2];
        Sums::load(a, join, t, tpr, j, n);
        if (LN) Sums::load(b, join + n, t, tpr, j, n);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          dg[j][i] = __fadd2_rn(dg[j][i], a[i]);
          if (LN) db[j][i] = __fadd2_rn(db[j][i], b[i]);
        }
      }
    }
  }
  if (mine == 0 && holds) {
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * (LN ? 2 : 1) * n;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      Sums::store(out, dg[j], t, tpr, j, n);
      if (LN) Sums::store(out + n, db[j], t, tpr, j, n);
    }
  }
}

// Rows too long for a block: the sums over rows column by
// column, and dx row by row (read twice).
template <class T, bool LN>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdParams p) {
  __shared__ float2 red[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const T* res = static_cast<const T*>(p.dres) + row * p.lddres;
  const float mean = LN ? p.mean[row] : 0.0f, rstd = load_rstd(p, row);
  const auto gamma = [&](int64_t c) {
    return p.gamma == nullptr ? 1.0f
           : p.p32            ? static_cast<const float*>(p.gamma)[c]
                              : to_float(static_cast<const T*>(p.gamma)[c]);
  };
  float2 s = make_float2(0.0f, 0.0f);
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    const float g = to_float(dy[c]) * gamma(c);
    s.x += g;
    s.y = fmaf(g, (to_float(x[c]) - mean) * rstd, s.y);
  }
  s = block_sum2(s, red);
  const float c1 = LN ? s.x * p.inv_n : 0.0f, c2 = s.y * p.inv_n;
  T* dx = static_cast<T*>(p.dx) + row * p.lddx;
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    float g = fmaf(to_float(dy[c]), gamma(c), -c1);
    g = fmaf(-((to_float(x[c]) - mean) * rstd), c2, g) * rstd;
    if (p.dres != nullptr) g += to_float(res[c]);
    dx[c] = from_float<T>(g);
  }
}

template <class T, bool LN>
__global__ void __launch_bounds__(256) norm_cols_kernel(const BwdParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.N) return;
  float dg = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float d = to_float(static_cast<const T*>(p.dy)[row * p.lddy + c]);
    const float xv = to_float(static_cast<const T*>(p.x)[row * p.ldx + c]);
    dg = fmaf(d, (xv - (LN ? p.mean[row] : 0.0f)) * load_rstd(p, row), dg);
    db += d;
  }
  if (p.partial == nullptr) {  // few rows: one block a column
    write_sum(p.dgamma, c, dg, p.accumulate);
    if (LN) write_sum(p.dbeta, c, db, p.accumulate);
    return;
  }
  float* out = p.partial + static_cast<int64_t>(blockIdx.y) * (LN ? 2 : 1) * p.N;
  out[c] = dg;
  if (LN) out[p.N + c] = db;
}

template <class T, int COLS, int R, int SUB, bool LN, bool RES, bool ALIGNED>
cudaError_t run_as(BwdParams p, const RowPlan& b, cudaStream_t stream) {
  if (b.cols != COLS || b.rows != R || (SUB < 32 && b.tpr != SUB)) return cudaErrorInvalidValue;  // a plan without a kernel
  p.tpr = b.tpr;
  p.row_blocks = static_cast<int>(b.blocks);
  const int64_t slice = ALIGNED ? 128 / static_cast<int64_t>(sizeof(T)) : 32;
  const bool columns = p.dgamma != nullptr || p.dbeta != nullptr;
  const int64_t slices = columns ? (p.N + slice - 1) / slice : 0;
  const auto kern = norm_bwd_kernel<T, COLS, R, SUB, LN, RES, ALIGNED>;
  const int64_t smem = std::max<int64_t>(static_cast<int64_t>(b.ring.stage_bytes) * b.ring.stages +
                                             gamma_bytes(b, p.p32 || p.gamma == nullptr ? 4 : sizeof(T)),
                                         std::max<int64_t>(b.groups > 1 ? p.N * (LN ? 8 : 4) : 0,
                                                           columns ? kSliceFloats * 4 : 0));
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
  if (e != cudaSuccess) return e;
  if (columns && p.in_place) {  // the columns are summed before dx is written over them
    BwdParams q = p;
    q.row_blocks = 0;
    kern<<<static_cast<unsigned>(slices), b.tpr * b.groups, smem, stream>>>(q, b.ring);
    kern<<<static_cast<unsigned>(b.blocks), b.tpr * b.groups, smem, stream>>>(p, b.ring);
  } else {
    return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks + slices)), dim3(b.tpr * b.groups), smem, stream, p, b.ring);
  }
  return cudaGetLastError();
}

template <class T, int COLS, int R, int SUB, bool LN, bool ALIGNED>
cudaError_t run(const BwdParams& p, const RowPlan& b, cudaStream_t stream) {
  return p.dres != nullptr ? run_as<T, COLS, R, SUB, LN, true, ALIGNED>(p, b, stream)
                           : run_as<T, COLS, R, SUB, LN, false, ALIGNED>(p, b, stream);
}

template <class T, bool LN, bool ALIGNED>
cudaError_t run_plan(const BwdParams& p, const RowPlan& b, cudaStream_t stream) {
  if (b.tpr == 8) {
    if (b.cols == 8) return run<T, 8, 2, 8, LN, ALIGNED>(p, b, stream);
    return b.rows == 2 ? run<T, 16, 2, 8, LN, ALIGNED>(p, b, stream) : run<T, 16, 1, 8, LN, ALIGNED>(p, b, stream);
  }
  if constexpr (ALIGNED && sizeof(T) == 4)
    if (b.cols == 4) return run<T, 4, 4, 32, LN, ALIGNED>(p, b, stream);
  switch (b.cols) {
    case 8: return b.rows == 4 ? run<T, 8, 4, 32, LN, ALIGNED>(p, b, stream) : run<T, 8, 2, 32, LN, ALIGNED>(p, b, stream);
    case 16: return b.rows == 2 ? run<T, 16, 2, 32, LN, ALIGNED>(p, b, stream) : run<T, 16, 1, 32, LN, ALIGNED>(p, b, stream);
    default: return run<T, 32, 1, 32, LN, ALIGNED>(p, b, stream);
  }
}

template <class T, bool LN>
cudaError_t bwd_of_type(const BwdParams& p, const RowPlan& b, bool aligned, int64_t blocks, cudaStream_t stream) {
  if (b.cols == 0) {
    if (p.partial != nullptr || p.dgamma != nullptr || p.dbeta != nullptr) {  // before dx, which may be written over dy or x
      const dim3 grid(static_cast<unsigned>((p.N + 255) / 256), static_cast<unsigned>(blocks));
      norm_cols_kernel<T, LN><<<grid, 256, 0, stream>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    norm_bwd_long_kernel<T, LN><<<static_cast<unsigned>(p.M), 1024, 0, stream>>>(p);
    return cudaGetLastError();
  }
  return aligned ? run_plan<T, LN, true>(p, b, stream) : run_plan<T, LN, false>(p, b, stream);
}

}  // namespace

template <class T>
cudaError_t run_norm_bwd(const BwdParams& p, const RowPlan& b, bool layernorm, bool aligned, int64_t blocks,
                         cudaStream_t stream) {
  return layernorm ? bwd_of_type<T, true>(p, b, aligned, blocks, stream)
                   : bwd_of_type<T, false>(p, b, aligned, blocks, stream);
}

}  // namespace fp8bq
