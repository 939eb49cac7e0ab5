// norm_fwd.cu -- LayerNorm's forward pass (RMSNorm's is the quantizing producer
// in quant_tiles.cu).
//
//   mean = avg(x), var = avg((x - mean)^2), rstd = 1 / sqrt(var + eps)
//   y = (x - mean) * rstd * gamma + beta
//
// FP32 arithmetic, y rounded once.  Bound by HBM: every value is read once,
// through a ring of rows in shared memory, and worked on in registers.  The
// statistics take two passes over those registers: each warp sums its columns
// and then, about its own mean, their deviations and squares; the warps'
// results are joined about the first warp's mean, so that rows far from zero
// lose nothing and one barrier serves the rows between it and the next.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "row_ring.cuh"

namespace fp8bq {
namespace {

struct FwdParams {
  const void* x;
  void* y;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  int64_t N, ldx, ldy;
  float n, eps;
  bool p32;  // gamma and beta are FP32 (else the rows' type)
  int tpr;   // threads a row, a multiple of 32
};

// A variance that rounding left below 0 is 0; one that is NaN (a row with NaN or
// an infinity) gives NaN.
__device__ __forceinline__ float rstd_of(float var, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn((var < 0.0f ? 0.0f : var) + eps));
}

// A sum over each SUB lanes.
template <int SUB>
__device__ __forceinline__ float sub_sum(float v) {
#pragma unroll
  for (int o = SUB / 2; o >= 1; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A team of tpr threads takes a row at a time (SUB = 8: a team of one warp four
// rows, 8 lanes each), COLS columns a thread, which stay in registers from one
// pass to the next.  Teams share nothing but gamma and beta: SHARED keeps
// those in shared memory, as FP32 pairs, else (few rows, or the longest; one
// team a block) in registers.  Few threads with many columns, because the sums
// over a team cost as much for one column as for many: [16384, 2048] BF16
// takes 26.3 us (5.1 TB/s, 78% of the copy rate) with one warp a row, 36 us
// with 128 threads a row and 16 columns each.  FULL: the threads' columns are
// the row's, without checks (5-7% faster than zero padding).
template <class T, int COLS, int SUB, bool ALIGNED, bool FULL, bool SHARED>
__global__ void __launch_bounds__(512, COLS <= 24 ? 2 : 1) ln_fwd_kernel(const __grid_constant__ FwdParams p,
                                                     const __grid_constant__ RingParams rp) {
  constexpr int W = ALIGNED ? 16 / static_cast<int>(sizeof(T)) : 8, G = COLS / W;
  constexpr int R = 32 / SUB;  // rows a team takes at a time
  using Cols = Group<T, W, ALIGNED, FULL>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[16][kMostStages];
  __shared__ int abort_flag;
  __shared__ float centre[2][16], sums[2][16], squares[2][16], held[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int members = SUB < 32 ? 32 : p.tpr, team = tid / members, teams = blockDim.x / members;
  const int tpr = SUB < 32 ? SUB : p.tpr, t = SUB < 32 ? lane % SUB : tid - team * members;  // threads a row
  const int warps = members >> 5, warp0 = team * warps;
  const int n = rp.n;
  cudaGridDependencySynchronize();

  // rows over the SMs first
  const int64_t first_row = (blockIdx.x + static_cast<int64_t>(gridDim.x) * team) * R;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
  float4* const params = reinterpret_cast<float4*>(smem);  // [COLS / 2][tpr]: a pair's gammas, its betas
  uint8_t* const rings = smem + (SHARED ? COLS / 2 * tpr * static_cast<int>(sizeof(float4)) : 0);
  RowRing<T, 1, ALIGNED> ring(rp, rings + team * rp.stages * rp.stage_bytes, bars[team], &abort_flag, first_row, step);
  if constexpr (ALIGNED && !FULL) {  // rows are padded with zeros to the threads' columns
    const int rows = teams * rp.stages * R, tail = static_cast<int>(rp.pitch - rp.row_bytes) / 16;
    for (int i = tid; i < rows * tail; i += blockDim.x) {
      const int r = i / tail;
      *reinterpret_cast<uint4*>(rings + r * rp.pitch + rp.row_bytes + (i - r * tail) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  const bool leader = tid == team * members;
  ring.init(leader);
  if (warp == warp0) ring.start();

  float2 gam[SHARED ? 1 : G][W / 2], bet[SHARED ? 1 : G][W / 2];
  if constexpr (SHARED) {
    for (int j = tid / tpr; j < G; j += blockDim.x / tpr) {
      float2 g[W / 2], b[W / 2];
      Cols::load_param(g, p.gamma, p.p32, 1.0f, t, tpr, j, n);
      Cols::load_param(b, p.beta, p.p32, 0.0f, t, tpr, j, n);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) params[(j * (W / 2) + i) * tpr + t] = make_float4(g[i].x, g[i].y, b[i].x, b[i].y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      Cols::load_param(gam[j], p.gamma, p.p32, 1.0f, t, tpr, j, n);
      Cols::load_param(bet[j], p.beta, p.p32, 0.0f, t, tpr, j, n);
    }
  }
  float count = 0.0f;  // this warp's columns
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int k = 0; k < W; ++k) count += FULL || Cols::column(t, tpr, j, k) < n ? 1.0f : 0.0f;
  count = sub_sum<SUB>(count);
  const float inv_count = count > 0.0f ? __fdiv_rn(1.0f, count) : 0.0f;
  if (lane == 0) held[warp] = count;
  __syncthreads();

  int buf = 0;
  for (int64_t row0 = first_row; row0 < rp.M; row0 += step, buf ^= 1) {
    ring.wait();
    const int64_t row = row0 + (SUB < 32 ? lane / SUB : 0);
    const T* x = ring.row(0, row0, SUB < 32 ? lane / SUB : 0);
    float2 v[G][W / 2];
    float2 sum = make_float2(0.0f, 0.0f), sum2 = sum;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if constexpr (ALIGNED)
        Cols::load_padded(v[j], x, t, tpr, j);
      else
        Cols::load(v[j], x, t, tpr, j, n);
#pragma unroll
      for (int i = 0; i < W / 2; i += 2) {
        sum = __fadd2_rn(sum, v[j][i]);
        sum2 = __fadd2_rn(sum2, v[j][i + 1]);
      }
    }
    sum = __fadd2_rn(sum, sum2);
    const float mid = sub_sum<SUB>(sum.x + sum.y) * inv_count;
    const float2 m2 = make_float2(-mid, -mid);
    float2 sq = make_float2(0.0f, 0.0f), sq2 = sq;
    sum = sum2 = sq;
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) v[j][i] = __fadd2_rn(v[j][i], m2);
      Cols::clear_rest(v[j], t, tpr, j, n);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        float2& s = i % 2 ? sum2 : sum;
        float2& q = i % 2 ? sq2 : sq;
        s = __fadd2_rn(s, v[j][i]);
        q = __ffma2_rn(v[j][i], v[j][i], q);
      }
    }
    sum = __fadd2_rn(sum, sum2);
    sq = __fadd2_rn(sq, sq2);
    const float s = sub_sum<SUB>(sum.x + sum.y), q = sub_sum<SUB>(sq.x + sq.y);
    // the row's mean is base + avg: base a rounded mean, avg what it is off by
    float base = mid, avg, var;
    if (warps > 1) {
      if (lane == 0) {
        centre[buf][warp] = mid;
        sums[buf][warp] = s;
        squares[buf][warp] = q;
      }
      named_bar_sync(team + 1, tpr);  // the row is in the team's registers
      if (warp == warp0) ring.fetch();
      base = centre[buf][warp0];
      const int w = warp0 + (lane < warps ? lane : 0);
      const float c = lane < warps ? held[w] : 0.0f, off = centre[buf][w] - base, sw = lane < warps ? sums[buf][w] : 0.0f;
      avg = __fdiv_rn(warp_sum(fmaf(c, off, sw)), p.n);
      // about the mean: sum (d + a)^2 = sum d^2 + 2 a sum d + count a^2
      const float a = off - avg;
      var = __fdiv_rn(warp_sum(lane < warps ? fmaf(a, fmaf(c, a, 2.0f * sw), squares[buf][w]) : 0.0f), p.n);
    } else {
      __syncwarp();
      ring.fetch();
      avg = __fdiv_rn(s, p.n);
      var = __fdiv_rn(fmaf(-avg, s, q), p.n);
    }
    const float rstd = rstd_of(var, p.eps);
    const bool live = SUB == 32 || row < rp.M;
    if (t == 0 && live) {
      if (p.mean != nullptr) p.mean[row] = base + avg;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    const float a = mid - base - avg;
    const float2 a2 = make_float2(a, a), rs2 = make_float2(rstd, rstd);
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        float2 g, b;
        if constexpr (SHARED) {
          const float4 both_params = params[(j * (W / 2) + i) * tpr + t];
          g = make_float2(both_params.x, both_params.y);
          b = make_float2(both_params.z, both_params.w);
        } else {
          g = gam[j][i];
          b = bet[j][i];
        }
        v[j][i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[j][i], a2), rs2), g, b);
      }
      if (live) Cols::store(y, v[j], t, tpr, j, n);
    }
    ring.next();
  }
  ring.finish(leader);
}

// Rows too long for a block: read three times.
template <class T>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(const FwdParams p) {
  __shared__ float2 red[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  float2 s = make_float2(0.0f, 0.0f);
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) s.x += to_float(x[c]);
  const float m = __fdiv_rn(block_sum2(s, red[0]).x, p.n);
  s = make_float2(0.0f, 0.0f);
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    const float d = to_float(x[c]) - m;
    s.x += d;
    s.y = fmaf(d, d, s.y);
  }
  s = block_sum2(s, red[1]);
  const float avg = __fdiv_rn(s.x, p.n), rstd = rstd_of(__fdiv_rn(fmaf(-avg, s.x, s.y), p.n), p.eps);
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = m + avg;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * p.ldy;
  const auto param = [&](const void* v, int64_t c, float none) {
    return v == nullptr ? none : p.p32 ? static_cast<const float*>(v)[c] : to_float(static_cast<const T*>(v)[c]);
  };
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x)
    y[c] = from_float<T>(fmaf((to_float(x[c]) - m - avg) * rstd, param(p.gamma, c, 1.0f), param(p.beta, c, 0.0f)));
}

template <class T, int COLS, int SUB, bool ALIGNED, bool FULL, bool SHARED>
cudaError_t run_as(FwdParams p, const RowPlan& b, cudaStream_t stream) {
  p.tpr = b.tpr;
  const auto kern = ln_fwd_kernel<T, COLS, SUB, ALIGNED, FULL, SHARED>;
  const int smem = static_cast<int>(b.ring.stage_bytes) * b.ring.stages * b.groups + (SHARED ? b.tpr * COLS * 8 : 0);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(static_cast<unsigned>(b.blocks)), dim3(std::max(32, b.tpr) * b.groups), smem, stream, p,
                          b.ring);
}

template <class T, int COLS, int SUB, bool ALIGNED, bool SHARED>
cudaError_t run(const FwdParams& p, const RowPlan& b, cudaStream_t stream) {
  if constexpr (ALIGNED && SHARED)
    if (p.N == static_cast<int64_t>(b.tpr) * COLS) return run_as<T, COLS, SUB, true, true, SHARED>(p, b, stream);
  return run_as<T, COLS, SUB, ALIGNED, false, SHARED>(p, b, stream);
}

template <class T, bool ALIGNED>
cudaError_t run_plan(const FwdParams& p, const RowPlan& b, cudaStream_t stream) {
  if (b.tpr == 8) {
    if (b.cols == 8) return run<T, 8, 8, ALIGNED, true>(p, b, stream);
    if (b.cols == 16) return run<T, 16, 8, ALIGNED, true>(p, b, stream);
    return run<T, 32, 8, ALIGNED, true>(p, b, stream);
  }
  switch (b.cols) {
    case 8: return run<T, 8, 32, ALIGNED, false>(p, b, stream);
    case 16: return run<T, 16, 32, ALIGNED, true>(p, b, stream);
    case 32: return b.tpr == 32 ? run<T, 32, 32, ALIGNED, true>(p, b, stream) : run<T, 32, 32, ALIGNED, false>(p, b, stream);
    case 24: return run<T, 24, 32, ALIGNED, true>(p, b, stream);
    case 40: return run<T, 40, 32, ALIGNED, true>(p, b, stream);
    case 48: return run<T, 48, 32, ALIGNED, true>(p, b, stream);
    default: return run<T, 64, 32, ALIGNED, true>(p, b, stream);
  }
}

// Few rows, not too long: a block each, 8 columns a thread ([200, 1283] FP32
// 4.7 us; the teams below, which first bring gamma and beta to shared memory,
// 6.9; [290, 640] FP32 3.6 and 4.9, [290, 4096] BF16 4.8 and 4.2, [600, 2048]
// 6.3 and 4.2).
// Rows of up to 256 columns: 8 lanes each.  Else teams of one warp where 64
// columns a thread hold the row, or the team and columns (48 or 64) that leave
// the fewest idle; as many teams a block, up to 16 warps, as leave each two
// stages.  The longest rows, whose gamma and beta do not fit beside two
// stages, take one team of 32 columns a thread.
RowPlan plan_fwd(int64_t M, int64_t N, int64_t size, bool aligned, bool packed, int sms) {
  RowPlan b{};
  const int64_t row = N * size;
  const auto threads = [&](int cols) { return ((N + cols - 1) / cols + 31) / 32 * 32; };
  int64_t room = kRingBytes - kRingExtra;
  int on_sm = 1, rows = 1;  // blocks that the registers allow; rows a team takes at a time
  bool shared = true;
  if (M <= 2 * sms && N <= 256 * 8) {
    b.cols = 8;
    b.tpr = static_cast<int>(threads(8));
    on_sm = 2;
    shared = false;
  } else if (N <= 256) {
    b.cols = N <= 64 ? 8 : N <= 128 ? 16 : 32;
    b.tpr = 8;
    rows = 4;
    on_sm = b.cols <= 16 ? 2 : 1;
  } else if (N <= 2048) {
    b.cols = N <= 512 ? 16 : N <= 768 ? 24 : N <= 1024 ? 32 : N <= 1280 ? 40 : N <= 1536 ? 48 : 64;
    b.tpr = 32;
    on_sm = b.cols <= 24 ? 2 : 1;
  } else {
    b.cols = threads(48) * 48 < threads(64) * 64 ? 48 : 64;
    b.tpr = static_cast<int>(threads(b.cols));
  }
  const auto pitch_of = [&] {
    return aligned ? static_cast<int64_t>(b.tpr) * b.cols * size : packed ? row : (row + 30) / 16 * 16;
  };
  int64_t pitch = pitch_of(), stage = aligned ? pitch * rows : (pitch * rows + 30) / 16 * 16;
  room = kRingBytes / on_sm - kRingExtra - (shared ? static_cast<int64_t>(b.tpr) * b.cols * 8 : 0);
  b.groups = static_cast<int>(std::min<int64_t>(shared ? 512 / std::max(32, b.tpr) : 1, room / (2 * stage)));
  if (b.groups < 1) {
    if (threads(32) > 512) return RowPlan{};
    b.cols = 32;
    b.tpr = static_cast<int>(threads(32));
    b.groups = 1;
    on_sm = 1;
    room = kRingBytes - kRingExtra;
    pitch = pitch_of();
    stage = aligned ? pitch : (pitch + 30) / 16 * 16;
    if (room < 2 * stage) return RowPlan{};
  }
  b.rows = rows;
  const int64_t row_blocks = (M + rows - 1) / rows;
  b.blocks = std::min<int64_t>(row_blocks, static_cast<int64_t>(on_sm) * sms);
  b.ring.M = M;
  b.ring.n = static_cast<int>(N);
  b.ring.rows = rows;
  b.ring.stages = static_cast<int>(std::min<int64_t>(shared ? kMostStages : 2, room / (b.groups * stage)));
  b.ring.row_bytes = static_cast<uint32_t>(row);
  b.ring.pitch = static_cast<uint32_t>(pitch);
  b.ring.tensor_bytes = b.ring.stage_bytes = static_cast<uint32_t>(stage);
  b.ring.packed = packed && (!aligned || pitch == row);
  return b;
}

template <class T>
cudaError_t fwd_of_type(const NormFwd& a, int sms, int* status, cudaStream_t stream) {
  const FwdParams p{a.x, a.y, a.gamma, a.beta, a.mean, a.rstd, a.N, a.ldx, a.ldy, static_cast<float>(a.N), a.eps,
                    a.param_dtype == FP8BQ_FP32, 0};
  const bool aligned = (a.N * sizeof(T)) % 16 == 0 && rows_aligned(a.x, a.ldx, sizeof(T), 16) &&
                       rows_aligned(a.y, a.ldy, sizeof(T), 16) && rows_aligned(a.gamma, 0, 1, 16) &&
                       rows_aligned(a.beta, 0, 1, 16);
  RowPlan b = plan_fwd(a.M, a.N, sizeof(T), aligned, a.ldx == a.N, sms);
  if (b.cols == 0) {
    ln_fwd_long_kernel<T><<<static_cast<unsigned>(a.M), 1024, 0, stream>>>(p);
    return cudaGetLastError();
  }
  b.ring.src[0] = a.x;
  b.ring.ld[0] = a.ldx;
  b.ring.status = status;
  return aligned ? run_plan<T, true>(p, b, stream) : run_plan<T, false>(p, b, stream);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const NormFwd& a, cudaStream_t stream) {
  int sms = 0;
  int* status = nullptr;
  cudaError_t e = device_sm_count(&sms);
  if (e == cudaSuccess) e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  switch (a.dtype) {
    case FP8BQ_BF16: return fwd_of_type<__nv_bfloat16>(a, sms, status, stream);
    case FP8BQ_FP16: return fwd_of_type<__half>(a, sms, status, stream);
    default: return fwd_of_type<float>(a, sms, status, stream);
  }
}

}  // namespace fp8bq
