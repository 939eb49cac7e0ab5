// norm.cu -- LayerNorm's forward pass and the backward passes of LayerNorm
// and RMSNorm (the RMSNorm forward pass is the quantizing producer in
// quant_tiles.cu, which returns the rstd read here).
//
//   forward   mean = avg(x), var = avg((x - mean)^2), rstd = 1 / sqrt(var + eps)
//             y = (x - mean) * rstd * gamma + beta
//   backward  xh = (x - mean) * rstd (RMSNorm: mean = 0), g = dy * gamma
//             dx = rstd * (g - avg(g) - xh * avg(g * xh)) [+ dres]
//             (RMSNorm: without avg(g));  dgamma = sum over rows of dy * xh,
//             dbeta = sum over rows of dy
//
// All arithmetic is FP32; every output is rounded once.  Both passes are
// bound by HBM: a row is read once into registers and its sums taken there.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8bq {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// gamma or beta at columns [c, c + VEC): NULL stands for `none`.
template <class T, int VEC>
__device__ __forceinline__ void load_params(float (&out)[VEC], const void* src, bool f32, int64_t c, float none) {
  if (src == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = none;
  } else if (f32) {
    Pack<float, VEC> p;
    load_pack(p, static_cast<const float*>(src) + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = p.v[i];
  } else {
    Pack<T, VEC> p;
    load_pack(p, static_cast<const T*>(src) + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = p.f(i);
  }
}

// Sums of two values over the block (every thread gets them), through
// red[2 * warps].  The caller separates uses of one `red` by a barrier.
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

// ---------------------------------------------------------------- forward --
struct FwdParams {
  const void* x;
  void* y;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  int64_t M, N, ldx, ldy;
  float n, eps;
  bool p32;  // gamma and beta are FP32 (else the rows' type)
};

// rstd from the sums of d = x - m and d^2, m the rounded mean: the mean is
// m + shift exactly where m alone is not (rows far from zero).
__device__ __forceinline__ float2 finish_stats(float2 s, const FwdParams& p) {
  const float shift = __fdiv_rn(s.x, p.n);
  const float var = fmaxf(fmaf(-shift, shift, __fdiv_rn(s.y, p.n)), 0.0f);
  return make_float2(shift, __fdiv_rn(1.0f, __fsqrt_rn(var + p.eps)));
}

// One row per warp (WARP) or per block, held in registers: NV packs of VEC
// elements a thread.
template <class T, int VEC, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) ln_fwd_kernel(const FwdParams p) {
  __shared__ float2 red[2][32];
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int stride = WARP ? 32 : blockDim.x;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.M) return;  // WARP: whole warps only
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const int n = static_cast<int>(p.N);
  Pack<T, VEC> v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * stride) * VEC;
    if (c < n) load_pack<true>(v[j], x + c);
  }
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((t + j * stride) * VEC < n) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) s.x += v[j].f(i);
    }
  const float m = __fdiv_rn(WARP ? warp_sum(s.x) : block_sum2(s, red[0]).x, p.n);
  s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((t + j * stride) * VEC < n) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = v[j].f(i) - m;
        s.x += d;
        s.y = fmaf(d, d, s.y);
      }
    }
  s = WARP ? make_float2(warp_sum(s.x), warp_sum(s.y)) : block_sum2(s, red[1]);
  const float2 st = finish_stats(s, p);
  if (t == 0) {
    if (p.mean != nullptr) p.mean[row] = m + st.x;
    if (p.rstd != nullptr) p.rstd[row] = st.y;
  }
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * stride) * VEC;
    if (c < n) {
      float g[VEC], b[VEC];
      load_params<T, VEC>(g, p.gamma, p.p32, c, 1.0f);
      load_params<T, VEC>(b, p.beta, p.p32, c, 0.0f);
      Pack<T, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        o.v[i] = from_float<T>(fmaf((v[j].f(i) - m - st.x) * st.y, g[i], b[i]));
      store_pack(y + c, o);
    }
  }
}

// Rows too long for the registers of one block: read three times.
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
  const float2 st = finish_stats(block_sum2(s, red[1]), p);
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = m + st.x;
    if (p.rstd != nullptr) p.rstd[row] = st.y;
  }
  T* y = static_cast<T*>(p.y) + row * p.ldy;
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    float g[1], b[1];
    load_params<T, 1>(g, p.gamma, p.p32, c, 1.0f);
    load_params<T, 1>(b, p.beta, p.p32, c, 0.0f);
    y[c] = from_float<T>(fmaf((to_float(x[c]) - m - st.x) * st.y, g[0], b[0]));
  }
}

// Whether gamma, beta can be read in packs of `vec` elements.
bool params_aligned(const void* p, bool f32, int64_t size, int vec) {
  const int64_t bytes = std::min<int64_t>(16, (f32 ? 4 : size) * vec);
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

template <class T, int VEC, int NV>
cudaError_t run_fwd(const FwdParams& p, int threads, cudaStream_t stream) {
  if (threads == 0)
    ln_fwd_kernel<T, VEC, NV, true><<<static_cast<unsigned>((p.M + 7) / 8), 256, 0, stream>>>(p);
  else
    ln_fwd_kernel<T, VEC, NV, false><<<static_cast<unsigned>(p.M), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

// The smallest number of packs a thread that fits a row of `slots` packs into
// a warp, a block of 256 threads, of 512 or of 1024; 0 threads: a warp.
template <class T, int VEC>
cudaError_t pick_fwd(const FwdParams& p, cudaStream_t stream) {
  constexpr int kMost = VEC == 8 ? 8 : 16;
  const int64_t slots = (p.N + VEC - 1) / VEC;
  for (int limit : {32, 256, 512, 1024})
    for (int nv = 1; nv <= kMost; nv *= 2) {
      const int64_t threads = ((slots + nv - 1) / nv + 31) / 32 * 32;
      if (threads > limit) continue;
      const int th = limit == 32 ? 0 : static_cast<int>(threads);
      switch (nv) {
        case 1: return run_fwd<T, VEC, 1>(p, th, stream);
        case 2: return run_fwd<T, VEC, 2>(p, th, stream);
        case 4: return run_fwd<T, VEC, 4>(p, th, stream);
        case 8: return run_fwd<T, VEC, 8>(p, th, stream);
        default:
          if constexpr (kMost == 16) return run_fwd<T, VEC, 16>(p, th, stream);
      }
    }
  ln_fwd_long_kernel<T><<<static_cast<unsigned>(p.M), 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class T>
cudaError_t fwd_of_type(const FwdParams& p, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  if (p.N % kVec == 0 && rows_aligned(p.x, p.ldx, sizeof(T), 16) && rows_aligned(p.y, p.ldy, sizeof(T), 16) &&
      params_aligned(p.gamma, p.p32, sizeof(T), kVec) && params_aligned(p.beta, p.p32, sizeof(T), kVec))
    return pick_fwd<T, kVec>(p, stream);
  return pick_fwd<T, 1>(p, stream);
}

// --------------------------------------------------------------- backward --
struct BwdParams {
  const void* dy;
  const void* x;
  const void* dres;  // or NULL
  void* dx;
  const void* gamma;  // or NULL
  const float* mean;
  const void* rstd;
  float* partial;  // [blocks][LN ? 2 : 1][N] sums of dgamma, dbeta, or NULL
  int64_t M, N, lddy, ldx, lddres, lddx;
  float inv_n;
  bool p32, rstd64;
  int tpr;  // threads a row: a multiple of 32
  // the ring of rows in shared memory
  int stages;
  bool packed;  // every tensor's rows follow one another without gaps
  int* status;
};

__device__ __forceinline__ float load_rstd(const BwdParams& p, int64_t row) {
  return p.rstd64 ? static_cast<float>(static_cast<const double*>(p.rstd)[row]) : static_cast<const float*>(p.rstd)[row];
}

// A block of G = blockDim.x / tpr rows at a time, tpr threads each; a thread
// keeps its columns (NV packs of VEC) for the whole launch, with their gamma
// and their sums of dgamma and dbeta in registers.
template <class T, int VEC, int NV, bool LN>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const BwdParams p) {
  __shared__ float2 red[2][16];
  extern __shared__ float join[];  // [LN ? 2 : 1][N], blocks of several rows only
  const int tpr = p.tpr, groups = blockDim.x / tpr;
  const int group = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int warps = tpr >> 5, warp0 = group * warps;  // the row's warps
  const int n = static_cast<int>(p.N);
  float gam[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * tpr) * VEC;
    if (c < n) load_params<T, VEC>(gam[j], p.gamma, p.p32, c, 1.0f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[j][i] = db[j][i] = 0.0f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int buf = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < p.M; row0 += step, buf ^= 1) {
    const int64_t row = row0 + group;
    const bool live = row < p.M;
    Pack<T, VEC> vx[NV], vy[NV], vr[NV];
    float mean = 0.0f, rstd = 0.0f;
    float2 s = make_float2(0.0f, 0.0f);
    if (live) {
      const T* x = static_cast<const T*>(p.x) + row * p.ldx;
      const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
      const T* res = static_cast<const T*>(p.dres) + row * p.lddres;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        if (c < n) {
          load_pack<true>(vx[j], x + c);
          load_pack<true>(vy[j], dy + c);
          if (p.dres != nullptr) load_pack<true>(vr[j], res + c);
        }
      }
      if (LN) mean = p.mean[row];
      rstd = load_rstd(p, row);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if ((t + j * tpr) * VEC < n) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float xh = (vx[j].f(i) - mean) * rstd, d = vy[j].f(i), g = d * gam[j][i];
            if (LN) s.x += g;
            s.y = fmaf(g, xh, s.y);
            dg[j][i] = fmaf(d, xh, dg[j][i]);
            if (LN) db[j][i] += d;
          }
        }
    }
    if (LN) s.x = warp_sum(s.x);
    s.y = warp_sum(s.y);
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = s;
      __syncthreads();  // the next use of this buffer is two barriers away
      s = make_float2(0.0f, 0.0f);
      for (int w = 0; w < warps; ++w) {
        s.x += red[buf][warp0 + w].x;
        s.y += red[buf][warp0 + w].y;
      }
    }
    if (live) {
      const float c1 = s.x * p.inv_n, c2 = s.y * p.inv_n;
      T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        if (c < n) {
          Pack<T, VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float xh = (vx[j].f(i) - mean) * rstd;
            float g = fmaf(vy[j].f(i), gam[j][i], LN ? -c1 : 0.0f);
            g = fmaf(-xh, c2, g) * rstd;
            if (p.dres != nullptr) g += vr[j].f(i);
            o.v[i] = from_float<T>(g);
          }
          store_pack(dx + c, o);
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  // the block's groups in order, through shared memory, then one row of sums
  for (int k = 1; k < groups; ++k) {
    __syncthreads();
    if (group == k) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int c = (t + j * tpr) * VEC + i;
          if (c < n) {
            join[c] = dg[j][i];
            if (LN) join[n + c] = db[j][i];
          }
        }
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int c = (t + j * tpr) * VEC + i;
          if (c < n) {
            dg[j][i] += join[c];
            if (LN) db[j][i] += join[n + c];
          }
        }
    }
  }
  if (group == 0) {
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * (LN ? 2 : 1) * n;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int c = (t + j * tpr) * VEC + i;
        if (c < n) {
          out[c] = dg[j][i];
          if (LN) out[n + c] = db[j][i];
        }
      }
  }
}

// K sums over the warp at once (K a power of two): halves of the values change
// places with halves of the lanes, so that K + log2(32 / K) shuffles do the
// work of 5 K.  The lane with its low bits 0 holds value `index`.
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

constexpr int kMostStages = 8;
constexpr int kTimeoutNorm = 30;

// The backward pass for 16-byte aligned rows.  A block takes groups * R rows
// at a time, tpr threads each row; bulk copies fill a ring of `stages` such
// row blocks in shared memory, so that the loads run ahead of the sums (the
// first kernel, which loaded rows into registers, spent its time waiting for
// them: 2.8 TB/s at [16384, 2048] BF16 with a residual).  A thread keeps its
// columns for the whole launch, their dgamma and dbeta in registers; x and dy
// are read from shared memory twice, before and after the row's sums.
// FULL: every thread has columns (N = tpr * NV * VEC); RES: dres is given.
template <class T, int NV, int R, bool LN, bool RES, bool FULL>
__global__ void __launch_bounds__(512) norm_bwd_ring_kernel(const BwdParams p) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int K = LN ? 2 * R : R;       // sums a thread takes part in
  constexpr bool kGammaRegs = NV * VEC <= 16;  // else read again for each row
  constexpr int kTensors = RES ? 3 : 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][16][K];
  __shared__ __align__(8) uint64_t full_bar[kMostStages];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tpr = p.tpr, groups = blockDim.x / tpr;
  const int group = tid / tpr, t = tid - group * tpr;
  const int warps = tpr >> 5, warp0 = group * warps;
  const int n = static_cast<int>(p.N);
  const int rows_a_block = groups * R;
  const uint32_t row_bytes = static_cast<uint32_t>(n * sizeof(T));
  const uint32_t tensor_bytes = row_bytes * rows_a_block, stage_bytes = tensor_bytes * kTensors;
  const int64_t row_blocks = (p.M + rows_a_block - 1) / rows_a_block;
  const int mine = static_cast<int>((row_blocks - 1 - blockIdx.x) / gridDim.x) + 1;  // row blocks of this block
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * rows_a_block;
  const WaitGuard guard{&abort_flag, p.status, 2000000000ull};  // every wait is bounded

  // warp 0: the copies of this block's next row block into the next stage
  int64_t fetch_row = static_cast<int64_t>(blockIdx.x) * rows_a_block;
  int fetch_stage = 0;
  auto fetch = [&]() {
    const int64_t row0 = fetch_row;
    if (row0 >= p.M || *guard.abort_flag != 0) return;
    const int rows = static_cast<int>(min(static_cast<int64_t>(rows_a_block), p.M - row0));
    const uint32_t bar = smem_u32(&full_bar[fetch_stage]), dst = smem_u32(ring) + fetch_stage * stage_bytes;
    if (lane == 0) mbar_arrive_expect_tx(bar, rows * kTensors * row_bytes);
    __syncwarp();
    if (p.packed) {
      if (lane < kTensors) {
        const T* src = static_cast<const T*>(lane == 0 ? p.x : lane == 1 ? p.dy : p.dres);
        bulk_load(dst + lane * tensor_bytes, src + row0 * n, rows * row_bytes, bar);
      }
    } else {
      for (int i = lane; i < kTensors * rows; i += 32) {
        const int r = i / kTensors, tensor = i - r * kTensors;
        const T* src = static_cast<const T*>(tensor == 0 ? p.x : tensor == 1 ? p.dy : p.dres);
        const int64_t ld = tensor == 0 ? p.ldx : tensor == 1 ? p.lddy : p.lddres;
        bulk_load(dst + tensor * tensor_bytes + r * row_bytes, src + (row0 + r) * ld, row_bytes, bar);
      }
    }
    fetch_row += row_step;
    fetch_stage = fetch_stage + 1 == p.stages ? 0 : fetch_stage + 1;
  };

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&full_bar[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == 0)
    for (int i = 0; i < p.stages; ++i) fetch();

  float2 gam[kGammaRegs ? NV : 1][VEC / 2];
  float2 dg[NV][VEC / 2], db[NV][VEC / 2];
  auto gamma_at = [&](int c, float2 (&out)[VEC / 2]) {
    float g[VEC];
    load_params<T, VEC>(g, p.gamma, p.p32, c, 1.0f);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) out[i] = make_float2(g[2 * i], g[2 * i + 1]);
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * tpr) * VEC;
    if constexpr (kGammaRegs)
      if (FULL || c < n) gamma_at(c, gam[j]);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) dg[j][i] = db[j][i] = make_float2(0.0f, 0.0f);
  }
  // The rows' statistics, fetched one row block ahead: lane r holds row r's
  // rstd, lane R + r its mean; zeros for rows past the last.
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_a_block + group * R;
  const float* stat = LN && lane >= R ? p.mean : static_cast<const float*>(p.rstd);
  const int stat_row = LN && lane >= R ? lane - R : lane;
  const bool stat_lane = lane < K && !(p.rstd64 && lane < R);
  float next = 0.0f;
  double next64 = 0.0;
  auto statistics = [&](int64_t row) {
    next = 0.0f;
    if (stat_lane && row + stat_row < p.M) next = stat[row + stat_row];
    if (p.rstd64) {
      next64 = 0.0;
      if (lane < R && row + lane < p.M) next64 = static_cast<const double*>(p.rstd)[row + lane];
    }
  };
  statistics(row0);

  int stage = 0, buf = 0;
  uint32_t parity = 0;
  for (int it = 0; it < mine; ++it, buf ^= 1, row0 += row_step) {
    float2 mean[R];  // negated
    float rstd[R];
    if (p.rstd64 && lane < R) next = static_cast<float>(next64);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = __shfl_sync(0xffffffffu, next, r);
      const float a = LN ? -__shfl_sync(0xffffffffu, next, R + r) : 0.0f;
      mean[r] = make_float2(a, a);
    }
    statistics(row0 + row_step);
    const int live = static_cast<int>(min(static_cast<int64_t>(R), p.M - row0));  // rows of this group, or less than 1
    mbar_wait(smem_u32(&full_bar[stage]), parity, guard, kTimeoutNorm);
    T* sx = reinterpret_cast<T*>(ring + stage * stage_bytes + group * R * row_bytes);
    T* sy = reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(sx) + tensor_bytes);
    const T* sr = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(sy) + tensor_bytes);
    if (live < R) {  // rows past the last add nothing: each thread clears the values it reads
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (t + j * tpr) * VEC;
          if (r >= live && (FULL || c < n)) {
            *reinterpret_cast<uint4*>(sx + r * n + c) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(sy + r * n + c) = make_uint4(0, 0, 0, 0);
          }
        }
    }
    float v[K];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
      const float2 rs = make_float2(rstd[r], rstd[r]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        if (FULL || c < n) {
          Pack<T, VEC> x, y;
          load_pack(x, sx + r * n + c);
          load_pack(y, sy + r * n + c);
          float2 gj[VEC / 2];
          if constexpr (!kGammaRegs) gamma_at(c, gj);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float2 d = y.f2(i), g = __fmul2_rn(d, kGammaRegs ? gam[kGammaRegs ? j : 0][i] : gj[i]);
            const float2 xh = __fmul2_rn(LN ? __fadd2_rn(x.f2(i), mean[r]) : x.f2(i), rs);
            if (LN) s1 = __fadd2_rn(s1, g);
            s2 = __ffma2_rn(g, xh, s2);
            dg[j][i] = __ffma2_rn(d, xh, dg[j][i]);
            if (LN) db[j][i] = __fadd2_rn(db[j][i], d);
          }
        }
      }
      v[r] = s2.x + s2.y;
      if constexpr (LN) v[R + r] = s1.x + s1.y;
    }
    int index;
    const float part = warp_sums<K>(v, lane, index);
    if ((lane & (32 / K - 1)) == 0) red[buf][warp][index] = part;
    __syncthreads();  // the last use of `red[buf]` and of the previous stage is over
    if (warp == 0 && it > 0) fetch();
    // lane w * K + k adds value k of every (32 / K)-th warp from w on
    float sum = 0.0f;
    for (int w = lane / K; w < warps; w += 32 / K) sum += red[buf][warp0 + w][lane % K];
#pragma unroll
    for (int o = K; o < 32; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum *= -p.inv_n;
    // dx = rstd * g + (-rstd * c1) + (x - mean) * (-rstd^2 * c2)
    T* dx = static_cast<T*>(p.dx) + row0 * p.lddx;
#pragma unroll
    for (int r = 0; r < R; ++r, dx += p.lddx) {
      const float k2 = __shfl_sync(0xffffffffu, sum, r) * rstd[r] * rstd[r];
      const float k1 = LN ? __shfl_sync(0xffffffffu, sum, (R + r) % 32) * rstd[r] : 0.0f;
      const float2 c1 = make_float2(k1, k1), c2 = make_float2(k2, k2), rs = make_float2(rstd[r], rstd[r]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        if (FULL || c < n) {
          Pack<T, VEC> x, y, z, o;
          load_pack(x, sx + r * n + c);
          load_pack(y, sy + r * n + c);
          if (RES) load_pack(z, sr + r * n + c);
          float2 gj[VEC / 2];
          if constexpr (!kGammaRegs) gamma_at(c, gj);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float2 g = __fmul2_rn(y.f2(i), kGammaRegs ? gam[kGammaRegs ? j : 0][i] : gj[i]);
            float2 d = LN ? __ffma2_rn(__fadd2_rn(x.f2(i), mean[r]), c2, c1) : __fmul2_rn(x.f2(i), c2);
            d = __ffma2_rn(g, rs, d);
            o.set2(i, RES ? __fadd2_rn(d, z.f2(i)) : d);
          }
          if (r < live) store_pack(dx + c, o);
        }
      }
    }
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1;
    }
  }
  __syncthreads();
  if (*static_cast<volatile int*>(&abort_flag) != 0) {
    // a copy never came: give the ones in flight some more time before the
    // shared memory they write is given up
    if (tid == 0) {
      const WaitGuard last{&abort_flag, p.status, 100000000ull};
      for (int i = 0; i < p.stages; ++i) {
        abort_flag = 0;
        mbar_wait(smem_u32(&full_bar[i]), i < stage ? parity ^ 1 : parity, last, kTimeoutNorm);
      }
    }
    __syncthreads();
    return;
  }
  if (p.partial == nullptr) return;
  float* join = reinterpret_cast<float*>(ring);  // [LN ? 2 : 1][N]: no copy is in flight any more
  for (int k = 1; k < groups; ++k) {
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      __syncthreads();
      if (group != (turn == 0 ? k : 0)) continue;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + j * tpr) * VEC;
        if (c < n) {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            float2* a = reinterpret_cast<float2*>(join + c) + i;
            float2* b = reinterpret_cast<float2*>(join + n + c) + i;
            if (turn == 0) {
              *a = dg[j][i];
              if (LN) *b = db[j][i];
            } else {
              dg[j][i] = __fadd2_rn(dg[j][i], *a);
              if (LN) db[j][i] = __fadd2_rn(db[j][i], *b);
            }
          }
        }
      }
    }
  }
  if (group == 0) {
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * (LN ? 2 : 1) * n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * tpr) * VEC;
      if (c < n) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          reinterpret_cast<float2*>(out + c)[i] = dg[j][i];
          if (LN) reinterpret_cast<float2*>(out + n + c)[i] = db[j][i];
        }
      }
    }
  }
}

// Rows too long for the registers of one block: the sums over rows column by
// column, and dx row by row (read twice).
template <class T, bool LN>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdParams p) {
  __shared__ float2 red[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const T* res = static_cast<const T*>(p.dres) + row * p.lddres;
  const float mean = LN ? p.mean[row] : 0.0f, rstd = load_rstd(p, row);
  float2 s = make_float2(0.0f, 0.0f);
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    float gam[1];
    load_params<T, 1>(gam, p.gamma, p.p32, c, 1.0f);
    const float g = to_float(dy[c]) * gam[0];
    s.x += g;
    s.y = fmaf(g, (to_float(x[c]) - mean) * rstd, s.y);
  }
  s = block_sum2(s, red);
  const float c1 = LN ? s.x * p.inv_n : 0.0f, c2 = s.y * p.inv_n;
  T* dx = static_cast<T*>(p.dx) + row * p.lddx;
  for (int64_t c = threadIdx.x; c < p.N; c += blockDim.x) {
    float gam[1];
    load_params<T, 1>(gam, p.gamma, p.p32, c, 1.0f);
    float g = fmaf(to_float(dy[c]), gam[0], -c1);
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
  float* out = p.partial + static_cast<int64_t>(blockIdx.y) * (LN ? 2 : 1) * p.N;
  out[c] = dg;
  if (LN) out[p.N + c] = db;
}

// dgamma and dbeta from the blocks' partial sums, in a fixed order: a block
// takes 32 columns, its 16 warps every 16th partial each.
__global__ void __launch_bounds__(512) norm_param_grad_kernel(const float* __restrict__ partial, int64_t parts,
                                                              int64_t width, int64_t N, float* dgamma, float* dbeta,
                                                              bool accumulate) {
  __shared__ float red[16][33];
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < width) {
#pragma unroll 4
    for (int64_t k = warp; k < parts; k += 16) s += partial[k * width + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= width) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += red[w][lane];
  float* out = c < N ? dgamma : dbeta;
  if (out == nullptr) return;
  out += c < N ? c : c - N;
  *out = accumulate ? *out + s : s;
}

// How a backward pass is laid out: threads a row and packs a thread, rows a
// block, blocks and the ring's stages (0: rows loaded straight into
// registers).  nv = 0: rows too long for a block's registers.
struct BwdPlan {
  int vec, nv, tpr, groups, rows, stages;
  int64_t blocks;
};

constexpr int64_t kRingBytes = 224 * 1024;  // of an SM's shared memory, for the rings of its blocks

// Bytes of dynamic shared memory a block needs beside its ring (none) and
// statically, rounded up, with what the system keeps of it.
constexpr int64_t kRingExtra = 3 * 1024;

BwdPlan plan_ring(int64_t M, int64_t N, int64_t size, int tensors, int sms) {
  const int vec = static_cast<int>(16 / size);
  BwdPlan b{vec, 0, 0, 1, 1, 0, 0};
  if (N % vec != 0) return b;
  const int64_t slots = N / vec;
  // One pack a thread where 256 threads hold the row, 16 columns where 512
  // do, 32 for the longest rows.
  for (const auto& [limit, most] : {std::pair<int, int>{256, vec}, {256, 16}, {512, 16}, {512, 32}}) {
    for (int nv = 1; nv * vec <= most && b.nv == 0; nv *= 2) {
      const int64_t tpr = ((slots + nv - 1) / nv + 31) / 32 * 32;
      if (tpr <= limit) {
        b.nv = nv;
        b.tpr = static_cast<int>(tpr);
      }
    }
  }
  if (b.nv == 0) return b;
  // As many rows between two barriers as leave the ring two stages (measured
  // at [16384, 2048] BF16 with a residual, LayerNorm: 75 us with one row, 57
  // with two, 51 with four).
  b.groups = std::max(1, 256 / b.tpr);
  const int per_sm = b.tpr > 256 ? 1 : 2;
  const int64_t room = kRingBytes / per_sm - kRingExtra, row = N * size * tensors * b.groups;
  b.rows = b.nv * vec <= 8 ? 4 : b.nv * vec <= 16 ? 2 : 1;
  while (b.rows > 1 && room / (row * b.rows) < 2) b.rows /= 2;
  b.stages = static_cast<int>(std::min<int64_t>(kMostStages, room / (row * b.rows)));
  if (b.stages < 2) {
    b.nv = 0;
    return b;
  }
  const int64_t row_blocks = (M + b.groups * b.rows - 1) / (b.groups * b.rows);
  b.blocks = std::min<int64_t>(row_blocks, static_cast<int64_t>(per_sm) * sms);
  return b;
}

BwdPlan plan_direct(int64_t M, int64_t N, int sms) {
  BwdPlan b{1, 0, 0, 1, 1, 0, 0};
  for (int limit : {256, 512})
    for (int nv = 1; nv <= 16 && b.nv == 0; nv *= 2) {
      const int64_t tpr = ((N + nv - 1) / nv + 31) / 32 * 32;
      if (tpr <= limit) {
        b.nv = nv;
        b.tpr = static_cast<int>(tpr);
      }
    }
  if (b.nv == 0) {
    b.blocks = std::min<int64_t>(M, std::max<int64_t>(1, 4 * sms / ((N + 255) / 256)));
    return b;
  }
  b.groups = std::max(1, 256 / b.tpr);
  b.blocks = std::min<int64_t>((M + b.groups - 1) / b.groups, sms * (b.tpr > 256 ? 1 : 2));
  return b;
}

template <class T, int NV, bool LN>
cudaError_t run_direct(BwdParams p, const BwdPlan& b, cudaStream_t stream) {
  p.tpr = b.tpr;
  const size_t smem = b.groups > 1 && p.partial != nullptr ? static_cast<size_t>(p.N) * (LN ? 8 : 4) : 0;
  norm_bwd_kernel<T, 1, NV, LN><<<static_cast<unsigned>(b.blocks), b.tpr * b.groups, smem, stream>>>(p);
  return cudaGetLastError();
}

template <class T, int NV, int R, bool LN, bool RES, bool FULL>
cudaError_t run_ring_as(BwdParams p, const BwdPlan& b, cudaStream_t stream) {
  p.tpr = b.tpr;
  p.stages = b.stages;
  const int64_t row = p.N * static_cast<int64_t>(sizeof(T));
  p.packed = p.ldx == p.N && p.lddy == p.N && (p.dres == nullptr || p.lddres == p.N);
  const int64_t smem = std::max<int64_t>(row * (RES ? 3 : 2) * b.groups * R * b.stages,
                                         b.groups > 1 ? p.N * (LN ? 8 : 4) : 0);
  const auto kern = norm_bwd_ring_kernel<T, NV, R, LN, RES, FULL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(b.blocks), b.tpr * b.groups, smem, stream>>>(p);
  return cudaGetLastError();
}

template <class T, int NV, int R, bool LN>
cudaError_t run_ring_rows(const BwdParams& p, const BwdPlan& b, cudaStream_t stream) {
  const bool full = p.N == static_cast<int64_t>(b.tpr) * NV * (16 / sizeof(T));
  if (p.dres != nullptr)
    return full ? run_ring_as<T, NV, R, LN, true, true>(p, b, stream) : run_ring_as<T, NV, R, LN, true, false>(p, b, stream);
  return full ? run_ring_as<T, NV, R, LN, false, true>(p, b, stream) : run_ring_as<T, NV, R, LN, false, false>(p, b, stream);
}

template <class T, int NV, bool LN>
cudaError_t run_ring(const BwdParams& p, const BwdPlan& b, cudaStream_t stream) {
  constexpr int kCols = NV * (16 / static_cast<int>(sizeof(T)));
  if constexpr (kCols <= 8)
    if (b.rows == 4) return run_ring_rows<T, NV, 4, LN>(p, b, stream);
  if constexpr (kCols <= 16)
    if (b.rows == 2) return run_ring_rows<T, NV, 2, LN>(p, b, stream);
  return run_ring_rows<T, NV, 1, LN>(p, b, stream);
}

template <class T, bool LN>
cudaError_t bwd_of_type(const BwdParams& p, const BwdPlan& b, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  if (b.nv == 0) {
    if (p.partial != nullptr) {  // before dx, which may be written over dy or x
      const dim3 grid(static_cast<unsigned>((p.N + 255) / 256), static_cast<unsigned>(b.blocks));
      norm_cols_kernel<T, LN><<<grid, 256, 0, stream>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    norm_bwd_long_kernel<T, LN><<<static_cast<unsigned>(p.M), 1024, 0, stream>>>(p);
    return cudaGetLastError();
  }
  if (b.stages != 0) {
    switch (b.nv) {
      case 1: return run_ring<T, 1, LN>(p, b, stream);
      case 2: return run_ring<T, 2, LN>(p, b, stream);
      case 4: return run_ring<T, 4, LN>(p, b, stream);
      default:
        if constexpr (kVec == 4) return run_ring<T, 8, LN>(p, b, stream);
    }
  }
  switch (b.nv) {
    case 1: return run_direct<T, 1, LN>(p, b, stream);
    case 2: return run_direct<T, 2, LN>(p, b, stream);
    case 4: return run_direct<T, 4, LN>(p, b, stream);
    case 8: return run_direct<T, 8, LN>(p, b, stream);
    default: return run_direct<T, 16, LN>(p, b, stream);
  }
}

}  // namespace

cudaError_t launch_layernorm_fwd(const NormFwd& a, cudaStream_t stream) {
  const FwdParams p{a.x, a.y, a.gamma, a.beta, a.mean, a.rstd, a.M, a.N, a.ldx, a.ldy,
                    static_cast<float>(a.N), a.eps, a.param_dtype == FP8BQ_FP32};
  switch (a.dtype) {
    case FP8BQ_BF16: return fwd_of_type<__nv_bfloat16>(p, stream);
    case FP8BQ_FP16: return fwd_of_type<__half>(p, stream);
    default: return fwd_of_type<float>(p, stream);
  }
}

int64_t norm_bwd_workspace_bytes(int64_t M, int64_t N, int sms) {
  int64_t most = plan_direct(M, N, sms).blocks;
  for (int64_t size : {2, 4})
    for (int tensors : {2, 3}) most = std::max(most, plan_ring(M, N, size, tensors, sms).blocks);
  return most * 2 * N * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_norm_bwd(const fp8bq_norm_grad& a, bool layernorm, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  const int64_t size = a.dtype == FP8BQ_FP32 ? 4 : 2;
  const int vec = static_cast<int>(16 / size);
  const bool p32 = a.param_dtype == FP8BQ_FP32;
  const bool wide = a.N % vec == 0 && rows_aligned(a.x, a.ldx, size, 16) && rows_aligned(a.dy, a.lddy, size, 16) &&
                    rows_aligned(a.dx, a.lddx, size, 16) &&
                    (a.dres == nullptr || rows_aligned(a.dres, a.lddres, size, 16)) &&
                    params_aligned(a.gamma, p32, size, vec);
  BwdPlan b{};
  if (wide) b = plan_ring(a.M, a.N, size, a.dres != nullptr ? 3 : 2, sms);
  if (b.nv == 0) b = plan_direct(a.M, a.N, sms);
  int* status = nullptr;
  e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  const BwdParams p{a.dy, a.x, a.dres, a.dx, a.gamma, a.mean, a.rstd,
                    sums ? static_cast<float*>(a.workspace) : nullptr,
                    a.M, a.N, a.lddy, a.ldx, a.lddres, a.lddx, 1.0f / static_cast<float>(a.N), p32,
                    (a.flags & FP8BQ_NORM_RSTD_F64) != 0, 0, 0, false, status};
  if (a.M > 0) {
    switch (a.dtype) {
      case FP8BQ_BF16:
        e = layernorm ? bwd_of_type<__nv_bfloat16, true>(p, b, stream) : bwd_of_type<__nv_bfloat16, false>(p, b, stream);
        break;
      case FP8BQ_FP16:
        e = layernorm ? bwd_of_type<__half, true>(p, b, stream) : bwd_of_type<__half, false>(p, b, stream);
        break;
      default: e = layernorm ? bwd_of_type<float, true>(p, b, stream) : bwd_of_type<float, false>(p, b, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  const int64_t width = a.N * (layernorm ? 2 : 1);
  return launch_dependent(norm_param_grad_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(512), 0, stream,
                          static_cast<const float*>(a.workspace), a.M > 0 ? b.blocks : int64_t{0}, width, a.N, a.dgamma,
                          layernorm ? a.dbeta : nullptr, (a.flags & FP8BQ_NORM_ACCUMULATE) != 0);
}

}  // namespace fp8bq
