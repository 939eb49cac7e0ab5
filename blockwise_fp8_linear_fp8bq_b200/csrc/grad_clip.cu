// grad_clip.cu -- the global norm of many gradients, and their clipping.
//
//   norm = sqrt(sum over all tensors and values of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Bound by HBM: the values are read once for the norm and once more to be
// scaled (402 M FP32 values: 726 us on the GPU for three passes, 6.65 TB/s, 741 a
// call in a loop; the norm's kernel reads at 7.0 TB/s).  Sums are taken in a fixed order (no floating-point atomics), in
// FP32 over eight values and in float64 beyond, so that the norm of billions
// of values, of tiny or of huge ones is right to FP32's rounding.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "internal.h"

namespace fp8bq {
namespace {

constexpr int kThreads = 256;
constexpr int kPack = 8;                      // values a thread takes at once
constexpr int kUnit = kThreads * kPack;       // values a block takes at once
constexpr int kUnits = 2;                     // units of a chunk
constexpr int kChunk = kUnits * kUnit;        // values of one tensor a block takes before it looks for more
constexpr int kNormBlocks = 8;                // blocks for each SM that take the norm
constexpr int kTensors = 128;                 // tensors a launch takes at most (its parameters hold their table)
constexpr int kFewTensors = 32;               // a short list's table: 0.5 us less to launch two kernels with
// A launch's chunks fit a grid: at most 2^35 values a tensor.
static_assert((int64_t{1} << 35) / kChunk * kTensors <= INT32_MAX, "chunks of a launch");

template <int CAP>
struct Table {
  const void* g[CAP];
  void* out[CAP];
  int64_t n[CAP];
  int64_t first[CAP];  // the tensor's first chunk among the launch's
  int8_t in_dtype[CAP], out_dtype[CAP];
  int64_t chunks;
  int count;
};

// The tensor that chunk k belongs to.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& t, int64_t k) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Eight squares in FP32 where neither the sum nor what matters of it leaves
// the normal range, else in float64.
template <class T>
__device__ __forceinline__ double sum_squares(const Pack<T, kPack>& v) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPack; ++i) s = fmaf(v.f(i), v.f(i), s);
  if (s > 0x1p-80f && s < 0x1p120f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kPack; ++i) {
    const double x = v.f(i);
    if (x != 0.0) d = fma(x, x, d);
  }
  return d;
}

// A chunk of n values from g on: whole packs where g is 16-byte aligned (two
// in flight a thread), then value by value.
template <class T>
__device__ __forceinline__ double chunk_squares(const T* g, int n) {
  double s = 0.0;
  const int packs = reinterpret_cast<uintptr_t>(g) % 16 == 0 ? n / kPack : 0;
  if (packs == kUnits * kThreads) {
    Pack<T, kPack> v[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) load_pack(v[j], g + (j * kThreads + threadIdx.x) * kPack);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) s += sum_squares(v[j]);
    return s;
  }
  for (int i = threadIdx.x; i < packs; i += kThreads) {
    Pack<T, kPack> v;
    load_pack(v, g + i * kPack);
    s += sum_squares(v);
  }
  for (int i0 = packs * kPack + threadIdx.x; i0 < n; i0 += kThreads * kPack) {
    Pack<T, kPack> v;
#pragma unroll
    for (int j = 0; j < kPack; ++j) v.v[j] = i0 + j * kThreads < n ? g[i0 + j * kThreads] : from_float<T>(0.0f);
    s += sum_squares(v);
  }
  return s;
}

__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ Table<CAP> t, double* partial) {
  __shared__ double red[kThreads / 32];
  cudaGridDependencySynchronize();
  double s = 0.0;
  for (int64_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const int i = tensor_of(t, k);
    const int64_t begin = (k - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(t.n[i] - begin, static_cast<int64_t>(kChunk)));
    switch (t.in_dtype[i]) {
      case FP8BQ_BF16: s += chunk_squares(static_cast<const __nv_bfloat16*>(t.g[i]) + begin, n); break;
      case FP8BQ_FP16: s += chunk_squares(static_cast<const __half*>(t.g[i]) + begin, n); break;
      default: s += chunk_squares(static_cast<const float*>(t.g[i]) + begin, n);
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the blocks' sums: every block that calls it gets the same.
__device__ __forceinline__ double norm_of(const double* partial, int64_t parts, double* red) {
  double s = 0.0;
  for (int64_t k = threadIdx.x; k < parts; k += kThreads) s += partial[k];
  return sqrt(block_sum(s, red));
}

// The factor a * b; NaN where the norm is, 1 for an infinite limit.  b is 1
// unless the factor is so small (gradients that blew up) that FP32 would hold it
// with few bits or none although the scaled values are ordinary: then it is the
// power of two that leaves a all its bits.
struct Factor {
  float a, b;
};
__device__ __forceinline__ Factor factor_of(double norm, double max_norm) {
  if (isinf(max_norm) && !isnan(norm)) return Factor{1.0f, 1.0f};
  const double q = max_norm / (norm + 1e-6);
  if (!(q > 0.0 && q < 0x1p-100)) return Factor{static_cast<float>(q >= 1.0 ? 1.0 : q), 1.0f};
  int e;
  frexp(q, &e);
  e = max(e, -149);
  return Factor{static_cast<float>(ldexp(q, -e)), static_cast<float>(ldexp(1.0, e))};
}

// The norm, and the factor for a scaling kernel of many blocks.
__global__ void __launch_bounds__(kThreads) norm_kernel(const double* partial, int64_t parts, double max_norm, float* norm,
                                                        Factor* factor) {
  __shared__ double red[kThreads / 32];
  cudaGridDependencySynchronize();
  const double r = norm_of(partial, parts, red);
  if (threadIdx.x != 0) return;
  *norm = static_cast<float>(r);
  if (factor != nullptr) *factor = factor_of(r, max_norm);
}

template <class T, class O>
__device__ __forceinline__ void scale_chunk(const T* g, O* out, int n, Factor f) {
  if (f.b != 1.0f) {  // rare; a second product in the loops below costs 1-2%
    for (int i = threadIdx.x; i < n; i += kThreads) out[i] = from_float<O>(to_float(g[i]) * f.a * f.b);
    return;
  }
  const int packs = (reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) % 16 == 0 ? n / kPack : 0;
  const auto put = [&](const Pack<T, kPack>& v, int i) {
    Pack<O, kPack> o;
#pragma unroll
    for (int j = 0; j < kPack; ++j) o.v[j] = from_float<O>(v.f(j) * f.a);
    store_pack<true>(out + i * kPack, o);
  };
  if (packs == kUnits * kThreads) {
    Pack<T, kPack> v[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) load_pack<true>(v[j], g + (j * kThreads + threadIdx.x) * kPack);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) put(v[j], j * kThreads + threadIdx.x);
    return;
  }
  for (int i = threadIdx.x; i < packs; i += kThreads) {
    Pack<T, kPack> v;
    load_pack<true>(v, g + i * kPack);
    put(v, i);
  }
#pragma unroll 4
  for (int i = packs * kPack + threadIdx.x; i < n; i += kThreads) out[i] = from_float<O>(to_float(g[i]) * f.a);
}

template <class T, int CAP>
__device__ __forceinline__ void scale_to(const Table<CAP>& t, int i, int64_t begin, int n, Factor f) {
  const T* g = static_cast<const T*>(t.g[i]) + begin;
  switch (t.out_dtype[i]) {
    case FP8BQ_BF16: scale_chunk(g, static_cast<__nv_bfloat16*>(t.out[i]) + begin, n, f); break;
    case FP8BQ_FP16: scale_chunk(g, static_cast<__half*>(t.out[i]) + begin, n, f); break;
    default: scale_chunk(g, static_cast<float*>(t.out[i]) + begin, n, f);
  }
}

// One chunk a block (blocks that stay and stride over the chunks: 564 us where
// this takes 466), in the reverse of the norm's order: those read last may
// still be in L2.  A short list's blocks take the factor from the norm's
// partial sums themselves (factor NULL).  Tensors scaled in place by a factor
// of 1 are left alone.
template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> t, const double* partial,
                                                         int64_t parts, double max_norm, float* norm, const Factor* factor) {
  __shared__ double red[kThreads / 32];
  cudaGridDependencySynchronize();
  Factor f;
  if (factor != nullptr) {
    f = *factor;
  } else {
    const double r = norm_of(partial, parts, red);
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm != nullptr) *norm = static_cast<float>(r);
    f = factor_of(r, max_norm);
  }
  const int64_t k = t.chunks - 1 - blockIdx.x;
  const int i = tensor_of(t, k);
  if (f.a == 1.0f && f.b == 1.0f && t.g[i] == t.out[i]) return;
  const int64_t begin = (k - t.first[i]) * kChunk;
  const int n = static_cast<int>(min(t.n[i] - begin, static_cast<int64_t>(kChunk)));
  switch (t.in_dtype[i]) {
    case FP8BQ_BF16: scale_to<__nv_bfloat16>(t, i, begin, n, f); break;
    case FP8BQ_FP16: scale_to<__half>(t, i, begin, n, f); break;
    default: scale_to<float>(t, i, begin, n, f);
  }
}

// The table of tensors [at, ...) of the list that one launch takes, empty
// tensors left out; returns where the next launch starts.
template <int CAP>
int fill_table(const fp8bq_grad* grads, int count, int at, Table<CAP>* t) {
  t->count = 0;
  t->chunks = 0;
  for (; at < count && t->count < CAP; ++at) {
    const fp8bq_grad& g = grads[at];
    if (g.n == 0) continue;
    const int i = t->count++;
    t->g[i] = g.g;
    t->out[i] = g.out;
    t->n[i] = g.n;
    t->first[i] = t->chunks;
    t->in_dtype[i] = static_cast<int8_t>(g.dtype);
    t->out_dtype[i] = static_cast<int8_t>(g.out_dtype);
    t->chunks += (g.n + kChunk - 1) / kChunk;
  }
  return at;
}

// Blocks of the norm's launch.
int64_t blocks_of(int64_t chunks, int sms) { return std::min<int64_t>(chunks, kNormBlocks * static_cast<int64_t>(sms)); }

template <int CAP>
cudaError_t run_grad_clip(const fp8bq_grad* grads, int count, double max_norm, bool clip, float* norm, void* workspace,
                          cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  Factor* factor = static_cast<Factor*>(workspace);
  double* partial = static_cast<double*>(workspace) + 2;
  int64_t parts = 0, chunks = 0;
  Table<CAP> t;
  for (int at = 0; at < count;) {
    at = fill_table(grads, count, at, &t);
    if (t.chunks == 0) break;
    const int64_t blocks = blocks_of(t.chunks, sms);
    e = launch_dependent(square_kernel<CAP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, t, partial + parts);
    if (e != cudaSuccess) return e;
    parts += blocks;
    chunks += t.chunks;
  }
  // Many chunks: the factor by a kernel of its own (10 M FP32 values: 24.1 us
  // against 24.8; 4 M: 12.7 against 12.4; 1 M: 6.6 against 5.7).
  const bool many = chunks > 8 * static_cast<int64_t>(sms);
  if (!clip || parts == 0 || many) {
    e = launch_dependent(norm_kernel, dim3(1), dim3(kThreads), 0, stream, static_cast<const double*>(partial), parts, max_norm,
                         norm, clip ? factor : nullptr);
    if (e != cudaSuccess || !clip) return e;
  }
  bool first = !many;
  for (int at = 0; at < count;) {
    at = fill_table(grads, count, at, &t);
    if (t.chunks == 0) break;
    e = launch_dependent(scale_kernel<CAP>, dim3(static_cast<unsigned>(t.chunks)), dim3(kThreads), 0, stream, t,
                         static_cast<const double*>(partial), parts, max_norm, first ? norm : nullptr,
                         many ? static_cast<const Factor*>(factor) : nullptr);
    if (e != cudaSuccess) return e;
    first = false;
  }
  return cudaSuccess;
}

}  // namespace

int64_t grad_clip_workspace_bytes(int count, int sms) {
  const int64_t launches = std::max(1, (count + kTensors - 1) / kTensors);
  return 16 + launches * kNormBlocks * sms * static_cast<int64_t>(sizeof(double));
}

cudaError_t launch_grad_clip(const fp8bq_grad* grads, int count, double max_norm, bool clip, float* norm,
                             void* workspace, cudaStream_t stream) {
  return count <= kFewTensors ? run_grad_clip<kFewTensors>(grads, count, max_norm, clip, norm, workspace, stream)
                              : run_grad_clip<kTensors>(grads, count, max_norm, clip, norm, workspace, stream);
}

}  // namespace fp8bq
