// embedding.cu -- embedding lookup with scaling and its gradient.
//
//   forward   y[t, :] = scale * W[id[t], :]
//   backward  dW[v, :] (+)= scale * sum over t with id[t] = v of dY[t, :]
//
// Both are bound by HBM (16384 tokens, table [151936, 2048] BF16: the lookup
// takes 17.2 us, 86% of the copy rate; the FP32 gradient 205 us, 98%; rows of
// 2047 values, moved one at a time, 43 and 262).  The
// gradient is summed without floating-point atomics, so equal inputs give
// equal bits: the tokens are sorted by id (a stable radix sort by one
// thread-block cluster, while the other SMs write the dense gradient's zeros),
// equal chunks of the sorted tokens are summed run by run, and a run that
// spans chunks is joined from its chunks' partial sums in order.
//
// An id outside [0, V) is never used as an address: it is recorded in the index
// word, which fp8bq_check() reports, and gives zeros or adds nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8bq {
namespace {

__device__ __forceinline__ int64_t load_id(const void* ids, bool i64, int64_t t) {
  return i64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
}

// ---------------------------------------------------------------- forward --
struct LookupParams {
  const void* w;
  const void* ids;
  void* y;
  int* index;
  int64_t V, T, ldw, ldy;
  int D, pieces;  // a row is `pieces` pieces of 32 lanes x 4 packs
  float scale;
  bool i64;
};

// A warp copies a piece of a row: four packs a lane in flight.
template <class W, class Y, int VEC>
__global__ void __launch_bounds__(256) lookup_kernel(const LookupParams p) {
  constexpr int kPacks = 4;
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t t = warp / p.pieces;
  if (t >= p.T) return;
  const int c0 = static_cast<int>(warp - t * p.pieces) * (32 * kPacks * VEC) + lane * VEC;
  const int64_t id = load_id(p.ids, p.i64, t);
  const bool ok = id >= 0 && id < p.V;
  if (!ok && c0 == 0) atomicCAS(p.index, 0, kStatusIndex);
  const W* w = static_cast<const W*>(p.w) + (ok ? id : 0) * p.ldw;
  Y* y = static_cast<Y*>(p.y) + t * p.ldy;
  Pack<W, VEC> v[kPacks];
#pragma unroll
  for (int j = 0; j < kPacks; ++j) {
    const int c = c0 + j * 32 * VEC;
    if (c < p.D && ok) load_pack(v[j], w + c);
  }
#pragma unroll
  for (int j = 0; j < kPacks; ++j) {
    const int c = c0 + j * 32 * VEC;
    if (c < p.D) {
      Pack<Y, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o.v[i] = from_float<Y>(ok ? v[j].f(i) * p.scale : 0.0f);
      store_pack(y + c, o);
    }
  }
}

template <class W, class Y>
cudaError_t run_lookup(LookupParams p, cudaStream_t stream) {
  constexpr int kVec = 16 / static_cast<int>(std::min(sizeof(W), sizeof(Y)));
  const bool wide = p.D % kVec == 0 && rows_aligned(p.w, p.ldw, sizeof(W), 16) && rows_aligned(p.y, p.ldy, sizeof(Y), 16);
  const int piece = 128 * (wide ? kVec : 1);
  p.pieces = static_cast<int>((static_cast<int64_t>(p.D) + piece - 1) / piece);
  const int64_t blocks = (p.T * p.pieces + 7) / 8;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (wide)
    return launch_dependent(lookup_kernel<W, Y, kVec>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
  return launch_dependent(lookup_kernel<W, Y, 1>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
}

template <class W>
cudaError_t lookup_to(const LookupParams& p, int out_dtype, cudaStream_t stream) {
  switch (out_dtype) {
    case FP8BQ_BF16: return run_lookup<W, __nv_bfloat16>(p, stream);
    case FP8BQ_FP16: return run_lookup<W, __half>(p, stream);
    default: return run_lookup<W, float>(p, stream);
  }
}

// --------------------------------------------------------------- backward --
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
// One cluster sorts any number of tokens (4096 take it 18.6 us with what
// follows, a single block 24.4).
constexpr int kSortCluster = 8;
constexpr int kKept = 4;  // rounds of 32 tokens a warp keeps in registers: all, up to 32768 tokens

// A sorted token: its id (V: none of the table's rows) and its position.
struct alignas(8) Token {
  uint32_t id, pos;
};

struct SortParams {
  const void* ids;
  Token* buf[2];  // the passes alternate, the last one writes buf[0]
  int* index;
  int64_t T, V, padding;
  int64_t per_warp;  // tokens a warp of the cluster owns, a multiple of 32
  int passes, bits;  // digits of `bits` bits
  bool i64;
};

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Stable radix sort of the tokens by id, least significant digit first.
// Every warp owns a contiguous run of tokens and ranks its tokens in order
// (equal digits in a warp's 32 found by a match), so no digit's order depends
// on timing.  Counts and ranks live in shared memory; the blocks of the
// cluster read one another's digit counts there.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
  extern __shared__ uint32_t count[];  // [kSortWarps][kBins]
  __shared__ uint32_t total[kBins], base[kBins], scan[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cudaGridDependencySynchronize();
  // the zeros need no result of this kernel, only that what came before it is done
  cudaTriggerProgrammaticLaunchCompletion();
  const uint32_t rank = cluster_ctarank();
  uint32_t* mine = count + warp * kBins;
  const int64_t begin = (static_cast<int64_t>(rank) * kSortWarps + warp) * p.per_warp;
  const int64_t end = min(begin + p.per_warp, p.T);
  const int bins = 1 << p.bits;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const Token* from = p.buf[(p.passes - pass) & 1];
    Token* to = p.buf[(p.passes - 1 - pass) & 1];
    auto read = [&](int64_t i) {
      Token k;
      if (pass == 0) {
        const int64_t id = load_id(p.ids, p.i64, i);
        const bool ok = id >= 0 && id < p.V;
        if (!ok) atomicCAS(p.index, 0, kStatusIndex);
        k.id = static_cast<uint32_t>(ok && id != p.padding ? id : p.V);
        k.pos = static_cast<uint32_t>(i);
      } else {
        const uint2 w = __ldcg(reinterpret_cast<const uint2*>(from + i));
        k.id = w.x;
        k.pos = w.y;
      }
      return k;
    };
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    // the warp's first tokens stay in registers for the second walk
    Token kept[kKept];
#pragma unroll
    for (int j = 0; j < kKept; ++j)
      if (begin + j * 32 + lane < end) kept[j] = read(begin + j * 32 + lane);
    const auto count_one = [&](bool live, Token k) {
      const uint32_t d = live ? (k.id >> shift) & (bins - 1) : bins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (live && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
    };
#pragma unroll
    for (int j = 0; j < kKept; ++j)
      if (begin + j * 32 < end) count_one(begin + j * 32 + lane < end, kept[j]);
    for (int64_t i0 = begin + kKept * 32; i0 < end; i0 += 32) {
      const bool live = i0 + lane < end;
      count_one(live, live ? read(i0 + lane) : Token{});
    }
    __syncthreads();
    // per digit: where each warp's tokens start within the block's
    if (tid < bins) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = count[w * kBins + tid];
        count[w * kBins + tid] = run;
        run += c;
      }
      total[tid] = run;
    }
    // and where the block's start in the whole array
    uint32_t before = 0, all = 0;
    cluster_sync();
    if (tid < bins) {
#pragma unroll
      for (uint32_t r = 0; r < kSortCluster; ++r) {
        const uint32_t c = ld_shared_cluster_u32(mapa_shared(smem_u32(&total[tid]), r));
        if (r < rank) before += c;
        all += c;
      }
    }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (tid < bins) {
      uint32_t lower = 0;
      for (int w = 0; w < warp; ++w) lower += scan[w];
      base[tid] = lower + incl - all + before;
    }
    __syncthreads();
    const auto place_one = [&](bool live, Token k) {
      const uint32_t d = live ? (k.id >> shift) & (bins - 1) : bins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      uint32_t at = 0;
      if (live) at = base[d] + mine[d] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (live && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
      if (live) __stcg(reinterpret_cast<uint2*>(to + at), make_uint2(k.id, k.pos));
    };
#pragma unroll
    for (int j = 0; j < kKept; ++j)
      if (begin + j * 32 < end) place_one(begin + j * 32 + lane < end, kept[j]);
    for (int64_t i0 = begin + kKept * 32; i0 < end; i0 += 32) {
      const bool live = i0 + lane < end;
      place_one(live, live ? read(i0 + lane) : Token{});
    }
    cluster_sync();  // the next pass reads what the whole cluster wrote, and rewrites `total`
  }
}

// Zeros for the dense gradient, written while the tokens are sorted: a small
// tile a block, in the order the blocks start, and no loop over the grid (7.2
// TB/s where blocks that stay and stride reach 6.2).  The last block waits
// for the sort, so that what waits for this kernel finds both done.
constexpr int64_t kZeroBytes = 32 * 1024;

struct ZeroParams {
  uint8_t* dw;
  int64_t V, row_bytes, ld_bytes, rows;  // rows a block
};

// Zeros over [p, p + bytes), shared by `n` threads of which this is the t-th.
__device__ __forceinline__ void zero_span(uint8_t* p, int64_t bytes, int64_t t, int64_t n) {
  const int64_t head = min(static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), bytes);
  const int64_t wide = (bytes - head) / 16, tail0 = head + wide * 16;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = t; i < wide; i += n) q[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = t * 2; i < head; i += n * 2) *reinterpret_cast<uint16_t*>(p + i) = 0;
  for (int64_t i = tail0 + t * 2; i < bytes; i += n * 2) *reinterpret_cast<uint16_t*>(p + i) = 0;
}

__global__ void __launch_bounds__(256) zero_kernel(const ZeroParams p) {
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * p.rows, v1 = min(v0 + p.rows, p.V);
  if (p.row_bytes == p.ld_bytes) {
    zero_span(p.dw + v0 * p.row_bytes, (v1 - v0) * p.row_bytes, threadIdx.x, 256);
  } else {
    for (int64_t v = v0 + threadIdx.x / 32; v < v1; v += 8) zero_span(p.dw + v * p.ld_bytes, p.row_bytes, threadIdx.x % 32, 32);
  }
  if (blockIdx.x == gridDim.x - 1) cudaGridDependencySynchronize();
}

struct GradParams {
  const Token* tokens;
  const void* dy;
  void* dw;
  float* partial;  // [chunks][2][D]: a chunk's first run where it began before, its last where it goes on
  int64_t T, V, lddy, lddw, chunks;
  int D, chunk;   // tokens a chunk
  int cols;       // threads across the columns of a block, a power of two
  float scale;
  bool accumulate;
};

template <class G, int VEC>
__device__ __forceinline__ void write_row(const GradParams& p, int64_t row, int64_t c, const float (&acc)[VEC]) {
  G* dst = static_cast<G*>(p.dw) + row * p.lddw + c;
  Pack<G, VEC> o;
  if (p.accumulate) {
    load_pack(o, dst);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.v[i] = from_float<G>(fmaf(p.scale, acc[i], o.f(i)));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.v[i] = from_float<G>(p.scale * acc[i]);
  }
  store_pack(dst, o);
}

// One chunk of sorted tokens a thread group, VEC columns a thread: rows of dY
// are fetched eight at a time and summed in order.
template <class T, class G, int VEC>
__global__ void __launch_bounds__(256) grad_chunk_kernel(const GradParams p) {
  constexpr int kBatch = 8;
  cudaGridDependencySynchronize();
  const int tx = threadIdx.x & (p.cols - 1), ty = threadIdx.x / p.cols;
  const int64_t chunk = static_cast<int64_t>(blockIdx.y) * (blockDim.x / p.cols) + ty;
  const int c = (blockIdx.x * p.cols + tx) * VEC;
  if (chunk >= p.chunks || c >= p.D) return;
  const int64_t begin = chunk * p.chunk, end = min(begin + p.chunk, p.T);
  const uint32_t none = static_cast<uint32_t>(p.V);
  uint32_t cur = p.tokens[begin].id;
  bool head = begin > 0 && p.tokens[begin - 1].id == cur;
  const T* dy = static_cast<const T*>(p.dy) + c;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  auto flush = [&](bool tail) {
    if (cur == none) return;
    if (head || tail) {
      float* dst = p.partial + (chunk * 2 + (head ? 0 : 1)) * static_cast<int64_t>(p.D) + c;
      Pack<float, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o.v[i] = acc[i];
      store_pack(dst, o);
    } else {
      write_row<G, VEC>(p, cur, c, acc);
    }
  };
  for (int64_t i0 = begin; i0 < end; i0 += kBatch) {
    Token tok[kBatch];
    Pack<T, VEC> v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) tok[k] = i0 + k < end ? p.tokens[i0 + k] : Token{none, 0};
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (tok[k].id != none) load_pack<true>(v[k], dy + tok[k].pos * p.lddy);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k >= end) break;
      if (tok[k].id != cur) {
        flush(false);
        cur = tok[k].id;
        head = false;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
      }
      if (cur != none) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] += v[k].f(i);
      }
    }
  }
  flush(end < p.T && p.tokens[end].id == cur);
}

// The runs that span chunks: the chunk where one begins adds the later
// chunks' partial sums to its own, in order.
template <class G, int VEC>
__global__ void __launch_bounds__(256) grad_join_kernel(const GradParams p) {
  cudaGridDependencySynchronize();
  const int64_t chunk = blockIdx.x, begin = chunk * p.chunk, end = min(begin + p.chunk, p.T);
  if (end >= p.T) return;
  const uint32_t cur = p.tokens[end - 1].id;
  if (cur == static_cast<uint32_t>(p.V) || p.tokens[end].id != cur) return;
  if (begin > 0 && p.tokens[begin - 1].id == cur) return;  // began earlier
  // the last chunk that holds the run: chunk k does while its first token is in it
  int64_t last = chunk + 1;
  for (;;) {
    const int64_t first = (last + 1 + (threadIdx.x & 31)) * p.chunk;
    const unsigned in = __ballot_sync(0xffffffffu, first < p.T && p.tokens[min(first, p.T - 1)].id == cur);
    const int more = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
    last += more;
    if (more < 32) break;
  }
  const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x * VEC;
  for (int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * VEC; c < p.D; c += step) {
    const float* src = p.partial + c;
    float acc[VEC];
    Pack<float, VEC> v;
    load_pack(v, src + (chunk * 2 + 1) * static_cast<int64_t>(p.D));
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = v.v[i];
    constexpr int kBatch = VEC == 8 ? 8 : 16;
    for (int64_t k0 = chunk + 1; k0 <= last; k0 += kBatch) {
      Pack<float, VEC> u[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k <= last) load_pack(u[k], src + (k0 + k) * 2 * static_cast<int64_t>(p.D));
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k <= last) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[i] += u[k].v[i];
        }
    }
    write_row<G, VEC>(p, cur, c, acc);
  }
}

// ---------------------------------------------------------- few tokens --
// One launch (509 tokens of a [1031, 640] table, ids as texts have them: 4.6 us,
// the kernels above 13) and no workspace: a block for each token, which sums the
// rows of all tokens with its id unless an earlier token has it, and blocks that
// write zeros to the rows no token names.  Every block finds its tokens by
// reading all the ids, so this is for few of them; its time is that of the most
// frequent id, whose rows one block adds eight at a time (509 tokens of one id:
// 40 us; 1024: 78, where the kernels above take 23).
constexpr int kFewTokens = 1024;
// Of a dense gradient: beyond, every block's reading of the ids shows (1000
// tokens: 16.3 us against 18.0 at 61 MB, 27.1 and 27.4 at 133 MB, 196 against
// 176 at 1.2 GB).
constexpr int64_t kFewBytes = int64_t{128} << 20;
constexpr int kFewRows = 1024;                     // rows a block of zeros takes at most

struct FewParams {
  GradParams g;
  ZeroParams z;
  const void* ids;
  int64_t padding;
  int* index;
  bool i64;
};

template <class T, class G, int VEC>
__global__ void __launch_bounds__(256) grad_few_kernel(const FewParams p) {
  __shared__ int list[kFewTokens], counts[8];
  __shared__ uint8_t named[kFewRows];
  cudaGridDependencySynchronize();
  const GradParams& g = p.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T_ = static_cast<int>(g.T);
  if (blockIdx.x >= static_cast<unsigned>(T_)) {
    const int64_t v0 = static_cast<int64_t>(blockIdx.x - T_) * p.z.rows, v1 = min(v0 + p.z.rows, p.z.V);
    for (int i = tid; i < v1 - v0; i += 256) named[i] = 0;
    __syncthreads();
    bool any = false;
    for (int i = tid; i < T_; i += 256) {
      const int64_t id = load_id(p.ids, p.i64, i);
      if (id >= v0 && id < v1 && id != p.padding) {
        named[id - v0] = 1;
        any = true;
      }
    }
    if (!__syncthreads_or(any) && p.z.row_bytes == p.z.ld_bytes) {
      zero_span(p.z.dw + v0 * p.z.row_bytes, (v1 - v0) * p.z.row_bytes, tid, 256);
    } else {
      for (int64_t v = v0 + warp; v < v1; v += 8)
        if (!named[v - v0]) zero_span(p.z.dw + v * p.z.ld_bytes, p.z.row_bytes, lane, 32);
    }
    return;
  }
  const int t = static_cast<int>(blockIdx.x);
  const int64_t id = load_id(p.ids, p.i64, t);
  if (id < 0 || id >= g.V) {
    if (tid == 0) atomicCAS(p.index, 0, kStatusIndex);
    return;
  }
  if (id == p.padding) return;
  // the tokens with this id, in order: 256 at a time, counted by warp
  bool earlier = false;
  int found = 0;
  for (int i0 = 0; i0 < T_; i0 += 256) {
    const int i = i0 + tid;
    const bool same = i < T_ && load_id(p.ids, p.i64, i) == id;
    earlier |= same && i < t;
    const unsigned ballot = __ballot_sync(0xffffffffu, same);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = found;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += counts[w];
      found += counts[w];
    }
    if (same) list[before + __popc(ballot & ((1u << lane) - 1u))] = i;
    __syncthreads();
  }
  if (__syncthreads_or(earlier)) return;
  constexpr int kBatch = 8;
  for (int c = tid * VEC; c < g.D; c += 256 * VEC) {
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < found; k0 += kBatch) {
      Pack<T, VEC> v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < found) load_pack(v[k], static_cast<const T*>(g.dy) + list[k0 + k] * g.lddy + c);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < found) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[i] += v[k].f(i);
        }
    }
    write_row<G, VEC>(g, id, c, acc);
  }
}

bool few_tokens(int64_t T, int64_t V, int64_t D) { return T > 0 && T <= kFewTokens && V * D <= kFewBytes / 4; }

// Tokens a chunk: few enough that short batches fill the GPU, and at most
// about a thousand chunks, whose partial sums are the workspace.
int chunk_tokens(int64_t T) {
  if (T <= 4096) return 8;
  if (T <= 32768) return 32;
  return static_cast<int>((T + 1023) / 1024);
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

template <class T, class G, int VEC>
cudaError_t run_grad(GradParams p, cudaStream_t stream) {
  const int64_t slots = (static_cast<int64_t>(p.D) + VEC - 1) / VEC;
  p.cols = 1;
  while (p.cols < slots && p.cols < 256) p.cols *= 2;
  const int rows = 256 / p.cols;
  // the pieces of a row next to each other, so that they are read together
  const dim3 grid(static_cast<unsigned>((slots + p.cols - 1) / p.cols), static_cast<unsigned>((p.chunks + rows - 1) / rows));
  cudaError_t e = launch_dependent(grad_chunk_kernel<T, G, VEC>, grid, dim3(256), 0, stream, p);
  if (e != cudaSuccess || p.chunks < 2) return e;
  const int threads = static_cast<int>(std::min<int64_t>(256, (slots + 31) / 32 * 32));
  // a grid's second dimension ends at 65535: blocks of longer rows take several pieces
  const int64_t pieces = std::min<int64_t>(65535, (slots + threads - 1) / threads);
  const dim3 join(static_cast<unsigned>(p.chunks - 1), static_cast<unsigned>(pieces));
  return launch_dependent(grad_join_kernel<G, VEC>, join, dim3(threads), 0, stream, p);
}

template <class T, class G>
cudaError_t grad_of_type(const FewParams& f, bool few, cudaStream_t stream) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  const GradParams& p = f.g;
  const bool wide = p.D % kVec == 0 && rows_aligned(p.dy, p.lddy, sizeof(T), 16) && rows_aligned(p.dw, p.lddw, sizeof(G), 16);
  const bool pairs = sizeof(T) == 2 && p.D % 2 == 0 && rows_aligned(p.dy, p.lddy, sizeof(T), 4) &&
                     rows_aligned(p.dw, p.lddw, sizeof(G), 2 * sizeof(G));
  if (!few) {
    if (wide) return run_grad<T, G, kVec>(p, stream);
    if constexpr (sizeof(T) == 2)
      if (pairs) return run_grad<T, G, 2>(p, stream);
    return run_grad<T, G, 1>(p, stream);
  }
  const int64_t zeros = p.accumulate ? 0 : (f.z.V + f.z.rows - 1) / f.z.rows;
  const unsigned blocks = static_cast<unsigned>(p.T + zeros);
  if (wide)
    return launch_dependent(grad_few_kernel<T, G, kVec>, dim3(blocks), dim3(256), 0, stream, f);
  return launch_dependent(grad_few_kernel<T, G, 1>, dim3(blocks), dim3(256), 0, stream, f);
}

cudaError_t grad_of_types(const FewParams& f, int dtype, int dw_dtype, bool few, cudaStream_t stream) {
  switch (dtype) {
    case FP8BQ_BF16:
      return dw_dtype == FP8BQ_FP32 ? grad_of_type<__nv_bfloat16, float>(f, few, stream)
                                    : grad_of_type<__nv_bfloat16, __nv_bfloat16>(f, few, stream);
    case FP8BQ_FP16:
      return dw_dtype == FP8BQ_FP32 ? grad_of_type<__half, float>(f, few, stream)
                                    : grad_of_type<__half, __half>(f, few, stream);
    default: return grad_of_type<float, float>(f, few, stream);
  }
}

}  // namespace

cudaError_t launch_embedding_fwd(const EmbeddingFwd& a, cudaStream_t stream) {
  int* index = nullptr;
  const cudaError_t e = device_index_word(&index);
  if (e != cudaSuccess) return e;
  const LookupParams p{a.w, a.ids, a.y, index, a.V, a.T, a.ldw, a.ldy, static_cast<int>(a.D), 0, a.scale, a.ids_i64};
  switch (a.dtype) {
    case FP8BQ_BF16: return lookup_to<__nv_bfloat16>(p, a.out_dtype, stream);
    case FP8BQ_FP16: return lookup_to<__half>(p, a.out_dtype, stream);
    default: return lookup_to<float>(p, a.out_dtype, stream);
  }
}

int64_t embedding_bwd_workspace_bytes(int64_t T, int64_t D, int64_t V) {
  if (T == 0 || few_tokens(T, V, D)) return 0;
  const int64_t chunks = (T + chunk_tokens(T) - 1) / chunk_tokens(T);
  return 2 * round256(T * static_cast<int64_t>(sizeof(Token))) + chunks * 2 * D * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_embedding_bwd(const EmbeddingBwd& a, cudaStream_t stream) {
  int* index = nullptr;
  cudaError_t e = device_index_word(&index);
  if (e != cudaSuccess) return e;
  const int64_t size = a.dw_dtype == FP8BQ_FP32 ? 4 : 2;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int64_t tokens_bytes = round256(a.T * static_cast<int64_t>(sizeof(Token)));
  FewParams f{};
  GradParams& g = f.g;
  g.tokens = reinterpret_cast<Token*>(ws);
  g.dy = a.dy;
  g.dw = a.dw;
  g.T = a.T;
  g.V = a.V;
  g.lddy = a.lddy;
  g.lddw = a.lddw;
  g.D = static_cast<int>(a.D);
  g.scale = a.scale;
  g.accumulate = a.accumulate;
  f.z = ZeroParams{static_cast<uint8_t*>(a.dw), a.V, a.D * size, a.lddw * size, 0};
  f.z.rows = std::min<int64_t>(kFewRows, std::max<int64_t>(1, kZeroBytes / f.z.row_bytes));
  if (few_tokens(a.T, a.V, a.D)) {
    f.ids = a.ids;
    f.padding = a.padding;
    f.index = index;
    f.i64 = a.ids_i64;
    return grad_of_types(f, a.dtype, a.dw_dtype, true, stream);
  }
  SortParams s{};
  s.ids = a.ids;
  s.buf[0] = reinterpret_cast<Token*>(ws);
  s.buf[1] = reinterpret_cast<Token*>(ws + tokens_bytes);
  s.index = index;
  s.T = a.T;
  s.V = a.V;
  s.padding = a.padding;
  s.i64 = a.ids_i64;
  int bits = 1;
  while ((a.V >> bits) != 0) ++bits;  // ids 0 .. V, V standing for none
  s.passes = (bits + kDigitBits - 1) / kDigitBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  const int64_t warps = int64_t{kSortCluster} * kSortWarps;
  s.per_warp = ((a.T + warps - 1) / warps + 31) / 32 * 32;
  constexpr size_t kSmem = sizeof(uint32_t) * kSortWarps * kBins;
  static_assert(kSmem + sizeof(uint32_t) * (2 * kBins + kSortWarps) <= 227 * 1024, "shared memory of one block");
  e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCluster, 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sort_kernel, s);
  if (e != cudaSuccess) return e;
  if (!a.accumulate) {
    const int64_t blocks = std::max<int64_t>(1, (a.V + f.z.rows - 1) / f.z.rows);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    e = launch_dependent(zero_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, f.z);
    if (e != cudaSuccess) return e;
  }
  if (a.T == 0) return cudaSuccess;
  g.partial = reinterpret_cast<float*>(ws + 2 * tokens_bytes);
  g.chunk = chunk_tokens(a.T);
  g.chunks = (a.T + g.chunk - 1) / g.chunk;
  return grad_of_types(f, a.dtype, a.dw_dtype, false, stream);
}

}  // namespace fp8bq
