// norm_bwd.cu -- the backward passes of LayerNorm and RMSNorm: how a launch is
// laid out, and the join of the blocks' dgamma and dbeta.  The kernels are in
// norm_bwd.cuh.
#include "norm_bwd.cuh"

namespace fp8bq {

extern template cudaError_t run_norm_bwd<__nv_bfloat16>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);
extern template cudaError_t run_norm_bwd<__half>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);
extern template cudaError_t run_norm_bwd<float>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);

namespace {

// dgamma and dbeta from the blocks' partial sums, in a fixed order: a block
// takes 32 columns, its 32 warps every 32nd partial each, eight of them in
// flight (latency is all there is: a few MB from L2).
__global__ void __launch_bounds__(1024) norm_param_grad_kernel(const float* partial, int64_t parts, int64_t width,
                                                               int64_t N, float* dgamma, float* dbeta, bool accumulate) {
  __shared__ float red[32][33];
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < width) {
    const float* p = partial + c;
    for (int64_t k0 = warp; k0 < parts; k0 += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k0 + 32 * i < parts ? p[(k0 + 32 * i) * width] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  // warp w adds column w's 32 sums
  s = warp_sum(red[lane][warp]);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane != 0 || col >= width) return;
  if (col < N)
    write_sum(dgamma, col, s, accumulate);
  else
    write_sum(dbeta, col - N, s, accumulate);
}

// Rows of up to 128 columns: 8 lanes each.  Else the fewest threads and
// columns a thread that hold the row, 512 threads an SM, and as many rows
// between two barriers as leave the ring two stages (measured at [16384, 2048]
// BF16 with a residual, LayerNorm, 8 columns a thread: 75 us with one row, 57
// with two, 51 with four).
RowPlan plan_bwd(int64_t M, int64_t N, int64_t size, int tensors, bool aligned, bool packed, bool wide_gamma, int sms) {
  if (aligned && (N * size) % 16 != 0) return RowPlan{};
  struct Choice {
    int threads, cols, rows;
  };
  const int least = aligned ? static_cast<int>(16 / size) : 8;
  const Choice choices[] = {{256, least, 4}, {256, 8, 4}, {256, 16, 2}, {512, 16, 2}, {512, 32, 1}};
  RowPlan b{};
  if (N <= 128) {
    b.tpr = 8;
    b.cols = N <= 64 ? 8 : 16;
    b.rows = 2;
    b.groups = 256 / b.tpr;
  }
  for (const Choice& c : choices) {
    if (b.cols != 0) break;
    const int64_t tpr = ((N + c.cols - 1) / c.cols + 31) / 32 * 32;
    if (tpr > c.threads) continue;
    b.cols = c.cols;
    b.tpr = static_cast<int>(tpr);
    b.rows = c.rows;
    b.groups = 1;
    for (int g = 2; g * b.tpr <= 256; ++g)  // the groups that leave the fewest of 512 threads out
      if (512 / (g * b.tpr) * g >= 512 / (b.groups * b.tpr) * b.groups) b.groups = g;
  }
  if (b.cols == 0) return b;
  const int per_sm = 512 / (b.tpr * b.groups);
  const int64_t row = N * size;
  const int64_t pitch = aligned ? static_cast<int64_t>(b.tpr) * b.cols * size : packed ? row : (row + 30) / 16 * 16;
  const int64_t room = kRingBytes / per_sm - kRingExtra - gamma_bytes(b, wide_gamma ? 4 : size);
  const auto stage = [&](int rows) {
    const int64_t bytes = pitch * b.groups * rows;
    return (aligned ? bytes : (bytes + 30) / 16 * 16) * tensors;
  };
  while (b.rows > 1 && room / stage(b.rows) < 2) b.rows /= 2;
  const int64_t stages = std::min<int64_t>(kMostStages, room / stage(b.rows));
  if (stages < 2) return RowPlan{};
  const int64_t rows = static_cast<int64_t>(b.groups) * b.rows;
  b.blocks = std::min<int64_t>((M + rows - 1) / rows, static_cast<int64_t>(per_sm) * sms);
  b.ring.M = M;
  b.ring.n = static_cast<int>(N);
  b.ring.rows = static_cast<int>(rows);
  b.ring.stages = static_cast<int>(stages);
  b.ring.row_bytes = static_cast<uint32_t>(row);
  b.ring.pitch = static_cast<uint32_t>(pitch);
  b.ring.stage_bytes = static_cast<uint32_t>(stage(b.rows));
  b.ring.tensor_bytes = b.ring.stage_bytes / static_cast<uint32_t>(tensors);
  b.ring.packed = packed && pitch == row;
  return b;
}

// Rows too long for a block: the blocks that share each column's sum.
int64_t long_blocks(int64_t M, int64_t N, int sms) {
  return std::min<int64_t>(M, std::max<int64_t>(1, 4 * sms / ((N + 255) / 256)));
}

// Few rows: their sums are taken from L2 in the same launch, beside the rows.
// At [509, 2048] BF16 5.6 us against 6.3 with the second kernel, whose launch
// also costs the host 3.5 us; at [777, 6144] FP32, 17.5 against 16.6.
bool small_batch(int64_t M, int64_t N) { return M <= 1024 && M * N <= int64_t{1} << 22; }

}  // namespace

int64_t norm_bwd_workspace_bytes(int64_t M, int64_t N, int sms) {
  if (M == 0 || N == 0 || small_batch(M, N)) return 0;
  int64_t most = long_blocks(M, N, sms);
  for (int64_t size : {2, 4})
    for (int tensors : {2, 3})
      for (int how = 0; how < 8; ++how)
        most = std::max(most, plan_bwd(M, N, size, tensors, (how & 1) != 0, (how & 2) != 0, (how & 4) != 0, sms).blocks);
  return most * 2 * N * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_norm_bwd(const fp8bq_norm_grad& a, bool layernorm, cudaStream_t stream) {
  int sms = 0;
  int* status = nullptr;
  cudaError_t e = device_sm_count(&sms);
  if (e == cudaSuccess) e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  const bool few = a.M > 0 && small_batch(a.M, a.N);
  const bool accumulate = (a.flags & FP8BQ_NORM_ACCUMULATE) != 0;
  int64_t blocks = 0;
  if (a.M > 0) {
    const int64_t size = a.dtype == FP8BQ_FP32 ? 4 : 2;
    const bool res = a.dres != nullptr;
    const auto overlap = [&](const void* p, int64_t ldp, const void* q, int64_t ldq) {
      const uintptr_t pa = reinterpret_cast<uintptr_t>(p), qa = reinterpret_cast<uintptr_t>(q);
      const auto span = [&](int64_t ld) { return static_cast<uintptr_t>(((a.M - 1) * ld + a.N) * size); };
      return pa < qa + span(ldq) && qa < pa + span(ldp);
    };
    const bool aligned = (a.N * size) % 16 == 0 && rows_aligned(a.x, a.ldx, size, 16) &&
                         rows_aligned(a.dy, a.lddy, size, 16) && rows_aligned(a.dx, a.lddx, size, 16) &&
                         (!res || rows_aligned(a.dres, a.lddres, size, 16)) && rows_aligned(a.gamma, 0, 1, 16);
    const bool packed = a.ldx == a.N && a.lddy == a.N && (!res || a.lddres == a.N);
    RowPlan b = plan_bwd(a.M, a.N, size, res ? 3 : 2, aligned, packed,
                         a.param_dtype == FP8BQ_FP32 || a.gamma == nullptr, sms);
    blocks = b.cols != 0 ? b.blocks : few ? 1 : long_blocks(a.M, a.N, sms);
    b.ring.src[0] = a.x;
    b.ring.src[1] = a.dy;
    b.ring.src[2] = a.dres;
    b.ring.ld[0] = a.ldx;
    b.ring.ld[1] = a.lddy;
    b.ring.ld[2] = a.lddres;
    b.ring.status = status;
    const BwdParams p{a.dy, a.x, a.dres, a.dx, a.gamma, a.mean, a.rstd,
                      sums && !few ? static_cast<float*>(a.workspace) : nullptr, few ? a.dgamma : nullptr,
                      few && layernorm ? a.dbeta : nullptr, 0, accumulate,
                      overlap(a.dx, a.lddx, a.x, a.ldx) || overlap(a.dx, a.lddx, a.dy, a.lddy), a.M, a.N, a.lddy, a.ldx, a.lddres, a.lddx, 1.0f / static_cast<float>(a.N),
                      a.param_dtype == FP8BQ_FP32, (a.flags & FP8BQ_NORM_RSTD_F64) != 0, 0};
    switch (a.dtype) {
      case FP8BQ_BF16: e = run_norm_bwd<__nv_bfloat16>(p, b, layernorm, aligned, blocks, stream); break;
      case FP8BQ_FP16: e = run_norm_bwd<__half>(p, b, layernorm, aligned, blocks, stream); break;
      default: e = run_norm_bwd<float>(p, b, layernorm, aligned, blocks, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums || few) return cudaSuccess;
  const int64_t width = a.N * (layernorm ? 2 : 1);
  return launch_dependent(norm_param_grad_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(1024), 0, stream,
                          static_cast<const float*>(a.workspace), blocks, width, a.N, a.dgamma,
                          layernorm ? a.dbeta : nullptr, accumulate);
}

}  // namespace fp8bq
