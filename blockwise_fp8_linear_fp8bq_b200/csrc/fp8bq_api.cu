// fp8bq_api.cu -- the C ABI declared in include/fp8bq.h: argument checks,
// status codes and dispatch to the kernels.  Nothing here allocates device
// memory or synchronizes, except fp8bq_check().
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <mutex>
#include <new>

#include "fp8bq.h"
#include "fp8bq_testing.h"
#include "internal.h"
#include "quant_math.cuh"

namespace {
thread_local int t_last_cuda_error = 0;
}  // namespace

namespace fp8bq {

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FP8BQ_OK;
  t_last_cuda_error = static_cast<int>(e);
  return FP8BQ_ERR_CUDA;
}

unsigned long long current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(f);
    f = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(f);
  });
  if (get_current == nullptr || get_id == nullptr) return 0;
  CUcontext ctx = nullptr;
  if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
  unsigned long long id = 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

}  // namespace fp8bq

namespace {

using fp8bq::cuda_status;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_fmt(int fmt) { return fmt == FP8BQ_SCALE_FP32 || fmt == FP8BQ_SCALE_UE8M0; }

// Kernels need an sm_100 device; checked once per device.
int device_ok() {
  static int cached[64] = {};  // 0 unknown, 1 ok, 2 unsupported
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= 64) return FP8BQ_ERR_UNSUPPORTED;
  if (cached[dev] == 0) {
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_status(e);
    e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e != cudaSuccess) return cuda_status(e);
    cached[dev] = (major == 10 && minor == 0) ? 1 : 2;
  }
  return cached[dev] == 1 ? FP8BQ_OK : FP8BQ_ERR_UNSUPPORTED;
}

int check_quant_args(const void* x, int64_t rows, int64_t cols, int64_t ld, const void* q,
                     const void* scales, int fmt) {
  if (!x || !q || !scales) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_fmt(fmt)) return FP8BQ_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || ld < cols) return FP8BQ_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || (ld % 8) != 0) return FP8BQ_ERR_ALIGN;
  return FP8BQ_OK;
}

// Bytes of a row operator's element type, 0 for another dtype.
int64_t elem_bytes(int dtype) {
  switch (dtype) {
    case FP8BQ_BF16:
    case FP8BQ_FP16: return 2;
    case FP8BQ_FP32: return 4;
    default: return 0;
  }
}

bool aligned_to(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

constexpr int64_t kMostRows = INT32_MAX - 1;

// Rows and columns of a row operator.
bool valid_rows(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMostRows && cols <= kMostRows;
}

// Token ids and the scale of an embedding call.
int check_ids(const void* ids, int ids_i64, float scale) {
  if ((ids_i64 != 0 && ids_i64 != 1) || !std::isfinite(scale)) return FP8BQ_ERR_INVALID_ARG;
  return aligned_to(ids, ids_i64 ? 8 : 4) ? FP8BQ_OK : FP8BQ_ERR_ALIGN;
}

int norm_backward(const fp8bq_norm_grad* a, bool layernorm, cudaStream_t stream) {
  if (a == nullptr) return FP8BQ_ERR_INVALID_ARG;
  const int64_t e = elem_bytes(a->dtype);
  if (e == 0 || (a->param_dtype != a->dtype && a->param_dtype != FP8BQ_FP32)) return FP8BQ_ERR_INVALID_ARG;
  if ((a->flags & ~(FP8BQ_NORM_ACCUMULATE | FP8BQ_NORM_RSTD_F64)) != 0) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_rows(a->M, a->N)) return FP8BQ_ERR_SHAPE;
  if (a->lddy < a->N || a->ldx < a->N || a->lddx < a->N || (a->dres != nullptr && a->lddres < a->N))
    return FP8BQ_ERR_SHAPE;
  if (a->M > 0 && a->N > 0 &&
      (!a->dy || !a->x || !a->dx || !a->rstd || (layernorm && !a->mean)))
    return FP8BQ_ERR_INVALID_ARG;
  if (!aligned_to(a->dy, e) || !aligned_to(a->x, e) || !aligned_to(a->dx, e) || !aligned_to(a->dres, e) ||
      !aligned_to(a->gamma, elem_bytes(a->param_dtype)) || !aligned_to(a->mean, 4) ||
      !aligned_to(a->rstd, (a->flags & FP8BQ_NORM_RSTD_F64) != 0 ? 8 : 4) || !aligned_to(a->dgamma, 4) ||
      !aligned_to(a->dbeta, 4) || !aligned16(a->workspace))
    return FP8BQ_ERR_ALIGN;
  fp8bq_norm_grad b = *a;
  if (!layernorm) {
    b.mean = nullptr;
    b.dbeta = nullptr;
  }
  const bool sums = b.dgamma != nullptr || b.dbeta != nullptr;
  if (b.N == 0 || (b.M == 0 && !sums)) return FP8BQ_OK;
  int st = device_ok();
  if (st != FP8BQ_OK) return st;
  if (sums && b.M > 0) {
    int sms = 0;
    const cudaError_t err = fp8bq::device_sm_count(&sms);
    if (err != cudaSuccess) return cuda_status(err);
    const int64_t need = fp8bq::norm_bwd_workspace_bytes(b.M, b.N, sms);
    if (need > 0 && (!b.workspace || b.workspace_bytes < need)) return FP8BQ_ERR_INVALID_ARG;
  }
  return cuda_status(fp8bq::launch_norm_bwd(b, layernorm, stream));
}

// Whether a tensor that clipping writes overlaps another listed one (its own
// input, at the same address, apart).
int check_overlaps(const fp8bq_grad* grads, int count) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[2 * static_cast<size_t>(count) + 1]);
  if (!spans) return FP8BQ_ERR_UNSUPPORTED;
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const fp8bq_grad& g = grads[i];
    if (g.n == 0) continue;
    const auto add = [&](const void* p, int dtype, bool written) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(p);
      spans[n++] = Span{b, b + static_cast<uintptr_t>(g.n * elem_bytes(dtype)), written};
    };
    add(g.out, g.out_dtype, true);
    if (g.g != g.out) add(g.g, g.dtype, false);
  }
  std::sort(spans.get(), spans.get() + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;  // where the spans so far end
  for (size_t i = 0; i < n; ++i) {
    if (spans[i].begin < (spans[i].written ? any : written)) return FP8BQ_ERR_INVALID_ARG;
    any = std::max(any, spans[i].end);
    if (spans[i].written) written = std::max(written, spans[i].end);
  }
  return FP8BQ_OK;
}

int grad_list(const fp8bq_grad* grads, int count, double max_norm, bool clip, float* norm, void* workspace,
              int64_t workspace_bytes, cudaStream_t stream) {
  if (count < 0) return FP8BQ_ERR_SHAPE;
  if ((grads == nullptr && count > 0) || norm == nullptr || !(max_norm >= 0.0)) return FP8BQ_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const fp8bq_grad& g = grads[i];
    const int64_t e = elem_bytes(g.dtype), o = clip ? elem_bytes(g.out_dtype) : 1;
    if (e == 0 || o == 0) return FP8BQ_ERR_INVALID_ARG;
    if (g.n < 0 || g.n > (int64_t{1} << 35)) return FP8BQ_ERR_SHAPE;
    if (g.n > 0 && (!g.g || (clip && !g.out))) return FP8BQ_ERR_INVALID_ARG;
    if (clip && g.n > 0 && g.g == g.out && g.dtype != g.out_dtype) return FP8BQ_ERR_INVALID_ARG;
    if (!aligned_to(g.g, e) || (clip && !aligned_to(g.out, o))) return FP8BQ_ERR_ALIGN;
  }
  if (!aligned_to(norm, 4) || !aligned16(workspace)) return FP8BQ_ERR_ALIGN;
  int st = clip ? check_overlaps(grads, count) : FP8BQ_OK;
  if (st != FP8BQ_OK) return st;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  int sms = 0;
  const cudaError_t err = fp8bq::device_sm_count(&sms);
  if (err != cudaSuccess) return cuda_status(err);
  if (!workspace || workspace_bytes < fp8bq::grad_clip_workspace_bytes(count, sms)) return FP8BQ_ERR_INVALID_ARG;
  return cuda_status(fp8bq::launch_grad_clip(grads, count, max_norm, clip, norm, workspace, stream));
}

// Operand checks shared by A and B; fills the internal form.
int convert_operand(const fp8bq_operand* op, int64_t rows, int64_t K, bool is_a, fp8bq::GemmOperand* out) {
  if (!op || !op->data) return FP8BQ_ERR_INVALID_ARG;
  if (op->dtype != FP8BQ_E4M3 && op->dtype != FP8BQ_BF16) return FP8BQ_ERR_INVALID_ARG;
  if (op->gran != FP8BQ_GRAN_ROW_1x128 && op->gran != FP8BQ_GRAN_BLOCK_128x128 &&
      op->gran != FP8BQ_GRAN_ROW_1x32)
    return FP8BQ_ERR_INVALID_ARG;
  if (!valid_fmt(op->fmt)) return FP8BQ_ERR_INVALID_ARG;
  const int fmt = op->fmt;
  if (op->k_major != 0 && op->k_major != 1) return FP8BQ_ERR_INVALID_ARG;
  const bool bf16 = op->dtype == FP8BQ_BF16;
  if (bf16 && (!is_a || !op->k_major)) return FP8BQ_ERR_UNSUPPORTED;
  const int64_t esz = bf16 ? 2 : 1;
  if (!aligned16(op->data) || (op->ld * esz) % 16 != 0) return FP8BQ_ERR_ALIGN;
  const int64_t inner = op->k_major ? K : rows;
  if (op->ld < inner) return FP8BQ_ERR_SHAPE;
  if (!bf16) {
    if (!op->scales) return FP8BQ_ERR_INVALID_ARG;
    if (!aligned16(op->scales)) return FP8BQ_ERR_ALIGN;
    if (op->gran == FP8BQ_GRAN_ROW_1x32 && fmt != FP8BQ_SCALE_UE8M0) return FP8BQ_ERR_UNSUPPORTED;
    if (op->gran == FP8BQ_GRAN_ROW_1x128 || op->gran == FP8BQ_GRAN_ROW_1x32) {
      if (!op->k_major) return FP8BQ_ERR_UNSUPPORTED;
      if (op->s_stride_r != 1 || op->s_stride_k % 128 != 0 || op->s_stride_k < rows)
        return FP8BQ_ERR_SHAPE;
    } else {
      if (is_a) return FP8BQ_ERR_UNSUPPORTED;
      const int64_t nrb = (rows + 127) / 128;
      const int64_t nkb = K / 128;
      const bool plain = op->s_stride_r == 1 && op->s_stride_k >= nrb;
      const bool transposed = op->s_stride_k == 1 && op->s_stride_r >= nkb;
      if (!plain && !transposed) return FP8BQ_ERR_SHAPE;
    }
  } else if (op->gran != FP8BQ_GRAN_ROW_1x128) {
    return FP8BQ_ERR_UNSUPPORTED;  // BF16 A is quantized in 1x128 row groups
  }
  out->data = op->data;
  out->ld = op->ld;
  out->bf16 = bf16;
  out->k_major = op->k_major != 0;
  out->scales = op->scales;
  out->row_groups = op->gran == FP8BQ_GRAN_ROW_1x128 || op->gran == FP8BQ_GRAN_ROW_1x32;
  out->mx = op->gran == FP8BQ_GRAN_ROW_1x32;
  out->s_stride_k = op->s_stride_k;
  out->s_stride_r = op->s_stride_r;
  return FP8BQ_OK;
}

}  // namespace

namespace fp8bq {

int validate_gemm(const fp8bq_operand* A, const fp8bq_operand* B, void* D, int64_t M, int64_t N, int64_t K,
                  int64_t ldd, uint32_t flags, GemmProblem* p) {
  if (!A || !B || !D || !p) return FP8BQ_ERR_INVALID_ARG;
  if ((flags & ~static_cast<uint32_t>(FP8BQ_GEMM_ACCUMULATE_F32)) != 0) return FP8BQ_ERR_INVALID_ARG;
  const bool acc = (flags & FP8BQ_GEMM_ACCUMULATE_F32) != 0;
  if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0 || N % 8 != 0 || ldd < N) return FP8BQ_ERR_SHAPE;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return FP8BQ_ERR_SHAPE;
  if (!aligned16(D) || ldd % 8 != 0) return FP8BQ_ERR_ALIGN;
  int st = convert_operand(A, M, K, true, &p->a);
  if (st != FP8BQ_OK) return st;
  st = convert_operand(B, N, K, false, &p->b);
  if (st != FP8BQ_OK) return st;
  if (p->a.mx != p->b.mx) return FP8BQ_ERR_UNSUPPORTED;  // MX blocks on both operands or neither
  // A BF16 A is quantized inside the GEMM in its own format; B must share it
  if (p->a.bf16 && A->fmt != B->fmt) return FP8BQ_ERR_UNSUPPORTED;
  // FP32 accumulation is built for the weight-gradient layout only
  if (acc && (p->a.bf16 || !p->a.row_groups || !p->b.row_groups || !p->b.k_major)) return FP8BQ_ERR_UNSUPPORTED;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  p->d = D;
  p->M = M;
  p->N = N;
  p->K = K;
  p->ldd = ldd;
  // both UE8M0: the block-scaled MMA; otherwise the FP32 promotion path, with
  // an operand's UE8M0 scales decoded to 2^e where they are staged
  const bool both_u8 = A->fmt == FP8BQ_SCALE_UE8M0 && B->fmt == FP8BQ_SCALE_UE8M0;
  p->fmt = both_u8 ? kFmtUe8m0 : kFmtFp32;
  p->a_u8 = !both_u8 && A->fmt == FP8BQ_SCALE_UE8M0;
  p->b_u8 = !both_u8 && B->fmt == FP8BQ_SCALE_UE8M0;
  p->acc_f32 = acc;
  p->ws = nullptr;
  p->ws_bytes = 0;
  return FP8BQ_OK;
}

int run_gemm(const GemmProblem& p, cudaStream_t stream) {
  bool unsupported = false;
  cudaError_t e = launch_gemm(p, stream, &unsupported);
  if (unsupported) return FP8BQ_ERR_UNSUPPORTED;
  return cuda_status(e);
}

}  // namespace fp8bq

extern "C" {

int fp8bq_quantize_act(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* scales,
                       int fmt, fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if (K % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, q, scales, nullptr, nullptr, fmt, 128,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_act_t(const void* x, int64_t M, int64_t K, int64_t ldx, void* qt, void* scales,
                         int fmt, fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, qt, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if (M % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (K % 8 != 0) return FP8BQ_ERR_ALIGN;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, nullptr, nullptr, qt, scales, fmt, 128,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_act_dual(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* scales,
                            void* qt, void* scales_t, int fmt, fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  st = check_quant_args(x, M, K, ldx, qt, scales_t, fmt);
  if (st != FP8BQ_OK) return st;
  if (K % 128 != 0 || M % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, q, scales, qt, scales_t, fmt, 128,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_act_mx(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* scales,
                          fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, FP8BQ_SCALE_UE8M0);
  if (st != FP8BQ_OK) return st;
  if (K % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, q, scales, nullptr, nullptr, FP8BQ_SCALE_UE8M0, 32,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_act_t_mx(const void* x, int64_t M, int64_t K, int64_t ldx, void* qt, void* scales,
                            fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, qt, scales, FP8BQ_SCALE_UE8M0);
  if (st != FP8BQ_OK) return st;
  if (M % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (K % 8 != 0) return FP8BQ_ERR_ALIGN;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, nullptr, nullptr, qt, scales, FP8BQ_SCALE_UE8M0, 32,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_act_dual_mx(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* scales,
                               void* qt, void* scales_t, fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, FP8BQ_SCALE_UE8M0);
  if (st != FP8BQ_OK) return st;
  st = check_quant_args(x, M, K, ldx, qt, scales_t, FP8BQ_SCALE_UE8M0);
  if (st != FP8BQ_OK) return st;
  if (K % 128 != 0 || M % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_tiles(x, M, K, ldx, q, scales, qt, scales_t, FP8BQ_SCALE_UE8M0, 32,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_swiglu_quantize(const void* gu, int64_t M, int64_t F, int64_t ldgu, void* h, void* q, void* scales,
                          void* qt, void* scales_t, int fmt, fp8bq_stream_t stream) {
  const bool exact = (fmt & FP8BQ_SWIGLU_EXACT) != 0;
  fmt &= ~FP8BQ_SWIGLU_EXACT;
  int st = check_quant_args(gu, M, 2 * F, ldgu, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if ((qt == nullptr) != (scales_t == nullptr)) return FP8BQ_ERR_INVALID_ARG;
  if (qt != nullptr && (!aligned16(qt) || !aligned16(scales_t))) return FP8BQ_ERR_ALIGN;
  if (h != nullptr && !aligned16(h)) return FP8BQ_ERR_ALIGN;
  if (F % 128 != 0 || (qt != nullptr && M % 128 != 0)) return FP8BQ_ERR_SHAPE;
  if (M == 0 || F == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_swiglu_quant(gu, M, F, ldgu, h, q, scales, qt, scales_t, fmt, exact,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_rmsnorm_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, const void* gamma, float eps,
                           float* rstd, void* h, void* q, void* scales, void* qt, void* scales_t, int fmt,
                           fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if (gamma == nullptr || rstd == nullptr) return FP8BQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8BQ_ERR_INVALID_ARG;  // finite, not negative
  if ((qt == nullptr) != (scales_t == nullptr)) return FP8BQ_ERR_INVALID_ARG;
  if (!aligned16(gamma) || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0) return FP8BQ_ERR_ALIGN;
  if (qt != nullptr && (!aligned16(qt) || !aligned16(scales_t))) return FP8BQ_ERR_ALIGN;
  if (h != nullptr && !aligned16(h)) return FP8BQ_ERR_ALIGN;
  if (K % 128 != 0 || (qt != nullptr && M % 128 != 0)) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_rmsnorm_quant(x, M, K, ldx, gamma, eps, rstd, h, q, scales, qt, scales_t, fmt,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_rmsnorm_quantize_exact(const void* x, int64_t M, int64_t K, int64_t ldx, const void* gamma, double eps,
                                 double* rstd, void* h, void* q, void* scales, void* qt, void* scales_t, int fmt,
                                 fp8bq_stream_t stream) {
  int st = check_quant_args(x, M, K, ldx, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if (gamma == nullptr || rstd == nullptr) return FP8BQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return FP8BQ_ERR_INVALID_ARG;  // finite, not negative
  if ((qt == nullptr) != (scales_t == nullptr)) return FP8BQ_ERR_INVALID_ARG;
  if (!aligned16(gamma) || (reinterpret_cast<uintptr_t>(rstd) & 7u) != 0) return FP8BQ_ERR_ALIGN;
  if (qt != nullptr && (!aligned16(qt) || !aligned16(scales_t))) return FP8BQ_ERR_ALIGN;
  if (h != nullptr && !aligned16(h)) return FP8BQ_ERR_ALIGN;
  if (K % 128 != 0 || (qt != nullptr && M % 128 != 0)) return FP8BQ_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_rmsnorm_quant_exact(x, M, K, ldx, gamma, eps, rstd, h, q, scales, qt, scales_t,
                                                       fmt, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_embedding_forward(const void* w, int64_t V, int64_t D, int64_t ldw, const void* ids, int ids_i64, int64_t T,
                            float scale, void* y, int64_t ldy, int dtype, int out_dtype, fp8bq_stream_t stream) {
  const int64_t e = elem_bytes(dtype), o = elem_bytes(out_dtype);
  if (e == 0 || o == 0) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_rows(V, D) || T < 0 || T > kMostRows || ldw < D || ldy < D) return FP8BQ_ERR_SHAPE;
  int st = check_ids(ids, ids_i64, scale);
  if (st != FP8BQ_OK) return st;
  if (!aligned_to(w, e) || !aligned_to(y, o)) return FP8BQ_ERR_ALIGN;
  if (T == 0 || D == 0) return FP8BQ_OK;
  if (!ids || !y || (!w && V > 0)) return FP8BQ_ERR_INVALID_ARG;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  const fp8bq::EmbeddingFwd a{w, ids, y, V, D, ldw, T, ldy, scale, dtype, out_dtype, ids_i64 != 0};
  return cuda_status(fp8bq::launch_embedding_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_embedding_backward(const void* dy, int64_t T, int64_t D, int64_t lddy, const void* ids, int ids_i64, int64_t V,
                             float scale, int64_t padding_id, void* dw, int64_t lddw, int dtype, int dw_dtype,
                             uint32_t flags, void* workspace, int64_t workspace_bytes, fp8bq_stream_t stream) {
  const int64_t e = elem_bytes(dtype);
  if (e == 0 || (dw_dtype != dtype && dw_dtype != FP8BQ_FP32)) return FP8BQ_ERR_INVALID_ARG;
  if ((flags & ~static_cast<uint32_t>(FP8BQ_EMBEDDING_ACCUMULATE)) != 0) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_rows(V, D) || T < 0 || T > kMostRows || lddy < D || lddw < D) return FP8BQ_ERR_SHAPE;
  int st = check_ids(ids, ids_i64, scale);
  if (st != FP8BQ_OK) return st;
  if (!aligned_to(dy, e) || !aligned_to(dw, elem_bytes(dw_dtype)) || !aligned16(workspace)) return FP8BQ_ERR_ALIGN;
  const bool accumulate = (flags & FP8BQ_EMBEDDING_ACCUMULATE) != 0;
  if (D == 0 || (T == 0 && (accumulate || V == 0))) return FP8BQ_OK;
  if ((!dw && V > 0) || (T > 0 && (!dy || !ids))) return FP8BQ_ERR_INVALID_ARG;
  const int64_t need = fp8bq::embedding_bwd_workspace_bytes(T, D, V);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FP8BQ_ERR_INVALID_ARG;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  const fp8bq::EmbeddingBwd a{dy,   ids,  dw,         workspace, T, D, lddy, V, lddw, padding_id, scale,
                              dtype, dw_dtype, ids_i64 != 0, accumulate};
  return cuda_status(fp8bq::launch_embedding_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t fp8bq_embedding_workspace_bytes(int64_t T, int64_t D, int64_t V) {
  return valid_rows(T, D) && valid_rows(V, D) ? fp8bq::embedding_bwd_workspace_bytes(T, D, V) : -1;
}

int fp8bq_layernorm_forward(const void* x, int64_t M, int64_t N, int64_t ldx, const void* gamma, const void* beta,
                            float eps, void* y, int64_t ldy, float* mean, float* rstd, int dtype, int param_dtype,
                            fp8bq_stream_t stream) {
  const int64_t e = elem_bytes(dtype);
  if (e == 0 || (param_dtype != dtype && param_dtype != FP8BQ_FP32)) return FP8BQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_rows(M, N) || ldx < N || ldy < N) return FP8BQ_ERR_SHAPE;
  if (M > 0 && N > 0 && (!x || !y)) return FP8BQ_ERR_INVALID_ARG;
  const int64_t pe = elem_bytes(param_dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(gamma, pe) || !aligned_to(beta, pe) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return FP8BQ_ERR_ALIGN;
  if (M == 0 || N == 0) return FP8BQ_OK;
  const int st = device_ok();
  if (st != FP8BQ_OK) return st;
  const fp8bq::NormFwd a{x, gamma, beta, y, mean, rstd, M, N, ldx, ldy, eps, dtype, param_dtype};
  return cuda_status(fp8bq::launch_layernorm_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_layernorm_backward(const fp8bq_norm_grad* args, fp8bq_stream_t stream) {
  return norm_backward(args, true, reinterpret_cast<cudaStream_t>(stream));
}

int fp8bq_rmsnorm_backward(const fp8bq_norm_grad* args, fp8bq_stream_t stream) {
  return norm_backward(args, false, reinterpret_cast<cudaStream_t>(stream));
}

int64_t fp8bq_norm_workspace_bytes(int64_t M, int64_t N) {
  int sms = 0;
  if (!valid_rows(M, N) || device_ok() != FP8BQ_OK || fp8bq::device_sm_count(&sms) != cudaSuccess) return -1;
  return fp8bq::norm_bwd_workspace_bytes(M, N, sms);
}

int fp8bq_grad_norm(const fp8bq_grad* grads, int count, float* norm, void* workspace, int64_t workspace_bytes,
                    fp8bq_stream_t stream) {
  return grad_list(grads, count, 0.0, false, norm, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int fp8bq_grad_clip(const fp8bq_grad* grads, int count, double max_norm, float* norm, void* workspace,
                    int64_t workspace_bytes, fp8bq_stream_t stream) {
  return grad_list(grads, count, max_norm, true, norm, workspace, workspace_bytes,
                   reinterpret_cast<cudaStream_t>(stream));
}

int64_t fp8bq_grad_workspace_bytes(int count) {
  int sms = 0;
  if (count < 0 || device_ok() != FP8BQ_OK || fp8bq::device_sm_count(&sms) != cudaSuccess) return -1;
  return fp8bq::grad_clip_workspace_bytes(count, sms);
}

int fp8bq_quantize_weight(const void* w, int64_t N, int64_t K, int64_t ldw, void* q, void* scales,
                          int fmt, fp8bq_stream_t stream) {
  int st = check_quant_args(w, N, K, ldw, q, scales, fmt);
  if (st != FP8BQ_OK) return st;
  if (K % 128 != 0) return FP8BQ_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8BQ_OK;
  if ((st = device_ok()) != FP8BQ_OK) return st;
  const fp8bq::QuantJob job{w, N, K, ldw, q, scales, nullptr, nullptr, true};
  return cuda_status(fp8bq::launch_quant_group(&job, 1, fmt, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_quantize_group(const fp8bq_quant_job* jobs, int njobs, int fmt, fp8bq_stream_t stream) {
  if (jobs == nullptr || njobs < 1 || njobs > 8) return FP8BQ_ERR_INVALID_ARG;
  if (!valid_fmt(fmt)) return FP8BQ_ERR_INVALID_ARG;
  fp8bq::QuantJob jb[8];
  for (int i = 0; i < njobs; ++i) {
    const fp8bq_quant_job& j = jobs[i];
    const bool rows = j.kind == FP8BQ_QUANT_ACT || j.kind == FP8BQ_QUANT_ACT_DUAL || j.kind == FP8BQ_QUANT_WEIGHT;
    const bool cols = j.kind == FP8BQ_QUANT_ACT_T || j.kind == FP8BQ_QUANT_ACT_DUAL;
    if (!rows && !cols) return FP8BQ_ERR_INVALID_ARG;
    int st = FP8BQ_OK;
    if (rows && (st = check_quant_args(j.x, j.rows, j.cols, j.ldx, j.q, j.scales, fmt)) != FP8BQ_OK) return st;
    if (cols && (st = check_quant_args(j.x, j.rows, j.cols, j.ldx, j.qt, j.scales_t, fmt)) != FP8BQ_OK) return st;
    if (rows && j.cols % 128 != 0) return FP8BQ_ERR_SHAPE;
    if (cols && j.rows % 128 != 0) return FP8BQ_ERR_SHAPE;
    if (cols && j.cols % 8 != 0) return FP8BQ_ERR_ALIGN;
    jb[i] = fp8bq::QuantJob{j.x, j.rows, j.cols, j.ldx, rows ? j.q : nullptr, rows ? j.scales : nullptr,
                            cols ? j.qt : nullptr, cols ? j.scales_t : nullptr, j.kind == FP8BQ_QUANT_WEIGHT};
  }
  bool any = false;
  for (int i = 0; i < njobs; ++i) any = any || (jb[i].rows > 0 && jb[i].cols > 0);
  if (!any) return FP8BQ_OK;
  int st = device_ok();
  if (st != FP8BQ_OK) return st;
  return cuda_status(fp8bq::launch_quant_group(jb, njobs, fmt, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8bq_gemm(const fp8bq_operand* A, const fp8bq_operand* B, void* D, int64_t M, int64_t N,
               int64_t K, int64_t ldd, uint32_t flags, fp8bq_stream_t stream) {
  return fp8bq_gemm_ws(A, B, D, M, N, K, ldd, flags, nullptr, 0, stream);
}

int64_t fp8bq_gemm_workspace_bytes(void) {
  if (device_ok() != FP8BQ_OK) return -1;
  int sms = 0;
  if (fp8bq::device_sm_count(&sms) != cudaSuccess) return -1;
  return static_cast<int64_t>(sms / 2) * fp8bq::kWsSlotBytes;
}

int fp8bq_gemm_ws(const fp8bq_operand* A, const fp8bq_operand* B, void* D, int64_t M, int64_t N, int64_t K,
                  int64_t ldd, uint32_t flags, void* workspace, int64_t workspace_bytes, fp8bq_stream_t stream) {
  if (workspace != nullptr && workspace_bytes < 0) return FP8BQ_ERR_INVALID_ARG;
  if (workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return FP8BQ_ERR_ALIGN;
  fp8bq::GemmProblem p;
  int st = fp8bq::validate_gemm(A, B, D, M, N, K, ldd, flags, &p);
  if (st != FP8BQ_OK) return st;
  p.ws = workspace;
  p.ws_bytes = workspace != nullptr ? workspace_bytes : 0;
  return fp8bq::run_gemm(p, reinterpret_cast<cudaStream_t>(stream));
}

int fp8bq_testing_gemm_ws_withhold(const fp8bq_operand* A, const fp8bq_operand* B, void* D, int64_t M, int64_t N,
                                   int64_t K, int64_t ldd, uint32_t flags, void* workspace, int64_t workspace_bytes,
                                   int withhold_pair, int64_t wait_limit_ns, fp8bq_stream_t stream) {
  if (workspace == nullptr || workspace_bytes < 0 || withhold_pair < 0) return FP8BQ_ERR_INVALID_ARG;
  if (wait_limit_ns < 100000 || wait_limit_ns > 2000000000LL) return FP8BQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return FP8BQ_ERR_ALIGN;
  fp8bq::GemmProblem p;
  int st = fp8bq::validate_gemm(A, B, D, M, N, K, ldd, flags, &p);
  if (st != FP8BQ_OK) return st;
  p.ws = workspace;
  p.ws_bytes = workspace_bytes;
  p.withhold_cluster = withhold_pair;
  p.wait_limit_ns = static_cast<uint64_t>(wait_limit_ns);
  return fp8bq::run_gemm(p, reinterpret_cast<cudaStream_t>(stream));
}

int64_t fp8bq_row_scale_ld(int64_t rows) { return rows < 0 ? -1 : fp8bq::round_up128(rows); }

int64_t fp8bq_scales_bytes(int gran, int fmt, int64_t rows, int64_t contraction) {
  if (!valid_fmt(fmt) || rows < 0 || contraction < 0 || contraction % 128 != 0) return -1;
  const int64_t esz = fmt == FP8BQ_SCALE_FP32 ? 4 : 1;
  const int64_t nkb = contraction / 128;
  if (gran == FP8BQ_GRAN_ROW_1x128) return nkb * fp8bq::round_up128(rows) * esz;
  if (gran == FP8BQ_GRAN_ROW_1x32)
    return fmt == FP8BQ_SCALE_UE8M0 ? (contraction / 32) * fp8bq::round_up128(rows) : -1;
  if (gran == FP8BQ_GRAN_BLOCK_128x128) return nkb * ((rows + 127) / 128) * esz;
  return -1;
}

int fp8bq_check(fp8bq_stream_t stream) {
  int status = 0;
  cudaError_t e = fp8bq::read_and_clear_device_status(reinterpret_cast<cudaStream_t>(stream), &status);
  if (e != cudaSuccess) return cuda_status(e);
  if (status == fp8bq::kStatusIndex) return FP8BQ_ERR_INDEX;
  return status != 0 ? FP8BQ_ERR_TIMEOUT : FP8BQ_OK;
}

int fp8bq_set_clock_counters(unsigned long long* counters) {
  if (counters != nullptr && (reinterpret_cast<uintptr_t>(counters) & 7u) != 0) return FP8BQ_ERR_ALIGN;
  int st = device_ok();
  if (st != FP8BQ_OK) return st;
  return cuda_status(fp8bq::set_clock_counters(counters));
}

int fp8bq_last_cuda_error(void) { return t_last_cuda_error; }

const char* fp8bq_status_string(int status) {
  switch (status) {
    case FP8BQ_OK: return "ok";
    case FP8BQ_ERR_INVALID_ARG: return "invalid argument";
    case FP8BQ_ERR_SHAPE: return "bad shape";
    case FP8BQ_ERR_ALIGN: return "misaligned pointer or leading dimension";
    case FP8BQ_ERR_UNSUPPORTED: return "unsupported device or operand combination";
    case FP8BQ_ERR_CUDA: return "CUDA error";
    case FP8BQ_ERR_TIMEOUT: return "device wait timed out";
    case FP8BQ_ERR_INDEX: return "token id outside the embedding table";
    default: return "unknown status";
  }
}

int fp8bq_version(void) { return 100; }

}  // extern "C"
