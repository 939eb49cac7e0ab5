// row_binding.cpp -- the Python side of the row operators (embedding, norms,
// gradient clipping): checks of the tensors, new outputs and workspaces, the
// current stream, and the call of the C ABI in include/fp8bq.h.
//
// Compiled, unlike the ctypes binding of the other calls, because these
// operators run for a few microseconds on small batches: with checks and
// allocations in Python and ctypes' conversions, LayerNorm at [8, 2048] took
// 13.1 us of the host's time, here 6.1 (the launch alone about 3.5).  Nothing
// is computed here.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/extension.h>

#include <optional>
#include <tuple>
#include <vector>

#include "fp8bq.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

struct Library {
  decltype(&fp8bq_embedding_forward) embedding_forward;
  decltype(&fp8bq_embedding_backward) embedding_backward;
  decltype(&fp8bq_embedding_workspace_bytes) embedding_workspace_bytes;
  decltype(&fp8bq_layernorm_forward) layernorm_forward;
  decltype(&fp8bq_layernorm_backward) layernorm_backward;
  decltype(&fp8bq_rmsnorm_backward) rmsnorm_backward;
  decltype(&fp8bq_norm_workspace_bytes) norm_workspace_bytes;
  decltype(&fp8bq_grad_norm) grad_norm;
  decltype(&fp8bq_grad_clip) grad_clip;
  decltype(&fp8bq_grad_workspace_bytes) grad_workspace_bytes;
} lib;

// Takes the entry points from libfp8bq.so.
void load(const std::string& path) {
  void* h = dlopen(path.c_str(), RTLD_NOW | RTLD_LOCAL);
  if (h == nullptr) throw py::import_error(dlerror());
  const auto take = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    if (f == nullptr) throw py::import_error(std::string(name) + " is missing from " + path);
  };
  take(lib.embedding_forward, "fp8bq_embedding_forward");
  take(lib.embedding_backward, "fp8bq_embedding_backward");
  take(lib.embedding_workspace_bytes, "fp8bq_embedding_workspace_bytes");
  take(lib.layernorm_forward, "fp8bq_layernorm_forward");
  take(lib.layernorm_backward, "fp8bq_layernorm_backward");
  take(lib.rmsnorm_backward, "fp8bq_rmsnorm_backward");
  take(lib.norm_workspace_bytes, "fp8bq_norm_workspace_bytes");
  take(lib.grad_norm, "fp8bq_grad_norm");
  take(lib.grad_clip, "fp8bq_grad_clip");
  take(lib.grad_workspace_bytes, "fp8bq_grad_workspace_bytes");
}

// A failed call becomes the package's Fp8bqError.
void check(int status, const char* what) {
  if (status != FP8BQ_OK) py::module_::import("blockwise_fp8_linear_fp8bq_b200").attr("_raise")(status, what);
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return FP8BQ_BF16;
    case at::kHalf: return FP8BQ_FP16;
    case at::kFloat: return FP8BQ_FP32;
    default: return 0;
  }
}

void check_cuda(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda(), "fp8bq runs on CUDA tensors only (no CPU path)"); }

// Checks a 2-D row-major bf16, fp16 or fp32 CUDA tensor; its leading dimension.
int64_t rows(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(code_of(t.scalar_type()) != 0, name, " must be bf16, fp16 or fp32");
  TORCH_CHECK_VALUE(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1), name, " must be a 2-D row-major tensor");
  check_cuda(t);
  return t.size(0) > 1 || t.stride(0) >= t.size(1) ? t.stride(0) : t.size(1);
}

// The same of x's shape, dtype and device.
int64_t rows_like(const Tensor& t, const char* name, const Tensor& x) {
  TORCH_CHECK_VALUE(t.sizes() == x.sizes() && t.scalar_type() == x.scalar_type() && t.device() == x.device(), name,
                    " must have shape ", x.sizes(), ", dtype ", x.scalar_type(), " and device ", x.device());
  return rows(t, name);
}

// Checks a contiguous vector of n entries; its address.
template <class P = void>
P* vector(const Tensor& t, const char* name, int64_t n, at::ScalarType a, at::ScalarType b, const Tensor& x) {
  TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n && t.is_contiguous() && t.device() == x.device() &&
                        (t.scalar_type() == a || t.scalar_type() == b),
                    name, " must be a contiguous vector of ", n, " entries of dtype ", a, " or ", b, " on ", x.device());
  return static_cast<P*>(t.data_ptr());
}

// A new contiguous tensor on x's device, past the dispatcher (0.4 us less).
Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& x) {
  return Tensor(at::detail::empty_cuda(shape, dtype, x.device(), std::nullopt));
}

Tensor new_rows(const Tensor& x) { return empty(x.sizes(), x.scalar_type(), x); }

// An FP32 vector to write: the one given, or a new one.
float* output(Maybe& t, const char* name, int64_t n, const Tensor& x) {
  if (t) return vector<float>(*t, name, n, at::kFloat, at::kFloat, x);
  t = empty({n}, at::kFloat, x);
  return static_cast<float*>(t->data_ptr());
}

// A workspace of n bytes (none for 0).
Tensor workspace(int64_t n, const Tensor& x, const char* what) {
  TORCH_CHECK(n >= 0, what, ": bad arguments or no usable device");
  return n == 0 ? Tensor() : empty({n}, at::kByte, x);
}
void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The device made current, and its current stream.
struct Call {
  explicit Call(const Tensor& t)
      : guard(t.device()),
        stream(reinterpret_cast<fp8bq_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream())) {}
  c10::cuda::CUDAGuard guard;
  fp8bq_stream_t stream;
};

int wide_ids(const Tensor& ids, const Tensor& x) {
  TORCH_CHECK_VALUE((ids.scalar_type() == at::kLong || ids.scalar_type() == at::kInt) && ids.is_contiguous() &&
                        ids.device() == x.device(),
                    "ids must be a contiguous int32 or int64 tensor on ", x.device());
  return ids.scalar_type() == at::kLong ? 1 : 0;
}

Tensor embedding_forward(const Tensor& w, const Tensor& ids, double scale, const Maybe& out,
                         std::optional<at::ScalarType> dtype) {
  const int64_t ldw = rows(w, "w"), V = w.size(0), D = w.size(1), T = ids.numel();
  const int wide = wide_ids(ids, w);
  Tensor y;
  int64_t ldy = D;
  if (out) {
    y = *out;
    ldy = rows(y, "out");
    TORCH_CHECK_VALUE(y.size(0) == T && y.size(1) == D && y.device() == w.device() && (!dtype || y.scalar_type() == *dtype),
                      "out must have shape [", T, ", ", D, "], the dtype asked for and w's device");
  } else {
    auto shape = ids.sizes().vec();
    shape.push_back(D);
    y = empty(shape, dtype.value_or(w.scalar_type()), w);
  }
  const Call call(w);
  check(lib.embedding_forward(w.data_ptr(), V, D, ldw, ids.data_ptr(), wide, T, static_cast<float>(scale), y.data_ptr(), ldy,
                              code_of(w.scalar_type()), code_of(y.scalar_type()), call.stream),
        "fp8bq_embedding_forward");
  return y;
}

Tensor embedding_backward(const Tensor& dy_, const Tensor& ids, int64_t vocab, double scale, int64_t padding, const Maybe& out,
                          bool accumulate, at::ScalarType dtype) {
  const int64_t T = ids.numel(), D = dy_.dim() > 0 ? dy_.size(-1) : 0;
  Tensor dy = dy_;
  if (dy.dim() != 2) {
    auto shape = ids.sizes().vec();
    shape.push_back(D);
    TORCH_CHECK_VALUE(dy.sizes() == shape && dy.is_contiguous(),
                      "dy must be [ids.numel(), D], or contiguous [*ids.shape, D]");
    dy = dy.view({T, D});
  }
  const int64_t lddy = rows(dy, "dy");
  TORCH_CHECK_VALUE(dy.size(0) == T, "dy must have a row for each id");
  TORCH_CHECK_VALUE(vocab >= 0, "vocab must not be negative");
  const int wide = wide_ids(ids, dy);
  Tensor dw;
  int64_t lddw = D;
  if (out) {
    dw = *out;
    lddw = rows(dw, "out");
    TORCH_CHECK_VALUE(dw.size(0) == vocab && dw.size(1) == D && dw.device() == dy.device(), "out must have shape [", vocab, ", ",
                      D, "] and dy's device");
  } else {
    TORCH_CHECK_VALUE(!accumulate, "accumulate=True needs the tensor to add into");
    dw = empty({vocab, D}, dtype, dy);
  }
  const Call call(dy);
  const int64_t n = lib.embedding_workspace_bytes(T, D, vocab);
  const Tensor ws = workspace(n, dy, "fp8bq_embedding_workspace_bytes");
  check(lib.embedding_backward(dy.data_ptr(), T, D, lddy, ids.data_ptr(), wide, vocab, static_cast<float>(scale), padding,
                               dw.data_ptr(), lddw, code_of(dy.scalar_type()), code_of(dw.scalar_type()),
                               accumulate ? FP8BQ_EMBEDDING_ACCUMULATE : 0, address(ws), n, call.stream),
        "fp8bq_embedding_backward");
  return dw;
}

std::tuple<Tensor, Tensor, Tensor> layernorm_forward(const Tensor& x, const Maybe& gamma, const Maybe& beta, double eps, Maybe y,
                                                     Maybe mean, Maybe rstd) {
  const int64_t ldx = rows(x, "x"), M = x.size(0), N = x.size(1);
  const auto dt = x.scalar_type();
  auto pdt = gamma ? gamma->scalar_type() : beta ? beta->scalar_type() : dt;
  const void* g = gamma ? vector(*gamma, "gamma", N, dt, at::kFloat, x) : nullptr;
  const void* b = beta ? vector(*beta, "beta", N, gamma ? pdt : dt, gamma ? pdt : at::kFloat, x) : nullptr;
  const int64_t ldy = y ? rows_like(*y, "y", x) : N;
  if (!y) y = new_rows(x);
  float* pm = output(mean, "mean", M, x);
  float* pr = output(rstd, "rstd", M, x);
  const Call call(x);
  check(lib.layernorm_forward(x.data_ptr(), M, N, ldx, g, b, static_cast<float>(eps), y->data_ptr(), ldy, pm, pr, code_of(dt),
                              code_of(pdt), call.stream),
        "fp8bq_layernorm_forward");
  return {*y, *mean, *rstd};
}

std::tuple<Tensor, Maybe, Maybe> norm_backward(bool layernorm, const Tensor& dy, const Tensor& x, const Maybe& mean,
                                               const Tensor& rstd, const Maybe& gamma, const Maybe& dres, bool params, Maybe dx,
                                               Maybe dgamma, Maybe dbeta, bool accumulate) {
  fp8bq_norm_grad a{};
  const auto dt = x.scalar_type();
  a.ldx = rows(x, "x");
  a.M = x.size(0);
  a.N = x.size(1);
  a.x = x.data_ptr();
  a.lddy = rows_like(dy, "dy", x);
  a.dy = dy.data_ptr();
  if (dres) {
    a.lddres = rows_like(*dres, "dres", x);
    a.dres = dres->data_ptr();
  }
  a.lddx = dx ? rows_like(*dx, "dx", x) : a.N;
  if (gamma) a.gamma = vector(*gamma, "gamma", a.N, dt, at::kFloat, x);
  TORCH_CHECK_VALUE(!layernorm || mean, "mean is missing");
  if (layernorm) a.mean = vector<const float>(*mean, "mean", a.M, at::kFloat, at::kFloat, x);
  a.rstd = vector(rstd, "rstd", a.M, at::kFloat, at::kDouble, x);
  a.dtype = code_of(dt);
  a.param_dtype = gamma ? code_of(gamma->scalar_type()) : a.dtype;
  a.flags = (accumulate ? FP8BQ_NORM_ACCUMULATE : 0u) | (rstd.scalar_type() == at::kDouble ? FP8BQ_NORM_RSTD_F64 : 0u);
  if (!dx) dx = new_rows(x);
  a.dx = dx->data_ptr();
  const Call call(x);
  Tensor ws;
  if (params) {
    TORCH_CHECK_VALUE(!accumulate || (dgamma && (dbeta || !layernorm)), "accumulate=True needs the tensors to add into");
    a.dgamma = output(dgamma, "dgamma", a.N, x);
    if (layernorm) a.dbeta = output(dbeta, "dbeta", a.N, x);
    a.workspace_bytes = lib.norm_workspace_bytes(a.M, a.N);
    ws = workspace(a.workspace_bytes, x, "fp8bq_norm_workspace_bytes");
    a.workspace = address(ws);
  } else {
    dgamma.reset();
    dbeta.reset();
  }
  if (layernorm)
    check(lib.layernorm_backward(&a, call.stream), "fp8bq_layernorm_backward");
  else
    check(lib.rmsnorm_backward(&a, call.stream), "fp8bq_rmsnorm_backward");
  return {*dx, dgamma, dbeta};
}

// The norm of the listed gradients, and with max_norm their clipped values.
Tensor grads(const std::vector<Tensor>& g, const std::optional<std::vector<Tensor>>& out, std::optional<double> max_norm) {
  TORCH_CHECK_VALUE(!g.empty(), "no gradients");
  TORCH_CHECK_VALUE(g.size() <= INT32_MAX && (!out || out->size() == g.size()), "as many outputs as gradients");
  check_cuda(g[0]);
  std::vector<fp8bq_grad> table(g.size());
  for (size_t i = 0; i < g.size(); ++i) {
    const Tensor& o = out ? (*out)[i] : g[i];
    TORCH_CHECK_VALUE(code_of(g[i].scalar_type()) != 0 && g[i].device() == g[0].device(),
                      "the gradients must be bf16, fp16 or fp32 tensors on one CUDA device");
    TORCH_CHECK_VALUE(g[i].is_non_overlapping_and_dense(), "a gradient must fill one span of memory");
    TORCH_CHECK_VALUE(o.is_same(g[i]) || (code_of(o.scalar_type()) != 0 && o.sizes() == g[i].sizes() &&
                                          o.device() == g[0].device() &&
                                          ((o.is_contiguous() && g[i].is_contiguous()) || o.strides() == g[i].strides())),
                      "each output must be bf16, fp16 or fp32 of its gradient's shape, strides and device");
    table[i] = fp8bq_grad{g[i].data_ptr(), o.data_ptr(), g[i].numel(), code_of(g[i].scalar_type()), code_of(o.scalar_type())};
  }
  const Call call(g[0]);
  const int count = static_cast<int>(g.size());
  const int64_t n = lib.grad_workspace_bytes(count);
  const Tensor ws = workspace(n, g[0], "fp8bq_grad_workspace_bytes");
  const Tensor norm = empty({}, at::kFloat, g[0]);
  float* p = static_cast<float*>(norm.data_ptr());
  if (max_norm)
    check(lib.grad_clip(table.data(), count, *max_norm, p, address(ws), n, call.stream), "fp8bq_grad_clip");
  else
    check(lib.grad_norm(table.data(), count, p, address(ws), n, call.stream), "fp8bq_grad_norm");
  return norm;
}

}  // namespace

PYBIND11_MODULE(_row_binding, m) {
  m.attr("torch_version") = FP8BQ_TORCH_VERSION;  // the package refuses the module beside another
  m.def("load", &load);
  m.def("embedding_forward", &embedding_forward);
  m.def("embedding_backward", &embedding_backward);
  m.def("layernorm_forward", &layernorm_forward);
  m.def("norm_backward", &norm_backward);
  m.def("grads", &grads);
}
