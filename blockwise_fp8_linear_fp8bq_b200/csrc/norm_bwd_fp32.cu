// norm_bwd_fp32.cu -- the norms' backward kernels for FP32 rows.
#include "norm_bwd.cuh"

namespace fp8bq {

template cudaError_t run_norm_bwd<float>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);

}  // namespace fp8bq
