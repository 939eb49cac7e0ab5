// norm_bwd_bf16.cu -- the norms' backward kernels for BF16 rows.
#include "norm_bwd.cuh"

namespace fp8bq {

template cudaError_t run_norm_bwd<__nv_bfloat16>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);

}  // namespace fp8bq
