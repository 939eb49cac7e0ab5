// norm_bwd_fp16.cu -- the norms' backward kernels for FP16 rows.
#include "norm_bwd.cuh"

namespace fp8bq {

template cudaError_t run_norm_bwd<__half>(const BwdParams&, const RowPlan&, bool, bool, int64_t, cudaStream_t);

}  // namespace fp8bq
