// qta_norm_bf16.cu -- the row kernels of the norms for bf16 activations.
#include "qta_norm_rows.cuh"

namespace qta {

cudaError_t launch_norm_rows_bf16(const NormParams& p, const RowPlan& q, int sms, cudaStream_t stream)
{
    return pick_row_kernel<0>(p.aligned, p.residual, p.cols, q, RunFwd{p, q, sms, stream});
}

cudaError_t launch_norm_bwd_rows_bf16(const NormBwdParams& p, const RowPlan& q, cudaStream_t stream)
{
    return pick_row_kernel<0>(p.aligned, p.dsum, p.cols, q, RunBwd{p, q, stream});
}

}  // namespace qta
