// qta_norm_fp32.cu -- the row kernels of the norms for fp32 activations.
#include "qta_norm_rows.cuh"

namespace qta {

cudaError_t launch_norm_rows_fp32(const NormParams& p, const RowPlan& q, int sms, cudaStream_t stream)
{
    return pick_row_kernel<2>(p.aligned, p.residual, p.cols, q, RunFwd{p, q, sms, stream});
}

cudaError_t launch_norm_bwd_rows_fp32(const NormBwdParams& p, const RowPlan& q, cudaStream_t stream)
{
    return pick_row_kernel<2>(p.aligned, p.dsum, p.cols, q, RunBwd{p, q, stream});
}

}  // namespace qta
