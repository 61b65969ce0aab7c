// qta_norm.cuh -- residual add + norm of rows, its backward pass, and the
// column sums of the weights' and biases' gradients.
#pragma once

#include "qta_act.cuh"

namespace qta {

struct NormParams {
    const void* x;
    const void* residual;   // NULL: none
    const void* gamma;
    const void* beta;       // NULL: none
    void* y;
    void* sum;              // NULL: not stored
    float* mean;            // NULL: not stored
    float* rstd;            // NULL: not stored
    int64_t rows, cols;
    int64_t ld_x, ld_r, ld_y, ld_s;
    float eps;
    int dt, w_dt, rms;
    int shift;              // elements from a 16-byte boundary to row 0
    int w_smem;             // gamma and beta are kept in shared memory
    int aligned, w_vec;     // rows are whole aligned vectors; gamma and beta are 16-byte aligned
};

struct NormBwdParams {
    const void* dy;
    const void* s;
    const void* gamma;
    const float* mean;      // NULL: RMS
    const float* rstd;
    const void* dsum;       // NULL: none
    void* dx;
    float* part;            // [parts][2][cols] partial sums of dgamma, dbeta
    float* dgamma;
    float* dbeta;           // NULL: not computed
    int64_t rows, cols;
    int64_t ld_dy, ld_s, ld_ds, ld_dx;
    int parts;
    int dt, w_dt, rms;
    int shift, aligned, w_vec, w_smem;   // as above
};

}  // namespace qta
