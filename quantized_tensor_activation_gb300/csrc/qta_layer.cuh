// qta_layer.cuh -- host-side launchers of the layer operators (internal).
#pragma once

#include "qta_gemm.cuh"
#include "qta_launch.h"
#include "qta_norm.cuh"

namespace qta {

// Partial column sums of the backward passes: at most this many rows of them.
constexpr int64_t MAX_PARTS = 304;

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormBwdParams& p, int sms, cudaStream_t stream);
cudaError_t launch_col_sum(const void* a, int64_t ld, int dt, int64_t rows, int64_t cols, int parts, float* part,
                           cudaStream_t stream);
cudaError_t launch_col_finish(const float* part, int64_t stride, int parts, int64_t cols, float* out,
                              cudaStream_t stream);

// The operand forms of the products: both contiguous along the contraction
// (forward), B contiguous along its output index (dx = dz w), both (dw = dz^T x).
enum GemmForm : int { FORM_NT = 0, FORM_NN = 1, FORM_TN = 2 };

// Tile of a product: output rows and columns, rows of the TMA box of a
// contraction-contiguous B, CTAs that split its contraction (0: a pair's tile),
// accumulator columns.
struct GemmTile {
    int rows, cols, b_box, split, bn;
};
GemmTile gemm_tile(int epi, int64_t M, int64_t N, int64_t blocks, int groups, int sms, bool shared);
cudaError_t launch_gemm(int form, int epi, const GemmParams& p, int sms, cudaStream_t stream);

// dx (FORM_NN) and dw (FORM_TN) in one launch, where both are the split
// kernel's in clusters of one size; else nothing is launched.
bool launch_gemm_both(const GemmParams& dx, const GemmParams& dw, cudaStream_t stream, cudaError_t* e);

// Whether qta_skinny.cu takes a forward product (`dual`: of two weights): up to
// 8 tokens; up to 16 but for long contractions of two weights; up to 32 where the
// contraction is short.  Its time against the split kernel's, us, n_in x outputs:
//     one weight   16 tokens: 8192 x 2048 11.0, 11.1; 3584 x 8192 14.2, 14.0; 1024 x 1024 2.7, 4.2
//                  32 tokens: 2048 x 4096  7.2,  7.8; 1024 x 1024  3.8,  4.3; 4096 x 1024 9.7, 7.2
//     two          16 tokens: 2048 x 2048  6.8,  8.0; 3584 x 4096 12.6, 13.9; 4096 x  512 10.3, 7.2
//                  32 tokens:  512 x 1024  3.6,  4.2; 1024 x  512  4.8,  4.6; 2048 x 2048 8.5, 8.0
inline bool skinny(int64_t rows, int64_t n_in, bool dual)
{
    if (rows <= 8) return true;
    if (rows <= 16) return !dual || n_in < 4096;
    return rows <= 32 && n_in <= (dual ? 1024 : 2048);
}

struct SkinnyParams {
    const uint8_t* x;
    int64_t ldx;
    const uint8_t* w[2];    // the weight, or the gate's and the up projection's
    int64_t ldw[2];
    int M, N, K;
    int act;
    const void* bias;
    int bias_dt;
    const void* aux;        // residual of type out_dt (NULL: none)
    int64_t ld_aux;
    void* out;
    int64_t ld_out;
    int out_dt;
};
cudaError_t launch_skinny(int dt, bool dual, const SkinnyParams& p, cudaStream_t stream);

}  // namespace qta
