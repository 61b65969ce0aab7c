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

// Whether qta_skinny.cu takes a forward product: up to 16 tokens, and up to 32
// where the contraction is short (n_in, tokens: its time against the split
// kernel's; 1024, 32: 7.2 and 8.4 us; 2048, 32: 6.9 and 8.2; 3584, 32: 18.8 and
// 15.2; 4096, 17: 9.1 and 7.4).
inline bool skinny(int64_t rows, int64_t n_in) { return rows <= 16 || (rows <= 32 && n_in <= 2048); }

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
