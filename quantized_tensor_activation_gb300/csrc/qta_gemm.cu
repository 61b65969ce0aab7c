// qta_gemm.cu -- instantiations and launcher of the matrix-product kernels.
#include "qta_layer.cuh"

namespace qta {

constexpr int BN_ALL = 128;

int gemm_tile_cols(int, int epi) { return epi == EPI_GATED || epi == EPI_GATED_BWD ? BN_ALL / 2 : BN_ALL; }

template <int BN, bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_g(const GemmParams& p, int sms, cudaStream_t stream)
{
    using C = GemmCfg<BN>;
    static std::atomic<unsigned> done{0};
    auto fn = gemm_kernel<BN, A_MN, B_MN, EPI>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fn), C::SMEM, &done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    GemmParams q = p;
    q.idesc |= idesc_f16(GEMM_BM, BN, false, A_MN, B_MN);
    return launch_pdl(fn, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(GEMM_THREADS), C::SMEM, stream,
                      q);
}

cudaError_t launch_gemm(int form, int epi, const GemmParams& p, int sms, cudaStream_t stream)
{
    if (form == FORM_NN) return launch_g<BN_ALL, false, true, EPI_LINEAR>(p, sms, stream);
    if (form == FORM_TN) return launch_g<BN_ALL, true, true, EPI_LINEAR>(p, sms, stream);
    switch (epi) {
    case EPI_LINEAR: return launch_g<BN_ALL, false, false, EPI_LINEAR>(p, sms, stream);
    case EPI_LINEAR_BWD: return launch_g<BN_ALL, false, false, EPI_LINEAR_BWD>(p, sms, stream);
    case EPI_GATED: return launch_g<BN_ALL, false, false, EPI_GATED>(p, sms, stream);
    case EPI_GATED_BWD: return launch_g<BN_ALL, false, false, EPI_GATED_BWD>(p, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qta
