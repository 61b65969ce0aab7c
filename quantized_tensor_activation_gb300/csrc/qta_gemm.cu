// qta_gemm.cu -- instantiations and launcher of the matrix-product kernels.
#include "qta_layer.cuh"

namespace qta {

// Tiles of a launch.
struct Plan {
    int cg, bn;
};

static Plan plan_of(int form, int epi, int64_t M, int64_t N, int groups, int sms)
{
    const bool dual = epi == EPI_GATED || epi == EPI_GATED_BWD;
    const int64_t pairs = ((M + 255) / 256) * ((N + (dual ? 127 : 255)) / (dual ? 128 : 256)) * groups;
    if (pairs >= sms / 2) return {2, 256};
    return {1, 128};
}

GemmTile gemm_tile(int form, int epi, int64_t M, int64_t N, int groups, int sms)
{
    const bool dual = epi == EPI_GATED || epi == EPI_GATED_BWD;
    const Plan q = plan_of(form, epi, M, N, groups, sms);
    return {q.cg * GEMM_BM, dual ? q.bn / 2 : q.bn, dual ? 128 * q.bn / 256 : q.bn / q.cg, q.cg, q.bn};
}

template <int CG, int BN, bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_g(const GemmParams& p, int sms, cudaStream_t stream)
{
    using C = GemmCfg<CG, BN>;
    static std::atomic<unsigned> done{0};
    auto fn = gemm_kernel<CG, BN, A_MN, B_MN, EPI>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fn), C::SMEM, &done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    int64_t slots = sms;
    if constexpr (CG == 2) {   // pairs that can be resident at once (an odd SM of a cluster of SMs has no partner)
        static std::atomic<int> pairs{0};
        int n = pairs.load();
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
            cfg.blockDim = dim3(GEMM_THREADS);
            cfg.dynamicSmemBytes = C::SMEM;
            if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) n = sms / 2;
            pairs.store(n);
        }
        slots = n;
    }
    GemmParams q = p;
    q.idesc |= idesc_f16(GEMM_BM * CG, BN, false, A_MN, B_MN);
    return launch_pdl(fn, dim3(static_cast<unsigned>((tiles < slots ? tiles : slots) * CG)), dim3(GEMM_THREADS),
                      C::SMEM, stream, q);
}

template <bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_t(const GemmTile& t, const GemmParams& p, int sms, cudaStream_t stream)
{
    if (t.cg == 2) return launch_g<2, 256, A_MN, B_MN, EPI>(p, sms, stream);
    return launch_g<1, 128, A_MN, B_MN, EPI>(p, sms, stream);
}

cudaError_t launch_gemm(int form, int epi, const GemmTile& t, const GemmParams& p, int sms, cudaStream_t stream)
{
    if (form == FORM_NN) return launch_t<false, true, EPI_LINEAR>(t, p, sms, stream);
    if (form == FORM_TN) return launch_t<true, true, EPI_LINEAR>(t, p, sms, stream);
    switch (epi) {
    case EPI_LINEAR: return launch_t<false, false, EPI_LINEAR>(t, p, sms, stream);
    case EPI_LINEAR_BWD: return launch_t<false, false, EPI_LINEAR_BWD>(t, p, sms, stream);
    case EPI_GATED: return launch_t<false, false, EPI_GATED>(t, p, sms, stream);
    case EPI_GATED_BWD: return launch_t<false, false, EPI_GATED_BWD>(t, p, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qta
