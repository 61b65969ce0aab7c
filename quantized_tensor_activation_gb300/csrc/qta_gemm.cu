// qta_gemm.cu -- instantiations and launcher of the matrix-product kernels.
#include "qta_layer.cuh"

namespace qta {

// Clusters of `size` CTAs of the split kernel that can be resident at once (an
// SM has room for one CTA; clusters of 8 leave 32 of 152 SMs without one).
static int resident_clusters(int size, int sms)
{
    static std::atomic<int> cache[4];
    const int i = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    int n = cache[i].load();
    if (n) return n;
    auto fn = gemm_split_kernel<false, false, EPI_LINEAR>;
    static std::atomic<unsigned> done{0};
    if (ensure_smem_attr(reinterpret_cast<const void*>(fn), SPLIT_SMEM, &done) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / size * size));
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = SPLIT_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) return 0;
    cache[i].store(n);
    return n;
}

// Pairs of CTAs on 256 x 256 tiles where the 128 x 128 tiles are more than the
// SMs, else the split kernel on those (1021 x 1000 -> 1096, bf16: 9 us against
// 22 in 20 pairs).  The contraction of each is split while the clusters are
// resident at once (in half the GPU where two such launches run side by side)
// and a CTA keeps at least 4 blocks: a block takes 0.30 us, the join as long
// as 5 to 8 of them (512 x 1024, S = 1, 2, 4: 16 blocks 9.8, 8.2, 8.1 us; 8
// blocks 7.1, 6.5, 7.2 us; 1021 x 1096: 16 blocks 9.9, 8.9 us; 8 blocks 7.2,
// 7.4 us).
constexpr int SPLIT_MIN_BLOCKS = 12;

GemmTile gemm_tile(int epi, int64_t M, int64_t N, int64_t blocks, int groups, int sms, bool shared)
{
    const bool dual = epi == EPI_GATED || epi == EPI_GATED_BWD;
    const int64_t tile_n = dual ? 64 : 128, tiles = ((M + 127) / 128) * ((N + tile_n - 1) / tile_n) * groups;
    if (tiles > sms) return {256, dual ? 128 : 256, 128, 0};
    int s = 1;
    if (blocks >= SPLIT_MIN_BLOCKS)
        while (s < 8 && tiles * (shared ? 2 : 1) <= resident_clusters(2 * s, sms) && blocks >= 4 * (2 * s)) s *= 2;
    return {128, static_cast<int>(tile_n), static_cast<int>(tile_n), s};
}

template <bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_pairs(const GemmParams& p, int sms, cudaStream_t stream)
{
    static std::atomic<unsigned> done{0};
    auto fn = gemm_kernel<A_MN, B_MN, EPI>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fn), GEMM_SMEM, &done);
    if (e != cudaSuccess) return e;
    // pairs that can be resident at once (an odd SM of a cluster of SMs has no partner)
    static std::atomic<int> slots{0};
    int n = slots.load();
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
        cfg.blockDim = dim3(GEMM_THREADS);
        cfg.dynamicSmemBytes = GEMM_SMEM;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) n = sms / 2;
        slots.store(n);
    }
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.groups;
    GemmParams q = p;
    q.idesc |= idesc_f16(2 * GEMM_BM, 256, false, A_MN, B_MN);
    return launch_pdl(fn, dim3(static_cast<unsigned>((tiles < n ? tiles : n) * 2)), dim3(GEMM_THREADS), GEMM_SMEM,
                      stream, q);
}

template <bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_split(const GemmParams& p, cudaStream_t stream)
{
    static std::atomic<unsigned> done{0};
    auto fn = gemm_split_kernel<A_MN, B_MN, EPI>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fn), SPLIT_SMEM, &done);
    if (e != cudaSuccess) return e;
    GemmParams q = p;
    q.idesc |= idesc_f16(GEMM_BM, 128, false, A_MN, B_MN);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.tiles_m * p.tiles_n * p.groups * p.split));
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = SPLIT_SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, q);
}

template <bool A_MN, bool B_MN, int EPI>
static cudaError_t launch_t(const GemmParams& p, int sms, cudaStream_t stream)
{
    return p.split ? launch_split<A_MN, B_MN, EPI>(p, stream) : launch_pairs<A_MN, B_MN, EPI>(p, sms, stream);
}

cudaError_t launch_gemm(int form, int epi, const GemmParams& p, int sms, cudaStream_t stream)
{
    if (form == FORM_NN) return launch_t<false, true, EPI_LINEAR>(p, sms, stream);
    if (form == FORM_TN) return launch_t<true, true, EPI_LINEAR>(p, sms, stream);
    switch (epi) {
    case EPI_LINEAR: return launch_t<false, false, EPI_LINEAR>(p, sms, stream);
    case EPI_LINEAR_BWD: return launch_t<false, false, EPI_LINEAR_BWD>(p, sms, stream);
    case EPI_GATED: return launch_t<false, false, EPI_GATED>(p, sms, stream);
    case EPI_GATED_BWD: return launch_t<false, false, EPI_GATED_BWD>(p, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qta
