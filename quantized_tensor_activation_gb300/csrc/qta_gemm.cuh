// qta_gemm.cuh -- matrix products of the layer operators on the tensor cores.
//
//   D[m, n] = sum_k A[m, k] B[n, k]   (FP32 accumulators in TMEM)
//
// with an epilogue that finishes the operator in registers.  A pair of CTAs
// (or one CTA) computes tiles of 256 (128) x BN: warp 0 loads A and B in blocks
// of 64 contraction elements by TMA into a ring of shared-memory stages, warp
// 1 issues tcgen05.mma on them, warps 2-5 read the accumulators of the
// previous tile (TMEM holds two) and run the epilogue.  In a pair each CTA
// loads and keeps half of B, so a byte of shared memory feeds twice the
// products that it feeds in a single CTA: the single CTA's 128 x 128 tile is
// bound by shared memory.  Operands whose contraction index is
// not the contiguous one (the backward products) are read as they lie, with
// MN-major descriptors: nothing is transposed in memory.
//
// Rows and columns past an operand's end are filled with zeros by TMA, and
// contraction elements past its end too, so ragged sizes need no other path.
#pragma once

#include "qta_act.cuh"
#include "qta_tc.cuh"

namespace qta {

enum Epi : int {
    EPI_LINEAR = 0,      // f(D + bias) + residual
    EPI_LINEAR_BWD = 1,  // dz = aux f'(D + bias), column sums of dz
    EPI_GATED = 2,       // f(G) U, the tile's columns: half of G, half of U
    EPI_GATED_BWD = 3    // aux U f'(G) and aux f(G)
};

struct GemmParams {
    // k blocks below nk0 read (a[0], b[0]), the others (a[1], b[1]): a sum of
    // two products.  With groups == 2 instead, group g reads a[g] and writes
    // out[g].  The gated epilogues read their tile's columns from b[0] and b[1].
    CUtensorMap a[2], b[2];
    int M, N;                   // output rows and columns (of one group)
    int nk0, nk;                // contraction blocks of 64: of the first product, of both
    int tiles_m, tiles_n, groups;
    uint32_t idesc;
    int act;
    const void* bias;
    int bias_dt;
    const void* aux;            // residual (EPI_LINEAR), dy / dh (the backward epilogues)
    int64_t ld_aux;
    int aux_dt;
    void* out[2];
    int64_t ld_out[2];
    int out_dt;
    float* colsum;              // EPI_LINEAR_BWD: [tiles_m][N] partial column sums (NULL: none)
    unsigned int* err;
};

constexpr int GEMM_BM = 128;   // rows of one CTA's share of a tile
constexpr int GEMM_BK = 64;
constexpr int GEMM_THREADS = 192;

// CG CTAs compute one tile of CG * 128 x BN; each holds its 128 rows of A and
// its BN / CG rows of B.
template <int CG, int BN>
struct GemmCfg {
    static constexpr int BN_CTA = BN / CG;
    static constexpr int A_BYTES = GEMM_BM * GEMM_BK * 2;
    static constexpr int B_BYTES = BN_CTA * GEMM_BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int SMEM = STAGES * STAGE + 1024;   // + slack to start on 1024 bytes
    static constexpr uint32_t TMEM_COLS = 2 * BN;        // two accumulators
};

// Tiles in an order that keeps a wave of CTAs on few rows and columns of
// tiles: GROUP_M row tiles side by side, all column tiles of them, then the
// next rows.  What a wave reads then stays in L2 while its CTAs share it.
constexpr int GROUP_M = 8;

__device__ __forceinline__ void tile_coords(int r, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int band = r / (GROUP_M * tiles_n), first = band * GROUP_M;
    const int height = min(GROUP_M, tiles_m - first);
    const int in = r - band * GROUP_M * tiles_n;
    tm = first + in % height;
    tn = in / height;
}

// 32 elements of one row from column c0 on, n of them in range.
__device__ __forceinline__ void row_load32(const void* base, int64_t off, int dt, int n, float (&v)[32])
{
    const uint8_t* p = static_cast<const uint8_t*>(base) + off * dt_size(dt);
    if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        if (dt == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 w = q[i];
                v[4 * i] = __uint_as_float(w.x);
                v[4 * i + 1] = __uint_as_float(w.y);
                v[4 * i + 2] = __uint_as_float(w.z);
                v[4 * i + 3] = __uint_as_float(w.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 w = q[i];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2(ws[j], dt);
                    v[8 * i + 2 * j] = f.x;
                    v[8 * i + 2 * j + 1] = f.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < n ? load_elem(p, i, dt) : 0.0f;
    }
}

__device__ __forceinline__ void row_store32(void* base, int64_t off, int dt, int n, const float (&v)[32])
{
    uint8_t* p = static_cast<uint8_t*>(base) + off * dt_size(dt);
    if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        uint4* q = reinterpret_cast<uint4*>(p);
        if (dt == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = make_uint4(pack2(v[8 * i], v[8 * i + 1], dt), pack2(v[8 * i + 2], v[8 * i + 3], dt),
                                  pack2(v[8 * i + 4], v[8 * i + 5], dt), pack2(v[8 * i + 6], v[8 * i + 7], dt));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) store_elem(p, i, dt, v[i]);
    }
}

// Sum of each of 32 columns over the 32 lanes, in a fixed order: in step s a
// lane keeps the half of its columns that its bit s selects and adds its
// partner's copy of that half, so lane j ends with column j (31 shuffles
// instead of 5 for each column).
__device__ __forceinline__ float column_sum32(float (&v)[32], int lane)
{
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float send = up ? v[i] : v[i + s];
            const float keep = up ? v[i + s] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    return v[0];
}

template <int CG, int BN, bool A_MN, bool B_MN, int EPI>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(GEMM_THREADS, 1) gemm_kernel(const __grid_constant__ GemmParams p)
{
    using C = GemmCfg<CG, BN>;
    constexpr bool DUAL = EPI == EPI_GATED || EPI == EPI_GATED_BWD;
    constexpr int TILE_N = DUAL ? BN / 2 : BN;   // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[C::STAGES], empty[C::STAGES], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ float colsum_s[EPI == EPI_LINEAR_BWD ? 4 * BN : 1];

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4 * CG);
        }
        mbar_init(&drain, 1);
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == 1) tmem_alloc<CG>(&tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();   // the barriers of both CTAs exist before either signals the other
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    // after the allocation: a successor that starts early allocates only once this CTA has what it needs
    pdl_trigger();

    const int per_group = p.tiles_m * p.tiles_n;
    const int n_tiles = per_group * p.groups;
    if (warp == 0) {
        if (lane == 0) {
            int s = 0, done = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; ok && t < n_tiles; t += step) {
                const int g = t / per_group, r = t - g * per_group;
                int tm, tn;
                tile_coords(r, p.tiles_m, p.tiles_n, tm, tn);
                const int m0 = (tm * CG + rank) * GEMM_BM, n0 = tn * TILE_N;
                const int nb = DUAL ? n0 : n0 + rank * C::BN_CTA;   // this CTA's rows of B
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (!mbar_wait(&empty[s], ph ^ 1u, p.err)) {
                        ok = false;
                        break;
                    }
                    const int second = kb >= p.nk0;
                    const int k0 = (second ? kb - p.nk0 : kb) * GEMM_BK;
                    const CUtensorMap* ma = &p.a[second | g];
                    const CUtensorMap* mb = &p.b[second];
                    uint8_t* sa = smem + s * C::STAGE;
                    uint8_t* sb = sa + C::A_BYTES;
                    auto load = [&](uint8_t* dst, const CUtensorMap* map, int c0, int c1) {
                        if constexpr (CG == 2)
                            tma_load_2d_pair(dst, map, c0, c1, leader_addr(&full[s]));
                        else
                            tma_load_2d(dst, map, c0, c1, &full[s]);
                    };
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * C::STAGE);
                    if constexpr (A_MN) {
#pragma unroll
                        for (int i = 0; i < GEMM_BM / 64; ++i) load(sa + i * BOX_BYTES, ma, m0 + 64 * i, k0);
                    } else {
                        load(sa, ma, k0, m0);
                    }
                    if constexpr (DUAL && CG == 2) {
                        load(sb, &p.b[rank], k0, nb);
                    } else if constexpr (DUAL) {
                        load(sb, &p.b[0], k0, nb);
                        load(sb + C::B_BYTES / 2, &p.b[1], k0, nb);
                    } else if constexpr (B_MN) {
#pragma unroll
                        for (int i = 0; i < C::BN_CTA / 64; ++i) load(sb + i * BOX_BYTES, mb, nb + 64 * i, k0);
                    } else {
                        load(sb, mb, k0, nb);
                    }
                    ++done;
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // let the loads in flight land before the shared memory goes away (with a pair, the even CTA's barriers
            // count both CTAs' loads, and neither leaves before both are here)
            if (!ok && rank == 0) {
                const int n = done < C::STAGES ? done : C::STAGES;
                const uint64_t until = globaltimer_ns() + 2000000000ull;
                for (int i = 1; i <= n; ++i) {
                    const int j = done - i;
                    mbar_wait_until(&full[j % C::STAGES], (j / C::STAGES) & 1u, until);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int s = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; ok && t < n_tiles; t += step, ++it) {
                const int buf = it & 1;
                const uint32_t drained = ((it >> 1) & 1) ^ 1u;
                if (!(CG == 2 ? mbar_wait_cluster(&acc_empty[buf], drained, p.err)
                              : mbar_wait(&acc_empty[buf], drained, p.err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (!mbar_wait(&full[s], ph, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = smem_desc<A_MN>(smem_u32(smem + s * C::STAGE));
                    const uint64_t db = smem_desc<B_MN>(smem_u32(smem + s * C::STAGE + C::A_BYTES));
#pragma unroll
                    for (int k = 0; k < GEMM_BK / 16; ++k)
                        tc_mma<CG>(tmem + buf * BN, da + k * K16_STEP<A_MN>, db + k * K16_STEP<B_MN>, p.idesc,
                               kb > 0 || k > 0);
                    tc_commit<CG>(&empty[s]);
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) tc_commit<CG>(&acc_full[buf]);
            }
            if (!ok) {   // the products in flight end before TMEM is freed
                tc_commit<CG>(&drain);
                mbar_wait_until(&drain, 0, globaltimer_ns() + 2000000000ull);
            }
        }
    } else {
        const int q = warp & 3;   // the TMEM lanes (rows) this warp may read: 32 q ...
        int it = 0;
        bool ok = true;   // after an expired wait a warp still takes part in the barriers below, without work
        for (int t = first; t < n_tiles; t += step, ++it) {
            const int buf = it & 1;
            const int g = t / per_group, r = t - g * per_group;
            int tm, tn;
            tile_coords(r, p.tiles_m, p.tiles_n, tm, tn);
            const int m0 = (tm * CG + rank) * GEMM_BM, n0 = tn * TILE_N;
            const int row = m0 + 32 * q + lane;
            const bool live = row < p.M;
            const int64_t row64 = row;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (it >> 1) & 1, p.err));
            tc_fence_after();
            const uint32_t acc = tmem + buf * BN + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
            for (int c = 0; ok && c < TILE_N; c += 32) {
                const int col = n0 + c;
                const int n = p.N - col;   // columns in range (may be <= 0)
                float v[32];
                tmem_ld32(acc + c, v);
                if constexpr (EPI == EPI_LINEAR) {
                    tmem_ld_wait();
                    if (n > 0) {
                        if (p.bias) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < n) v[i] += load_elem(p.bias, col + i, p.bias_dt);
                        }
                        if (p.act != ACT_NONE) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], p.act);
                        }
                        if (live) {
                            if (p.aux) {
                                float res[32];
                                row_load32(p.aux, row64 * p.ld_aux + col, p.aux_dt, n, res);
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] += res[i];
                            }
                            row_store32(p.out[g], row64 * p.ld_out[g] + col, p.out_dt, n, v);
                        }
                    }
                } else if constexpr (EPI == EPI_LINEAR_BWD) {
                    tmem_ld_wait();
                    float dy[32];
                    if (live && n > 0) {
                        row_load32(p.aux, row64 * p.ld_aux + col, p.aux_dt, n, dy);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float f, df;
                            const float z = v[i] + (p.bias && i < n ? load_elem(p.bias, col + i, p.bias_dt) : 0.0f);
                            act_both(z, p.act, f, df);
                            v[i] = i < n ? dy[i] * df : 0.0f;
                        }
                        row_store32(p.out[0], row64 * p.ld_out[0] + col, p.out_dt, n, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                    }
                    if (p.colsum) colsum_s[q * BN + c + lane] = column_sum32(v, lane);
                } else {
                    float u[32];
                    tmem_ld32(acc + TILE_N + c, u);
                    tmem_ld_wait();
                    if (live && n > 0) {
                        if constexpr (EPI == EPI_GATED) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], p.act) * u[i];
                            row_store32(p.out[0], row64 * p.ld_out[0] + col, p.out_dt, n, v);
                        } else {
                            float dh[32];
                            row_load32(p.aux, row64 * p.ld_aux + col, p.aux_dt, n, dh);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                float f, df;
                                act_both(v[i], p.act, f, df);
                                v[i] = dh[i] * u[i] * df;
                                u[i] = dh[i] * f;
                            }
                            row_store32(p.out[0], row64 * p.ld_out[0] + col, p.out_dt, n, v);
                            row_store32(p.out[1], row64 * p.ld_out[1] + col, p.out_dt, n, u);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    mbar_arrive_cluster(leader_addr(&acc_empty[buf]));
                else
                    mbar_arrive(&acc_empty[buf]);
            }
            if constexpr (EPI == EPI_LINEAR_BWD) {
                if (p.colsum) {   // the four warps' sums, in warp order
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    for (int c = threadIdx.x - 64; c < BN; c += 128)
                        if (n0 + c < p.N && m0 < p.M)
                            p.colsum[static_cast<int64_t>(m0 / GEMM_BM) * p.N + n0 + c] =
                                (colsum_s[c] + colsum_s[BN + c]) + (colsum_s[2 * BN + c] + colsum_s[3 * BN + c]);
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<CG>(tmem, C::TMEM_COLS);
}

}  // namespace qta
