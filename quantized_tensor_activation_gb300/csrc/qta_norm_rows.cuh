// qta_norm_rows.cuh -- norm kernels that hold a row in registers.
//
// Forward and backward read each byte once: a thread keeps VPT 16-byte
// vectors of its row, the statistics come from registers (the variance about
// the mean, in a second pass over registers), and the next row's vectors are
// on their way meanwhile.  What bounds them is HBM.
//
// Rows may start anywhere: where every matrix of a call has its rows at the
// same distance from a 16-byte boundary (one base alignment, row distances
// equal modulo a vector), vector v of a row holds the columns
// v * VEC - shift ... with shift that row's distance, so that all vectors but
// the first and last are aligned, whole ones.  AL: shift is 0 and cols whole
// vectors.
#pragma once

#include "qta_layer.cuh"

namespace qta {

template <int DT>
struct Vec {
    static constexpr int N = DT == 2 ? 4 : 8;
    static constexpr int ES = DT == 2 ? 4 : 2;

    static __device__ __forceinline__ void unpack(const uint4 w, float (&f)[N])
    {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == 2) {
                f[j] = __uint_as_float(ws[j]);
            } else {
                const float2 t = unpack2(ws[j], DT);
                f[2 * j] = t.x;
                f[2 * j + 1] = t.y;
            }
        }
    }

    static __device__ __forceinline__ uint4 pack(const float (&f)[N])
    {
        if constexpr (DT == 2)
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
        else
            return make_uint4(pack2(f[0], f[1], DT), pack2(f[2], f[3], DT), pack2(f[4], f[5], DT),
                              pack2(f[6], f[7], DT));
    }

    // Vector of the columns c0 ... of the row at `row`, zeros outside [0, cols).
    template <bool AL>
    static __device__ __forceinline__ uint4 load(const uint8_t* row, int c0, int cols)
    {
        if (c0 >= 0 && c0 + N <= cols) return __ldcs(reinterpret_cast<const uint4*>(row + c0 * ES));
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!AL) {
            uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (c0 + k >= 0 && c0 + k < cols) {
                    if constexpr (DT == 2)
                        ws[k] = reinterpret_cast<const uint32_t*>(row)[c0 + k];
                    else
                        ws[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[c0 + k])
                                     << (16 * (k & 1));
                }
        }
        return w;
    }

    template <bool AL>
    static __device__ __forceinline__ void store(uint8_t* row, int c0, int cols, const float (&f)[N])
    {
        const uint4 w = pack(f);
        if (c0 >= 0 && c0 + N <= cols) {
            *reinterpret_cast<uint4*>(row + c0 * ES) = w;
        } else if constexpr (!AL) {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (c0 + k >= 0 && c0 + k < cols) {
                    if constexpr (DT == 2)
                        reinterpret_cast<uint32_t*>(row)[c0 + k] = ws[k];
                    else
                        reinterpret_cast<uint16_t*>(row)[c0 + k] = static_cast<uint16_t>(ws[k / 2] >> (16 * (k & 1)));
                }
        }
    }

    // gamma or beta of the columns c0 ..., zeros outside.  `vec`: 16-byte aligned.
    template <bool AL>
    static __device__ __forceinline__ void weights(const void* w, int w_dt, bool vec, int c0, int cols, float (&f)[N])
    {
        if (AL && vec) {
            if (c0 < cols) {
                if (w_dt == DT) {
                    unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(w) + c0 * ES)), f);
                } else {   // fp32 weights of a 16-bit activation
                    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0);
#pragma unroll
                    for (int j = 0; j < N / 4; ++j) {
                        const float4 t = __ldg(q + j);
                        f[4 * j] = t.x;
                        f[4 * j + 1] = t.y;
                        f[4 * j + 2] = t.z;
                        f[4 * j + 3] = t.w;
                    }
                }
                return;
            }
#pragma unroll
            for (int k = 0; k < N; ++k) f[k] = 0.0f;
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = c0 + k >= 0 && c0 + k < cols ? load_elem(w, c0 + k, w_dt) : 0.0f;
    }
};

// A CTA works on G rows at a time, T threads (whole warps) on each.
constexpr int FWD_MAX_THREADS = 512;
constexpr int BWD_MAX_THREADS = 640;   // 96 registers: two rows of 5120 16-bit channels at a time
constexpr int MAX_GROUPS = 16;

// Sums of two values over the T threads of a row's group.  `buf` alternates
// from call to call, so that one barrier suffices.
__device__ __forceinline__ void row_sums(float& a, float& b, int T, int group, float2 (*scratch)[BWD_MAX_THREADS / 32],
                                         int& buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (T == 32) return;
    if ((threadIdx.x & 31) == 0) scratch[buf][threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
    const int n = T >> 5, w0 = group * n;
    a = b = 0.0f;
    for (int w = 0; w < n; ++w) {
        const float2 t = scratch[buf][w0 + w];
        a += t.x;
        b += t.y;
    }
    buf ^= 1;
}

template <int DT, int VPT, bool AL>
__global__ void __launch_bounds__(FWD_MAX_THREADS, VPT == 2 ? 2 : 1) norm_fwd_kernel(const NormParams p, const int T)
{
    using V = Vec<DT>;
    constexpr int N = V::N;
    __shared__ float2 scratch[2][BWD_MAX_THREADS / 32];
    int buf = 0;
    const int group = threadIdx.x / T, tid = threadIdx.x - group * T, G = blockDim.x / T;
    const int64_t first = blockIdx.x * int64_t(G) + group, step = gridDim.x * int64_t(G);
    const int cols = static_cast<int>(p.cols);
    const uint8_t* x = static_cast<const uint8_t*>(p.x);
    const uint8_t* res = static_cast<const uint8_t*>(p.residual);
    const float inv = 1.0f / static_cast<float>(cols);
    pdl_wait();
    pdl_trigger();

    uint4 nx[VPT], nr[VPT];
    auto shift_of = [&](int64_t r) { return AL ? 0 : static_cast<int>((p.shift + r * p.ld_x) & (N - 1)); };
    auto fetch = [&](int64_t r) {
        const int sh = shift_of(r);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c0 = (tid + i * T) * N - sh;
            nx[i] = V::template load<AL>(x + r * p.ld_x * V::ES, c0, cols);
            if (res) nr[i] = V::template load<AL>(res + r * p.ld_r * V::ES, c0, cols);
        }
    };
    if (first < p.rows) fetch(first);
    for (int64_t r = first; r < p.rows; r += step) {
        const int sh = shift_of(r);
        float s[VPT][N];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            V::unpack(nx[i], s[i]);
            if (res) {
                float t[N];
                V::unpack(nr[i], t);
#pragma unroll
                for (int k = 0; k < N; ++k) s[i][k] += t[k];
            }
        }
        if (r + step < p.rows) fetch(r + step);
        float mean = 0.0f, dummy = 0.0f;
        if (!p.rms) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int k = 0; k < N; ++k) a += s[i][k];
            row_sums(a, dummy, T, group, scratch, buf);
            mean = a * inv;
        }
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c0 = (tid + i * T) * N - sh;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float d = s[i][k] - mean;
                if (AL ? c0 < cols : (c0 + k >= 0 && c0 + k < cols)) q = fmaf(d, d, q);
            }
        }
        row_sums(q, dummy, T, group, scratch, buf);
        const float rstd = 1.0f / sqrtf(fmaf(q, inv, p.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c0 = (tid + i * T) * N - sh;
            if (c0 >= cols) continue;
            float g[N], o[N];
            if (p.sum) V::template store<AL>(static_cast<uint8_t*>(p.sum) + r * p.ld_s * V::ES, c0, cols, s[i]);
            V::template weights<AL>(p.gamma, p.w_dt, p.w_vec, c0, cols, g);
#pragma unroll
            for (int k = 0; k < N; ++k) o[k] = (s[i][k] - mean) * rstd * g[k];
            if (p.beta) {
                V::template weights<AL>(p.beta, p.w_dt, p.w_vec, c0, cols, g);
#pragma unroll
                for (int k = 0; k < N; ++k) o[k] += g[k];
            }
            V::template store<AL>(static_cast<uint8_t*>(p.y) + r * p.ld_y * V::ES, c0, cols, o);
        }
        if (tid == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// One 16-byte piece into shared memory; the calling thread alone reads it,
// after cp_wait.
__device__ __forceinline__ void cp_async16(uint4* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Backward: dx of each row, and the CTA's share of dgamma and dbeta kept in
// registers over its rows (a CTA's rows have one shift: the grid is a
// multiple of a vector's elements, or every row has the same), then written
// as row blockIdx.x of the partial sums.
//
// Registers hold those sums (VPT vectors of two), so the rows in flight wait
// in shared memory instead: every thread copies its own vectors of the next
// BWD_STAGES - 1 rows there asynchronously and reads them back itself, without
// a barrier.
template <int VPT>
constexpr int BWD_STAGES = VPT == 2 ? 3 : 2;

template <int DT, int VPT, bool AL>
__global__ void __launch_bounds__(BWD_MAX_THREADS, 1) norm_bwd_kernel(const NormBwdParams p, const int T)
{
    using V = Vec<DT>;
    constexpr int N = V::N, S = BWD_STAGES<VPT>;
    __shared__ float2 scratch[2][BWD_MAX_THREADS / 32];
    extern __shared__ uint4 stage_s[];   // [S][dy, s, dsum][VPT][threads]; in the end G > 1: [2][cols] sums
    int buf = 0;
    const int group = threadIdx.x / T, tid = threadIdx.x - group * T, G = blockDim.x / T;
    const int64_t first = blockIdx.x + int64_t(gridDim.x) * group, step = gridDim.x * int64_t(G);
    const int cols = static_cast<int>(p.cols);
    const uint8_t* mats[3] = {static_cast<const uint8_t*>(p.dy), static_cast<const uint8_t*>(p.s),
                              static_cast<const uint8_t*>(p.dsum)};
    const int64_t lds[3] = {p.ld_dy, p.ld_s, p.ld_ds};
    const int n_mats = p.dsum ? 3 : 2;
    const float inv = 1.0f / static_cast<float>(cols);
    pdl_wait();
    pdl_trigger();

    const int sh = AL ? 0 : static_cast<int>((p.shift + first * p.ld_s) & (N - 1));
    auto slot = [&](int st, int m, int i) { return stage_s + ((st * n_mats + m) * VPT + i) * blockDim.x + threadIdx.x; };
    auto fetch = [&](int64_t r, int st) {
        if (r < p.rows) {
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                if (m == n_mats) break;
                const uint8_t* row = mats[m] + r * lds[m] * V::ES;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c0 = (tid + i * T) * N - sh;
                    if (c0 >= 0 && c0 + N <= cols)
                        cp_async16(slot(st, m, i), row + c0 * V::ES);
                    else
                        *slot(st, m, i) = V::template load<AL>(row, c0, cols);
                }
            }
        }
        cp_commit();
    };
    float dg[VPT][N], db[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) dg[i][k] = db[i][k] = 0.0f;
    float nmean = 0.0f, nrstd = 0.0f;
    if (first < p.rows) {
        if (!p.rms) nmean = __ldg(p.mean + first);
        nrstd = __ldg(p.rstd + first);
    }
#pragma unroll
    for (int j = 0; j < S - 1; ++j) fetch(first + j * step, j);
    int st = 0;
    for (int64_t r = first; r < p.rows; r += step) {
        const float mean = nmean, rstd = nrstd;
        fetch(r + (S - 1) * step, st == 0 ? S - 1 : st - 1);
        if (r + step < p.rows) {
            if (!p.rms) nmean = __ldg(p.mean + r + step);
            nrstd = __ldg(p.rstd + r + step);
        }
        cp_wait<S - 1>();
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c0 = (tid + i * T) * N - sh;
            float g[N], d[N], xh[N];
            V::template weights<AL>(p.gamma, p.w_dt, p.w_vec, c0, cols, g);
            V::unpack(*slot(st, 0, i), d);
            V::unpack(*slot(st, 1, i), xh);
#pragma unroll
            for (int k = 0; k < N; ++k) {   // (past the row's ends dy and gamma are 0)
                xh[k] = (xh[k] - mean) * rstd;
                dg[i][k] = fmaf(d[k], xh[k], dg[i][k]);
                db[i][k] += d[k];
                const float t = d[k] * g[k];
                a += t;
                b = fmaf(t, xh[k], b);
            }
        }
        row_sums(a, b, T, group, scratch, buf);
        const float mt = p.rms ? 0.0f : a * inv, mtx = b * inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c0 = (tid + i * T) * N - sh;
            if (c0 >= cols) continue;
            float g[N], d[N], xh[N];
            V::template weights<AL>(p.gamma, p.w_dt, p.w_vec, c0, cols, g);
            V::unpack(*slot(st, 0, i), d);
            V::unpack(*slot(st, 1, i), xh);
#pragma unroll
            for (int k = 0; k < N; ++k) d[k] = fmaf(-((xh[k] - mean) * rstd), mtx, d[k] * g[k] - mt) * rstd;
            if (n_mats == 3) {
                V::unpack(*slot(st, 2, i), xh);
#pragma unroll
                for (int k = 0; k < N; ++k) d[k] += xh[k];
            }
            V::template store<AL>(static_cast<uint8_t*>(p.dx) + r * p.ld_dx * V::ES, c0, cols, d);
        }
        st = st == S - 1 ? 0 : st + 1;
    }
    cp_wait<0>();
    float* acc_s = reinterpret_cast<float*>(stage_s);
    __syncthreads();   // every row has been read
    float* part = p.part + 2LL * blockIdx.x * cols;
    if (G > 1) {
        for (int w = 0; w < G; ++w) {
            if (group == w) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const int c = (tid + i * T) * N - sh + k;
                        if (c >= 0 && c < cols) {
                            acc_s[c] = (w ? acc_s[c] : 0.0f) + dg[i][k];
                            acc_s[cols + c] = (w ? acc_s[cols + c] : 0.0f) + db[i][k];
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) part[c] = acc_s[c];
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int c = (tid + i * T) * N - sh + k;
                if (c >= 0 && c < cols) {
                    part[c] = dg[i][k];
                    part[cols + c] = db[i][k];
                }
            }
    }
}

// Threads per row, vectors per thread and rows at a time for rows of nv
// vectors (the first and last of a shifted row included).
struct RowPlan {
    int vpt, T, G;
};

inline bool row_plan(int64_t nv, int max_threads, RowPlan* q)
{
    q->vpt = nv <= 1024 ? 2 : 4;
    const int64_t T = ((nv + q->vpt - 1) / q->vpt + 31) / 32 * 32;
    if (T > 512) return false;
    q->T = static_cast<int>(T);
    q->G = max_threads / q->T > 1 ? max_threads / q->T : 1;
    if (q->G > MAX_GROUPS) q->G = MAX_GROUPS;
    if (q->T > 32 && q->G > 8) q->G = 8;   // one named barrier each
    return true;
}

template <int DT, int VPT, bool AL>
cudaError_t launch_norm_fwd_1(const NormParams& p, const RowPlan& q, int sms, cudaStream_t stream)
{
    const int threads = q.T * q.G;
    const int64_t units = (p.rows + q.G - 1) / q.G, most = static_cast<int64_t>(sms) * (1024 / threads);
    return launch_pdl(norm_fwd_kernel<DT, VPT, AL>, dim3(static_cast<unsigned>(units < most ? units : most)),
                      dim3(threads), 0, stream, p, q.T);
}

template <int DT, int VPT, bool AL>
cudaError_t launch_norm_bwd_1(const NormBwdParams& p, const RowPlan& q, cudaStream_t stream)
{
    // the ring of rows holds the sums of both vectors afterwards: two floats for each element of a row's slots
    const int smem = BWD_STAGES<VPT> * (p.dsum ? 3 : 2) * VPT * 16 * q.T * q.G;
    static std::atomic<unsigned> done{0};
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(norm_bwd_kernel<DT, VPT, AL>), smem, &done);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_bwd_kernel<DT, VPT, AL>, dim3(p.parts), dim3(q.T * q.G), smem, stream, p, q.T);
}

// f.run<DT, VPT, AL>() of the form that the call needs.
template <int DT, typename P, typename F>
cudaError_t pick_row_kernel(const P& p, const RowPlan& q, F&& f)
{
    if (q.vpt == 2) return p.aligned ? f.template run<DT, 2, true>() : f.template run<DT, 2, false>();
    return p.aligned ? f.template run<DT, 4, true>() : f.template run<DT, 4, false>();
}

struct RunFwd {
    const NormParams& p;
    const RowPlan& q;
    int sms;
    cudaStream_t s;
    template <int DT, int VPT, bool AL>
    cudaError_t run() const { return launch_norm_fwd_1<DT, VPT, AL>(p, q, sms, s); }
};

struct RunBwd {
    const NormBwdParams& p;
    const RowPlan& q;
    cudaStream_t s;
    template <int DT, int VPT, bool AL>
    cudaError_t run() const { return launch_norm_bwd_1<DT, VPT, AL>(p, q, s); }
};

}  // namespace qta
