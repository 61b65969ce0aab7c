// qta_norm.cu -- norm kernels and launchers of the layer operators.
#include "qta_norm_rows.cuh"

namespace qta {

constexpr int ROW_THREADS = 256;

// Sum over a CTA of ROW_THREADS threads, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();   // the scratch of an earlier sum has been read
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < ROW_THREADS / 32; ++w) v += scratch[w];
    return v;
}

// One CTA per row, three passes over it: the mean, the sum of squares about
// it, the output.
__global__ void __launch_bounds__(ROW_THREADS) norm_rows_kernel(const NormParams p)
{
    __shared__ float scratch[ROW_THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        auto value = [&](int64_t c) {
            float v = load_elem(p.x, r * p.ld_x + c, p.dt);
            if (p.residual) v += load_elem(p.residual, r * p.ld_r + c, p.dt);
            return v;
        };
        float mean = 0.0f;
        if (!p.rms) {
            float a = 0.0f;
            for (int64_t c = threadIdx.x; c < p.cols; c += ROW_THREADS) a += value(c);
            mean = block_sum(a, scratch) * inv;
        }
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += ROW_THREADS) {
            const float d = value(c) - mean;
            q = fmaf(d, d, q);
        }
        const float rstd = 1.0f / sqrtf(fmaf(block_sum(q, scratch), inv, p.eps));
        for (int64_t c = threadIdx.x; c < p.cols; c += ROW_THREADS) {
            const float v = value(c);
            float o = (v - mean) * rstd * load_elem(p.gamma, c, p.w_dt);
            if (p.beta) o += load_elem(p.beta, c, p.w_dt);
            store_elem(p.y, r * p.ld_y + c, p.dt, o);
            if (p.sum) store_elem(p.sum, r * p.ld_s + c, p.dt, v);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// dx of one row per CTA: two passes (the row means <t> and <t xh>, the output).
__global__ void __launch_bounds__(ROW_THREADS) norm_bwd_rows_kernel(const NormBwdParams p)
{
    __shared__ float scratch[ROW_THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const float mean = p.rms ? 0.0f : p.mean[r], rstd = p.rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += ROW_THREADS) {
            const float t = load_elem(p.dy, r * p.ld_dy + c, p.dt) * load_elem(p.gamma, c, p.w_dt);
            const float xh = (load_elem(p.s, r * p.ld_s + c, p.dt) - mean) * rstd;
            a += t;
            b = fmaf(t, xh, b);
        }
        const float mt = p.rms ? 0.0f : block_sum(a, scratch) * inv;
        const float mtx = block_sum(b, scratch) * inv;
        for (int64_t c = threadIdx.x; c < p.cols; c += ROW_THREADS) {
            const float t = load_elem(p.dy, r * p.ld_dy + c, p.dt) * load_elem(p.gamma, c, p.w_dt);
            const float xh = (load_elem(p.s, r * p.ld_s + c, p.dt) - mean) * rstd;
            float d = fmaf(-xh, mtx, t - mt) * rstd;
            if (p.dsum) d += load_elem(p.dsum, r * p.ld_ds + c, p.dt);
            store_elem(p.dx, r * p.ld_dx + c, p.dt, d);
        }
    }
}

// Partial column sums of dy xh and dy: CTA (x, y) sums rows y, y + parts, ...
// of 256 columns.
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const NormBwdParams p)
{
    pdl_wait();
    pdl_trigger();
    const int64_t c = blockIdx.x * 256LL + threadIdx.x;
    if (c >= p.cols) return;
    float g = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < p.rows; r += p.parts) {
        const float mean = p.rms ? 0.0f : p.mean[r];
        const float dy = load_elem(p.dy, r * p.ld_dy + c, p.dt);
        g = fmaf(dy, (load_elem(p.s, r * p.ld_s + c, p.dt) - mean) * p.rstd[r], g);
        b += dy;
    }
    p.part[(2LL * blockIdx.y) * p.cols + c] = g;
    p.part[(2LL * blockIdx.y + 1) * p.cols + c] = b;
}

// Partial column sums of a matrix: CTA (x, y) sums rows y, y + parts, ...
__global__ void __launch_bounds__(256) col_sum_kernel(const void* a, int64_t ld, int dt, int64_t rows, int64_t cols,
                                                      int parts, float* part)
{
    pdl_wait();
    pdl_trigger();
    const int64_t c = blockIdx.x * 256LL + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += parts) s += load_elem(a, r * ld + c, dt);
    part[static_cast<int64_t>(blockIdx.y) * cols + c] = s;
}

// out0[c] = sum over i < parts of part[i * stride + c], out1 the same one
// block of `cols` further: the partial sums in a fixed order (warp w of 16
// adds the rows w, w + 16, ..., then the warps in turn).
constexpr int FINISH_WARPS = 16;
__global__ void __launch_bounds__(32 * FINISH_WARPS) col_finish_kernel(const float* part, int64_t stride, int parts,
                                                                       int64_t cols, float* out0, float* out1)
{
    __shared__ float sums[FINISH_WARPS][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32LL + lane;
    float* out = blockIdx.y ? out1 : out0;
    const float* p = part + blockIdx.y * cols + c;
    float s = 0.0f;
    if (c < cols && out) {
#pragma unroll 4
        for (int i = warp; i < parts; i += FINISH_WARPS) s += p[i * stride];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols && out) {
#pragma unroll
        for (int w = 1; w < FINISH_WARPS; ++w) s += sums[w][lane];
        out[c] = s;
    }
}

cudaError_t launch_norm_rows_bf16(const NormParams&, const RowPlan&, int, cudaStream_t);
cudaError_t launch_norm_rows_fp16(const NormParams&, const RowPlan&, int, cudaStream_t);
cudaError_t launch_norm_rows_fp32(const NormParams&, const RowPlan&, int, cudaStream_t);
cudaError_t launch_norm_bwd_rows_bf16(const NormBwdParams&, const RowPlan&, cudaStream_t);
cudaError_t launch_norm_bwd_rows_fp16(const NormBwdParams&, const RowPlan&, cudaStream_t);
cudaError_t launch_norm_bwd_rows_fp32(const NormBwdParams&, const RowPlan&, cudaStream_t);

// Whether the row kernels take matrices whose rows start at these addresses
// (n of them, NULL: absent), and the vectors of a row.
static bool row_form(const void* const* base, const int64_t* ld, int n, int64_t rows, int64_t cols, int dt,
                     int sms, int max_threads, int short_T, int* shift, int* aligned, RowPlan* q)
{
    const int es = dt_size(dt), N = 16 / es;
    bool all = true;
    *shift = static_cast<int>((reinterpret_cast<uintptr_t>(base[0]) / es) % N);
    for (int i = 0; i < n; ++i) {
        if (!base[i]) continue;
        if (static_cast<int>((reinterpret_cast<uintptr_t>(base[i]) / es) % N) != *shift || (ld[i] - ld[0]) % N)
            return false;
        all = all && ld[i] % N == 0;
    }
    *aligned = all && *shift == 0 && cols % N == 0;
    if (cols > (1 << 20)) return false;
    return row_plan(*aligned ? cols / N : (cols + N - 1) / N + 1, rows, sms, max_threads, short_T, q);
}

static bool vec16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

cudaError_t launch_norm(const NormParams& in, int sms, cudaStream_t stream)
{
    NormParams p = in;
    p.w_vec = vec16(p.gamma) && vec16(p.beta);
    const void* base[4] = {p.x, p.residual, p.y, p.sum};
    const int64_t ld[4] = {p.ld_x, p.ld_r, p.ld_y, p.ld_s};
    RowPlan q;
    if (row_form(base, ld, 4, p.rows, p.cols, p.dt, sms, FWD_MAX_THREADS, 512, &p.shift, &p.aligned, &q)) {
        if (p.dt == 0) return launch_norm_rows_bf16(p, q, sms, stream);
        if (p.dt == 1) return launch_norm_rows_fp16(p, q, sms, stream);
        return launch_norm_rows_fp32(p, q, sms, stream);
    }
    const int64_t most = 16LL * sms;
    return launch_pdl(norm_rows_kernel, dim3(static_cast<unsigned>(p.rows < most ? p.rows : most)), dim3(ROW_THREADS),
                      0, stream, p);
}

cudaError_t launch_norm_bwd(const NormBwdParams& in, int sms, cudaStream_t stream)
{
    NormBwdParams p = in;
    p.w_vec = vec16(p.gamma);
    const void* base[4] = {p.s, p.dy, p.dsum, p.dx};
    const int64_t ld[4] = {p.ld_s, p.ld_dy, p.ld_ds, p.ld_dx};
    RowPlan q;
    cudaError_t e;
    const unsigned nf = static_cast<unsigned>((p.cols + 31) / 32);
    if (row_form(base, ld, 4, p.rows, p.cols, p.dt, sms, BWD_MAX_THREADS, 384, &p.shift, &p.aligned, &q)) {
        // CTAs: what fits on the GPU, or the rows; a multiple of 8 where the rows' shifts differ
        int64_t parts = (p.rows + q.G - 1) / q.G;
        if (parts > sms) parts = sms;
        if (parts > MAX_PARTS) parts = MAX_PARTS;
        if (!p.aligned) parts = parts < 8 ? 8 : parts / 8 * 8;
        p.parts = static_cast<int>(parts);
        if (p.dt == 0)
            e = launch_norm_bwd_rows_bf16(p, q, stream);
        else if (p.dt == 1)
            e = launch_norm_bwd_rows_fp16(p, q, stream);
        else
            e = launch_norm_bwd_rows_fp32(p, q, stream);
        if (e != cudaSuccess) return e;
        return launch_pdl(col_finish_kernel, dim3(nf, p.dbeta ? 2 : 1), dim3(32 * FINISH_WARPS), 0, stream,
                          static_cast<const float*>(p.part), 2 * p.cols, p.parts, p.cols, p.dgamma, p.dbeta);
    }
    const int64_t most = 16LL * sms;
    const unsigned nc = static_cast<unsigned>((p.cols + 255) / 256);
    e = launch_pdl(norm_bwd_rows_kernel, dim3(static_cast<unsigned>(p.rows < most ? p.rows : most)),
                               dim3(ROW_THREADS), 0, stream, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(norm_bwd_cols_kernel, dim3(nc, p.parts), dim3(256), 0, stream, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(col_finish_kernel, dim3(nf, 2), dim3(32 * FINISH_WARPS), 0, stream,
                      static_cast<const float*>(p.part), 2 * p.cols, p.parts, p.cols, p.dgamma, p.dbeta);
}

cudaError_t launch_col_sum(const void* a, int64_t ld, int dt, int64_t rows, int64_t cols, int parts, float* part,
                           cudaStream_t stream)
{
    return launch_pdl(col_sum_kernel, dim3(static_cast<unsigned>((cols + 255) / 256), parts), dim3(256), 0, stream, a,
                      ld, dt, rows, cols, parts, part);
}

cudaError_t launch_col_finish(const float* part, int64_t stride, int parts, int64_t cols, float* out,
                              cudaStream_t stream)
{
    return launch_pdl(col_finish_kernel, dim3(static_cast<unsigned>((cols + 31) / 32), 1), dim3(32 * FINISH_WARPS), 0,
                      stream, part, stride, parts, cols, out, static_cast<float*>(nullptr));
}

}  // namespace qta
