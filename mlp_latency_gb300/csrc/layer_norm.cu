// layer_norm.cu -- layer norm, forward and backward (C ABI in include/mlp_block.h).
//
// Per row of C columns: mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps),
// xh = (x - mean) rstd, y = xh gamma + beta.  Backward, with g = dy gamma:
// dx = rstd (g - mean(g) - xh mean(g xh)), dgamma = sum_rows dy xh, dbeta = sum_rows dy.
// A handful of operations per element: the memory system is the bound, so every kernel reads its rows
// once, in the widest loads that the addresses allow, and keeps them in registers between the passes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mlp_block.h"

namespace {

constexpr int kMaxThreads = 1024;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&f)[V])
{
    const Vec<T, V> x = *reinterpret_cast<const Vec<T, V> *>(p);
#pragma unroll
    for (int j = 0; j < V; ++j)
        f[j] = to_f32<T>(x.v[j]);
}

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V])
{
    Vec<T, V> x;
#pragma unroll
    for (int j = 0; j < V; ++j)
        x.v[j] = from_f32<T>(f[j]);
    *reinterpret_cast<Vec<T, V> *>(p) = x;
}

// gamma or beta, columns c .. c + V - 1 (NULL: `none`).  kind: 0 bf16, 1 fp32; + 2: aligned to V of them
// (at most 16 bytes), read in vectors.
template <int V>
__device__ __forceinline__ void load_w(const void *w, int kind, int64_t c, float none, float (&f)[V])
{
    constexpr int V4 = V < 4 ? V : 4;
    if (!w) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            f[j] = none;
    } else if (kind == 2) {
        load<__nv_bfloat16, V>(static_cast<const __nv_bfloat16 *>(w) + c, f);
    } else if (kind == 3) {
#pragma unroll
        for (int j = 0; j < V; j += V4) {
            const Vec<float, V4> x = *reinterpret_cast<const Vec<float, V4> *>(static_cast<const float *>(w) + c + j);
#pragma unroll
            for (int k = 0; k < V4; ++k)
                f[j + k] = x.v[k];
        }
    } else if (kind == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            f[j] = static_cast<const float *>(w)[c + j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            f[j] = __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c + j]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N values over the threads of a row's team (a warp, or the whole block), in a fixed order.
template <int N, bool kWarpTeam>
__device__ __forceinline__ void team_sum(float (&v)[N], float *scratch)
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = warp_sum(v[n]);
    if (kWarpTeam)
        return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, warps = (blockDim.x + 31) / 32;
    __syncthreads();   // the scratch may still be read from the sum before
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; ++n)
            scratch[n * 32 + warp] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = warp_sum(lane < warps ? scratch[n * 32 + lane] : 0.0f);
}

struct NormParams {
    const void *x, *dy, *add;
    void *y, *dx;
    const void *gamma, *beta;
    float *mean, *rstd;            // outputs (forward), inputs (backward)
    const float *mean_in, *rstd_in;
    int64_t rows, cols, ldx, ldy, lddy, ldadd, lddx;
    float eps, inv_cols;
    int32_t w_f32, w_kind;         // dtype of the weights; how load_w reads them
    float *part;                   // column sums: blocks x 2 x cols
    int64_t block_rows;
    int32_t blocks;
};

// One row per team, the row in registers (kItems vectors of V per thread): moments, then the output.
template <typename T, int V, int kItems, bool kWarpTeam, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormParams p)
{
    __shared__ float scratch[32];
    const int team = kWarpTeam ? 32 : static_cast<int>(blockDim.x);
    const int t = kWarpTeam ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t row = kWarpTeam ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (row >= p.rows)
        return;   // a whole team leaves (warp teams share no barrier)
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    float v[kItems][V];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * team + t) * V;
        if (c < p.cols) {
            load<T, V>(x + c, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j)
                s[0] += v[i][j];
        }
    }
    team_sum<1, kWarpTeam>(s, scratch);
    const float mean = s[0] / static_cast<float>(p.cols);   // (a division: a constant row gives exact zeros)
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * team + t) * V;
        if (c < p.cols)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[i][j] - mean;
                s[0] = fmaf(d, d, s[0]);
            }
    }
    team_sum<1, kWarpTeam>(s, scratch);
    const float rstd = rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
    if (t == 0) {
        if (p.mean)
            p.mean[row] = mean;
        if (p.rstd)
            p.rstd[row] = rstd;
    }
    T *y = static_cast<T *>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * team + t) * V;
        if (c < p.cols) {
            float g[V], b[V], o[V];
            load_w<V>(p.gamma, p.w_kind, c, 1.0f, g);
            load_w<V>(p.beta, p.w_kind, c, 0.0f, b);
#pragma unroll
            for (int j = 0; j < V; ++j)
                o[j] = fmaf((v[i][j] - mean) * rstd, g[j], b[j]);
            store<T, V>(y + c, o);
        }
    }
}

// Rows too wide for registers: three passes over the row (the later ones come from L2).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_wide_kernel(const NormParams p)
{
    __shared__ float scratch[32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x)
        s[0] += to_f32<T>(x[c]);
    team_sum<1, false>(s, scratch);
    const float mean = s[0] / static_cast<float>(p.cols);   // (a division: a constant row gives exact zeros)
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
        const float d = to_f32<T>(x[c]) - mean;
        s[0] = fmaf(d, d, s[0]);
    }
    team_sum<1, false>(s, scratch);
    const float rstd = rsqrtf(fmaf(s[0], p.inv_cols, p.eps));
    if (threadIdx.x == 0) {
        if (p.mean)
            p.mean[row] = mean;
        if (p.rstd)
            p.rstd[row] = rstd;
    }
    T *y = static_cast<T *>(p.y) + row * p.ldy;
    for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float g[1], b[1];
        load_w<1>(p.gamma, p.w_kind, c, 1.0f, g);
        load_w<1>(p.beta, p.w_kind, c, 0.0f, b);
        y[c] = from_f32<T>(fmaf((to_f32<T>(x[c]) - mean) * rstd, g[0], b[0]));
    }
}

// dx of one row per block: two sums over the row, then the output; the row is read twice (the second
// time from L1 or L2), so any width fits.
template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_dx_kernel(const NormParams p)
{
    __shared__ float scratch[64];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
    const T *add = p.add ? static_cast<const T *>(p.add) + row * p.ldadd : nullptr;
    T *dx = static_cast<T *>(p.dx) + row * p.lddx;
    const float mean = p.mean_in[row], rstd = p.rstd_in[row];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < p.cols; c += static_cast<int64_t>(blockDim.x) * V) {
        float a[V], d[V], g[V];
        load<T, V>(x + c, a);
        load<T, V>(dy + c, d);
        load_w<V>(p.gamma, p.w_kind, c, 1.0f, g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float gd = g[j] * d[j];
            s[0] += gd;
            s[1] = fmaf(gd, (a[j] - mean) * rstd, s[1]);
        }
    }
    team_sum<2, false>(s, scratch);
    const float m0 = s[0] * p.inv_cols, m1 = s[1] * p.inv_cols;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < p.cols; c += static_cast<int64_t>(blockDim.x) * V) {
        float a[V], d[V], g[V], o[V];
        load<T, V>(x + c, a);
        load<T, V>(dy + c, d);
        load_w<V>(p.gamma, p.w_kind, c, 1.0f, g);
#pragma unroll
        for (int j = 0; j < V; ++j)
            o[j] = rstd * (fmaf(g[j], d[j], -m0) - (a[j] - mean) * rstd * m1);
        if (add) {
            float r[V];
            load<T, V>(add + c, r);
#pragma unroll
            for (int j = 0; j < V; ++j)
                o[j] += r[j];
        }
        store<T, V>(dx + c, o);
    }
}

// Column sums of dy xh and dy over one block of rows: 32 lanes x V columns, 8 warps over the rows.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_colsum_kernel(const NormParams p)
{
    __shared__ float red[2][8][32 * V];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V;
    const int64_t lo = static_cast<int64_t>(blockIdx.y) * p.block_rows, hi = min(lo + p.block_rows, p.rows);
    float sg[V], sb[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        sg[j] = sb[j] = 0.0f;
    if (c < p.cols) {
#pragma unroll 4
        for (int64_t r = lo + warp; r < hi; r += 8) {
            float a[V], d[V];
            load<T, V>(static_cast<const T *>(p.x) + r * p.ldx + c, a);
            load<T, V>(static_cast<const T *>(p.dy) + r * p.lddy + c, d);
            const float mean = p.mean_in[r], rstd = p.rstd_in[r];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sb[j] += d[j];
                sg[j] = fmaf(d[j], (a[j] - mean) * rstd, sg[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        red[0][warp][lane * V + j] = sg[j];
        red[1][warp][lane * V + j] = sb[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * 32 * V; i += 256) {
        const int w = i / (32 * V), k = i % (32 * V);
        const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * V + k;
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s += red[w][q][k];
        if (col < p.cols)
            p.part[(static_cast<int64_t>(blockIdx.y) * 2 + w) * p.cols + col] = s;
    }
}

// dgamma and dbeta: the partial rows in block order.  32 columns per block, 8 interleaved row sets.
__global__ void __launch_bounds__(256) norm_colsum_finish_kernel(const NormParams p, void *dgamma, void *dbeta)
{
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, set = threadIdx.x / 32;
    const int w = blockIdx.y;
    void *out = w ? dbeta : dgamma;
    if (!out)
        return;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < p.cols)
#pragma unroll 4
        for (int b = set; b < p.blocks; b += 8)
            s += p.part[(static_cast<int64_t>(b) * 2 + w) * p.cols + c];
    red[set][lane] = s;
    __syncthreads();
    if (set == 0 && c < p.cols) {
        s = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s += red[q][lane];
        if (p.w_f32)
            static_cast<float *>(out)[c] = s;
        else
            static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kColsumBlocks = 64;   // row blocks of the column sums, at most

bool aligned(const void *p, int64_t ld, size_t esz, size_t bytes)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && static_cast<size_t>(ld) * esz % bytes == 0);
}

bool bad_dtype(mlp_dtype d) { return d != MLP_DT_BF16 && d != MLP_DT_F32; }

bool bad_rows(const void *p, int64_t ld, int64_t cols, size_t esz)
{
    return !p || reinterpret_cast<uintptr_t>(p) % esz != 0 || ld < cols;
}

template <typename T, int V, int kItems, int kThreads>
void launch_forward(const NormParams &p, int64_t nvec, cudaStream_t st)
{
    if (nvec <= 32 * kItems) {
        const int teams = 4;
        norm_forward_kernel<T, V, kItems, true, 128><<<static_cast<unsigned>(cdiv(p.rows, teams)), 32 * teams, 0, st>>>(p);
    } else {
        const int threads = static_cast<int>(cdiv(cdiv(nvec, kItems), 32) * 32);
        norm_forward_kernel<T, V, kItems, false, kThreads><<<static_cast<unsigned>(p.rows), threads, 0, st>>>(p);
    }
}

// Vectors per thread.  Few rows: one, so that a row's loads go out at once from as many threads as there
// are.  Many rows: four, so that several rows share an SM and one row's reductions hide behind the others'
// loads.  Wider rows take what fits a block's registers.
template <typename T, int V>
void forward_v(const NormParams &p, cudaStream_t st)
{
    const int64_t nvec = cdiv(p.cols, V);
    const bool many = p.rows > 304;
    if (nvec <= (many ? 64 : 1024))
        launch_forward<T, V, 1, 1024>(p, nvec, st);
    else if (nvec <= 4 * 256)
        launch_forward<T, V, 4, 256>(p, nvec, st);
    else if (nvec <= 4 * 512)
        launch_forward<T, V, 4, 512>(p, nvec, st);
    else if (nvec <= 4 * 1024)
        launch_forward<T, V, 4, 1024>(p, nvec, st);
    else if (V <= 2 && nvec <= 16 * 1024)
        launch_forward<T, V, V <= 2 ? 16 : 1, 1024>(p, nvec, st);
    else
        norm_forward_wide_kernel<T><<<static_cast<unsigned>(p.rows), kMaxThreads, 0, st>>>(p);
}

template <typename T, int V>
void backward_v(const NormParams &p, bool want_w, cudaStream_t st)
{
    if (p.dx) {
        const int threads = static_cast<int>(std::min<int64_t>(cdiv(cdiv(p.cols, V), 32) * 32, kMaxThreads));
        norm_dx_kernel<T, V><<<static_cast<unsigned>(p.rows), threads, 0, st>>>(p);
    }
    if (want_w)
        norm_colsum_kernel<T, V><<<dim3(static_cast<unsigned>(cdiv(p.cols, 32 * V)), static_cast<unsigned>(p.blocks)), 256, 0, st>>>(p);
}

}  // namespace

extern "C" mlp_status mlp_layernorm_forward(int64_t rows, int64_t cols, const void *x, int64_t ldx, mlp_dtype dtype,
                                            const void *gamma, const void *beta, mlp_dtype w_dtype, float eps, void *y,
                                            int64_t ldy, float *mean, float *rstd, void *stream)
{
    if (rows < 0 || rows >= (int64_t{1} << 31) || cols < 1 || cols >= (int64_t{1} << 31) || !(eps >= 0.0f))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype) || bad_dtype(w_dtype))
        return MLP_ERR_UNSUPPORTED;
    if (rows == 0)
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4, wsz = w_dtype == MLP_DT_BF16 ? 2 : 4;
    if (bad_rows(x, ldx, cols, esz) || bad_rows(y, ldy, cols, esz) || !aligned(gamma, 0, wsz, wsz) ||
        !aligned(beta, 0, wsz, wsz) || !aligned(mean, 0, 4, 4) || !aligned(rstd, 0, 4, 4))
        return MLP_ERR_INVALID_ARG;
    NormParams p = {};
    p.x = x;
    p.y = y;
    p.gamma = gamma;
    p.beta = beta;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.ldy = ldy;
    p.eps = eps;
    p.inv_cols = 1.0f / static_cast<float>(cols);
    p.w_f32 = w_dtype == MLP_DT_F32;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.w_kind = p.w_f32 + (aligned(gamma, 0, wsz, 16) && aligned(beta, 0, wsz, 16) ? 2 : 0);
    auto wide = [&](size_t bytes) {
        return static_cast<size_t>(cols) * esz % bytes == 0 && aligned(x, ldx, esz, bytes) && aligned(y, ldy, esz, bytes);
    };
    if (dtype == MLP_DT_BF16) {
        if (wide(16))
            forward_v<__nv_bfloat16, 8>(p, st);
        else if (wide(4))
            forward_v<__nv_bfloat16, 2>(p, st);
        else
            forward_v<__nv_bfloat16, 1>(p, st);
    } else if (wide(16)) {
        forward_v<float, 4>(p, st);
    } else {
        forward_v<float, 1>(p, st);
    }
    return cudaGetLastError() == cudaSuccess ? MLP_OK : MLP_ERR_CUDA;
}

extern "C" mlp_status mlp_layernorm_workspace_size(int64_t rows, int64_t cols, size_t *bytes)
{
    if (rows < 0 || cols < 1 || !bytes)
        return MLP_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(kColsumBlocks) * 2 * static_cast<size_t>(cols) * 4;
    return MLP_OK;
}

extern "C" mlp_status mlp_layernorm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *x,
                                             int64_t ldx, mlp_dtype dtype, const void *gamma, mlp_dtype w_dtype,
                                             const float *mean, const float *rstd, const void *dx_add, int64_t ldadd,
                                             void *dx, int64_t lddx, void *dgamma, void *dbeta, void *workspace,
                                             void *stream)
{
    if (rows < 0 || rows >= (int64_t{1} << 31) || cols < 1 || cols >= (int64_t{1} << 31))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype) || bad_dtype(w_dtype))
        return MLP_ERR_UNSUPPORTED;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4, wsz = w_dtype == MLP_DT_BF16 ? 2 : 4;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!aligned(dgamma, 0, wsz, wsz) || !aligned(dbeta, 0, wsz, wsz) || !aligned(gamma, 0, wsz, wsz))
        return MLP_ERR_INVALID_ARG;
    const bool want_w = dgamma || dbeta;
    if (rows == 0) {
        if ((dgamma && cudaMemsetAsync(dgamma, 0, static_cast<size_t>(cols) * wsz, st) != cudaSuccess) ||
            (dbeta && cudaMemsetAsync(dbeta, 0, static_cast<size_t>(cols) * wsz, st) != cudaSuccess))
            return MLP_ERR_CUDA;
        return MLP_OK;
    }
    if (bad_rows(dy, lddy, cols, esz) || bad_rows(x, ldx, cols, esz) || (dx && bad_rows(dx, lddx, cols, esz)) ||
        (dx_add && bad_rows(dx_add, ldadd, cols, esz)) || !mean || !rstd || !aligned(mean, 0, 4, 4) ||
        !aligned(rstd, 0, 4, 4) || (want_w && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)))
        return MLP_ERR_INVALID_ARG;
    NormParams p = {};
    p.x = x;
    p.dy = dy;
    p.add = dx_add;
    p.dx = dx;
    p.gamma = gamma;
    p.mean_in = mean;
    p.rstd_in = rstd;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.lddy = lddy;
    p.ldadd = ldadd;
    p.lddx = lddx;
    p.inv_cols = 1.0f / static_cast<float>(cols);
    p.w_f32 = w_dtype == MLP_DT_F32;
    p.w_kind = p.w_f32 + (aligned(gamma, 0, wsz, 16) ? 2 : 0);
    p.part = static_cast<float *>(workspace);
    p.block_rows = std::max<int64_t>(cdiv(rows, kColsumBlocks), 8);
    p.blocks = static_cast<int32_t>(cdiv(rows, p.block_rows));
    // The column sums read dy and x, which dx may overwrite: they go first.
    NormParams sums = p;
    sums.dx = nullptr;
    auto wide = [&](size_t bytes) {
        return static_cast<size_t>(cols) * esz % bytes == 0 && aligned(x, ldx, esz, bytes) && aligned(dy, lddy, esz, bytes) &&
               aligned(dx, lddx, esz, bytes) && aligned(dx_add, ldadd, esz, bytes);
    };
    auto run = [&](auto vec) {
        vec(sums, want_w);
        vec(p, false);
    };
    if (dtype == MLP_DT_BF16) {
        if (wide(16))
            run([&](const NormParams &q, bool w) { backward_v<__nv_bfloat16, 8>(q, w, st); });
        else if (wide(4))
            run([&](const NormParams &q, bool w) { backward_v<__nv_bfloat16, 2>(q, w, st); });
        else
            run([&](const NormParams &q, bool w) { backward_v<__nv_bfloat16, 1>(q, w, st); });
    } else if (wide(16)) {
        run([&](const NormParams &q, bool w) { backward_v<float, 4>(q, w, st); });
    } else {
        run([&](const NormParams &q, bool w) { backward_v<float, 1>(q, w, st); });
    }
    if (want_w)
        norm_colsum_finish_kernel<<<dim3(static_cast<unsigned>(cdiv(cols, 32)), 2), 256, 0, st>>>(p, dgamma, dbeta);
    return cudaGetLastError() == cudaSuccess ? MLP_OK : MLP_ERR_CUDA;
}
