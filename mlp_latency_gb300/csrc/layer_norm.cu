// layer_norm.cu -- layer norm, forward and backward (C ABI in include/mlp_block.h).
//
// Per row of C columns: mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps),
// xh = (x - mean) rstd, y = xh gamma + beta.  Backward, with g = dy gamma:
// dx = rstd (g - mean(g) - xh mean(g xh)), dgamma = sum_rows dy xh, dbeta = sum_rows dy.
// A handful of operations per element: the memory system is the bound, so rows that fit registers or shared memory are read
// once, in the widest loads that the addresses allow, and kept there between the passes.  Wider ones, and gradients of
// arrays whose rows start at different places, are read again for each pass.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mlp_block.h"
#include "cuda_call.h"

using mlpc::succeeded;

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

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// V elements at an address aligned to V of them (at most 16 bytes) as they are in memory.  Loads keep this form until
// the values are used: a conversion next to the load would wait for memory before the next load goes out.
template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> { using type = unsigned short; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };
template <typename T, int V>
using Raw = typename RawOf<static_cast<int>(sizeof(T)) * V>::type;

template <typename T>
__device__ __forceinline__ void unpack(unsigned short x, float (&f)[1]) { f[0] = bf16_lo(x); }
template <typename T>
__device__ __forceinline__ void unpack(uint32_t x, float (&f)[1]) { f[0] = __uint_as_float(x); }
template <typename T>
__device__ __forceinline__ void unpack(uint32_t x, float (&f)[2])
{
    f[0] = bf16_lo(x);
    f[1] = bf16_hi(x);
}
template <typename T>
__device__ __forceinline__ void unpack(uint2 x, float (&f)[2])
{
    f[0] = __uint_as_float(x.x);
    f[1] = __uint_as_float(x.y);
}
template <typename T>
__device__ __forceinline__ void unpack(uint2 x, float (&f)[4])
{
    f[0] = bf16_lo(x.x);
    f[1] = bf16_hi(x.x);
    f[2] = bf16_lo(x.y);
    f[3] = bf16_hi(x.y);
}
template <typename T>
__device__ __forceinline__ void unpack(uint4 x, float (&f)[4])
{
    f[0] = __uint_as_float(x.x);
    f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z);
    f[3] = __uint_as_float(x.w);
}
template <typename T>
__device__ __forceinline__ void unpack(uint4 x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
    }
}

// Vectors at columns c, c + step, ... below cols.  (I: int where the width is known to fit.)
template <typename T, int V, int N, typename I>
__device__ __forceinline__ void load_batch(const T *p, I c, I step, I cols, Raw<T, V> (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c + i * step < cols)
            r[i] = *reinterpret_cast<const Raw<T, V> *>(p + c + i * step);
}

template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&f)[V])
{
    unpack<T>(*reinterpret_cast<const Raw<T, V> *>(p), f);
}

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V])
{
    if constexpr (sizeof(T) == 2 && V == 8)
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    else if constexpr (sizeof(T) == 2 && V == 2)
        *reinterpret_cast<uint32_t *>(p) = pack_bf16(f[0], f[1]);
    else if constexpr (sizeof(T) == 4 && V == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else {
        static_assert(V == 1, "no such vector");
        *p = from_f32<T>(f[0]);
    }
}

// gamma or beta: N vectors of V columns at c, c + step, ... below cols (NULL: `none`).  kind: 0 bf16, 1 fp32; + 2:
// aligned to V of them (at most 16 bytes), read in vectors.  Nothing that a kernel stores is read this way, so these
// loads may move above stores.
template <typename U, int V, int N, typename I>
__device__ __forceinline__ void load_w_as(const U *w, I c, I step, I cols, float (&f)[N][V])
{
    if constexpr (sizeof(U) * V > 16) {   // two loads of half the columns
        float lo[N][V / 2], hi[N][V / 2];
        load_w_as<U, V / 2, N, I>(w, c, step, cols, lo);
        load_w_as<U, V / 2, N, I>(w + V / 2, c, step, static_cast<I>(cols - V / 2), hi);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                f[i][j] = lo[i][j];
                f[i][j + V / 2] = hi[i][j];
            }
    } else {
        Raw<U, V> r[N] = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i * step < cols)
                r[i] = __ldg(reinterpret_cast<const Raw<U, V> *>(w + c + i * step));
#pragma unroll
        for (int i = 0; i < N; ++i)
            unpack<U>(r[i], f[i]);
    }
}

template <typename U, int V, int N, typename I>
__device__ __forceinline__ void load_w_scalar(const U *w, I c, I step, I cols, float (&f)[N][V])
{
    Raw<U, 1> r[N][V] = {};
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c + i * step < cols)
#pragma unroll
            for (int j = 0; j < V; ++j)
                r[i][j] = __ldg(reinterpret_cast<const Raw<U, 1> *>(w + c + i * step + j));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[1];
            unpack<U>(r[i][j], x);
            f[i][j] = x[0];
        }
}

template <int V, int N, typename I>
__device__ __forceinline__ void load_w(const void *w, int kind, I c, I step, I cols, float none, float (&f)[N][V])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                f[i][j] = none;
    } else if (kind == 2) {
        load_w_as<__nv_bfloat16, V, N, I>(static_cast<const __nv_bfloat16 *>(w), c, step, cols, f);
    } else if (kind == 3) {
        load_w_as<float, V, N, I>(static_cast<const float *>(w), c, step, cols, f);
    } else if (kind == 1) {
        load_w_scalar<float, V, N, I>(static_cast<const float *>(w), c, step, cols, f);
    } else {
        load_w_scalar<__nv_bfloat16, V, N, I>(static_cast<const __nv_bfloat16 *>(w), c, step, cols, f);
    }
}

// The same for columns at any place in a 16-byte word, zero where a column is outside [0, cols): whole words, shifted in
// registers (read by single columns, 2000 x 5111 took 4 us longer).  Vectors whose words are not all inside are read by columns.
template <typename U, int V, int N>
__device__ __forceinline__ void load_w_shifted(const U *w, int c, int step, int cols, float (&f)[N][V])
{
    constexpr int kOut = V * static_cast<int>(sizeof(U)) / 4, kIn = (kOut + 3) / 4 + 1;   // 4-byte words of a vector; 16-byte words it touches
    uint4 raw[N][kIn];
    bool whole[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(w + c + i * step) & ~uintptr_t{15};
        whole[i] = at >= reinterpret_cast<uintptr_t>(w) && at + 16 * kIn <= reinterpret_cast<uintptr_t>(w + cols);
#pragma unroll
        for (int k = 0; k < kIn; ++k)
            raw[i][k] = whole[i] ? __ldg(reinterpret_cast<const uint4 *>(at) + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(w + c + i * step)) & 15;
        uint32_t q[4 * kIn];
#pragma unroll
        for (int k = 0; k < kIn; ++k) {
            q[4 * k] = raw[i][k].x;
            q[4 * k + 1] = raw[i][k].y;
            q[4 * k + 2] = raw[i][k].z;
            q[4 * k + 3] = raw[i][k].w;
        }
#pragma unroll
        for (int k = 0; k + 2 < 4 * kIn; ++k)
            q[k] = shift & 8 ? q[k + 2] : q[k];
#pragma unroll
        for (int k = 0; k + 1 < 4 * kIn; ++k)
            q[k] = shift & 4 ? q[k + 1] : q[k];
#pragma unroll
        for (int k = 0; k < kOut; ++k) {
            const uint32_t v = __funnelshift_r(q[k], q[k + 1], (shift & 2) * 8);
            if constexpr (sizeof(U) == 2) {
                f[i][2 * k] = bf16_lo(v);
                f[i][2 * k + 1] = bf16_hi(v);
            } else {
                f[i][k] = __uint_as_float(v);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (!whole[i])
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int k = c + i * step + j;
                if (k >= 0 && k < cols)
                    f[i][j] = to_f32<U>(__ldg(w + k));
            }
}

// One vector, which is inside the row.  (The bound is the vector's end: where it is read in two halves, each is checked.)
template <int V>
__device__ __forceinline__ void load_w(const void *w, int kind, int64_t c, float none, float (&f)[V])
{
    load_w<V, 1, int64_t>(w, kind, c, 0, c + V, none, *reinterpret_cast<float(*)[1][V]>(&f));
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// First statement of every kernel here: the next launch on the stream may come onto the SMs while this one runs, and
// this one waits for the one before (which waited for those before it).  A launch then costs its own work and not the
// start and end of a grid as well.
__device__ __forceinline__ void take_turn()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    int64_t part_ld;               // its row pitch
    int64_t block_rows;
    int32_t blocks;
    int32_t gamma_smem;            // the backward ring kernel holds it in shared memory
    int32_t part_step, part_mask;  // block b's row begins at element (b part_step) & part_mask
};

// ---- element-wise arithmetic on a vector of V columns: pairs through the two-wide fp32 instructions of
// sm_100 and later, which halve the instructions of kernels that are bound by issue as much as by memory.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d)); }

// d = a * b + c
template <int V>
__device__ __forceinline__ void fma_v(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V])
{
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t r;
            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])), "l"(pair(c[j], c[j + 1])));
            unpair(r, d[j], d[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            d[j] = fmaf(a[j], b[j], c[j]);
    }
}

// d = a * b + c with scalars b, c
template <int V>
__device__ __forceinline__ void fma_s(float (&d)[V], const float (&a)[V], float b, float c)
{
    float bv[V], cv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bv[j] = b;
        cv[j] = c;
    }
    fma_v<V>(d, a, bv, cv);
}

template <int V>
__device__ __forceinline__ void fma_sv(float (&d)[V], const float (&a)[V], float b, const float (&c)[V])
{
    float bv[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        bv[j] = b;
    fma_v<V>(d, a, bv, c);
}

template <int V>
__device__ __forceinline__ void mul_v(float (&d)[V], const float (&a)[V], const float (&b)[V])
{
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t r;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
            unpair(r, d[j], d[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            d[j] = a[j] * b[j];
    }
}

template <int V>
__device__ __forceinline__ void mul_s(float (&d)[V], const float (&a)[V], float b)
{
    float bv[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        bv[j] = b;
    mul_v<V>(d, a, bv);
}

template <int V>
__device__ __forceinline__ void add_v(float (&d)[V], const float (&a)[V], const float (&b)[V])
{
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t r;
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
            unpair(r, d[j], d[j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            d[j] = a[j] + b[j];
    }
}

// Running sums of a vector's columns, kept as min(V, 2) partial sums.
template <int V>
struct Sum {
    static constexpr int kW = V % 2 == 0 ? 2 : 1;
    float w[kW];
    __device__ __forceinline__ Sum()
    {
#pragma unroll
        for (int k = 0; k < kW; ++k)
            w[k] = 0.0f;
    }
    __device__ __forceinline__ void add(const float (&a)[V])
    {
#pragma unroll
        for (int j = 0; j < V; j += kW) {
            float x[kW];
#pragma unroll
            for (int k = 0; k < kW; ++k)
                x[k] = a[j + k];
            add_v<kW>(w, w, x);
        }
    }
    __device__ __forceinline__ void fma(const float (&a)[V], const float (&b)[V])
    {
#pragma unroll
        for (int j = 0; j < V; j += kW) {
            float x[kW], y[kW];
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                x[k] = a[j + k];
                y[k] = b[j + k];
            }
            fma_v<kW>(w, x, y, w);
        }
    }
    __device__ __forceinline__ float total() const { return kW == 2 ? w[0] + w[kW - 1] : w[0]; }
};

// ---- sums over a block, once per row of a loop.  The scratch (32 floats, zero where a warp is absent) alternates between
// two halves, so one barrier suffices: no thread can be two rows ahead of another.
__device__ __forceinline__ void block_sum_init(float (*scratch)[32])
{
    if (threadIdx.x < 32)
        scratch[0][threadIdx.x] = scratch[1][threadIdx.x] = 0.0f;
}

__device__ __forceinline__ float block_sum(float v, float (*scratch)[32], int parity)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    v = warp_sum(v);
    if (lane == 0)
        scratch[parity][warp] = v;
    __syncthreads();
    return warp_sum(scratch[parity][lane]);
}

// Two sums at once, blocks of at most 512 threads: after the first exchange the lower half of a warp carries one value and the upper half the
// other, so both take one chain of shuffles.
__device__ __forceinline__ void block_sum2(float &a, float &b, float (*scratch)[32], int parity)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const bool upper = lane >= 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((lane & 15) == 0)
        scratch[parity][(lane & 16) + warp] = v;
    __syncthreads();
    v = scratch[parity][lane];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// ------------------------------------------------------------------------- rows through a ring --
// A block walks over rows; the next rows are on their way into shared memory while it works on one.  Each
// thread copies exactly the columns that it reads, so the copies need no barrier, only the thread's own
// wait_group.
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// `bytes` of them, and zeros for the rest
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory"); }


// Rows that start or end inside a 16-byte word (kOdd) are handled on the words of memory all the same: the first and the
// last word of a row are partly another's, are read as zeros there and stored element by element.  The place `o` of a row's
// first column in its word repeats after at most V rows, and the grid is a multiple of V, so it is the same for all rows of
// a block and a thread still keeps its columns from row to row.  All arrays share it (their base addresses are multiples of
// 16 bytes and their row strides are equal modulo V).  The elements before a row that are read lie in the same array: row 0
// has o = 0.

// kStages slots of `bufs` rows, kItems vectors of V elements (16 bytes) per thread and row.
template <typename T, int V, int kItems, int kStages, bool kOdd>
struct RowRing {
    static constexpr int kBytes = 16;
    static_assert(V * sizeof(T) == 16, "words of 16 bytes");
    uint32_t first, last;        // this thread's place in the first and last slot
    uint32_t rd, wr;             // ... in the slot to read and to fill next
    uint32_t item, row, slot;    // strides of vectors, rows and slots
    int cols, c0, cstep;         // this thread's first column (-o for thread 0), and the step to its next vector
    int o;
    __device__ __forceinline__ RowRing(const void *smem, int bufs, int n_cols, int64_t ld) : cols(n_cols)
    {
        o = kOdd ? static_cast<int>(blockIdx.x * ld) & (V - 1) : 0;
        item = blockDim.x * kBytes;
        row = item * kItems;
        slot = row * static_cast<uint32_t>(bufs);
        first = rd = wr = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * kBytes;
        last = first + slot * (kStages - 1);
        c0 = static_cast<int>(threadIdx.x) * V - o;
        cstep = static_cast<int>(blockDim.x) * V;
    }
    // vector i is partly outside the row / its element j is outside
    __device__ __forceinline__ bool edge(int i) const { return kOdd && ((i == 0 && c0 < 0) || c0 + i * cstep + V > cols); }
    __device__ __forceinline__ bool outside(int i, int j) const { return static_cast<unsigned>(c0 + i * cstep + j) >= static_cast<unsigned>(cols); }
    __device__ __forceinline__ void clear_outside(int i, float (&f)[V]) const
    {
        if (edge(i))
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (outside(i, j))
                    f[j] = 0.0f;
    }
    // vector i of the row of which p is this thread's first column
    __device__ __forceinline__ void write(T *p, int i, const float (&f)[V]) const
    {
        if (edge(i)) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (!outside(i, j))
                    p[i * cstep + j] = from_f32<T>(f[j]);
        } else {
            store<T, V>(p + i * cstep, f);
        }
    }
    // gamma or beta at this thread's columns, zero outside the row
    __device__ __forceinline__ void weights(const void *w, int kind, float none, float (&f)[kItems][V]) const
    {
        if constexpr (!kOdd) {
            load_w<V, kItems>(w, kind, c0, cstep, cols, none, f);
        } else {
            if (!w) {
#pragma unroll
                for (int i = 0; i < kItems; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        f[i][j] = none;
            } else if (kind & 1) {
                load_w_shifted<float, V, kItems>(static_cast<const float *>(w), c0, cstep, cols, f);
            } else {
                load_w_shifted<__nv_bfloat16, V, kItems>(static_cast<const __nv_bfloat16 *>(w), c0, cstep, cols, f);
            }
        }
    }
    __device__ __forceinline__ bool has(int i) const { return c0 + i * cstep < cols; }
    __device__ __forceinline__ void advance(uint32_t &at) const { at = at == last ? first : at + slot; }
    // one row into buffer `buf` of the slot to fill
    __device__ __forceinline__ void fetch(int buf, const T *src) const
    {
        src += c0;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (has(i)) {
                if constexpr (kOdd)
                    copy_async(wr + buf * row + i * item, src + i * cstep, min(V, cols - c0 - i * cstep) * static_cast<uint32_t>(sizeof(T)));
                else
                    copy_async(wr + buf * row + i * item, src + i * cstep);
            }
    }
    // vector i of buffer `buf` of the slot to read
    __device__ __forceinline__ void read(int buf, int i, float (&f)[V]) const
    {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(rd + buf * row + i * item)
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2) {
                f[2 * j] = bf16_lo(w[j]);
                f[2 * j + 1] = bf16_hi(w[j]);
            } else {
                f[j] = __uint_as_float(w[j]);
            }
        }
        if constexpr (kOdd)
            if (i == 0)   // (the copies put zeros behind the row's end)
#pragma unroll
                for (int j = 0; j < V - 1; ++j)
                    f[j] = c0 + j < 0 ? 0.0f : f[j];
    }
};

// Forward over many rows.  A thread keeps its columns from row to row, so gamma and beta stay in registers.
// 2048 x 8192 bf16: 14.1 us, 4.8 TB/s of read and written bytes; its first loads and last stores bound so short a kernel.
// Rows inside words: 2000 x 5111 16.6 us.  fp32: 2048 x 8192 22.3 us, 4096 x 4096 23.7 (6.0 and 5.7 TB/s).
template <typename T, int V, int kItems, int kStages, bool kOdd>
__global__ void __launch_bounds__(512) norm_forward_ring_kernel(const NormParams p)
{
    take_turn();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s1[2][32], s2[2][32];
    RowRing<T, V, kItems, kStages, kOdd> ring(smem, 1, static_cast<int>(p.cols), p.ldx);
    const int64_t step = gridDim.x;
    const T *ahead = static_cast<const T *>(p.x) + blockIdx.x * p.ldx;   // next row to fetch
    T *y = static_cast<T *>(p.y) + blockIdx.x * p.ldy + ring.c0;
    int left = static_cast<int>((p.rows - blockIdx.x + step - 1) / step);   // rows of this block
    int to_fetch = left;
    auto fetch = [&] {
        if (to_fetch > 0)
            ring.fetch(0, ahead);
        copy_commit();
        ring.advance(ring.wr);
        ahead += step * p.ldx;
        --to_fetch;
    };
    for (int s = 0; s < kStages - 1; ++s)
        fetch();
    block_sum_init(s1);
    block_sum_init(s2);
    float g[kItems][V], b[kItems][V];
    ring.weights(p.gamma, p.w_kind, 1.0f, g);
    ring.weights(p.beta, p.w_kind, 0.0f, b);
    __syncthreads();
    int parity = 0;
    for (int64_t row = blockIdx.x; left > 0; --left, row += step, parity ^= 1) {
        copy_wait<kStages - 2>();
        fetch();
        float v[kItems][V];
        Sum<V> sum, sq;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (ring.has(i)) {
                ring.read(0, i, v[i]);
                sum.add(v[i]);
            }
        ring.advance(ring.rd);
        const float mean = __fdiv_rn(block_sum(sum.total(), s1, parity), static_cast<float>(ring.cols));
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (ring.has(i)) {
                fma_s<V>(v[i], v[i], 1.0f, -mean);
                ring.clear_outside(i, v[i]);
                sq.fma(v[i], v[i]);
            }
        const float rstd = rsqrtf(fmaf(block_sum(sq.total(), s2, parity), p.inv_cols, p.eps));
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (ring.has(i)) {
                mul_s<V>(v[i], v[i], rstd);
                fma_v<V>(v[i], v[i], g[i], b[i]);
                ring.write(y, i, v[i]);
            }
        y += step * p.ldy;
    }
}

// Backward: dx of each row, and this block's column sums of dy xh and dy in registers (each thread keeps its
// columns from row to row), so x and dy are read once for all three gradients.  Up to 16 columns a thread also
// keep gamma and, over the row's reduction, g and xh; more columns are read and computed again.  (x rstd -
// mean rstd would save an instruction, but leaves rounding errors where x = mean.)  The sums of the blocks are added
// by norm_colsum_finish_kernel.  4096 x 8192 bf16 with dx_add: 43.4 us, 6.2 TB/s, of 49 with the finish; the issue of
// instructions (53 % of cycles) and memory come close to each other.
template <typename T, int V, int kItems, int kStages, bool kOdd>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormParams p)
{
    take_turn();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[2][32];
    constexpr bool kKeep = V * kItems <= 16;
    constexpr int kK = kKeep ? kItems : 1;
    RowRing<T, V, kItems, kStages, kOdd> ring(smem, p.add ? 3 : 2, static_cast<int>(p.cols), p.ldx);
    const int64_t step = gridDim.x;
    const int cols = ring.cols;
    const int64_t r0 = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + r0 * p.ldx, *dy = static_cast<const T *>(p.dy) + r0 * p.lddy;
    const T *add = p.add ? static_cast<const T *>(p.add) + r0 * p.ldadd : nullptr;
    T *dx = p.dx ? static_cast<T *>(p.dx) + r0 * p.lddx + ring.c0 : nullptr;
    const int mine = static_cast<int>((p.rows - r0 + step - 1) / step);   // rows of this block
    int to_fetch = mine;
    // x, dy and add run ahead: they point to the next row to fetch
    auto fetch = [&] {
        if (to_fetch > 0) {
            ring.fetch(0, x);
            ring.fetch(1, dy);
            if (add)
                ring.fetch(2, add);
        }
        copy_commit();
        ring.advance(ring.wr);
        --to_fetch;
        x += step * p.ldx;
        dy += step * p.lddy;
        if (add)
            add += step * p.ldadd;
    };
    for (int s = 0; s < kStages - 1; ++s)
        fetch();
    block_sum_init(scratch);
    float ag[kItems][V], ab[kItems][V], gk[kK][V];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            ag[i][j] = ab[i][j] = 0.0f;
    }
    // gamma of more columns: behind the ring in fp32, where each thread lays out its own (1898 x 11248 58 -> 45 us), or,
    // without room there, from global memory
    float4 *gs = reinterpret_cast<float4 *>(smem + kStages * ring.slot) + threadIdx.x;
    if constexpr (kKeep) {
        ring.weights(p.gamma, p.w_kind, 1.0f, gk);
    } else if (kOdd || p.gamma_smem) {
        float w[kItems][V];
        ring.weights(p.gamma, p.w_kind, 1.0f, w);
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
            for (int j = 0; j < V; j += 4)
                gs[(i * V + j) / 4 * blockDim.x] = make_float4(w[i][j], w[i][j + 1], w[i][j + 2], w[i][j + 3]);
    }
    // mean and rstd of 32 rows at a time, a row a lane, the next 32 on their way: one row ahead is not enough for
    // memory under load
    const int lane = static_cast<int>(threadIdx.x & 31);
    auto load_stats = [&](int first, float &m, float &r) {
        const int64_t q = r0 + static_cast<int64_t>(min(first + lane, mine - 1)) * step;
        m = p.mean_in[q];
        r = p.rstd_in[q];
    };
    float mean_c, rstd_c, mean_n, rstd_n;
    load_stats(0, mean_c, rstd_c);
    load_stats(32, mean_n, rstd_n);
    __syncthreads();
    int parity = 0;
    for (int it = 0; it < mine; ++it, parity ^= 1) {
        copy_wait<kStages - 2>();
        fetch();
        if (it > 0 && (it & 31) == 0) {
            mean_c = mean_n;
            rstd_c = rstd_n;
            load_stats(it + 32, mean_n, rstd_n);
        }
        const float mean = __shfl_sync(0xffffffffu, mean_c, it & 31), rstd = __shfl_sync(0xffffffffu, rstd_c, it & 31);
        Sum<V> sum0, sum1;
        float gd[kK][V], xh[kK][V];
        auto terms = [&](int i, float (&d)[V], float (&go)[V], float (&xo)[V]) {   // dy, g and xh of vector i
            float a[V];
            ring.read(0, i, a);
            ring.read(1, i, d);
            fma_s<V>(xo, a, 1.0f, -mean);
            mul_s<V>(xo, xo, rstd);
            if constexpr (kKeep) {
                mul_v<V>(go, gk[kKeep ? i : 0], d);
            } else {
                float w[V];
                if (kOdd || p.gamma_smem) {
#pragma unroll
                    for (int j = 0; j < V; j += 4) {
                        const float4 q = gs[(i * V + j) / 4 * blockDim.x];
                        w[j] = q.x;
                        w[j + 1] = q.y;
                        w[j + 2] = q.z;
                        w[j + 3] = q.w;
                    }
                } else {
                    load_w<V>(p.gamma, p.w_kind, ring.c0 + i * ring.cstep, 1.0f, w);
                }
                mul_v<V>(go, w, d);
            }
        };
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (ring.has(i)) {
                float d[V];
                const int k = kKeep ? i : 0;
                terms(i, d, gd[k], xh[k]);
                add_v<V>(ab[i], ab[i], d);
                fma_v<V>(ag[i], d, xh[k], ag[i]);
                sum0.add(gd[k]);
                sum1.fma(gd[k], xh[k]);
            }
        if (dx) {
            float m0 = sum0.total(), m1 = sum1.total();
            block_sum2(m0, m1, scratch, parity);
            m0 *= -rstd * p.inv_cols;   // dx = rstd g + (m0' + m1' xh), m' = -rstd * mean of g, of g xh
            m1 *= -rstd * p.inv_cols;
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (ring.has(i)) {
                    float o[V], d[V];
                    const int k = kKeep ? i : 0;
                    if constexpr (!kKeep)
                        terms(i, d, gd[k], xh[k]);
                    fma_s<V>(o, xh[k], m1, m0);
                    fma_sv<V>(o, gd[k], rstd, o);
                    if (add) {
                        float r[V];
                        ring.read(2, i, r);
                        add_v<V>(o, o, r);
                    }
                    ring.write(dx, i, o);
                }
            dx += step * p.lddx;
        }
        ring.advance(ring.rd);
    }
    if (p.part) {
        float *out = p.part + r0 * 2 * p.part_ld;   // (with kOdd its first column is column -o)
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int c = ring.c0 + ring.o + i * ring.cstep;
            if (ring.has(i)) {
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    *reinterpret_cast<float4 *>(out + c + j) = make_float4(ag[i][j], ag[i][j + 1], ag[i][j + 2], ag[i][j + 3]);
                    *reinterpret_cast<float4 *>(out + p.part_ld + c + j) = make_float4(ab[i][j], ab[i][j + 1], ab[i][j + 2], ab[i][j + 3]);
                }
            }
        }
    }
}

// One row per team, the row in registers (kItems vectors of V per thread): moments, then the output.  For few rows
// or narrow ones: latency (one row of 4096 4.2 us, back to back 2.2 by the host).
template <typename T, int V, int kItems, bool kWarpTeam, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormParams p)
{
    take_turn();
    __shared__ float scratch[32];
    const int team = kWarpTeam ? 32 : static_cast<int>(blockDim.x);
    const int t = kWarpTeam ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t row = kWarpTeam ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (row >= p.rows)
        return;   // a whole team leaves (warp teams share no barrier)
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    float v[kItems][V];
    float s[1] = {0.0f};
    const int64_t c0 = static_cast<int64_t>(t) * V, cstep = static_cast<int64_t>(team) * V;
    Raw<T, V> raw[kItems] = {};
    load_batch<T, V, kItems>(x, c0, cstep, p.cols, raw);
    // The weights of at most 16 columns at a time; where that is all of them, they are on their way during the sums.
    constexpr int kB = V * kItems <= 16 ? kItems : 16 / V > 0 ? 16 / V : 1;
    constexpr bool kEarly = kB == kItems;
    float g[kB][V], b[kB][V];
    if (kEarly) {
        load_w<V, kB>(p.gamma, p.w_kind, c0, cstep, p.cols, 1.0f, g);
        load_w<V, kB>(p.beta, p.w_kind, c0, cstep, p.cols, 0.0f, b);
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        unpack<T>(raw[i], v[i]);   // (zeros past the row's end)
#pragma unroll
        for (int j = 0; j < V; ++j)
            s[0] += v[i][j];
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
    for (int k = 0; k < kItems; k += kB) {
        if (!kEarly) {
            load_w<V, kB>(p.gamma, p.w_kind, c0 + k * cstep, cstep, p.cols, 1.0f, g);
            load_w<V, kB>(p.beta, p.w_kind, c0 + k * cstep, cstep, p.cols, 0.0f, b);
        }
#pragma unroll
        for (int i = 0; i < kB; ++i)
            if (c0 + (k + i) * cstep < p.cols) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j)
                    o[j] = fmaf((v[k + i][j] - mean) * rstd, g[i][j], b[i][j]);
                store<T, V>(y + c0 + (k + i) * cstep, o);
            }
    }
}

// ------------------------------------------------------------------------ rows without 16-byte alignment --
// Any width and stride, in loops over the columns.  Forward, a thread works on two neighbouring bf16 columns or one fp32
// column at a time (bf16 pairs of a row that starts between two 4-byte words are loaded and stored as halves).  Each
// round first requests the loads of kBatch vectors and then works on them: a loop that uses a value where it loads it waits for
// memory once per vector (one row of 14876 columns took 28 us that way).
template <typename T>
constexpr int kLoopV = sizeof(T) == 2 ? 2 : 1;

template <typename T>
__device__ __forceinline__ bool between_words(const void *row) { return sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(row) & 2) != 0; }

// Vectors of a row at columns c, c + step, ... below cols, as they were loaded: a value or a word of two, or the two halves
// of a pair between words (nothing here uses a loaded value, so all loads go out before any is waited for).  The half of a
// pair past the row's end is zero.
struct Loaded {
    uint32_t a, b;
};

template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, bool split, int c, int step, int cols, Loaded (&r)[N])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i * step < cols)
                r[i].a = *reinterpret_cast<const uint32_t *>(p + c + i * step);
    } else {
        const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
        if (!split) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = c + i * step;
                if (k + 1 < cols)
                    r[i].a = *reinterpret_cast<const uint32_t *>(h + k);
                else if (k < cols)
                    r[i].a = h[k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = c + i * step;
                r[i].b = 0;
                if (k < cols)
                    r[i].a = h[k];
                if (k + 1 < cols)
                    r[i].b = h[k + 1];
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void unpack_row(bool split, const Loaded &r, float (&f)[kLoopV<T>])
{
    if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(r.a);
    } else {
        f[0] = bf16_lo(r.a);
        f[1] = split ? bf16_lo(r.b) : bf16_hi(r.a);
    }
}

template <typename T>
__device__ __forceinline__ void store_row(T *p, bool split, int k, int cols, const float (&f)[kLoopV<T>])
{
    if constexpr (sizeof(T) == 4) {
        p[k] = f[0];
    } else {
        const uint32_t w = pack_bf16(f[0], f[1]);
        unsigned short *h = reinterpret_cast<unsigned short *>(p);
        if (!split && k + 1 < cols) {
            *reinterpret_cast<uint32_t *>(h + k) = w;
        } else {
            h[k] = static_cast<unsigned short>(w);
            if (k + 1 < cols)
                h[k + 1] = static_cast<unsigned short>(w >> 16);
        }
    }
}

// gamma or beta at those columns.
template <int V, int N>
__device__ __forceinline__ void load_w_row(const void *w, int kind, int c, int step, int cols, float none, float (&f)[N][V])
{
    if constexpr (V == 1) {
        load_w<1, N>(w, kind, c, step, cols, none, f);
    } else {
        const int pairs = cols & ~1;   // a last single column is read by itself
        load_w<2, N>(w, kind, c, step, pairs, none, f);
        if (w && (cols & 1))
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c + i * step == cols - 1)
                    f[i][0] = kind & 1 ? __ldg(static_cast<const float *>(w) + cols - 1)
                                       : __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(w) + cols - 1));
    }
}

// Forward: the row waits in shared memory in fp32 between its three passes.  For arrays whose rows start at different
// places in their words: 2000 x 5111 30.5 us, bound by the issue of narrow loads and stores.
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_staged_kernel(const NormParams p)
{
    take_turn();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s1[2][32], s2[2][32];
    constexpr int kBatch = 8, V = kLoopV<T>;
    float *buf = reinterpret_cast<float *>(smem);
    const int cols = static_cast<int>(p.cols), c0 = static_cast<int>(threadIdx.x) * V, cstep = static_cast<int>(blockDim.x) * V;
    block_sum_init(s1);
    block_sum_init(s2);
    __syncthreads();
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        T *y = static_cast<T *>(p.y) + row * p.ldy;
        const bool sx = between_words<T>(x), sy = between_words<T>(y);
        float s = 0.0f;
        for (int c = c0; c < cols; c += kBatch * cstep) {   // (each thread reads back only what it wrote: no barrier)
            Loaded raw[kBatch];
            load_row<T, kBatch>(x, sx, c, cstep, cols, raw);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (c + i * cstep < cols) {
                    float v[V];
                    unpack_row<T>(sx, raw[i], v);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        s += v[j];
                    if constexpr (V == 2)
                        *reinterpret_cast<float2 *>(buf + c + i * cstep) = make_float2(v[0], v[1]);
                    else
                        buf[c + i * cstep] = v[0];
                }
        }
        const float mean = __fdiv_rn(block_sum(s, s1, parity), static_cast<float>(cols));
        s = 0.0f;
#pragma unroll 4
        for (int c = c0; c < cols; c += cstep) {
            if constexpr (V == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(buf + c);
                const float d = v.x - mean, e = c + 1 < cols ? v.y - mean : 0.0f;
                s = fmaf(d, d, fmaf(e, e, s));
            } else {
                const float d = buf[c] - mean;
                s = fmaf(d, d, s);
            }
        }
        const float rstd = rsqrtf(fmaf(block_sum(s, s2, parity), p.inv_cols, p.eps));
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
        for (int c = c0; c < cols; c += kBatch * cstep) {
            float g[kBatch][V], b[kBatch][V], o[V];
            load_w_row<V, kBatch>(p.gamma, p.w_kind, c, cstep, cols, 1.0f, g);
            load_w_row<V, kBatch>(p.beta, p.w_kind, c, cstep, cols, 0.0f, b);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (c + i * cstep < cols) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        o[j] = fmaf((buf[c + i * cstep + j] - mean) * rstd, g[i][j], b[i][j]);
                    store_row<T>(y, sy, c + i * cstep, cols, o);
                }
        }
    }
}

// (The backward kernels take bf16 in pairs only where rows are in 4-byte units: with pairs between words their loops
// took twice as long as with single columns.)

// Backward, R rows at a time: a column's R contributions to dgamma and dbeta are added in registers and then to the
// block's running sums in shared memory; dx reads its rows a second time (from L1 or L2).  Fewer rows than R at the end
// go one by one.  2000 x 5111 47 us, bound by the issue of loads of single columns.
struct StagedSums {
    float *ag, *ab;      // running sums of the block (a thread touches only its own columns) ...
    float *pg, *pb;      // ... or, with one round per block, the partial row itself
    bool want, once;
};

template <typename T, int V, int R>
__device__ __forceinline__ void backward_rows(const NormParams &p, int64_t row, const StagedSums &q, float (*scratch)[16])
{
    constexpr int kBatch = R == 1 ? 4 : 2;
    const int cols = static_cast<int>(p.cols), c0 = static_cast<int>(threadIdx.x) * V, cstep = static_cast<int>(blockDim.x) * V;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, warps = blockDim.x / 32;
    const T *x[R], *dy[R];
    float mean[R], rstd[R], s0[R], s1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = static_cast<const T *>(p.x) + (row + r) * p.ldx;
        dy[r] = static_cast<const T *>(p.dy) + (row + r) * p.lddy;
        mean[r] = p.mean_in[row + r];
        rstd[r] = p.rstd_in[row + r];
        s0[r] = s1[r] = 0.0f;
    }
    for (int c = c0; c < cols; c += kBatch * cstep) {
        Raw<T, V> ra[R][kBatch], rd[R][kBatch];
        float g[kBatch][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            load_batch<T, V, kBatch>(x[r], c, cstep, cols, ra[r]);
            load_batch<T, V, kBatch>(dy[r], c, cstep, cols, rd[r]);
        }
        load_w<V, kBatch>(p.gamma, p.w_kind, c, cstep, cols, 1.0f, g);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (c + i * cstep < cols) {
                float dg[V], db[V];
#pragma unroll
                for (int j = 0; j < V; ++j)
                    dg[j] = db[j] = 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float a[V], d[V];
                    unpack<T>(ra[r][i], a);
                    unpack<T>(rd[r][i], d);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float xh = (a[j] - mean[r]) * rstd[r], gd = g[i][j] * d[j];
                        db[j] += d[j];
                        dg[j] = fmaf(d[j], xh, dg[j]);
                        s0[r] += gd;
                        s1[r] = fmaf(gd, xh, s1[r]);
                    }
                }
                if (q.want) {
                    const int k = c + i * cstep;
                    if (q.once)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            q.pg[k + j] = dg[j];
                            q.pb[k + j] = db[j];
                        }
                    else
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            q.ag[k + j] += dg[j];
                            q.ab[k + j] += db[j];
                        }
                }
            }
    }
    if (!p.dx)
        return;
    __syncthreads();   // the sums of the rows before have been read
#pragma unroll
    for (int r = 0; r < R; ++r) {
        s0[r] = warp_sum(s0[r]);
        s1[r] = warp_sum(s1[r]);
        if (lane == 0) {
            scratch[2 * r][warp] = s0[r];
            scratch[2 * r + 1][warp] = s1[r];
        }
    }
    __syncthreads();
    float m0[R], m1[R];   // dx = rstd g + (m0 + m1 xh)
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float u = (lane & 15) < warps ? scratch[2 * r][lane & 15] : 0.0f, w = (lane & 15) < warps ? scratch[2 * r + 1][lane & 15] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            u += __shfl_xor_sync(0xffffffffu, u, o);
            w += __shfl_xor_sync(0xffffffffu, w, o);
        }
        m0[r] = -rstd[r] * p.inv_cols * u;
        m1[r] = -rstd[r] * p.inv_cols * w;
    }
    for (int c = c0; c < cols; c += kBatch * cstep) {
        Raw<T, V> ra[R][kBatch], rd[R][kBatch], rq[R][kBatch];
        float g[kBatch][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            load_batch<T, V, kBatch>(x[r], c, cstep, cols, ra[r]);
            load_batch<T, V, kBatch>(dy[r], c, cstep, cols, rd[r]);
            if (p.add)
                load_batch<T, V, kBatch>(static_cast<const T *>(p.add) + (row + r) * p.ldadd, c, cstep, cols, rq[r]);
        }
        load_w<V, kBatch>(p.gamma, p.w_kind, c, cstep, cols, 1.0f, g);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (c + i * cstep < cols)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float o[V], a[V], d[V], e[V];
                    unpack<T>(ra[r][i], a);
                    unpack<T>(rd[r][i], d);
                    unpack<T>(rq[r][i], e);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        o[j] = fmaf(g[i][j] * d[j], rstd[r], fmaf((a[j] - mean[r]) * rstd[r], m1[r], m0[r]));
                        if (p.add)
                            o[j] += e[j];
                    }
                    store<T, V>(static_cast<T *>(p.dx) + (row + r) * p.lddx + c + i * cstep, o);
                }
    }
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(512) norm_backward_staged_kernel(const NormParams p)
{
    take_turn();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[2 * R][16];
    const int cols = static_cast<int>(p.cols), c0 = static_cast<int>(threadIdx.x) * V, cstep = static_cast<int>(blockDim.x) * V;
    StagedSums q;
    q.want = p.part != nullptr;
    q.once = static_cast<int64_t>(gridDim.x) * R >= p.rows && p.rows % R == 0;
    q.ag = reinterpret_cast<float *>(smem);
    q.ab = q.ag + cols;
    q.pg = p.part + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    q.pb = q.pg + cols;
    if (q.want && !q.once)
        for (int c = c0; c < cols; c += cstep)
#pragma unroll
            for (int j = 0; j < V; ++j)
                q.ag[c + j] = q.ab[c + j] = 0.0f;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * R; row < p.rows; row += static_cast<int64_t>(gridDim.x) * R) {
        if (R == 1 || row + R <= p.rows)
            backward_rows<T, V, R>(p, row, q, scratch);
        else
            for (int64_t r = row; r < p.rows; ++r)
                backward_rows<T, V, 1>(p, r, q, scratch);
    }
    if (q.want && !q.once)
        for (int c = c0; c < cols; c += cstep)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                q.pg[c + j] = q.ag[c + j];
                q.pb[c + j] = q.ab[c + j];
            }
}

// Rows too wide for registers and shared memory: three passes over the row (the later ones come from L2).  256 x 40000
// bf16: 49 us, bound by its narrow loads; such rows are here to be right.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_wide_kernel(const NormParams p)
{
    take_turn();
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
// time from L1 or L2), so any width fits.  256 x 40000 bf16: 16 us.
template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_dx_kernel(const NormParams p)
{
    take_turn();
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

// Column sums of dy xh and dy over one block of rows: 32 lanes x V columns, 8 warps over the rows.  256 x 40000 bf16:
// 27 us, bound by the latency of few rows a thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_colsum_kernel(const NormParams p)
{
    take_turn();
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

// dgamma and dbeta: the blocks' partial rows, added in a fixed order.  Latency is all there is to it (10 MB from L2 for
// 152 rows of 8192), so L = 8 threads of a warp take a row (32 where the rows are few and blocks would be many), a block
// 256 / L interleaved sets of rows, and a thread requests 8 rows at once: V = 4 columns each where the rows are in 16-byte
// units, else one.  (One thread a column and 32 rows a block of 1024 threads: 3 us longer at 152 x 8192.)
template <int V, int L>
__global__ void __launch_bounds__(256) norm_colsum_finish_kernel(const NormParams p, void *dgamma, void *dbeta)
{
    __shared__ float red[8][L * V];
    take_turn();
    constexpr int kBatch = 8, kSets = 256 / L;
    const int lane = threadIdx.x & (L - 1), set = threadIdx.x / L;
    const int w = blockIdx.y;
    void *out = w ? dbeta : dgamma;
    if (!out)
        return;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * L + lane) * V;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        s[j] = 0.0f;
    if (c < p.cols)
        for (int b0 = set; b0 < p.blocks; b0 += kSets * kBatch) {
            Raw<float, V> r[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int b = b0 + kSets * i;
                if (b < p.blocks)
                    r[i] = *reinterpret_cast<const Raw<float, V> *>(p.part + (static_cast<int64_t>(b) * 2 + w) * p.part_ld + c +
                                                                    ((b * p.part_step) & p.part_mask));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (b0 + kSets * i < p.blocks) {
                    float x[V];
                    unpack<float>(r[i], x);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        s[j] += x[j];
                }
        }
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int o = L; o < 32; o *= 2)
            s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
        if ((threadIdx.x & 31) < L)
            red[threadIdx.x / 32][lane * V + j] = s[j];
    }
    __syncthreads();
    const int64_t k = static_cast<int64_t>(blockIdx.x) * L * V + threadIdx.x;
    if (threadIdx.x < L * V && k < p.cols) {
        float t = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            t += red[q][threadIdx.x];
        if (p.w_f32)
            static_cast<float *>(out)[k] = t;
        else
            static_cast<__nv_bfloat16 *>(out)[k] = __float2bfloat16_rn(t);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kSms = 152;
constexpr int kColsumBlocks = 64;     // row blocks of the two-kernel backward pass, at most
constexpr int64_t kOddLeast = 16;     // words a row (forward_odd)
constexpr size_t kRingLimit = 200 * 1024;
constexpr size_t kAloneLimit = 226 * 1024;       // of a block that has an SM to itself
constexpr int64_t kFusedCols = kRingLimit / 8;   // its widest rows
constexpr int64_t kLoopCols = int64_t{1} << 30;  // the widest rows of kernels that count columns in int

// Vectors per thread of the backward ring kernel, for at most 512 threads and 32 columns a thread.  0: too wide.
int ring_items(int64_t nvec, int v)
{
    if (nvec <= 256)
        return 1;
    for (int items = 2; items <= 32 / v; items *= 2)
        if (nvec <= 512 * items)
            return items;
    return 0;
}

int ring_threads(int64_t nvec, int items) { return static_cast<int>(cdiv(cdiv(nvec, items), 32) * 32); }

// Threads of the kernels that loop over columns in rounds of `batch` vectors: as few rounds as `most` threads need, and no
// more threads than fill those (a round that is mostly past the row's end costs as much as a full one).
int loop_threads(int64_t nvec, int batch, int most)
{
    const int64_t rounds = cdiv(nvec, static_cast<int64_t>(batch) * most);
    return static_cast<int>(std::max<int64_t>(64, cdiv(cdiv(nvec, rounds * batch), 32) * 32));
}

// Blocks per SM of the fused backward kernels: as many as its 65536 registers hold (64, 96 or 128 a thread for 4, 8 or
// more columns).
int ring_per_sm(int threads, int columns)
{
    return std::max(1, std::min(8, 65536 / ((columns <= 4 ? 64 : columns <= 8 ? 96 : 128) * threads)));
}
int staged_per_sm(int threads, size_t smem, int at_a_time)
{
    return std::max(1, std::min({8, (at_a_time == 1 ? 1536 : 1024) / threads, static_cast<int>(kRingLimit / smem)}));
}

// Words that a row of `cols` columns touches at most, from the place in its first word on.
int64_t odd_words(int64_t cols, int v) { return cdiv(cols + v - 1, v); }

// The most blocks that a fused backward kernel uses at this width, over the kinds of alignment.
int64_t most_fused_blocks(int64_t cols)
{
    int per_sm = 1;
    for (int v = 1; v <= 8; v *= 2)
        for (const int64_t nvec : {cdiv(cols, v), odd_words(cols, v)}) {
            if (v <= 2)
                per_sm = std::max(per_sm, staged_per_sm(loop_threads(nvec, 4, 512), static_cast<size_t>(cols) * 8, 1));
            else if (const int items = ring_items(nvec, v))
                per_sm = std::max(per_sm, ring_per_sm(ring_threads(nvec, items), items * v));
        }
    return static_cast<int64_t>(per_sm) * kSms;
}

// A call's launches: none after one that failed.
struct Stream {
    cudaStream_t stream;
    bool failed = false;
};

// A kernel's limit is raised to the same value whatever a launch takes: the limit belongs to the kernel, and another thread may
// be about to launch it with more.
template <typename K>
bool allow_smem(K *kernel, size_t bytes)
{
    return bytes <= 47 * 1024 ||   // (the blocks also hold up to 1 KB of static shared memory)
           succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kAloneLimit)));
}

bool aligned(const void *p, int64_t ld, size_t esz, size_t bytes)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && static_cast<size_t>(ld) * esz % bytes == 0);
}

bool bad_dtype(mlp_dtype d) { return d != MLP_DT_BF16 && d != MLP_DT_F32; }

bool bad_rows(const void *p, int64_t ld, int64_t cols, size_t esz)
{
    return !p || reinterpret_cast<uintptr_t>(p) % esz != 0 || ld < cols;
}

// (see take_turn)
template <typename... A, typename... B>
void launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, Stream &st, B... args)
{
    if (st.failed)
        return;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    st.failed = !succeeded(cudaLaunchKernelEx(&cfg, kernel, A(args)...));
}

template <typename T, int V, int kItems, int kThreads>
void launch_forward(const NormParams &p, int64_t nvec, Stream &st)
{
    if (nvec <= 32 * kItems) {
        const int teams = 4;
        launch(norm_forward_kernel<T, V, kItems, true, 128>, static_cast<unsigned>(cdiv(p.rows, teams)), 32 * teams, 0, st, p);
    } else {
        const int threads = static_cast<int>(cdiv(cdiv(nvec, kItems), 32) * 32);
        launch(norm_forward_kernel<T, V, kItems, false, kThreads>, static_cast<unsigned>(p.rows), threads, 0, st, p);
    }
}

template <typename T, int V, int kItems, bool kOdd>
bool launch_forward_ring(const NormParams &p, int64_t nvec, Stream &st)
{
    constexpr int kStages = 3;   // (4 and 5 slots measured no faster at 2048 x 8192)
    const int threads = static_cast<int>(cdiv(cdiv(nvec, kItems), 32) * 32);
    const size_t smem = static_cast<size_t>(kStages) * kItems * threads * V * sizeof(T);
    if (smem > kRingLimit)
        return false;
    // Blocks per SM: as many as fit registers (40, 64 or 128 a thread for 4, 8 or 32 columns) and rings, unless fewer leave
    // the last round fuller (the blocks of an SM share its throughput, so a round of n rows per SM costs n).
    const int most = std::max(1, std::min({12, (V * kItems <= 4 ? 1536 : V * kItems <= 8 ? 1024 : 512) / threads,
                                            static_cast<int>(kRingLimit / smem)}));
    int per_sm = most;
    for (int n = most; n >= std::max(1, most / 2); --n)
        if (cdiv(p.rows, static_cast<int64_t>(n) * kSms) * n < cdiv(p.rows, static_cast<int64_t>(per_sm) * kSms) * per_sm)
            per_sm = n;
    static_assert(kSms % V == 0, "rows of a block start at the same place in a word");
    auto kernel = norm_forward_ring_kernel<T, V, kItems, kStages, kOdd>;
    if (!allow_smem(kernel, smem))
        return false;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.rows, static_cast<int64_t>(per_sm) * kSms));
    launch(kernel, grid, threads, smem, st, p);
    return true;
}

template <typename T>
bool launch_forward_staged(const NormParams &p, Stream &st)
{
    const int threads = loop_threads(cdiv(p.cols, kLoopV<T>), 8, 1024);
    const size_t smem = static_cast<size_t>((p.cols + 1) & ~int64_t{1}) * 4;
    auto kernel = norm_forward_staged_kernel<T>;
    if (smem > kRingLimit || !allow_smem(kernel, smem))
        return false;
    const int per_sm = std::max(1, std::min({16, 1024 / threads, static_cast<int>(kRingLimit / smem)}));
    launch(kernel, static_cast<unsigned>(std::min<int64_t>(p.rows, static_cast<int64_t>(per_sm) * kSms)), threads, smem, st, p);
    return true;
}

// Rows of any width and stride on the words of memory (2000 x 5111 16.6 us, staged 30.5); false where they are too wide, or
// too narrow: up to 16 words a row the kernels for other rows are as fast (8000 x 71 8 us, through the ring 14).
template <typename T>
bool forward_odd(const NormParams &p, Stream &st)
{
    constexpr int V = 16 / sizeof(T), kMost = 32 / V;
    const int64_t nvec = odd_words(p.cols, V);
    if (nvec <= kOddLeast)
        return false;
    if constexpr (V == 4)   // (8 vectors a thread: 4000 x 2001 22.6 us, 2: 18.4; in bf16 2 instead of 4 gained as often as it lost)
        if (nvec > 256 && nvec <= 512)
            return launch_forward_ring<T, V, 2, true>(p, nvec, st);
    return nvec <= 256 ? launch_forward_ring<T, V, 1, true>(p, nvec, st)
                       : nvec <= 512 * kMost && launch_forward_ring<T, V, kMost, true>(p, nvec, st);
}

// Rows in 16-byte units.  Few rows: one vector per thread and one row per block, so that a row's loads go out at once
// from as many threads as there are.  Many rows: narrow ones a warp each, wide ones through the ring.  Other rows
// (those that forward_odd leaves): narrow ones a warp each, wide ones staged.  What fits none of these takes three passes over the row.
template <typename T, int V>
void forward_v(const NormParams &p, Stream &st)
{
    const int64_t nvec = cdiv(p.cols, V);
    const bool many = p.rows > 2 * kSms;
    if constexpr (V * sizeof(T) == 16) {
        constexpr int kMost = 32 / V;   // 32 columns a thread
        if (many && nvec > 128 &&
            ((nvec <= 256 && launch_forward_ring<T, V, 1, false>(p, nvec, st)) ||
             (nvec > 256 && nvec <= 512 * kMost && launch_forward_ring<T, V, kMost, false>(p, nvec, st))))
            return;
        if (nvec <= (many ? 32 : 1024))
            return launch_forward<T, V, 1, 1024>(p, nvec, st);
        if (nvec <= 4 * 512)
            return launch_forward<T, V, 4, 512>(p, nvec, st);
        if (nvec <= 4 * 1024)
            return launch_forward<T, V, 4, 1024>(p, nvec, st);
    } else {
        if (nvec <= 32)
            return launch_forward<T, V, 1, 1024>(p, nvec, st);
        if (nvec <= 128)
            return launch_forward<T, V, 4, 512>(p, nvec, st);
        if (launch_forward_staged<T>(p, st))
            return;
    }
    launch(norm_forward_wide_kernel<T>, static_cast<unsigned>(p.rows), kMaxThreads, 0, st, p);
}

template <typename T, int V, int kItems, int kStages, bool kOdd>
bool launch_backward(const NormParams &p, int threads, size_t smem, Stream &st)
{
    auto kernel = norm_backward_kernel<T, V, kItems, kStages, kOdd>;
    if (!allow_smem(kernel, smem))
        return false;
    launch(kernel, static_cast<unsigned>(p.blocks), threads, smem, st, p);
    return true;
}

// Through a ring of 4 slots, or 2 where the rows are wide; false where they are too wide.
template <typename T, int V, int kItems, bool kOdd>
bool backward_ring(NormParams &p, int64_t nvec, Stream &st)
{
    const int threads = ring_threads(nvec, kItems);
    p.blocks = static_cast<int32_t>(std::min<int64_t>(p.rows, static_cast<int64_t>(ring_per_sm(threads, kItems * V)) * kSms));
    const size_t slot = static_cast<size_t>(p.add ? 3 : 2) * kItems * threads * 16;
    const size_t more = V * kItems > 16 ? static_cast<size_t>(kItems) * threads * V * 4 : 0;   // gamma
    const size_t limit = p.blocks <= kSms ? kAloneLimit : kRingLimit;
    p.gamma_smem = 2 * slot + more <= limit;
    if (!kOdd && !p.gamma_smem)
        return 2 * slot <= kRingLimit && launch_backward<T, V, kItems, 2, kOdd>(p, threads, 2 * slot, st);
    if ((4 * slot + more) * cdiv(p.blocks, kSms) <= limit)
        return launch_backward<T, V, kItems, 4, kOdd>(p, threads, 4 * slot + more, st);
    return p.gamma_smem && launch_backward<T, V, kItems, 2, kOdd>(p, threads, 2 * slot + more, st);
}

template <typename T, int V, bool kOdd>
bool backward_rings(NormParams &p, int64_t nvec, Stream &st)
{
    const int items = ring_items(nvec, V);
    if constexpr (V == 4)
        if (items == 8)
            return backward_ring<T, V, 8, kOdd>(p, nvec, st);
    return (items == 1 && backward_ring<T, V, 1, kOdd>(p, nvec, st)) || (items == 2 && backward_ring<T, V, 2, kOdd>(p, nvec, st)) ||
           (items == 4 && backward_ring<T, V, 4, kOdd>(p, nvec, st));
}

template <typename T, int V, int R>
bool backward_staged_r(NormParams &p, int threads, size_t smem, Stream &st)
{
    auto kernel = norm_backward_staged_kernel<T, V, R>;
    if (!allow_smem(kernel, smem))
        return false;
    launch(kernel, static_cast<unsigned>(p.blocks), threads, smem, st, p);
    return true;
}

// Other rows, four at a time where there are enough to keep every SM busy.
template <typename T, int V>
bool backward_staged(NormParams &p, Stream &st)
{
    const int threads = loop_threads(cdiv(p.cols, V), 4, 512);
    if (p.cols > (p.part ? kFusedCols : kLoopCols))
        return false;
    const size_t sums = static_cast<size_t>(p.cols) * 8, smem = p.part ? sums : 0;
    auto most = [&](int r) { return static_cast<int64_t>(staged_per_sm(threads, sums, r)) * kSms; };
    const bool four = p.rows >= 2 * most(4);
    p.blocks = static_cast<int32_t>(four ? std::min(cdiv(p.rows, 4), most(4)) : std::min(p.rows, most(1)));
    return four ? backward_staged_r<T, V, 4>(p, threads, smem, st) : backward_staged_r<T, V, 1>(p, threads, smem, st);
}

template <typename T>
bool backward_odd(NormParams &p, int64_t ld, Stream &st)
{
    constexpr int V = 16 / sizeof(T);
    const NormParams keep = p;
    p.part_ld = odd_words(p.cols, V) * V;
    p.part_step = static_cast<int32_t>(ld & (V - 1));
    p.part_mask = V - 1;
    if (odd_words(p.cols, V) > kOddLeast && backward_rings<T, V, true>(p, odd_words(p.cols, V), st))
        return true;
    p = keep;
    return false;
}

// One kernel for all gradients; false where the rows are too wide for it.  dx alone needs no room for the sums, so any width
// would fit the staged kernel; but rows in 16-byte units are read faster by norm_dx_kernel (256 x 40000 bf16, from cold caches, 21 us,
// staged 40).  Others stay here (4000 x 30002 263 us, there 504).
template <typename T, int V>
bool backward_v(NormParams &p, Stream &st)
{
    if constexpr (V * sizeof(T) == 16) {
        if (backward_rings<T, V, false>(p, cdiv(p.cols, V), st))
            return true;
        if (p.cols > kFusedCols)
            return false;
    }
    return backward_staged<T, V * sizeof(T) == 16 ? (sizeof(T) == 2 ? 2 : 1) : V>(p, st);
}

// Rows wider than a block's registers: the column sums first (dx may overwrite what they read), then dx.
template <typename T, int V>
void backward_wide(NormParams &p, Stream &st)
{
    p.block_rows = std::max<int64_t>(cdiv(p.rows, kColsumBlocks), 8);
    p.blocks = static_cast<int32_t>(cdiv(p.rows, p.block_rows));
    if (p.part)
        launch(norm_colsum_kernel<T, V>, dim3(static_cast<unsigned>(cdiv(p.cols, 32 * V)), static_cast<unsigned>(p.blocks)), 256, 0, st, p);
    if (p.dx)
        launch(norm_dx_kernel<T, V>, static_cast<unsigned>(p.rows), kMaxThreads, 0, st, p);
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
    Stream st{static_cast<cudaStream_t>(stream)};
    p.w_kind = p.w_f32 + (aligned(gamma, 0, wsz, 16) && aligned(beta, 0, wsz, 16) ? 2 : 0);
    auto wide = [&](size_t bytes) {
        return static_cast<size_t>(cols) * esz % bytes == 0 && aligned(x, ldx, esz, bytes) && aligned(y, ldy, esz, bytes);
    };
    const int64_t mod = 16 / static_cast<int64_t>(esz);
    const bool odd = aligned(x, 0, esz, 16) && aligned(y, 0, esz, 16) && ldx % mod == ldy % mod;
    if (dtype == MLP_DT_BF16) {
        if (wide(16))
            forward_v<__nv_bfloat16, 8>(p, st);
        else if (odd && forward_odd<__nv_bfloat16>(p, st))
            ;
        else if (wide(4))
            forward_v<__nv_bfloat16, 2>(p, st);
        else
            forward_v<__nv_bfloat16, 1>(p, st);
    } else if (wide(16)) {
        forward_v<float, 4>(p, st);
    } else if (!(odd && forward_odd<float>(p, st))) {
        forward_v<float, 1>(p, st);
    }
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
}

extern "C" mlp_status mlp_layernorm_workspace_size(int64_t rows, int64_t cols, size_t *bytes)
{
    if (rows < 0 || cols < 1 || !bytes)
        return MLP_ERR_INVALID_ARG;
    const int64_t blocks = cols <= kFusedCols ? std::min<int64_t>(std::max<int64_t>(rows, kColsumBlocks), std::max<int64_t>(most_fused_blocks(cols), kColsumBlocks))
                                              : kColsumBlocks;
    *bytes = static_cast<size_t>(blocks) * 2 * static_cast<size_t>(cols + 14) * 4;   // (row pitch: at most 14 more)
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
    Stream st{static_cast<cudaStream_t>(stream)};
    if (!aligned(dgamma, 0, wsz, wsz) || !aligned(dbeta, 0, wsz, wsz) || !aligned(gamma, 0, wsz, wsz))
        return MLP_ERR_INVALID_ARG;
    const bool want_w = dgamma || dbeta;
    if (rows == 0) {
        if ((dgamma && !succeeded(cudaMemsetAsync(dgamma, 0, static_cast<size_t>(cols) * wsz, st.stream))) ||
            (dbeta && !succeeded(cudaMemsetAsync(dbeta, 0, static_cast<size_t>(cols) * wsz, st.stream))))
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
    p.part = want_w ? static_cast<float *>(workspace) : nullptr;
    p.part_ld = cols;
    auto wide = [&](size_t bytes) {
        return static_cast<size_t>(cols) * esz % bytes == 0 && aligned(x, ldx, esz, bytes) && aligned(dy, lddy, esz, bytes) &&
               aligned(dx, lddx, esz, bytes) && aligned(dx_add, ldadd, esz, bytes);
    };
    const int64_t mod = 16 / static_cast<int64_t>(esz);
    const bool odd = !wide(16) && aligned(x, 0, esz, 16) && aligned(dy, 0, esz, 16) && aligned(dx, 0, esz, 16) &&
                     aligned(dx_add, 0, esz, 16) && ldx % mod == lddy % mod && (!dx || ldx % mod == lddx % mod) &&
                     (!dx_add || ldx % mod == ldadd % mod);
    if (odd && (dtype == MLP_DT_BF16 ? backward_odd<__nv_bfloat16>(p, ldx, st) : backward_odd<float>(p, ldx, st))) {
        // launched
    } else if (dtype == MLP_DT_BF16) {
        if (!(wide(16) ? backward_v<__nv_bfloat16, 8>(p, st) : wide(4) ? backward_v<__nv_bfloat16, 2>(p, st)
                                                                       : backward_v<__nv_bfloat16, 1>(p, st)))
            wide(16) ? backward_wide<__nv_bfloat16, 8>(p, st) : backward_wide<__nv_bfloat16, 1>(p, st);
    } else if (!(wide(16) ? backward_v<float, 4>(p, st) : backward_v<float, 1>(p, st))) {
        wide(16) ? backward_wide<float, 4>(p, st) : backward_wide<float, 1>(p, st);
    }
    if (want_w) {
        if (cols % 4 == 0 && p.part_ld % 4 == 0 && p.part_step == 0)
            launch(norm_colsum_finish_kernel<4, 8>, dim3(static_cast<unsigned>(cdiv(cols, 32)), 2), 256, 0, st, p, dgamma, dbeta);
        else if (p.blocks <= 64)
            launch(norm_colsum_finish_kernel<1, 32>, dim3(static_cast<unsigned>(cdiv(cols, 32)), 2), 256, 0, st, p, dgamma, dbeta);
        else
            launch(norm_colsum_finish_kernel<1, 8>, dim3(static_cast<unsigned>(cdiv(cols, 8)), 2), 256, 0, st, p, dgamma, dbeta);
    }
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
}
