// exchange.cu -- rows between token order and expert order, forward and backward (C ABI in include/mlp_experts.h).
//
//   gather   out[t] = sum_j g[t][j] in[slots[t][j]] + add[t]    combine, and dispatch's gradient (g = 1)
//   scatter  out[slots[t][j]] = g[t][j] in[t]                   dispatch (g = 1), and combine's gradient, which also takes
//            dg[t][j] = sum_c in[t][c] z[slots[t][j]][c]
//
// Copies with a few operations per element: the memory system is the bound.  Both walk the tokens, so a token's row is read or
// written once however many experts it has, and the table that says where its rows are is read along.  A token's rows are found
// through the table, two latencies in a row, so what keeps memory busy is many small blocks, no more registers than let them share
// an SM, and several words of several rows requested together; a grid of as many blocks as run at a time, which fetch the next token's
// entries early, was slower (combine of 4096 x 2048 from four rows 24 us, one block a token 18).
#include <algorithm>

#include "../../include/mlp_experts.h"
#include "elements.cuh"
#include "launch.h"

using namespace mlpc;

namespace {

struct Exchange {
    const void *in, *z, *add;
    void *out;
    const float *gates;
    float *dgates;
    const int32_t *slots;
    int64_t tokens, cols, rows, ldin, ldz, ldadd, ldout;
    int32_t top;
    uint32_t tiles;
};

constexpr int kThreads = 256, kOddThreads = 512, kMostWarps = kOddThreads / 32;
constexpr int kAtOnce = 4;   // rows of a token that are requested together, at most

template <typename T>
constexpr int kWord = 16 / static_cast<int>(sizeof(T));   // elements of 16 bytes

// Where J of a token's rows from the j0-th choice on are (-1: none), and their gates.
template <int J>
struct Choices {
    int32_t at[J];
    float gate[J];

    __device__ __forceinline__ Choices(const Exchange &p, int64_t t, int j0, bool gates)
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = t * p.top + j0 + j;
            at[j] = j0 + j < p.top ? p.slots[i] : -1;
            gate[j] = gates && j0 + j < p.top ? p.gates[i] : 1.0f;
            if (at[j] >= p.rows)
                at[j] = -1;
        }
    }
    __device__ __forceinline__ bool there(int j) const { return at[j] >= 0; }
};

template <typename T>
__device__ __forceinline__ const T *row(const void *base, int64_t i, int64_t ld) { return static_cast<const T *>(base) + i * ld; }
template <typename T>
__device__ __forceinline__ T *row(void *base, int64_t i, int64_t ld) { return static_cast<T *>(base) + i * ld; }

// ---- rows in words of V elements throughout, 16 or 4 bytes.  A block has a tile of a token's row (p.tiles of them), or narrow rows of blockDim.y tokens.
__device__ __forceinline__ int64_t token_of(const Exchange &p) { return static_cast<int64_t>(blockIdx.x / p.tiles) * blockDim.y + threadIdx.y; }

// J rows at once, kItems words a thread.  4096 x 8192 bf16 from two rows each with the residual, 268 MB: 43.6 us, 91 % of the copy rate;
// 4096 x 2048 from four 18.1, 82 %.
template <typename T, int V, int J, int kItems>
__global__ void __launch_bounds__(kThreads, kItems == 1 ? 4 : 5) gather_kernel(const Exchange p)
{
    using R = Raw<T, V>;
    take_turn();
    const int64_t t = kItems == 1 ? token_of(p) : blockIdx.x / p.tiles, step = blockDim.x * V;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * kItems * blockDim.x + threadIdx.x) * V;
    if (t >= p.tokens)
        return;
    R add[kItems] = {};
    if (p.add)
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (c + i * step < p.cols)
                add[i] = *reinterpret_cast<const R *>(row<T>(p.add, t, p.ldadd) + c + i * step);
    float s[kItems][V];
    for (int j0 = 0; j0 < p.top; j0 += J) {
        const Choices<J> now(p, t, j0, p.gates);
        R x[J][kItems] = {};
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (now.there(j))
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (c + i * step < p.cols)
                        x[j][i] = *reinterpret_cast<const R *>(row<T>(p.in, now.at[j], p.ldin) + c + i * step);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (j0 == 0)
                unpack<T>(add[i], s[i]);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (now.there(j)) {
                    float f[V];
                    unpack<T>(x[j][i], f);
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        s[i][v] = fmaf(now.gate[j], f[v], s[i][v]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        if (c + i * step < p.cols)
            store<T, V>(row<T>(p.out, t, p.ldout) + c + i * step, s[i]);
}

// 4096 x 8192 bf16 to two rows each, 201 MB: 30.7 us, 97 % of the copy rate; 2048 x 4096 (50 MB) 9.1, 81 %.
template <typename T, int V, int kItems>
__global__ void __launch_bounds__(kThreads, 8) scatter_kernel(const Exchange p)
{
    using R = Raw<T, V>;
    take_turn();
    const int64_t t = token_of(p), step = blockDim.x * V;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * kItems * blockDim.x + threadIdx.x) * V;
    if (t >= p.tokens)
        return;
    R x[kItems] = {};
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        if (c + i * step < p.cols)
            x[i] = *reinterpret_cast<const R *>(row<T>(p.in, t, p.ldin) + c + i * step);
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        const Choices<kAtOnce> now(p, t, j0, p.gates);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (now.there(j))
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (c + i * step < p.cols) {
                        T *to = row<T>(p.out, now.at[j], p.ldout) + c + i * step;
                        if (p.gates) {
                            float f[V];
                            unpack<T>(x[i], f);
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                f[v] *= now.gate[j];
                            store<T, V>(to, f);
                        } else {
                            *reinterpret_cast<R *>(to) = x[i];
                        }
                    }
    }
}

// Sums of kAtOnce values over a block, for its first threads: thread j has the j-th.  part: one of two buffers in turn, so that one
// barrier a call is enough.
__device__ __forceinline__ float block_sums(const float (&d)[kAtOnce], float (&part)[kAtOnce][kMostWarps])
{
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
        const float s = warp_sum(d[j]);
        if ((threadIdx.x & 31) == 0)
            part[j][threadIdx.x / 32] = s;
    }
    __syncthreads();
    float all = 0.0f;
    if (threadIdx.x < kAtOnce)
        for (unsigned w = 0; w < blockDim.x / 32; ++w)
            all += part[threadIdx.x][w];
    return all;
}

// combine's gradient with the gates': a block a token.  4096 x 8192 bf16 of two rows each, 336 MB: 54.2 us, 91 % of the copy rate.  (Two
// words a thread at once, with half the blocks on an SM: 67 us.)
template <typename T, int V, int kItems>
__global__ void __launch_bounds__(kThreads, 5) scatter_dot_kernel(const Exchange p)
{
    using R = Raw<T, V>;
    __shared__ float part[2][kAtOnce][kMostWarps];
    int turn = 0;
    take_turn();
    const int64_t t = blockIdx.x, step = blockDim.x * V;
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        const Choices<kAtOnce> now(p, t, j0, p.out);
        float d[kAtOnce] = {};
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < p.cols; c += kItems * step) {
            R x[kItems] = {}, z[kAtOnce][kItems] = {};
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (c + i * step < p.cols) {
                    x[i] = *reinterpret_cast<const R *>(row<T>(p.in, t, p.ldin) + c + i * step);
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j)
                        if (now.there(j))
                            z[j][i] = *reinterpret_cast<const R *>(row<T>(p.z, now.at[j], p.ldz) + c + i * step);
                }
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float f[V];
                unpack<T>(x[i], f);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    if (now.there(j) && c + i * step < p.cols) {
                        float g[V];
                        unpack<T>(z[j][i], g);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            d[j] = fmaf(f[v], g[v], d[j]);
                            g[v] = now.gate[j] * f[v];
                        }
                        if (p.out)
                            store<T, V>(row<T>(p.out, now.at[j], p.ldout) + c + i * step, g);
                    }
            }
        }
        const float all = block_sums(d, part[turn]);
        turn ^= 1;
        if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < p.top)
            p.dgates[t * p.top + j0 + threadIdx.x] = all;
    }
}

// ---- rows anywhere (of bf16: any row of fp32 lies in words of 4 bytes).
//
// The gates' gradient: a block a token, a thread a 16-byte word of what is written.  The columns of a word lie across two words of a row
// that is read; both are requested whole and shifted in registers, or read by element where they are not all inside the row.  (The
// second word from the next lane instead: 4096 x 8191 of two rows each 90 us, requested 82.)
template <typename T>
struct Word {
    uint4 x, y;
    uint32_t shift;
    bool whole;

    // The columns c ... c + kWord - 1 of a row.
    __device__ __forceinline__ void request(const T *first, int64_t cols, int64_t c)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(first + c), lo = a & ~uintptr_t{15};
        shift = static_cast<uint32_t>(a & 15);
        whole = lo >= reinterpret_cast<uintptr_t>(first) && lo + (shift ? 32 : 16) <= reinterpret_cast<uintptr_t>(first + cols);
        if (whole) {
            x = reinterpret_cast<const uint4 *>(lo)[0];
            y = reinterpret_cast<const uint4 *>(lo)[shift ? 1 : 0];
        }
    }
    // Where they are whole.
    __device__ __forceinline__ uint4 shifted() const
    {
        uint32_t q[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 6; ++i)
            q[i] = shift & 8 ? q[i + 2] : q[i];
#pragma unroll
        for (int i = 0; i < 5; ++i)
            q[i] = shift & 4 ? q[i + 1] : q[i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = __funnelshift_r(q[i], q[i + 1], (shift & 2) * 8);
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
    // Zeros outside the row.
    __device__ __forceinline__ void values(const T *first, int64_t cols, int64_t c, float (&f)[kWord<T>]) const
    {
        if (whole) {
            unpack<T>(shifted(), f);
        } else {
#pragma unroll
            for (int i = 0; i < kWord<T>; ++i)
                f[i] = c + i >= 0 && c + i < cols ? to_f32<T>(first[c + i]) : 0.0f;
        }
    }
};

template <typename T>
__device__ __forceinline__ void put(T *first, int64_t cols, int64_t c, const float (&f)[kWord<T>])
{
    if (c >= 0 && c + kWord<T> <= cols)
        store<T, kWord<T>>(first + c, f);
    else
#pragma unroll
        for (int i = 0; i < kWord<T>; ++i)
            if (c + i >= 0 && c + i < cols)
                first[c + i] = from_f32<T>(f[i]);
}

// The column of a row's first word: 0, or before it.
template <typename T>
__device__ __forceinline__ int64_t first_column(const T *first)
{
    return -static_cast<int64_t>((reinterpret_cast<uintptr_t>(first) & 15) / sizeof(T));
}

// (Two rows at a time were slower: 4096 x 8191 of two rows each 91 us, one at a time 82; columns read one by one, as below, 142.)
template <typename T, int kMost>
__global__ void __launch_bounds__(kMost) scatter_dot_odd_kernel(const Exchange p)
{
    constexpr int V = kWord<T>;
    __shared__ float part[2][kAtOnce][kMostWarps];
    int turn = 0;
    take_turn();
    const int64_t t = blockIdx.x;
    const T *in = row<T>(p.in, t, p.ldin);
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        const Choices<kAtOnce> now(p, t, j0, p.gates && p.out);
        float d[kAtOnce] = {};
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (!now.there(j))
                continue;
            T *out = p.out ? row<T>(p.out, now.at[j], p.ldout) : nullptr;
            const T *z = row<T>(p.z, now.at[j], p.ldz);
            for (int64_t c = first_column(out ? out : z) + static_cast<int64_t>(threadIdx.x) * V; c < p.cols; c += static_cast<int64_t>(blockDim.x) * V) {
                Word<T> x, y;
                float f[V], g[V];
                x.request(in, p.cols, c);
                y.request(z, p.cols, c);
                x.values(in, p.cols, c, f);
                y.values(z, p.cols, c, g);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    d[j] = fmaf(f[v], g[v], d[j]);
                if (out) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        f[v] *= now.gate[j];
                    put(out, p.cols, c, f);
                }
            }
        }
        const float all = block_sums(d, part[turn]);
        turn ^= 1;
        if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < p.top)
            p.dgates[t * p.top + j0 + threadIdx.x] = all;
    }
}

// The other directions: a thread has pairs of columns that are a 4-byte word of what is written, and reads their columns one by one; so a
// warp's loads are of one line of memory, whatever their place.
struct Pair {
    uint32_t a, b;

    __device__ __forceinline__ void request(const __nv_bfloat16 *row, int64_t cols, int64_t c)   // zeros outside the row
    {
        const unsigned short *p = reinterpret_cast<const unsigned short *>(row);
        a = c >= 0 && c < cols ? p[c] : 0u;
        b = c + 1 < cols ? p[c + 1] : 0u;
    }
    __device__ __forceinline__ uint32_t value() const { return a | b << 16; }
};

__device__ __forceinline__ void put_pair(__nv_bfloat16 *row, int64_t cols, int64_t c, uint32_t v)
{
    unsigned short *p = reinterpret_cast<unsigned short *>(row);
    if (c >= 0 && c + 1 < cols) {
        *reinterpret_cast<uint32_t *>(row + c) = v;
    } else {
        if (c >= 0 && c < cols)
            p[c] = static_cast<unsigned short>(v);
        if (c + 1 >= 0 && c + 1 < cols)
            p[c + 1] = static_cast<unsigned short>(v >> 16);
    }
}

// How far a row's first word of 4 bytes begins before its first column.
__device__ __forceinline__ int back_of(const void *row) { return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 1); }

// (By whole words of what is written, as above: 4096 x 2047 from four rows each 37.5 us, so 28.8; 1000 x 4095 from eight 35, so 24; 4096 x
// 8191 from two 77, so 74.)
template <typename T, int J, int kItems>
__global__ void __launch_bounds__(kThreads, 4) gather_odd_kernel(const Exchange p)
{
    take_turn();
    const int64_t t = blockIdx.x / p.tiles, step = blockDim.x * 2;
    T *out = row<T>(p.out, t, p.ldout);
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * kItems * blockDim.x + threadIdx.x) * 2 - back_of(out);
    Pair add[kItems];
    if (p.add)
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            add[i].request(row<T>(p.add, t, p.ldadd), p.cols, c + i * step);
    float s[kItems][2] = {};
    for (int j0 = 0; j0 < p.top; j0 += J) {
        const Choices<J> now(p, t, j0, p.gates);
        Pair x[J][kItems];
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (now.there(j))
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    x[j][i].request(row<T>(p.in, now.at[j], p.ldin), p.cols, c + i * step);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (j0 == 0 && p.add)
                unpack<T>(add[i].value(), s[i]);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (now.there(j)) {
                    float f[2];
                    unpack<T>(x[j][i].value(), f);
                    s[i][0] = fmaf(now.gate[j], f[0], s[i][0]);
                    s[i][1] = fmaf(now.gate[j], f[1], s[i][1]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        put_pair(out, p.cols, c + i * step, pack_bf16(s[i][0], s[i][1]));
}

// A thread has columns of a token and writes them as words of 4 bytes wherever a row's words begin.  (By whole words of what is written, as
// above: 4096 x 2047 to four rows each 24 us, so 18.6; 1000 x 4095 to eight 25, so 16; 4096 x 8191 to two 41, so 44.)
template <typename T, int kItems>
__global__ void __launch_bounds__(kThreads, 8) scatter_odd_kernel(const Exchange p)
{
    take_turn();
    const int64_t t = blockIdx.x / p.tiles, step = blockDim.x * 2;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.tiles) * kItems * blockDim.x + threadIdx.x) * 2;
    const unsigned short *in = reinterpret_cast<const unsigned short *>(row<T>(p.in, t, p.ldin));
    // the columns c - 1, c and c + 1: a word of what is written is the first two or the last two
    uint32_t x[kItems][3] = {};
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int n = 0; n < 3; ++n)
            if (c + i * step + n - 1 >= 0 && c + i * step + n - 1 < p.cols)
                x[i][n] = in[c + i * step + n - 1];
    for (int j0 = 0; j0 < p.top; j0 += kAtOnce) {
        const Choices<kAtOnce> now(p, t, j0, p.gates);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (now.there(j)) {
                T *out = row<T>(p.out, now.at[j], p.ldout);
                const int back = back_of(out);
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    uint32_t v = back ? x[i][0] | x[i][1] << 16 : x[i][1] | x[i][2] << 16;
                    if (p.gates)
                        v = pack_bf16(now.gate[j] * bf16_lo(v), now.gate[j] * bf16_hi(v));
                    put_pair(out, p.cols, c + i * step - back, v);
                }
            }
    }
}

// Few tokens leave SMs idle: then a row of the gates' gradient has more threads (333 rows of 1357, fp32 in this kernel, of three each 8.9 us,
// 7.1 so; 4096 of 8191 bf16 76, 105 so).
constexpr int64_t kFewTokens = 4 * kSms;

template <typename T>
void run_odd(bool gather, Exchange &p, Stream &st)
{
    if (!gather && p.dgates) {
        const bool few = p.tokens <= kFewTokens;
        const int64_t words = cdiv(p.cols, kWord<T>) + 1, rounds = cdiv(words, few ? kOddThreads : kThreads);
        return launch(few ? scatter_dot_odd_kernel<T, kOddThreads> : scatter_dot_odd_kernel<T, kThreads>, static_cast<unsigned>(p.tokens),
                      static_cast<unsigned>(cdiv(cdiv(words, rounds), 32) * 32), 0, st, p);
    }
    constexpr int kItems = 4;
    const int64_t pairs = p.cols / 2 + 1, rounds = cdiv(pairs, kItems * kThreads), threads = cdiv(cdiv(pairs, rounds * kItems), 32) * 32;
    p.tiles = static_cast<uint32_t>(cdiv(pairs, kItems * threads));
    launch(gather ? gather_odd_kernel<T, 2, kItems> : scatter_odd_kernel<T, kItems>, static_cast<unsigned>(p.tokens * p.tiles),
           static_cast<unsigned>(threads), 0, st, p);
}

// Rows in words of 16 bytes.
template <typename T>
void run_words(bool gather, Exchange &p, Stream &st)
{
    constexpr int V = kWord<T>;
    const int64_t words = p.cols / V;
    if (!gather && p.dgates) {
        const int64_t threads = std::min<int64_t>(kThreads, cdiv(words, 32) * 32);
        return launch(scatter_dot_kernel<T, V, 1>, static_cast<unsigned>(p.tokens), static_cast<unsigned>(threads), 0, st, p);
    }
    // Two words of each of two rows a thread, or narrow rows: 4096 x 8192 of two rows each 43.5 us, one word 48; of four rows (4096 x 2048)
    // 18.1, one word of all four 20.
    const bool two = gather && words > 64;
    const int64_t threads = std::min<int64_t>(kThreads, cdiv(cdiv(words, two ? 2 : 1), 32) * 32);
    const dim3 block(static_cast<unsigned>(threads), static_cast<unsigned>(two ? 1 : std::min<int64_t>(kThreads / threads, p.tokens)));
    p.tiles = static_cast<uint32_t>(cdiv(words, (two ? 2 : 1) * threads));
    const unsigned grid = static_cast<unsigned>(cdiv(p.tokens, block.y) * p.tiles);
    launch(!gather ? scatter_kernel<T, V, 1> : two ? gather_kernel<T, V, 2, 2> : gather_kernel<T, V, 4, 1>, grid, block, 0, st, p);
}

// Rows in words of 4 bytes, which a warp reads as fast as larger ones: several a thread, or narrow rows of several tokens a block.  (Found
// across words of 16 bytes, as odd rows are: 4096 x 2046 bf16 of four rows each 37 us, so 25.)
template <typename T>
void run_small_words(bool gather, Exchange &p, Stream &st)
{
    constexpr int V = 4 / static_cast<int>(sizeof(T)), kItems = 4, kDotItems = 3;
    const int64_t words = p.cols / V;
    if (!gather && p.dgates) {
        const int64_t rounds = cdiv(words, kDotItems * kThreads), threads = cdiv(cdiv(words, rounds * kDotItems), 32) * 32;
        return launch(scatter_dot_kernel<T, V, kDotItems>, static_cast<unsigned>(p.tokens), static_cast<unsigned>(threads), 0, st, p);
    }
    const bool narrow = words <= 128;   // (16384 rows of 70 fp32 to eight each: 17.6 us in blocks of one token, 13.7)
    const int64_t items = narrow ? 1 : kItems, rounds = cdiv(words, items * kThreads), threads = cdiv(cdiv(words, rounds * items), 32) * 32;
    const dim3 block(static_cast<unsigned>(threads), static_cast<unsigned>(narrow ? std::min<int64_t>(kThreads / threads, p.tokens) : 1));
    p.tiles = static_cast<uint32_t>(cdiv(words, items * threads));
    auto kernel = gather ? gather_kernel<T, V, 2, kItems> : scatter_kernel<T, V, kItems>;
    if (narrow)
        kernel = gather ? gather_kernel<T, V, 4, 1> : scatter_kernel<T, V, 1>;
    launch(kernel, static_cast<unsigned>(cdiv(p.tokens, block.y) * p.tiles), block, 0, st, p);
}

template <typename T>
void run(bool gather, int word, Exchange &p, Stream &st)
{
    p.tiles = 1;
    if (word == 16)
        run_words<T>(gather, p, st);
    else if (word == 4)
        run_small_words<T>(gather, p, st);
    else if constexpr (sizeof(T) == 2)
        run_odd<T>(gather, p, st);
}

bool bad_sizes(int64_t tokens, int64_t cols, int32_t top, int64_t rows)
{
    return tokens < 0 || rows < 0 || rows >= (int64_t{1} << 31) || cols < 1 || cols >= (int64_t{1} << 31) || top < 1 || top > MLP_MAX_TOP ||
           tokens > ((int64_t{1} << 31) - 1) / top;
}

mlp_status start(bool gather, Exchange &p, mlp_dtype dtype, void *stream)
{
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    auto in_words = [&](size_t bytes) {
        return static_cast<size_t>(p.cols) * esz % bytes == 0 && aligned(p.in, p.ldin, esz, bytes) && aligned(p.z, p.ldz, esz, bytes) &&
               aligned(p.add, p.ldadd, esz, bytes) && aligned(p.out, p.ldout, esz, bytes);
    };
    const int word = in_words(16) ? 16 : in_words(4) ? 4 : 2;
    if (p.tokens * cdiv(p.cols, 32 * 4 / static_cast<int64_t>(esz)) >= int64_t{1} << 31)
        return MLP_ERR_INVALID_ARG;
    Stream st{static_cast<cudaStream_t>(stream)};
    dtype == MLP_DT_BF16 ? run<__nv_bfloat16>(gather, word, p, st) : run<float>(gather, word, p, st);
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
}

}  // namespace

extern "C" mlp_status mlp_dispatch_forward(int64_t tokens, int64_t cols, int32_t top, const void *x, int64_t ldx, mlp_dtype dtype,
                                           const int32_t *slots, int64_t rows, void *y, int64_t ldy, void *stream)
{
    if (bad_sizes(tokens, cols, top, rows))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    if (tokens == 0 || rows == 0)
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if (bad_rows(x, ldx, cols, esz) || bad_rows(y, ldy, cols, esz) || !slots || !aligned(slots, 0, 4, 4))
        return MLP_ERR_INVALID_ARG;
    Exchange p = {};
    p.in = x;
    p.ldin = ldx;
    p.out = y;
    p.ldout = ldy;
    p.slots = slots;
    p.tokens = tokens;
    p.cols = cols;
    p.rows = rows;
    p.top = top;
    return start(false, p, dtype, stream);
}

extern "C" mlp_status mlp_dispatch_backward(int64_t tokens, int64_t cols, int32_t top, const void *dy, int64_t lddy, mlp_dtype dtype,
                                            const int32_t *slots, int64_t rows, const void *dx_add, int64_t ldadd, void *dx, int64_t lddx,
                                            void *stream)
{
    if (bad_sizes(tokens, cols, top, rows))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    if (tokens == 0)
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if ((rows && bad_rows(dy, lddy, cols, esz)) || bad_rows(dx, lddx, cols, esz) || (dx_add && bad_rows(dx_add, ldadd, cols, esz)) ||
        !slots || !aligned(slots, 0, 4, 4))
        return MLP_ERR_INVALID_ARG;
    Exchange p = {};
    p.in = rows ? dy : nullptr;
    p.ldin = lddy;
    p.add = dx_add;
    p.ldadd = ldadd;
    p.out = dx;
    p.ldout = lddx;
    p.slots = slots;
    p.tokens = tokens;
    p.cols = cols;
    p.rows = rows;
    p.top = top;
    return start(true, p, dtype, stream);
}

extern "C" mlp_status mlp_combine_forward(int64_t tokens, int64_t cols, int32_t top, const void *z, int64_t ldz, mlp_dtype dtype,
                                          const float *gates, const int32_t *slots, int64_t rows, const void *residual, int64_t ldr, void *y,
                                          int64_t ldy, void *stream)
{
    if (bad_sizes(tokens, cols, top, rows))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    if (tokens == 0)
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if ((rows && bad_rows(z, ldz, cols, esz)) || bad_rows(y, ldy, cols, esz) || (residual && bad_rows(residual, ldr, cols, esz)) ||
        !slots || !aligned(slots, 0, 4, 4) || !gates || !aligned(gates, 0, 4, 4))
        return MLP_ERR_INVALID_ARG;
    Exchange p = {};
    p.in = rows ? z : nullptr;
    p.ldin = ldz;
    p.add = residual;
    p.ldadd = ldr;
    p.out = y;
    p.ldout = ldy;
    p.gates = gates;
    p.slots = slots;
    p.tokens = tokens;
    p.cols = cols;
    p.rows = rows;
    p.top = top;
    return start(true, p, dtype, stream);
}

extern "C" mlp_status mlp_combine_backward(int64_t tokens, int64_t cols, int32_t top, const void *dy, int64_t lddy, const void *z,
                                           int64_t ldz, mlp_dtype dtype, const float *gates, const int32_t *slots, int64_t rows, void *dz,
                                           int64_t lddz, float *dgates, void *stream)
{
    if (bad_sizes(tokens, cols, top, rows))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    if (tokens == 0 || (!dz && !dgates))
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if (bad_rows(dy, lddy, cols, esz) || (dgates && rows && bad_rows(z, ldz, cols, esz)) || (dz && rows && bad_rows(dz, lddz, cols, esz)) ||
        !slots || !aligned(slots, 0, 4, 4) || !aligned(dgates, 0, 4, 4) || (dz && (!gates || !aligned(gates, 0, 4, 4))))
        return MLP_ERR_INVALID_ARG;
    Exchange p = {};
    p.in = dy;
    p.ldin = lddy;
    p.z = dgates && rows ? z : nullptr;
    p.ldz = ldz;
    p.out = rows ? dz : nullptr;
    p.ldout = lddz;
    p.gates = gates;
    p.dgates = dgates;
    p.slots = slots;
    p.tokens = tokens;
    p.cols = cols;
    p.rows = rows;
    p.top = top;
    return start(false, p, dtype, stream);
}
