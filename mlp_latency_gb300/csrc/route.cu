// route.cu -- the router of the products by expert: top choices, gates, rows in expert order and the balance loss, and the
// gradient of the logits (C ABI in include/mlp_experts.h).
//
// Per token: p = softmax(l); choices are the largest l; gate = p or p / sum of the chosen p.  Over tokens: the choices of each
// expert are counted, every choice gets the next row of its expert in token order, and
//   loss = E k / M^2 sum_e counts_e P_e,  P_e = sum_t p_te,  M = sum_e counts_e.
// Backward, with g_e = dloss E k counts_e / M^2 (+ dgate at a chosen e, without normalize):
//   dl = p (g - sum_e g_e p_e) (+ gate (dgate - sum gate dgate) at the chosen ones, with normalize).
//
// A few instructions per logit and a table of counts: what bounds it is latency for few tokens (one to 2 of 8 experts 2.4 us, of
// which an empty launch is 2.3; 2048 in one launch 4.5) and the rate of instructions for many (8192 to 8 of 256, 4.2 MB of logits,
// 14.4 us, or 13.5 where the same logits are read again and L2 has them: 6.3 million instructions of a warp, some 560 a token of 256
// experts, at half the rate of issue; then 2.3 us of the second launch).  A group of lanes takes a token, 8 experts a lane (16 or 32
// where there are more than 256), so a warp has up to 32 tokens at a time.  The rows are a counting sort: a warp ranks its tokens'
// choices, a block adds its warps' counts up, a cluster its blocks', and a second launch the clusters' (none where one cluster has all
// tokens).  The times below are of calls in a row with the same logits.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "../../include/mlp_experts.h"
#include "elements.cuh"
#include "launch.h"

using namespace mlpc;

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kCluster = 8;           // blocks that add their counts up through each other's shared memory
// Clusters of a launch: as many as run at a time on the one device there is code for (of 512 threads with 64 registers two blocks share
// an SM, with more one); where fewer ran, the others would come after them.  8192 tokens to 8 of 256 experts: 20 clusters 21.0 us,
// 30 16.8, 32 18.6; 4096 tokens to 8 of 512: 12 18.9, 15 17.6, 18 27.2.
constexpr int kMostClusters = 30, kMostWideClusters = 15;
constexpr int kStageBytes = 48 * 1024;   // a block's choices, kept until their rows are known
constexpr int kPlaceThreads = 1024;
// Tables of 16 warps x 512 experts or 8 x 1024, two of 8 blocks x 1024, and what is staged: kStageBytes, or one step of 16 warps x 256
// choices.
constexpr int kRouteSmem = 2 * 4 * 8192 + 2 * 4 * kCluster * MLP_MAX_EXPERTS + kStageBytes;
constexpr uint32_t kLeast = 0x00800000u;   // the key of the lowest finite value
constexpr uint32_t kUnknown = 1;           // no key

struct Route {
    const void *logits;
    const uint8_t *mask;
    float *gates, *loss;
    int32_t *chosen, *slots, *offsets, *counts;
    int32_t *hist;   // [clusters][experts]: choices of each cluster
    float *part;     // likewise: sums of p
    int64_t tokens, ldl, tokens_of_cluster;
    int32_t experts, top, normalize, clusters, warps, steps, staged, split;
};

// Logits in the order of their values, NaN first of all; -inf, which is never chosen, below kLeast.  (The sum makes -0 0 and any
// NaN the positive one.)
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key ^ (static_cast<uint32_t>(static_cast<int32_t>(~key) >> 31) | 0x80000000u));
}

// A lane's N experts, from e0 on, and the best two of them that are not chosen yet.  After two wins of a lane its next two are
// found again; that is rare, so a round costs a few instructions instead of a pass over N.
//
// fp32: the order is that of the keys, of equal ones that of the places.
template <typename T, int N>
struct Choice {
    uint32_t key[N], first, second;   // second: kUnknown after a win
    int at = 0, at2 = 0;

    __device__ __forceinline__ void look()
    {
        first = second = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool a = key[i] > first, b = key[i] > second;
            second = a ? first : b ? key[i] : second;
            at2 = a ? at : b ? i : at2;
            first = a ? key[i] : first;
            at = a ? i : at;
        }
    }
    __device__ __forceinline__ Choice(const float (&l)[N], int)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            key[i] = order_of(l[i]);
        look();
    }
    __device__ __forceinline__ int expert(int e0) const { return e0 + at; }
    // Where its first, of key `most`, was chosen (won), a lane goes on to its next.
    __device__ __forceinline__ void next(bool won, uint32_t most)
    {
        const int was = at;
        first = won ? second : first;
        at = won ? at2 : at;
        second = won ? kUnknown : second;
        if (first == kUnknown) {
            // what is chosen is what comes before this one: higher, or equal and no later
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (key[i] > most || (key[i] == most && i <= was))
                    key[i] = 0;
            look();
        }
    }
    static __device__ __forceinline__ float value(uint32_t most) { return value_of(most); }
};

// bf16: the upper 16 bits of a key say it all, and the lower ones hold the expert, so keys differ and the highest is the winner.
template <int N>
struct Choice<__nv_bfloat16, N> {
    uint32_t key[N], first, second;

    __device__ __forceinline__ int expert(int) const { return 0xffff - static_cast<int>(first & 0xffffu); }
    template <bool kAllOfThem>
    __device__ __forceinline__ void look(uint32_t below)
    {
        first = second = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t k = kAllOfThem || key[i] < below ? key[i] : 0;
            second = max(second, min(first, k));
            first = max(first, k);
        }
    }
    __device__ __forceinline__ Choice(const float (&l)[N], int e0)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            key[i] = (order_of(l[i]) & 0xffff0000u) | static_cast<uint32_t>(0xffff - (e0 + i));
        look<true>(0);
    }
    __device__ __forceinline__ void next(bool won, uint32_t most)
    {
        first = won ? second : first;
        second = won ? kUnknown : second;
        if (first == kUnknown)
            look<false>(most);
    }
    static __device__ __forceinline__ float value(uint32_t most)
    {
        return value_of(most & 0x80000000u ? (most >= 0xffff0000u ? kAll : most & 0xffff0000u) : most | 0xffffu);
    }
};

// A lane's N logits of a token as they are in memory, in loads of V; -inf where there is no expert.
template <typename T, int N, int V>
struct Logits {
    Raw<T, V> r[N / V];

    __device__ __forceinline__ Logits()
    {
        float none[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            none[i] = __uint_as_float(0xff800000u);
#pragma unroll
        for (int q = 0; q < N / V; ++q)
            store<T, V>(reinterpret_cast<T *>(&r[q]), none);
    }
    __device__ __forceinline__ void load(const T *row, int e0, int experts)
    {
#pragma unroll
        for (int q = 0; q < N / V; ++q)
            if (e0 + q * V < experts)
                r[q] = *reinterpret_cast<const Raw<T, V> *>(row + e0 + q * V);
    }
    __device__ __forceinline__ void values(float (&l)[N]) const
    {
#pragma unroll
        for (int q = 0; q < N / V; ++q) {
            float x[V];
            unpack<T>(r[q], x);
#pragma unroll
            for (int i = 0; i < V; ++i)
                l[q * V + i] = x[i];
        }
    }
};

// Exclusive sums of total[0 .. experts) in place, by all threads of a block (a multiple of 32), as many experts at a time; returns the sum
// of all.  Starts and ends with the block in step.
__device__ __forceinline__ int32_t scan_experts(int32_t *total, int experts)
{
    __shared__ int32_t of_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    int32_t carry = 0;
    for (int e0 = 0; e0 < experts; e0 += blockDim.x) {
        __syncthreads();
        const int e = e0 + threadIdx.x;
        const int32_t own = e < experts ? total[e] : 0;
        int32_t v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(kAll, v, o);
            if (lane >= o)
                v += u;
        }
        if (lane == 31)
            of_warp[warp] = v;
        __syncthreads();
        int32_t t = lane < warps ? of_warp[lane] : 0;
        const int32_t before = __reduce_add_sync(kAll, lane < warp ? t : 0);
        t = __reduce_add_sync(kAll, t);
        if (e < experts)
            total[e] = carry + before + v - own;
        carry += t;
    }
    __syncthreads();
    return carry;
}

// What is known when all choices are counted: first[e] the first row of e, all of them, sums[e] the sum of its p.  A block.
__device__ __forceinline__ void finish(const Route &p, const int32_t *first, int32_t all, const float *sums)
{
    __shared__ float of_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    float s = 0.0f;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        const int32_t n = (e + 1 < p.experts ? first[e + 1] : all) - first[e];
        p.offsets[e] = first[e];
        if (p.counts)
            p.counts[e] = n;
        if (p.loss)
            s += static_cast<float>(n) * sums[e];
    }
    if (threadIdx.x == 0)
        p.offsets[p.experts] = all;
    if (p.loss) {
        s = warp_sum(s);
        if (lane == 0)
            of_warp[warp] = s;
        __syncthreads();
        if (warp == 0) {
            s = warp_sum(lane < static_cast<int>(blockDim.x) / 32 ? of_warp[lane] : 0.0f);
            const float m = static_cast<float>(all);
            if (lane == 0)
                *p.loss = all ? s / m * (static_cast<float>(p.experts) * static_cast<float>(p.top) / m) : 0.0f;
        }
    }
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (G == 32) {
        return __reduce_max_sync(kAll, v);
    } else {
#pragma unroll
        for (int o = 1; o < G; o <<= 1)
            v = max(v, __shfl_xor_sync(kAll, v, o));
        return v;
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = 1; o < G; o <<= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Up to 32 tokens (8 where there are more than 256 experts) in one block, a warp each: which tokens chose an expert is a word, so a row
// is a count of bits.  All of it is latency: one token to 2 of 8 experts 2.4 us, 32 tokens 3.3 (route_kernel: 4.0 and 4.1).
template <typename T, int N>
__global__ void __launch_bounds__(N <= 8 ? 1024 : 256) route_few_kernel(const Route p)
{
    extern __shared__ float of_token[];   // [tokens][experts]: p, where the loss is wanted
    __shared__ uint32_t tokens_of[MLP_MAX_EXPERTS];
    __shared__ int32_t first[MLP_MAX_EXPERTS];
    __shared__ float sums[MLP_MAX_EXPERTS];
    const int t = threadIdx.x / 32, lane = threadIdx.x & 31, E = p.experts, k = p.top, e0 = lane * N;
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        tokens_of[e] = 0;
    take_turn();
    const int tokens = static_cast<int>(p.tokens);
    Logits<T, N, 1> l;
    bool real = t < tokens;
    if (real) {
        l.load(static_cast<const T *>(p.logits) + t * p.ldl, e0, E);
        real = !p.mask || p.mask[t];
    }
    float x[N];
    l.values(x);
    __syncthreads();
    Choice<T, N> left(x, e0);
    uint32_t most = __reduce_max_sync(kAll, real ? left.first : 0u), my_key = 0;
    const bool any = most >= kLeast;
    int32_t mine = -1;
    float gate = 0.0f, all = 0.0f;
    if (any) {
        const float top = left.value(most);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = expf(x[i] - top);
            all += x[i];
        }
        all = warp_sum(all);
        for (int j = 0; j < k && most >= kLeast; ++j) {
            const int winner = __ffs(__ballot_sync(kAll, left.first == most)) - 1;
            const int32_t e = __shfl_sync(kAll, left.expert(e0), winner);
            if (lane == j) {
                mine = e;
                my_key = most;
            }
            left.next(lane == winner, most);
            most = __reduce_max_sync(kAll, left.first);
        }
        gate = mine >= 0 ? expf(left.value(my_key) - top) : 0.0f;
        const float sum = p.normalize ? warp_sum(gate) : all;
        gate = mine >= 0 ? gate / sum : 0.0f;   // (the sum may be NaN)
    }
    if (p.loss)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (t < tokens && e0 + i < E)
                of_token[t * E + e0 + i] = any ? x[i] / all : 0.0f;
    if (mine >= 0)
        atomicOr(&tokens_of[mine], 1u << t);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float s = 0.0f;
        if (p.loss)
            for (int i = 0; i < tokens; ++i)
                s += of_token[i * E + e];
        first[e] = __popc(tokens_of[e]);
        sums[e] = s;
    }
    const int32_t of_all = scan_experts(first, E);
    if (t < tokens && lane < k) {
        p.gates[t * k + lane] = gate;
        p.chosen[t * k + lane] = mine;
        p.slots[t * k + lane] = mine >= 0 ? first[mine] + __popc(tokens_of[mine] & ((1u << t) - 1)) : -1;
    }
    finish(p, first, of_all, sums);
}

template <int N>
constexpr int kRouteThreads = N <= 16 ? 512 : 256;   // 64 registers a thread with 8 experts a lane: two blocks per SM

// What a block's shared memory holds, in this order (4-byte cells).
struct RouteCells {
    int count, sum, counts_of, sums_of, stage, all;
};
__host__ __device__ inline RouteCells route_cells(int warps, int experts, int pairs)
{
    RouteCells c;
    c.count = 0;                                           // [warps][experts]: choices
    c.sum = warps * experts;                               // [warps][experts]: sums of p
    c.counts_of = 2 * warps * experts;                     // [kCluster][experts]: choices of the cluster's blocks
    c.sums_of = c.counts_of + kCluster * experts;          // [kCluster][experts]: their sums of p, as far as this block adds them up
    c.stage = c.sums_of + kCluster * experts;              // [3][warps][pairs]: experts, gates, ranks
    c.all = c.stage + 3 * warps * pairs;
    return c;
}

// The choices of a block's tokens, 32 / G tokens of a warp at a time.  Where there is one cluster (or one block) this is all;
// otherwise it leaves in slots the row within the cluster's rows of its expert, and place_kernel follows.
template <typename T, int N, int G, int V>
__global__ void __launch_bounds__(kRouteThreads<N>, N <= 8 ? 2 : 1) route_kernel(const Route p)
{
    extern __shared__ int32_t smem[];
    __shared__ int32_t base[MLP_MAX_EXPERTS], first[MLP_MAX_EXPERTS];
    __shared__ float sums[MLP_MAX_EXPERTS];
    namespace cg = cooperative_groups;
    constexpr int kTokens = 32 / G;
    constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31, E = p.experts, k = p.top;
    const int member = lane % G, group = lane / G, e0 = member * N;
    const uint32_t lower = ((1u << lane) - 1) & ~((1u << group * G) - 1);   // the lanes before this one in its group
    const int pairs = kTokens * k * (p.staged ? p.steps : 1);
    const RouteCells cells = route_cells(warps, E, pairs);
    int32_t *count = smem + cells.count, *my_count = count + warp * E;
    float *sum = reinterpret_cast<float *>(smem + cells.sum);
    int32_t *st_expert = smem + cells.stage + warp * pairs, *st_rank = st_expert + 2 * warps * pairs;
    float *st_gate = reinterpret_cast<float *>(st_expert + warps * pairs);
    auto cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    if (blocks > 1)
        (void)cluster.barrier_arrive();   // this block is there: the others may write to its shared memory
    for (int e = lane; e < E; e += 32)
        my_count[e] = 0;
    __syncwarp();
    float acc[N] = {};
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * warps + warp) * p.steps * kTokens, t1 = min(t0 + p.steps * kTokens, p.tokens);
    const T *logits = static_cast<const T *>(p.logits);
    Logits<T, N, V> next;
    bool next_real = false;
    auto request = [&](int64_t t) {
        next_real = t < t1;
        if (next_real) {
            next.load(logits + t * p.ldl, e0, E);
            if (p.mask)
                next_real = p.mask[t];
        }
    };
    // The ranks of pairs in their order: 32 at a time, equal experts by the lanes before.
    auto rank_pairs = [&](const int32_t *expert, int32_t *rank_of, int n) {
        for (int q0 = 0; q0 < n; q0 += 32) {
            const int q = q0 + lane;
            const int32_t e = q < n ? expert[q] : -1;
            const uint32_t peers = __match_any_sync(kAll, e), lower = peers & ((1u << lane) - 1);
            const int32_t r = e >= 0 ? my_count[e] + __popc(lower) : -1;
            __syncwarp();
            if (e >= 0 && (peers >> lane) == 1u)   // the last of them
                my_count[e] = r + 1;
            if (q < n)
                rank_of[q] = r;
            __syncwarp();
        }
    };
    take_turn();
    request(t0 + group);
    for (int64_t t = t0; t < t1; t += kTokens) {
        float x[N];
        const bool real = next_real;
        next.values(x);
        request(t + kTokens + group);
        Choice<T, N> left(x, e0);
        if (!real)
            left.first = 0;
        uint32_t most = group_max<G>(left.first);
        const bool any = most >= kLeast;
        const float top = left.value(most);
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = expf(x[i] - top);
            all += x[i];
        }
        all = group_sum<G>(all);
        if (p.loss && any) {
            const float scale = 1.0f / all;
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] = fmaf(x[i], scale, acc[i]);
        }
        int found = 0;   // choices made
        uint32_t *key_of = reinterpret_cast<uint32_t *>(st_gate + group * k);   // (until all are known)
        int32_t *expert_of = st_expert + group * k;
#pragma unroll (N <= 16 ? 4 : 2)
        for (int j = 0; j < k; ++j) {
            const bool there = most >= kLeast;
            bool won = there && left.first == most;
            if constexpr (!kBf16 && G > 1) {   // of equal ones the lowest lane, which has the lowest experts
                const uint32_t equal = __ballot_sync(kAll, won);   // (by all lanes: not within the condition)
                won = won && (equal & lower) == 0;
            }
            if (won) {
                key_of[j] = most;
                if constexpr (!kBf16)
                    expert_of[j] = left.expert(e0);
            }
            found += there;
            left.next(won, most);
            most = group_max<G>(left.first);
        }
        __syncwarp();
        float chosen = 0.0f;
        for (int j = member; j < k; j += G) {
            const int at = group * k + j;
            const uint32_t key = key_of[j];
            const float gate = j < found ? expf(left.value(key) - top) : 0.0f;
            st_gate[at] = gate;
            if (kBf16 || j >= found)
                st_expert[at] = j < found ? 0xffff - static_cast<int>(key & 0xffffu) : -1;
            chosen += gate;
        }
        if (p.normalize)
            all = group_sum<G>(chosen);
        const float scale = 1.0f / all;
        for (int j = member; j < found; j += G)
            st_gate[group * k + j] *= scale;
        __syncwarp();
        if (p.staged) {   // their ranks are found when there are more of them
            st_expert += kTokens * k;
            st_gate += kTokens * k;
        } else {
            const int here = static_cast<int>(min(static_cast<int64_t>(kTokens), t1 - t)) * k;
            rank_pairs(st_expert, st_rank, here);
            for (int q = lane; q < here; q += 32) {
                p.gates[t * k + q] = st_gate[q];
                p.chosen[t * k + q] = st_expert[q];
                p.slots[t * k + q] = st_rank[q];
            }
            __syncwarp();
        }
    }
    if (p.staged) {
        st_expert = smem + cells.stage + warp * pairs;
        st_gate = reinterpret_cast<float *>(st_expert + warps * pairs);
        rank_pairs(st_expert, st_rank, static_cast<int>(max(t1 - t0, int64_t{0})) * k);
    }
    if (p.loss) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int o = G; o < 32; o <<= 1)
                acc[i] += __shfl_xor_sync(kAll, acc[i], o);
            if (group == 0 && e0 + i < E)
                sum[warp * E + e0 + i] = acc[i];
        }
    }
    __syncthreads();
    // Per expert: the warps before each; all of them, which every block of the cluster is told; and the sums of p, for the block that
    // adds them up.  Those are other threads' work, as far as there are others.
    if (blocks > 1)
        cluster.barrier_wait();
    const int other = threadIdx.x < blockDim.x / 2 ? threadIdx.x + (blockDim.x + 1) / 2 : threadIdx.x - blockDim.x / 2;
    const int each = p.clusters == 1 ? E : (E + kCluster - 1) / kCluster;   // experts whose sums a block adds up
    int32_t *counts_of = smem + cells.counts_of;
    float *sums_of = reinterpret_cast<float *>(smem + cells.sums_of);
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t n = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            int32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m[i] = w0 + i < warps ? count[(w0 + i) * E + e] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (w0 + i < warps) {
                    count[(w0 + i) * E + e] = n;
                    n += m[i];
                }
        }
        int32_t *to = counts_of + rank * E + e;
        if (blocks > 1)
#pragma unroll
            for (int r = 0; r < kCluster; ++r)
                *cluster.map_shared_rank(to, r) = n;
        else
            *to = n;
    }
    if (p.loss)
        for (int e = other; e < E; e += blockDim.x) {
            float s = 0.0f;
            for (int w0 = 0; w0 < warps; w0 += 8)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s += w0 + i < warps ? sum[(w0 + i) * E + e] : 0.0f;
            float *to = sums_of + rank * E + e;
            *(blocks > 1 ? cluster.map_shared_rank(to, e / each) : to) = s;
        }
    blocks > 1 ? cluster.sync() : __syncthreads();
    // the blocks before this one in the cluster, and all of them
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t n = 0, before = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r)
            if (r < blocks) {
                const int32_t v = counts_of[r * E + e];
                before += r < rank ? v : 0;
                n += v;
            }
        base[e] = before;
        first[e] = n;
        if (p.clusters > 1 && e / each == rank)
            p.hist[static_cast<int>(blockIdx.x) / kCluster * E + e] = n;
    }
    if (p.loss)
        for (int e = other + rank * each; e < min((rank + 1) * each, E); e += blockDim.x) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < kCluster; ++r)
                if (r < blocks)
                    s += sums_of[r * E + e];
            if (p.clusters > 1)
                p.part[static_cast<int>(blockIdx.x) / kCluster * E + e] = s;
            else
                sums[e] = s;
        }
    if (p.clusters == 1) {
        const int32_t all_of_them = scan_experts(first, E);
        if (rank == 0)
            finish(p, first, all_of_them, sums);
        for (int e = threadIdx.x; e < E; e += blockDim.x)
            base[e] += first[e];
    }
    __syncthreads();
    if (p.staged) {
        const int n = static_cast<int>(max(t1 - t0, int64_t{0})) * k;
        for (int q = lane; q < n; q += 32) {
            const int32_t e = st_expert[q];
            p.gates[t0 * k + q] = st_gate[q];
            p.chosen[t0 * k + q] = e;
            p.slots[t0 * k + q] = e >= 0 ? st_rank[q] + my_count[e] + base[e] : -1;
        }
    } else {
        for (int64_t i = t0 * k + lane; i < t1 * k; i += 32) {
            const int32_t e = p.chosen[i];
            if (e >= 0)
                p.slots[i] += my_count[e] + base[e];
        }
    }
}

// Rows within clusters to rows of all: a block adds up what the clusters before its own chose, a thread an expert's counts.
// p.split blocks share a cluster's tokens.  The last block has none and writes the offsets, counts and the loss.
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const Route p)
{
    __shared__ int32_t first[MLP_MAX_EXPERTS], before[MLP_MAX_EXPERTS];
    __shared__ float sums[MLP_MAX_EXPERTS];
    constexpr int kAhead = 2;
    const int E = p.experts, mine = static_cast<int>(blockIdx.x) / p.split;
    const bool last = mine >= p.clusters;
    const int64_t chunk = static_cast<int64_t>(p.tokens_of_cluster) * p.top;   // pairs of a cluster
    const int64_t piece = (chunk + p.split - 1) / p.split, end = min((mine + 1) * chunk, p.tokens * p.top);
    const int64_t i0 = mine * chunk + static_cast<int>(blockIdx.x) % p.split * piece, i1 = last ? i0 : min(i0 + piece, end);
    take_turn();
    int32_t expert[kAhead], slot[kAhead];   // of the first pairs, requested before the sums
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t at = i0 + i * kPlaceThreads + threadIdx.x;
        expert[i] = at < i1 ? p.chosen[at] : -1;
        slot[i] = at < i1 ? p.slots[at] : -1;
    }
    if (const int e = threadIdx.x; e < E) {
        // from this block's own cluster on, round: were all blocks to begin with the first, they would wait for the same lines of L2
        int32_t n[kMostClusters], all = 0, some = 0;
        auto turn = [&](int c) { return c + mine - (c + mine >= p.clusters ? p.clusters : 0); };
#pragma unroll
        for (int c = 0; c < kMostClusters; ++c)
            n[c] = c < p.clusters ? p.hist[turn(c) * E + e] : 0;
#pragma unroll
        for (int c = 0; c < kMostClusters; ++c) {
            all += n[c];
            some += turn(c) < mine ? n[c] : 0;
        }
        first[e] = all;
        before[e] = some;
    }
    if (const int e = threadIdx.x ^ (kPlaceThreads / 2); last && p.loss && e < E) {   // (other threads, as far as there are others)
        float s[kMostClusters], all = 0.0f;
#pragma unroll
        for (int c = 0; c < kMostClusters; ++c)
            s[c] = c < p.clusters ? p.part[c * E + e] : 0.0f;
#pragma unroll
        for (int c = 0; c < kMostClusters; ++c)
            all += s[c];
        sums[e] = all;
    }
    const int32_t all = scan_experts(first, E);
    if (last) {
        finish(p, first, all, sums);
        return;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (expert[i] >= 0)
            p.slots[i0 + i * kPlaceThreads + threadIdx.x] = slot[i] + first[expert[i]] + before[expert[i]];
    for (int64_t at = i0 + kAhead * kPlaceThreads + threadIdx.x; at < i1; at += kPlaceThreads) {
        const int32_t e = p.chosen[at];
        if (e >= 0)
            p.slots[at] += first[e] + before[e];
    }
}

struct RouteGrad {
    const void *logits;
    void *dlogits;
    const int32_t *chosen, *offsets;
    const float *dgates, *dloss;
    int64_t tokens, ldl, ldd;
    int32_t experts, top, normalize;
};

template <int G>
__device__ __forceinline__ float group_most(float v)   // NaN where there is one
{
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
        const float u = __shfl_xor_sync(kAll, v, o);
        v = u > v || u != u ? u : v;
    }
    return v;
}

template <int N>
constexpr int kGradThreads = N <= 16 ? 256 : 128;

// Lanes have tokens and experts as in route_kernel.  Reads the logits once and writes as much: 16000 x 32 fp32 (4.6 MB) 3.6 us (4.0 with
// other logits each time), of which 1.3 are more than an empty launch; 8192 x 256 bf16 7.1, with normalize 9.2: the rate of instructions
// again.
template <typename T, int N, int G, int V>
__global__ void __launch_bounds__(kGradThreads<N>) route_grad_kernel(const RouteGrad p)
{
    constexpr int kTokens = 32 / G;
    constexpr int kPitch = N + 4;   // of a lane's experts: no two lanes of eight read the same banks
    // Of a warp's tokens and their experts: the chosen gates' gradients, and which are chosen.  (Found by comparing each lane's experts with
    // each choice instead, 8192 tokens to 8 of 256 took 10.6 us.)
    __shared__ __align__(16) float grad_of[kGradThreads<N> / 32][32 * kPitch], chosen_of[kGradThreads<N> / 32][32 * kPitch];
    float *grads = grad_of[threadIdx.x / 32], *flags = chosen_of[threadIdx.x / 32];
    const float inf = __uint_as_float(0x7f800000u);
    const int lane = threadIdx.x & 31, E = p.experts, k = p.top, e0 = lane % G * N, group = lane / G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kGradThreads<N> / 32) * kTokens;
    take_turn();
    // what the loss pulls at each expert's p
    float pull[N] = {};
    if (p.dloss) {
        int32_t at[N + 1];
#pragma unroll
        for (int i = 0; i <= N; ++i)
            at[i] = p.offsets[min(e0 + i, E)];
        const float m = static_cast<float>(max(p.offsets[E] - p.offsets[0], 1));
        const float scale = *p.dloss * (static_cast<float>(E) * static_cast<float>(k) / m / m);
#pragma unroll
        for (int i = 0; i < N; ++i)
            pull[i] = scale * static_cast<float>(at[i + 1] - at[i]);
    }
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kGradThreads<N> / 32) + threadIdx.x / 32) * kTokens; t0 < p.tokens; t0 += step) {
        const int64_t t = t0 + group;
        const bool here = t < p.tokens;
        Logits<T, N, V> raw;
        if (here)
            raw.load(static_cast<const T *>(p.logits) + t * p.ldl, e0, E);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            *reinterpret_cast<float4 *>(grads + (lane * kPitch + i)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            *reinterpret_cast<float4 *>(flags + (lane * kPitch + i)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncwarp();
        for (int j = lane % G; j < k; j += G) {
            const int32_t e = here ? p.chosen[t * k + j] : -1;
            const float v = here && p.dgates ? p.dgates[t * k + j] : 0.0f;
            if (e >= 0 && e < E) {
                const int at = (group * G + e / N) * kPitch + e % N;
                grads[at] = v;
                flags[at] = 1.0f;
            }
        }
        __syncwarp();
        float d[N];
        uint32_t chosen = 0;        // which of the lane's experts are chosen
#pragma unroll
        for (int i = 0; i < N; ++i) {
            d[i] = grads[lane * kPitch + i];
            chosen |= flags[lane * kPitch + i] != 0.0f ? 1u << i : 0u;
        }
        __syncwarp();
        float x[N], most = -inf, all = 0.0f, dot = 0.0f;
        raw.values(x);
#pragma unroll
        for (int i = 0; i < N; ++i)
            most = x[i] > most || x[i] != x[i] ? x[i] : most;
        most = group_most<G>(most);
        float gate[N] = {};
        if (p.normalize) {   // among the chosen ones alone, whose p may all be small
            float top = -inf, sum = 0.0f, mean = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (chosen >> i & 1u)
                    top = x[i] > top || x[i] != x[i] ? x[i] : top;
            top = group_most<G>(top);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                gate[i] = chosen >> i & 1u ? expf(x[i] - top) : 0.0f;
                sum += gate[i];
                mean += gate[i] * d[i];
            }
            const float scale = 1.0f / group_sum<G>(sum);
            mean = group_sum<G>(mean) * scale;
#pragma unroll
            for (int i = 0; i < N; ++i)
                gate[i] = chosen >> i & 1u ? gate[i] * scale * (d[i] - mean) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float g = p.normalize ? pull[i] : pull[i] + d[i];
            x[i] = x[i] == -inf ? 0.0f : expf(x[i] - most);
            all += x[i];
            dot += x[i] * g;
            d[i] = g;
        }
        const float scale = 1.0f / group_sum<G>(all);
        dot = group_sum<G>(dot) * scale;
        uint32_t routed = chosen;
#pragma unroll
        for (int o = 1; o < G; o <<= 1)
            routed |= __shfl_xor_sync(kAll, routed, o);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = routed ? x[i] * scale * (d[i] - dot) + gate[i] : 0.0f;
        if (here) {
            T *out = static_cast<T *>(p.dlogits) + t * p.ldd + e0;
#pragma unroll
            for (int q = 0; q < N / V; ++q)
                if (e0 + q * V < E) {
                    if constexpr (V == 1)
                        out[q] = from_f32<T>(x[q]);
                    else
                        store<T, V>(out + q * V, *reinterpret_cast<float(*)[V]>(&x[q * V]));
                }
        }
    }
}

bool bad_sizes(int64_t tokens, int64_t experts, int32_t top)
{
    return tokens < 0 || experts < 1 || experts > MLP_MAX_EXPERTS || top < 1 || top > MLP_MAX_TOP || top > experts ||
           tokens > ((int64_t{1} << 31) - 1) / top;
}

// Tables of the clusters' counts, and of their sums of p: cells of each.
int64_t table_cells(int64_t experts) { return kMostClusters * experts; }

template <typename T, int N, int G>
void forward_as(Route &p, Stream &st)
{
    constexpr int V = std::min(N, 16 / static_cast<int>(sizeof(T))), kTokens = 32 / G;
    const int most = kRouteThreads<N> / 32;   // warps of a block
    // Rows of whole vectors, or else one value at a time: 8192 tokens to 8 of 256 bf16 13.5 and 13.9 us, 16384 to 4 of 64 11.1 and 11.4 (of
    // 60 11.4).
    const bool wide = p.experts % V == 0 && aligned(p.logits, p.ldl, sizeof(T), V * sizeof(T));
    const int64_t units = cdiv(p.tokens, kTokens);   // of a warp's tokens at a time
    int cluster = kCluster;
    p.clusters = 1;
    p.steps = 1;
    if (units <= most) {
        p.warps = std::max(1, static_cast<int>(units));
        cluster = 1;
    } else if (units <= most * kCluster) {
        p.warps = static_cast<int32_t>(cdiv(units, kCluster));
    } else {
        constexpr int kClusters = N <= 8 ? kMostClusters : kMostWideClusters;
        p.steps = static_cast<int32_t>(cdiv(units, most * kCluster * kClusters));
        p.warps = static_cast<int32_t>(std::max<int64_t>(most * 3 / 4, cdiv(units, static_cast<int64_t>(p.steps) * kCluster * kClusters)));
        p.clusters = static_cast<int32_t>(cdiv(units, static_cast<int64_t>(p.steps) * p.warps * kCluster));
    }
    p.tokens_of_cluster = static_cast<int64_t>(p.steps) * p.warps * kCluster * kTokens;
    p.split = static_cast<int32_t>(std::min<int64_t>(8, cdiv(p.tokens_of_cluster * p.top, 4 * kPlaceThreads)));
    const int64_t pairs = static_cast<int64_t>(p.steps) * kTokens * p.top;
    p.staged = pairs * p.warps * 12 <= kStageBytes;
    const RouteCells cells = route_cells(p.warps, p.experts, p.staged ? static_cast<int>(pairs) : kTokens * p.top);
    const size_t smem = static_cast<size_t>(cells.all) * 4;
    auto kernel = wide ? route_kernel<T, N, G, V> : route_kernel<T, N, G, 1>;
    if (smem > 28 * 1024 && !succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem))) {
        st.failed = true;
        return;
    }
    launch_clusters(kernel, static_cast<unsigned>(p.clusters * cluster), cluster, p.warps * 32, smem, st, p);
    if (p.clusters > 1)
        launch(place_kernel, static_cast<unsigned>(p.clusters * p.split + 1), kPlaceThreads, 0, st, p);
}

template <typename T, int N>
void forward_few(const Route &p, Stream &st)
{
    launch(route_few_kernel<T, N>, 1, static_cast<int>(std::max<int64_t>(p.tokens, 1)) * 32, static_cast<size_t>(p.loss ? p.tokens * p.experts * 4 : 0), st, p);
}

template <typename T>
void forward(Route &p, Stream &st)
{
    const int64_t E = p.experts;
    if (p.tokens <= (E <= 256 ? 32 : 8))
        return E <= 32    ? forward_few<T, 1>(p, st)
               : E <= 64  ? forward_few<T, 2>(p, st)
               : E <= 128 ? forward_few<T, 4>(p, st)
               : E <= 256 ? forward_few<T, 8>(p, st)
                          : forward_few<T, 32>(p, st);
    E <= 8     ? forward_as<T, 8, 1>(p, st)
    : E <= 16  ? forward_as<T, 8, 2>(p, st)
    : E <= 32  ? forward_as<T, 8, 4>(p, st)
    : E <= 64  ? forward_as<T, 8, 8>(p, st)
    : E <= 128 ? forward_as<T, 8, 16>(p, st)
    : E <= 256 ? forward_as<T, 8, 32>(p, st)
    : E <= 512 ? forward_as<T, 16, 32>(p, st)
               : forward_as<T, 32, 32>(p, st);
}

template <typename T, int N, int G>
void backward_as(const RouteGrad &p, Stream &st)
{
    constexpr int V = std::min(N, 16 / static_cast<int>(sizeof(T)));
    // (as above: 8192 x 256 bf16 7.1 and 10.0 us, 16384 x 64 3.7 and 6.2, 16384 x 60 5.8)
    const bool wide = p.experts % V == 0 && aligned(p.logits, p.ldl, sizeof(T), V * sizeof(T)) && aligned(p.dlogits, p.ldd, sizeof(T), V * sizeof(T));
    const int64_t blocks = cdiv(p.tokens, 32 / G * (kGradThreads<N> / 32));
    launch(wide ? route_grad_kernel<T, N, G, V> : route_grad_kernel<T, N, G, 1>, static_cast<unsigned>(std::min<int64_t>(blocks, 8 * kSms)),
           kGradThreads<N>, 0, st, p);
}

template <typename T>
void backward(const RouteGrad &p, Stream &st)
{
    const int64_t E = p.experts;
    E <= 8     ? backward_as<T, 8, 1>(p, st)
    : E <= 16  ? backward_as<T, 8, 2>(p, st)
    : E <= 32  ? backward_as<T, 8, 4>(p, st)
    : E <= 64  ? backward_as<T, 8, 8>(p, st)
    : E <= 128 ? backward_as<T, 8, 16>(p, st)
    : E <= 256 ? backward_as<T, 8, 32>(p, st)
    : E <= 512 ? backward_as<T, 16, 32>(p, st)
               : backward_as<T, 32, 32>(p, st);
}

}  // namespace

extern "C" mlp_status mlp_route_workspace_size(int64_t tokens, int64_t experts, size_t *bytes)
{
    if (tokens < 0 || experts < 1 || experts > MLP_MAX_EXPERTS || !bytes)
        return MLP_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(table_cells(experts)) * 8;
    return MLP_OK;
}

extern "C" mlp_status mlp_route_forward(int64_t tokens, int64_t experts, int32_t top, const void *logits, int64_t ldl, mlp_dtype dtype,
                                        const uint8_t *mask, int32_t normalize, float *gates, int32_t *chosen, int32_t *slots,
                                        int32_t *offsets, int32_t *counts, float *loss, void *workspace, void *stream)
{
    if (bad_sizes(tokens, experts, top))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if (!offsets || !aligned(offsets, 0, 4, 4) || !aligned(counts, 0, 4, 4) || !aligned(loss, 0, 4, 4) ||
        (tokens && (bad_rows(logits, ldl, experts, esz) || !gates || !aligned(gates, 0, 4, 4) || !chosen || !aligned(chosen, 0, 4, 4) ||
                    !slots || !aligned(slots, 0, 4, 4) || !workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)))
        return MLP_ERR_INVALID_ARG;
    Route p = {};
    p.logits = logits;
    p.ldl = ldl;
    p.mask = mask;
    p.gates = gates;
    p.chosen = chosen;
    p.slots = slots;
    p.offsets = offsets;
    p.counts = counts;
    p.loss = loss;
    p.tokens = tokens;
    p.experts = static_cast<int32_t>(experts);
    p.top = top;
    p.normalize = normalize;
    p.hist = static_cast<int32_t *>(workspace);
    p.part = reinterpret_cast<float *>(p.hist + table_cells(experts));
    Stream st{static_cast<cudaStream_t>(stream)};
    dtype == MLP_DT_BF16 ? forward<__nv_bfloat16>(p, st) : forward<float>(p, st);
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
}

extern "C" mlp_status mlp_route_backward(int64_t tokens, int64_t experts, int32_t top, const void *logits, int64_t ldl, mlp_dtype dtype,
                                         int32_t normalize, const int32_t *chosen, const int32_t *offsets, const float *dgates,
                                         const float *dloss, void *dlogits, int64_t ldd, void *stream)
{
    if (bad_sizes(tokens, experts, top))
        return MLP_ERR_INVALID_ARG;
    if (bad_dtype(dtype))
        return MLP_ERR_UNSUPPORTED;
    if (tokens == 0)
        return MLP_OK;
    const size_t esz = dtype == MLP_DT_BF16 ? 2 : 4;
    if (bad_rows(logits, ldl, experts, esz) || bad_rows(dlogits, ldd, experts, esz) || !chosen || !aligned(chosen, 0, 4, 4) || !offsets ||
        !aligned(offsets, 0, 4, 4) || !aligned(dgates, 0, 4, 4) || !aligned(dloss, 0, 4, 4))
        return MLP_ERR_INVALID_ARG;
    RouteGrad p = {};
    p.logits = logits;
    p.ldl = ldl;
    p.dlogits = dlogits;
    p.ldd = ldd;
    p.chosen = chosen;
    p.offsets = offsets;
    p.dgates = dgates;
    p.dloss = dloss;
    p.tokens = tokens;
    p.experts = static_cast<int32_t>(experts);
    p.top = top;
    p.normalize = normalize;
    Stream st{static_cast<cudaStream_t>(stream)};
    dtype == MLP_DT_BF16 ? backward<__nv_bfloat16>(p, st) : backward<float>(p, st);
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
}
