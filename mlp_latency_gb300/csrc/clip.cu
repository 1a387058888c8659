// clip.cu -- the norm of many tensors, and clipping by it (C ABI in include/mlp_clip.h).
//
//   n = sqrt(sum x^2),  c = min(1, max_norm / (n + eps)),  out = c x
//
// Two or three operations per element: the memory system is the bound, first reading everything, then (where c < 1, or out is
// another place) reading and writing it.  The tensors are cut into pieces of a block's registers; the list travels in the
// kernel's parameters, so a call needs no copy to the device and a captured one keeps its own.  134 million bf16 values to another
// place 122 us, in place 121: the first pass reads 268 MB in 42 (93 % of the copy rate), the second what L2 does not have of them, and
// writes.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/mlp_clip.h"
#include "elements.cuh"
#include "launch.h"

using namespace mlpc;

namespace {

constexpr int kThreads = 256, kWords = 4;           // a piece: 256 threads x 4 words of 16 bytes
constexpr int64_t kPiece = kThreads * kWords;       // words
constexpr int kMostBlocks = 8 * kSms;               // of a launch: all on the SMs at once; partial sums
constexpr int kScaleBlocks = 4 * kSms;              // of the second pass (6 an SM: 36 tensors, 21.7 MB, 13.8 us, 4 13.0; 3 14.1)
// What the first pass leaves in L2 for the second: 64 MB, the last pieces.  (134 million bf16 values to another place: none kept 128.0 us,
// 32 MB 126.2, 64 MB 123.0, 128 MB, which is all of L2, 126.8.)
constexpr uint32_t kKeptPieces = (64 << 20) / (kPiece * 16);

// Sums of the blocks of the first pass (big, mid, small: see Squares), `from` of them by the launches before.
struct Partial {
    float4 *sums;
    int32_t from;
};

// One tensor: `head` elements, `words` words of 16 bytes, `tail` elements; or, for the second pass where out lies differently in its words
// than data, elements throughout (`words` counts elements then).
struct Part {
    const char *data;
    char *out;
    int64_t words;
    uint32_t last;        // pieces up to and with this tensor
    uint8_t f32, by_element, head, tail;
};

template <int N>
struct List {
    Part part[N];
    int32_t parts;
};

__device__ __forceinline__ float element(const char *p, bool f32, int64_t i)
{
    return f32 ? reinterpret_cast<const float *>(p)[i] : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void put_element(char *p, bool f32, int64_t i, float v)
{
    if (f32)
        reinterpret_cast<float *>(p)[i] = v;
    else
        reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// The tensor of a piece; `lo` is that of another one (0 at first), which most often is the same.
template <int N>
__device__ __forceinline__ int part_of(const List<N> &l, uint32_t piece, int lo)
{
    if (piece < l.part[lo].last && (lo == 0 || piece >= l.part[lo - 1].last))
        return lo;
    int hi = l.parts - 1;
    lo = 0;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (l.part[mid].last > piece)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// A sum of squares that keeps the exponent's range: a group of words, 16 or 32 values, whose squares would leave fp32's is summed apart,
// scaled by a power of two.  Groups above 2^90 (big) by 2^-96: a value of 2^128 adds 2^64, the largest of such a group 2^-107 at least.
// Groups below 2^-80 (small) by 2^84: a value of 2^-149 adds 2^-130, a group at most 2^88.  A call takes fewer than 2^40 values, in 2^36
// groups, so no sum leaves the range: big 2^104, in between 2^126, small 2^124.
struct Squares {
    float big = 0.0f, mid = 0.0f, small = 0.0f;
};
constexpr float kBig = 0x1p-96f, kSmall = 0x1p84f;

__device__ __forceinline__ float squares(uint4 w, bool f32, float scale, float s)
{
    if (f32) {
        float x[4];
        unpack<float>(w, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = x[i] * scale;
            s = fmaf(v, v, s);
        }
    } else {
        float x[8];
        unpack<__nv_bfloat16>(w, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = x[i] * scale;
            s = fmaf(v, v, s);
        }
    }
    return s;
}

// 16 bytes, read or written with a policy of their own in L2.
__device__ __forceinline__ uint64_t passing()   // not wanted again
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint4 load_with(const void *p, uint64_t policy)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ void store_with(void *p, uint4 v, uint64_t policy)
{
    asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "l"(policy) : "memory");
}

// What values are multiplied by: c, then a power of two, which is 1 unless max_norm / norm is below fp32's normal numbers.
struct Factor {
    float c, power;

    __device__ __forceinline__ float of(float x) const { return x * c * power; }
};

// min(1, max_norm / (norm + eps)).  Where fp32 has few bits or none for the quotient, or none for the sum (a norm or norm + eps past its
// range), it is found in 64 bits; c is then between 1/2 and 1, so that its product with a value of any size keeps its bits until the power is
// applied.  (The least power there is, 2^-149, goes with a smaller c; below 2^-275 c is subnormal too, and so is all that is left.)
__device__ __forceinline__ Factor factor_of(double exact, float max_norm, float eps)
{
    const float norm = static_cast<float>(exact), sum = norm + eps;
    if (norm == 0.0f || max_norm >= sum)
        return {1.0f, 1.0f};
    const float c = max_norm / sum;   // (a NaN stays one)
    if (!(c < 0x1p-126f) || isinf(exact))
        return {c, 1.0f};
    int e;
    const double f = static_cast<double>(max_norm) / (exact + static_cast<double>(eps)), half = frexp(f, &e);
    return {static_cast<float>(ldexp(half, min(e + 149, 0))), ldexpf(1.0f, max(e, -149))};
}

template <typename T>
__device__ __forceinline__ uint4 times(uint4 w, Factor f);
template <>
__device__ __forceinline__ uint4 times<float>(uint4 w, Factor f)
{
    return make_uint4(__float_as_uint(f.of(__uint_as_float(w.x))), __float_as_uint(f.of(__uint_as_float(w.y))),
                      __float_as_uint(f.of(__uint_as_float(w.z))), __float_as_uint(f.of(__uint_as_float(w.w))));
}
template <>
__device__ __forceinline__ uint4 times<__nv_bfloat16>(uint4 w, Factor f)
{
    auto two = [f](uint32_t v) { return pack_bf16(f.of(bf16_lo(v)), f.of(bf16_hi(v))); };
    return make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
}

// Which sum a thread's values belong to: by their sum of squares without a scale.
__device__ __forceinline__ int range_of(float s) { return s >= 0x1p-80f && s <= 0x1p90f ? 1 : s < 0x1p-80f ? 2 : 0; }

__device__ __forceinline__ void add_element(Squares &q, float x)
{
    const float s = x * x;
    const int r = range_of(s);
    if (r == 1)
        q.mid += s;
    else if (r == 2)
        q.small = fmaf(x * kSmall, x * kSmall, q.small);
    else
        q.big = fmaf(x * kBig, x * kBig, q.big);
}

// 8 blocks an SM of 4 words a thread: 128 KB of an SM's are on their way, and the last round of pieces is short (8 words and five blocks:
// 134 MB from cold caches 24.0 us, so 22.1).
template <int N>
__global__ void __launch_bounds__(kThreads, 8) norm_kernel(const __grid_constant__ List<N> l, uint32_t pieces, uint32_t passing_pieces, Partial partial)
{
    __shared__ float red[3][kThreads / 32];
    take_turn();
    const uint64_t policy = passing();
    Squares q;
    int k = 0;
    for (uint32_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        k = part_of(l, piece, k);
        const Part &t = l.part[k];
        const int64_t w0 = static_cast<int64_t>(piece - (k ? l.part[k - 1].last : 0)) * kPiece;
        const bool f32 = t.f32;
        const char *body = t.data + static_cast<int>(t.head) * (f32 ? 4 : 2);
        uint4 w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int64_t at = w0 + i * kThreads + threadIdx.x;
            w[i] = at >= t.words ? make_uint4(0, 0, 0, 0) : piece < passing_pieces ? load_with(body + at * 16, policy) : *reinterpret_cast<const uint4 *>(body + at * 16);
        }
        float of_word[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            of_word[i] = squares(w[i], f32, 1.0f, 0.0f);
        const float s = (of_word[0] + of_word[1]) + (of_word[2] + of_word[3]);
        const int r = range_of(s);
        if (r == 1) {
            q.mid += s;
        } else {
            const float scale = r == 0 ? kBig : kSmall;
            float &sum = r == 0 ? q.big : q.small;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                sum = squares(w[i], f32, scale, sum);
        }
        if (w0 == 0 && threadIdx.x < t.head + t.tail)
            add_element(q, threadIdx.x < t.head ? element(t.data, f32, threadIdx.x)
                                                : element(body + t.words * 16, f32, threadIdx.x - t.head));
    }
    const float v[3] = {q.big, q.mid, q.small};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const float s = warp_sum(v[n]);
        if ((threadIdx.x & 31) == 0)
            red[n][threadIdx.x / 32] = s;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            sum += red[threadIdx.x][w];
        reinterpret_cast<float *>(partial.sums + partial.from + blockIdx.x)[threadIdx.x] = sum;
    }
}

// The norm from the partial sums, in a fixed order, for thread 0 of a block.  In 64 bits only where a scaled sum takes part: there are
// few units for it, and a square root of every thread took 15 us.
__device__ __forceinline__ double total_norm(const Partial &p)
{
    __shared__ float red[3][kThreads / 32];
    float v[3] = {};
    constexpr int kRounds = (kMostBlocks + kThreads - 1) / kThreads;   // of a launch's sums, requested at once
    // the blocks' warps begin at different places: all at the same one, they would wait for the same lines of L2
    constexpr int kWarps = kThreads / 32;
    const int warp = (threadIdx.x / 32 + blockIdx.x) % kWarps, lane = threadIdx.x & 31;
    for (int i0 = warp * 32 + lane; i0 < p.from; i0 += kRounds * kThreads) {
        float4 x[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            x[r] = i0 + r * kThreads < p.from ? p.sums[i0 + r * kThreads] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            v[0] += x[r].x;
            v[1] += x[r].y;
            v[2] += x[r].z;
        }
    }
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        v[n] = warp_sum(v[n]);
        if (lane == 0)
            red[n][warp] = v[n];
    }
    __syncthreads();
    if (threadIdx.x != 0)
        return 0.0;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        v[n] = red[n][0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w)
            v[n] += red[n][w];
    }
    if (v[0] == 0.0f && v[2] == 0.0f)
        return sqrtf(v[1]);
    return sqrt(static_cast<double>(v[0]) * 0x1p192 + static_cast<double>(v[1]) + static_cast<double>(v[2]) * 0x1p-168);
}

__global__ void __launch_bounds__(kThreads) finish_kernel(Partial partial, float *norm)
{
    take_turn();
    const double v = total_norm(partial);
    if (threadIdx.x == 0)
        *norm = static_cast<float>(v);
}

// The pieces from the last on: those that the pass before read last are in L2.  (A piece requested before the norm is known gained
// nothing: other blocks' loads are on their way then.)
template <int N>
__global__ void __launch_bounds__(kThreads, 4) scale_kernel(const __grid_constant__ List<N> l, uint32_t pieces, Partial partial, bool in_place,
                                                           float max_norm, float eps, float *norm)
{
    __shared__ Factor factor;
    take_turn();
    const double exact = total_norm(partial);
    if (threadIdx.x == 0) {
        if (norm && blockIdx.x == 0)
            *norm = static_cast<float>(exact);
        factor = factor_of(exact, max_norm, eps);
    }
    __syncthreads();
    const Factor f = factor;
    const bool whole = f.c * f.power == 1.0f;
    if (whole && in_place)
        return;
    const uint64_t policy = passing();
    int k = l.parts - 1;
    for (uint32_t turn = blockIdx.x; turn < pieces; turn += gridDim.x) {
        const uint32_t piece = pieces - 1 - turn;
        k = part_of(l, piece, k);
        const Part &t = l.part[k];
        if (whole && t.out == t.data)
            continue;
        const int64_t w0 = static_cast<int64_t>(piece - (k ? l.part[k - 1].last : 0)) * kPiece;
        const bool f32 = t.f32;
        if (t.by_element) {   // (67 million bf16 values 230 us, 33 million fp32 133; lying alike 58 and 57)
            for (int64_t i = w0 + threadIdx.x; i < min(w0 + kPiece, t.words); i += kThreads)
                put_element(t.out, f32, i, f.of(element(t.data, f32, i)));
            continue;
        }
        const int64_t head = static_cast<int>(t.head) * (f32 ? 4 : 2);
        uint4 w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int64_t at = w0 + i * kThreads + threadIdx.x;
            if (at < t.words)
                w[i] = load_with(t.data + head + at * 16, policy);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int64_t at = w0 + i * kThreads + threadIdx.x;
            if (at < t.words)
                store_with(t.out + head + at * 16, f32 ? times<float>(w[i], f) : times<__nv_bfloat16>(w[i], f), policy);
        }
        if (w0 == 0 && threadIdx.x < t.head + t.tail) {
            const int64_t at = threadIdx.x < t.head ? threadIdx.x : t.words * (f32 ? 4 : 8) + threadIdx.x;
            put_element(t.out, f32, at, f.of(element(t.data, f32, at)));
        }
    }
}

// Tensors of a launch: 2 KB of parameters, or about the most that a launch takes (32764 bytes), which cost the host and the device
// 1.3 us a launch whatever is in them (tensors of 4096 fp32 in place, two launches: 2 of them 5.5 us with the short list and 8.2 with the
// long one, 64 6.3 and 8.7; 65 8.8, 400 12.0, 1000 18.6).
constexpr int kFew = 64, kMost = 1000;

size_t size_of(mlp_dtype d) { return d == MLP_DT_BF16 ? 2 : 4; }

Part part_for(const mlp_tensor &t, bool write)
{
    Part p = {};
    const size_t esz = size_of(t.dtype);
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.data);
    p.data = static_cast<const char *>(t.data);
    p.out = static_cast<char *>(t.out);
    p.f32 = t.dtype == MLP_DT_F32;
    p.by_element = write && (at ^ reinterpret_cast<uintptr_t>(t.out)) % 16 != 0;
    if (p.by_element) {
        p.words = t.count;
        return p;
    }
    const int64_t per = 16 / static_cast<int64_t>(esz), head = std::min<int64_t>(t.count, static_cast<int64_t>((16 - at % 16) % 16 / esz));
    p.head = static_cast<uint8_t>(head);
    p.words = (t.count - head) / per;
    p.tail = static_cast<uint8_t>(t.count - head - p.words * per);
    return p;
}

// The next launch's tensors from `i` on; empty ones are left out.  Returns its pieces.
template <int N>
uint32_t fill(List<N> &l, int64_t &i, int64_t tensors, const mlp_tensor *list, bool write, bool &in_place)
{
    uint32_t pieces = 0;
    l.parts = 0;
    in_place = true;
    for (; i < tensors && l.parts < N; ++i) {
        if (list[i].count == 0)
            continue;
        Part p = part_for(list[i], write);
        const int64_t n = std::max<int64_t>(1, cdiv(p.words, kPiece));
        pieces += static_cast<uint32_t>(n);
        p.last = pieces;
        in_place = in_place && p.out == p.data;
        l.part[l.parts++] = p;
    }
    return pieces;
}

template <int N>
void run(int64_t tensors, const mlp_tensor *list, bool clip, float max_norm, float eps, float *norm, Partial partial, Stream &st)
{
    List<N> l;
    uint32_t pieces = 0;
    bool in_place = true, one = false;
    for (int64_t i = 0; i < tensors;) {
        const int64_t from = i;
        pieces = fill(l, i, tensors, list, false, in_place);
        if (!pieces)
            break;
        one = from == 0 && i == tensors;
        const unsigned grid = std::min<uint32_t>(pieces, kMostBlocks);
        launch(norm_kernel<N>, grid, kThreads, 0, st, l, pieces, pieces > kKeptPieces ? pieces - kKeptPieces : 0u, partial);
        partial.from += static_cast<int32_t>(grid);
    }
    if (!clip || !partial.from) {
        launch(finish_kernel, 1, kThreads, 0, st, partial, norm);
        return;
    }
    for (int64_t i = 0; i < tensors; norm = nullptr) {
        if (one && in_place)
            i = tensors;   // (l is that of the only launch)
        else
            pieces = fill(l, i, tensors, list, true, in_place);
        if (!pieces)
            break;
        launch(scale_kernel<N>, std::min<uint32_t>(pieces, kScaleBlocks), kThreads, 0, st, l, pieces, partial, in_place, max_norm, eps, norm);
    }
}

int64_t launches_of(int64_t tensors) { return std::max<int64_t>(1, cdiv(tensors, kMost)); }

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// Whether a place that is written is also another tensor's, or partly its own data.
bool overlap(int64_t tensors, const mlp_tensor *list)
{
    bool ascending = true;
    uintptr_t end = 0;
    for (int64_t i = 0; i < tensors && ascending; ++i) {   // the common case: each tensor after the one before, in place
        if (!list[i].count)
            continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(list[i].data);
        ascending = list[i].out == list[i].data && lo >= end;
        end = lo + static_cast<size_t>(list[i].count) * size_of(list[i].dtype);
    }
    if (ascending)
        return false;
    Span *s = new Span[static_cast<size_t>(2 * tensors)];
    int64_t n = 0;
    for (int64_t i = 0; i < tensors; ++i) {
        const size_t bytes = static_cast<size_t>(list[i].count) * size_of(list[i].dtype);
        const uintptr_t from = reinterpret_cast<uintptr_t>(list[i].data), to = reinterpret_cast<uintptr_t>(list[i].out);
        if (!bytes)
            continue;
        s[n++] = {to, to + bytes, true};
        if (from != to)
            s[n++] = {from, from + bytes, false};
    }
    std::sort(s, s + n, [](const Span &a, const Span &b) { return a.lo < b.lo; });
    bool bad = false;
    uintptr_t any = 0, written = 0;   // the farthest ends so far
    for (int64_t i = 0; i < n && !bad; ++i) {
        bad = s[i].lo < written || (s[i].out && s[i].lo < any);
        any = std::max(any, s[i].hi);
        if (s[i].out)
            written = std::max(written, s[i].hi);
    }
    delete[] s;
    return bad;
}

mlp_status start(int64_t tensors, const mlp_tensor *list, bool clip, float max_norm, float eps, float *norm, void *workspace, void *stream)
try {
    if (tensors < 0 || tensors > (int64_t{1} << 20) || (tensors && !list) || !norm || !aligned(norm, 0, 4, 4) || !workspace ||
        reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || (clip && (!(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps))))
        return MLP_ERR_INVALID_ARG;
    for (int64_t i = 0; i < tensors; ++i)
        if (bad_dtype(list[i].dtype))
            return MLP_ERR_UNSUPPORTED;
    int64_t elements = 0;
    for (int64_t i = 0; i < tensors; ++i) {
        const mlp_tensor &t = list[i];
        const size_t esz = size_of(t.dtype);
        if (t.count < 0 || t.count >= (int64_t{1} << 40) || (elements += t.count) >= (int64_t{1} << 40) || (t.count && (!t.data || !aligned(t.data, 0, esz, esz))) ||
            (clip && t.count && (!t.out || !aligned(t.out, 0, esz, esz))))
            return MLP_ERR_INVALID_ARG;
    }
    if (clip && overlap(tensors, list))
        return MLP_ERR_INVALID_ARG;
    Stream st{static_cast<cudaStream_t>(stream)};
    const Partial partial = {static_cast<float4 *>(workspace), 0};
    if (tensors <= kFew)
        run<kFew>(tensors, list, clip, max_norm, eps, norm, partial, st);
    else
        run<kMost>(tensors, list, clip, max_norm, eps, norm, partial, st);
    return st.failed ? MLP_ERR_CUDA : MLP_OK;
} catch (const std::bad_alloc &) {
    return MLP_ERR_OOM;
}

}  // namespace

extern "C" mlp_status mlp_clip_workspace_size(int64_t tensors, size_t *bytes)
{
    if (tensors < 0 || tensors > (int64_t{1} << 20) || !bytes)
        return MLP_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(launches_of(tensors)) * kMostBlocks * sizeof(float4);
    return MLP_OK;
}

extern "C" mlp_status mlp_gradient_norm(int64_t tensors, const mlp_tensor *list, float *norm, void *workspace, void *stream)
{
    return start(tensors, list, false, 0.0f, 0.0f, norm, workspace, stream);
}

extern "C" mlp_status mlp_clip_gradients(int64_t tensors, const mlp_tensor *list, float max_norm, float eps, float *norm, void *workspace,
                                         void *stream)
{
    return start(tensors, list, true, max_norm, eps, norm, workspace, stream);
}
