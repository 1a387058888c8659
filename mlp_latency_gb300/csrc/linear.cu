// linear.cu -- C ABI of mlp_linear (include/mlp_block.h): handle, choice of the kernel variant, tensor
// maps, launches, and the elementwise part of the backward pass.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/mlp_block.h"
#include "cuda_call.h"
#include "linear_kernel.cuh"
#include "row_blocks.h"

using namespace mlpl;

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (!succeeded(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q)) ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Views of bf16 rows of `inner` elements, `ld` apart, `outer` per group: (inner, outer, group) with boxes of 64 x
// box_outer; or, for tiles of several 64-column boxes that start on a box, (64, outer, inner / 64, group) with all of a
// tile's boxes in one.
bool encode(CUtensorMap *map, const void *ptr, int64_t inner, int64_t outer, int64_t groups, int64_t ld, int box_outer)
{
    EncodeFn fn = encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * static_cast<cuuint64_t>(outer)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_outer), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemLimit = 227 * 1024;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int kForm, int kFormB>
bool allow_smem()
{
    constexpr bool kWide = kForm == kRowsT && kFormB < 0;
    auto allow = [](void (*kernel)(LinearParams)) {
        return succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit));
    };
    return allow(linear_kernel<kForm, kFormB, 1, false>) && allow(linear_kernel<kForm, kFormB, 2, false>) &&
           (!kWide || allow(linear_kernel<kForm, kFormB, 2, kWide>));
}

bool encode_boxed(CUtensorMap *map, const void *ptr, int64_t inner, int64_t outer, int64_t groups, int64_t ld, int boxes)
{
    EncodeFn fn = encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(inner / 64), static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, 128, static_cast<cuuint64_t>(ld) * 2 * static_cast<cuuint64_t>(outer)};
    const cuuint32_t box[4] = {64, kKB, static_cast<cuuint32_t>(boxes), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Operand `op` of a launch.  K-major: `outer` rows of the reduction extent `inner`, `cols` of them per tile.  MN-major:
// `inner` columns, the reduction outside, `cols` columns per tile.
bool operand(Problem &p, int op, bool mn, const void *ptr, int64_t inner, int64_t outer, int64_t groups, int64_t ld, int cols)
{
    p.mn[op] = mn;
    if (!mn) {
        p.copy_bytes[op] = static_cast<uint32_t>(cols) * 128u;
        return encode(&p.map[op], ptr, inner, outer, groups, ld, cols);
    }
    p.copy_bytes[op] = q_tile_bytes(cols, true);
    if (inner % 64 == 0 && cols % 64 == 0 && encode_boxed(&p.map[op], ptr, inner, outer, groups, ld, cols / 64)) {
        p.boxed[op] = 1;
        return true;
    }
    return encode(&p.map[op], ptr, inner, outer, groups, ld, kKB);
}

struct Plan {
    int form, pair, bn, split, pipe;
    uint32_t slot, recv_bytes;
    int recv_bufs, part_align;
    int q_tiles;             // kRowsT, one group: tiles along the rows
};

}  // namespace

struct mlp_linear {
    mlp_linear_desc d;
    int groups;
    int num_sms;
    int max_clusters[9];   // co-resident clusters of 1 to 8 CTAs
    uint32_t *status;
};

namespace {

int accumulators(int bn) { return bn <= 256 ? 2 : 1; }

// Ring depth and exchange buffers of a chosen variant.
void finish_plan(const mlp_linear *h, Plan &pl, bool q_mn)
{
    const bool rows_t = pl.form == kRowsT;
    pl.slot = kPBytes + q_tile_bytes(pl.bn / pl.pair, q_mn);
    // an accumulator next to another one of full width leaves no columns to over-read
    pl.part_align = accumulators(pl.bn) * pl.bn + 32 <= 512 && rows_t ? 8 : 32;
    const int part = static_cast<int>(cdiv(cdiv(pl.bn, pl.split), pl.part_align)) * pl.part_align;
    pl.recv_bytes = static_cast<uint32_t>((pl.split - 1) * part) * kPRows * 4;
    pl.recv_bufs = pl.split > 1 && rows_t ? (pl.recv_bytes <= 24 * 1024 ? 2 : pl.recv_bytes <= 64 * 1024 ? 1 : 0) : 0;
    const size_t fixed = linear_smem_bytes(pl.form != kRows, 0, static_cast<uint32_t>(pl.recv_bufs) * pl.recv_bytes, h->groups);
    pl.pipe = static_cast<int>(std::min<size_t>(kMaxRing, (kSmemLimit - fixed) / pl.slot));
}

// An estimate of a product's time in SM cycles: of all its tiles on the whole GPU, of one tile, and the sum over the
// tiles divided by the tiles that run at a time.
struct Estimate {
    double time, tile, work;
};

// Row pitch of dZ: its rows start on 128-byte lines, without which every copy of 64 columns takes two requests to L2.
int64_t dz_pitch(int64_t N) { return (N + 63) & ~int64_t{63}; }

// Requests to L2 for rows of this pitch (elements), copied in pieces of 128 bytes: a piece that does not start on a line of
// 128 bytes takes two, and one that does not start on a sector of 32 a sector more.  (Measured as bytes a cycle: 9700 on
// lines, about 6000 on sectors, 3900 on neither.)
double l2_cost(int64_t pitch) { return pitch % 64 == 0 ? 1.0 : pitch % 16 == 0 ? 1.6 : 2.5; }

// A rows product.  rows: of the whole call; out_cols, red: output columns and reduction extent; w_mn: the weights' tile
// is MN-major; a_pitch: of the activations' rows.
Estimate estimate_rows(const mlp_linear *h, const Plan &pl, int64_t rows, int64_t out_cols, int64_t red, bool w_mn, int64_t a_pitch)
{
    const int64_t groups = std::min<int64_t>(h->groups, rows), kb = cdiv(red, kKB);
    const int bm = kPRows * pl.pair, u = 16 * pl.pair;
    // groups of ragged size: at least a tile each, and half a tile (a column step) too much
    int64_t items;
    double n = pl.bn;
    if (pl.form == kRows) {
        items = (h->groups > 1 ? std::max(groups, cdiv(rows, bm) + groups / 2) : cdiv(rows, bm)) * cdiv(out_cols, pl.bn);
    } else if (h->groups > 1) {
        const int64_t tiles = std::max(groups, cdiv(rows, pl.bn) + groups / 2);
        items = tiles * cdiv(out_cols, bm);
        n = std::min<double>(pl.bn, static_cast<double>(rows) / static_cast<double>(tiles) + u / 2);
    } else {
        items = pl.q_tiles * cdiv(out_cols, bm);
        n = static_cast<double>(cdiv(rows, u) * u) / static_cast<double>(pl.q_tiles);
    }
    // MMA: 2 n cycles per k block, at least 310 to issue its four instructions; fill: what a CTA loads per k block
    // at 64 bytes a cycle.  (Wide tiles do not hide all of one behind the other.)
    const double act = pl.form == kRows ? 16384.0 : (h->groups > 1 ? pl.bn : n) * 128.0 / pl.pair;
    const double wgt = pl.form == kRows ? q_tile_bytes(pl.bn / pl.pair, w_mn) : 16384.0;
    const double mma = std::max(2.0 * n, 310.0), fill = (act + wgt) / 64.0;
    const double m2 = mma * mma, f2 = fill * fill;
    const double step = n < 160.0 ? std::max(mma, fill) : std::sqrt(std::sqrt(m2 * m2 + f2 * f2));
    Estimate e;
    e.tile = static_cast<double>(cdiv(kb, pl.split)) * step + 400.0;
    // one accumulator: no epilogue is hidden (with an activation, Z and a residual)
    if (accumulators(pl.bn) == 1)
        e.tile += 40.0 * n;
    // the last epilogue of a CTA is not hidden, nor are the exchanges of a split tile; clusters start later
    if (pl.split > 1)
        e.tile += 2500.0 + n * 512.0 * (pl.split - 1) / pl.split / 18.0;
    const double at_once = h->max_clusters[pl.pair * pl.split], rounds = static_cast<double>(items) / at_once;
    // What L2 needs for a tile: it serves all SMs together with 9700 bytes a cycle
    const double l2 = static_cast<double>(kb) * pl.pair * (act * l2_cost(a_pitch) + wgt * l2_cost(w_mn ? out_cols : red)) / 9700.0;
    // (tiles of ragged groups differ, so their last round is rarely a full one)
    const double full = std::floor(rounds), rest = (rounds - full) * at_once, round = std::max(e.tile, at_once * l2);
    e.work = rounds * round;
    e.time = h->groups > 1 ? std::max(std::max(1.0, rounds + 0.3) * e.tile, static_cast<double>(items) * l2)
                           : full * round + (rest > 0.0 ? std::max(e.tile, rest * l2) : 0.0);
    e.time += (accumulators(pl.bn) == 1 ? 0.0 : 12.0 * n) + (pl.pair > 1 ? 1500.0 : 0.0);
    return e;
}

// The variant of a rows product with the lowest estimate.  any: of all forms, else of the unsplit kRowsT ones on `pair`
// CTAs.
Plan plan_rows(const mlp_linear *h, int64_t rows, int64_t out_cols, int64_t red, bool w_mn, int64_t a_pitch, bool any = true,
               int only_pair = 0)
{
    const int64_t kb = cdiv(red, kKB);
    Plan best{kRowsT, only_pair ? only_pair : 1, 32, 1, 0, 0, 0, 0, 0, static_cast<int>(cdiv(rows, 32))};
    double best_t = 1e300;
    for (int form = any ? kRows : kRowsT; form <= kRowsT; ++form)
        for (int pair = 1; pair <= 2; ++pair)
            for (int bn = 32; bn <= (any && pair == 2 && form == kRowsT ? 512 : 256); bn += bn < 256 ? 32 : 64)
                for (int s = 1; s * pair <= 8 && s <= (any ? 4 : 1); ++s) {
                    if (only_pair && pair != only_pair)
                        continue;
                    if ((form == kRows && bn < 128) || (any && pair == 2 && rows <= (form == kRows ? kPRows : 32)))
                        continue;   // (a pair's second half would have no rows)
                    if (h->max_clusters[pair * s] < 1 || (s > 1 && kb < 4 * s))
                        continue;
                    // tiles along the rows: as few as hold them, or up to two more for a fuller last round (never more
                    // than there are column steps: every tile gets at least one)
                    const int64_t least = form == kRowsT ? cdiv(rows, bn) : 1;
                    const int64_t most = form == kRowsT && h->groups == 1 ? std::min<int64_t>(least + 2, cdiv(rows, 16 * pair)) : least;
                    if (bn > 256 && (s > 1 || rows <= 256))
                        continue;   // (the exchange of such tiles took longer than it saved)
                    for (int64_t tq = least; tq <= most; ++tq) {
                        const Plan pl{form, pair, bn, s, 0, 0, 0, 0, 0, static_cast<int>(tq)};
                        const double t = estimate_rows(h, pl, rows, out_cols, red, w_mn, a_pitch).time;
                        if (t < best_t) {
                            best_t = t;
                            best = pl;
                        }
                    }
                }
    finish_plan(h, best, best.form == kRows && w_mn);
    return best;
}

// The weights' gradient: 256 x 256 tiles on pairs, or 128 x 128 ones where those would leave half of the SMs idle.  Its reduction
// is not split, so a small weight over many rows keeps few SMs busy: 4096 rows of 256 x 256 are 4 tiles, 17.9 us.
Plan plan_reduce(const mlp_linear *h, int64_t p_ext, int64_t q_ext)
{
    Plan pl{kReduce, 2, 256, 1, 0, 0, 0, 0, 0, 0};
    if (h->groups * cdiv(p_ext, 256) * cdiv(q_ext, 256) * 2 < h->num_sms)
        pl.pair = 1, pl.bn = 128;
    finish_plan(h, pl, true);
    return pl;
}

Estimate estimate_reduce(const mlp_linear *h, const Plan &pl, int64_t rows, int64_t p_ext, int64_t q_ext)
{
    const double kb = static_cast<double>(rows) / static_cast<double>(h->groups) / kKB + (h->groups > 1 ? 0.5 : 0.0);
    const double items = static_cast<double>(h->groups * cdiv(p_ext, kPRows * pl.pair) * cdiv(q_ext, pl.bn));
    Estimate e;
    // k blocks as above; a tile's stores leave the SM at about 18 bytes a cycle
    e.tile = std::max(kb * std::max(2.0 * pl.bn, 512.0), 128.0 * pl.bn * 2.0 / 18.0) + 400.0;
    const double at_once = h->max_clusters[pl.pair];
    e.work = items * e.tile / at_once;
    e.time = std::ceil(items / at_once) * e.tile + 12.0 * pl.bn;
    return e;
}

// The backward pass: variants of both gradients, and whether they share a launch when both are asked for.  That saves a
// launch, a set-up and a last round that is partly idle: 29 rows of 3160 x 1024 23 us against 30, 3343 rows of 6624 x
// 2336 154 against 166.  Not where few long tiles of the input's gradient would outlast everything else (a launch of two
// splits no tile), and not past a few hundred microseconds, where two working sets in L2 cost more (2048 rows of 8192 x
// 8192 338 us against 331).  The input's gradient takes the same variant either way, so its bits do not depend on what
// else is asked for.
struct GradPlan {
    Plan x, w;
    bool together;
};

GradPlan plan_grads(const mlp_linear *h, int64_t rows)
{
    const int64_t K = h->d.K, N = h->d.N;
    const bool kn = h->d.weight_layout == 0;
    const int64_t pe = kn ? K : N, qe = kn ? N : K;
    GradPlan g;
    g.w = plan_reduce(h, pe, qe);
    const int64_t pitch = h->d.activation != MLP_ACT_NONE ? dz_pitch(N) : N;
    g.x = plan_rows(h, rows, K, N, !kn, pitch);
    const Plan x = plan_rows(h, rows, K, N, !kn, pitch, false, g.w.pair);
    const Estimate ex = estimate_rows(h, x, rows, K, N, !kn, pitch), ew = estimate_reduce(h, g.w, rows, pe, qe);
    const double both = std::max(ex.work + ew.work, std::max(ex.tile, ew.tile)) + 3000.0;
    const double apart = estimate_rows(h, g.x, rows, K, N, !kn, pitch).time + ew.time + 6000.0;
    g.together = both <= apart && both < 400e3;
    if (g.together)
        g.x = x;
    return g;
}

template <int kForm, int kFormB, int kPair, bool kWide = false>
bool launch_one(const LinearParams &p, int clusters, int cs, size_t smem, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    // set up while the kernel before it on the stream ends (every role waits for that end before it touches
    // global memory that a kernel may have written or may still read)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cs), 1, 1);
    cfg.blockDim = dim3(kLThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return succeeded(cudaLaunchKernelEx(&cfg, linear_kernel<kForm, kFormB, kPair, kWide>, p));
}

// One product (w NULL), or a kRowsT one with the weights' gradient.  items: of the launch, or an upper bound where the
// counts of groups are on the device.
mlp_status launch(const mlp_linear *h, LinearParams &p, const Plan &pl, const Plan *w, int64_t items, cudaStream_t st)
{
    p.groups = h->groups;
    for (int i = 0; i < 2; ++i)
        p.pr[i].raster = 16 / pl.pair;
    p.pr[0].bn = pl.bn;
    if (w)
        p.pr[1].bn = w->bn;
    p.acc_cols = w ? std::max(pl.bn, w->bn) : pl.bn;
    p.split = pl.split;
    p.slot_bytes = w ? std::max(pl.slot, w->slot) : pl.slot;
    p.num_pipe = w ? std::min(pl.pipe, w->pipe) : pl.pipe;
    p.part_align = pl.part_align;
    p.recv_bufs = pl.recv_bufs;
    p.recv_bytes = pl.recv_bytes;
    // parts of a split tile that are no multiple of 32 columns are over-read
    const uint32_t cols = static_cast<uint32_t>(accumulators(p.acc_cols) * p.acc_cols) + (pl.split > 1 && pl.part_align < 32 ? 32u : 0u);
    p.tmem_cols = 32;
    while (p.tmem_cols < cols)
        p.tmem_cols *= 2;
    p.status = h->status;
    // By default two seconds and a microsecond for each k block of the longest reduction, which takes 0.2 to 0.3 (600 million
    // rows of 8 x 8: 2.5 s for the one tile)
    const int64_t kb = cdiv(std::max({p.pr[0].k_ext, p.pr[1].k_ext, w || pl.form == kReduce ? p.rows : 0}), kKB);
    p.timeout_ns = h->d.timeout_us ? h->d.timeout_us * 1000ull : 2000000000ull + static_cast<uint64_t>(kb) * 1000ull;
    const int cs = pl.pair * pl.split;
    const int clusters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(items, h->max_clusters[cs])));
    const size_t smem = linear_smem_bytes(pl.form != kRows, static_cast<uint32_t>(p.num_pipe) * p.slot_bytes,
                                          static_cast<uint32_t>(pl.recv_bufs) * pl.recv_bytes, h->groups);
    bool ok = false;
    const bool two = pl.pair == 2;
    if (w)
        ok = two ? launch_one<kRowsT, kReduce, 2>(p, clusters, cs, smem, st) : launch_one<kRowsT, kReduce, 1>(p, clusters, cs, smem, st);
    else if (pl.form == kRows)
        ok = two ? launch_one<kRows, -1, 2>(p, clusters, cs, smem, st) : launch_one<kRows, -1, 1>(p, clusters, cs, smem, st);
    else if (pl.bn > 256)
        ok = launch_one<kRowsT, -1, 2, true>(p, clusters, cs, smem, st);
    else if (pl.form == kRowsT)
        ok = two ? launch_one<kRowsT, -1, 2>(p, clusters, cs, smem, st) : launch_one<kRowsT, -1, 1>(p, clusters, cs, smem, st);
    else
        ok = two ? launch_one<kReduce, -1, 2>(p, clusters, cs, smem, st) : launch_one<kReduce, -1, 1>(p, clusters, cs, smem, st);
    return ok ? MLP_OK : MLP_ERR_CUDA;
}

// out[rows, out_cols] = A[rows, red] * B, B stored out_cols-major (b_mn: red x out_cols) or red-major.  Returns the
// product's items (at most), or 0 if a tensor map could not be made.
int64_t describe_rows(const mlp_linear *h, Problem &q, const Plan &pl, int64_t rows, const void *A, int64_t lda, const void *B,
                      int64_t out_cols, int64_t red, bool b_mn, bool offsets)
{
    q.k_ext = static_cast<int32_t>(red);
    const int64_t b_in = b_mn ? out_cols : red, b_out = b_mn ? red : out_cols;
    int64_t items;
    if (pl.form == kRows) {
        // (a box never reaches past the last row of a short matrix: copies that are mostly out of range measured
        // several times slower than full ones)
        const int prows = static_cast<int>(std::min<int64_t>(kPRows, rows));
        if (!operand(q, 0, false, A, red, rows, 1, lda, prows) || !operand(q, 1, b_mn, B, b_in, b_out, h->groups, b_in, pl.bn / pl.pair))
            return 0;
        q.q_ext = static_cast<int32_t>(out_cols);
        items = (cdiv(rows, kPRows * pl.pair) + h->groups - 1) * cdiv(out_cols, pl.bn);
    } else {
        const int qrows = static_cast<int>(std::min<int64_t>(pl.bn / pl.pair, rows));
        if (pl.bn > 256) {   // two halves, each a copy and an MMA of its own
            q.wide = static_cast<uint32_t>(pl.bn / 2 / pl.pair) * 128u;
            if (!operand(q, 1, false, A, red, rows, 1, lda, std::min(pl.bn / 2 / pl.pair, qrows)))
                return 0;
            if (q.copy_bytes[1] != q.wide)
                return 0;
            q.copy_bytes[1] *= 2;
        } else if (!operand(q, 1, false, A, red, rows, 1, lda, qrows)) {
            return 0;
        }
        if (!operand(q, 0, b_mn, B, b_in, b_out, h->groups, b_in, kPRows))
            return 0;
        q.p_ext = static_cast<int32_t>(out_cols);
        if (!offsets)
            q.dense_q_tiles = pl.q_tiles;
        items = (offsets ? cdiv(rows, pl.bn) + h->groups - 1 : pl.q_tiles) * cdiv(out_cols, kPRows * pl.pair);
    }
    q.dense_items = static_cast<int32_t>(items);
    return items;
}

// dW: P and Q have `rows` rows of pe and qe columns.
int64_t describe_reduce(const mlp_linear *h, Problem &q, const Plan &pl, int64_t rows, const void *P, int64_t ldp, int64_t pe,
                        const void *Q, int64_t ldq, int64_t qe, void *dW, bool f32)
{
    q.p_ext = static_cast<int32_t>(pe);
    q.q_ext = static_cast<int32_t>(qe);
    q.out = dW;
    q.out_f32 = f32;
    q.ld_out = qe;
    if (!operand(q, 0, true, P, pe, rows, 1, ldp, kPRows) || !operand(q, 1, true, Q, qe, rows, 1, ldq, pl.bn / pl.pair))
        return 0;
    const int64_t items = h->groups * cdiv(pe, kPRows * pl.pair) * cdiv(qe, pl.bn);
    q.dense_items = static_cast<int32_t>(items);
    return items;
}

// ------------------------------------------------------- dZ = dY act'(Z) and the bias gradient --
// With e = e^-t and s = sigmoid(t) = 1 / (1 + e): 1 - s = e s, without cancellation.
//   silu'(z) = s + z s (1 - s), t = z;   gelu'(z) = s + z s (1 - s) t', t = 2u.
// z is clamped to where e stays finite; beyond, the derivative is 0 or 1 to 23 digits (NaN stays NaN).  Two elements at a
// time in the two-wide fp32 instructions: the kernel below is bound by issue (element by element 4000 x 4096 took 26 us,
// and takes 21).  The product with dy is also summed, and in these instructions cannot become part of an fma in one of the
// places where it is used.
__device__ __forceinline__ uint64_t two(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 each(uint64_t d)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float clamp_nan(float x, float lim)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(lim));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(d), "f"(-lim));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}

// dy act'(z) of two elements.
template <int kAct>
__device__ __forceinline__ uint64_t act_grad(float2 dy, float2 z)
{
    if (kAct == kActNone)
        return two(dy.x, dy.y);
    if (kAct == kActRelu)
        return two(z.x <= 0.0f ? 0.0f : dy.x, z.y <= 0.0f ? 0.0f : dy.y);
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr float kLim = kAct == kActGelu ? 8.5f : 80.0f;
    const uint64_t v = two(clamp_nan(z.x, kLim), clamp_nan(z.y, kLim)), one = two(1.0f, 1.0f);
    uint64_t t, dt = one;   // -t log2(e), and t' (1 for silu)
    if (kAct == kActGelu) {
        const uint64_t q = mul2(v, v);
        constexpr float a = -2.0f * kGeluC * kGeluA * kLog2e, b = -2.0f * kGeluC * kLog2e;
        constexpr float c = 6.0f * kGeluC * kGeluA, d = 2.0f * kGeluC;
        t = mul2(v, fma2(two(a, a), q, two(b, b)));
        dt = fma2(two(c, c), q, two(d, d));
    } else {
        t = mul2(v, two(-kLog2e, -kLog2e));
    }
    const float2 tt = each(t);
    const uint64_t e = two(exp2_approx(tt.x), exp2_approx(tt.y));
    const float2 n = each(add2(e, one));
    const uint64_t s = two(rcp_approx(n.x), rcp_approx(n.y));
    uint64_t w = mul2(v, mul2(e, s));
    if (kAct == kActGelu)
        w = mul2(w, dt);
    return mul2(two(dy.x, dy.y), fma2(w, s, s));
}

struct GradParams {
    const __nv_bfloat16 *dy, *z;
    __nv_bfloat16 *dz;          // or null
    int64_t ld_dy, ld_z, ld_dz;
    int32_t rows, N, groups, block_rows, blocks;
    const int32_t *offsets;
    float *part;                // (blocks + groups) x N column sums, or null
};

// Rows of group e of the offsets `off` (device or shared memory; null: one group), clamped to the matrix.
__device__ __forceinline__ void group_range(const int32_t *off, int32_t rows, int32_t e, int32_t &lo, int32_t &hi)
{
    lo = off ? min(max(off[e], 0), rows) : 0;
    hi = off ? min(max(off[e + 1], lo), rows) : rows;
}

// dZ leaves rounded to bf16, the type of the tensor cores' operands beside bf16 X and W: 2^-9 of each element, which takes
// the gradients' error against 64 bits from 0.0017, that of their own bf16, to 0.0023.  (As two bf16 parts it would be exact
// enough to return to 0.0017, for twice the products: 2048 x 8192 x 8192 about 700 us instead of 370.)  The bias gradient
// sums what was not rounded; without an activation dZ is dY.
// One CTA: a block of rows x 256 columns.  Memory-bound: reads dY and Z once, writes dZ once; the column
// sums stay in registers and leave as one fp32 row per (block, group) pair.  Blocks and groups are both
// ascending ranges, so block + group numbers those pairs without collisions.  Rows are requested 32 at a time whatever
// groups they belong to (a group at a time, 25 rows of 7 groups took 5 us longer).  4000 x 4096 gelu, 32 groups: 21.3 us,
// 4.6 TB/s, 61 % of the issue slots.
template <int kAct>
__global__ void __launch_bounds__(256, 4) act_grad_kernel(const GradParams p)
{
    __shared__ __align__(8) float red[8][kStrip];
    __shared__ int32_t off_s[MLP_MAX_EXPERTS + 1];
    griddep_launch_dependents();
    griddep_wait();   // launched while the kernel before it runs, as all kernels here are
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int32_t col = blockIdx.x * kStrip + lane * 8;
    const bool col_ok = col < p.N;
    const int32_t b_lo = blockIdx.y * p.block_rows, b_hi = block_end(b_lo, p.block_rows, p.rows);
    const int32_t *off = nullptr;
    int32_t e = 0;
    if (p.offsets) {   // first group that ends past the block's start
        for (int32_t i = threadIdx.x; i <= p.groups; i += 256)
            off_s[i] = p.offsets[i];
        __syncthreads();
        off = off_s;
        int32_t lo = 0, hi = p.groups;
        while (lo < hi) {
            const int32_t mid = (lo + hi) / 2;
            if (off[mid + 1] > b_lo)
                hi = mid;
            else
                lo = mid + 1;
        }
        e = lo;
    }
    uint64_t acc[4] = {0, 0, 0, 0};   // pairs of columns
    auto flush = [&] {   // the sums of group e over this block's rows
        if (p.part) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float2 *>(&red[warp][lane * 8 + 2 * j]) = each(acc[j]);
            __syncthreads();
            const int32_t c = blockIdx.x * kStrip + threadIdx.x;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                s += red[w][threadIdx.x];
            if (c < p.N)
                p.part[static_cast<int64_t>(blockIdx.y + e) * p.N + c] = s;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = 0;
    };
    int32_t g_lo = 0, g_hi = 0;
    for (int32_t r0 = b_lo; r0 < b_hi && e < p.groups; r0 += 32) {
        const int32_t end = min(r0 + 32, b_hi);
        // all loads before any store: the stores of one row could be the loads of the next for all the compiler knows
        uint4 dyv[4], zv[4];
        if (col_ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t q = min(r0 + warp + 8 * i, end - 1);
                dyv[i] = __ldg(reinterpret_cast<const uint4 *>(p.dy + q * p.ld_dy + col));
                if (kAct != kActNone)
                    zv[i] = __ldg(reinterpret_cast<const uint4 *>(p.z + q * p.ld_z + col));
            }
        }
        for (; e < p.groups; ++e) {
            group_range(off, p.rows, e, g_lo, g_hi);
            if (g_lo >= end)
                break;
            if (col_ok) {
                const int32_t lo = max(g_lo, r0), hi = min(g_hi, end);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t r = r0 + warp + 8 * i;
                    if (r < lo || r >= hi)
                        continue;
                    const uint32_t dw[4] = {dyv[i].x, dyv[i].y, dyv[i].z, dyv[i].w};
                    uint32_t zw[4] = {0u, 0u, 0u, 0u};
                    if (kAct != kActNone) {
                        zw[0] = zv[i].x;
                        zw[1] = zv[i].y;
                        zw[2] = zv[i].z;
                        zw[3] = zv[i].w;
                    }
                    uint32_t ow[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t g = act_grad<kAct>(unpack2(dw[j]), unpack2(zw[j]));
                        acc[j] = add2(acc[j], g);
                        const float2 o = each(g);
                        ow[j] = pack2(o.x, o.y);
                    }
                    if (p.dz)
                        *reinterpret_cast<uint4 *>(p.dz + r * p.ld_dz + col) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                }
            }
            if (g_hi > end)
                break;   // it goes on
            if (g_hi > max(g_lo, b_lo))
                flush();
        }
    }
    if (e < p.groups && g_lo < b_hi && g_hi > b_hi)
        flush();   // it goes on in the next block
}

// dbias where no product is asked for that would add the sums on its way.
__global__ void __launch_bounds__(256) bias_grad_kernel(const BiasSums q, const int32_t *offsets, int32_t rows, uint32_t *status)
{
    griddep_launch_dependents();
    griddep_wait();
    if (ld_relaxed_gpu_u32(status) == kStTimeout)
        return;
    const int32_t e = static_cast<int32_t>(blockIdx.y);
    int32_t lo, hi;
    group_range(offsets, rows, e, lo, hi);
    if (offsets && threadIdx.x == 0 && (lo != offsets[e] || hi != offsets[e + 1]))
        atomicCAS(status, 0u, kStBadOffsets);
    add_bias_sums(q, e, blockIdx.x * 256 + threadIdx.x, lo, hi);
}

// Without an activation dZ is dY.  Where the bias gradient reads dY anyway, a copy of it whose rows start on those lines
// pays for itself in the products of many rows.
bool copies_dy(const mlp_linear *h, int64_t rows) { return h->d.activation == MLP_ACT_NONE && h->d.N % 64 != 0 && rows >= 256; }

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

bool misaligned(const void *p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool bad_matrix(const void *p, int64_t ld, int64_t cols) { return !p || misaligned(p) || ld < cols || ld % 8 != 0; }

bool bad_call(const mlp_linear *h, int64_t rows, const int32_t *offsets)
{
    return rows < 0 || rows > (int64_t{1} << 31) - 1024 || (h->d.experts > 0) != (offsets != nullptr) ||
           (offsets && misaligned(offsets, 4));
}

}  // namespace

extern "C" mlp_status mlp_linear_create(const mlp_linear_desc *d, mlp_linear_t *out)
{
    if (!d || !out)
        return MLP_ERR_INVALID_ARG;
    *out = nullptr;
    const int64_t lim = (int64_t{1} << 31) - 1024;
    if (d->K < 8 || d->N < 8 || d->K % 8 || d->N % 8 || d->K > lim || d->N > lim || d->experts < 0 ||
        d->experts > MLP_MAX_EXPERTS || d->weight_layout < 0 || d->weight_layout > 1 || d->device < 0)
        return MLP_ERR_INVALID_ARG;
    if (d->activation < MLP_ACT_NONE || d->activation > MLP_ACT_SILU ||
        (d->bias_dtype != MLP_DT_BF16 && d->bias_dtype != MLP_DT_F32) ||
        (d->dw_dtype != MLP_DT_BF16 && d->dw_dtype != MLP_DT_F32))
        return MLP_ERR_UNSUPPORTED;
    const OnDevice on(d->device);
    if (!on)
        return MLP_ERR_CUDA;
    mlp_linear *h = new (std::nothrow) mlp_linear();
    if (!h)
        return MLP_ERR_OOM;
    h->d = *d;
    h->groups = d->experts ? d->experts : 1;
    h->status = nullptr;
    mlp_status st = MLP_OK;
    if (!succeeded(cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, d->device)) ||
        !allow_smem<kRows, -1>() || !allow_smem<kRowsT, -1>() || !allow_smem<kReduce, -1>() || !allow_smem<kRowsT, kReduce>()) {
        st = MLP_ERR_CUDA;
    }
    for (int cs = 1; cs <= 8 && st == MLP_OK; ++cs) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(cs), 1, 1);
        cfg.blockDim = dim3(kLThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmemLimit;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (!succeeded(cudaOccupancyMaxActiveClusters(&n, linear_kernel<kRows, -1, 1, false>, &cfg)) || (n < 1 && cs <= 2))
            st = MLP_ERR_CUDA;
        h->max_clusters[cs] = n;
    }
    if (st == MLP_OK && !succeeded(cudaMalloc(&h->status, 256))) {
        h->status = nullptr;
        st = MLP_ERR_OOM;
    }
    if (st == MLP_OK && !succeeded(cudaMemset(h->status, 0, 256)))
        st = MLP_ERR_CUDA;
    if (st != MLP_OK) {
        if (h->status)
            cudaFree(h->status);
        delete h;
        return st;
    }
    *out = h;
    return MLP_OK;
}

extern "C" mlp_status mlp_linear_destroy(mlp_linear_t h)
{
    if (!h)
        return MLP_ERR_INVALID_ARG;
    const OnDevice on(h->d.device);
    succeeded(cudaFree(h->status));
    delete h;
    return MLP_OK;
}

// dZ, then the partial column sums.
static void workspace_layout(const mlp_linear *h, int64_t rows, size_t *part, size_t *total)
{
    const size_t dz = h->d.activation == MLP_ACT_NONE && !copies_dy(h, rows) ? 0 : align256(static_cast<size_t>(rows) * dz_pitch(h->d.N) * 2);
    const int64_t blocks = cdiv(rows, grad_block_rows(h->d.N, h->num_sms, rows));
    *part = dz;
    *total = dz + align256(static_cast<size_t>(blocks + h->groups) * h->d.N * 4);
}

extern "C" mlp_status mlp_linear_workspace_size(mlp_linear_t h, int64_t rows, size_t *bytes)
{
    if (!h || !bytes || rows < 0)
        return MLP_ERR_INVALID_ARG;
    size_t part;
    workspace_layout(h, rows, &part, bytes);
    return MLP_OK;
}

extern "C" mlp_status mlp_linear_forward(mlp_linear_t h, int64_t rows, const void *X, int64_t ldx, const void *W,
                                         const void *bias, const void *residual, int64_t ldr, const int32_t *offsets,
                                         void *Z, int64_t ldz, void *Y, int64_t ldy, void *stream)
{
    if (!h || bad_call(h, rows, offsets))
        return MLP_ERR_INVALID_ARG;
    const int64_t K = h->d.K, N = h->d.N;
    if (rows == 0)
        return MLP_OK;
    if (bad_matrix(X, ldx, K) || bad_matrix(Y, ldy, N) || !W || misaligned(W) || (residual && bad_matrix(residual, ldr, N)) ||
        (Z && bad_matrix(Z, ldz, N)) || (bias && misaligned(bias, h->d.bias_dtype == MLP_DT_F32 ? 4 : 2)))
        return MLP_ERR_INVALID_ARG;
    const OnDevice on(h->d.device);
    if (!on)
        return MLP_ERR_CUDA;
    LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.offsets = offsets;
    p.rows = static_cast<int32_t>(rows);
    Problem &q = p.pr[0];
    q.act = h->d.activation;
    q.bias = bias;
    q.bias_f32 = h->d.bias_dtype == MLP_DT_F32;
    q.res = static_cast<const __nv_bfloat16 *>(residual);
    q.ld_res = ldr;
    q.z = static_cast<__nv_bfloat16 *>(Z);
    q.ld_z = ldz;
    q.out = Y;
    q.ld_out = ldy;
    const bool kn = h->d.weight_layout == 0;
    const Plan pl = plan_rows(h, rows, N, K, kn, K);
    const int64_t items = describe_rows(h, q, pl, rows, X, ldx, W, N, K, kn, offsets != nullptr);
    return items ? launch(h, p, pl, nullptr, items, static_cast<cudaStream_t>(stream)) : MLP_ERR_CUDA;
}

extern "C" mlp_status mlp_linear_backward(mlp_linear_t h, int64_t rows, const void *dY, int64_t lddy, const void *X,
                                          int64_t ldx, const void *W, const void *Z, int64_t ldz, const int32_t *offsets,
                                          void *dX, int64_t lddx, void *dW, void *dbias, void *workspace, void *stream)
{
    if (!h || bad_call(h, rows, offsets))
        return MLP_ERR_INVALID_ARG;
    const int64_t K = h->d.K, N = h->d.N;
    const bool act = h->d.activation != MLP_ACT_NONE;
    const size_t bias_esz = h->d.bias_dtype == MLP_DT_F32 ? 4 : 2, dw_esz = h->d.dw_dtype == MLP_DT_F32 ? 4 : 2;
    if ((dW && misaligned(dW)) || (dbias && misaligned(dbias, bias_esz)))
        return MLP_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        const OnDevice on(h->d.device);
        if (!on || (dW && !succeeded(cudaMemsetAsync(dW, 0, static_cast<size_t>(h->groups) * K * N * dw_esz, st))) ||
            (dbias && !succeeded(cudaMemsetAsync(dbias, 0, static_cast<size_t>(h->groups) * N * bias_esz, st))))
            return MLP_ERR_CUDA;
        return MLP_OK;
    }
    if (bad_matrix(dY, lddy, N) || (act && bad_matrix(Z, ldz, N)) || (dW && bad_matrix(X, ldx, K)) ||
        (dX && (bad_matrix(dX, lddx, K) || !W || misaligned(W))) ||
        (((act && (dX || dW)) || dbias) && (!workspace || misaligned(workspace, 256))))
        return MLP_ERR_INVALID_ARG;
    const OnDevice on(h->d.device);
    if (!on)
        return MLP_ERR_CUDA;
    const void *dz = dY;
    int64_t ld_dz = lddy;
    BiasSums bias = {};
    if ((act && (dX || dW)) || dbias) {
        size_t part, total;
        workspace_layout(h, rows, &part, &total);
        GradParams g;
        std::memset(&g, 0, sizeof(g));
        g.dy = static_cast<const __nv_bfloat16 *>(dY);
        g.ld_dy = lddy;
        g.z = static_cast<const __nv_bfloat16 *>(Z);
        g.ld_z = ldz;
        if ((act || copies_dy(h, rows)) && (dX || dW)) {
            g.dz = static_cast<__nv_bfloat16 *>(workspace);
            dz = workspace;
            ld_dz = g.ld_dz = dz_pitch(N);
        }
        g.rows = static_cast<int32_t>(rows);
        g.N = static_cast<int32_t>(N);
        g.groups = h->groups;
        g.block_rows = grad_block_rows(h->d.N, h->num_sms, rows);
        g.blocks = static_cast<int32_t>(cdiv(rows, g.block_rows));
        g.offsets = offsets;
        g.part = dbias ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part) : nullptr;
        bias = BiasSums{g.part, dbias, g.N, g.block_rows, bias_esz == 4};
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(cdiv(N, kStrip)), static_cast<unsigned>(g.blocks));
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void (*const kernels[])(GradParams) = {act_grad_kernel<kActNone>, act_grad_kernel<kActRelu>, act_grad_kernel<kActGelu>,
                                               act_grad_kernel<kActSilu>};
        if (!succeeded(cudaLaunchKernelEx(&cfg, kernels[h->d.activation], g)))
            return MLP_ERR_CUDA;
        cfg.gridDim = dim3(static_cast<unsigned>(cdiv(N, 256)), static_cast<unsigned>(h->groups));
        if (dbias && !dX && !dW && !succeeded(cudaLaunchKernelEx(&cfg, bias_grad_kernel, bias, offsets, g.rows, h->status)))
            return MLP_ERR_CUDA;
    }
    if (!dX && !dW)
        return MLP_OK;
    const bool kn = h->d.weight_layout == 0;
    LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.offsets = offsets;
    p.rows = static_cast<int32_t>(rows);
    p.bias = bias;
    // dX[m, k] = sum_n dZ[m, n] W(k, n): W stored K x N has the reduction inside
    auto input_grad = [&](const Plan &pl) {
        p.pr[0].out = dX;
        p.pr[0].ld_out = lddx;
        return describe_rows(h, p.pr[0], pl, rows, dz, ld_dz, W, K, N, !kn, offsets != nullptr);
    };
    const int64_t pe = kn ? K : N, qe = kn ? N : K;
    auto weight_grad = [&](Problem &q, const Plan &pl) {
        return describe_reduce(h, q, pl, rows, kn ? X : dz, kn ? ldx : ld_dz, pe, kn ? dz : X, kn ? ld_dz : ldx, qe, dW, dw_esz == 4);
    };
    const GradPlan plans = plan_grads(h, rows);
    const Plan &px = plans.x, &pw = plans.w;
    if (dX && dW && plans.together) {
        const int64_t a = input_grad(px), b = weight_grad(p.pr[1], pw);
        return a && b ? launch(h, p, px, &pw, a + b, st) : MLP_ERR_CUDA;
    }
    if (dX) {
        const int64_t items = input_grad(px);
        const mlp_status r = items ? launch(h, p, px, nullptr, items, st) : MLP_ERR_CUDA;
        if (r != MLP_OK)
            return r;
        p.bias.out = nullptr;   // done
    }
    if (dW) {
        std::memset(p.pr, 0, sizeof(p.pr));
        const int64_t items = weight_grad(p.pr[0], pw);
        return items ? launch(h, p, pw, nullptr, items, st) : MLP_ERR_CUDA;
    }
    return MLP_OK;
}

extern "C" mlp_status mlp_linear_check(mlp_linear_t h, void *stream)
{
    if (!h)
        return MLP_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t v = 0;
    const OnDevice on(h->d.device);
    if (!on || !succeeded(cudaMemcpyAsync(&v, h->status, 4, cudaMemcpyDeviceToHost, st)) || !succeeded(cudaStreamSynchronize(st)))
        return MLP_ERR_CUDA;
    if (v && (!succeeded(cudaMemsetAsync(h->status, 0, 4, st)) || !succeeded(cudaStreamSynchronize(st))))
        return MLP_ERR_CUDA;
    return static_cast<mlp_status>(v);
}

extern "C" mlp_status mlp_linear_get_plan(mlp_linear_t h, int64_t rows, int32_t pass, mlp_linear_plan *plan)
{
    if (!h || !plan || rows < 1 || pass < 0 || pass > 2)
        return MLP_ERR_INVALID_ARG;
    const Plan pl = pass == 0 ? plan_rows(h, rows, h->d.N, h->d.K, h->d.weight_layout == 0, h->d.K)
                              : pass == 1 ? plan_grads(h, rows).x : plan_grads(h, rows).w;
    plan->form = pl.form;
    plan->cta_pair = pl.pair;
    plan->tile_cols = pl.bn;
    plan->k_split = pl.split;
    plan->pipe_stages = pl.pipe;
    return MLP_OK;
}
