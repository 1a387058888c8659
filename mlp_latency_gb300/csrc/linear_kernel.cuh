// linear_kernel.cuh -- the persistent, warp-specialised tcgen05 kernel behind mlp_linear: products of
// bf16 matrices with fp32 accumulators in TMEM, in three forms that differ in which dimension is
// ragged (the row ranges [start_e, start_e + cnt_e) of the groups; a dense product is one group):
//
//   kRows    D[rows of e, n] = sum_k A[row, k] B_e[k, n]      forward, and the input's gradient
//            (MMA rows = activation rows, MMA columns = weight columns)
//   kRowsT   the same product with the operands exchanged: MMA rows = weight columns, MMA columns =
//            activation rows.  An MMA always works on 128 rows; with few activation rows they are the
//            narrow operand here, so a tile reads 128 weight columns and 16 to 256 activation rows
//            per k block instead of 128 mostly empty activation rows.
//   kReduce  D_e[i, j] = sum_{rows of e} A[row, i] B[row, j]  the weights' gradient
//
// In MMA terms every form is D[p, q] = sum_k P[p, k] Q[q, k] with operands that are K-major or
// MN-major in memory (the descriptors' and the TMA boxes' business only).
//
// Roles (384 threads): warps 0 and 3 copy P and Q tiles into a ring (one thread each, for its even and its odd slots: a
// thread issues one 16 KB copy per ~400 cycles, longer than a fill's MMAs), warp 1 issues MMAs and owns TMEM, warp 2 builds
// the group tables and masks ragged reduction tails, warps 4-11 run the epilogue (two per TMEM lane quarter, on
// alternating column chunks).
// The accumulator is double buffered, so a tile's epilogue runs under the next tile's MMAs.  Tiles are dealt out
// statically, in an order that lets the CTAs running at one time share operand panels in L2.
//
// kWide (kRowsT on pairs): tiles of 257 to 512 activation rows, each k block two MMAs that share the weights' tile, in one
// accumulator, whose epilogue then runs under no MMA.  (As a flag at run time it cost the other tiles 10 %.)
//
// kFormB >= 0: a launch of two products, kForm's and kFormB's, whose tiles every CTA takes in turn.  The backward pass
// runs the input's and the weights' gradient this way.
//
// kPair = 2 runs 256-row tiles on CTA pairs (cta_group::2): each CTA loads its 128 rows of P and half
// of Q's tile, a third less to fetch per SM and flop.  split > 1 shares one tile's reduction among the
// CTAs (or pairs) of a cluster, each taking a range of k blocks; every CTA then finishes a range of the
// tile's columns, for which the others send it their partial sums through distributed shared memory, and
// adds them in slice order, so the result does not depend on timing.
//
// What bounds it, measured alone (bf16):
//   1 x 4096 x 14336            21.0 us   memory: 5.6 TB/s of weights, set-up and the last epilogue
//   128 x 4096 x 4096, split 4  13.6 us   set-up, exchange and epilogue; the k loop is a third
//   301 x 14336 x 4096          38.0 us   an SM's intake (64 bytes a cycle), 128 of 152 SMs at work
//   2048 x 8192 x 8192          185 us    1.5 PFLOP/s at the power cap (the first 60 launches after a pause 168), 3.8 rounds of 4
//   4000 rows, 32 experts of 2048 x 4096, both gradients  245 us   the order of the tiles (Walk::next)
// Tiles of 256 columns on pairs need the whole of that intake (32 KB per 512 cycles), which is why narrower ones do not get
// faster in proportion.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace mlpl {

using namespace mlpc;

enum Form { kRows = 0, kRowsT = 1, kReduce = 2 };
enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

constexpr int kLThreads = 384;
constexpr int kEpi = 8;                        // epilogue warps
constexpr int kPRows = 128;                    // rows of P per CTA (= TMEM lanes)
constexpr int kKB = 64;                        // reduction depth of one ring slot: 128 bytes of bf16
constexpr uint32_t kPBytes = kPRows * kKB * 2;
constexpr uint32_t kBoxBytes = kKB * 128;      // one MN-major box: 64 k rows of 64 columns
constexpr int kMaxRing = 10;
constexpr uint32_t kStageWarpBytes = 32 * 64;  // epilogue staging: 32 rows x 64 bytes per warp
constexpr uint32_t kStTimeout = 5, kStBadOffsets = 1;

// Shared memory of one CTA's share of a Q tile: `cols` K-major rows of 128 bytes, or whole boxes of 64 columns.
__host__ __device__ inline uint32_t q_tile_bytes(int32_t cols, bool mn)
{
    return mn ? static_cast<uint32_t>((cols + 63) / 64) * kBoxBytes : static_cast<uint32_t>(cols) * 128u;
}

// One product of a launch.
struct Problem {
    CUtensorMap map[2];             // P and Q: (inner, outer, group) views, or (64, outer, inner / 64, group)
    uint32_t copy_bytes[2];         // what one fill copies of each into a CTA
    uint32_t wide;                  // kRowsT on pairs, tiles of more than 256 columns: bytes of one of Q's two halves
    int32_t boxed[2];               // the four-dimensional view: all boxes of an MN-major tile in one copy
    int32_t mn[2];                  // operand stored MN-major (else K-major)
    int32_t dense_items;            // items without offsets
    int32_t dense_q_tiles;          // kRowsT, dense: tiles along the rows, from rows / bn up to one per column step
    int32_t p_ext, q_ext, k_ext;    // extents of the dimensions that are not ragged
    int32_t bn;                     // columns of a tile (the pair's)
    int32_t raster;                 // row panels sharing a sweep over the column tiles
    int32_t act;
    int32_t bias_f32, out_f32;
    const void *bias;               // groups x (output columns), or null
    const __nv_bfloat16 *res;       // or null
    __nv_bfloat16 *z;               // pre-activation output, or null
    void *out;
    int64_t ld_out, ld_res, ld_z;   // row strides in elements
};

// The bias gradient: partial rows of column sums, one per (block of rows, group) pair at block + group, to be added.
struct BiasSums {
    const float *part;
    void *out;                      // groups x N, or null
    int32_t N, block_rows, f32;
};

struct LinearParams {
    Problem pr[2];
    BiasSums bias;                  // added by the epilogue warps before their first tile
    const int32_t *offsets;         // device, groups + 1 entries, or null: one group of `rows` rows
    int32_t groups, rows;
    int32_t acc_cols;               // TMEM columns of one accumulator
    int32_t split;                  // CTAs, or pairs, sharing a tile's reduction
    int32_t part_align;             // granularity of the column ranges that they finish: 8 or 32
    int32_t recv_bufs;              // receive buffers for partial sums, of recv_bytes each; 0: the ring
    uint32_t recv_bytes;            // serves as the one buffer and the next tile's copies wait for it
    int32_t num_pipe;
    uint32_t slot_bytes;
    uint32_t tmem_cols;
    uint32_t *status;
    uint64_t timeout_ns;
};

struct __align__(8) LCtrl {
    uint64_t full[kMaxRing], empty[kMaxRing], tail[kMaxRing];
    uint64_t go[kMaxRing];   // leader to peer: the fill is armed
    uint64_t tfull[2], tempty[2];
    uint64_t drain, rdy[2], got[2], ringfree;
    uint64_t left;           // the copying threads and the MMA thread are through, and have noted what they leave in flight:
    uint32_t fills[2], tail_ph[2];   // of each copying thread
    uint32_t masked[kMaxRing];       // a slot's last masked fill
    uint32_t issued;
    uint32_t tmem_base;
    volatile int32_t abort_flag;
    int32_t skip;
    int32_t n_items[2];
};

// Shared memory: ring (1024-byte aligned), receive buffers, staging per epilogue warp, a chunk's bias per epilogue warp
// (kRows only), control block, group tables.
struct SmemMap {
    uint32_t recv, stage, bias, ctrl, tab;
    __host__ __device__ SmemMap(bool no_bias, uint32_t ring_bytes, uint32_t recv_total)
    {
        recv = ring_bytes;
        stage = recv + recv_total;
        bias = stage + kEpi * kStageWarpBytes;
        ctrl = bias + (no_bias ? 0u : kEpi * 32u * 4u);
        tab = ctrl + static_cast<uint32_t>((sizeof(LCtrl) + 15) / 16 * 16);
    }
};
__host__ inline size_t linear_smem_bytes(bool no_bias, uint32_t ring_bytes, uint32_t recv_total, int groups)
{
    return 1024 + SmemMap(no_bias, ring_bytes, recv_total).tab + (3 * static_cast<size_t>(groups) + 1) * 4;
}

__device__ __forceinline__ uint64_t policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Each thread of the warp reads 8 consecutive 32-bit columns of its own TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                                                 int32_t c3, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}

// True in one lane of a converged warp.  (elect.sync rather than a comparison of the lane number: the compiler then
// knows that the code under it runs in a single thread, and the uniform operands of tcgen05 and TMA instructions need
// no loop over the lanes.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t pred = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 r;\n\t"
        "elect.sync r|p, 0xffffffff;\n\t"
        "@p mov.u32 %0, 1;\n\t}\n"
        : "+r"(pred));
    return pred != 0;
}

// Order this thread's generic-proxy accesses of its CTA's shared memory with later async-proxy ones
// (TMA copies, MMA operand reads).
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------------------ bounded waits --
// On expiry: first error wins in the status word, the CTA's abort flag stops the other roles.  Draining waits (for own
// copies and MMAs in flight after an abort) ignore the flag and use a short limit.
__device__ __forceinline__ bool lwait(uint64_t *bar, uint32_t parity, LCtrl *c, const LinearParams &p,
                                      bool cluster = false, bool draining = false)
{
    auto probe = [&]() { return cluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (probe())
        return true;
    const uint64_t t0 = globaltimer_ns();
    const uint64_t limit = draining ? 200000000ull : p.timeout_ns;
    while (true) {
        if (probe())
            return true;
        if (!draining && c->abort_flag)
            return false;
        if (globaltimer_ns() - t0 > limit) {
            atomicCAS(p.status, 0u, kStTimeout);
            c->abort_flag = 1;
            return false;
        }
    }
}

// After an abort, before the CTA's shared memory and TMEM go away: waits for all copies and MMAs in flight.  By a thread of the
// first epilogue warp, since that one knows: if it saw all its tiles' accumulators, every MMA is over and every copy was
// read by one.  (The copying and MMA threads do not: another role's wait can run out after they are through.  Waits of
// their own at the end of every run cost 0.6 us of 13.4 where tiles have one k block.)
template <int kPair>
__device__ __noinline__ void land(LCtrl *c, const LinearParams &p)
{
    if (!lwait(&c->left, 0, c, p, false, true))
        return;
    const bool half = kPair == 2 && (cluster_ctarank() & 1u) != 0;
    if (c->issued && !lwait(&c->drain, 0, c, p, false, true))
        return;
    // Each copy on its slot's last barrier phase.  Unmasked fills of a pair complete on the leader's barriers (the peer fills
    // only what the leader armed, and keeps its shared memory until the cluster barriers at the end); masked fills complete
    // on each CTA's own.  A wait that ran out was long enough for the rest.
    const bool shared_ring = p.split > 1 && p.recv_bufs == 0;
    const uint32_t num_pipe = static_cast<uint32_t>(p.num_pipe);
    for (uint32_t which = 0; which < (shared_ring ? 1u : 2u); ++which)
        for (uint32_t fills = c->fills[which], f = fills > num_pipe ? fills - num_pipe : 0u; f < fills; ++f) {
            const uint32_t slot = f % num_pipe;
            if (!shared_ring && (slot & 1u) != which)
                continue;
            if (c->masked[slot] == f) {
                if (!lwait(&c->tail[slot], (c->tail_ph[which] >> slot & 1u) ^ 1u, c, p, false, true))
                    return;
            } else if (!half && !lwait(&c->full[slot], (f / num_pipe) & 1u, c, p, false, true)) {
                return;
            }
        }
}

// Accumulator of an item, and the parity of its uses.  Wide tiles have one: two are more than TMEM holds.
template <bool kWide>
__device__ __forceinline__ uint32_t acc_of(uint32_t tiles) { return kWide ? 0u : tiles & 1u; }
template <bool kWide>
__device__ __forceinline__ uint32_t acc_parity(uint32_t tiles) { return (kWide ? tiles : tiles >> 1) & 1u; }

// Columns of the first of a wide tile's two MMAs.
template <int kPair>
__device__ __forceinline__ int32_t first_half(int32_t n)
{
    constexpr int32_t u = 16 * kPair;
    return (n / u + 1) / 2 * u;
}

// Lane 0 waits, then every lane acquires the completed phase itself.
__device__ __forceinline__ bool lwait_warp(uint64_t *bar, uint32_t parity, LCtrl *c, const LinearParams &p,
                                           bool cluster = false)
{
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0)
        ok = lwait(bar, parity, c, p, cluster) ? 1u : 0u;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok)
        return false;
    if (cluster)
        mbar_try_wait_cluster(bar, parity);
    else
        mbar_try_wait(bar, parity);
    return true;
}

// ---------------------------------------------------------------------------------- activations --
// x sigmoid(t) as x / (1 + e^-t): relative accuracy for every sign of t (a tanh form cancels for
// t << 0) down to t = -87, where the result is below 2^-119; from there on the quotient is the limit 0.
__device__ __forceinline__ float x_sigmoid(float x, float t) { return __fdividef(x, 1.0f + __expf(-t)); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// gelu(x) = x (1 + tanh u) / 2 = x sigmoid(2u), u = c (x + a x^3)
__device__ __forceinline__ float act_fwd(int act, float x)
{
    if (act == kActGelu)
        return x_sigmoid(x, x * fmaf(2.0f * kGeluC * kGeluA, x * x, 2.0f * kGeluC));
    if (act == kActSilu)
        return x_sigmoid(x, x);
    if (act == kActRelu)
        return x < 0.0f ? 0.0f : x;   // NaN stays NaN
    return x;
}

// ---------------------------------------------------------------------------------------- items --
struct GroupTab {
    int32_t *start, *cnt, *base;   // rows of each group; items before each group (groups + 1)
};

struct Tile {
    int32_t which;       // product of the launch
    int32_t e, start, cnt;
    int32_t p0, q0;      // origin in the P and Q extents (inside the group's rows for a ragged one)
    int32_t n;           // MMA columns: bn, or what is left of the group's rows for kRowsT
    int32_t kb0, kb1;    // k blocks of this CTA's slice
};

// kRowsT: tiles that a group's rows are dealt over.
__device__ __forceinline__ int32_t q_tiles(const Problem &q, int32_t cnt)
{
    return q.dense_q_tiles ? q.dense_q_tiles : (cnt + q.bn - 1) / q.bn;
}

template <int kForm, int kPair>
__device__ __forceinline__ int32_t items_of(const Problem &q, int32_t cnt)
{
    constexpr int32_t bm = kPRows * kPair;
    if (kForm == kRows)
        return (cnt + bm - 1) / bm * ((q.q_ext + q.bn - 1) / q.bn);
    if (kForm == kRowsT)
        return q_tiles(q, cnt) * ((q.p_ext + bm - 1) / bm);
    return (q.p_ext + bm - 1) / bm * ((q.q_ext + q.bn - 1) / q.bn);
}

// One role's walk over its CTA's items: a product's ids grow, so the group only ever advances.
template <int kForm, int kFormB, int kPair>
struct Walk {
    int32_t id, id_b, step, e, slice, turn;
    __device__ __forceinline__ Walk(const LinearParams &p)
        : id(static_cast<int32_t>(cluster_id_x())), step(static_cast<int32_t>(num_clusters_x())), e(0),
          slice(p.split > 1 ? static_cast<int32_t>(cluster_ctarank()) / kPair : 0), turn(0)
    {
        id_b = step - 1 - id;   // (dealt from the other end: a CTA with one tile more of one has fewer of the other)
    }
    __device__ __forceinline__ bool next(const LinearParams &p, const GroupTab &g, int32_t n_items, int32_t n_items_b, Tile &t)
    {
        if (kFormB < 0) {
            if (id >= n_items)
                return false;
            t.which = 0;
            place<kForm>(p, g, id, true, t);
            id += step;
            return true;
        }
        const bool a = id < n_items, b = id_b < n_items_b;
        if (!a && !b)
            return false;
        // (One to one while both have tiles left.  Where one product has many more, as the weights' gradient of many small
        // experts has, the other's come all at the start: the input's gradient reads the weights first, and what is left
        // only writes, at the 3.9 TB/s of write-only traffic instead of the 6.8 of a copy.)
        t.which = a && b ? turn : b;
        turn ^= 1;
        if (t.which == 0) {
            place<kForm>(p, g, id, true, t);
            id += step;
        } else {
            place<kFormB < 0 ? kForm : kFormB>(p, g, id_b, false, t);
            id_b += step;
        }
        return true;
    }
    // tabled: the group tables count this product's items (else every group has the same number)
    template <int kF>
    __device__ __forceinline__ void place(const LinearParams &p, const GroupTab &g, int32_t item, bool tabled, Tile &t)
    {
        const Problem &q = p.pr[kFormB < 0 ? 0 : t.which];
        constexpr int32_t bm = kPRows * kPair;
        const int32_t tiles_q = (q.q_ext + q.bn - 1) / q.bn;   // (not for kRowsT)
        int32_t i = item;
        t.e = 0;
        t.start = 0;
        t.cnt = p.rows;
        if (p.offsets) {
            if (kF == kReduce) {
                const int32_t each = (q.p_ext + bm - 1) / bm * tiles_q;
                t.e = item / each;
                i = item - t.e * each;
            } else {
                while (item >= g.base[e + 1])
                    ++e;
                t.e = e;
                i = item - g.base[e];
            }
            t.start = g.start[t.e];
            t.cnt = g.cnt[t.e];
        }
        const int32_t kext = kF == kReduce ? t.cnt : q.k_ext;
        const int32_t nkb = (kext + kKB - 1) / kKB;
        if (kF == kRowsT) {
            // the group's rows in units of the MMA's column step, dealt evenly over the tiles
            constexpr int32_t u = 16 * kPair;
            const int32_t units = (t.cnt + u - 1) / u;
            const int32_t tq = q_tiles(q, t.cnt);
            const int32_t pi = i / tq, qi = i - pi * tq;
            const int32_t each = units / tq, more = units - each * tq;
            t.p0 = pi * bm;
            t.q0 = (qi * each + min(qi, more)) * u;
            t.n = (each + (qi < more ? 1 : 0)) * u;
        } else {
            const int32_t tp = ((kF == kRows ? t.cnt : q.p_ext) + bm - 1) / bm;
            const int32_t band = i / (q.raster * tiles_q), first = band * q.raster;
            const int32_t h = min(q.raster, tp - first), r = i - first * tiles_q;
            t.q0 = r / h * q.bn;
            t.p0 = (first + r % h) * bm;
            t.n = q.bn;
        }
        if (p.split > 1) {
            const int32_t per = (nkb + p.split - 1) / p.split;
            t.kb0 = min(slice * per, nkb);
            t.kb1 = min(t.kb0 + per, nkb);
        } else {
            t.kb0 = 0;
            t.kb1 = nkb;
        }
    }
};

// The form of a tile's product: known at compile time in a launch of one.
template <int kForm, int kFormB>
__device__ __forceinline__ int form_of(const Tile &t)
{
    return kFormB < 0 ? kForm : t.which ? kFormB : kForm;
}
template <int kFormB>
__device__ __forceinline__ const Problem &problem_of(const LinearParams &p, const Tile &t)
{
    return p.pr[kFormB < 0 ? 0 : t.which];
}

// A group's last k block holds rows of the next group when the reduction runs over a group's rows:
// they are zeroed in shared memory.  (At the very end of the matrix the copy fills zeros itself.)
__device__ __forceinline__ int32_t masked_rows(int form, const LinearParams &p, const Tile &t, int32_t kb)
{
    if (form != kReduce)
        return 0;
    const int32_t have = t.cnt - kb * kKB;
    return have < kKB && t.start + t.cnt < p.rows ? kKB - have : 0;
}

// ------------------------------------------------------------------------------- TMA producers --
// One of two threads, `which` = 0 or 1: the fills of the ring's even or odd slots.  (A slot always has the same thread: with
// fills in turn and an odd number of slots, a pair's second CTA could take the barrier by which its leader armed one fill of a
// slot for that of the fill after next, when the leader's other thread lagged.)
template <int kForm, int kFormB, int kPair, bool kWide>
__device__ __forceinline__ void l_role_tma(const LinearParams &p, LCtrl *c, const GroupTab g, uint8_t *ring, uint32_t which,
                                           Walk<kForm, kFormB, kPair> w, Tile t, bool have)
{
    constexpr bool kMasks = kForm == kReduce || kFormB == kReduce;
    const uint32_t num_pipe = static_cast<uint32_t>(p.num_pipe);
    const uint32_t slot_bytes = p.slot_bytes;
    const uint32_t rank = cluster_ctarank();
    const uint32_t half = kPair == 2 ? (rank & 1u) : 0u;
    const uint32_t full_lead0 = kPair == 2 ? map_to_rank(&c->full[0], rank & ~1u) : 0u;
    const uint32_t go_peer0 = kPair == 2 ? map_to_rank(&c->go[0], rank | 1u) : 0u;
    const uint32_t tail_own0 = kPair == 2 ? map_to_rank(&c->tail[0], rank) : 0u;
    const bool shared_ring = p.split > 1 && p.recv_bufs == 0;
    const int32_t n_items = c->n_items[0], n_items_b = c->n_items[1];
    const uint64_t pol = policy_evict_normal();
    uint32_t fills = 0, tail_ph = 0, item_ph = 0;
    uint32_t ps = 0, pph = 0;
    bool ok = true, first = true;
    griddep_wait();   // a programmatic launch: the kernel before this one is complete from here on
    for (; ok && have; have = w.next(p, g, n_items, n_items_b, t)) {
        const int form = form_of<kForm, kFormB>(t);
        const Problem &q = problem_of<kFormB>(p, t);
        const bool p_mn = q.mn[0] != 0, q_mn = q.mn[1] != 0, p_boxed = q.boxed[0] != 0, q_boxed = q.boxed[1] != 0;
        const uint32_t bytes = q.copy_bytes[0] + q.copy_bytes[1];
        const int32_t q_boxes = static_cast<int32_t>(q.copy_bytes[1] / kBoxBytes);
        const CUtensorMap *const map_p = &q.map[0], *const map_q = &q.map[1];
        // The ring was the exchange buffer of the previous item.  (One thread makes all copies then: a thread without a
        // copy in some item could fall a phase of this barrier behind.)
        if (shared_ring && which == 0) {
            if (!first) {
                if (!lwait(&c->ringfree, item_ph, c, p))
                    break;
                item_ph ^= 1;
            }
            first = false;
        }
        // first row (column of an MN-major operand) of this CTA's share of each tile, and the group
        const int32_t p_row = (form == kRows ? t.start : 0) + t.p0 + static_cast<int32_t>(half) * kPRows;
        const int32_t n1 = kWide ? first_half<kPair>(t.n) : t.n;
        const int32_t q_row = (form == kRowsT ? t.start : 0) + t.q0 + static_cast<int32_t>(half) * (n1 / kPair);
        const int32_t q_row2 = t.start + t.q0 + n1 + static_cast<int32_t>(half) * ((t.n - n1) / kPair);
        const int32_t p_grp = form == kRowsT ? t.e : 0, q_grp = form == kRows ? t.e : 0;
        int32_t k = (form == kReduce ? t.start : 0) + t.kb0 * kKB;
        for (int32_t kb = t.kb0; kb < t.kb1; ++kb, k += kKB) {
            if (shared_ring ? which == 0 : (ps & 1u) == which) {
                if (kPair == 2 && half) {
                    if (!lwait(&c->go[ps], pph, c, p, true)) {   // the leader armed this fill
                        ok = false;
                        break;
                    }
                } else if (!lwait(&c->empty[ps], pph ^ 1u, c, p)) {
                    ok = false;
                    break;
                }
                const bool masked = kMasks && masked_rows(form, p, t, kb) != 0;
                if (masked) {
                    // completes on this CTA's own tail barrier; warp 2 zeroes the rows and completes `full`
                    mbar_arrive_expect_tx(&c->tail[ps], bytes);
                    c->masked[ps] = fills;
                } else if (!half) {
                    mbar_arrive_expect_tx(&c->full[ps], kPair * bytes);
                    if (kMasks && kPair == 2)
                        mbar_arrive(&c->full[ps]);   // (the count is 2: one per CTA's warp 2 on a masked fill)
                }
                if (kPair == 2 && !half)
                    mbar_arrive_relaxed_cluster(go_peer0 + 8u * ps, 1);   // publishes no data
                uint8_t *a = ring + ps * slot_bytes, *b = a + kPBytes;
                const uint32_t fb = kPair == 2 ? (masked ? tail_own0 : full_lead0) + 8u * ps : 0u;
                uint64_t *lb = masked ? &c->tail[ps] : &c->full[ps];
                auto load3 = [&](uint8_t *dst, const CUtensorMap *m, int32_t c0, int32_t c1, int32_t c2) {
                    if (kPair == 2)
                        tma_load_3d_pair(dst, m, fb, c0, c1, c2, pol);
                    else
                        tma_load_3d(dst, m, lb, c0, c1, c2, pol);
                };
                auto load4 = [&](uint8_t *dst, const CUtensorMap *m, int32_t c1, int32_t c2, int32_t c3) {
                    if (kPair == 2)
                        tma_load_4d_pair(dst, m, fb, 0, c1, c2, c3, pol);
                    else
                        tma_load_4d(dst, m, lb, 0, c1, c2, c3, pol);
                };
                if (!p_mn) {
                    load3(a, map_p, k, p_row, p_grp);
                } else if (p_boxed) {
                    load4(a, map_p, k, p_row >> 6, p_grp);
                } else {
                    load3(a, map_p, p_row, k, p_grp);
                    load3(a + kBoxBytes, map_p, p_row + 64, k, p_grp);
                }
                if (!q_mn) {
                    load3(b, map_q, k, q_row, q_grp);
                    if (kWide)
                        load3(b + q.wide, map_q, k, q_row2, q_grp);
                } else if (q_boxed) {
                    load4(b, map_q, k, q_row >> 6, q_grp);
                } else {
                    for (int32_t j = 0; j < q_boxes; ++j)
                        load3(b + j * kBoxBytes, map_q, q_row + 64 * j, k, q_grp);
                }
            }
            if (kMasks && masked_rows(form, p, t, kb) != 0)
                tail_ph ^= 1u << ps;   // (the other thread's too: the slot's tail barrier counts both)
            ++fills;
            if (++ps == num_pipe) {
                ps = 0;
                pph ^= 1u;
            }
        }
    }
    c->fills[which] = fills;
    c->tail_ph[which] = tail_ph;
    mbar_arrive(&c->left);
}

// ---------------------------------------------------------------------------------- MMA issuer --
template <int kForm, int kFormB, int kPair, bool kWide>
__device__ __forceinline__ void l_role_mma(const LinearParams &p, LCtrl *c, const GroupTab g, uint8_t *ring,
                                           uint32_t tmem_base)
{
    if (kPair == 2 && (cluster_ctarank() & 1u)) {   // the leader issues for both
        c->issued = 0;
        mbar_arrive(&c->left);
        return;
    }
    const int32_t num_pipe = p.num_pipe;
    const uint32_t acc_cols = static_cast<uint32_t>(p.acc_cols);
    const uint32_t tfull_peer0 = kPair == 2 ? map_to_rank(&c->tfull[0], cluster_ctarank() | 1u) : 0u;
    const uint32_t base = smem_u32(ring);
    const uint64_t slot16 = p.slot_bytes >> 4;
    const int32_t n_items = c->n_items[0], n_items_b = c->n_items[1];
    // K-major: 8-row groups 1024 bytes apart, a 16-deep k step 32 bytes along the row.  MN-major: 64
    // columns x 64 k per box, boxes kBoxBytes apart, a k step 16 rows of 128 bytes.  Slot offsets add to
    // the 14-bit address field in 16-byte units (shared memory is below 2^18 bytes: no carry).
    uint32_t idesc0 = 0;
    uint64_t pd = 0, qd = 0, pstep = 0, qstep = 0;
    auto describe = [&](const Problem &q) {
        idesc0 = idesc_bf16_f32(kPRows * kPair, 0, q.mn[1] ? 1u : 0u) | (q.mn[0] ? 1u << 15 : 0u);
        pd = q.mn[0] ? smem_desc(base, kBoxBytes, 1024u, 2u) : smem_desc(base, 16u, 1024u, 2u);
        qd = q.mn[1] ? smem_desc(base + kPBytes, kBoxBytes, 1024u, 2u) : smem_desc(base + kPBytes, 16u, 1024u, 2u);
        pstep = q.mn[0] ? 128u : 2u;
        qstep = q.mn[1] ? 128u : 2u;
    };
    if (kFormB < 0)
        describe(p.pr[0]);
    int32_t ps = 0;
    uint32_t pph = 0, tiles = 0;
    bool issued = false, ok = true;
    Walk<kForm, kFormB, kPair> w(p);
    Tile t;
    while (w.next(p, g, n_items, n_items_b, t)) {
        if (kFormB >= 0)
            describe(problem_of<kFormB>(p, t));
        const uint32_t acc = acc_of<kWide>(tiles);
        if (!lwait(&c->tempty[acc], acc_parity<kWide>(tiles) ^ 1u, c, p, kPair == 2))
            break;
        tc_fence_after();
        // As the copying threads do: what is left of the kernel before counts against no wait's limit.  (Only now, when all that
        // a tile needs is at hand: before the walk it cost 0.2 us of 14.)
        if (tiles == 0)
            griddep_wait();
        const uint32_t d = tmem_base + acc * acc_cols;
        const uint32_t n1 = static_cast<uint32_t>(kWide ? first_half<kPair>(t.n) : t.n), n2 = static_cast<uint32_t>(t.n) - n1;
        const uint32_t idesc = idesc0 | (n1 >> 3) << 17, idesc2 = idesc0 | (n2 >> 3) << 17;
        const uint64_t wide16 = p.pr[0].wide >> 4;
        uint32_t accum = 0;
        for (int32_t kb = t.kb0; kb < t.kb1; ++kb) {
            if (!lwait(&c->full[ps], pph, c, p, kPair == 2)) {
                ok = false;
                break;
            }
            const uint64_t off = static_cast<uint64_t>(ps) * slot16;
#pragma unroll
            for (uint32_t kk = 0; kk < kKB / 16; ++kk) {
                mma_bf16_ss_g<kPair>(d, pd + off + pstep * kk, qd + off + qstep * kk, idesc, accum);
                if (kWide && n2 != 0)   // (an MMA has at most 256 columns)
                    mma_bf16_ss_g<kPair>(d + n1, pd + off + pstep * kk, qd + off + wide16 + qstep * kk, idesc2, accum);
                accum = 1u;
            }
            issued = true;
            mma_commit_g<kPair>(smem_u32(&c->empty[ps]));
            if (++ps == num_pipe) {
                ps = 0;
                pph ^= 1;
            }
        }
        if (!ok)
            break;
        mma_commit_g<kPair>(smem_u32(&c->tfull[acc]));
        if (kPair == 2)
            mma_commit_g<kPair>(tfull_peer0 + acc * 8u);
        ++tiles;
    }
    if (issued)
        mma_commit_g<kPair>(smem_u32(&c->drain));
    c->issued = issued;
    mbar_arrive(&c->left);
}

// ---------------------------------------------------------------- ragged reduction tails (warp 2) --
template <int kForm, int kFormB, int kPair>
__device__ __forceinline__ void l_role_mask(const LinearParams &p, LCtrl *c, const GroupTab g, uint8_t *ring)
{
    const int32_t lane = threadIdx.x & 31;
    const int32_t num_pipe = p.num_pipe;
    const uint32_t boxes = (kPBytes + q_tile_bytes(p.pr[kFormB < 0 ? 0 : 1].bn / kPair, true)) / kBoxBytes;   // P's two, then Q's
    const uint32_t full_lead0 = kPair == 2 ? map_to_rank(&c->full[0], cluster_ctarank() & ~1u) : 0u;
    const int32_t n_items = c->n_items[0], n_items_b = c->n_items[1];
    uint32_t fills = 0, tail_ph = 0;
    Walk<kForm, kFormB, kPair> w(p);
    Tile t;
    while (w.next(p, g, n_items, n_items_b, t)) {
        if (t.kb1 <= t.kb0)
            continue;
        const int32_t zero = masked_rows(form_of<kForm, kFormB>(t), p, t, t.kb1 - 1);
        fills += static_cast<uint32_t>(t.kb1 - t.kb0);
        if (!zero)
            continue;
        const int32_t ps = static_cast<int32_t>((fills - 1) % static_cast<uint32_t>(num_pipe));
        if (!lwait_warp(&c->tail[ps], (tail_ph >> ps) & 1u, c, p))
            return;
        tail_ph ^= 1u << ps;
        // a k row is 128 contiguous bytes of each box (the swizzle permutes inside them)
        uint8_t *s = ring + static_cast<size_t>(ps) * p.slot_bytes;
        const uint32_t segs = static_cast<uint32_t>(zero) * 8u;
        for (uint32_t b = 0; b < boxes; ++b)
            for (uint32_t i = lane; i < segs; i += 32)
                *reinterpret_cast<uint4 *>(s + b * kBoxBytes + (kKB - zero) * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (kPair == 2)
                mbar_arrive_cluster(full_lead0 + 8u * static_cast<uint32_t>(ps));
            else
                mbar_arrive(&c->full[ps]);
        }
    }
}

// ------------------------------------------------------------------------------------- epilogue --
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Offset of 16-byte segment `seg` (0-3) of row `row` in a warp's 32 x 64-byte staging buffer.  kSwizzle: accessed a
// row per lane, so the XOR spreads eight consecutive rows over all banks.
template <bool kSwizzle>
__device__ __forceinline__ uint32_t stg(int row, int seg)
{
    return static_cast<uint32_t>(row * 64 + ((kSwizzle ? seg ^ ((row >> 1) & 3) : seg) * 16));
}

// Where a lane's 16-byte pieces of a 32 x 64-byte chunk lie in global memory: rows (lane >> 2) + 8 i, segment lane & 3.
struct Piece {
    uint8_t *at;        // of the chunk at hand
    int64_t step;       // eight rows
    int64_t next;       // to this warp's next chunk
    __device__ __forceinline__ void init(const void *base, int64_t row, int32_t col, int64_t ld, int32_t esz, bool down, int32_t lane)
    {
        const int64_t ldb = ld * esz;
        at = const_cast<uint8_t *>(static_cast<const uint8_t *>(base)) + (row + (lane >> 2)) * ldb + static_cast<int64_t>(col) * esz +
             (lane & 3) * 16;
        step = 8 * ldb;
        next = down ? 8 * step : 64 * esz;   // 64 rows or 64 columns on
    }
};

// The staged 32 rows x 4 segments to global memory; rows and segments past the limits are skipped.
template <bool kSwizzle>
__device__ __forceinline__ void stage_store(const uint8_t *stage, const Piece &g, int32_t row_lim, int32_t seg_lim, int32_t lane)
{
    const int32_t r0 = lane >> 2, sg = lane & 3;
    // (eight rows on, the swizzle is the same: (row >> 1) & 3 has period 8)
    const uint4 *s = reinterpret_cast<const uint4 *>(stage + stg<kSwizzle>(r0, sg));
    const uint4 a = s[0], b = s[32], c = s[64], d = s[96];
    if (row_lim >= 32 && seg_lim >= 4) {
        *reinterpret_cast<uint4 *>(g.at) = a;
        *reinterpret_cast<uint4 *>(g.at + g.step) = b;
        *reinterpret_cast<uint4 *>(g.at + 2 * g.step) = c;
        *reinterpret_cast<uint4 *>(g.at + 3 * g.step) = d;
    } else if (sg < seg_lim) {
        if (r0 < row_lim)
            *reinterpret_cast<uint4 *>(g.at) = a;
        if (r0 + 8 < row_lim)
            *reinterpret_cast<uint4 *>(g.at + g.step) = b;
        if (r0 + 16 < row_lim)
            *reinterpret_cast<uint4 *>(g.at + 2 * g.step) = c;
        if (r0 + 24 < row_lim)
            *reinterpret_cast<uint4 *>(g.at + 3 * g.step) = d;
    }
}

// The residual's piece of a chunk: requested early, staged when it is needed.
__device__ __forceinline__ void res_load(uint4 (&x)[4], const Piece &g, int32_t row_lim, int32_t seg_lim, int32_t lane)
{
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        x[it] = make_uint4(0u, 0u, 0u, 0u);
        if (it * 8 + (lane >> 2) < row_lim && (lane & 3) < seg_lim)
            x[it] = *reinterpret_cast<const uint4 *>(g.at + it * g.step);
    }
}
template <bool kSwizzle>
__device__ __forceinline__ void res_stage(const uint4 (&x)[4], uint8_t *stage, int32_t lane)
{
#pragma unroll
    for (int it = 0; it < 4; ++it)
        *reinterpret_cast<uint4 *>(stage + stg<kSwizzle>(it * 8 + (lane >> 2), lane & 3)) = x[it];
    __syncwarp();
}

__device__ __forceinline__ float load_bias(const Problem &p, int64_t i)
{
    return p.bias_f32 ? static_cast<const float *>(p.bias)[i]
                      : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[i]);
}

// A 32 x 32 chunk of the output on its way out.  Rows are output rows, so with TMEM lane = output row (kLaneRow) a
// lane holds a row of the chunk, and with lane = output column (kRowsT) a column; both go through the staging buffer
// so that global memory is touched in 64-byte row pieces.
template <bool kLaneRow>
__device__ __forceinline__ void put_bf16(const float (&v)[32], uint8_t *stage, int32_t lane)
{
    if (kLaneRow) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            *reinterpret_cast<uint4 *>(stage + stg<true>(lane, s)) =
                make_uint4(pack2(v[8 * s], v[8 * s + 1]), pack2(v[8 * s + 2], v[8 * s + 3]),
                           pack2(v[8 * s + 4], v[8 * s + 5]), pack2(v[8 * s + 6], v[8 * s + 7]));
    } else {
        __nv_bfloat16 *mine = reinterpret_cast<__nv_bfloat16 *>(stage) + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            mine[32 * j] = __float2bfloat16_rn(v[j]);
    }
    __syncwarp();
}

template <int kAct, bool kLaneRow>
__device__ __forceinline__ void finish_chunk(const Problem &p, float (&v)[32], uint8_t *stage, const Piece &out, const Piece &zp,
                                             const uint4 (&res)[4], int32_t row_lim, int32_t seg_lim, int32_t lane)
{
    if (p.z) {
        put_bf16<kLaneRow>(v, stage, lane);
        stage_store<kLaneRow>(stage, zp, row_lim, seg_lim, lane);
        __syncwarp();
    }
    if (kAct != kActNone) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[j] = act_fwd(kAct, v[j]);
    }
    if (p.res) {
        res_stage<kLaneRow>(res, stage, lane);
        if (kLaneRow) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint4 x = *reinterpret_cast<const uint4 *>(stage + stg<true>(lane, s));
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2(xw[j]);
                    v[8 * s + 2 * j] += f.x;
                    v[8 * s + 2 * j + 1] += f.y;
                }
            }
        } else {
            const __nv_bfloat16 *mine = reinterpret_cast<const __nv_bfloat16 *>(stage) + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] += __bfloat162float(mine[32 * j]);
        }
        __syncwarp();
    }
    put_bf16<kLaneRow>(v, stage, lane);
    stage_store<kLaneRow>(stage, out, row_lim, seg_lim, lane);
    __syncwarp();
}

// 32 x 32 fp32 values, 16 columns at a time.
__device__ __forceinline__ void finish_f32(const float (&v)[32], uint8_t *stage, Piece out, int32_t row_lim, int32_t cols, int32_t lane)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            *reinterpret_cast<float4 *>(stage + stg<true>(lane, s)) =
                make_float4(v[16 * h + 4 * s], v[16 * h + 4 * s + 1], v[16 * h + 4 * s + 2], v[16 * h + 4 * s + 3]);
        __syncwarp();
        stage_store<true>(stage, out, row_lim, (cols - 16 * h) / 4, lane);
        out.at += 64;
        __syncwarp();
    }
}

// What a warp of the epilogue carries from item to item.
struct EpiState {
    int32_t quarter, which, lane;   // TMEM lane quarter (= warp % 4); of its two warps the even or odd chunks
    uint32_t rank, half;
    uint8_t *stage, *recv_base;
    float *bias_s;
    uint32_t tmem_lanes;            // TMEM address of its lanes
    uint32_t tempty_lead0;
    uint32_t tiles;
    int32_t buf;                    // receive buffer of this item, and how often it was used before (parity)
    uint32_t buf_ph;
    int32_t keep;                   // -1, or 0: the launch before ended in a wait that ran out, and this one stores nothing
};

// One tile; false after an abort.
template <int kForm, int kPair, bool kWide>
__device__ __forceinline__ bool epilogue_tile(const LinearParams &lp, const Problem &p, LCtrl *c, EpiState &st, const Tile &t)
{
    constexpr bool kLaneRow = kForm != kRowsT;
    const int32_t quarter = st.quarter, which = st.which, lane = st.lane, buf = st.buf;
    const uint32_t half = st.half, tiles = st.tiles, buf_ph = st.buf_ph;
    uint8_t *stage = st.stage;
    float *bias_s = st.bias_s;
    const bool splitk = lp.split > 1;
    const int32_t S = splitk ? lp.split : 1;
    const int32_t me = splitk ? static_cast<int32_t>(st.rank) / kPair : 0;
    const int32_t nbuf = lp.recv_bufs > 0 ? lp.recv_bufs : 1;
    auto cta_of = [&](int32_t slice) { return static_cast<uint32_t>(slice * kPair) + half; };   // same half, other slice
    {
        const uint32_t acc = acc_of<kWide>(tiles);
        const uint32_t ph = acc_parity<kWide>(tiles);
        // the columns of the tile that this CTA finishes
        const int32_t part = splitk ? ((t.n + S - 1) / S + lp.part_align - 1) / lp.part_align * lp.part_align : t.n;
        const int32_t c_lo = min(me * part, t.n), c_hi = min(c_lo + part, t.n);
        // This warp's chunks: accumulator columns col .. col + 31 of its lanes, for col = first, first + 64, ...
        const int32_t first = c_lo + 32 * which;
        const int32_t prow = t.p0 + static_cast<int32_t>(half) * kPRows + quarter * 32;   // first MMA row of this warp
        const int64_t row0 = kForm == kRows     ? static_cast<int64_t>(t.start) + prow
                             : kForm == kRowsT ? static_cast<int64_t>(t.start) + t.q0 + first
                                               : static_cast<int64_t>(t.e) * p.p_ext + prow;
        const int32_t col0 = kLaneRow ? t.q0 + first : prow;
        Piece out, zp, rp;
        out.init(p.out, row0, col0, p.ld_out, kForm == kReduce && p.out_f32 ? 4 : 2, !kLaneRow, lane);
        if (p.z)
            zp.init(p.z, row0, col0, p.ld_z, 2, !kLaneRow, lane);
        if (p.res)
            rp.init(p.res, row0, col0, p.ld_res, 2, !kLaneRow, lane);
        // rows and 16-byte segments (of bf16) of a chunk that exist
        const int32_t lim_fix = kLaneRow ? (kForm == kRows ? t.cnt : p.p_ext) - prow : (p.p_ext - prow) / 8;
        auto row_lim_of = [&](int32_t col) { return kLaneRow ? lim_fix : min(c_hi - col, t.cnt - t.q0 - col); };
        auto seg_lim_of = [&](int32_t col) { return kLaneRow ? min(c_hi - col, p.q_ext - t.q0 - col) / 8 : lim_fix; };
        uint4 res[4];
        auto request_res = [&](int32_t col) {
            if (p.res && col < c_hi)
                res_load(res, rp, row_lim_of(col), seg_lim_of(col), lane);
        };
        // ---- bias and residual of the first chunk are requested while the tile's MMAs run, of later ones a chunk
        // ahead.  A lane holds one column's bias: its own for kRowsT, column col + lane of the chunk otherwise.
        float bias = 0.0f;
        auto request_bias = [&](int32_t col) {
            const int32_t n = kLaneRow ? t.q0 + col + lane : prow + lane, ext = kLaneRow ? p.q_ext : p.p_ext;
            if (p.bias && col < c_hi)
                bias = n < ext ? load_bias(p, static_cast<int64_t>(t.e) * ext + n) : 0.0f;
        };
        request_bias(first);
        request_res(first);
        if (!lwait_warp(&c->tfull[acc], ph, c, lp, kPair == 2))
            return false;
        tc_fence_after();
        const uint32_t d = st.tmem_lanes + acc * static_cast<uint32_t>(lp.acc_cols);
        const bool have_k = t.kb1 > t.kb0;
        uint8_t *recv = st.recv_base + static_cast<uint32_t>(buf) * lp.recv_bytes;
        if (splitk) {
            // Wait until the others can receive: with the ring as buffer, until every CTA's MMAs of this
            // item are done; with buffers of their own, until they have read this one's previous content.
            if (lp.recv_bufs == 0) {
                if (lane == 0)
                    for (int32_t r = 0; r < S; ++r)
                        mbar_arrive_relaxed_cluster(map_to_rank(&c->rdy[0], cta_of(r)), 1);   // publishes no data
                if (!lwait_warp(&c->rdy[0], buf_ph, c, lp, true))
                    return false;
            } else if (tiles >= static_cast<uint32_t>(nbuf)) {
                if (!lwait_warp(&c->rdy[buf], buf_ph ^ 1u, c, lp, true))
                    return false;
            }
            // layout: [source][4-column block][128 lanes] float4
            for (int32_t o = 1; o < S; ++o) {
                const int32_t r = (me + o) % S;
                const uint32_t dst = map_to_rank(recv, cta_of(r));
                const int32_t slot = me < r ? me : me - 1;
                const int32_t r_lo = min(r * part, t.n), r_n = min(part, t.n - r_lo);
                for (int32_t j = 8 * which; j < r_n; j += 16) {
                    uint32_t x[8];
                    tmem_ld_32x32b_x8(d + static_cast<uint32_t>(r_lo + j), x);
                    tmem_ld_wait();
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t off = (static_cast<uint32_t>(slot * (part / 4) + j / 4 + b) * 128u +
                                              static_cast<uint32_t>(quarter * 32 + lane)) * 16u;
                        st_cluster_v4_f32(dst + off, have_k ? __uint_as_float(x[4 * b]) : 0.0f,
                                          have_k ? __uint_as_float(x[4 * b + 1]) : 0.0f,
                                          have_k ? __uint_as_float(x[4 * b + 2]) : 0.0f,
                                          have_k ? __uint_as_float(x[4 * b + 3]) : 0.0f);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {   // one fence, then arrivals: together the release of the warp's stores
                fence_acq_rel_cluster();
                for (int32_t o = 1; o < S; ++o)
                    mbar_arrive_relaxed_cluster(map_to_rank(&c->got[buf], cta_of((me + o) % S)), 1);
            }
            if (!lwait_warp(&c->got[buf], buf_ph, c, lp, true))
                return false;
        }
        bool freed = false;
        for (int32_t col = first; col < c_hi; col += 64) {
            const int32_t row_lim = row_lim_of(col) & st.keep, seg_lim = seg_lim_of(col);
            // accumulator columns [col, col + 32) of this lane, partial sums of all slices in slice order
            float v[32];
            {
                uint32_t x[32];
                tmem_ld_32x32b_x32(d + static_cast<uint32_t>(col), x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __uint_as_float(x[j]);
                if (!have_k) {   // an empty reduction
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = 0.0f;
                }
            }
            if (col + 64 >= c_hi) {   // this warp's last read of the accumulator
                freed = true;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_relaxed_cluster(st.tempty_lead0 + 8u * acc, 1);
            }
            if (splitk) {
                const int32_t blocks = min(8, (c_hi - col + 3) / 4);
                float own[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    own[j] = v[j];
                    v[j] = 0.0f;
                }
                for (int32_t s = 0; s < S; ++s) {
                    if (s == me) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] += own[j];
                        continue;
                    }
                    const int32_t slot = s < me ? s : s - 1;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (b < blocks) {
                            const float4 q = *reinterpret_cast<const float4 *>(
                                recv + (static_cast<uint32_t>(slot * (part / 4) + (col - c_lo) / 4 + b) * 128u +
                                        static_cast<uint32_t>(quarter * 32 + lane)) * 16u);
                            v[4 * b] += q.x;
                            v[4 * b + 1] += q.y;
                            v[4 * b + 2] += q.z;
                            v[4 * b + 3] += q.w;
                        }
                    }
                }
            }
            if (kForm == kReduce) {
                if (p.out_f32) {
                    finish_f32(v, stage, out, row_lim, 8 * seg_lim, lane);
                } else {
                    put_bf16<true>(v, stage, lane);
                    stage_store<true>(stage, out, row_lim, seg_lim, lane);
                    __syncwarp();
                }
                out.at += out.next;
                continue;
            }
            if (p.bias) {
                if (kLaneRow) {
                    bias_s[lane] = bias;
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 b = kLaneRow ? *reinterpret_cast<const float4 *>(bias_s + j) : make_float4(bias, bias, bias, bias);
                    v[j] += b.x;
                    v[j + 1] += b.y;
                    v[j + 2] += b.z;
                    v[j + 3] += b.w;
                }
                if (kLaneRow) {
                    __syncwarp();
                    request_bias(col + 64);
                }
            }
            if (row_lim > 0 && seg_lim > 0) {
                switch (p.act) {
                case kActGelu: finish_chunk<kActGelu, kLaneRow>(p, v, stage, out, zp, res, row_lim, seg_lim, lane); break;
                case kActSilu: finish_chunk<kActSilu, kLaneRow>(p, v, stage, out, zp, res, row_lim, seg_lim, lane); break;
                case kActRelu: finish_chunk<kActRelu, kLaneRow>(p, v, stage, out, zp, res, row_lim, seg_lim, lane); break;
                default: finish_chunk<kActNone, kLaneRow>(p, v, stage, out, zp, res, row_lim, seg_lim, lane); break;
                }
            }
            out.at += out.next;
            if (p.z)
                zp.at += zp.next;
            if (p.res)
                rp.at += rp.next;
            request_res(col + 64);
        }
        __syncwarp();
        if (splitk && lp.recv_bufs == 0) {
            fence_proxy_async_shared();   // these reads of the ring before the producers' next copies
            __syncwarp();
        }
        if (lane == 0) {
            if (!freed) {
                tc_fence_before();
                mbar_arrive_relaxed_cluster(st.tempty_lead0 + 8u * acc, 1);
            }
            if (splitk && lp.recv_bufs == 0) {
                mbar_arrive(&c->ringfree);
            } else if (splitk) {
                fence_acq_rel_cluster();   // this warp's reads of the buffer before the others' next stores to it
                for (int32_t o = 1; o < S; ++o)
                    mbar_arrive_relaxed_cluster(map_to_rank(&c->rdy[buf], cta_of((me + o) % S)), 1);
            }
        }
    }
    ++st.tiles;
    if (++st.buf == nbuf) {
        st.buf = 0;
        st.buf_ph ^= 1u;
    }
    return true;
}

// out[e, c]: the partial rows of the blocks that hold rows lo .. hi - 1 (those of group e), in block order.
__device__ __forceinline__ void add_bias_sums(const BiasSums &q, int32_t e, int32_t c, int32_t lo, int32_t hi)
{
    if (c >= q.N)
        return;
    float s = 0.0f;
    if (hi > lo) {
        const int32_t b1 = (hi - 1) / q.block_rows;
#pragma unroll 8
        for (int32_t b = lo / q.block_rows; b <= b1; ++b)
            s += q.part[static_cast<int64_t>(b + e) * q.N + c];
    }
    const int64_t o = static_cast<int64_t>(e) * q.N + c;
    if (q.f32)
        static_cast<float *>(q.out)[o] = s;
    else
        static_cast<__nv_bfloat16 *>(q.out)[o] = __float2bfloat16_rn(s);
}

// False after an abort.
template <int kForm, int kFormB, int kPair, bool kWide>
__device__ __forceinline__ bool l_role_epilogue(const LinearParams &p, LCtrl *c, const GroupTab g, uint8_t *recv_base,
                                                uint8_t *stage_all, float *bias_all, uint32_t tmem_base)
{
    const int32_t ew = static_cast<int32_t>(threadIdx.x / 32) - 4;
    EpiState st;
    st.quarter = ew & 3;
    st.which = ew >> 2;
    st.lane = threadIdx.x & 31;
    st.rank = cluster_ctarank();
    st.half = kPair == 2 ? (st.rank & 1u) : 0u;
    st.stage = stage_all + ew * kStageWarpBytes;
    st.recv_base = recv_base;
    st.bias_s = bias_all + ew * 32;
    st.tmem_lanes = tmem_base + (static_cast<uint32_t>(st.quarter * 32) << 16);
    st.tempty_lead0 = map_to_rank(&c->tempty[0], kPair == 2 ? st.rank & ~1u : st.rank);
    st.tiles = 0;
    st.buf = 0;
    st.buf_ph = 0;
    const int32_t n_items = c->n_items[0], n_items_b = c->n_items[1];
    griddep_wait();
    // (from here on only this launch or another stream's can report a wait that ran out)
    st.keep = ld_relaxed_gpu_u32(p.status) == kStTimeout ? 0 : -1;
    if (p.bias.out && st.keep) {   // (while the first tile's products run: a launch of its own took 3 us)
        const int32_t strips = (p.bias.N + kEpi * 32 - 1) / (kEpi * 32), todo = strips * p.groups;
        for (int32_t i = static_cast<int32_t>(blockIdx.x); i < todo; i += static_cast<int32_t>(gridDim.x)) {
            const int32_t e = i / strips, lo = p.offsets ? g.start[e] : 0;
            add_bias_sums(p.bias, e, (i - e * strips) * kEpi * 32 + ew * 32 + st.lane, lo, p.offsets ? lo + g.cnt[e] : p.rows);
        }
    }
    Walk<kForm, kFormB, kPair> w(p);
    Tile t;
    while (w.next(p, g, n_items, n_items_b, t)) {
        if constexpr (kFormB < 0) {
            if (!epilogue_tile<kForm, kPair, kWide>(p, p.pr[0], c, st, t))
                return false;
        } else if (t.which == 0) {
            if (!epilogue_tile<kForm, kPair, kWide>(p, p.pr[0], c, st, t))
                return false;
        } else {
            if (!epilogue_tile<kFormB, kPair, kWide>(p, p.pr[1], c, st, t))
                return false;
        }
    }
    return true;
}

// --------------------------------------------------------------------------------------- kernel --
template <int kForm, int kFormB, int kPair, bool kWide>
__global__ void __launch_bounds__(kLThreads, 1) linear_kernel(const __grid_constant__ LinearParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((base + 1023u) & ~1023u) - base);
    const SmemMap sm(kForm == kRowsT || kForm == kReduce, static_cast<uint32_t>(p.num_pipe) * p.slot_bytes,
                     static_cast<uint32_t>(p.recv_bufs) * p.recv_bytes);
    LCtrl *c = reinterpret_cast<LCtrl *>(ring + sm.ctrl);
    GroupTab g;
    g.start = reinterpret_cast<int32_t *>(ring + sm.tab);
    g.cnt = g.start + p.groups;
    g.base = g.cnt + p.groups;
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    griddep_launch_dependents();   // every wait of a dependent kernel is for this grid's end

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&p.pr[0].map[0]);
            prefetch_tensormap(&p.pr[0].map[1]);
            if (kFormB >= 0) {
                prefetch_tensormap(&p.pr[1].map[0]);
                prefetch_tensormap(&p.pr[1].map[1]);
            }
        }
        for (int32_t i = lane; i < p.num_pipe; i += 32) {
            mbar_init(&c->full[i], kForm == kReduce || kFormB == kReduce ? kPair : 1);
            mbar_init(&c->empty[i], 1);
            mbar_init(&c->go[i], 1);
            mbar_init(&c->tail[i], 1);
            c->masked[i] = 0xffffffffu;
        }
        if (lane < 2) {
            mbar_init(&c->tfull[lane], 1);
            mbar_init(&c->tempty[lane], kEpi * kPair);
        }
        if (lane == 0) {
            const int32_t S = p.split > 1 ? p.split : 1;
            mbar_init(&c->drain, 1);
            mbar_init(&c->left, 3);
            for (int b = 0; b < 2; ++b) {   // epilogue warps of the other CTAs (and, sharing the ring, of this one)
                mbar_init(&c->rdy[b], p.recv_bufs == 0 ? kEpi * S : S > 1 ? kEpi * (S - 1) : 1);
                mbar_init(&c->got[b], S > 1 ? kEpi * (S - 1) : 1);
            }
            mbar_init(&c->ringfree, kEpi);
            c->abort_flag = 0;
            // a wait that ran out is sticky: do nothing.  (Bad offsets are not: a CTA of this very grid may have just
            // reported them.)  The launch before may still be running and report one: see EpiState::keep.
            c->skip = ld_relaxed_gpu_u32(p.status) == kStTimeout;
        }
        fence_barrier_init();
    } else if (warp == 1) {
        tmem_alloc_g<kPair>(&c->tmem_base, p.tmem_cols);
        tmem_relinquish_g<kPair>();
    } else if (warp == 2 && !p.offsets) {
        if (lane == 0) {
            c->n_items[0] = p.pr[0].dense_items;
            c->n_items[1] = p.pr[1].dense_items;
        }
    } else if (warp == 2) {
        griddep_wait();
        // Group tables.  Offsets come from device memory: anything out of order or out of range is
        // clamped, so no access can leave the matrices, and reported through the status word.
        int32_t carry = 0;
        bool bad = false;
        for (int32_t e0 = 0; e0 < p.groups; e0 += 32) {
            const int32_t e = e0 + lane;
            int32_t items = 0;
            if (e < p.groups) {
                const int32_t lo0 = p.offsets[e], hi0 = p.offsets[e + 1];
                const int32_t lo = min(max(lo0, 0), p.rows), hi = min(max(hi0, lo), p.rows);
                bad |= lo != lo0 || hi != hi0;
                g.start[e] = lo;
                g.cnt[e] = hi - lo;
                items = items_of<kForm, kPair>(p.pr[0], hi - lo);
            }
            int32_t sum = items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += v;
            }
            if (e < p.groups)
                g.base[e] = carry + sum - items;
            carry += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) {
            g.base[p.groups] = carry;
            c->n_items[0] = carry;
            c->n_items[1] = kFormB >= 0 ? p.groups * items_of<kFormB < 0 ? kForm : kFormB, kPair>(p.pr[1], 0) : 0;
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0)
            atomicCAS(p.status, 0u, kStBadOffsets);
    }
    // a dense product's first tile needs no tables: its coordinates are worked out before the barrier
    Walk<kForm, kFormB, kPair> w(p);
    Tile t;
    bool have = false;
    if (!p.offsets && (warp == 0 || warp == 3))
        have = w.next(p, g, p.pr[0].dense_items, p.pr[1].dense_items, t);
    tc_fence_before();
    cluster_sync_all();   // barriers initialised before any remote arrival
    tc_fence_after();
    const uint32_t tmem_base = c->tmem_base;
    if (!ld_cluster_s32(map_to_rank(&c->skip, 0))) {   // the CTAs of a cluster agree: they wait for one another
        if (warp == 0) {
            if (p.offsets)
                have = w.next(p, g, c->n_items[0], c->n_items[1], t);
            if (elect_one())
                l_role_tma<kForm, kFormB, kPair, kWide>(p, c, g, ring, 0, w, t, have);
        } else if (warp == 1) {
            if (elect_one())
                l_role_mma<kForm, kFormB, kPair, kWide>(p, c, g, ring, tmem_base);
        } else if (warp == 2) {
            if ((kForm == kReduce || kFormB == kReduce) && p.offsets)
                l_role_mask<kForm, kFormB, kPair>(p, c, g, ring);
        } else if (warp == 3) {
            if (p.offsets)
                have = w.next(p, g, c->n_items[0], c->n_items[1], t);
            if (elect_one())
                l_role_tma<kForm, kFormB, kPair, kWide>(p, c, g, ring, 1, w, t, have);
        } else {
            const bool ok = l_role_epilogue<kForm, kFormB, kPair, kWide>(p, c, g, ring + (p.recv_bufs ? sm.recv : 0u), ring + sm.stage,
                                                                         reinterpret_cast<float *>(ring + sm.bias), tmem_base);
            if (!ok && warp == 4 && lane == 0)
                land<kPair>(c, p);
        }
    }
    __syncwarp();
    griddep_wait();       // (also after a skipped run: this grid must not end before the one it may have overtaken)
    tc_fence_before();
    cluster_sync_all();   // MMAs, epilogues and exchanges of every CTA of the cluster are over
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_g<kPair>(tmem_base, p.tmem_cols);
    }
    if (kPair == 2)
        cluster_sync_all();   // a pair's CTAs free their TMEM together
}

}  // namespace mlpl
