// paged_chunk.cu -- attention of chunks of new tokens over a paged key/value
// cache on the tcgen05 tensor cores (sequences with more query rows than the
// decode kernel takes).
//
//   x_ij = scale_log2 * q_i . k_j,  o_i = sum_j 2^(x_ij - m_i) v_j / sum_j 2^(x_ij - m_i)
//
// over the keys j < visible(i), with the running shift m_i raised only when a
// row's maximum outgrew it by 2^8.  The weights are rounded to the data type as the
// tensor cores take them (off by up to 2^-8 of each in bf16, 2^-11 in fp16, where the
// shift stands 2^7 below the maximum: weight_room in paged_sched.h); row sums add the
// unrounded ones, and O, m and l stay in fp32.
//
// Bound: the tensor cores (4 d flops per row and visible key), then exp2 on the
// MUFU.  An item is two 128-row tiles against the keys they see; a row tile packs
// 128 / g tokens of all g query heads of one key/value head, so each key tile that
// is loaded serves every head that shares it.  The pipeline of one persistent block:
//
//   warps 0-3, 4-7  softmax of row tile 0, 1 (thread = row)
//   warps 8-11      epilogue: O / l, or a partial result of an item that other
//                   blocks compute parts of
//   warp 12         TMA producer of K and V: 128-key tiles gathered page by page
//   warp 13         MMA issuer, owns TMEM
//   warp 14         TMA producer of Q
//   warp 15         edge tiles of V: rows behind the last key become zeros, and
//                   non-finite values of keys that some row must not see are
//                   taken out of the product (0 * NaN would reach every row) and
//                   added by the epilogue to the rows that see them
//
// A one-block kernel first lists the items and where each block's run of them
// starts (the lengths live on the device).  Runs are equal in cost.  An item that
// crosses a cut is computed in parts; two parts are joined by the block that
// finishes last (an arrival count per item; nobody waits), more by
// paged_chunk_join_kernel.  Either way the parts are added in the order of the
// keys, so results do not depend on who was last.
//
// An item with a single row tile (few tokens, or the last of a sequence) would
// leave one softmax group idle and the other's chain score -> weight -> product
// bare.  There the groups take turns at the key tiles: the even ones go through S0,
// O0, the odd ones through S1, O1, and the epilogue adds the two.
//
// A key tile's weights are computed with the shift as it is, beside the tile's
// maximum, and the maximum is looked at afterwards: it is off the chain score ->
// weight -> product unless it outgrew the shift, and then the tile's weights are
// computed again.  (Handing the weights over in two halves, so that the first
// half's product runs beside the second half's weights, was slower, 730 against
// 707 us: each further wait and commit of the MMA warp is a gap in the tensor pipe,
// which takes only a few products in advance.)
//
// 2,048 tokens behind 30,011 (32 query and 8 key/value heads): at d = 128 686 to 690 us
// alone, 726 to 755 among other calls (1,380 to 1,520 TFLOP/s; the tensor pipe active 66%
// of the time), at d = 64 511 us (1,020).  At d = 128 a key tile takes 1.45 us, of which
// the chain of one row tile is 1.4 (scores 0.28, weights 0.6, product 0.28, and the
// barriers between them).  256 items of 243 key tiles on average are 409 such steps on
// each of 152 SMs, 593 us; the rest (first tiles, joins, page lookups, 84 bytes of
// registers that the softmax warps spill at d = 128) has not been taken apart.
//
// Every wait is bounded.
#include <cuda_bf16.h>

#include "clis_internal.h"
#include "paged_internal.h"
#include "sm103_ptx.cuh"

namespace clis {

__device__ unsigned int g_chunk_error_word = 0;

namespace {

constexpr int BM = kChunkRows, BN = kChunkKeys;
constexpr int kThreads = 512;
constexpr int kNStageMax = 8;
constexpr float kTau = 8.0f;
constexpr int kSchedThreads = 256;
// Items of three parts or more: every block but the last adds at most one part to
// the items' number, so there are at most (grid - 1) / 2 of them.
int max_joins(int grid) { return (grid - 1) / 2 + 1; }

// Error-word bits of waits that gave up (the forward kernel's meanings).
constexpr unsigned kErrProducer = 1u << 0, kErrMma = 1u << 1, kErrSoftmax = 1u << 2, kErrEpilogue = 1u << 3,
                   kErrDrain = 1u << 4, kErrEdge = 1u << 5;

template <int D>
struct Cfg {
    static constexpr int NSTAGE = (D == 128) ? 4 : 8;
    static constexpr int NBOX = D / 64;
    static constexpr int BOX_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = NBOX * BOX_BYTES;
    static constexpr int SMEM_BYTES = 2 * TILE_BYTES + NSTAGE * TILE_BYTES + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t TM_S0 = 0, TM_S1 = 128, TM_O0 = 256, TM_O1 = 256 + D;
};

struct ChunkParams {
    PagedArgs a;
    int g, tpt;           // query heads per key/value head; tokens per row tile
    int rows_small;       // sequences of up to so many rows are the decode kernel's
    int grid, least;      // blocks; cost of a block's run, at least
    int box_rows;         // rows of a K/V TMA box: min(page size, 128)
    int list;             // places of the list of items
    ChunkItem *items;
    unsigned long long *head;  // {items, total cost, blocks that take part}
    int *run_first;       // [grid] first item of each block's run
    int *arrived;         // [grid] parts done of the item that the block starts and does not finish
    int2 *join;           // [max_joins] {parts, item} of items of three parts or more
    int *joins;           // their number
    float *part_o;        // [2 * grid][D / 4][256][4]: slot 2 c + 1 if block c starts the item, 2 c if it goes on with it
    float2 *part_ml;      // [2 * grid][256]
};

struct __align__(8) Ctl {
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[kNStageMax], kv_empty[kNStageMax];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t o_free[2], epi_full[2];
    uint64_t edge_go;  // an edge tile of V has been loaded
    uint64_t edge_ok;  // and is ready for the product
    uint64_t drain;
    float epi_l[2][BM], epi_shift[2][BM];
    int dirty[8];  // per item (mod 8): non-finite values were taken out
    uint32_t tmem_base;
    int last;  // epilogue: the item's other parts are done
    int abort_flag;
};

__device__ __forceinline__ SeqLen seq_len(const PagedArgs &a, int s)
{
    return clip_seq(__ldg(a.cu_q + s), __ldg(a.cu_q + s + 1), __ldg(a.kv_len + s), a.T, a.width << a.page_shift);
}

// ------------------------------------------------------------------ schedule

__device__ __forceinline__ ChunkItem load_item(const ChunkParams &p, int i)
{
    union { int4 v[3]; ChunkItem c; } u;
    const int4 *src = reinterpret_cast<const int4 *>(p.items + i);
    u.v[0] = src[0];
    u.v[1] = src[1];
    u.v[2] = src[2];
    return u.c;
}

// Exclusive prefix sum over the block's threads; the total in *total.
template <typename T>
__device__ __forceinline__ T block_scan(T mine, T *s_warp, T *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    T before = 0, all = 0;
    for (int w = 0; w < kSchedThreads / 32; w++) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
    }
    __syncthreads();
    *total = all;
    return before + incl - mine;
}

__global__ void __launch_bounds__(kSchedThreads) paged_chunk_schedule_kernel(const ChunkParams p)
{
    extern __shared__ int s_first[];  // [S + 1] first item of each sequence
    __shared__ unsigned long long s_warp[kSchedThreads / 32];
    __shared__ int s_joins;
    const PagedArgs &a = p.a;
    const int tid = threadIdx.x;
    const bool causal = a.causal != 0;
    unsigned int bad = 0;
    pdl_launch();  // the decode kernel does not read what is written here
    for (int c = tid; c < p.grid; c += kSchedThreads) p.arrived[c] = 0;
    if (tid == 0) s_joins = 0;  // (read after the scans' barriers)

    const int per = (a.S + kSchedThreads - 1) / kSchedThreads;
    const int s0 = min(a.S, tid * per), s1 = min(a.S, s0 + per);
    auto items_of = [&](const SeqLen &q) -> int { return chunk_items(q, p.g, p.rows_small, a.Hkv); };
    unsigned long long mine = 0, all;
    for (int s = s0; s < s1; s++) {
        const SeqLen q = seq_len(a, s);
        if (q.bad) bad |= CLIS_PAGED_LENGTH_BIT;
        mine += items_of(q);
    }
    unsigned long long run = block_scan(mine, s_warp, &all);
    for (int s = s0; s < s1; s++) {
        s_first[s] = chunk_place(run, p.list);
        run += items_of(seq_len(a, s));
    }
    const int W = chunk_place(all, p.list);
    if (all > static_cast<unsigned long long>(W)) bad |= CLIS_PAGED_LENGTH_BIT;
    if (tid == 0) s_first[a.S] = W;
    __syncthreads();

    // Costs: a run of consecutive items per thread, then over the threads.
    const int iper = (W + kSchedThreads - 1) / kSchedThreads;
    const int i0 = min(W, tid * iper), i1 = min(W, i0 + iper);
    int seq = 0;
    if (i0 < i1) {  // the sequence of item i0
        int hi = a.S;
        while (hi - seq > 1) {
            const int mid = (seq + hi) >> 1;
            if (s_first[mid] <= i0) seq = mid;
            else hi = mid;
        }
    }
    auto item_at = [&](int i, int &s) -> ChunkItem {
        while (s_first[s + 1] <= i) s++;
        return chunk_item(seq_len(a, s), s, p.g, i - s_first[s], causal);
    };
    mine = 0;
    for (int i = i0, s = seq; i < i1; i++) {
        const ChunkItem t = item_at(i, s);
        mine += chunk_cost(t.n_kv, t.nt);
    }
    unsigned long long U;
    unsigned long long first = block_scan(mine, s_warp, &U);
    const int nb = chunk_blocks(U, p.grid, p.least);
    const ChunkCuts cuts = chunk_cuts(U, nb);
    for (int i = i0, s = seq; i < i1; i++) {
        ChunkItem t = item_at(i, s);
        t.first = first;
        p.items[i] = t;
        first += chunk_cost(t.n_kv, t.nt);
        // Blocks whose runs start in this item.
        int c = chunk_block_of(cuts, t.first);
        if (cuts.cut(c) < t.first) c++;
        for (; c < nb && cuts.cut(c) < first; c++) p.run_first[c] = i;
        const ChunkOwners o = chunk_owners(t, cuts);
        // (the order of the list does not matter: it only says which block joins what)
        if (o.count > 2) p.join[atomicAdd(&s_joins, 1)] = make_int2(o.count, i);
    }
    __syncthreads();
    if (tid == 0) {
        p.head[0] = W;
        p.head[1] = U;
        p.head[2] = nb;
        *p.joins = s_joins;
    }
    if (bad) atomicOr(&g_chunk_error_word, bad);
}

// A block's run of items.
struct Run {
    int first, items;      // its first item; items in all
    unsigned long long lo, hi;
    ChunkCuts cuts;
};

// One item of the run: the key tiles [start, start + n) of it are this block's.
struct Work {
    ChunkItem t;
    int start, n;
    bool whole;
};

__device__ __forceinline__ bool load_work(const ChunkParams &p, const Run &r, int i, Work &k)
{
    k.t = load_item(p, i);
    const ChunkRange g = chunk_range(k.t, r.lo, r.hi);
    k.start = g.t0;
    k.n = g.t1 - g.t0;
    k.whole = g.t0 == 0 && g.t1 == k.t.n_kv;
    return k.t.first < r.hi;  // false: behind the run
}

// Loop over the block's items that have key tiles in its run.
#define CLIS_FOR_WORK(K)                                                              \
    Work K;                                                                           \
    for (int i_ = R.first; i_ < R.items && load_work(p, R, i_, K); ++i_)              \
        if (K.n > 0)

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > 200000000ull) {
            atomicOr(&g_chunk_error_word, kErrDrain);
            return;
        }
    }
}

// ----------------------------------------------------------------- producers

template <int D>
__device__ void q_producer_role(const ChunkParams &p, Ctl &c, const CUtensorMap *tm_q, uint32_t sQ0, const Run &R)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const bool leader = elect_one();
    const uint64_t pol = policy_evict_first();
    int wt[2] = {0, 0};
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            if (t >= T.nt) break;
            if (!mbar_wait_warp(smem_u32(&c.q_empty[t]), (wt[t] & 1) ^ 1, ab, err, kErrProducer)) goto abort;
            if (leader) {
                const uint32_t bar = smem_u32(&c.q_full[t]);
                mbar_arrive_expect_tx(bar, C::NBOX * p.g * p.tpt * 128);
#pragma unroll
                for (int bx = 0; bx < C::NBOX; bx++)
                    tma_load_3d_hint(sQ0 + t * C::TILE_BYTES + bx * C::BOX_BYTES, tm_q, bar, bx * 64, T.h * p.g,
                                     T.q0 + T.tok0 + t * p.tpt, pol);
            }
            __syncwarp();
            ++wt[t];
        }
    }
    return;
abort:
    for (int t = 0; t < 2; t++)
        if (wt[t] > 0) drain_wait(smem_u32(&c.q_full[t]), (wt[t] - 1) & 1);
}

template <int D>
__device__ void producer_role(const ChunkParams &p, Ctl &c, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                              uint32_t sKV, const Run &R)
{
    using C = Cfg<D>;
    const PagedArgs &a = p.a;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int lane = threadIdx.x & 31;
    const int npg = BN / p.box_rows;  // pages per key tile, at most 16: lane l < npg loads the l-th
    const uint32_t box_bytes = p.box_rows * 128;
    const uint64_t pol = policy_evict_last();
    uint32_t it = 0, gq = 0;
    unsigned int bad = 0;
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
        // Whether the lane has rows of key tile kt to load (none behind the last key), and
        // their page.  What the table holds is looked at when it is used, a tile later (any
        // number can stand there, so none can say that there is nothing to load).
        auto has_rows = [&](int kt) { return lane < npg && kt * BN + lane * p.box_rows < T.kv; };
        auto page_of = [&](int kt) -> int {
            return has_rows(kt) ? __ldg(a.block_table + T.s * a.bt_s + ((kt * BN + lane * p.box_rows) >> a.page_shift)) : -1;
        };
        int pg_k = page_of(K.start), pg_v = -1;
        // Groups of loads as the MMA warp needs them: {K_0}, {V_0, K_1}, ..., {V_{n-1}}.
        for (int gi = 0; gi <= K.n; gi++) {
            const bool has_v = gi > 0, has_k = gi < K.n;
            const int nl = (has_v ? 1 : 0) + (has_k ? 1 : 0);
            const bool rows_v = has_v && has_rows(K.start + gi - 1), rows_k = has_k && has_rows(K.start + gi);
            const int pg_next = gi + 1 < K.n ? page_of(K.start + gi + 1) : -1;
            for (int l = 0; l < nl; l++) {
                const uint32_t li = it + l;
                if (!mbar_wait_warp(smem_u32(&c.kv_empty[li % C::NSTAGE]), ((li / C::NSTAGE) & 1) ^ 1, ab, err,
                                    kErrProducer))
                    goto abort;
            }
            const uint32_t bar = smem_u32(&c.kv_full[gq % C::NSTAGE]);
            const int live = __popc(__ballot_sync(~0u, rows_v)) + __popc(__ballot_sync(~0u, rows_k));
            if (lane == 0) mbar_arrive_expect_tx(bar, live * C::NBOX * box_bytes);
            __syncwarp();
#pragma unroll
            for (int l = 0; l < 2; l++) {
                const bool is_v = l == 0;
                if (is_v ? !rows_v : !rows_k) continue;
                int pg = is_v ? pg_v : pg_k;
                if (pg < 0 || pg >= a.num_pages) {
                    bad |= CLIS_PAGED_INDEX_BIT;
                    pg = static_cast<int>(a.num_pages);  // out of the map: its rows read as zeros
                }
                const uint32_t slot = (it + (is_v ? 0 : nl - 1)) % C::NSTAGE;
                const int key = (K.start + (is_v ? gi - 1 : gi)) * BN + lane * p.box_rows;
                const uint32_t dst = sKV + slot * C::TILE_BYTES + lane * box_bytes;
                const CUtensorMap *tm = is_v ? tm_v : tm_k;
#pragma unroll
                for (int bx = 0; bx < C::NBOX; bx++)
                    tma_load_4d_hint(dst + bx * C::BOX_BYTES, tm, bar, bx * 64, key & ((1 << a.page_shift) - 1), T.h, pg,
                                     pol);
            }
            __syncwarp();
            it += nl;
            ++gq;
            pg_v = pg_k;
            pg_k = pg_next;
        }
    }
    if (bad) atomicOr(err, bad);
    return;
abort:
    for (uint32_t k = (gq > C::NSTAGE ? gq - C::NSTAGE : 0); k < gq; k++)
        drain_wait(smem_u32(&c.kv_full[k % C::NSTAGE]), (k / C::NSTAGE) & 1);
}

// ---------------------------------------------------------------- edge tiles

// 16 bytes of shared memory.
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int DT>
__device__ __forceinline__ bool scrub(uint32_t &u)
{
    constexpr uint32_t E = DT ? 0x7C00u : 0x7F80u;
    uint32_t keep = 0xFFFFFFFFu;
    if ((u & E) == E) keep &= 0xFFFF0000u;
    if (((u >> 16) & E) == E) keep &= 0x0000FFFFu;
    u &= keep;
    return keep != 0xFFFFFFFFu;
}

template <int D, int DT>
__device__ void edge_role(const ChunkParams &p, Ctl &c, uint32_t sKV, const Run &R)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int lane = threadIdx.x & 31;
    uint32_t it = 0, gq = 0, nedge = 0;
    int w = 0;
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
        // Items without an edge tile are followed too: a wait then spans one item, however
        // many of them come first.  (Q of the next item is not loaded before this arrival, so
        // this phase is the barrier's last.)
        if (!mbar_wait_warp(smem_u32(&c.q_full[0]), w & 1, ab, err, kErrEdge)) return;
        if (lane == 0) mbar_arrive(smem_u32(&c.q_empty[0]));
        const int first = chunk_first_masked(T, p.a.causal != 0);
        // Keys that all rows, and that some row of the item sees.
        const int lim_all = visible_keys(T.n, T.kv, T.tok0, p.a.causal);
        const int lim_any = visible_keys(T.n, T.kv, min(T.n, T.tok0 + 2 * p.tpt) - 1, p.a.causal);
        bool dirty = false;
        for (int j = 0; j < K.n; j++) {
            const int kt = K.start + j;
            if (kt < first) continue;
            // V_j is in load group j + 1 and in ring slot 2 j + 1 of the item's
            // (K_0, V_0, K_1, V_1, ...).  The MMA warp, which waits for every group,
            // says when it has arrived; this warp skips groups, and a barrier whose
            // phases are skipped cannot be told apart by parity.  Once it is said, the
            // group's phase is the barrier's last (the slot is not loaded again
            // before the product), so the second wait returns at once.
            const uint32_t grp = gq + j + 1, vs = it + 2 * j + 1;
            if (!mbar_wait_warp(smem_u32(&c.edge_go), nedge & 1, ab, err, kErrEdge)) return;
            ++nedge;
            if (!mbar_wait_warp(smem_u32(&c.kv_full[grp % C::NSTAGE]), (grp / C::NSTAGE) & 1, ab, err, kErrEdge)) return;
            const uint32_t base = sKV + (vs % C::NSTAGE) * C::TILE_BYTES;
            // Rows [0, lo) are keys that every row of the item sees: left alone.  Rows [lo, hi)
            // are seen by some: scrubbed.  Rows from hi on are seen by none, or hold no key:
            // zeros.  (One warp: only what has to be touched is.  Going over all of the tile
            // took 4 us, in every item.)
            const int lo = min(max(lim_all - kt * BN, 0), BN), hi = min(max(lim_any - kt * BN, lo), BN);
            // (the swizzle permutes 16-byte pieces within a 128-byte row: a row is a row)
            for (int bx = 0; bx < C::NBOX; bx++) {
                const uint32_t box = base + bx * C::BOX_BYTES;
                for (int i0 = lo * 8; i0 < hi * 8; i0 += 4 * 32) {
                    uint4 u[4];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (i0 + e * 32 + lane < hi * 8) u[e] = lds128(box + (i0 + e * 32 + lane) * 16);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        if (i0 + e * 32 + lane >= hi * 8) continue;
                        const bool d0 = scrub<DT>(u[e].x), d1 = scrub<DT>(u[e].y), d2 = scrub<DT>(u[e].z), d3 = scrub<DT>(u[e].w);
                        if (d0 | d1 | d2 | d3) {
                            sts128(box + (i0 + e * 32 + lane) * 16, u[e]);
                            dirty = true;
                        }
                    }
                }
#pragma unroll 4
                for (int i = hi * 8 + lane; i < BN * 8; i += 32) sts128(box + i * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            const bool any = __any_sync(~0u, dirty);
            if (lane == 0) {
                // (set before the arrival that the product, and through it the epilogue, waits for)
                *reinterpret_cast<volatile int *>(&c.dirty[w & 7]) = any ? 1 : 0;
                __threadfence_block();
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.edge_ok));
        }
        it += 2 * K.n;
        gq += K.n + 1;
        ++w;
    }
}

// ----------------------------------------------------------------------- MMA

template <int D, int DT>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t qd, uint64_t kd)
{
    using C = Cfg<D>;
    constexpr uint32_t IDESC_S = idesc_f16kind_f32(BM, BN, false, DT ? 0u : 1u);
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++) {
        const uint32_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
        umma_ss(d_tmem, qd + off, kd + off, IDESC_S, kk > 0 ? 1u : 0u);
    }
}

template <int D, int DT>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t accumulate)
{
    constexpr uint32_t IDESC_O = idesc_f16kind_f32(BM, D, true, DT ? 0u : 1u);
#pragma unroll
    for (int kk = 0; kk < BN / 16; kk++)
        umma_ts(o_tmem, p_tmem + kk * 8, vd + ((kk * 2048) >> 4), IDESC_O, (accumulate | kk) ? 1u : 0u);
}

// O_t (+)= P_t V_j, in the MMA role's loop: the group is a compile-time constant, so
// that addresses and descriptors stay in uniform registers.
#define CLIS_PRODUCT(t, fresh, frees)                                                                               \
    do {                                                                                                            \
        if (!mbar_wait_warp(smem_u32(&c.p_full[t]), (steps >> (t)) & 1, ab, err, kErrMma)) goto abort;               \
        if (fresh)                                                                                                  \
            if (!mbar_wait_warp(smem_u32(&c.o_free[t]), (items & 1) ^ 1, ab, err, kErrMma)) goto abort;              \
        tc_fence_after();                                                                                           \
        if (leader) {                                                                                               \
            issue_pv<D, DT>(tmem + ((t) ? C::TM_O1 : C::TM_O0), tmem + ((t) ? C::TM_S1 : C::TM_S0), vd,              \
                            (fresh) ? 0u : 1u);                                                                     \
            umma_commit(smem_u32(&c.pv_done[t]));                                                                   \
            if (frees) umma_commit(smem_u32(&c.kv_empty[vs]));                                                      \
        }                                                                                                           \
        __syncwarp();                                                                                               \
        steps ^= 1u << (t);                                                                                         \
    } while (0)

template <int D, int DT>
__device__ void mma_role(const ChunkParams &p, Ctl &c, uint32_t tmem, uint32_t sQ0, uint32_t sKV, const Run &R)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const bool leader = elect_one();
    uint32_t it = 0, gq = 0, nedge = 0;
    uint32_t items = 0;             // parities: of the items,
    uint32_t steps = 0, q_par = 0;  // of each group's steps and Q tiles (bit t)
    const uint64_t qd0 = sdesc_sw128(sQ0, 16, 1024);
    const uint64_t qd1 = sdesc_sw128(sQ0 + C::TILE_BYTES, 16, 1024);
    const uint64_t kvd_k = sdesc_sw128(sKV, 16, 1024);
    const uint64_t kvd_v = sdesc_sw128(sKV, C::BOX_BYTES, 1024);
    auto stage_off = [](uint32_t s) -> uint64_t { return (s * C::TILE_BYTES) >> 4; };
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
        const int nt = T.nt;
        const int first = chunk_first_masked(T, p.a.causal != 0);
        for (int t = 0; t < nt; t++) {
            if (!mbar_wait_warp(smem_u32(&c.q_full[t]), (q_par >> t) & 1, ab, err, kErrMma)) goto abort;
            q_par ^= 1u << t;
        }
        {
            const uint32_t ks = it % C::NSTAGE;
            if (!mbar_wait_warp(smem_u32(&c.kv_full[gq % C::NSTAGE]), (gq / C::NSTAGE) & 1, ab, err, kErrMma))
                goto abort;
            ++gq;
            tc_fence_after();
            const uint64_t kd = kvd_k + stage_off(ks);
            if (leader) {
                issue_qk<D, DT>(tmem + C::TM_S0, qd0, kd);
                umma_commit(smem_u32(&c.s_full[0]));
                if (nt == 2) {
                    issue_qk<D, DT>(tmem + C::TM_S1, qd1, kd);
                    umma_commit(smem_u32(&c.s_full[1]));
                }
                umma_commit(smem_u32(&c.kv_empty[ks]));
                if (K.n == 1)
                    for (int t = 0; t < nt; t++) umma_commit(smem_u32(&c.q_empty[t]));
            }
            __syncwarp();
            ++it;
        }
        for (int j = 0; j < K.n; j++) {
            const bool has_next = j + 1 < K.n;
            const uint32_t vs = it % C::NSTAGE;
            if (!mbar_wait_warp(smem_u32(&c.kv_full[gq % C::NSTAGE]), (gq / C::NSTAGE) & 1, ab, err, kErrMma))
                goto abort;
            ++gq;
            const bool edge = K.start + j >= first;
            if (edge && leader) mbar_arrive(smem_u32(&c.edge_go));
            const uint64_t vd = kvd_v + stage_off(vs);
            const uint32_t kns = (it + 1) % C::NSTAGE;
            const uint64_t kd = kvd_k + stage_off(kns);
            const bool last_k = j + 1 == K.n - 1;  // K_{j+1} is the item's last key tile
            if (edge) {
                if (!mbar_wait_warp(smem_u32(&c.edge_ok), nedge & 1, ab, err, kErrMma)) goto abort;
                ++nedge;
            }
            if (nt == 2) {
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    CLIS_PRODUCT(t, j == 0, t == 1);
                    if (has_next) {
                        if (leader) {
                            issue_qk<D, DT>(tmem + (t ? C::TM_S1 : C::TM_S0), t ? qd1 : qd0, kd);
                            umma_commit(smem_u32(&c.s_full[t]));
                            if (t == 1) umma_commit(smem_u32(&c.kv_empty[kns]));
                            if (last_k) umma_commit(smem_u32(&c.q_empty[t]));
                        }
                        __syncwarp();
                    }
                }
            } else {
                // One row tile: the other group's next scores first (its last product was
                // issued before), then this group's product.
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    if ((j & 1) != t) continue;
                    if (has_next) {
                        if (leader) {
                            issue_qk<D, DT>(tmem + (t ? C::TM_S0 : C::TM_S1), qd0, kd);
                            umma_commit(smem_u32(&c.s_full[t ^ 1]));
                            umma_commit(smem_u32(&c.kv_empty[kns]));
                            if (last_k) umma_commit(smem_u32(&c.q_empty[0]));
                        }
                        __syncwarp();
                    }
                    CLIS_PRODUCT(t, j < 2, true);
                }
            }
            it += has_next ? 2 : 1;
        }
        ++items;
    }
    return;
abort:
    if (leader) umma_commit(smem_u32(&c.drain));
    __syncwarp();
    drain_wait(smem_u32(&c.drain), 0);
}

// ------------------------------------------------------------------- softmax

// Weights of a row's 128 scores for a shift, p = 2^(scale_log2 s - shift), packed in
// pairs over the first 64 columns of the scores, all of which have been read;
// returns their sum (before rounding).
template <int DT>
__device__ __forceinline__ float weights128(const uint32_t *s, float sl2, float nshift, uint32_t tP)
{
    const float2 sc2 = make_float2(sl2, sl2), sh2 = make_float2(nshift, nshift);
    float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
    for (int c32 = 0; c32 < BN / 32; c32++) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const float2 x = ffma2(
                make_float2(__uint_as_float(s[c32 * 32 + 2 * e]), __uint_as_float(s[c32 * 32 + 2 * e + 1])), sc2, sh2);
            const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            if (e & 1) lb = fadd2(lb, pp);
            else la = fadd2(la, pp);
            pk[e] = pack2<DT>(pp.x, pp.y);
        }
        tmem_st16(tP + c32 * 16, pk);
    }
    const float2 l = fadd2(la, lb);
    return l.x + l.y;
}

template <int D, int DT>
__device__ void softmax_role(const ChunkParams &p, Ctl &c, uint32_t tmem, int warp, int lane, const Run &R)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int t = warp >> 2;
    const int quarter = warp & 3;
    const int rl = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + (t ? C::TM_S1 : C::TM_S0) + lane_off;
    const uint32_t tO = tmem + (t ? C::TM_O1 : C::TM_O0) + lane_off;
    const float sl2 = p.a.scale_log2;
    const int row_tok = rl / p.g;  // token within the row tile
    uint32_t g = 0;
    int w = 0;
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
        const bool single = T.nt == 1;  // the groups share the row tile, key tiles in turn
        const int tok = T.tok0 + (single ? 0 : t * p.tpt) + row_tok;
        const bool row_ok = row_tok < p.tpt && tok < T.n;
        const int lim = row_ok ? visible_keys(T.n, T.kv, tok, p.a.causal) : 0;  // keys [0, lim) are visible
        const int step = single ? 2 : 1;
        float m_run = -INFINITY, l_run = 0.f;
        bool begun = false;  // O holds a product of this item
#pragma unroll 1
        for (int j = single ? t : 0; j < K.n; j += step) {
            if (!mbar_wait(smem_u32(&c.s_full[t]), g & 1, ab, err, kErrSoftmax)) return;
            tc_fence_after();
            uint32_t s[BN];
            tmem_ld32(tS + 0, s + 0);
            tmem_ld32(tS + 32, s + 32);
            tmem_ld32(tS + 64, s + 64);
            tmem_ld32(tS + 96, s + 96);
            tmem_wait_ld();
            const int key0 = (K.start + j) * BN;
            if (key0 + BN > lim) {
#pragma unroll
                for (int cc = 0; cc < BN; cc++)
                    if (key0 + cc >= lim) s[cc] = 0xFF800000u;  // -inf
            }
            float l = 0.f;
            if (begun) l = weights128<DT>(s, sl2, (m_run == -INFINITY) ? 0.f : -m_run, tS);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int cc = 0; cc < BN; cc += 8) {
#pragma unroll
                for (int q4 = 0; q4 < 4; q4++)
                    mx[q4] = fmax3(mx[q4], __uint_as_float(s[cc + 2 * q4]), __uint_as_float(s[cc + 2 * q4 + 1]));
            }
            const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
            const bool grow = m_tile > m_run + (kTau + weight_room(DT));  // always true where a row's first visible key is
            if (__any_sync(0xFFFFFFFFu, grow) || !begun) {
                // Raise the shift, compute the tile's weights (again), and shrink O once the
                // last product is in it.
                const float m_new = m_tile - weight_room(DT);
                const float alpha = grow ? ex2_approx(m_run - m_new) : 1.f;
                if (grow) m_run = m_new;
                l_run *= alpha;
                // (stores to TMEM are asynchronous: the weights that these replace must be in place)
                if (begun) tmem_wait_st();
                l = weights128<DT>(s, sl2, (m_run == -INFINITY) ? 0.f : -m_run, tS);
                if (begun) {
                    if (!mbar_wait(smem_u32(&c.pv_done[t]), (g - 1) & 1, ab, err, kErrSoftmax)) return;
                    tc_fence_after();
                    const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
                    for (int c16 = 0; c16 < D / 16; c16++) {
                        uint32_t r[16];
                        tmem_ld16(tO + c16 * 16, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 o2 = fmul2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), a2);
                            r[e] = __float_as_uint(o2.x);
                            r[e + 1] = __float_as_uint(o2.y);
                        }
                        tmem_st16(tO + c16 * 16, r);
                    }
                }
            }
            l_run += l;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.p_full[t]));  // one arrival per warp
            begun = true;
            ++g;
        }
        // Row sum and shift for the epilogue, which must have read the previous ones.
        if (w > 0 && !mbar_wait(smem_u32(&c.o_free[t]), (w - 1) & 1, ab, err, kErrSoftmax)) return;
        c.epi_l[t][rl] = l_run;
        c.epi_shift[t][rl] = m_run;
        mbar_arrive(smem_u32(&c.epi_full[t]));
        ++w;
    }
}

// ------------------------------------------------------------------ epilogue

// Adds to 16 columns of an output row the non-finite values of the keys [from, see).
template <int DT>
__device__ __forceinline__ void add_not_finite(float *o, const ChunkItem &T, int from, int see, int col, const ChunkParams &p)
{
    const PagedArgs &a = p.a;
#pragma unroll 1
    for (int key = from; key < see; key++) {
        const int pg = __ldg(a.block_table + T.s * a.bt_s + (key >> a.page_shift));
        if (pg < 0 || pg >= a.num_pages) continue;
        const uint32_t *vs = reinterpret_cast<const uint32_t *>(
            a.vc + static_cast<int64_t>(pg) * a.vc_sp + T.h * a.vc_sh +
            static_cast<int64_t>(key & ((1 << a.page_shift) - 1)) * a.vc_sn + col);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t u = __ldg(vs + e);
            const float lo = elem_lo<DT>(u), hi = elem_hi<DT>(u);
            if (!isfinite(lo)) o[2 * e] += lo;
            if (!isfinite(hi)) o[2 * e + 1] += hi;
        }
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The same barrier; true in all threads if `bad` in one.
__device__ __forceinline__ bool epilogue_any(bool bad)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(bad ? 1u : 0u)
        : "memory");
    return r != 0;
}

// Partial result of place `slot` [D / 4][256][4] (a warp's rows lie side by side).
template <int D>
__device__ __forceinline__ float4 *part_at(const ChunkParams &p, int64_t slot, int c4, int r)
{
    return reinterpret_cast<float4 *>(p.part_o) + (slot * (D / 4) + c4) * (2 * BM) + r;
}

// 16 columns of an output row; inv = 1 / l, none: the row sees no key.
template <int DT>
__device__ __forceinline__ void store16(uint16_t *dst, const float *o, float inv, bool none, uint64_t pol)
{
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 8; e++) pk[e] = none ? 0u : pack2<DT>(o[2 * e] * inv, o[2 * e + 1] * inv);
    st_global_v4_hint(dst, make_uint4(pk[0], pk[1], pk[2], pk[3]), pol);
    st_global_v4_hint(dst + 8, make_uint4(pk[4], pk[5], pk[6], pk[7]), pol);
}

template <int D, int DT>
__device__ void epilogue_role(const ChunkParams &p, Ctl &c, uint32_t tmem, uint32_t sKV, int warp, int lane, const Run &R)
{
    using C = Cfg<D>;
    const PagedArgs &a = p.a;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int quarter = warp & 3;
    const int rl = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int row_tok = rl / p.g, row_head = rl - row_tok * p.g;
    const bool lead = rl == 0;
    const uint64_t pol = policy_evict_first();
    uint32_t g0 = 0, g1 = 0;  // steps of the two groups
    int w = 0;
    CLIS_FOR_WORK(K)
    {
        const ChunkItem &T = K.t;
        const int first = chunk_first_masked(T, a.causal != 0);
        const bool edges = K.start + K.n > first;
        ChunkOwners own = {static_cast<int>(blockIdx.x), 1};
        if (!K.whole) own = chunk_owners(T, R.cuts);
        const int me = static_cast<int>(blockIdx.x) - own.c;
        // The second of two parts done already (the usual case: the first part is the
        // last work of its block, the second the first of the next block): the first
        // need not go through memory.
        bool direct = false;
        if (own.count == 2 && me == 0) {
            if (lead) {
                int n;
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(p.arrived + own.c) : "memory");
                c.last = n == 1;
            }
            epilogue_barrier();
            direct = c.last != 0;
            epilogue_barrier();  // (c.last is written again below or by the next item)
        }
        const bool to_memory = own.count > 1 && !direct;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (K.start == 0 ? 1 : 0);
        const int64_t slot0 = 2 * own.c + 1, slot1 = 2 * (own.c + 1);  // the two parts' places

        // A single row tile's own values are the sum of both groups'.
        const bool single = T.nt == 1;
        float w_even = 1.f, w_odd = 0.f;
        bool has_odd = false;
        auto own16 = [&](uint32_t tO, int c16, float *o) {
            uint32_t x[16];
            tmem_ld16(tO + c16 * 16, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e++) o[e] = __uint_as_float(x[e]);
            if (has_odd) {
                tmem_ld16(tO + (C::TM_O1 - C::TM_O0) + c16 * 16, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] = fmaf(w_odd, __uint_as_float(x[e]), w_even * o[e]);
            }
        };
        // Joins the two parts of row tile t: the first from TMEM (staged = the place of
        // the second in shared memory) or, with staged = 0, both from memory.
        auto join_rows = [&](int t, uint32_t staged, float l0, float m0, int key_from, int see) {
            const int r = t * BM + rl, tok = T.tok0 + t * p.tpt + row_tok;
            const bool row_ok = row_tok < p.tpt && tok < T.n;
            float2 a0 = make_float2(m0, l0), a1 = make_float2(-INFINITY, 0.f);
            if (row_ok) {
                if (!staged) a0 = __ldcg(p.part_ml + slot0 * (2 * BM) + r);
                a1 = __ldcg(p.part_ml + slot1 * (2 * BM) + r);
            }
            // (a part none of whose keys the row sees adds nothing)
            const bool any0 = a0.y != 0.f, any1 = a1.y != 0.f;
            const float M = !any0 ? a1.x : !any1 ? a0.x : fmaxf(a0.x, a1.x);
            const float w0 = any0 ? ex2_approx(a0.x - M) : 0.f, w1 = any1 ? ex2_approx(a1.x - M) : 0.f;
            float l = any0 ? w0 * a0.y : 0.f;
            if (any1) l = fmaf(w1, a1.y, l);
            const int hd = T.h * p.g + row_head;
            uint16_t *orow = a.o + static_cast<int64_t>(T.q0 + tok) * a.o_st + hd * a.o_sh;
            const uint32_t tO = tmem + (t ? C::TM_O1 : C::TM_O0) + lane_off;
            const float inv = 1.f / l;
#pragma unroll 1
            for (int c16 = 0; c16 < D / 16; c16++) {
                float o[16];
                if (staged) {
                    own16(tO, c16, o);
                    if (key_from >= 0) add_not_finite<DT>(o, T, key_from, see, c16 * 16, p);
                }
                if (!row_ok) continue;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (!staged) {
                        const float4 x = __ldcg(part_at<D>(p, slot0, c16 * 4 + e, r));
                        o[4 * e] = x.x; o[4 * e + 1] = x.y; o[4 * e + 2] = x.z; o[4 * e + 3] = x.w;
                    }
                    float4 y;
                    if (staged) {
                        const uint4 u = lds128(staged + ((t * (D / 4) + c16 * 4 + e) * BM + rl) * 16);
                        y = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
                    } else {
                        y = __ldcg(part_at<D>(p, slot1, c16 * 4 + e, r));
                    }
                    const float yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int f = 0; f < 4; f++) {
                        const float x = any0 ? w0 * o[4 * e + f] : 0.f;
                        o[4 * e + f] = any1 ? fmaf(w1, yy[f], x) : x;
                    }
                }
                store16<DT>(orow + c16 * 16, o, inv, l == 0.f, pol);
            }
            if (row_ok && a.lse2) a.lse2[static_cast<int64_t>(T.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : M + log2f(l);
        };

        // Row sum and shift of row tile t (a single row tile's: of both groups).
        auto row_sums = [&](int t, float &l, float &shift) {
            l = c.epi_l[t][rl];
            shift = c.epi_shift[t][rl];
            if (single) {
                const float l1 = c.epi_l[1][rl], m1 = c.epi_shift[1][rl];
                const float M = l == 0.f ? m1 : l1 == 0.f ? shift : fmaxf(shift, m1);
                has_odd = K.n > 1;
                w_even = l == 0.f ? 0.f : ex2_approx(shift - M);  // (a group none of whose keys the row sees adds nothing)
                w_odd = l1 == 0.f ? 0.f : ex2_approx(m1 - M);
                l = (l == 0.f ? 0.f : w_even * l) + (l1 == 0.f ? 0.f : w_odd * l1);
                shift = M;
            }
        };
        // Non-finite values of keys from here on that a row sees were left out of the
        // product (-1: none were); to be asked once the products are done.
        auto left_out = [&]() -> int {
            return edges && *reinterpret_cast<volatile int *>(&c.dirty[w & 7]) != 0 ? max(first, K.start) * BN : -1;
        };
        auto seen = [&](int tok) { return min(visible_keys(T.n, T.kv, tok, a.causal), (K.start + K.n) * BN); };

#pragma unroll 1
        for (int t = 0; t < T.nt; t++) {
            bool ok;
            if (single) {
                g0 += (K.n + 1) / 2;
                g1 += K.n / 2;
                ok = mbar_wait(smem_u32(&c.epi_full[0]), w & 1, ab, err, kErrEpilogue) &&
                     mbar_wait(smem_u32(&c.epi_full[1]), w & 1, ab, err, kErrEpilogue) &&
                     mbar_wait(smem_u32(&c.pv_done[0]), (g0 - 1) & 1, ab, err, kErrEpilogue) &&
                     (K.n < 2 || mbar_wait(smem_u32(&c.pv_done[1]), (g1 - 1) & 1, ab, err, kErrEpilogue));
            } else {
                const uint32_t steps = t ? g1 += K.n : g0 += K.n;
                ok = mbar_wait(smem_u32(&c.epi_full[t]), w & 1, ab, err, kErrEpilogue) &&
                     mbar_wait(smem_u32(&c.pv_done[t]), (steps - 1) & 1, ab, err, kErrEpilogue);
            }
            // A wait that gave up ends all four warps together: one that went on would
            // stay at the barriers of a later item.
            if (epilogue_any(!ok)) return;
            tc_fence_after();
            if (direct) continue;  // (below, with both row tiles done)
            const uint32_t tO = tmem + (t ? C::TM_O1 : C::TM_O0) + lane_off;
            const int tok = T.tok0 + t * p.tpt + row_tok;
            const bool row_ok = row_tok < p.tpt && tok < T.n;
            float l, shift;
            row_sums(t, l, shift);
            const int key_from = left_out();
            const int see = row_ok ? seen(tok) : 0;
            const int hd = T.h * p.g + row_head;
            const float inv = 1.f / l;
            uint16_t *orow = a.o + static_cast<int64_t>(T.q0 + tok) * a.o_st + hd * a.o_sh;
#pragma unroll 1
            for (int c16 = 0; c16 < D / 16; c16++) {
                float o[16];
                own16(tO, c16, o);
                if (c16 == D / 16 - 1) {  // O has been read: the next item's products may start
                    tc_fence_before();
                    mbar_arrive(smem_u32(&c.o_free[t]));
                    if (single) mbar_arrive(smem_u32(&c.o_free[1]));
                }
                if (!row_ok) continue;
                if (key_from >= 0) add_not_finite<DT>(o, T, key_from, see, c16 * 16, p);
                if (to_memory) {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        __stcg(part_at<D>(p, slot, c16 * 4 + e, t * BM + rl),
                               make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                } else {
                    store16<DT>(orow + c16 * 16, o, inv, l == 0.f, pol);
                }
            }
            if (row_ok) {
                if (to_memory)
                    __stcg(p.part_ml + slot * (2 * BM) + t * BM + rl, make_float2(shift, l));
                else if (a.lse2)
                    a.lse2[static_cast<int64_t>(T.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : shift + log2f(l);
            }
        }
        // Who joins two parts: this block if the other part is done.
        bool joins = direct;
        if (to_memory && own.count == 2) {
            __threadfence();
            epilogue_barrier();
            if (lead) c.last = atomicAdd(p.arrived + own.c, 1) == 1;
            epilogue_barrier();
            joins = c.last != 0;
            if (joins) __threadfence();
            epilogue_barrier();
        }
        if (joins && me == 0) {
            // The block's last work: its own part is still in TMEM, and the K/V ring, free
            // after the last product, takes the other part, each thread its own row.
            tc_fence_after();
            for (int t = 0; t < T.nt; t++) {
                if (row_tok >= p.tpt || T.tok0 + t * p.tpt + row_tok >= T.n) continue;  // never written
#pragma unroll 8
                for (int c4 = 0; c4 < D / 4; c4++)
                    cp_async16(sKV + ((t * (D / 4) + c4) * BM + rl) * 16, part_at<D>(p, slot1, c4, t * BM + rl));
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
            for (int t = 0; t < T.nt; t++) {
                const int tok = T.tok0 + t * p.tpt + row_tok;
                float l, shift;
                row_sums(t, l, shift);
                join_rows(t, sKV, l, shift, left_out(), row_tok < p.tpt && tok < T.n ? seen(tok) : 0);
            }
        } else if (joins) {
#pragma unroll 1
            for (int t = 0; t < T.nt; t++) join_rows(t, 0u, 0.f, 0.f, -1, 0);
        }
        ++w;
    }
}

// -------------------------------------------------------------------- kernel

template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const ChunkParams p)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t dsmem[];
    __shared__ Ctl ctl;
    const uint32_t sbase = (smem_u32(dsmem) + 1023u) & ~1023u;
    const uint32_t sQ0 = sbase;
    const uint32_t sKV = sbase + 2 * C::TILE_BYTES;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(smem_u32(&ctl.q_full[t]), 1);
            mbar_init(smem_u32(&ctl.q_empty[t]), t == 0 ? 2 : 1);  // the first: products and the edge warp
            mbar_init(smem_u32(&ctl.s_full[t]), 1);
            mbar_init(smem_u32(&ctl.p_full[t]), BM / 32);
            mbar_init(smem_u32(&ctl.pv_done[t]), 1);
            mbar_init(smem_u32(&ctl.o_free[t]), BM);
            mbar_init(smem_u32(&ctl.epi_full[t]), BM);
        }
        for (int s = 0; s < C::NSTAGE; s++) {
            mbar_init(smem_u32(&ctl.kv_full[s]), 1);
            mbar_init(smem_u32(&ctl.kv_empty[s]), 1);
        }
        mbar_init(smem_u32(&ctl.edge_go), 1);
        mbar_init(smem_u32(&ctl.edge_ok), 1);
        mbar_init(smem_u32(&ctl.drain), 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 13) {
        tmem_alloc(smem_u32(&ctl.tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;

    pdl_wait();
    pdl_launch();
    Run R;
    {
        const int nb = static_cast<int>(p.head[2]);
        const unsigned long long U = p.head[1];
        const int c = blockIdx.x;
        R.items = c < nb ? static_cast<int>(p.head[0]) : 0;  // no items: nothing to do
        R.first = c < nb ? p.run_first[c] : 0;
        R.cuts = chunk_cuts(U, nb);
        R.lo = R.cuts.cut(c);
        R.hi = R.cuts.cut(c + 1);
    }

    // Register split (launch: 512 threads x 128 = 65536): softmax 2 x 128 x 176,
    // epilogue 128 x 80, the other four warps 128 x 80.
    if (warp < 8) {
        setmaxnreg_inc<176>();
        softmax_role<D, DT>(p, ctl, tmem, warp, lane, R);
    } else if (warp < 12) {
        setmaxnreg_dec<80>();
        epilogue_role<D, DT>(p, ctl, tmem, sKV, warp, lane, R);
    } else {
        setmaxnreg_dec<80>();
        if (warp == 12) producer_role<D>(p, ctl, &tm_k, &tm_v, sKV, R);
        if (warp == 13) mma_role<D, DT>(p, ctl, tmem, sQ0, sKV, R);
        if (warp == 14) q_producer_role<D>(p, ctl, &tm_q, sQ0, R);
        if (warp == 15) edge_role<D, DT>(p, ctl, sKV, R);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Adds the partial results of items of three parts or more: part 0 in place
// 2 c + 1, part k in place 2 (c + k), c the block that started the item.  A block
// takes 32 rows (lane = row) and 16 columns, its warps every eighth part; sums
// over parts run in a fixed order.
constexpr int kJoinWarps = 8;

template <int D, int DT>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_chunk_join_kernel(const ChunkParams p)
{
    const PagedArgs &a = p.a;
    __shared__ float s_o[kJoinWarps][16][33], s_m[kJoinWarps][32], s_l[kJoinWarps][32];
    pdl_wait();
    const int joins = *p.joins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * 32 + lane, tile = r / BM, rl = r % BM, c16 = blockIdx.z;
    const int rt = rl / p.g;
    for (int i = blockIdx.x; i < joins; i += gridDim.x) {
        const int2 jn = p.join[i];
        const int parts = jn.x;
        const ChunkItem T = load_item(p, jn.y);
        if (static_cast<int>(blockIdx.y) * 32 / BM >= T.nt) continue;
        const int tok = T.tok0 + tile * p.tpt + rt;
        const bool row_ok = rt < p.tpt && tok < T.n;  // (other rows' partial results were never written)
        const int nb = static_cast<int>(p.head[2]);
        const int c = chunk_owners(T, chunk_cuts(p.head[1], nb)).c;
        float M = -INFINITY, l = 0.f, o[16];
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] = 0.f;
        if (row_ok) {
#pragma unroll 2
            for (int k = warp; k < parts; k += kJoinWarps) {
                const int64_t s = k == 0 ? 2 * c + 1 : 2 * (c + k);
                const float2 ml = p.part_ml[s * (2 * BM) + r];
                float4 u[4];
#pragma unroll
                for (int e = 0; e < 4; e++) u[e] = *part_at<D>(p, s, c16 * 4 + e, r);
                if (ml.y == 0.f) continue;  // a part none of whose keys the row sees adds nothing
                const float m = fmaxf(M, ml.x);
                const bool none = l == 0.f;
                const float w0 = none ? 0.f : ex2_approx(M - m), w = ex2_approx(ml.x - m);
                M = m;
                l = none ? w * ml.y : fmaf(l, w0, w * ml.y);
                const float x[16] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w,
                                     u[2].x, u[2].y, u[2].z, u[2].w, u[3].x, u[3].y, u[3].z, u[3].w};
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] = none ? w * x[e] : fmaf(o[e], w0, w * x[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 16; e++) s_o[warp][e][lane] = o[e];
        s_m[warp][lane] = M;
        s_l[warp][lane] = l;
        __syncthreads();
        if (warp < 2 && row_ok) {
            // Warps 0 and 1: eight columns each, over the warps' sums in order.
            M = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; w++)
                if (s_l[w][lane] != 0.f) M = fmaxf(M, s_m[w][lane]);
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; w++) {
                const float lw = s_l[w][lane];
                if (lw == 0.f) continue;
                const float g = ex2_approx(s_m[w][lane] - M);
                l = fmaf(g, lw, l);
#pragma unroll
                for (int e = 0; e < 8; e++) o[e] = fmaf(g, s_o[w][warp * 8 + e][lane], o[e]);
            }
            const float inv = 1.f / l;
            const int hd = T.h * p.g + (rl - rt * p.g);
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; e++) pk[e] = l == 0.f ? 0u : pack2<DT>(o[2 * e] * inv, o[2 * e + 1] * inv);
            *reinterpret_cast<uint4 *>(a.o + static_cast<int64_t>(T.q0 + tok) * a.o_st + hd * a.o_sh + c16 * 16 + warp * 8) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
            if (c16 == 0 && warp == 0 && a.lse2)
                a.lse2[static_cast<int64_t>(T.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : M + log2f(l);
        }
        __syncthreads();  // (the sums are written again)
    }
}

// ------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult qres;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qres) ==
                cudaSuccess &&
            qres == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

bool encode(CUtensorMap *map, const void *base, int dtype, int rank, const cuuint64_t *dims, const int64_t *elem_strides,
            const cuuint32_t *box)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t strides[3];
    for (int i = 0; i + 1 < rank; i++) {
        // A stride of a size-1 dimension is never used; give it a canonical value.
        const int64_t s = dims[i + 1] == 1 ? static_cast<int64_t>(dims[0]) : elem_strides[i];
        strides[i] = static_cast<cuuint64_t>(s) * 2;
    }
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, dtype == CLIS_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int64_t max_items(const PagedArgs &a) { return chunk_list(a.T, a.S, a.H / a.Hkv, a.Hkv); }

template <int D, int DT>
clis_status_t launch_impl(const ChunkParams &p, cudaStream_t stream)
{
    using C = Cfg<D>;
    const PagedArgs &a = p.a;
    if (cudaFuncSetAttribute(paged_chunk_kernel<D, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
        return CLIS_ERR_CUDA;
    CUtensorMap mq, mk, mv;
    {
        const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.T)};
        const int64_t st[2] = {a.q_sh, a.q_st};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.g), static_cast<cuuint32_t>(p.tpt)};
        if (!encode(&mq, a.q, DT, 3, dims, st, box)) return CLIS_ERR_CUDA;
    }
    {
        const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(1) << a.page_shift, static_cast<cuuint64_t>(a.Hkv),
                                    static_cast<cuuint64_t>(a.num_pages)};
        const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.box_rows), 1, 1};
        const int64_t ks[3] = {a.kc_sn, a.kc_sh, a.kc_sp}, vs[3] = {a.vc_sn, a.vc_sh, a.vc_sp};
        if (!encode(&mk, a.kc, DT, 4, dims, ks, box) || !encode(&mv, a.vc, DT, 4, dims, vs, box)) return CLIS_ERR_CUDA;
    }
    if (launch_pdl(paged_chunk_kernel<D, DT>, dim3(p.grid), kThreads, C::SMEM_BYTES, stream, mq, mk, mv, p) != cudaSuccess)
        return CLIS_ERR_CUDA;
    // One wave of blocks over the list; mostly it is short or empty.
    const int64_t items = max_items(a), wave = p.grid / 8;
    const int joins = static_cast<int>(imin(max_joins(p.grid), static_cast<int>(items < wave ? items : wave > 1 ? wave : 1)));
    if (launch_pdl(paged_chunk_join_kernel<D, DT>, dim3(joins, 2 * BM / 32, D / 16), 32 * kJoinWarps, 0, stream, p) !=
        cudaSuccess)
        return CLIS_ERR_CUDA;
    return CLIS_OK;
}

}  // namespace

size_t paged_chunk_workspace(const PagedArgs &a, int nsm)
{
    const size_t grid = static_cast<size_t>(nsm);
    return 256 + 2 * up256(grid * sizeof(int)) + up256(max_joins(nsm) * sizeof(int2)) +
           up256(static_cast<size_t>(max_items(a)) * sizeof(ChunkItem)) + up256(2 * grid * 2 * BM * sizeof(float2)) +
           up256(2 * grid * 2 * BM * a.d * sizeof(float));
}

namespace {

ChunkParams chunk_params(const PagedArgs &a, int rows_small, void *workspace, int nsm)
{
    ChunkParams p;
    p.a = a;
    p.g = a.H / a.Hkv;
    p.tpt = BM / p.g;
    p.rows_small = rows_small;
    p.grid = nsm;
    p.least = 2 * kChunkOverhead;
    p.box_rows = imin(1 << a.page_shift, BN);
    p.list = static_cast<int>(max_items(a));  // (below 10^9, which the entry point checks)
    const size_t grid = static_cast<size_t>(nsm);
    char *w = static_cast<char *>(workspace);
    p.head = reinterpret_cast<unsigned long long *>(w);
    p.joins = reinterpret_cast<int *>(w + 128);
    w += 256;
    p.run_first = reinterpret_cast<int *>(w);
    w += up256(grid * sizeof(int));
    p.arrived = reinterpret_cast<int *>(w);
    w += up256(grid * sizeof(int));
    p.join = reinterpret_cast<int2 *>(w);
    w += up256(max_joins(nsm) * sizeof(int2));
    p.items = reinterpret_cast<ChunkItem *>(w);
    w += up256(static_cast<size_t>(max_items(a)) * sizeof(ChunkItem));
    p.part_ml = reinterpret_cast<float2 *>(w);
    w += up256(2 * grid * 2 * BM * sizeof(float2));
    p.part_o = reinterpret_cast<float *>(w);
    return p;
}

}  // namespace

clis_status_t launch_paged_chunk_schedule(const PagedArgs &a, int rows_small, void *workspace, int nsm,
                                          cudaStream_t stream)
{
    const ChunkParams p = chunk_params(a, rows_small, workspace, nsm);
    const size_t smem = sizeof(int) * (static_cast<size_t>(a.S) + 1);
    if (smem > 48 * 1024 && cudaFuncSetAttribute(paged_chunk_schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem)) != cudaSuccess)
        return CLIS_ERR_CUDA;
    paged_chunk_schedule_kernel<<<1, kSchedThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t launch_paged_chunk(const PagedArgs &a, int rows_small, void *workspace, int nsm, cudaStream_t stream)
{
    const ChunkParams p = chunk_params(a, rows_small, workspace, nsm);
    const bool f16 = a.dtype == CLIS_DT_FP16;
    if (a.d == 128) return f16 ? launch_impl<128, 1>(p, stream) : launch_impl<128, 0>(p, stream);
    return f16 ? launch_impl<64, 1>(p, stream) : launch_impl<64, 0>(p, stream);
}

clis_status_t read_chunk_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_chunk_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_chunk_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_chunk_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
