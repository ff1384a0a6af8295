// paged_chunk.cu -- attention of chunks of new tokens over a paged key/value
// cache on the tcgen05 tensor cores (sequences with more query rows than the
// decode kernel takes).
//
//   x_ij = scale_log2 * q_i . k_j,  o_i = sum_j 2^(x_ij - m_i) v_j / sum_j 2^(x_ij - m_i)
//
// over the keys j < visible(i), with the running shift m_i raised only when a
// row's maximum outgrew it by 2^8.
//
// Bound: the tensor cores (4 d flops per row and visible key), then exp2 on the
// MUFU.  A work tile is two 128-row tiles; a row tile packs 128 / g tokens of
// all g query heads of one key/value head, so each key tile that is loaded
// serves every head that shares it.  The pipeline of one persistent block:
//
//   warps 0-3, 4-7  softmax of row tile 0, 1 (thread = row)
//   warps 8-11      epilogue: O / l, or a partial result where the keys of a
//                   work tile are shared out
//   warp 12         TMA producer of K and V: 128-key tiles gathered page by page
//   warp 13         MMA issuer, owns TMEM
//   warp 14         TMA producer of Q
//   warp 15         edge tiles of V: rows behind the last key become zeros, and
//                   non-finite values of keys that some row must not see are
//                   taken out of the product (0 * NaN would reach every row) and
//                   added by the epilogue to the rows that see them
//
// A one-block kernel first writes the list of work tiles (the lengths live on
// the device); block i takes tiles i, 2 G - 1 - i, 2 G + i, ... (G blocks), which
// evens out costs that rise or fall along the list.  Every wait is bounded.
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
constexpr int kSchedThreads = 1024;

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
    int slots, least;     // places for tiles when keys are shared out; key tiles per part
    int box_rows;         // rows of a K/V TMA box: min(page size, 128)
    ChunkTile *tiles;
    int *count;           // {tiles, first work tile of a sequence whose keys are shared out: 0/1}
    float *part_o;        // [slots'][256][D]
    float2 *part_ml;      // [slots'][256]
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
    int dirty[8];  // per work tile (mod 8): non-finite values were taken out
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ SeqLen seq_len(const PagedArgs &a, int s)
{
    return clip_seq(__ldg(a.cu_q + s), __ldg(a.cu_q + s + 1), __ldg(a.kv_len + s), a.T, a.width << a.page_shift);
}

// ------------------------------------------------------------------ schedule

__global__ void __launch_bounds__(kSchedThreads) paged_chunk_schedule_kernel(const ChunkParams p)
{
    extern __shared__ int s_first[];  // [S + 1] first tile of each sequence
    __shared__ unsigned long long s_total, s_items;
    __shared__ int s_warp[kSchedThreads / 32];
    const PagedArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned int bad = 0;
    if (tid == 0) s_total = s_items = 0;
    __syncthreads();
    unsigned long long total = 0, items = 0;
    for (int s = tid; s < a.S; s += kSchedThreads) {
        const SeqLen q = seq_len(a, s);
        if (q.bad) bad |= CLIS_PAGED_LENGTH_BIT;
        if (q.n == 0 || is_decode(q, p.g, p.rows_small)) continue;
        const unsigned long long it = static_cast<unsigned long long>(a.Hkv) * chunk_q_tiles(q.n, p.g);
        items += it;
        total += it * chunk_max_cost(q);
    }
    // (integer sums: the order in which they are added does not matter)
    if (items) {
        atomicAdd(&s_items, items);
        atomicAdd(&s_total, total);
    }
    __syncthreads();
    const int len = chunk_part_len(s_total, s_items, p.slots, p.least);
    const int per = (a.S + kSchedThreads - 1) / kSchedThreads;
    const int s0 = min(a.S, tid * per), s1 = min(a.S, s0 + per);
    auto tiles_of = [&](int s) -> int {
        const SeqLen q = seq_len(a, s);
        if (q.n == 0 || is_decode(q, p.g, p.rows_small)) return 0;
        return a.Hkv * chunk_q_tiles(q.n, p.g) * chunk_parts(q, len);
    };
    int mine = 0;
    for (int s = s0; s < s1; s++) mine += tiles_of(s);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int run = incl - mine;
    for (int w = 0; w < warp; w++) run += s_warp[w];
    for (int s = s0; s < s1; s++) {
        s_first[s] = run;
        run += tiles_of(s);
    }
    if (s0 < a.S && s1 == a.S) s_first[a.S] = run;
    __syncthreads();
    const int W = s_first[a.S];
    for (int t = tid; t < W; t += kSchedThreads) {
        int lo = 0, hi = a.S;  // s_first[lo] <= t < s_first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_first[mid] <= t) lo = mid;
            else hi = mid;
        }
        const SeqLen q = seq_len(a, lo);
        p.tiles[t] = chunk_tile(q, lo, p.g, chunk_parts(q, len), t - s_first[lo], a.causal != 0);
    }
    if (tid == 0) *p.count = W;
    if (bad) atomicOr(&g_chunk_error_word, bad);
}

// i-th tile of this block (-1: no more).
__device__ __forceinline__ int tile_at(int i, int W)
{
    const int G = gridDim.x;
    const int t = i * G + ((i & 1) ? G - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
    if (i * static_cast<int64_t>(G) >= W) return -1;
    return t < W ? t : -2;  // -2: this round has no tile for the block
}

__device__ __forceinline__ ChunkTile load_tile(const ChunkParams &p, int t)
{
    union { int4 v[3]; ChunkTile c; } u;
    const int4 *src = reinterpret_cast<const int4 *>(p.tiles + t);
    u.v[0] = __ldg(src);
    u.v[1] = __ldg(src + 1);
    u.v[2] = __ldg(src + 2);
    return u.c;
}

// Loop over this block's work tiles; `w` counts them.
#define CLIS_FOR_TILES(T)                                                  \
    for (int i_ = 0, t_; (t_ = tile_at(i_, W)) != -1; ++i_)                \
        if (t_ >= 0)                                                       \
            if (const ChunkTile T = load_tile(p, t_); true)

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
__device__ void q_producer_role(const ChunkParams &p, Ctl &c, const CUtensorMap *tm_q, uint32_t sQ0, int W)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const bool leader = elect_one();
    const uint64_t pol = policy_evict_first();
    int wt[2] = {0, 0};
    CLIS_FOR_TILES(T)
    {
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
                              uint32_t sKV, int W)
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
    CLIS_FOR_TILES(T)
    {
        // Page of the lane's rows of key tile kt; -2: behind the last key, not loaded.
        auto page_of = [&](int kt) -> int {
            const int key = kt * BN + lane * p.box_rows;
            if (lane >= npg || key >= T.kv) return -2;
            return __ldg(a.block_table + T.s * a.bt_s + (key >> a.page_shift));
        };
        int pg_k = page_of(T.start), pg_v = -2;
        // Groups of loads as the MMA warp needs them: {K_0}, {V_0, K_1}, ..., {V_{n-1}}.
        for (int gi = 0; gi <= T.n_kv; gi++) {
            const bool has_v = gi > 0, has_k = gi < T.n_kv;
            const int nl = (has_v ? 1 : 0) + (has_k ? 1 : 0);
            const int pg_next = gi + 1 < T.n_kv ? page_of(T.start + gi + 1) : -2;
            for (int l = 0; l < nl; l++) {
                const uint32_t li = it + l;
                if (!mbar_wait_warp(smem_u32(&c.kv_empty[li % C::NSTAGE]), ((li / C::NSTAGE) & 1) ^ 1, ab, err,
                                    kErrProducer))
                    goto abort;
            }
            const uint32_t bar = smem_u32(&c.kv_full[gq % C::NSTAGE]);
            const int live = __popc(__ballot_sync(~0u, has_v && pg_v != -2)) + __popc(__ballot_sync(~0u, has_k && pg_k != -2));
            if (lane == 0) mbar_arrive_expect_tx(bar, live * C::NBOX * box_bytes);
            __syncwarp();
#pragma unroll
            for (int l = 0; l < 2; l++) {
                const bool is_v = l == 0;
                if (is_v ? !has_v : !has_k) continue;
                int pg = is_v ? pg_v : pg_k;
                if (pg == -2) continue;
                if (pg < 0 || pg >= a.num_pages) {
                    bad |= CLIS_PAGED_INDEX_BIT;
                    pg = static_cast<int>(a.num_pages);  // out of the map: its rows read as zeros
                }
                const uint32_t slot = (it + (is_v ? 0 : nl - 1)) % C::NSTAGE;
                const int key = (T.start + (is_v ? gi - 1 : gi)) * BN + lane * p.box_rows;
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
__device__ void edge_role(const ChunkParams &p, Ctl &c, uint32_t sKV, int W)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int lane = threadIdx.x & 31;
    uint32_t it = 0, gq = 0, nedge = 0;
    int w = 0;
    CLIS_FOR_TILES(T)
    {
        const int first = chunk_first_masked(T, p.a.causal != 0);
        bool dirty = false;
        for (int j = 0; j < T.n_kv; j++) {
            const int kt = T.start + j;
            if (kt < first) continue;
            // V_j is in load group j + 1 and in ring slot 2 j + 1 of the work tile's
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
            const int live = min(BN, T.kv - kt * BN);  // rows that hold keys (may be <= 0)
            // Rows of 128 bytes, two boxes at d = 128; the swizzle permutes 16-byte
            // pieces within a row, so a row is a row.
            if (p.a.causal) {
#pragma unroll 4
                for (int i = lane; i < C::NBOX * BN * 8; i += 32) {
                    const int row = (i >> 3) & (BN - 1);
                    const uint32_t at = base + i * 16;
                    if (row < live) {
                        uint4 u = lds128(at);
                        const bool d0 = scrub<DT>(u.x), d1 = scrub<DT>(u.y), d2 = scrub<DT>(u.z), d3 = scrub<DT>(u.w);
                        if (d0 | d1 | d2 | d3) {
                            sts128(at, u);
                            dirty = true;
                        }
                    } else {
                        sts128(at, make_uint4(0u, 0u, 0u, 0u));
                    }
                }
            } else {
                const int from = max(live, 0) * 8;
                for (int bx = 0; bx < C::NBOX; bx++)
                    for (int i = from + lane; i < BN * 8; i += 32)
                        sts128(base + bx * C::BOX_BYTES + i * 16, make_uint4(0u, 0u, 0u, 0u));
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
        it += 2 * T.n_kv;
        gq += T.n_kv + 1;
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

template <int D, int DT>
__device__ void mma_role(const ChunkParams &p, Ctl &c, uint32_t tmem, uint32_t sQ0, uint32_t sKV, int W)
{
    using C = Cfg<D>;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const bool leader = elect_one();
    uint32_t it = 0, gq = 0, nedge = 0;
    uint32_t wt[2] = {0, 0}, gt[2] = {0, 0};  // per row tile: work tiles, steps
    const uint64_t qd0 = sdesc_sw128(sQ0, 16, 1024);
    const uint64_t qd1 = sdesc_sw128(sQ0 + C::TILE_BYTES, 16, 1024);
    const uint64_t kvd_k = sdesc_sw128(sKV, 16, 1024);
    const uint64_t kvd_v = sdesc_sw128(sKV, C::BOX_BYTES, 1024);
    auto stage_off = [](uint32_t s) -> uint64_t { return (s * C::TILE_BYTES) >> 4; };
    CLIS_FOR_TILES(T)
    {
        const int nt = T.nt;
        const int first = chunk_first_masked(T, p.a.causal != 0);
        for (int t = 0; t < nt; t++)
            if (!mbar_wait_warp(smem_u32(&c.q_full[t]), wt[t] & 1, ab, err, kErrMma)) goto abort;
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
                if (T.n_kv == 1)
                    for (int t = 0; t < nt; t++) umma_commit(smem_u32(&c.q_empty[t]));
            }
            __syncwarp();
            ++it;
        }
        for (int j = 0; j < T.n_kv; j++) {
            const bool has_next = j + 1 < T.n_kv;
            const uint32_t vs = it % C::NSTAGE;
            if (!mbar_wait_warp(smem_u32(&c.kv_full[gq % C::NSTAGE]), (gq / C::NSTAGE) & 1, ab, err, kErrMma))
                goto abort;
            ++gq;
            const bool edge = T.start + j >= first;
            if (edge && leader) mbar_arrive(smem_u32(&c.edge_go));
            if (edge) {
                if (!mbar_wait_warp(smem_u32(&c.edge_ok), nedge & 1, ab, err, kErrMma)) goto abort;
                ++nedge;
            }
            const uint64_t vd = kvd_v + stage_off(vs);
            const uint32_t kns = (it + 1) % C::NSTAGE;
            const uint64_t kd = kvd_k + stage_off(kns);
#pragma unroll
            for (int t = 0; t < 2; t++) {
                if (t >= nt) break;
                const bool last = t == nt - 1;
                if (!mbar_wait_warp(smem_u32(&c.p_full[t]), gt[t] & 1, ab, err, kErrMma)) goto abort;
                if (j == 0)
                    if (!mbar_wait_warp(smem_u32(&c.o_free[t]), (wt[t] & 1) ^ 1, ab, err, kErrMma)) goto abort;
                tc_fence_after();
                if (leader) {
                    issue_pv<D, DT>(tmem + (t ? C::TM_O1 : C::TM_O0), tmem + (t ? C::TM_S1 : C::TM_S0), vd,
                                    j > 0 ? 1u : 0u);
                    umma_commit(smem_u32(&c.pv_done[t]));
                    if (last) umma_commit(smem_u32(&c.kv_empty[vs]));
                    if (has_next) {
                        issue_qk<D, DT>(tmem + (t ? C::TM_S1 : C::TM_S0), t ? qd1 : qd0, kd);
                        umma_commit(smem_u32(&c.s_full[t]));
                        if (last) umma_commit(smem_u32(&c.kv_empty[kns]));
                        if (j + 1 == T.n_kv - 1) umma_commit(smem_u32(&c.q_empty[t]));
                    }
                }
                __syncwarp();
                ++gt[t];
            }
            it += has_next ? 2 : 1;
        }
        for (int t = 0; t < nt; t++) ++wt[t];
    }
    return;
abort:
    if (leader) umma_commit(smem_u32(&c.drain));
    __syncwarp();
    drain_wait(smem_u32(&c.drain), 0);
}

// ------------------------------------------------------------------- softmax

template <int D, int DT>
__device__ void softmax_role(const ChunkParams &p, Ctl &c, uint32_t tmem, int warp, int lane, int W)
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
    CLIS_FOR_TILES(T)
    {
        if (t >= T.nt) continue;
        const int tok = T.tok0 + t * p.tpt + row_tok;
        const bool row_ok = row_tok < p.tpt && tok < T.n && !T.masked;
        const int lim = row_ok ? visible_keys(T.n, T.kv, tok, p.a.causal) : 0;  // keys [0, lim) are visible
        float m_run = -INFINITY, l_run = 0.f;
        for (int j = 0; j < T.n_kv; j++) {
            if (!mbar_wait(smem_u32(&c.s_full[t]), g & 1, ab, err, kErrSoftmax)) return;
            tc_fence_after();
            uint32_t s[BN];
            tmem_ld32(tS + 0, s + 0);
            tmem_ld32(tS + 32, s + 32);
            tmem_ld32(tS + 64, s + 64);
            tmem_ld32(tS + 96, s + 96);
            tmem_wait_ld();
            const int key0 = (T.start + j) * BN;
            if (key0 + BN > lim) {
#pragma unroll
                for (int cc = 0; cc < BN; cc++)
                    if (key0 + cc >= lim) s[cc] = 0xFF800000u;  // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int cc = 0; cc < BN; cc += 8) {
#pragma unroll
                for (int q4 = 0; q4 < 4; q4++)
                    mx[q4] = fmax3(mx[q4], __uint_as_float(s[cc + 2 * q4]), __uint_as_float(s[cc + 2 * q4 + 1]));
            }
            const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
            float alpha = 1.f;
            const bool grow = m_tile > m_run + kTau;
            if (grow) {
                if (j > 0) alpha = ex2_approx(m_run - m_tile);
                m_run = m_tile;
            }
            const bool rescale = j > 0 && __any_sync(0xFFFFFFFFu, grow);
            const float nshift = (m_run == -INFINITY) ? 0.f : -m_run;
            const float2 sc2 = make_float2(sl2, sl2), sh2 = make_float2(nshift, nshift);
            float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
            for (int c32 = 0; c32 < BN / 32; c32++) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const float2 x = ffma2(make_float2(__uint_as_float(s[c32 * 32 + 2 * e]),
                                                       __uint_as_float(s[c32 * 32 + 2 * e + 1])),
                                           sc2, sh2);
                    const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    if (e & 1) lb = fadd2(lb, pp);
                    else la = fadd2(la, pp);
                    pk[e] = pack2<DT>(pp.x, pp.y);
                }
                tmem_st16(tS + c32 * 16, pk);
            }
            const float2 lab = fadd2(la, lb);
            l_run = l_run * alpha + (lab.x + lab.y);
            if (rescale) {
                // O of the warp's rows shrinks to the new shift once the previous product
                // is in it, before this step's arrival lets the next one start.
                if (!mbar_wait(smem_u32(&c.pv_done[t]), (g - 1) & 1, ab, err, kErrSoftmax)) return;
                tc_fence_after();
                const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
                for (int c32 = 0; c32 < D / 32; c32++) {
                    uint32_t r[32];
                    tmem_ld32(tO + c32 * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 o2 = fmul2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), a2);
                        r[e] = __float_as_uint(o2.x);
                        r[e + 1] = __float_as_uint(o2.y);
                    }
                    tmem_st32(tO + c32 * 32, r);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&c.p_full[t]));
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

template <int D, int DT>
__device__ void epilogue_role(const ChunkParams &p, Ctl &c, uint32_t tmem, int warp, int lane, int W)
{
    using C = Cfg<D>;
    const PagedArgs &a = p.a;
    volatile int *ab = &c.abort_flag;
    unsigned *err = &g_chunk_error_word;
    const int quarter = warp & 3;
    const int rl = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int row_tok = rl / p.g, row_head = rl - row_tok * p.g;
    const uint64_t pol_o = policy_evict_first();
    uint32_t gt[2] = {0, 0}, wt[2] = {0, 0};
    int w = 0;
    CLIS_FOR_TILES(T)
    {
        const int first = chunk_first_masked(T, a.causal != 0);
        const bool edges = T.start + T.n_kv > first;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            if (t >= T.nt) break;
            gt[t] += T.n_kv;
            if (!mbar_wait(smem_u32(&c.epi_full[t]), wt[t] & 1, ab, err, kErrEpilogue)) return;
            if (!mbar_wait(smem_u32(&c.pv_done[t]), (gt[t] - 1) & 1, ab, err, kErrEpilogue)) return;
            tc_fence_after();
            const bool dirty = edges && *reinterpret_cast<volatile int *>(&c.dirty[w & 7]) != 0;
            const uint32_t tO = tmem + (t ? C::TM_O1 : C::TM_O0) + lane_off;
            const int tok = T.tok0 + t * p.tpt + row_tok;
            const bool row_ok = row_tok < p.tpt && tok < T.n;
            const float l = c.epi_l[t][rl], shift = c.epi_shift[t][rl];
            const float inv = 1.f / l;
            const int see = min(visible_keys(T.n, T.kv, tok, a.causal), (T.start + T.n_kv) * BN);
            const int hd = T.h * p.g + row_head;
            uint16_t *orow = a.o + static_cast<int64_t>(T.q0 + tok) * a.o_st + hd * a.o_sh;
            const int64_t prow = static_cast<int64_t>(t_) * (2 * BM) + t * BM + rl;
#pragma unroll 1
            for (int c32 = 0; c32 < D / 32; c32++) {
                uint32_t r[32];
                tmem_ld32(tO + c32 * 32, r);
                tmem_wait_ld();
                if (!row_ok) continue;
                if (dirty && !T.masked) {
                    // Non-finite values of keys that this row sees and that were left out.
#pragma unroll 1
                    for (int key = max(first, T.start) * BN; key < see; key++) {
                        const int pg = __ldg(a.block_table + T.s * a.bt_s + (key >> a.page_shift));
                        if (pg < 0 || pg >= a.num_pages) continue;
                        const uint16_t *vs = a.vc + static_cast<int64_t>(pg) * a.vc_sp + T.h * a.vc_sh +
                                             static_cast<int64_t>(key & ((1 << a.page_shift) - 1)) * a.vc_sn + c32 * 32;
#pragma unroll
                        for (int e = 0; e < 32; e++) {
                            const float x = elem_lo<DT>(__ldg(vs + e));
                            if (!isfinite(x)) r[e] = __float_as_uint(__uint_as_float(r[e]) + x);
                        }
                    }
                }
                if (T.parts > 1) {
                    float4 *d4 = reinterpret_cast<float4 *>(p.part_o + prow * D + c32 * 32);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        d4[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                            __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
                } else {
                    uint32_t pk[16];
                    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const float2 o2 =
                            fmul2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), inv2);
                        pk[e] = l == 0.f ? 0u : pack2<DT>(o2.x, o2.y);  // a row that sees no key
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(orow + c32 * 32);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        st_global_v4_hint(dst + e,
                                          make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]), pol_o);
                }
            }
            if (row_ok) {
                if (T.parts > 1)
                    p.part_ml[prow] = make_float2(shift, l);
                else if (a.lse2)
                    a.lse2[static_cast<int64_t>(T.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : shift + log2f(l);
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&c.o_free[t]));
            ++wt[t];
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
    const int W = __ldg(p.count);

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(smem_u32(&ctl.q_full[t]), 1);
            mbar_init(smem_u32(&ctl.q_empty[t]), 1);
            mbar_init(smem_u32(&ctl.s_full[t]), 1);
            mbar_init(smem_u32(&ctl.p_full[t]), BM);
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

    // Register split (launch: 512 threads x 128 = 65536): softmax 2 x 128 x 176,
    // epilogue 128 x 80, the other four warps 128 x 80.
    if (warp < 8) {
        setmaxnreg_inc<176>();
        softmax_role<D, DT>(p, ctl, tmem, warp, lane, W);
    } else if (warp < 12) {
        setmaxnreg_dec<80>();
        epilogue_role<D, DT>(p, ctl, tmem, warp, lane, W);
    } else {
        setmaxnreg_dec<80>();
        if (warp == 12) producer_role<D>(p, ctl, &tm_k, &tm_v, sKV, W);
        if (warp == 13) mma_role<D, DT>(p, ctl, tmem, sQ0, sKV, W);
        if (warp == 14) q_producer_role<D>(p, ctl, &tm_q, sQ0, W);
        if (warp == 15) edge_role<D, DT>(p, ctl, sKV, W);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the parts of work tiles whose keys were shared out: a warp per row, the
// parts in order (fixed, so reruns agree bit for bit).
template <int D, int DT>
__global__ void __launch_bounds__(256) paged_chunk_join_kernel(const ChunkParams p)
{
    constexpr int V = D / 32;
    const PagedArgs &a = p.a;
    const int t = blockIdx.x;
    if (t >= __ldg(p.count)) return;
    const ChunkTile T = load_tile(p, t);
    if (T.parts == 1 || T.part != 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nqt = chunk_q_tiles(T.n, p.g);
    const int rows = p.tpt * p.g;
    for (int r = blockIdx.y * 8 + warp; r < 2 * BM; r += gridDim.y * 8) {
        const int tile = r / BM, rl = r % BM;
        const int rt = rl / p.g, tok = T.tok0 + tile * p.tpt + rt;
        if (tile >= T.nt || rl >= rows || tok >= T.n) continue;
        float M = -INFINITY;
        for (int k = lane; k < T.parts; k += 32) {
            const float2 ml = p.part_ml[(static_cast<int64_t>(t) + static_cast<int64_t>(k) * nqt) * (2 * BM) + r];
            if (ml.y != 0.f) M = fmaxf(M, ml.x);
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
        float l = 0.f, o[V];
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = 0.f;
#pragma unroll 4
        for (int k = 0; k < T.parts; k++) {
            const int64_t at = (static_cast<int64_t>(t) + static_cast<int64_t>(k) * nqt) * (2 * BM) + r;
            const float2 ml = p.part_ml[at];
            if (ml.y == 0.f) continue;
            const float w = ex2_approx(ml.x - M);
            l = fmaf(w, ml.y, l);
            if (V == 4) {
                const float4 u = *reinterpret_cast<const float4 *>(p.part_o + at * D + lane * 4);
                o[0] = fmaf(w, u.x, o[0]);
                o[1] = fmaf(w, u.y, o[1]);
                o[2 % V] = fmaf(w, u.z, o[2 % V]);
                o[3 % V] = fmaf(w, u.w, o[3 % V]);
            } else {
                const float2 u = *reinterpret_cast<const float2 *>(p.part_o + at * D + lane * 2);
                o[0] = fmaf(w, u.x, o[0]);
                o[1] = fmaf(w, u.y, o[1]);
            }
        }
        const float inv = 1.f / l;
        const int hd = T.h * p.g + (rl - rt * p.g);
        uint16_t *dst = a.o + static_cast<int64_t>(T.q0 + tok) * a.o_st + hd * a.o_sh + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2)
            *reinterpret_cast<uint32_t *>(dst + e) = l == 0.f ? 0u : pack2<DT>(o[e] * inv, o[e + 1] * inv);
        if (lane == 0 && a.lse2)
            a.lse2[static_cast<int64_t>(T.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : M + log2f(l);
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

// Work tiles if no keys are shared out, at most.
int64_t max_items(const PagedArgs &a)
{
    const int g = a.H / a.Hkv;
    return static_cast<int64_t>(a.Hkv) * (a.T / chunk_tokens(g) + static_cast<int64_t>(a.S) + 1);
}

// Places for tiles when keys are shared out (a few rounds of the grid).
int part_places(int nsm) { return 2 * nsm; }

// Tiles whose keys are shared out, at most: chunk_part_len cuts the work into
// `places` pieces, and each of fewer than `places` work tiles adds at most one.
int64_t max_parts(const PagedArgs &a, int nsm)
{
    const int64_t places = part_places(nsm), items = max_items(a);
    return places + (items < places ? items : places);
}

template <int D, int DT>
clis_status_t launch_impl(const ChunkParams &p, int nsm, cudaStream_t stream)
{
    using C = Cfg<D>;
    const PagedArgs &a = p.a;
    if (cudaFuncSetAttribute(paged_chunk_kernel<D, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
        return CLIS_ERR_CUDA;
    const size_t sched_smem = sizeof(int) * (static_cast<size_t>(a.S) + 1);
    if (sched_smem > 48 * 1024 &&
        cudaFuncSetAttribute(paged_chunk_schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sched_smem)) != cudaSuccess)
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
    paged_chunk_schedule_kernel<<<1, kSchedThreads, sched_smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    const int64_t tiles = max_items(a) + max_parts(a, nsm);
    const int grid = static_cast<int>(tiles < nsm ? tiles : nsm);
    paged_chunk_kernel<D, DT><<<grid, kThreads, C::SMEM_BYTES, stream>>>(mq, mk, mv, p);
    if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    paged_chunk_join_kernel<D, DT><<<dim3(static_cast<unsigned>(max_parts(a, nsm)), 8), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace

size_t paged_chunk_workspace(const PagedArgs &a, int nsm)
{
    const size_t parts = static_cast<size_t>(max_parts(a, nsm));
    return 256 + up256(static_cast<size_t>(max_items(a) + max_parts(a, nsm)) * sizeof(ChunkTile)) +
           up256(parts * 2 * BM * sizeof(float2)) + up256(parts * 2 * BM * a.d * sizeof(float));
}

clis_status_t launch_paged_chunk(const PagedArgs &a, int rows_small, void *workspace, int nsm, cudaStream_t stream)
{
    ChunkParams p;
    p.a = a;
    p.g = a.H / a.Hkv;
    p.tpt = BM / p.g;
    p.rows_small = rows_small;
    p.slots = part_places(nsm);
    p.least = 4;
    p.box_rows = imin(1 << a.page_shift, BN);
    char *w = static_cast<char *>(workspace);
    p.count = reinterpret_cast<int *>(w);
    w += 256;
    p.tiles = reinterpret_cast<ChunkTile *>(w);
    const size_t parts = static_cast<size_t>(max_parts(a, nsm));
    w += up256(static_cast<size_t>(max_items(a) + max_parts(a, nsm)) * sizeof(ChunkTile));
    p.part_ml = reinterpret_cast<float2 *>(w);
    w += up256(parts * 2 * BM * sizeof(float2));
    p.part_o = reinterpret_cast<float *>(w);
    const bool f16 = a.dtype == CLIS_DT_FP16;
    if (a.d == 128) return f16 ? launch_impl<128, 1>(p, nsm, stream) : launch_impl<128, 0>(p, nsm, stream);
    return f16 ? launch_impl<64, 1>(p, nsm, stream) : launch_impl<64, 0>(p, nsm, stream);
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
