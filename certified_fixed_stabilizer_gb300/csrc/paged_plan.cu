// paged_plan.cu -- the plan of one serving step over a paged key/value cache,
// from the lengths of its requests: prefix sums of the new tokens, pages taken
// from (and given back to) a ring of free pages, block tables completed, and
// every new token's slot and position.
//
// All results are whole numbers and none depends on the order in which blocks
// run: the i-th page taken, counted over the sequences in order, is the i-th of
// the ring from its head on, so three exclusive prefix sums (tokens, pages
// taken, pages given back) say everything.  Bound: launch latency for a few
// requests, then the 12 bytes written per token.  One launch: every block
// computes the sums of all sequences for itself (16 bytes a sequence from L2;
// cheaper than a second launch) and then takes its share of the tokens, of the
// pages taken and of the pages given back.
#include <cuda_runtime.h>

#include "clis_internal.h"
#include "paged_internal.h"

namespace clis {

__device__ unsigned int g_plan_error_word = 0;

namespace {

constexpr int kPlanThreads = 512;
// Sums saturate here, so that lengths beyond any sense cannot wrap around.
constexpr uint32_t kCap = (1u << 31) - 1;  // (beyond any number of rows)

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }  // a, b <= kCap

struct Sums {
    uint32_t tok, taken, back;
};

__device__ __forceinline__ Sums add(const Sums &a, const Sums &b)
{
    return {sat_add(a.tok, b.tok), sat_add(a.taken, b.taken), sat_add(a.back, b.back)};
}

// Lengths of one sequence.  The cached one is brought into the range a block-table row
// can hold; the new tokens are counted as given, because their rows are in the packed
// batch whether they can be served or not.
struct Seq {
    int ctx, n, have, need;  // have, need: pages held and pages wanted
    bool gone;
    bool full;  // the block-table row cannot hold it: not served, takes no page
};

__device__ __forceinline__ Seq read_seq(const PlanArgs &a, int s)
{
    Seq q;
    const int cap = a.width << a.page_shift;
    const int mask = (1 << a.page_shift) - 1;
    const int c = __ldg(a.ctx_len + s), n = __ldg(a.new_len + s);
    q.gone = n < 0;
    q.ctx = min(max(c, 0), cap);
    q.n = q.gone ? 0 : n;
    q.full = c != q.ctx || q.n > cap - q.ctx;
    q.have = (q.ctx >> a.page_shift) + ((q.ctx & mask) ? 1 : 0);
    const int total = q.full ? q.ctx : q.ctx + q.n;
    q.need = (total >> a.page_shift) + ((total & mask) ? 1 : 0);
    return q;
}

__device__ __forceinline__ Sums sums_of(const Seq &q)
{
    return {min(static_cast<uint32_t>(q.n), kCap), static_cast<uint32_t>(q.need - q.have),
            q.gone ? static_cast<uint32_t>(q.have) : 0u};
}

// Last s with first[s] <= i, for i < first[S] (first is non-decreasing).
__device__ __forceinline__ int find(const uint32_t *first, int S, uint32_t i)
{
    int lo = 0, hi = S;  // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs a)
{
    extern __shared__ uint32_t sm[];
    uint32_t *s_tok = sm, *s_taken = sm + (a.S + 1), *s_back = sm + 2 * (a.S + 1);
    __shared__ Sums s_warp[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned int bad = 0;

    // Prefix sums: a run of consecutive sequences per thread, then over threads.
    const int per = (a.S + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(a.S, tid * per), s1 = min(a.S, s0 + per);
    Sums mine = {0, 0, 0};
    for (int s = s0; s < s1; s++) {
        const Seq q = read_seq(a, s);
        if (q.full) bad |= CLIS_PAGED_LENGTH_BIT;
        mine = add(mine, sums_of(q));
    }
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums up = {__shfl_up_sync(~0u, incl.tok, o), __shfl_up_sync(~0u, incl.taken, o),
                         __shfl_up_sync(~0u, incl.back, o)};
        if (lane >= o) incl = add(incl, up);
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    Sums run = {0, 0, 0};
    for (int w = 0; w < warp; w++) run = add(run, s_warp[w]);
    {
        const Sums up = {__shfl_up_sync(~0u, incl.tok, 1), __shfl_up_sync(~0u, incl.taken, 1),
                         __shfl_up_sync(~0u, incl.back, 1)};
        if (lane > 0) run = add(run, up);
    }
    for (int s = s0; s < s1; s++) {
        s_tok[s] = run.tok;
        s_taken[s] = run.taken;
        s_back[s] = run.back;
        run = add(run, sums_of(read_seq(a, s)));
    }
    // (the totals: from the thread with the last sequence, or zeros without any)
    if ((s0 < a.S && s1 == a.S) || (a.S == 0 && tid == 0)) {
        s_tok[a.S] = run.tok;
        s_taken[a.S] = run.taken;
        s_back[a.S] = run.back;
    }
    __syncthreads();
    const uint32_t tokens = s_tok[a.S], taken = s_taken[a.S], back = s_back[a.S];

    const int64_t F = a.ring_size;
    const int64_t head = a.state_in[0], tail = a.state_in[1];
    const int64_t held = tail - head;  // free pages in the ring
    if (held < 0 || held > F) bad |= CLIS_PAGED_POOL_BIT;
    const int64_t avail = held < 0 || held > F ? 0 : held;
    const uint32_t hm = static_cast<uint32_t>(((head % F) + F) % F), tm = static_cast<uint32_t>(((tail % F) + F) % F);
    const uint32_t Fu = static_cast<uint32_t>(F);
    // A sequence that the ring has too few pages for, or the batch too few rows, stays as
    // it was, and those behind it take no page either: `served` are served whatever they
    // need, the others only if they need no page and their rows are there.  One whose
    // block-table row is full stays as it was too, and is nobody else's concern: it wants
    // no page, and its rows are counted.
    int served = a.S;
    if (taken > avail) served = find(s_taken, a.S, static_cast<uint32_t>(avail));
    if (tokens > static_cast<uint32_t>(a.T)) served = min(served, find(s_tok, a.S, static_cast<uint32_t>(a.T)));
    const uint32_t used = s_taken[served];  // <= avail
    auto fits = [&](int s, const Seq &q) {
        if (q.full) return false;
        return s < served || q.n == 0 ||
               (q.need == q.have && s_tok[s] + static_cast<uint32_t>(q.n) <= static_cast<uint32_t>(a.T));
    };
    // The i-th page taken in this step, i < used.
    auto fresh = [&](uint32_t i) -> int {
        const int page = __ldg(a.ring + (hm + i) % Fu);
        if (page < 0 || page >= a.num_pages) bad |= CLIS_PAGED_INDEX_BIT;
        return page;
    };

    const uint32_t gtid = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    for (uint32_t s = gtid; s <= static_cast<uint32_t>(a.S); s += step) {
        a.cu_q[s] = min(s_tok[s], static_cast<uint32_t>(a.T));
        if (s < static_cast<uint32_t>(a.S)) {
            const Seq q = read_seq(a, s);
            a.kv_len[s] = q.gone ? 0 : fits(s, q) ? q.ctx + q.n : q.ctx;
        }
    }
    if (gtid == 0) {
        if (tokens > static_cast<uint32_t>(a.T)) bad |= CLIS_PAGED_LENGTH_BIT;
        if (taken > avail) bad |= CLIS_PAGED_POOL_BIT;
        a.state_out[0] = head + used;
        a.state_out[1] = tail + min(static_cast<int64_t>(back), F - avail);
    }
    // Pages taken go into the block tables behind the pages held.
    for (uint32_t i = gtid; i < used; i += step) {
        const int s = find(s_taken, a.S, i);
        const Seq q = read_seq(a, s);
        a.block_table[s * a.bt_s + q.have + (i - s_taken[s])] = fresh(i);
    }
    // Pages given back follow the ring's tail.  They lie outside the head ..
    // tail part that `fresh` reads, so neither waits for the other.
    for (uint32_t i = gtid; i < back; i += step) {
        const int s = find(s_back, a.S, i);
        if (avail + i >= F) {
            bad |= CLIS_PAGED_POOL_BIT;
            continue;
        }
        const int page = a.block_table[s * a.bt_s + (i - s_back[s])];
        if (page < 0 || page >= a.num_pages) bad |= CLIS_PAGED_INDEX_BIT;
        a.ring[(tm + i) % Fu] = page;
    }
    // Slots and positions; rows behind the last sequence get slot -1, position 0.
    const int mask = (1 << a.page_shift) - 1;
    for (uint32_t t = gtid; t < static_cast<uint32_t>(a.T); t += step) {
        int64_t slot = -1;
        int pos = 0;
        if (t < tokens) {
            const int s = find(s_tok, a.S, t);
            const Seq q = read_seq(a, s);
            pos = q.ctx + static_cast<int>(t - s_tok[s]);
            if (fits(s, q)) {
                const int col = pos >> a.page_shift;
                // A page held is read from the table, a page taken from the ring: this
                // launch writes the latter's table entry, the former's it leaves alone.
                const int page = col < q.have ? a.block_table[s * a.bt_s + col] : fresh(s_taken[s] + (col - q.have));
                if (page >= 0 && page < a.num_pages) slot = (static_cast<int64_t>(page) << a.page_shift) + (pos & mask);
                else bad |= CLIS_PAGED_INDEX_BIT;
            }
        }
        a.slots[t] = slot;
        a.pos[t] = pos;
    }
    if (bad) atomicOr(&g_plan_error_word, bad);
}

}  // namespace

clis_status_t launch_paged_plan(const PlanArgs &a, cudaStream_t stream)
{
    const size_t smem = 3 * sizeof(uint32_t) * (static_cast<size_t>(a.S) + 1);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return CLIS_ERR_CUDA;
    // About two tokens a thread, one block per SM at most (90,000 tokens: 8.5 us a call with
    // one or two, 10.3 with four).
    int64_t blocks = (static_cast<int64_t>(a.T) + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
    blocks = blocks < 1 ? 1 : blocks > 152 ? 152 : blocks;
    paged_plan_kernel<<<static_cast<unsigned>(blocks), kPlanThreads, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t read_plan_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_plan_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_plan_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_plan_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
