// beam.cu -- the next beams of a beam search: of each request's W * V continuations
// (beam w, token v) the K best by
//
//   score_w + logit_wv - log sum_u e^(logit_wu),
//
// best first, ties to the lowest w * V + v.
//
// Bound: the logits' bytes, read once (96 requests of 8 beams, 128,000 tokens, bf16, a fifth of the
// beams not in use: 47 us, of which the second kernel 11; 23 by the copy rate.  8 requests of 4 beams and
// 32,003 tokens: 12.4 us, two dependent launches).  A row is cut into chunks of 512 logits.  The
// first kernel leaves each chunk's largest logit and the row's maximum and sum.  At most K
// chunks can hold one of the K best: those whose largest logit leads to the K best such
// values, so the second kernel (a block per request) picks them, reads them again (a
// few KB, still in L2) and picks the K best of what they hold:
//
//  * Mostly no pick has to be exact but the last.  The K-th largest of 64 (K above 16: 256) groups'
//    leaders is no more than the K-th best value; chunks and then logits below it are left out,
//    which leaves little more than K candidates, and each counts those that are better.  Where many
//    are left (few chunks), a second such bound comes from groups of the logits themselves; where that
//    does not do either (ties), warps sort candidates 32 at a time and merge their lists in a tree.
//    Either way the order is exactly that of (value, index).  (Without the second bound 37 requests
//    of 7 beams and 2,397 tokens took 35 us, now 19; with 64 groups for all K 8 requests of 4 beams
//    and K = 64 took 87, now 38.  K rounds of a maximum over the block took 38 us for 96
//    requests of 8 beams and K = 16.)
//  * A value is a pair of fp32 numbers (their sum, to 48 bits): exact sums of score, logit and
//    the logarithm, which comes from 32-bit terms: off by 2^-22 each, their sums of up to 2^18 by
//    2^-19 at most, 4e-6 in all (measured: 3e-7 at most, from 1,000 to 4,000,037 normal logits of
//    deviations 0 to 20).  fp64 is a fiftieth of fp32's rate here: with doubles the picks took 28 us
//    for 8 requests of 4 beams and K = 8.  Within a beam the order is that of the logits, but for
//    those that differ by less than the 48 bits, which tie.
//  * Sums are taken in an order that depends on the places in the row alone, not on the
//    row's alignment: equal rows have equal sums, and ties between beams stay ties.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "clis_internal.h"
#include "paged_internal.h"
#include "sm103_ptx.cuh"

namespace clis {
namespace {

constexpr int kChunk = 512, kPer = kChunk / 32;  // logits of a chunk, of a lane
constexpr int kScanThreads = 256, kScanWarps = kScanThreads / 32;
// Chunks of a segment, on their way at a time, and blocks of an SM (registers).
constexpr int max_seg(int dtype) { return dtype == 2 ? 1 : 2; }
constexpr int scan_blocks(bool aligned) { return aligned ? 4 : 3; }
constexpr int kMaxListed = 8192; // rows
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;
constexpr int kGroups = 256;        // for the bounds, at most
constexpr int kFew = 128;           // candidates that are ranked at once
constexpr int kPool = kPickThreads; // candidates that are ranked by counting
constexpr int kAhead = 4;             // leaders of a thread that are loaded at once
constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
    BeamArgs a;
    int chunks;     // of a row
    int seg;        // chunks of a segment
    int segs;       // segments of a row
    bool listed;    // runs of segments of the beams in use; else a warp per segment
    float *lead;    // [R * W][chunks] largest logit
    float2 *part;   // [R * W][segs] maximum and sum
};

__device__ __forceinline__ float logit(const void *row, int dtype, int64_t i)
{
    if (dtype == 2) return __ldg(static_cast<const float *>(row) + i);
    const uint32_t u = __ldg(static_cast<const unsigned short *>(row) + i);
    return dtype == CLIS_DT_BF16 ? elem_lo<0>(u) : elem_lo<1>(u);
}

// Place in a chunk of a lane's e-th logit, rising with e: 16 bytes at a time.
template <int DT>
__device__ __forceinline__ int place(int lane, int e)
{
    constexpr int N = DT == 2 ? 4 : 8;
    return (e / N) * (32 * N) + lane * N + e % N;
}

// Four words from the 16 bytes at `lo` and the following ones at `hi`, WS words and
// (HALF) two bytes on.
template <int WS, bool HALF>
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi)
{
    const uint32_t w[9] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w, 0u};
    uint4 r;
    r.x = HALF ? __funnelshift_r(w[WS], w[WS + 1], 16) : w[WS];
    r.y = HALF ? __funnelshift_r(w[WS + 1], w[WS + 2], 16) : w[WS + 1];
    r.z = HALF ? __funnelshift_r(w[WS + 2], w[WS + 3], 16) : w[WS + 2];
    r.w = HALF ? __funnelshift_r(w[WS + 3], w[WS + 4], 16) : w[WS + 3];
    return r;
}

__device__ __forceinline__ uint4 shifted_by(const uint4 &lo, const uint4 &hi, int bytes)
{
    switch (bytes >> 1) {  // (uniform in a row)
    case 0: return lo;
    case 1: return shifted<0, true>(lo, hi);
    case 2: return shifted<1, false>(lo, hi);
    case 3: return shifted<1, true>(lo, hi);
    case 4: return shifted<2, false>(lo, hi);
    case 5: return shifted<2, true>(lo, hi);
    case 6: return shifted<3, false>(lo, hi);
    default: return shifted<3, true>(lo, hi);
    }
}

// Logits that are read once (without a place in L1: 2 us less for 96 requests of 8 beams).
__device__ __forceinline__ uint4 ldg_stream(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// What a lane loads of a chunk: its logits (the e-th at place(lane, e)) as they lie in
// memory.  A row that is not 16-byte aligned is read in aligned pieces, each lane two
// neighbouring ones; its first and last chunk one logit at a time, so that nothing outside
// of the row is touched.
template <int DT, bool ALIGNED>
struct Raw {
    static constexpr int SIZE = DT == 2 ? 4 : 2, N = 16 / SIZE, P = kPer / N;
    uint4 v[P], u[ALIGNED ? 1 : P];
    bool whole;

    __device__ __forceinline__ void load(const void *row, int64_t first, int V, int lane)
    {
        const int off = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
        whole = off == 0 ? first + kChunk <= V : first > 0 && first + kChunk + N <= V;
        if (!whole) return;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + first * SIZE - off);
#pragma unroll
        for (int j = 0; j < P; j++) v[j] = ldg_stream(src + j * 32 + lane);
        if (!ALIGNED && off != 0)
#pragma unroll
            for (int j = 0; j < P; j++) u[ALIGNED ? 0 : j] = __ldg(src + j * 32 + lane + 1);
    }
    // The logits; -inf behind the row's end.
    __device__ __forceinline__ void values(const void *row, int64_t first, int V, int lane, float *x) const
    {
        if (!whole) {
#pragma unroll
            for (int e = 0; e < kPer; e++) {
                const int64_t i = first + place<DT>(lane, e);
                x[e] = i < V ? logit(row, DT, i) : -INFINITY;
            }
            return;
        }
        const int off = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
#pragma unroll
        for (int j = 0; j < P; j++) {
            const uint4 y = ALIGNED ? v[j] : shifted_by(v[j], u[ALIGNED ? 0 : j], off);
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if constexpr (DT == 2) {
                    x[j * N + e] = __uint_as_float(w[e]);
                } else {
                    x[j * N + 2 * e] = elem_lo<DT>(w[e]);
                    x[j * N + 2 * e + 1] = elem_hi<DT>(w[e]);
                }
            }
        }
    }
};

// Floats as unsigned numbers of the same order.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t u)
{
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// Two running (maximum, sum of 2^((x - maximum) log2 e)) as one.
__device__ __forceinline__ void merge(float &m, float &s, float m1, float s1)
{
    const float mm = fmaxf(m, m1);
    if (mm == -INFINITY) {  // (no logit above -inf; the sums are 0, or no number)
        s += s1;
        return;
    }
    s = s * ex2_approx((m - mm) * kLog2e) + s1 * ex2_approx((m1 - mm) * kLog2e);
    m = mm;
}

// The rows of beams in use, in order, in s_rows; returns their number.
__device__ __forceinline__ int list_rows(const float *scores, int rows, uint16_t *s_rows, uint32_t *s_mask, int *s_sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, words = (rows + 31) / 32;
    for (int j = warp; j < words; j += kScanWarps) {
        const int r = j * 32 + lane;
        const uint32_t mask = __ballot_sync(~0u, r < rows && isfinite(__ldg(scores + min(r, rows - 1))));
        if (lane == 0) s_mask[j] = mask;
    }
    __syncthreads();
    static_assert(kMaxListed / 32 <= kScanThreads, "a thread per word");
    const int n = threadIdx.x < words ? __popc(s_mask[threadIdx.x]) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int at = incl - n, total = 0;
    for (int i = 0; i < kScanWarps; i++) {
        if (i < warp) at += s_sum[i];
        total += s_sum[i];
    }
    if (threadIdx.x < words)
        for (uint32_t mask = s_mask[threadIdx.x]; mask; mask &= mask - 1) s_rows[at++] = static_cast<uint16_t>(threadIdx.x * 32 + __ffs(mask) - 1);
    __syncthreads();
    return total;
}

// A warp reads segments of one or two chunks, the next one's chunks on their way as those of the one
// at hand have been looked at, also from row to row: runs of segments of the beams in use,
// as many for each warp (few logits: a warp per segment).  A block per 128 chunks of a row,
// which began and ended without loads on their way, took 5 us more for 96 requests of 8 beams;
// segments of four chunks with three blocks an SM 1.5, two blocks an SM 10: it is warps that hide
// a chunk's chain of instructions.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kScanThreads, scan_blocks(ALIGNED)) beam_scan_kernel(const BeamParams p)
{
    const BeamArgs &a = p.a;
    __shared__ uint16_t s_rows[kMaxListed];
    __shared__ uint32_t s_mask[kMaxListed / 32];
    __shared__ int s_sum[kScanWarps];
    const int lane = threadIdx.x & 31, worker = blockIdx.x * kScanWarps + (threadIdx.x >> 5), rows = a.R * a.W;
    pdl_launch();
    int64_t u = worker;  // its first segment
    int left = 1;        // and how many
    const bool list = p.listed && rows <= kMaxListed;  // (else those of beams not in use are read as well)
    if (p.listed) {
        const int64_t n = static_cast<int64_t>(list ? list_rows(a.scores, rows, s_rows, s_mask, s_sum) : rows) * p.segs;
        const int workers = gridDim.x * kScanWarps;
        u = n * worker / workers;
        left = static_cast<int>(n * (worker + 1) / workers - u);
    }
    if (left <= 0 || (!p.listed && u >= static_cast<int64_t>(rows) * p.segs)) return;
    int rank = static_cast<int>(u / p.segs), c = static_cast<int>(u - static_cast<int64_t>(rank) * p.segs) * p.seg;  // its first chunk
    int r = list ? s_rows[rank] : rank;
    auto row_of = [&](int i) {
        const int req = i / a.W, w = i - req * a.W;
        return static_cast<const uint8_t *>(a.logits) + (req * a.l_sr + w * a.l_sw) * (DT == 2 ? 4 : 2);
    };
    const uint8_t *row = row_of(r);
    constexpr int B = max_seg(DT);
    Raw<DT, ALIGNED> raw[B];
#pragma unroll
    for (int b = 0; b < B; b++)
        if (b < p.seg && c + b < p.chunks) raw[b].load(row, static_cast<int64_t>(c + b) * kChunk, a.V, lane);
    if (!p.listed && !isfinite(__ldg(a.scores + r))) return;  // a beam not in use (known only now: the loads do not wait for it)
    while (true) {
        // the segment after this one
        const uint8_t *row1 = row;
        int r1 = r, c1 = c + p.seg;
        if (left > 1 && c1 >= p.chunks) {
            rank++;
            r1 = list ? s_rows[rank] : rank;
            row1 = row_of(r1);
            c1 = 0;
        }
        float m = -INFINITY, s = 0.f;  // the segment's maximum, the lane's sum
#pragma unroll
        for (int b = 0; b < B; b++) {
            if (b >= p.seg) continue;
            float x[kPer];
            const bool has = c + b < p.chunks;
            if (has) raw[b].values(row, static_cast<int64_t>(c + b) * kChunk, a.V, lane, x);
            if (left > 1 && c1 + b < p.chunks) raw[b].load(row1, static_cast<int64_t>(c1 + b) * kChunk, a.V, lane);
            if (!has) continue;
            float mx = fmaxf(x[0], x[1]);  // (a NaN is left to the sum)
#pragma unroll
            for (int e = 2; e < kPer; e += 2) mx = fmax3(mx, x[e], x[e + 1]);
            mx = from_ordered(__reduce_max_sync(~0u, ordered(mx)));
            if (lane == 0) p.lead[static_cast<int64_t>(r) * p.chunks + c + b] = mx;
            if (mx > m) {
                s *= ex2_approx((m - mx) * kLog2e);
                m = mx;
            }
            const float base = m == -INFINITY ? 0.f : -m;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const float2 d = fmul2(fadd2(make_float2(x[e], x[e + 1]), make_float2(base, base)), make_float2(kLog2e, kLog2e));
                sum = fadd2(sum, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
            }
            s += sum.x + sum.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) p.part[static_cast<int64_t>(r) * p.segs + c / p.seg] = make_float2(m, s);
        if (--left == 0) break;
        r = r1;
        c = c1;
        row = row1;
    }
}

// hi + lo, exact sums of two numbers and of such pairs (to 48 bits).
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}

__device__ __forceinline__ Pair plus(const Pair &a, float b)
{
    const Pair t = two_sum(a.hi, b);
    const float e = __fadd_rn(t.lo, a.lo), s = __fadd_rn(t.hi, e);
    return {s, __fsub_rn(e, __fsub_rn(s, t.hi))};
}

// m + log(s), s a positive number: s = f 2^k with f in [0.7, 1.42), so that logf(f) is off by
// little, and k log 2 as a pair.
__device__ __forceinline__ Pair log_sum(float m, float s)
{
    int k = static_cast<int>(__float_as_uint(s) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(s) & 0x7FFFFFu) | 0x3F800000u);  // (sums are normal numbers)
    if (f > 1.41421356f) {
        f *= 0.5f;
        k++;
    }
    const float ln2 = 0.693147182f, rest = -1.90465429e-9f;  // log 2 - ln2
    const float x = static_cast<float>(k), p = __fmul_rn(x, ln2);
    const Pair t = plus(two_sum(m, p), __fmaf_rn(x, ln2, -p));
    return plus(t, __fmaf_rn(x, rest, logf(f)));
}

// score + (x - lse)
__device__ __forceinline__ Pair value(float score, float x, const Pair &lse)
{
    const Pair t = plus({-lse.hi, -lse.lo}, x);
    return plus(t, score);
}

// A candidate: its value as an unsigned number of the same order (0: none), and its place.
struct Best {
    uint64_t v;
    uint32_t at;
};

__device__ __forceinline__ Best no_one() { return {0ull, ~0u}; }

__device__ __forceinline__ Best best_of(const Pair &v, uint32_t at)
{
    // (no -0)
    return {isfinite(v.hi) ? static_cast<uint64_t>(ordered(v.hi + 0.f)) << 32 | ordered(v.lo + 0.f) : 0ull, at};
}

__device__ __forceinline__ bool better(const Best &a, const Best &b) { return a.v > b.v || (a.v == b.v && a.at < b.at); }
__device__ __forceinline__ Best from_lane(const Best &b, int l) { return {__shfl_sync(~0u, b.v, l), __shfl_sync(~0u, b.at, l)}; }

// One comparison of a sorting network: lanes whose bit o is clear keep the better one
// (down), or the worse.
__device__ __forceinline__ void exchange(Best &b, int o, bool down, int lane)
{
    const Best x = {__shfl_xor_sync(~0u, b.v, o), __shfl_xor_sync(~0u, b.at, o)};
    if (better(x, b) == (((lane & o) == 0) == down)) b = x;
}

// A bitonic sequence of 32, best first.  (Loops, not unrolled: a kernel this short waits for
// its instructions.)
__device__ __forceinline__ void sort_bitonic(Best &b, int lane)
{
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) exchange(b, o, true, lane);
}

__device__ __forceinline__ void sort32(Best &b, int lane)
{
#pragma unroll 1
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll 1
        for (int o = n / 2; o > 0; o >>= 1) exchange(b, o, (lane & n) == 0, lane);
}

// The K best of what a warp has seen, best first: lane i has the i-th and, where K is
// beyond 32, the (32 + i)-th.
struct Top {
    Best b[2];
    int K;

    // 32 sorted candidates join.
    __device__ __forceinline__ void join(const Best &sorted, int lane)
    {
        Best x = from_lane(sorted, 31 - lane);
        const bool take = better(x, b[0]);
        Best rest = take ? b[0] : x;
        if (take) b[0] = x;
        sort_bitonic(b[0], lane);
        if (K <= 32) return;
        sort_bitonic(rest, lane);
        x = from_lane(rest, 31 - lane);
        if (better(x, b[1])) b[1] = x;
        sort_bitonic(b[1], lane);
    }
    __device__ __forceinline__ void add(Best x, int lane)
    {
        // (nothing to do where no candidate is better than the K-th)
        const Best worst = K <= 32 ? from_lane(b[0], K - 1) : from_lane(b[1], K - 33);
        if (!__any_sync(~0u, better(x, worst))) return;
        sort32(x, lane);
        join(x, lane);
    }
};

// The lists of the block's first n warps (all threads call) become the first warp's.
__device__ __forceinline__ void join_warps(Top &top, int n, Best (*lists)[64])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = 1; d < n; d *= 2) {
        if (warp < n && (warp & (2 * d - 1)) == d) {
            lists[warp][lane] = top.b[0];
            if (top.K > 32) lists[warp][32 + lane] = top.b[1];
        }
        __syncthreads();
        if ((warp & (2 * d - 1)) == 0 && warp + d < n) {
            top.join(lists[warp + d][lane], lane);
            if (top.K > 32) top.join(lists[warp + d][32 + lane], lane);
        }
    }
}

struct Outputs {
    const BeamArgs &a;
    int64_t first;
    __device__ __forceinline__ void put(int k, const Best &b) const
    {
        const bool gone = b.v == 0;
        a.out_scores[first + k] = gone ? -INFINITY : from_ordered(static_cast<uint32_t>(b.v >> 32));
        a.parent[first + k] = gone ? -1 : static_cast<int>(b.at / static_cast<uint32_t>(a.V));
        a.token[first + k] = gone ? -1 : static_cast<int>(b.at % static_cast<uint32_t>(a.V));
    }
};

// The K-th largest of N groups (1: there are fewer); the block's first N threads take part.
template <int N>
__device__ __forceinline__ void kth_group(const uint32_t *group, int K, uint32_t *bound)
{
    const int tid = threadIdx.x;
    if (tid >= N) return;
    const uint32_t mine = group[tid];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < N; j += 4) {
        const uint4 g = *reinterpret_cast<const uint4 *>(group + j);
        rank += g.x > mine || (g.x == mine && j < tid);
        rank += g.y > mine || (g.y == mine && j + 1 < tid);
        rank += g.z > mine || (g.z == mine && j + 2 < tid);
        rank += g.w > mine || (g.w == mine && j + 3 < tid);
    }
    if (rank == K - 1) *bound = max(mine, 1u);
}

template <int DT>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamParams p)
{
    const BeamArgs &a = p.a;
    __shared__ Best s_lists[kPickWarps][64];
    __shared__ float s_score[kMaxBeams];
    __shared__ Pair s_lse[kMaxBeams];
    __shared__ bool s_ok[kMaxBeams];
    __shared__ Best s_pick[kMaxPicks];  // at: beam * chunks + chunk
    __shared__ __align__(16) uint32_t s_group[kGroups];
    __shared__ uint32_t s_bound;
    __shared__ int s_chunks, s_cands, s_chunk[kPool];
    Best *pool = &s_lists[0][0];  // [kPool]
    static_assert(kPool <= kPickWarps * 64, "the pool lies in the lists' place");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int req = blockIdx.x;
    const int groups = a.K <= 16 ? 64 : kGroups;  // of leaders (more take longer to rank)
    if (tid < kGroups) s_group[tid] = 0;
    if (tid == 0) s_chunks = s_cands = 0;
    pdl_wait();
    const int leads = a.W * p.chunks;
    const float *lead = p.lead + static_cast<int64_t>(req) * leads;
    const Outputs out{a, static_cast<int64_t>(req) * a.K};
    float ahead[kAhead];  // this thread's first leaders, beside the rows' sums (a beam not in use may hold anything)
#pragma unroll
    for (int j = 0; j < kAhead; j++) ahead[j] = tid + j * kPickThreads < leads ? lead[tid + j * kPickThreads] : 0.f;

    // ---- the rows' logarithms, in the order of the segments
    for (int w = warp; w < a.W; w += kPickWarps) {
        const int r = req * a.W + w;
        const float score = __ldg(a.scores + r);
        float m = -INFINITY, s = 0.f;
        for (int i0 = 0; i0 < p.segs; i0 += 32 * kAhead) {
            float2 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                const int i = i0 + j * 32 + lane;
                v[j] = i < p.segs ? p.part[static_cast<int64_t>(r) * p.segs + i] : make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kAhead; j++) merge(m, s, v[j].x, v[j].y);
        }
        bool ok = isfinite(score);
        if (ok) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float m1 = __shfl_down_sync(~0u, m, o), s1 = __shfl_down_sync(~0u, s, o);
                merge(m, s, m1, s1);
            }
            m = __shfl_sync(~0u, m, 0);
            s = __shfl_sync(~0u, s, 0);
            ok = isfinite(m) && isfinite(s) && s > 0.f;
        }
        if (lane == 0) {
            s_ok[w] = ok;
            s_score[w] = score;
            s_lse[w] = ok ? log_sum(m, s) : Pair{0.f, 0.f};
        }
    }
    __syncthreads();

    // The value of a chunk's leader as an unsigned number of its order (0: none).
    auto leader = [&](int i, float x) -> Best {
        const int w = i / p.chunks;
        return s_ok[w] && x != -INFINITY ? best_of(value(s_score[w], x, s_lse[w]), static_cast<uint32_t>(i)) : no_one();
    };
    // A quarter of a chunk: this lane's kChunk / 128 logits, their places w * V + v from `at` on in steps of 32.
    constexpr int E = kChunk / 128;
    auto quarter = [&](int chunk, int q, float *x, int &w, uint32_t &at) {
        w = chunk / p.chunks;
        const int64_t first = static_cast<int64_t>(chunk - w * p.chunks) * kChunk + q * 128 + lane;
        const void *row = static_cast<const uint8_t *>(a.logits) + (req * a.l_sr + w * a.l_sw) * (DT == 2 ? 4 : 2);
#pragma unroll
        for (int e = 0; e < E; e++) x[e] = first + e * 32 < a.V ? logit(row, DT, first + e * 32) : -INFINITY;
        at = static_cast<uint32_t>(static_cast<int64_t>(w) * a.V + first);
    };

    // The K best of n candidates, each by the number of those that are better.
    auto rank_pool = [&](int n) {
        const Best mine = tid < n ? pool[tid] : no_one();
        if (tid < n) {
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; j++) rank += better(pool[j], mine);
            if (rank < a.K) out.put(rank, mine);
        }
        if (tid >= n && tid < a.K) out.put(tid, no_one());
    };

    // ---- the bound, the chunks that reach it, the logits that do
    uint32_t first[kAhead];  // the first leaders' values
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
        const int i = tid + j * kPickThreads;
        first[j] = i < leads ? static_cast<uint32_t>(leader(i, ahead[j]).v >> 32) : 0u;
        if (first[j]) atomicMax(&s_group[i & (groups - 1)], first[j]);
    }
#pragma unroll 1
    for (int i = tid + kAhead * kPickThreads; i < leads; i += kPickThreads)
        atomicMax(&s_group[i & (groups - 1)], static_cast<uint32_t>(leader(i, lead[i]).v >> 32));
    __syncthreads();
    if (groups == 64) kth_group<64>(s_group, a.K, &s_bound);
    else kth_group<kGroups>(s_group, a.K, &s_bound);
    __syncthreads();
    uint32_t bound = s_bound;
    auto found_one = [&](int i) {
        const int k = atomicAdd(&s_chunks, 1);
        if (k < kPool) s_chunk[k] = i;
    };
#pragma unroll
    for (int j = 0; j < kAhead; j++)
        if (first[j] >= bound) found_one(tid + j * kPickThreads);
#pragma unroll 1
    for (int i = tid + kAhead * kPickThreads; i < leads; i += kPickThreads)
        if ((leader(i, lead[i]).v >> 32) >= bound) found_one(i);
    __syncthreads();
    const int found = s_chunks;
    if (found <= kPool) {
#pragma unroll 1
        for (int t = warp; t < 4 * found; t += kAhead * kPickWarps) {
            float x[kAhead][E];  // four quarters on their way
            int w[kAhead];
            uint32_t at[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                const int u = t + j * kPickWarps;
                if (u < 4 * found) quarter(s_chunk[u >> 2], u & 3, x[j], w[j], at[j]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                if (t + j * kPickWarps >= 4 * found) break;
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const Best b = x[j][e] == -INFINITY ? no_one() : best_of(value(s_score[w[j]], x[j][e], s_lse[w[j]]), at[j] + e * 32);
                    if ((b.v >> 32) < bound) continue;
                    const int k = atomicAdd(&s_cands, 1);
                    if (k < kPool) pool[k] = b;
                }
            }
            if (s_cands > kPool) break;  // (only to save time: looked at again below)
        }
        __syncthreads();
        const int n = s_cands;
        if (n <= kFew) {
            rank_pool(n);
            return;
        }
    }
    __syncthreads();  // (s_cands and the pool's place are written again)

    // ---- many logits reach it (leaders are few in a small vocabulary): the K-th largest of 128 groups
    // of those logits is the next bound
    if (found <= kPool) {
        auto logits = [&](auto use) {
#pragma unroll 1
            for (int t = warp; t < 4 * found; t += kPickWarps) {
                float x[E];
                int w;
                uint32_t at;
                quarter(s_chunk[t >> 2], t & 3, x, w, at);
#pragma unroll
                for (int e = 0; e < E; e++)
                    if (x[e] != -INFINITY) use(best_of(value(s_score[w], x[e], s_lse[w]), at + e * 32));
            }
        };
        uint32_t top = 0;
        logits([&](const Best &b) { top = max(top, static_cast<uint32_t>(b.v >> 32)); });
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        static_assert(kPickThreads / 4 <= kGroups, "a group for four threads");
        if ((tid & 3) == 0) s_group[tid >> 2] = top;
        if (tid == 0) s_cands = 0;
        __syncthreads();
        kth_group<kPickThreads / 4>(s_group, a.K, &s_bound);
        __syncthreads();
        bound = max(bound, s_bound);
        logits([&](const Best &b) {
            if ((b.v >> 32) < bound || *static_cast<volatile int *>(&s_cands) > kPool) return;
            const int k = atomicAdd(&s_cands, 1);
            if (k < kPool) pool[k] = b;
        });
        __syncthreads();
        const int n = s_cands;
        if (n <= kPool) {
            rank_pool(n);
            return;
        }
        __syncthreads();  // (the pool's place is written again)
    }

    // ---- the other way: the K best leaders, exactly
    Top top;
    top.K = a.K;
    top.b[0] = top.b[1] = no_one();
#pragma unroll 1
    for (int i0 = warp * 32; i0 < leads; i0 += kPickThreads) top.add(i0 + lane < leads ? leader(i0 + lane, lead[i0 + lane]) : no_one(), lane);
    join_warps(top, min((leads + 31) / 32, kPickWarps), s_lists);
    if (warp == 0) {
        if (lane < a.K) s_pick[lane] = top.b[0];
        if (32 + lane < a.K) s_pick[32 + lane] = top.b[1];
    }
    __syncthreads();

    // ---- what they hold, no worse than the last of their leaders: quarters of chunks
    int picks = 0;
    while (picks < a.K && s_pick[picks].v != 0) picks++;
    const Best last = picks == a.K ? s_pick[picks - 1] : no_one();
    top.b[0] = top.b[1] = no_one();
#pragma unroll 1
    for (int t = warp; t < 4 * picks; t += kPickWarps) {
        float x[E];
        int w;
        uint32_t at;
        quarter(static_cast<int>(s_pick[t >> 2].at), t & 3, x, w, at);
#pragma unroll 1
        for (int e = 0; e < E; e++) {
            Best b = x[0] == -INFINITY ? no_one() : best_of(value(s_score[w], x[0], s_lse[w]), at + e * 32);
            if (b.v < last.v) b = no_one();
            top.add(b, lane);
#pragma unroll
            for (int i = 1; i < E; i++) x[i - 1] = x[i];
        }
    }
    join_warps(top, min(4 * picks, kPickWarps), s_lists);
    if (warp > 0) return;
    if (lane < a.K) out.put(lane, top.b[0]);
    if (32 + lane < a.K) out.put(32 + lane, top.b[1]);
}

int chunks_of(const BeamArgs &a) { return (a.V + kChunk - 1) / kChunk; }

// Segments of one chunk and a warp for each while the GPU holds them all.
void plan(const BeamArgs &a, int nsm, BeamParams &p)
{
    p.a = a;
    p.chunks = chunks_of(a);
    const int64_t rows = static_cast<int64_t>(a.R) * a.W, workers = static_cast<int64_t>(scan_blocks(false)) * nsm * kScanWarps;
    p.listed = rows * p.chunks > workers;
    p.seg = p.listed ? max_seg(a.dtype) : 1;
    p.segs = (p.chunks + p.seg - 1) / p.seg;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <int DT, bool ALIGNED>
cudaError_t launch_impl(const BeamParams &p, int nsm, cudaStream_t stream)
{
    const int64_t units = static_cast<int64_t>(p.a.R) * p.a.W * p.segs, blocks = (units + kScanWarps - 1) / kScanWarps, most = scan_blocks(ALIGNED) * nsm;
    beam_scan_kernel<DT, ALIGNED><<<static_cast<unsigned>(blocks < most ? blocks : most), kScanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_pick_kernel<DT>, dim3(p.a.R), kPickThreads, 0, stream, p);
}

template <int DT>
cudaError_t launch_type(const BeamParams &p, bool aligned, int nsm, cudaStream_t stream)
{
    return aligned ? launch_impl<DT, true>(p, nsm, stream) : launch_impl<DT, false>(p, nsm, stream);
}

}  // namespace

size_t beam_workspace(const BeamArgs &a, int nsm)
{
    BeamParams p;
    plan(a, nsm, p);
    const size_t rows = static_cast<size_t>(a.R) * a.W;
    return up256(rows * p.chunks * sizeof(float)) + up256(rows * p.segs * sizeof(float2));
}

clis_status_t launch_beam(const BeamArgs &a, void *workspace, int nsm, cudaStream_t stream)
{
    BeamParams p;
    const int64_t size = a.dtype == 2 ? 4 : 2;
    const bool aligned = !((reinterpret_cast<uintptr_t>(a.logits) | a.l_sr * size | a.l_sw * size) & 15);
    plan(a, nsm, p);
    const size_t rows = static_cast<size_t>(a.R) * a.W;
    p.lead = static_cast<float *>(workspace);
    p.part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + up256(rows * p.chunks * sizeof(float)));
    const cudaError_t e = a.dtype == CLIS_DT_BF16 ? launch_type<CLIS_DT_BF16>(p, aligned, nsm, stream)
                          : a.dtype == CLIS_DT_FP16 ? launch_type<CLIS_DT_FP16>(p, aligned, nsm, stream)
                                                    : launch_type<2>(p, aligned, nsm, stream);
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
