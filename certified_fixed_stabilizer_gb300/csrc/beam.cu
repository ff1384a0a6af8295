// beam.cu -- the next beams of a beam search: of each request's W * V continuations
// (beam w, token v) the K best by
//
//   score_w + logit_wv - log sum_u e^(logit_wu),
//
// best first, ties to the lowest w * V + v.
//
// Bound: the logits' bytes, read once.  A row is cut into chunks of 512 logits.  The
// first kernel leaves each chunk's largest logit and the row's maximum and sum.  At most K
// chunks can hold one of the K best: those whose largest logit leads to the K best such
// values, so the second kernel (a block per request) picks them, reads them again (a
// few KB, still in L2) and picks the K best of what they hold.  Either pick is K rounds of
// a maximum over the block, each thread offering the best of what it has left: exact in
// the order of (value, index), whatever ties.
//
//  * Values are compared in 64 bits: score and logit as they are, the logarithm of the
//    sum from 32-bit terms, off by about 1e-7.  Within a beam the order is that of the
//    logits alone; fp64 is one addition per thread and round.
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
constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
    BeamArgs a;
    int chunks;     // of a row
    int per_warp;   // chunks that a warp of the first kernel takes
    int splits;     // blocks of a row
    float *lead;    // [R * W][chunks] largest logit
    float2 *part;   // [R * W][splits] maximum and sum
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

// A lane's logits of the chunk at `first`, the e-th at place(lane, e); -inf behind the
// row's end.  A row that is not 16-byte aligned is read in aligned pieces, each lane two
// neighbouring ones; its first and last chunk one logit at a time, so that nothing outside
// of the row is touched.
template <int DT>
__device__ __forceinline__ void load_chunk(const void *row, int64_t first, int V, int lane, float *x)
{
    constexpr int SIZE = DT == 2 ? 4 : 2, N = 16 / SIZE;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    if (off == 0 ? first + kChunk <= V : first > 0 && first + kChunk + N <= V) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + first * SIZE - off);
        uint4 v[kPer / N];
#pragma unroll
        for (int j = 0; j < kPer / N; j++) v[j] = __ldg(src + j * 32 + lane);
        if (off != 0) {
            uint4 u[kPer / N];
#pragma unroll
            for (int j = 0; j < kPer / N; j++) u[j] = __ldg(src + j * 32 + lane + 1);
#pragma unroll
            for (int j = 0; j < kPer / N; j++) v[j] = shifted_by(v[j], u[j], off);
        }
#pragma unroll
        for (int j = 0; j < kPer / N; j++) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (DT == 2) {
                    x[j * N + e] = __uint_as_float(w[e]);
                } else {
                    x[j * N + 2 * e] = elem_lo<DT == 2 ? 0 : DT>(w[e]);
                    x[j * N + 2 * e + 1] = elem_hi<DT == 2 ? 0 : DT>(w[e]);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < kPer; e++) {
        const int64_t i = first + place<DT>(lane, e);
        x[e] = i < V ? logit(row, DT, i) : -INFINITY;
    }
}

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

template <int DT>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamParams p)
{
    const BeamArgs &a = p.a;
    __shared__ float2 s_part[kScanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y, split = blockIdx.x;
    pdl_launch();
    if (!isfinite(__ldg(a.scores + r))) return;  // a beam not in use
    const int req = r / a.W, w = r - req * a.W;
    const void *row = static_cast<const uint8_t *>(a.logits) + (req * a.l_sr + w * a.l_sw) * (DT == 2 ? 4 : 2);
    const int c0 = (split * kScanWarps + warp) * p.per_warp, c1 = min(p.chunks, c0 + p.per_warp);
    float m = -INFINITY, s = 0.f;  // the warp's maximum, the lane's sum
    constexpr int B = 2;           // chunks in flight
    for (int c = c0; c < c1; c += B) {
        float x[B][kPer];
#pragma unroll
        for (int b = 0; b < B; b++)
            if (c + b < c1) load_chunk<DT>(row, static_cast<int64_t>(c + b) * kChunk, a.V, lane, x[b]);
#pragma unroll
        for (int b = 0; b < B; b++) {
            if (c + b >= c1) continue;
            float mx = x[b][0];
#pragma unroll
            for (int e = 1; e < kPer; e++) mx = fmaxf(mx, x[b][e]);  // (a NaN is left to the sum)
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
                const float2 d = fmul2(fadd2(make_float2(x[b][e], x[b][e + 1]), make_float2(base, base)), make_float2(kLog2e, kLog2e));
                sum = fadd2(sum, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
            }
            s += sum.x + sum.y;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) s_part[warp] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kScanWarps; i++) merge(m, s, s_part[i].x, s_part[i].y);
        p.part[static_cast<int64_t>(r) * p.splits + split] = make_float2(m, s);
    }
}

// A candidate: its value as an unsigned number of the same order (0: none), and its place.
struct Best {
    uint32_t hi, lo, at;
};

__device__ __forceinline__ Best best_of(double v, uint32_t at)
{
    uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    u = u >> 63 ? ~u : u | (uint64_t(1) << 63);
    if (!isfinite(v)) u = 0;
    return {static_cast<uint32_t>(u >> 32), static_cast<uint32_t>(u), at};
}

__device__ __forceinline__ double value_of(const Best &b)
{
    uint64_t u = (static_cast<uint64_t>(b.hi) << 32) | b.lo;
    u = u >> 63 ? u & ~(uint64_t(1) << 63) : ~u;
    return __longlong_as_double(static_cast<long long>(u));
}

__device__ __forceinline__ bool none(const Best &b) { return (b.hi | b.lo) == 0; }
__device__ __forceinline__ bool better(const Best &a, const Best &b)
{
    return a.hi != b.hi ? a.hi > b.hi : a.lo != b.lo ? a.lo > b.lo : a.at < b.at;
}

__device__ __forceinline__ Best warp_best(const Best &b)
{
    Best r;
    r.hi = __reduce_max_sync(~0u, b.hi);
    r.lo = __reduce_max_sync(~0u, b.hi == r.hi ? b.lo : 0u);
    r.at = __reduce_min_sync(~0u, b.hi == r.hi && b.lo == r.lo ? b.at : ~0u);
    return r;
}

// Of all threads' candidates; one barrier (the places alternate).
__device__ __forceinline__ Best block_best(const Best &b, Best (*places)[kPickWarps], int round)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Best w = warp_best(b);
    if (lane == 0) places[round & 1][warp] = w;
    __syncthreads();
    return warp_best(places[round & 1][lane]);
}

template <int DT>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamParams p)
{
    const BeamArgs &a = p.a;
    extern __shared__ float s_lead[];  // [W][chunks]
    __shared__ double s_score[kMaxBeams], s_lse[kMaxBeams];
    __shared__ bool s_ok[kMaxBeams];
    __shared__ Best s_best[2][kPickWarps];
    __shared__ int2 s_pick[kMaxPicks];  // beam and chunk
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int req = blockIdx.x;
    pdl_wait();

    // ---- the rows' logarithms, in the order of the splits
    for (int w = warp; w < a.W; w += kPickWarps) {
        const int r = req * a.W + w;
        const float score = __ldg(a.scores + r);
        bool ok = isfinite(score);
        float m = -INFINITY, s = 0.f;
        if (ok) {
            for (int i = lane; i < p.splits; i += 32) {
                const float2 v = p.part[static_cast<int64_t>(r) * p.splits + i];
                merge(m, s, v.x, v.y);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {  // (lane l with l + o: the same order in every lane that counts)
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
            s_lse[w] = ok ? static_cast<double>(m) + log(static_cast<double>(s)) : 0.0;
        }
    }
    for (int i = tid; i < a.W * p.chunks; i += kPickThreads)
        s_lead[i] = p.lead[static_cast<int64_t>(req) * a.W * p.chunks + i];
    __syncthreads();

    // ---- the chunks: a thread has every tpr-th of one beam
    const int tpr = kPickThreads / a.W;
    const int w = tid / tpr, sub = tid - w * tpr;
    const bool mine = w < a.W && s_ok[w < a.W ? w : 0];
    auto next_lead = [&]() -> Best {
        float top = -INFINITY;
        int at = -1;
        if (mine)
            for (int c = sub; c < p.chunks; c += tpr) {
                const float x = s_lead[w * p.chunks + c];
                if (x > top) {
                    top = x;
                    at = c;
                }
            }
        if (at < 0) return {0u, 0u, ~0u};
        return best_of(s_score[w] + (static_cast<double>(top) - s_lse[w]), static_cast<uint32_t>(w * p.chunks + at));
    };
    Best have = next_lead();
    int picks = 0;
    for (; picks < a.K; picks++) {
        const Best b = block_best(have, s_best, picks);
        if (none(b)) break;
        if (tid == 0) s_pick[picks] = make_int2(static_cast<int>(b.at) / p.chunks, static_cast<int>(b.at) % p.chunks);
        if (have.at == b.at && !none(have)) {
            s_lead[b.at] = -INFINITY;
            have = next_lead();
        }
    }
    __syncthreads();

    // ---- what they hold: up to two chunks a warp
    constexpr int Q = kMaxPicks / kPickWarps;
    float x[Q][kPer];
    Best own[Q];
    int beam[Q] = {};
    int64_t first[Q] = {};
    auto next_own = [&](int q) {
        float top = -INFINITY;
        int at = -1;
#pragma unroll
        for (int e = 0; e < kPer; e++)
            if (x[q][e] > top) {  // (the first of equal ones: places rise with e)
                top = x[q][e];
                at = e;
            }
        own[q] = at < 0 ? Best{0u, 0u, ~0u}
                        : best_of(s_score[beam[q]] + (static_cast<double>(top) - s_lse[beam[q]]),
                                  static_cast<uint32_t>(static_cast<int64_t>(beam[q]) * a.V + first[q] + place<DT>(lane, at)));
    };
#pragma unroll
    for (int q = 0; q < Q; q++) {
        const int i = q * kPickWarps + warp;
        const bool some = i < picks;
        const int2 pk = some ? s_pick[i] : make_int2(0, 0);
        beam[q] = pk.x;
        first[q] = static_cast<int64_t>(pk.y) * kChunk;
        const void *row = static_cast<const uint8_t *>(a.logits) + (req * a.l_sr + pk.x * a.l_sw) * (DT == 2 ? 4 : 2);
        if (some) load_chunk<DT>(row, first[q], a.V, lane, x[q]);
        else
#pragma unroll
            for (int e = 0; e < kPer; e++) x[q][e] = -INFINITY;
        next_own(q);
    }
    for (int k = 0; k < a.K; k++) {
        Best mineb = own[0];
#pragma unroll
        for (int q = 1; q < Q; q++)
            if (better(own[q], mineb)) mineb = own[q];
        const Best b = block_best(mineb, s_best, picks + 1 + k);
        const int64_t out = static_cast<int64_t>(req) * a.K + k;
        if (none(b)) {
            for (int i = k + tid; i < a.K; i += kPickThreads) {
                a.out_scores[out + i - k] = -INFINITY;
                a.parent[out + i - k] = -1;
                a.token[out + i - k] = -1;
            }
            break;
        }
        if (tid == 0) {
            a.out_scores[out] = static_cast<float>(value_of(b));
            a.parent[out] = static_cast<int>(b.at / static_cast<uint32_t>(a.V));
            a.token[out] = static_cast<int>(b.at % static_cast<uint32_t>(a.V));
        }
#pragma unroll
        for (int q = 0; q < Q; q++)
            if (own[q].at == b.at && !none(own[q])) {
                const int64_t at = static_cast<int64_t>(b.at) - static_cast<int64_t>(beam[q]) * a.V - first[q];
#pragma unroll
                for (int e = 0; e < kPer; e++)
                    if (place<DT>(lane, e) == at) x[q][e] = -INFINITY;
                next_own(q);
            }
    }
}

int chunks_of(const BeamArgs &a) { return (a.V + kChunk - 1) / kChunk; }

// Chunks per warp of the first kernel: about 16 warps a SM or more, up to 8 chunks each.
void plan(const BeamArgs &a, int nsm, BeamParams &p)
{
    p.a = a;
    p.chunks = chunks_of(a);
    const int64_t rows = static_cast<int64_t>(a.R) * a.W;
    p.per_warp = 1;
    while (p.per_warp < 8 && rows * p.chunks / (2 * p.per_warp) >= static_cast<int64_t>(nsm) * 32) p.per_warp *= 2;
    const int per_block = kScanWarps * p.per_warp;
    p.splits = (p.chunks + per_block - 1) / per_block;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <int DT>
cudaError_t launch_impl(const BeamParams &p, size_t smem, cudaStream_t stream)
{
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(beam_pick_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    beam_scan_kernel<DT><<<dim3(p.splits, p.a.R * p.a.W), kScanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_pick_kernel<DT>, dim3(p.a.R), kPickThreads, smem, stream, p);
}

}  // namespace

bool beam_fits(const BeamArgs &a) { return static_cast<int64_t>(a.W) * chunks_of(a) <= kMaxBeamChunks; }

size_t beam_workspace(const BeamArgs &a, int nsm)
{
    BeamParams p;
    plan(a, nsm, p);
    const size_t rows = static_cast<size_t>(a.R) * a.W;
    return up256(rows * p.chunks * sizeof(float)) + up256(rows * p.splits * sizeof(float2));
}

clis_status_t launch_beam(const BeamArgs &a, void *workspace, int nsm, cudaStream_t stream)
{
    BeamParams p;
    plan(a, nsm, p);
    const size_t rows = static_cast<size_t>(a.R) * a.W;
    p.lead = static_cast<float *>(workspace);
    p.part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + up256(rows * p.chunks * sizeof(float)));
    const size_t smem = static_cast<size_t>(a.W) * p.chunks * sizeof(float);
    const cudaError_t e = a.dtype == CLIS_DT_BF16 ? launch_impl<CLIS_DT_BF16>(p, smem, stream)
                          : a.dtype == CLIS_DT_FP16 ? launch_impl<CLIS_DT_FP16>(p, smem, stream)
                                                    : launch_impl<2>(p, smem, stream);
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
