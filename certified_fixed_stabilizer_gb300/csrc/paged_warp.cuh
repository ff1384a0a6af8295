// paged_warp.cuh -- what the kernels for a few query rows per sequence share, over a
// cache of 16-bit values (paged_decode.cu) and one of 8-bit codes (paged_q8.cu): the
// workers' runs of units, warp-level copies and matrix products, and the join of the
// items that several workers computed parts of.
//
// Each translation unit that includes it has a copy of its own.
#pragma once

#include "clis_internal.h"
#include "paged_internal.h"
#include "sm103_ptx.cuh"

namespace clis {
namespace {

constexpr int kDecodeWarps = 4;  // of a block
constexpr int kDecodeThreads = kDecodeWarps * 32;
constexpr int kJoinThreads = 256;

struct DecodeParams {
    PagedArgs a;
    int g, rows_max, least;
    int limit;   // query rows that a sequence may have (rows_max of them in an item)
    int workers; // warps of the grid
    int strict;  // no chunk kernel follows: a sequence of more rows is an error
    int one;     // (paged_q8.cu) a block per item, no parts
    float *part_o;   // [2 * workers][rows_max][D]: place 2 c + 1 if worker c starts the item, 2 c if it goes on with it
    float2 *part_ml; // [2 * workers][rows_max]
    int4 *meta;      // [workers] {parts, first row of q, new tokens and 2^16 times the item's first row, head} of the item
                     // the worker starts and does not finish
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t *r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if (DT)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ SeqLen seq_len(const PagedArgs &a, int s)
{
    return clip_seq(__ldg(a.cu_q + s), __ldg(a.cu_q + s + 1), __ldg(a.kv_len + s), a.T, a.width << a.page_shift);
}

// Position in the block's run: unit j of item (s, h).
// TR: an item has up to TR of a sequence's query rows, `tile` says which (0: all of them).
template <int TK, int TR = 0>
struct Pos {
    int s, h, j, units;
    int tile, tiles;
    SeqLen q;
    uint32_t left;  // units of the run from this one on

    __device__ __forceinline__ void set(const PagedArgs &a, int seq, int g)
    {
        s = seq;
        q = seq_len(a, s);
        units = decode_units(q, TK);
        tile = 0;
        tiles = TR ? ceil_div(q.n * g, TR) : 1;
    }
    // The next item of the run (there is one if units are left).
    __device__ __forceinline__ void next_item(const PagedArgs &a, int g, int limit)
    {
        j = 0;
        if (TR) {
            if (++tile < tiles) return;
            tile = 0;
        }
        if (++h < a.Hkv) return;
        h = 0;
        int n = s + 1;
        while (n < a.S) {
            set(a, n, g);
            if (is_decode(q, g, limit)) return;
            ++n;
        }
        left = 0;  // not reached while the run's units are counted alike
    }
};

// The runs of the block's workers (neighbouring runs go to different blocks): worker
// w * gridDim.x + blockIdx.x, w < NW, starts at unit s_rel[w] of sequence s_seq[w].  All
// threads take part; ends with a barrier.
struct Runs {
    uint64_t U;  // units of the batch
    int nb;      // workers that take part
};

template <int TK, int NW, int TR = 0>
__device__ __forceinline__ Runs block_runs(const DecodeParams &p, uint64_t *s_sum, int *s_seq, uint64_t *s_rel, unsigned int &bad)
{
    const PagedArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.S + kDecodeThreads - 1) / kDecodeThreads;
    const int sb = min(a.S, tid * per), se = min(a.S, sb + per);
    uint64_t mine = 0;
    for (int s = sb; s < se; s++) {
        const SeqLen q = seq_len(a, s);
        if (q.bad) bad |= CLIS_PAGED_LENGTH_BIT;
        if (is_decode(q, p.g, p.limit)) mine += static_cast<uint64_t>(a.Hkv * (TR ? ceil_div(q.n * p.g, TR) : 1)) * decode_units(q, TK);
        else if (p.strict && q.n > 0) bad |= CLIS_PAGED_LENGTH_BIT;
    }
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    uint64_t U = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kDecodeWarps; w++) {
        if (w < warp) before += s_sum[w];
        U += s_sum[w];
    }
    const uint64_t excl = before + incl - mine;
    const int nb = decode_workers(U, p.workers, p.least);
    for (int w = 0; w < NW; w++) {
        const int cw = w * gridDim.x + blockIdx.x;
        if (cw >= nb) break;
        const uint64_t u = decode_cut(U, nb, cw);
        if (u < excl || u >= excl + mine) continue;
        uint64_t rel = u - excl;
        for (int s = sb; s < se; s++) {
            const SeqLen q = seq_len(a, s);
            if (!is_decode(q, p.g, p.limit)) continue;
            const uint64_t n = static_cast<uint64_t>(a.Hkv * (TR ? ceil_div(q.n * p.g, TR) : 1)) * decode_units(q, TK);
            if (rel < n) {
                s_seq[w] = s;
                s_rel[w] = rel;
                break;
            }
            rel -= n;
        }
    }
    __syncthreads();
    return {U, nb};
}

// Adds the partial results of the items that workers of the decode kernel started
// and did not finish: worker c's own and those at the start of the following
// workers' runs, a few, or a hundred where there are few sequences.  A block looks
// after kJoinEach neighbouring workers; its warps share out the rows of the items
// that those started, and where there are fewer rows than warps the parts of each
// row too (by counts alone, and added in a fixed order: reruns agree bit for bit).
// blockIdx.y: where an item has many rows, blocks take turns.
constexpr int kJoinEach = 8;

template <int D, int DT>
__global__ void __launch_bounds__(kJoinThreads) paged_decode_join_kernel(const DecodeParams p)
{
    constexpr int V = D / 32, W = kJoinThreads / 32, B = 8;  // columns per lane, warps, loads in flight
    __shared__ int4 s_meta[kJoinEach];
    __shared__ float s_o[W][D];
    __shared__ float2 s_ml[W];
    const PagedArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = blockIdx.x * kJoinEach;
    pdl_wait();
    pdl_launch();
    if (tid < kJoinEach) s_meta[tid] = c0 + tid < p.workers ? p.meta[c0 + tid] : make_int4(0, 0, 0, 0);
    __syncthreads();
    auto rows_of = [&](int i) { return s_meta[i].x ? min((s_meta[i].z & 0xFFFF) * p.g - (s_meta[i].z >> 16), p.rows_max) : 0; };
    int rows = 0;
#pragma unroll
    for (int i = 0; i < kJoinEach; i++) rows += rows_of(i);
    const int mine = (rows + gridDim.y - 1) / gridDim.y;  // rows of this block
    int per = W;                                          // warps per row
    while (per > 1 && mine * per > W) per /= 2;
    for (int r0 = blockIdx.y * (W / per); r0 < rows; r0 += gridDim.y * (W / per)) {
        const int sub = warp % per;
        int row = r0 + warp / per, i = 0;
        const bool live = row < rows;
        if (live)
            while (true) {  // the item that the row belongs to
                const int n = rows_of(i);
                if (row < n) break;
                row -= n;
                i++;
            }
        const int4 mt = s_meta[live ? i : 0];
        const int c = c0 + i;
        float M = -INFINITY, l = 0.f, o[V];
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = 0.f;
        auto add = [&](float m1, float l1, const float *x) {
            if (l1 == 0.f) return;  // a part none of whose keys the row sees
            const float m = fmaxf(M, m1), w = ex2_approx(m1 - m);
            const bool none = l == 0.f;
            const float w0 = none ? 0.f : ex2_approx(M - m);
            M = m;
            l = none ? w * l1 : fmaf(l, w0, w * l1);
#pragma unroll
            for (int e = 0; e < V; e++) o[e] = none ? w * x[e] : fmaf(o[e], w0, w * x[e]);
        };
        if (live) {
            for (int k0 = sub; k0 < mt.x; k0 += B * per) {
                float2 ml[B];
                float x[B][V];
#pragma unroll
                for (int e = 0; e < B; e++) {
                    const int k = k0 + e * per;
                    ml[e] = make_float2(0.f, 0.f);
                    if (k >= mt.x) continue;
                    const int64_t at = static_cast<int64_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)) * p.rows_max + row;
                    ml[e] = p.part_ml[at];
                    if constexpr (V == 4) {
                        const float4 u = reinterpret_cast<const float4 *>(p.part_o + at * D)[lane];
                        x[e][0] = u.x; x[e][1] = u.y; x[e][2] = u.z; x[e][3] = u.w;
                    } else {
                        const float2 u = reinterpret_cast<const float2 *>(p.part_o + at * D)[lane];
                        x[e][0] = u.x; x[e][1] = u.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < B; e++) add(ml[e].x, ml[e].y, x[e]);
            }
        }
        if (per > 1) {
#pragma unroll
            for (int e = 0; e < V; e++) s_o[warp][lane * V + e] = o[e];
            if (lane == 0) s_ml[warp] = make_float2(M, l);
            __syncthreads();
            if (sub == 0)
                for (int w = 1; w < per; w++) add(s_ml[warp + w].x, s_ml[warp + w].y, &s_o[warp + w][lane * V]);
            __syncthreads();
        }
        if (live && sub == 0) {
            const float inv = 1.f / l;
            const int of = row + (mt.z >> 16), tok = of / p.g, hd = mt.w * p.g + (of - tok * p.g);
            uint16_t *dst = a.o + static_cast<int64_t>(mt.y + tok) * a.o_st + hd * a.o_sh + lane * V;
#pragma unroll
            for (int e = 0; e < V; e += 2)  // (zeros for a row that sees no key)
                *reinterpret_cast<uint32_t *>(dst + e) = l == 0.f ? 0u : pack2<DT>(o[e] * inv, o[e + 1] * inv);
            if (lane == 0 && a.lse2)
                a.lse2[static_cast<int64_t>(mt.y + tok) * a.H + hd] = l == 0.f ? -INFINITY : M + log2f(l);
        }
    }
}

// The item that a worker starts at unit j0 and does not finish: how many workers compute
// parts of it.  end: the item's last unit, counted over the batch.
__device__ __forceinline__ int item_parts(const Runs &r, int c, uint64_t end)
{
    int ce = static_cast<int>(div64(end * static_cast<uint32_t>(r.nb), r.U));
    while (ce > c && decode_cut(r.U, r.nb, ce) > end) ce--;
    while (ce + 1 < r.nb && decode_cut(r.U, r.nb, ce + 1) <= end) ce++;
    return ce - c + 1;
}

inline size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Workspace of `workers` workers with `rows` rows each: meta, part_ml, part_o.
inline size_t parts_workspace(size_t workers, size_t rows, int d)
{
    return up256(workers * sizeof(int4)) + up256(2 * workers * rows * sizeof(float2)) +
           up256(2 * workers * rows * d * sizeof(float));
}

inline void place_parts(DecodeParams &p, size_t workers, size_t rows, void *workspace)
{
    char *w = static_cast<char *>(workspace);
    p.workers = static_cast<int>(workers);
    p.rows_max = p.limit = static_cast<int>(rows);
    p.meta = reinterpret_cast<int4 *>(w);
    w += up256(workers * sizeof(int4));
    p.part_ml = reinterpret_cast<float2 *>(w);
    w += up256(2 * workers * rows * sizeof(float2));
    p.part_o = reinterpret_cast<float *>(w);
}

template <int D, int DT>
cudaError_t launch_join(const DecodeParams &p, cudaStream_t stream)
{
    return launch_pdl(paged_decode_join_kernel<D, DT>, dim3((p.workers + kJoinEach - 1) / kJoinEach, p.rows_max / 4), kJoinThreads,
                      0, stream, p);
}

}  // namespace
}  // namespace clis
