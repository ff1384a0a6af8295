// paged_read.cu -- cached keys and values as 16-bit rows again: packed rows of any
// ranges of the sequences' tokens (to move, inspect or use them in a dense call), or
// whole pages for the chunk kernel, which works on 16-bit tiles.
//
//   x = code * scale, rounded to fp32 and then to the data type (a cache of 16-bit values is
//   copied): off by half a step of the data type and by 2^-24 of the value
//
// Bound: bytes, d + 4 read and 2 d written per row.  A thread turns 8 codes into one 16-byte
// store, so that a warp's stores fill whole lines; eight such pieces are in flight at a time,
// and places are multiplied out once per token.  120,000 tokens of 8 heads, K and V, 600 MB: 99 us,
// 89% of the measured copy rate (16 codes and two stores a thread 124, places per piece 110).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "clis_internal.h"
#include "paged_internal.h"
#include "sm103_ptx.cuh"

namespace clis {

__device__ unsigned int g_read_error_word = 0;

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;  // of a block: a warp looks up their places
constexpr int kBatch = 8;        // pieces in flight

__device__ __forceinline__ float2 e4m3_floats(uint32_t lo16)
{
    uint32_t r;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(lo16));
    return __half22float2(*reinterpret_cast<const __half2 *>(&r));
}

// Four codes of a word as values.
template <int CODE>
__device__ __forceinline__ void values4(uint32_t w, float scale, float *f)
{
    if (CODE == CLIS_CODE_INT8) {
        // 2^23 + 128 + code, minus 2^23 + 128: exact.
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 4; e++) f[e] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + e)) - 8388736.f) * scale;
    } else {
        const float2 a = e4m3_floats(w & 0xFFFFu), b = e4m3_floats(w >> 16);
        f[0] = a.x * scale;
        f[1] = a.y * scale;
        f[2] = b.x * scale;
        f[3] = b.y * scale;
    }
}

// A piece: 8 elements of a row.
struct Piece {
    uint4 u;  // codes in x and y, or 16-bit values
    float scale;
};

template <int CODE>
__device__ __forceinline__ void load_piece(Piece &x, const uint8_t *row, const float *scale, int piece)
{
    if (CODE < 0) {
        x.u = __ldg(reinterpret_cast<const uint4 *>(row) + piece);
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row) + piece);
        x.u.x = v.x;
        x.u.y = v.y;
        x.scale = __ldg(scale);
    }
}

template <int CODE, int DT>
__device__ __forceinline__ void store_piece(const Piece &x, uint16_t *dst)
{
    uint4 y = x.u;
    if (CODE >= 0) {
        float f[8];
        values4<CODE>(x.u.x, x.scale, f);
        values4<CODE>(x.u.y, x.scale, f + 4);
        y = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
    }
    *reinterpret_cast<uint4 *>(dst) = y;
}

// 32 tokens of both caches by a block.  Iteration `it` is head it / IPH of K's heads, then of V's;
// a thread has one piece of a token in it, of the same IPH tokens throughout, so that their
// places are looked up and multiplied out once.
template <int D>
struct Split {
    static constexpr int PPR = D / 8, IPH = kReadTokens * PPR / kReadThreads;  // pieces of a row, iterations of a head
    static constexpr int PER = kReadTokens / IPH;                             // tokens of an iteration
};

// One token's rows: where they lie in the caches and where they go.  from: 0 nowhere (reads as
// zeros), 1 there; to: whether they are written.
struct Token {
    int64_t kc, vc, ks, vs, ko, vo;
    bool from, to;
};

// Heads it0 / IPH .. of the block's tokens, kBatch pieces in flight.  SCALED: K's values (else its
// codes as they are, and its scales times k_times to k_scale at their offset `ko` / D of the row).
template <int CODE, int DT, int D, bool SCALED>
__device__ __forceinline__ void convert(const uint8_t *kc, const uint8_t *vc, const float *ks, const float *vs, int64_t kc_sh, int64_t vc_sh,
                                        int64_t ks_sh, int64_t vs_sh, uint16_t *ko, uint16_t *vo, int64_t ko_sh, int64_t vo_sh, float *k_scale,
                                        int64_t k_scale_sh, float k_times, int Hkv, const Token *tok, int it0, int step)
{
    using S = Split<D>;
    constexpr int B = CODE < 0 ? 2 : 1;
    const int piece = threadIdx.x & (S::PPR - 1);
    for (; it0 < 2 * Hkv * S::IPH; it0 += step) {
        Piece x[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const int hh = (it0 + b) / S::IPH;
            const Token &t = tok[b % S::IPH];
            x[b].u = make_uint4(0, 0, 0, 0);
            x[b].scale = 0.f;
            if (hh >= 2 * Hkv || !t.from || !t.to) continue;
            if (hh < Hkv) load_piece<CODE>(x[b], kc + (t.kc + hh * kc_sh) * B, ks + t.ks + hh * ks_sh, piece);
            else load_piece<CODE>(x[b], vc + (t.vc + (hh - Hkv) * vc_sh) * B, vs + t.vs + (hh - Hkv) * vs_sh, piece);
        }
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const int hh = (it0 + b) / S::IPH;
            const Token &t = tok[b % S::IPH];
            if (hh >= 2 * Hkv || !t.to) continue;
            if (hh < Hkv) {
                if (!SCALED) {
                    if (piece == 0) k_scale[t.ko / D + hh * k_scale_sh] = x[b].scale * k_times;
                    x[b].scale = 1.f;
                }
                store_piece<CODE, DT>(x[b], ko + t.ko + hh * ko_sh + piece * 8);
            } else {
                store_piece<CODE, DT>(x[b], vo + t.vo + (hh - Hkv) * vo_sh + piece * 8);
            }
        }
    }
}

template <int CODE, int DT, int D>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const ReadArgs a)
{
    using S = Split<D>;
    __shared__ int2 s_at[kReadTokens];  // page (-1: reads as zeros, -2: not written) and row of it
    const int t0 = blockIdx.x * kReadTokens;
    if (threadIdx.x < kReadTokens) {
        const int t = t0 + threadIdx.x;
        int page = -2, in = 0;
        unsigned int bad = 0;
        if (t < a.T) {
            // The last sequence whose rows start at t or before (cu does not fall).
            int lo = 0, hi = a.S;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(a.cu + mid + 1) <= t) lo = mid + 1;
                else hi = mid;
            }
            const int first = lo < a.S ? __ldg(a.cu + lo) : 0;
            if (lo < a.S && first >= 0 && first <= t) {
                const int64_t key = (a.start ? static_cast<int64_t>(__ldg(a.start + lo)) : 0) + (t - first);
                page = -1;
                if (key < 0 || key >= static_cast<int64_t>(a.width) << a.page_shift) {
                    bad = CLIS_PAGED_LENGTH_BIT;
                } else {
                    page = __ldg(a.block_table + lo * a.bt_s + (key >> a.page_shift));
                    in = static_cast<int>(key) & ((1 << a.page_shift) - 1);
                    if (page < 0 || page >= a.num_pages) {
                        bad = CLIS_PAGED_INDEX_BIT;
                        page = -1;
                    }
                }
            } else if (lo < a.S) {
                bad = CLIS_PAGED_LENGTH_BIT;  // (prefix sums that do not start at 0, or fall)
            }
        }
        s_at[threadIdx.x] = make_int2(page, in);
        if (bad) atomicOr(&g_read_error_word, bad);
    }
    __syncthreads();
    Token tok[S::IPH];
#pragma unroll
    for (int i = 0; i < S::IPH; i++) {
        const int t = i * S::PER + threadIdx.x / S::PPR;
        const int2 at = s_at[t];
        const int64_t pg = max(at.x, 0), in = at.y, row = t0 + t;
        tok[i] = {pg * a.kc_sp + in * a.kc_sn, pg * a.vc_sp + in * a.vc_sn, pg * a.z.ks_sp + in * a.z.ks_sn, pg * a.z.vs_sp + in * a.z.vs_sn,
                  row * a.ko_st, row * a.vo_st, at.x >= 0, at.x != -2};
    }
    convert<CODE, DT, D, true>(a.z.kc, a.z.vc, a.z.ks, a.z.vs, a.kc_sh, a.vc_sh, a.z.ks_sh, a.z.vs_sh, a.ko, a.vo, a.ko_sh, a.vo_sh, nullptr, 0, 1.f,
                               a.Hkv, tok, blockIdx.y * kBatch, gridDim.y * kBatch);
}

// Whole pages, for the chunk kernel (K's codes stay unscaled: its softmax applies the scales).  Units of 32 keys (all heads) of the sequences that
// it works on, laid end to end and cut into equal runs, one per block.  Two sequences
// that share a page write the same bits.
constexpr int kUnitKeys = kReadTokens;

struct UnpackParams {
    PagedArgs a;
    QuantArgs z;
    uint16_t *ko, *vo;
    float *ks;
    int32_t *table;  // nullptr: the cache's page numbers
    int g, rows_small;
};

template <int CODE, int DT, int D>
__global__ void __launch_bounds__(kReadThreads) paged_unpack_kernel(const UnpackParams p)
{
    const PagedArgs &a = p.a;
    const QuantArgs &z = p.z;
    __shared__ unsigned long long s_sum[kReadThreads / 32];
    __shared__ int s_seq, s_unit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch();
    auto seq_len = [&](int s) {
        return clip_seq(__ldg(a.cu_q + s), __ldg(a.cu_q + s + 1), __ldg(a.kv_len + s), a.T, a.width << a.page_shift);
    };
    auto units = [&](int s) -> int {
        const SeqLen q = seq_len(s);
        return chunk_items(q, p.g, p.rows_small, 1) == 0 ? 0 : ceil_div(q.kv, kUnitKeys);
    };
    const int per = (a.S + kReadThreads - 1) / kReadThreads;
    const int sb = min(a.S, tid * per), se = min(a.S, sb + per);
    unsigned long long mine = 0;
    for (int s = sb; s < se; s++) mine += units(s);
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    unsigned long long U = 0, before = 0;
    for (int w = 0; w < kReadThreads / 32; w++) {
        if (w < warp) before += s_sum[w];
        U += s_sum[w];
    }
    const unsigned long long u0 = U * blockIdx.x / gridDim.x, u1 = U * (blockIdx.x + 1) / gridDim.x;
    const unsigned long long excl = before + incl - mine;
    if (u0 < u1 && u0 >= excl && u0 < excl + mine) {
        unsigned long long rel = u0 - excl;
        for (int s = sb; s < se; s++) {
            const unsigned long long n = units(s);
            if (rel < n) {
                s_seq = s;
                s_unit = static_cast<int>(rel);
                break;
            }
            rel -= n;
        }
    }
    __syncthreads();
    if (u0 >= u1) {
        pdl_wait();
        return;
    }
    int s = s_seq, j = s_unit, n = units(s), kv = seq_len(s).kv;
    using S = Split<D>;
    const int mask = (1 << a.page_shift) - 1;
    const int64_t head = static_cast<int64_t>(D) << a.page_shift;  // values of a head's page
    for (unsigned long long u = u0; u < u1; u++) {
        Token tok[S::IPH];
#pragma unroll
        for (int i = 0; i < S::IPH; i++) {
            const int key = j * kUnitKeys + i * S::PER + threadIdx.x / S::PPR;
            const int page = key < kv ? __ldg(a.block_table + s * a.bt_s + (key >> a.page_shift)) : -1;
            const bool ok = page >= 0 && page < a.num_pages;  // (the chunk kernel records the others)
            const int64_t pg = ok ? page : 0, in = key & mask;
            const int64_t place = p.table ? static_cast<int64_t>(s) * a.width + (key >> a.page_shift) : pg;
            const int64_t to = place * a.Hkv * head + in * D;
            if (p.table && in == 0 && key < kv && (threadIdx.x & (S::PPR - 1)) == 0) p.table[place] = ok ? static_cast<int>(place) : -1;
            tok[i] = {pg * a.kc_sp + in * a.kc_sn, pg * a.vc_sp + in * a.vc_sn, pg * z.ks_sp + in * z.ks_sn, pg * z.vs_sp + in * z.vs_sn,
                      to, to, ok, ok};
        }
        convert<CODE, DT, D, false>(z.kc, z.vc, z.ks, z.vs, a.kc_sh, a.vc_sh, z.ks_sh, z.vs_sh, p.ko, p.vo, head, head, p.ks, mask + 1, a.scale_log2, a.Hkv,
                                    tok, 0, kBatch);
        if (++j == n && u + 1 < u1) {
            do s++;
            while (s + 1 < a.S && units(s) == 0);
            j = 0;
            n = units(s);
            kv = seq_len(s).kv;
        }
    }
    pdl_wait();  // (the schedule kernel, whose results only later kernels read)
}

template <int CODE, int DT>
cudaError_t launch_read_impl(const ReadArgs &a, dim3 grid, cudaStream_t stream)
{
    if (a.d == 128) paged_read_kernel<CODE, DT, 128><<<grid, kReadThreads, 0, stream>>>(a);
    else paged_read_kernel<CODE, DT, 64><<<grid, kReadThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int CODE, int DT>
cudaError_t launch_unpack_impl(const UnpackParams &p, int grid, cudaStream_t stream)
{
    return launch_pdl(p.a.d == 128 ? paged_unpack_kernel<CODE, DT, 128> : paged_unpack_kernel<CODE, DT, 64>, dim3(grid), kReadThreads, 0, stream, p);
}

}  // namespace

clis_status_t launch_paged_read(const ReadArgs &a, cudaStream_t stream)
{
    const int64_t blocks = (static_cast<int64_t>(a.T) + kReadTokens - 1) / kReadTokens;
    // Blocks share out a token group's heads where there are few groups.
    const int its = 2 * a.Hkv * kReadTokens * (a.d / 8) / kReadThreads;
    const int split = blocks >= 152 * 8 ? 1 : (its + kBatch - 1) / kBatch;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(split));
    const bool half = a.dtype == CLIS_DT_FP16;
    const cudaError_t e = a.z.code < 0                 ? launch_read_impl<-1, 0>(a, grid, stream)  // (the type does not matter)
                          : a.z.code == CLIS_CODE_INT8 ? (half ? launch_read_impl<CLIS_CODE_INT8, 1>(a, grid, stream)
                                                               : launch_read_impl<CLIS_CODE_INT8, 0>(a, grid, stream))
                                                       : (half ? launch_read_impl<CLIS_CODE_E4M3, 1>(a, grid, stream)
                                                               : launch_read_impl<CLIS_CODE_E4M3, 0>(a, grid, stream));
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t launch_paged_unpack(const PagedArgs &a, const QuantArgs &z, int rows_small, uint16_t *k_pages, float *k_scale,
                                  uint16_t *v_pages, int32_t *table, int nsm, cudaStream_t stream)
{
    const UnpackParams p{a, z, k_pages, v_pages, k_scale, table, a.H / a.Hkv, rows_small};
    const int grid = 8 * nsm;
    const bool half = a.dtype == CLIS_DT_FP16;
    const cudaError_t e = z.code == CLIS_CODE_INT8 ? (half ? launch_unpack_impl<CLIS_CODE_INT8, 1>(p, grid, stream)
                                                           : launch_unpack_impl<CLIS_CODE_INT8, 0>(p, grid, stream))
                                                   : (half ? launch_unpack_impl<CLIS_CODE_E4M3, 1>(p, grid, stream)
                                                           : launch_unpack_impl<CLIS_CODE_E4M3, 0>(p, grid, stream));
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t read_read_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_read_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_read_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_read_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
