// paged_read.cu -- cached keys and values as 16-bit rows again: packed rows of any
// ranges of the sequences' tokens (to move, inspect or use them in a dense call), or
// whole pages for the chunk kernel, which works on 16-bit tiles.
//
//   x = code * scale, rounded once to the data type (a cache of 16-bit values is copied)
//
// Bound: bytes, d + 4 read and 2 d written per row.  A thread turns 16 codes into two
// 16-byte stores; four such pieces are in flight at a time.
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
constexpr int kBatch = 4;        // pieces in flight

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

// A piece: 16 elements of a row.
struct Piece {
    uint4 u, w;  // codes in u; 16-bit values in u and w
    float scale;
};

template <int CODE>
__device__ __forceinline__ void load_piece(Piece &x, const uint8_t *row, const float *scale, int chunk)
{
    if (CODE < 0) {
        const uint4 *src = reinterpret_cast<const uint4 *>(row + chunk * 32);
        x.u = __ldg(src);
        x.w = __ldg(src + 1);
    } else {
        x.u = __ldg(reinterpret_cast<const uint4 *>(row + chunk * 16));
        x.scale = __ldg(scale);
    }
}

template <int CODE, int DT>
__device__ __forceinline__ void store_piece(const Piece &x, uint16_t *dst)
{
    uint4 y0 = x.u, y1 = x.w;
    if (CODE >= 0) {
        float f[16];
        values4<CODE>(x.u.x, x.scale, f);
        values4<CODE>(x.u.y, x.scale, f + 4);
        values4<CODE>(x.u.z, x.scale, f + 8);
        values4<CODE>(x.u.w, x.scale, f + 12);
        y0 = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
        y1 = make_uint4(pack2<DT>(f[8], f[9]), pack2<DT>(f[10], f[11]), pack2<DT>(f[12], f[13]), pack2<DT>(f[14], f[15]));
    }
    reinterpret_cast<uint4 *>(dst)[0] = y0;
    reinterpret_cast<uint4 *>(dst)[1] = y1;
}

// A token's place: page (-1: reads as zeros, -2: not written) and row of it.
template <int CODE, int DT>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const ReadArgs a)
{
    __shared__ int2 s_at[kReadTokens];
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
    const int cpr = a.d >> 4, shift = a.d == 128 ? 3 : 2;  // pieces of a row
    const int all = kReadTokens * cpr * a.Hkv;
    for (int i0 = blockIdx.y * kReadThreads * kBatch + threadIdx.x; i0 < all; i0 += gridDim.y * kReadThreads * kBatch) {
        Piece k[kBatch], v[kBatch];
        int2 at[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const int i = i0 + b * kReadThreads, chunk = i & (cpr - 1), t = (i >> shift) & (kReadTokens - 1), h = (i >> shift) / kReadTokens;
            at[b] = i < all ? s_at[t] : make_int2(-2, 0);
            k[b].u = k[b].w = v[b].u = v[b].w = make_uint4(0, 0, 0, 0);
            k[b].scale = v[b].scale = 0.f;
            if (at[b].x < 0) continue;
            const int64_t pg = at[b].x, in = at[b].y;
            constexpr int B = CODE < 0 ? 2 : 1;
            load_piece<CODE>(k[b], a.z.kc + (pg * a.kc_sp + h * a.kc_sh + in * a.kc_sn) * B,
                             a.z.ks + pg * a.z.ks_sp + h * a.z.ks_sh + in * a.z.ks_sn, chunk);
            load_piece<CODE>(v[b], a.z.vc + (pg * a.vc_sp + h * a.vc_sh + in * a.vc_sn) * B,
                             a.z.vs + pg * a.z.vs_sp + h * a.z.vs_sh + in * a.z.vs_sn, chunk);
        }
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            if (at[b].x == -2) continue;
            const int i = i0 + b * kReadThreads, chunk = i & (cpr - 1), t = (i >> shift) & (kReadTokens - 1), h = (i >> shift) / kReadTokens;
            const int64_t row = t0 + t;
            store_piece<CODE, DT>(k[b], a.ko + row * a.ko_st + h * a.ko_sh + chunk * 16);
            store_piece<CODE, DT>(v[b], a.vo + row * a.vo_st + h * a.vo_sh + chunk * 16);
        }
    }
}

// Whole pages, for the chunk kernel (K's codes stay unscaled: its softmax applies the scales).  Units of 32 keys (all heads) of the sequences that
// it works on, laid end to end and cut into equal runs, one per block.  Two sequences
// that share a page write the same bits.
constexpr int kUnitKeys = 32;

struct UnpackParams {
    PagedArgs a;
    QuantArgs z;
    uint16_t *ko, *vo;
    float *ks;
    int g, rows_small;
};

template <int CODE, int DT>
__global__ void __launch_bounds__(kReadThreads) paged_unpack_kernel(const UnpackParams p)
{
    const PagedArgs &a = p.a;
    const QuantArgs &z = p.z;
    __shared__ unsigned long long s_sum[kReadThreads / 32];
    __shared__ int s_seq, s_unit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    if (u0 >= u1) return;
    int s = s_seq, j = s_unit, n = units(s), kv = seq_len(s).kv;
    const int cpr = a.d >> 4, shift = a.d == 128 ? 3 : 2, page = 1 << a.page_shift;
    const int all = kUnitKeys * cpr * a.Hkv;
    for (unsigned long long u = u0; u < u1; u++) {
        for (int i0 = tid; i0 < all; i0 += kReadThreads * kBatch) {
            Piece k[kBatch], v[kBatch];
            int64_t to[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                const int i = i0 + b * kReadThreads, chunk = i & (cpr - 1), h = (i >> shift) / kUnitKeys;
                const int key = j * kUnitKeys + ((i >> shift) & (kUnitKeys - 1));
                to[b] = -1;
                if (i >= all || key >= kv) continue;
                const int pg = __ldg(a.block_table + s * a.bt_s + (key >> a.page_shift));
                if (pg < 0 || pg >= a.num_pages) continue;  // (the chunk kernel records it)
                const int64_t in = key & (page - 1);
                load_piece<CODE>(k[b], z.kc + pg * a.kc_sp + h * a.kc_sh + in * a.kc_sn, z.ks + pg * z.ks_sp + h * z.ks_sh + in * z.ks_sn,
                                 chunk);
                load_piece<CODE>(v[b], z.vc + pg * a.vc_sp + h * a.vc_sh + in * a.vc_sn, z.vs + pg * z.vs_sp + h * z.vs_sh + in * z.vs_sn,
                                 chunk);
                to[b] = (((static_cast<int64_t>(pg) * a.Hkv + h) << a.page_shift) + in) * a.d + chunk * 16;
            }
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                if (to[b] < 0) continue;
                if ((to[b] & (a.d - 1)) == 0) p.ks[to[b] / a.d] = k[b].scale;
                k[b].scale = 1.f;  // (the codes as they are)
                store_piece<CODE, DT>(k[b], p.ko + to[b]);
                store_piece<CODE, DT>(v[b], p.vo + to[b]);
            }
        }
        if (++j == n && u + 1 < u1) {
            do s++;
            while (s + 1 < a.S && units(s) == 0);
            j = 0;
            n = units(s);
            kv = seq_len(s).kv;
        }
    }
}

template <int CODE>
cudaError_t launch_read_impl(const ReadArgs &a, dim3 grid, cudaStream_t stream)
{
    if (a.dtype == CLIS_DT_FP16 || CODE < 0) paged_read_kernel<CODE, 1><<<grid, kReadThreads, 0, stream>>>(a);
    else paged_read_kernel<CODE, 0><<<grid, kReadThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int CODE>
cudaError_t launch_unpack_impl(const UnpackParams &p, int grid, cudaStream_t stream)
{
    if (p.a.dtype == CLIS_DT_FP16) paged_unpack_kernel<CODE, 1><<<grid, kReadThreads, 0, stream>>>(p);
    else paged_unpack_kernel<CODE, 0><<<grid, kReadThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

clis_status_t launch_paged_read(const ReadArgs &a, cudaStream_t stream)
{
    const int64_t blocks = (static_cast<int64_t>(a.T) + kReadTokens - 1) / kReadTokens;
    // Blocks share out a token group's heads where there are few groups.
    const int pieces = kReadTokens * (a.d >> 4) * a.Hkv;
    int split = (pieces + kReadThreads * kBatch - 1) / (kReadThreads * kBatch);
    if (blocks >= 152 * 8) split = 1;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(split));
    const cudaError_t e = a.z.code < 0 ? launch_read_impl<-1>(a, grid, stream)
                          : a.z.code == CLIS_CODE_INT8 ? launch_read_impl<CLIS_CODE_INT8>(a, grid, stream)
                                                       : launch_read_impl<CLIS_CODE_E4M3>(a, grid, stream);
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t launch_paged_unpack(const PagedArgs &a, const QuantArgs &z, int rows_small, uint16_t *k_pages, float *k_scale,
                                  uint16_t *v_pages, int nsm, cudaStream_t stream)
{
    const UnpackParams p{a, z, k_pages, v_pages, k_scale, a.H / a.Hkv, rows_small};
    const int grid = 8 * nsm;
    const cudaError_t e = z.code == CLIS_CODE_INT8 ? launch_unpack_impl<CLIS_CODE_INT8>(p, grid, stream)
                                                   : launch_unpack_impl<CLIS_CODE_E4M3>(p, grid, stream);
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
