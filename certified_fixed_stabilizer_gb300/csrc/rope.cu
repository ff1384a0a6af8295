// rope.cu -- rotary positions with up to four axes for q and k in one launch,
// and the same rotation on the way into a paged key/value cache.
//
// Pair p of a head's row turns by the angle pos[axis_p] * inv_freq_p:
//   (y0, y1) = (x0 cos a - x1 sin a, x1 cos a + x0 sin a).
// The transposed rotation (the gradient) only changes the sign of sin a.
//
// Angles of far positions: a position times a frequency in fp32 is off by
// 2^-24 of the angle itself (0.06 rad at position 10^6), so the frequency is
// held as a 64-bit fraction of a turn and multiplied by the integer position
// modulo 2^64.  The product IS the fraction of a turn, whatever the position's
// size or sign, off by at most |pos| * 2^-54 turns (the frequency's own double
// rounding); its upper 32 bits as a signed number of 2^-31 half turns go to
// sincospif.  Position 10^6 is then as exact as position 1.
//
// Bound: HBM bytes (each row read once and written once; sin and cos are
// computed once for a token and group of heads, not per head).  A thread owns
// 16 elements (8 pairs) of a row and walks a group of heads with the eight
// angles in registers; loads of four heads are in flight at a time, the first
// of them while the angles are computed.  480p video q and k (671 MB read and
// written) take 102.6 us, 6.5 TB/s (a plain copy of as many bytes 104.6); a chunk
// of 8,192 tokens into a cache (201 MB) 39.3 us, 5.1 TB/s (a plain copy 37.0: what
// fits the L2 twice over does not reach the rate of long copies).  More loads in
// flight make it slower (blocks of 128 threads, 8 an SM: 45.2; two heads a thread
// at a time, 5 blocks an SM: 50.2; eight, 2 blocks: 39.9).  At three blocks an SM the
// kernels that write the cache spill 32 bytes of registers; the plain ones do not.
//
// Into a cache of codes a row's scale needs its largest magnitude: its 4 or 8 threads
// exchange it by shuffles and each writes its 16 codes.  The same chunk (185 MB) takes 41 us, 27
// by the copy rate: two blocks an SM (three, with spills, 51; in one launch with q's rotation 45 with 16
// heads a block, 60, 49, 47, 47 and 47 with 4, 8, 12, 24 and 48).
#include <cuda_bf16.h>

#include "clis_internal.h"
#include "paged_internal.h"
#include "sm103_ptx.cuh"

namespace clis {

__device__ unsigned int g_rot_error_word = 0;

namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxPairs = 64;  // d / 2 at d = 128
constexpr int kMaxAxes = 4;
constexpr int kHeadBatch = 4;  // heads whose loads are in flight together

// The eight pairs in u0, u1 by the angles cs, sn.  Interleaved: `first` and `second`
// say whether u0's and u1's pairs turn (what does not turn is not multiplied by 1
// and 0: an inf beside it would make a NaN).
template <int DT>
__device__ __forceinline__ void rotate8(uint4 &u0, uint4 &u1, const float *cs, const float *sn, bool interleaved,
                                        bool first, bool second)
{
    uint32_t a[4] = {u0.x, u0.y, u0.z, u0.w}, b[4] = {u1.x, u1.y, u1.z, u1.w};
    if (interleaved) {
        // a holds the first four pairs as (x0, x1) words, b the other four.
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float x0 = elem_lo<DT>(a[e]), x1 = elem_hi<DT>(a[e]);
            if (first) a[e] = pack2<DT>(fmaf(x0, cs[e], -x1 * sn[e]), fmaf(x1, cs[e], x0 * sn[e]));
            const float z0 = elem_lo<DT>(b[e]), z1 = elem_hi<DT>(b[e]);
            if (second) b[e] = pack2<DT>(fmaf(z0, cs[4 + e], -z1 * sn[4 + e]), fmaf(z1, cs[4 + e], z0 * sn[4 + e]));
        }
    } else {
        // a holds x0 of pairs 0..7, b their x1.
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float p0 = elem_lo<DT>(a[e]), p1 = elem_lo<DT>(b[e]);
            const float q0 = elem_hi<DT>(a[e]), q1 = elem_hi<DT>(b[e]);
            a[e] = pack2<DT>(fmaf(p0, cs[2 * e], -p1 * sn[2 * e]), fmaf(q0, cs[2 * e + 1], -q1 * sn[2 * e + 1]));
            b[e] = pack2<DT>(fmaf(p1, cs[2 * e], p0 * sn[2 * e]), fmaf(q1, cs[2 * e + 1], q0 * sn[2 * e + 1]));
        }
    }
    u0 = make_uint4(a[0], a[1], a[2], a[3]);
    u1 = make_uint4(b[0], b[1], b[2], b[3]);
}

// The same in fp32, unrounded: f0, f1 are the values of u0 and u1.
template <int DT>
__device__ __forceinline__ void rotate8f(const uint4 &u0, const uint4 &u1, float *f0, float *f1, const float *cs, const float *sn,
                                         bool interleaved, bool first, bool second)
{
    const uint32_t a[4] = {u0.x, u0.y, u0.z, u0.w}, b[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float p0 = elem_lo<DT>(a[e]), q0 = elem_hi<DT>(a[e]), p1 = elem_lo<DT>(b[e]), q1 = elem_hi<DT>(b[e]);
        f0[2 * e] = p0;
        f0[2 * e + 1] = q0;
        f1[2 * e] = p1;
        f1[2 * e + 1] = q1;
        if (interleaved) {
            if (first) {
                f0[2 * e] = fmaf(p0, cs[e], -q0 * sn[e]);
                f0[2 * e + 1] = fmaf(q0, cs[e], p0 * sn[e]);
            }
            if (second) {
                f1[2 * e] = fmaf(p1, cs[4 + e], -q1 * sn[4 + e]);
                f1[2 * e + 1] = fmaf(q1, cs[4 + e], p1 * sn[4 + e]);
            }
        } else if (first) {
            f0[2 * e] = fmaf(p0, cs[2 * e], -p1 * sn[2 * e]);
            f0[2 * e + 1] = fmaf(q0, cs[2 * e + 1], -q1 * sn[2 * e + 1]);
            f1[2 * e] = fmaf(p1, cs[2 * e], p0 * sn[2 * e]);
            f1[2 * e + 1] = fmaf(q1, cs[2 * e + 1], q0 * sn[2 * e + 1]);
        }
    }
}

// Eight values times `mul` as codes.  int8: adding 1.5 * 2^23 leaves the nearest whole
// number (ties to even) in the low bits; |value * mul| is at most 127.  The product is rounded
// first: ties (16-bit values meet them) are then those of value * mul in fp32.
template <int CODE>
__device__ __forceinline__ uint2 codes8(const float *f, float mul)
{
    if (CODE == CLIS_CODE_E4M3)
        return make_uint2(pack_e4m3x4(f[0] * mul, f[1] * mul, f[2] * mul, f[3] * mul),
                          pack_e4m3x4(f[4] * mul, f[5] * mul, f[6] * mul, f[7] * mul));
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; e++) w[e] = __float_as_uint(__fadd_rn(__fmul_rn(f[e], mul), 12582912.f));
    return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
}

// A row's 16 values of this thread (the row lies in NC neighbouring lanes) into codes
// at dst + e0 and dst + e1, and its scale.  The scale is the row's largest magnitude over
// that of the codes; a row below 2^-100 becomes zeros (1 / scale would overflow), one that
// holds a non-finite value gets the scale NaN and the codes 0, so it reads back as NaN.
template <int CODE, int NC>
__device__ __forceinline__ void store_codes(const float *f0, const float *f1, uint8_t *dst, int e0, int e1, float *scale)
{
    uint32_t top = 0;  // (bits of magnitudes are ordered, infinity and NaN above the numbers)
#pragma unroll
    for (int e = 0; e < 8; e++)
        top = max(top, max(__float_as_uint(f0[e]) & 0x7FFFFFFFu, __float_as_uint(f1[e]) & 0x7FFFFFFFu));
    const int lane = threadIdx.x & 31;
    const unsigned mask = ((1u << NC) - 1u) << (lane & ~(NC - 1));
#pragma unroll
    for (int o = 1; o < NC; o <<= 1) top = max(top, __shfl_xor_sync(mask, top, o));
    constexpr float kTop = CODE == CLIS_CODE_INT8 ? 127.f : 448.f;
    const float t = __uint_as_float(top);
    uint2 c0 = make_uint2(0u, 0u), c1 = c0;
    float sc = 0.f;
    if (top >= 0x7F800000u) {
        sc = __uint_as_float(0x7FC00000u);
    } else if (t >= 7.888609052210118e-31f) {  // 2^-100
        const float mul = kTop / t;
        sc = t / kTop;
        c0 = codes8<CODE>(f0, mul);
        c1 = codes8<CODE>(f1, mul);
    }
    *reinterpret_cast<uint2 *>(dst + e0) = c0;
    *reinterpret_cast<uint2 *>(dst + e1) = c1;
    if ((lane & (NC - 1)) == 0) *scale = sc;
}

// NC: 16-element chunks per row (d / 16).  MODE: 0 rotation, 1 into a
// cache, 2 + c into a cache of codes of kind c.  hg: heads per block row of the grid.
// The first heads are loaded before the angles are computed, so that the chain
// frequency -> turn -> sin, cos runs beside them.
template <int DT, int NC, int MODE>
__global__ void __launch_bounds__(kRotThreads, MODE > 1 ? 2 : 3) rot_kernel(const RotArgs a, const int hg)
{
    constexpr bool APPEND = MODE > 0;
    constexpr int CODE = MODE - 2;
    __shared__ unsigned long long s_step[kMaxPairs];
    if (MODE > 1) pdl_launch();
    __shared__ int s_axis[kMaxPairs];
    const int idx = blockIdx.x * kRotThreads + threadIdx.x;
    const bool live = idx < a.B * a.N * NC;
    const int tok = live ? idx / NC : 0, ch = idx % NC;
    const int b = tok / a.N, n = tok - b * a.N;

    // The thread's two 8-element vectors of a row and how many of their pairs turn.
    // Halves: x0 and x1 of pairs 8 ch .. 8 ch + 7.  Interleaved: pairs 4 ch .. 4 ch + 3
    // from the row's first half and as many from its second (a warp's accesses then
    // fill whole 128-byte lines).
    const bool inter = a.interleaved != 0;
    const bool rot = ch * 8 < a.pairs;  // (halves)
    const int e0 = inter || rot ? ch * 8 : ch * 16;
    const int e1 = inter ? NC * 8 + ch * 8 : rot ? a.pairs + ch * 8 : ch * 16 + 8;
    const int p0 = inter ? ch * 4 : ch * 8, p1 = inter ? NC * 4 + ch * 4 : ch * 8 + 4;  // pairs of angles 0-3, 4-7
    const bool turn0 = p0 < a.pairs, turn1 = p1 < a.pairs;  // (pairs is a multiple of 8)

    const int heads = a.Hq + (APPEND ? 2 : 1) * a.Hk;
    const int h0 = blockIdx.y * hg, h1 = live ? min(h0 + hg, heads) : h0;
    auto source = [&](int h) -> const uint16_t * {
        if (h < a.Hq) return a.q + b * a.q_sb + h * a.q_sh + n * a.q_sn;
        if (!APPEND || h < a.Hq + a.Hk) return a.k + b * a.k_sb + (h - a.Hq) * a.k_sh + n * a.k_sn;
        return a.v + (h - a.Hq - a.Hk) * a.v_sh + n * a.v_sn;
    };
    uint4 u0[kHeadBatch], u1[kHeadBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kHeadBatch; i++) {
            if (h + i >= h1) continue;
            const uint16_t *src = source(h + i);
            u0[i] = *reinterpret_cast<const uint4 *>(src + e0);
            u1[i] = *reinterpret_cast<const uint4 *>(src + e1);
        }
    };
    load(h0);
    const bool angles = MODE < 2 || h0 < a.Hq + a.Hk;  // (a block of V's heads alone turns nothing)
    int pos[kMaxAxes];
#pragma unroll
    for (int x = 0; x < kMaxAxes; x++)
        pos[x] = x < a.axes && a.pairs > 0 && angles ? __ldg(a.pos + b * a.p_sb + n * a.p_sn + x * a.p_sa) : 0;
    int64_t page = 0, in_page = 0;
    bool write_kv = true;
    if (APPEND) {
        const int64_t slot = live ? __ldg(a.slots + n) : -1;
        write_kv = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots) atomicOr(&g_rot_error_word, CLIS_PAGED_INDEX_BIT);
        page = slot >> a.page_shift;
        in_page = slot & ((int64_t(1) << a.page_shift) - 1);
    }
    for (int i = angles ? threadIdx.x : a.pairs; i < a.pairs; i += kRotThreads) {
        // Frequency as a fraction of a turn per position, 64-bit fixed point.
        double t = a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        t -= floor(t);
        s_step[i] = __double2ull_rn(t * 18446744073709551616.0);
        const int ax = a.axis[i];
        if (ax < 0 || ax >= a.axes) atomicOr(&g_rot_error_word, CLIS_PAGED_INDEX_BIT);
        s_axis[i] = ax;
    }
    __syncthreads();
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (!angles || (e < 4 ? !turn0 : !turn1)) continue;
        const int pr = e < 4 ? p0 + e : p1 + e - 4;
        const int ax = s_axis[pr];
        // (an axis index out of range turns by nothing)
        const int p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : ax == 3 ? pos[3] : 0;
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(p)) * s_step[pr];
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn[e], &cs[e]);
        if (a.inverse) sn[e] = -sn[e];
    }
    const bool turns = turn0 || turn1;
#pragma unroll 1
    for (int h = h0; h < h1; h += kHeadBatch) {
#pragma unroll
        for (int i = 0; i < kHeadBatch; i++) {
            const int hh = h + i;
            if (hh >= h1) continue;
            uint16_t *dst;
            bool turn = turns;
            if (hh < a.Hq) {
                dst = a.qo + b * a.qo_sb + hh * a.qo_sh + n * a.qo_sn;
            } else if (!APPEND) {
                dst = a.ko + b * a.ko_sb + (hh - a.Hq) * a.ko_sh + n * a.ko_sn;
            } else {
                if (!write_kv) continue;
                const int kh = hh - a.Hq;
                if constexpr (CODE >= 0) {
                    const bool is_k = kh < a.Hk;
                    const int vh = kh - a.Hk;
                    float f0[8], f1[8];
                    rotate8f<DT>(u0[i], u1[i], f0, f1, cs, sn, inter, is_k && turn0, is_k && turn1);
                    uint8_t *to = is_k ? reinterpret_cast<uint8_t *>(a.ko) + page * a.ko_sb + kh * a.ko_sh + in_page * a.ko_sn
                                       : reinterpret_cast<uint8_t *>(a.vo) + page * a.vo_sb + vh * a.vo_sh + in_page * a.vo_sn;
                    float *sc = is_k ? a.ks + page * a.ks_sp + kh * a.ks_sh + in_page * a.ks_sn
                                     : a.vs + page * a.vs_sp + vh * a.vs_sh + in_page * a.vs_sn;
                    store_codes<CODE, NC>(f0, f1, to, e0, e1, sc);
                    continue;
                }
                if (kh < a.Hk) {
                    dst = a.ko + page * a.ko_sb + kh * a.ko_sh + in_page * a.ko_sn;
                } else {  // v is copied as it is
                    dst = a.vo + page * a.vo_sb + (kh - a.Hk) * a.vo_sh + in_page * a.vo_sn;
                    turn = false;
                }
            }
            if (turn) rotate8<DT>(u0[i], u1[i], cs, sn, inter, turn0, turn1);
            *reinterpret_cast<uint4 *>(dst + e0) = u0[i];
            *reinterpret_cast<uint4 *>(dst + e1) = u1[i];
        }
        load(h + kHeadBatch);
    }
    if (MODE == 0) pdl_wait();  // (a write of codes beside it)
}

// A write of codes beside q's rotation: a launch each, since q's kernel has three blocks an SM
// and the other two.  Worth a second launch from 32 blocks of rows on where q has most of the
// heads (32 and 8, d = 128: 1,024 rows 12.6 us together, 11.2 apart; 8,192 45.4 and 41.2; 512 rows 8.5
// and 10.5; 8,192 rows of 32 and 32 heads 85.6 and 86.8).
template <int DT, int NC>
cudaError_t launch_codes_and_q(const RotArgs &a, int blocks, cudaStream_t stream)
{
    constexpr int KV = 8, Q = 16;  // heads per thread
    RotArgs kv = a, q = a;
    kv.Hq = 0;
    q.Hk = 0;
    q.slots = nullptr;
    const auto codes = a.code == CLIS_CODE_INT8 ? rot_kernel<DT, NC, 2> : rot_kernel<DT, NC, 3>;
    codes<<<dim3(blocks, (2 * a.Hk + KV - 1) / KV), kRotThreads, 0, stream>>>(kv, KV);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(rot_kernel<DT, NC, 0>, dim3(blocks, (a.Hq + Q - 1) / Q), kRotThreads, 0, stream, q, Q);
}

template <int DT, int NC>
cudaError_t launch_rot_impl(const RotArgs &a, dim3 grid, int hg, cudaStream_t stream)
{
    if (a.slots && a.code >= 0 && a.Hq >= 4 * a.Hk && grid.x >= 32) return launch_codes_and_q<DT, NC>(a, grid.x, stream);
    if (!a.slots)
        rot_kernel<DT, NC, 0><<<grid, kRotThreads, 0, stream>>>(a, hg);
    else if (a.code < 0)
        rot_kernel<DT, NC, 1><<<grid, kRotThreads, 0, stream>>>(a, hg);
    else if (a.code == CLIS_CODE_INT8)
        rot_kernel<DT, NC, 2><<<grid, kRotThreads, 0, stream>>>(a, hg);
    else
        rot_kernel<DT, NC, 3><<<grid, kRotThreads, 0, stream>>>(a, hg);
    return cudaGetLastError();
}

}  // namespace

clis_status_t launch_rot(const RotArgs &a, cudaStream_t stream)
{
    const int heads = a.Hq + (a.slots ? 2 : 1) * a.Hk;
    const int64_t threads = static_cast<int64_t>(a.B) * a.N * (a.d / 16);
    if (threads == 0 || heads == 0) return CLIS_OK;
    const int64_t blocks = (threads + kRotThreads - 1) / kRotThreads;
    // Heads per thread: sin and cos are shared by them, so 16, fewer where that
    // leaves the GPU without a few blocks per SM.  (8,192 rows of 48 heads into a
    // cache: 39.8 us with 16, 41.5 with 12, 45.5 with 4 or 24; 480p video q and k, 40
    // heads of 32,760 rows: 102.7 us with 16, 103.5 with 12, 108.2 with all.)
    int hg = 16;
    while (hg > kHeadBatch && blocks * ((heads + hg - 1) / hg) < 152 * 4) hg /= 2;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + hg - 1) / hg));
    cudaError_t e;
    if (a.d == 128)
        e = a.dtype == CLIS_DT_FP16 ? launch_rot_impl<1, 8>(a, grid, hg, stream)
                                    : launch_rot_impl<0, 8>(a, grid, hg, stream);
    else
        e = a.dtype == CLIS_DT_FP16 ? launch_rot_impl<1, 4>(a, grid, hg, stream)
                                    : launch_rot_impl<0, 4>(a, grid, hg, stream);
    return e == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t read_rot_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_rot_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_rot_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_rot_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
