// paged_decode.cu -- attention of a few new query rows per sequence (single
// tokens, drafted tokens) over a paged key/value cache.
//
//   x_ij = scale_log2 * q_i . k_j,  o_i = sum_j 2^(x_ij - m_i) v_j / sum_j 2^(x_ij - m_i)
//
// over the keys j < visible(i), with the running shift m_i raised only when a
// row's maximum outgrew it by 2^8 (the rescale is then rare).
//
// Bound: the cache's bytes.  All n * g query rows of a (sequence, key/value
// head) pair share each key and value that is loaded, in one m16n8k16 row tile
// (MT = 1) or two (MT = 2); 16 rows cost 64 flops per byte of cache, far below
// what even the warp-level matrix instructions deliver, so the tensor cores of
// the chunk kernel would gain nothing here.
//
//  * Work: paged_sched.h lays all items' units (16 keys, 32 at d = 64) end to end
//    and gives every warp an equal run, so ragged lengths balance; an item that
//    crosses a cut leaves partial results (unnormalised o, m, l) that
//    paged_decode_join_kernel adds in a fixed order.  A warp works alone: no
//    barrier, and items that end inside its run are written from registers.
//    (With a block of four warps per item, which then had to join its warps'
//    results, 1,000 sequences of 70 keys took 140 us.)
//  * Loads: each warp runs its own ring of cp.async stages of 8 KB, on into the next
//    item, so item ends do not drain it.  Rows past the length are filled with
//    zeros by the copy itself: what a page holds behind the last key is never
//    multiplied (0 * NaN would be NaN).
//  * P is rounded to the data type as the matrix instructions take it (off by up to
//    2^-8 of each weight in bf16, 2^-11 in fp16); the row sum adds the unrounded values,
//    and o, m, l stay in fp32.  fp16 ends at 2^-24, so there the shift stands 2^7 below
//    the row's maximum and weights reach up to 2^15 (weight_room in paged_sched.h).
//
// 64 requests of 1,000 to 16,000 keys (8 key/value heads, d = 128, 2.13 GB): 315 to 323
// us with the join (5 us), 97 to 100% of the measured copy rate.
#include <cuda_bf16.h>

#include "paged_warp.cuh"

namespace clis {

__device__ unsigned int g_decode_error_word = 0;

namespace {

constexpr int kWarps = kDecodeWarps;
constexpr int kThreads = kDecodeThreads;
constexpr float kTau = 8.0f;

template <int D>
struct DCfg {
    static constexpr int TK = decode_keys(D);           // keys per unit
    static constexpr int NST = 3;
    static constexpr int ROW = D * 2;                   // bytes of a row
    static constexpr int HALF = TK * ROW;               // K (or V) of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int SMEM = kWarps * NST * STAGE;
};

// Clears the non-finite halves of a pair; true if there was one.
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

template <int D, int DT, int MT>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_kernel(const DecodeParams p)
{
    using C = DCfg<D>;
    const PagedArgs &a = p.a;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_sum[kWarps];
    __shared__ int s_seq[kWarps];
    __shared__ uint64_t s_rel[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned int bad = 0;
    pdl_launch();

    const Runs runs = block_runs<C::TK, kWarps>(p, s_sum, s_seq, s_rel, bad);
    const uint64_t U = runs.U;
    const int nb = runs.nb;
    const int c = warp * gridDim.x + blockIdx.x;  // this worker
    if (lane == 0) p.meta[c] = make_int4(0, 0, 0, 0);
    if (bad && blockIdx.x == 0) atomicOr(&g_decode_error_word, bad);
    bad = 0;
    if (c >= nb) {  // nothing for this warp (U = 0 included)
        pdl_wait();
        return;
    }
    const uint64_t u0 = decode_cut(U, nb, c), u1 = decode_cut(U, nb, c + 1);

    Pos<C::TK> cur;
    cur.set(a, s_seq[warp], p.g);
    cur.h = static_cast<int>(div64(s_rel[warp], cur.units));
    cur.j = static_cast<int>(s_rel[warp] - static_cast<uint64_t>(cur.h) * cur.units);
    cur.left = static_cast<uint32_t>(u1 - u0);

    // ---- loader: one stage per unit, `ld` runs NST - 1 units ahead of `cur`
    constexpr int CPR = D / 8;         // 16-byte chunks per row
    constexpr int RPI = 32 / CPR;      // rows per copy instruction
    constexpr int NCP = C::TK / RPI;
    const uint32_t ring = smem_u32(smem) + warp * C::NST * C::STAGE;
    const int key_mask = (1 << a.page_shift) - 1;
    const int lrow = lane / CPR, lchunk = lane % CPR;
    Pos<C::TK> ld = cur;
    int ld_stage = 0;
    // Page of the lane's key of the tile that the loader is at, read one unit ahead.  What
    // the table holds is looked at when it is used (any number can stand there, so none
    // can say that there is no key: `lane_key` does).
    auto lane_key = [&](const Pos<C::TK> &q) { return q.j * C::TK + (lane & (C::TK - 1)); };
    auto page_at = [&](const Pos<C::TK> &q) -> int {
        const int key = lane_key(q);
        if (q.left == 0 || key >= q.q.kv) return -1;
        return __ldg(a.block_table + q.s * a.bt_s + (key >> a.page_shift));
    };
    int page = page_at(ld);
    auto load_step = [&]() {
        if (ld.left > 0) {
            if (page < 0 || page >= a.num_pages) {
                if (lane_key(ld) < ld.q.kv) bad |= CLIS_PAGED_INDEX_BIT;
                page = -1;  // its keys read as zeros
            }
            const uint32_t dst = ring + ld_stage * C::STAGE;
            const int key0 = ld.j * C::TK;
#pragma unroll
            for (int i = 0; i < NCP; i++) {
                const int row = i * RPI + lrow;
                const int pg = __shfl_sync(~0u, page, row);
                const bool ok = pg >= 0;
                const int64_t pi = ok ? pg : 0;
                const int in = ok ? (key0 + row) & key_mask : 0;
                const uint16_t *ks = a.kc + pi * a.kc_sp + ld.h * a.kc_sh + in * a.kc_sn + lchunk * 8;
                const uint16_t *vs = a.vc + pi * a.vc_sp + ld.h * a.vc_sh + in * a.vc_sn + lchunk * 8;
                const uint32_t at = row * C::ROW + ((lchunk ^ (row & 7)) << 4);
                cp_async16(dst + at, ks, ok ? 16 : 0);
                cp_async16(dst + C::HALF + at, vs, ok ? 16 : 0);
            }
            ld_stage = ld_stage + 1 == C::NST ? 0 : ld_stage + 1;
            ld.left--;
            if (++ld.j == ld.units && ld.left > 0) ld.next_item(a, p.g, p.rows_max);
            page = page_at(ld);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < C::NST - 1; i++) load_step();

    const float sl2 = a.scale_log2;
    const int r4 = lane >> 2, c2 = (lane & 3) * 2;
    int stage = 0;

    while (cur.left > 0) {
        // ---- one item, units j0 .. j1 - 1 of it
        const int j0 = cur.j;
        const int j1 = static_cast<int>(min(static_cast<uint32_t>(cur.units), j0 + cur.left));
        const int n = cur.q.n, kv = cur.q.kv, R = n * p.g, q0 = cur.q.q0;
        const int lim0 = visible_keys(n, kv, 0, a.causal);  // keys that every row sees

        uint32_t qf[MT][D / 16][4];
        int lim[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int row = mt * 16 + hf * 8 + r4;
                const bool ok = row < R;
                const int tok = ok ? row / p.g : 0, hd = cur.h * p.g + (ok ? row - tok * p.g : 0);
                lim[mt][hf] = ok ? visible_keys(n, kv, tok, a.causal) : 0;
                const uint16_t *src = a.q + static_cast<int64_t>(q0 + tok) * a.q_st + hd * a.q_sh + c2;
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
                    qf[mt][ks][hf] = ok ? __ldg(reinterpret_cast<const uint32_t *>(src + ks * 16)) : 0u;
                    qf[mt][ks][hf + 2] = ok ? __ldg(reinterpret_cast<const uint32_t *>(src + ks * 16 + 8)) : 0u;
                }
            }
        float o[MT][D / 8][4];
        float m_run[MT][2], l_run[MT][2], l_low[MT][2];  // l_low: what the last addition to l_run gained by rounding
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            m_run[mt][0] = m_run[mt][1] = -INFINITY;
            l_run[mt][0] = l_run[mt][1] = l_low[mt][0] = l_low[mt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; i++) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
        }
        bool dirty = false;

        for (int j = j0; j < j1; j++) {
            cp_async_wait<C::NST - 2>();
            __syncwarp();
            load_step();  // into the stage that the previous unit has been read from
            const int key0 = j * C::TK;
            const uint32_t sK = ring + stage * C::STAGE, sV = sK + C::HALF;
            stage = stage + 1 == C::NST ? 0 : stage + 1;
            if (key0 >= kv) continue;

            // S = Q K^T: 16 rows x TK keys per row tile
            constexpr int NB = C::TK / 8, KB = C::TK / 16;  // key blocks of 8 and of 16
            float s[MT][NB][4];
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int i = 0; i < NB; i++) s[mt][i][0] = s[mt][i][1] = s[mt][i][2] = s[mt][i][3] = 0.f;
            {
                const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
                const uint32_t base = sK + kr * C::ROW;
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
#pragma unroll
                    for (int kb = 0; kb < KB; kb++) {
                        uint32_t kf[4];
                        ldsm4(base + kb * 16 * C::ROW + (((ks * 2 + kc) ^ (kr & 7)) << 4), kf);
#pragma unroll
                        for (int mt = 0; mt < MT; mt++) {
                            mma16816<DT>(s[mt][2 * kb], qf[mt][ks], kf[0], kf[1]);
                            mma16816<DT>(s[mt][2 * kb + 1], qf[mt][ks], kf[2], kf[3]);
                        }
                    }
                }
            }
            const bool edge = key0 + C::TK > lim0;  // some row does not see some key
            if (edge) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int i = 0; i < NB; i++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (key0 + i * 8 + c2 + (e & 1) >= lim[mt][e >> 1]) s[mt][i][e] = -INFINITY;
            }
            float mx[MT][2];
            bool grow = false;
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float v = fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]);
#pragma unroll
                    for (int i = 1; i < NB; i++) v = fmax3(v, s[mt][i][2 * hf], s[mt][i][2 * hf + 1]);
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
                    mx[mt][hf] = v * sl2;
                    grow |= mx[mt][hf] > m_run[mt][hf] + (kTau + weight_room(DT));
                }
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        if (mx[mt][hf] > m_run[mt][hf] + (kTau + weight_room(DT))) {
                            const float m = mx[mt][hf] - weight_room(DT);
                            const float al = ex2_approx(m_run[mt][hf] - m);
                            m_run[mt][hf] = m;
                            l_run[mt][hf] *= al;
                            l_low[mt][hf] *= al;
#pragma unroll
                            for (int i = 0; i < D / 8; i++) {
                                o[mt][i][2 * hf] *= al;
                                o[mt][i][2 * hf + 1] *= al;
                            }
                        }
                    }
            }
            uint32_t pf[MT][KB][4];
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const float ns = m_run[mt][hf] == -INFINITY ? 0.f : -m_run[mt][hf];
                    float l = 0.f;
#pragma unroll
                    for (int i = 0; i < NB; i++) {
                        const float p0 = ex2_approx(fmaf(s[mt][i][2 * hf], sl2, ns));
                        const float p1 = ex2_approx(fmaf(s[mt][i][2 * hf + 1], sl2, ns));
                        l += p0 + p1;
                        pf[mt][i >> 1][2 * (i & 1) + hf] = pack2<DT>(p0, p1);
                    }
                    // Compensated: a run may be many thousands of units, each far below the sum.
                    const float y = l - l_low[mt][hf], t = l_run[mt][hf] + y;
                    l_low[mt][hf] = (t - l_run[mt][hf]) - y;
                    l_run[mt][hf] = t;
                }
            // O += P V
            {
                const int vr = lane & 15, vc = lane >> 4;
                const uint32_t base = sV + vr * C::ROW;
                auto pv = [&](bool clean) {
#pragma unroll
                    for (int kb = 0; kb < KB; kb++)
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            uint32_t vf[4];
                            ldsm4_t(base + kb * 16 * C::ROW + (((i * 2 + vc) ^ (vr & 7)) << 4), vf);
                            if (clean)
#pragma unroll
                                for (int e = 0; e < 4; e++) dirty |= scrub<DT>(vf[e]);
#pragma unroll
                            for (int mt = 0; mt < MT; mt++) {
                                mma16816<DT>(o[mt][2 * i], pf[mt][kb], vf[0], vf[1]);
                                mma16816<DT>(o[mt][2 * i + 1], pf[mt][kb], vf[2], vf[3]);
                            }
                        }
                };
                // Where a key is masked for some rows only, a non-finite v of it must
                // not reach them as 0 * inf: it is left out of the product and added to
                // the rows that see it at the end.
                if (edge && lim0 < kv) pv(true);
                else pv(false);
            }
        }

        // ---- write the rows: final, or partial
        const bool any_dirty = __any_sync(~0u, dirty);
        const bool whole = j0 == 0 && j1 == cur.units;
        const int64_t slot = 2 * static_cast<int64_t>(c) + (j0 == 0 ? 1 : 0);
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int row = mt * 16 + hf * 8 + r4;
                float l = l_run[mt][hf];
                l += __shfl_xor_sync(~0u, l, 1);
                l += __shfl_xor_sync(~0u, l, 2);
                if (row >= R) continue;
                const int tok = row / p.g, hd = cur.h * p.g + (row - tok * p.g);
                if (any_dirty) {
                    // Non-finite values of keys that this row sees and that were left out.
                    const int see = min(lim[mt][hf], j1 * C::TK);
#pragma unroll 1
                    for (int key = max(lim0 / C::TK * C::TK, j0 * C::TK); key < see; key++) {
                        const int pg = __ldg(a.block_table + cur.s * a.bt_s + (key >> a.page_shift));
                        if (pg < 0 || pg >= a.num_pages) continue;
                        const uint16_t *vs = a.vc + static_cast<int64_t>(pg) * a.vc_sp + cur.h * a.vc_sh +
                                             static_cast<int64_t>(key & key_mask) * a.vc_sn + c2;
#pragma unroll
                        for (int i = 0; i < D / 8; i++) {
                            const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(vs + i * 8));
                            const float x0 = elem_lo<DT>(u), x1 = elem_hi<DT>(u);
                            if (!isfinite(x0)) o[mt][i][2 * hf] += x0;
                            if (!isfinite(x1)) o[mt][i][2 * hf + 1] += x1;
                        }
                    }
                }
                const float m = m_run[mt][hf];
                if (whole) {
                    const float inv = 1.f / l;
                    uint16_t *dst = a.o + static_cast<int64_t>(q0 + tok) * a.o_st + hd * a.o_sh + c2;
#pragma unroll
                    for (int i = 0; i < D / 8; i++)  // (zeros for a row that sees no key)
                        *reinterpret_cast<uint32_t *>(dst + i * 8) =
                            l == 0.f ? 0u : pack2<DT>(o[mt][i][2 * hf] * inv, o[mt][i][2 * hf + 1] * inv);
                    if ((lane & 3) == 0 && a.lse2)
                        a.lse2[static_cast<int64_t>(q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : m + log2f(l);
                } else {
                    float *dst = p.part_o + (slot * p.rows_max + row) * D + c2;
#pragma unroll
                    for (int i = 0; i < D / 8; i++)
                        *reinterpret_cast<float2 *>(dst + i * 8) = make_float2(o[mt][i][2 * hf], o[mt][i][2 * hf + 1]);
                    if ((lane & 3) == 0) p.part_ml[slot * p.rows_max + row] = make_float2(m, l);
                }
            }
        if (!whole && j0 == 0 && lane == 0) {
            // The item's remaining units lie in the next workers' runs.
            const uint64_t end = u1 - cur.left + cur.units - 1;  // the item's last unit
            p.meta[c] = make_int4(item_parts(runs, c, end), q0, n, cur.h);
        }
        cur.left -= j1 - j0;
        cur.j = j1;
        if (cur.left > 0) cur.next_item(a, p.g, p.rows_max);
    }
    cp_async_wait<0>();
    if (bad) atomicOr(&g_decode_error_word, bad);
    pdl_wait();  // (the schedule kernel, whose results only later kernels read)
}

template <int D, int DT, int MT>
clis_status_t launch_impl(const DecodeParams &p, int grid, bool after_schedule, cudaStream_t stream)
{
    if (cudaFuncSetAttribute(paged_decode_kernel<D, DT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             DCfg<D>::SMEM) != cudaSuccess)
        return CLIS_ERR_CUDA;
    if (after_schedule) {
        if (launch_pdl(paged_decode_kernel<D, DT, MT>, dim3(grid), kThreads, DCfg<D>::SMEM, stream, p) != cudaSuccess)
            return CLIS_ERR_CUDA;
    } else {
        paged_decode_kernel<D, DT, MT><<<grid, kThreads, DCfg<D>::SMEM, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    }
    return launch_join<D, DT>(p, stream) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace

int paged_decode_row_tiles(int64_t max_q, int g, int d)
{
    // Rows of the largest sequence if it is small; else those of single tokens.  Two
    // row tiles at d = 128 would spill registers (64 sequences of 8,000 keys and 32
    // rows: 661 us, the chunk kernel 415 us): not built.
    const int most = d == 64 ? 32 : 16;
    const int64_t rows = max_q <= most && max_q * g <= most ? max_q * g : g;
    return rows <= 16 ? 1 : rows <= most ? 2 : 0;
}

size_t paged_decode_workspace(int d, int row_tiles, int nsm)
{
    if (row_tiles == 0) return 0;
    return parts_workspace(2 * static_cast<size_t>(nsm) * kWarps, 16 * static_cast<size_t>(row_tiles), d);
}

clis_status_t launch_paged_decode(const PagedArgs &a, int row_tiles, bool strict, bool after_schedule, void *workspace,
                                  int nsm, cudaStream_t stream)
{
    const int grid = 2 * nsm;  // two blocks fit an SM
    DecodeParams p;
    p.a = a;
    p.g = a.H / a.Hkv;
    p.least = 2;  // units of a worker's run: one token over 301 keys 12.8 us with 2, 14 with 1 or 4, 16.5 with 8
    p.strict = strict;
    place_parts(p, static_cast<size_t>(grid) * kWarps, 16 * static_cast<size_t>(row_tiles), workspace);
#define CLIS_DECODE(D, MT)                                                  \
    return a.dtype == CLIS_DT_FP16 ? launch_impl<D, 1, MT>(p, grid, after_schedule, stream) \
                                   : launch_impl<D, 0, MT>(p, grid, after_schedule, stream)
    if (a.d == 128) CLIS_DECODE(128, 1);
    if (row_tiles == 1) CLIS_DECODE(64, 1);
    CLIS_DECODE(64, 2);
#undef CLIS_DECODE
}

clis_status_t read_decode_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_decode_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_decode_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_decode_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
