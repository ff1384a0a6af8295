// paged_q8.cu -- attention of a few new query rows per sequence over a paged
// key/value cache held in 8 bits (int8 or E4M3 codes, one fp32 scale per token and
// key/value head for K and one for V).
//
//   x_ij = scale_log2 * ks_j * (q_i . kc_j),  o_i = sum_j 2^(x_ij) vs_j vc_j / sum_j 2^(x_ij)
//
// with the codes kc, vc and the scales ks, vs.  The codes go into the products as
// they are (both kinds are exact in fp16); the scales are applied to the scores and
// to the weights, one multiplication per query row and key instead of one per element.
//
// Bound: the cache's bytes, half of those of paged_decode.cu, and then the issue
// slots: per 8 KB of codes (32 keys at d = 128) a warp spends about 600 instructions
// on 16 query rows, two thirds of them on turning codes into fp16 pairs, about half of
// what an SM can issue while these bytes arrive.
//
//  * Work, runs and joins: as in paged_decode.cu.  A team of RT = 1, 2 or 4 warps
//    (16 query rows each) shares one ring of stages, so 17 to 64 rows (drafted tokens)
//    read the cache once as well; RT = 1 needs no barrier.
//  * int8 to fp16: the byte with its sign bit flipped is put below 0x64, which reads
//    1024 + 128 + code, and 1152 is subtracted: exact, and the byte permutation does
//    the transposition of V's pairs on the way.  E4M3 has its own instruction.
//  * The contraction over d takes the elements in the order in which a thread's
//    16-byte load of codes holds them; q's fragments are laid out the same way.
//  * q is scaled by a power of two per row so that its largest magnitude is between
//    2^14 and 2^15 and goes into fp16: exact for fp16 and bf16 values down to 2^-30 of
//    the row's largest.
//  * The weights of V carry vs_j, whose range has nothing to do with the softmax's, so
//    they have a shift of their own: w_ij = 2^(x_ij + log2(vs_j) - m'_i) with the running
//    maximum m'_i of the exponent, next to m_i for the row sum.  Both are raised
//    lazily.  w is rounded to fp16 as the matrix instructions take it (off by up to
//    2^-11, and by 2^-32 of the row's largest below that: weight_room in paged_sched.h).
#include <cuda_fp16.h>

#include "paged_warp.cuh"

namespace clis {

__device__ unsigned int g_q8_error_word = 0;

namespace {

constexpr float kTau = 8.0f;
constexpr float kRoom = weight_room(1);

template <int D, int RT>
struct QCfg {
    static constexpr int TK = 4096 / D;                  // keys per unit: 8 KB of codes
    static constexpr int TEAMS = kDecodeWarps / RT;
    static constexpr int NST = 3 * RT;
    static constexpr int HALF = TK * D;                  // bytes of K (or V) of a stage
    static constexpr int SCALES = 2 * HALF;              // [2][TK] floats behind the codes
    static constexpr int STAGE = 2 * HALF + 2 * TK * 4;
    static constexpr int SMEM = TEAMS * NST * STAGE;
};

// Place of a 16-byte chunk of a row of codes in its stage.  K is read by 16-byte loads
// of four threads per row, V by ldmatrix (8 rows, one chunk): either way a quarter warp
// touches all banks once.
template <int D>
__device__ __forceinline__ uint32_t at_k(int row, int chunk)
{
    return row * D + ((D == 128 ? chunk ^ ((row & 1) << 2) : chunk) << 4);
}

template <int D>
__device__ __forceinline__ uint32_t at_v(int row, int chunk)
{
    return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ float lg2_approx(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t lo16)
{
    uint32_t r;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(lo16));
    return r;
}

// Four codes of a word as two fp16 pairs: bytes (0, 1) and (2, 3), or TRANS: (0, 2) and
// (1, 3), the pairs of a transposed load.
template <int CODE, bool TRANS>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t &a, uint32_t &b)
{
    if (CODE == CLIS_CODE_INT8) {
        const uint32_t u = w ^ 0x80808080u;
        a = hsub2u(__byte_perm(u, 0x64646464u, TRANS ? 0x4240 : 0x4140), 0x64806480u);
        b = hsub2u(__byte_perm(u, 0x64646464u, TRANS ? 0x4341 : 0x4342), 0x64806480u);
    } else {
        if (TRANS) w = __byte_perm(w, 0, 0x3120);
        a = e4m3_pair(w & 0xFFFFu);
        b = e4m3_pair(w >> 16);
    }
}

// Clears the NaN halves of an fp16 pair; true if there was one.
__device__ __forceinline__ bool scrub(uint32_t &u)
{
    uint32_t keep = 0xFFFFFFFFu;
    if ((u & 0x7C00u) == 0x7C00u) keep &= 0xFFFF0000u;
    if (((u >> 16) & 0x7C00u) == 0x7C00u) keep &= 0x0000FFFFu;
    u &= keep;
    return keep != 0xFFFFFFFFu;
}

template <int RT>
__device__ __forceinline__ void team_sync(int team)
{
    if (RT == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(RT * 32) : "memory");
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

template <int D, int DT, int CODE, int RT>
__global__ void __launch_bounds__(kDecodeThreads, 2) paged_q8_kernel(const DecodeParams p, const QuantArgs z)
{
    using C = QCfg<D, RT>;
    constexpr int TK = C::TK, NB = TK / 8, KB = TK / 16;
    const PagedArgs &a = p.a;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_sum[kDecodeWarps];
    __shared__ int s_seq[C::TEAMS];
    __shared__ uint64_t s_rel[C::TEAMS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / RT, mt = warp % RT;  // this warp has rows 16 mt .. 16 mt + 15 of its team's items
    unsigned int bad = 0;
    pdl_launch();

    const Runs runs = block_runs<TK, C::TEAMS>(p, s_sum, s_seq, s_rel, bad);
    const int c = team * gridDim.x + blockIdx.x;  // this worker
    if (lane == 0 && mt == 0) p.meta[c] = make_int4(0, 0, 0, 0);
    if (bad && blockIdx.x == 0) atomicOr(&g_q8_error_word, bad);
    bad = 0;
    if (c >= runs.nb) {  // nothing for this team (U = 0 included)
        pdl_wait();
        return;
    }
    const uint64_t u0 = decode_cut(runs.U, runs.nb, c), u1 = decode_cut(runs.U, runs.nb, c + 1);

    Pos<TK> cur;
    cur.set(a, s_seq[team]);
    cur.h = static_cast<int>(div64(s_rel[team], cur.units));
    cur.j = static_cast<int>(s_rel[team] - static_cast<uint64_t>(cur.h) * cur.units);
    cur.left = static_cast<uint32_t>(u1 - u0);

    // ---- loader: one stage per unit, `ld` runs NST - 1 units ahead of `cur`; the team's
    // warps share out the rows
    constexpr int CPR = D / 16;           // 16-byte chunks per row
    constexpr int RPI = 32 / CPR;         // rows per copy instruction
    constexpr int NCP = TK / RT / RPI;
    constexpr int KPL = TK / 32;          // keys per lane of the page lookup (one page: at least 8 keys)
    const uint32_t ring = smem_u32(smem) + team * C::NST * C::STAGE;
    const uint8_t *ring_ptr = smem + team * C::NST * C::STAGE;
    const int key_mask = (1 << a.page_shift) - 1;
    const int lrow = mt * (TK / RT) + lane / CPR, lchunk = lane % CPR;
    Pos<TK> ld = cur;
    int ld_stage = 0;
    auto lane_key = [&](const Pos<TK> &q) { return q.j * TK + lane * KPL; };
    auto page_at = [&](const Pos<TK> &q) -> int {
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
            const int key0 = ld.j * TK;
#pragma unroll
            for (int i = 0; i < NCP; i++) {
                const int row = i * RPI + lrow;
                const int pg = __shfl_sync(~0u, page, row / KPL);
                const bool ok = pg >= 0 && key0 + row < ld.q.kv;
                const int64_t pi = ok ? pg : 0;
                const int in = ok ? (key0 + row) & key_mask : 0;
                cp_async16(dst + at_k<D>(row, lchunk), z.kc + pi * a.kc_sp + ld.h * a.kc_sh + in * a.kc_sn + lchunk * 16, ok ? 16 : 0);
                cp_async16(dst + C::HALF + at_v<D>(row, lchunk), z.vc + pi * a.vc_sp + ld.h * a.vc_sh + in * a.vc_sn + lchunk * 16,
                           ok ? 16 : 0);
            }
            // Scales: K's by the team's first warp, V's by its last.
#pragma unroll
            for (int i = 0; i < KPL; i++) {
                const bool ok = page >= 0 && key0 + lane * KPL + i < ld.q.kv;
                const int64_t pi = ok ? page : 0;
                const int in = ok ? (key0 + lane * KPL + i) & key_mask : 0;
                const uint32_t to = dst + C::SCALES + (lane * KPL + i) * 4;
                if (mt == 0) cp_async4(to, z.ks + pi * z.ks_sp + ld.h * z.ks_sh + in * z.ks_sn, ok ? 4 : 0);
                if (mt == RT - 1) cp_async4(to + TK * 4, z.vs + pi * z.vs_sp + ld.h * z.vs_sh + in * z.vs_sn, ok ? 4 : 0);
            }
            ld_stage = ld_stage + 1 == C::NST ? 0 : ld_stage + 1;
            ld.left--;
            if (++ld.j == ld.units && ld.left > 0) ld.next_item(a, p.g, p.rows_max);
            page = page_at(ld);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < C::NST - 1; i++) load_step();

    const int r4 = lane >> 2, t4 = lane & 3, c2 = t4 * 2;
    int stage = 0;

    while (cur.left > 0) {
        // ---- one item, units j0 .. j1 - 1 of it
        const int j0 = cur.j;
        const int j1 = static_cast<int>(min(static_cast<uint32_t>(cur.units), j0 + cur.left));
        const int n = cur.q.n, kv = cur.q.kv, R = n * p.g, q0 = cur.q.q0;
        const int lim0 = visible_keys(n, kv, 0, a.causal);  // keys that every row sees
        const bool live = mt * 16 < R;                      // (the team's barriers are met either way)

        // q's rows r4 and r4 + 8 of this tile: word w of a row's thread t4 holds elements
        // 16 t4 + 4 w .. (w < 4) or 64 + 16 t4 + 4 (w - 4) .. of d.
        uint32_t qf[D / 16][4];
        int lim[2];
        float cs[2];  // scale_log2 over the power of two that q's row was multiplied by
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
            const int row = mt * 16 + hf * 8 + r4;
            const bool ok = row < R;
            const int tok = ok ? row / p.g : 0, hd = cur.h * p.g + (ok ? row - tok * p.g : 0);
            lim[hf] = ok ? visible_keys(n, kv, tok, a.causal) : 0;
            const uint16_t *src = a.q + static_cast<int64_t>(q0 + tok) * a.q_st + hd * a.q_sh + t4 * 16;
            uint32_t u[D / 16][2];
#pragma unroll
            for (int w = 0; w < D / 16; w += 2) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4 *>(src + (w >> 2) * 64 + (w & 3) * 4)) : make_uint4(0, 0, 0, 0);
                u[w][0] = v.x;
                u[w][1] = v.y;
                u[w + 1][0] = v.z;
                u[w + 1][1] = v.w;
            }
            uint32_t top = 0;  // the row's largest magnitude: bits of non-negative floats are ordered
#pragma unroll
            for (int w = 0; w < D / 16; w++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    top = max(top, __float_as_uint(elem_lo<DT>(u[w][e])) & 0x7FFFFFFFu);
                    top = max(top, __float_as_uint(elem_hi<DT>(u[w][e])) & 0x7FFFFFFFu);
                }
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // (a row of zeros or with something non-finite is taken as it is)
            const int e = top == 0 || top >= 0x7F800000u ? 0 : min(14 - (static_cast<int>(top >> 23) - 127), 126);
            const float f = exp2_int(e);
            cs[hf] = a.scale_log2 * exp2_int(-e);
#pragma unroll
            for (int w = 0; w < D / 16; w++) {
                qf[w][hf] = pack2<1>(elem_lo<DT>(u[w][0]) * f, elem_hi<DT>(u[w][0]) * f);
                qf[w][hf + 2] = pack2<1>(elem_lo<DT>(u[w][1]) * f, elem_hi<DT>(u[w][1]) * f);
            }
        }
        // o[2 i], o[2 i + 1]: columns 16 i + 4 t4 + {0, 2} and + {1, 3} of rows r4 and r4 + 8.
        float o[D / 8][4];
        float m_run[2], l_run[2], l_low[2];  // l_low: what the last addition to l_run gained by rounding
        float m_val[2];                      // the shift of the weights of V
        m_run[0] = m_run[1] = m_val[0] = m_val[1] = -INFINITY;
        l_run[0] = l_run[1] = l_low[0] = l_low[1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        bool dirty = false;

#pragma unroll 1
        for (int j = j0; j < j1; j++) {
            cp_async_wait<C::NST - 2>();
            team_sync<RT>(team);
            load_step();  // into the stage that the previous unit has been read from
            const int key0 = j * TK;
            const uint8_t *sK = ring_ptr + stage * C::STAGE;
            const uint32_t sV = ring + stage * C::STAGE + C::HALF;
            const float *sS = reinterpret_cast<const float *>(sK + C::SCALES);
            stage = stage + 1 == C::NST ? 0 : stage + 1;
            if (key0 >= kv || !live) continue;

            // S = Q KC^T: 16 rows x TK keys
            float s[NB][4];
#pragma unroll
            for (int i = 0; i < NB; i++) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int hh = 0; hh < D / 64; hh++)
#pragma unroll
                for (int i0 = 0; i0 < NB; i0 += 4) {
                    uint4 kw[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        kw[i] = *reinterpret_cast<const uint4 *>(sK + at_k<D>((i0 + i) * 8 + r4, hh * 4 + t4));
#pragma unroll
                    for (int w = 0; w < 4; w++)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t b0, b1;
                            unpack<CODE, false>(w == 0 ? kw[i].x : w == 1 ? kw[i].y : w == 2 ? kw[i].z : kw[i].w, b0, b1);
                            mma16816<1>(s[i0 + i], qf[hh * 4 + w], b0, b1);
                        }
                }
            const bool edge = key0 + TK > lim0;  // some row does not see some key
            float mx[2] = {-INFINITY, -INFINITY}, my[2] = {-INFINITY, -INFINITY}, lv[NB][2];
#pragma unroll
            for (int i = 0; i < NB; i++) {
                const float2 ks = *reinterpret_cast<const float2 *>(sS + i * 8 + c2);
                const float2 vs = *reinterpret_cast<const float2 *>(sS + TK + i * 8 + c2);
                lv[i][0] = lg2_approx(vs.x);
                lv[i][1] = lg2_approx(vs.y);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[i][e] *= e & 1 ? ks.y : ks.x;
                    if (edge && key0 + i * 8 + c2 + (e & 1) >= lim[e >> 1]) s[i][e] = -INFINITY;
                }
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    mx[hf] = fmax3(mx[hf], s[i][2 * hf], s[i][2 * hf + 1]);
                    const float y0 = fmaf(s[i][2 * hf], cs[hf], lv[i][0]), y1 = fmaf(s[i][2 * hf + 1], cs[hf], lv[i][1]);
                    my[hf] = fmax3(my[hf], s[i][2 * hf] == -INFINITY ? -INFINITY : y0, s[i][2 * hf + 1] == -INFINITY ? -INFINITY : y1);
                }
            }
            bool grow = false;
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(~0u, mx[hf], 1));
                my[hf] = fmaxf(my[hf], __shfl_xor_sync(~0u, my[hf], 1));
                mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(~0u, mx[hf], 2)) * cs[hf];
                my[hf] = fmaxf(my[hf], __shfl_xor_sync(~0u, my[hf], 2));
                grow |= mx[hf] > m_run[hf] + kTau || my[hf] > m_val[hf] + (kTau + kRoom);
            }
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    if (mx[hf] > m_run[hf] + kTau) {
                        const float al = ex2_approx(m_run[hf] - mx[hf]);
                        m_run[hf] = mx[hf];
                        l_run[hf] *= al;
                        l_low[hf] *= al;
                    }
                    if (my[hf] > m_val[hf] + (kTau + kRoom)) {
                        const float m = my[hf] - kRoom;
                        const float al = ex2_approx(m_val[hf] - m);
                        m_val[hf] = m;
#pragma unroll
                        for (int i = 0; i < D / 8; i++) {
                            o[i][2 * hf] *= al;
                            o[i][2 * hf + 1] *= al;
                        }
                    }
                }
            }
            uint32_t pf[KB][4];
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const float ns = m_run[hf] == -INFINITY ? 0.f : -m_run[hf];
                const float nv = m_val[hf] == -INFINITY ? 0.f : -m_val[hf];
                float l = 0.f;
#pragma unroll
                for (int i = 0; i < NB; i++) {
                    const float x0 = s[i][2 * hf], x1 = s[i][2 * hf + 1];
                    l += ex2_approx(fmaf(x0, cs[hf], ns)) + ex2_approx(fmaf(x1, cs[hf], ns));
                    float w0 = ex2_approx(fmaf(x0, cs[hf], lv[i][0]) + nv), w1 = ex2_approx(fmaf(x1, cs[hf], lv[i][1]) + nv);
                    if (edge) {  // (a scale that is no number must not reach a row that does not see its key)
                        w0 = x0 == -INFINITY ? 0.f : w0;
                        w1 = x1 == -INFINITY ? 0.f : w1;
                    }
                    pf[i >> 1][2 * (i & 1) + hf] = pack2<1>(w0, w1);
                }
                // Compensated: a run may be many thousands of units, each far below the sum.
                const float y = l - l_low[hf], t = l_run[hf] + y;
                l_low[hf] = (t - l_run[hf]) - y;
                l_run[hf] = t;
            }
            // O += W VC: a transposed load gives 32 keys of 16 columns, in each word the codes
            // of two neighbouring columns and two neighbouring keys.
            auto pv = [&](bool clean) {
#pragma unroll
                for (int kb = 0; kb < KB; kb += 2)
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        uint32_t vw[4], b0[4], b1[4];
                        ldsm4_t(sV + at_v<D>(kb * 16 + lane, i), vw);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            unpack<CODE, true>(vw[e], b0[e], b1[e]);
                            if (CODE != CLIS_CODE_INT8 && clean) {
                                dirty |= scrub(b0[e]);
                                dirty |= scrub(b1[e]);
                            }
                        }
                        mma16816<1>(o[2 * i], pf[kb], b0[0], b0[1]);
                        mma16816<1>(o[2 * i + 1], pf[kb], b1[0], b1[1]);
                        mma16816<1>(o[2 * i], pf[kb + 1], b0[2], b0[3]);
                        mma16816<1>(o[2 * i + 1], pf[kb + 1], b1[2], b1[3]);
                    }
            };
            // Where a key is masked for some rows only, a NaN code of it must not reach them as
            // 0 * NaN: it is left out of the product and given to the rows that see it at the end.
            if (CODE != CLIS_CODE_INT8 && edge && lim0 < kv) pv(true);
            else pv(false);
        }

        // ---- write the rows: final, or partial
        const bool any_dirty = __any_sync(~0u, dirty);
        const bool whole = j0 == 0 && j1 == cur.units;
        const int64_t slot = 2 * static_cast<int64_t>(c) + (j0 == 0 ? 1 : 0);
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
            const int row = mt * 16 + hf * 8 + r4;
            float l = l_run[hf];
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            if (row >= R) continue;
            const int tok = row / p.g, hd = cur.h * p.g + (row - tok * p.g);
            if (CODE != CLIS_CODE_INT8 && any_dirty) {
                const int see = min(lim[hf], j1 * TK);
#pragma unroll 1
                for (int key = max(lim0 / TK * TK, j0 * TK); key < see; key++) {
                    const int pg = __ldg(a.block_table + cur.s * a.bt_s + (key >> a.page_shift));
                    if (pg < 0 || pg >= a.num_pages) continue;
                    const uint8_t *vs = z.vc + static_cast<int64_t>(pg) * a.vc_sp + cur.h * a.vc_sh +
                                        static_cast<int64_t>(key & key_mask) * a.vc_sn + 4 * t4;
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(vs + i * 16));
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (((u >> (8 * e)) & 0x7Fu) == 0x7Fu) o[2 * i + (e & 1)][2 * hf + (e >> 1)] = NAN;
                    }
                }
            }
            const float m = m_run[hf];
            // From the weights' shift to the row's.
            const float back = m_val[hf] == -INFINITY ? 0.f : ex2_approx(m_val[hf] - m);
            if (whole) {
                const float inv = l == 0.f ? 0.f : back / l;
                uint16_t *dst = a.o + static_cast<int64_t>(q0 + tok) * a.o_st + hd * a.o_sh + 4 * t4;
#pragma unroll
                for (int i = 0; i < D / 16; i++) {  // (zeros for a row that sees no key)
                    uint2 u = make_uint2(0u, 0u);
                    if (l != 0.f) {
                        u.x = pack2<DT>(o[2 * i][2 * hf] * inv, o[2 * i + 1][2 * hf] * inv);
                        u.y = pack2<DT>(o[2 * i][2 * hf + 1] * inv, o[2 * i + 1][2 * hf + 1] * inv);
                    }
                    *reinterpret_cast<uint2 *>(dst + i * 16) = u;
                }
                if (t4 == 0 && a.lse2) a.lse2[static_cast<int64_t>(q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : m + log2f(l);
            } else {
                float *dst = p.part_o + (slot * p.rows_max + row) * D + 4 * t4;
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    *reinterpret_cast<float4 *>(dst + i * 16) =
                        make_float4(o[2 * i][2 * hf] * back, o[2 * i + 1][2 * hf] * back, o[2 * i][2 * hf + 1] * back,
                                    o[2 * i + 1][2 * hf + 1] * back);
                if (t4 == 0) p.part_ml[slot * p.rows_max + row] = make_float2(m, l);
            }
        }
        if (!whole && j0 == 0 && lane == 0 && mt == 0) {
            const uint64_t end = u1 - cur.left + cur.units - 1;  // the item's last unit
            p.meta[c] = make_int4(item_parts(runs, c, end), q0, n, cur.h);
        }
        cur.left -= j1 - j0;
        cur.j = j1;
        if (cur.left > 0) cur.next_item(a, p.g, p.rows_max);
    }
    cp_async_wait<0>();
    if (bad) atomicOr(&g_q8_error_word, bad);
    pdl_wait();
}

template <int D, int DT, int CODE, int RT>
clis_status_t launch_impl(const DecodeParams &p, const QuantArgs &z, int grid, bool after_schedule, cudaStream_t stream)
{
    constexpr int smem = QCfg<D, RT>::SMEM;
    if (cudaFuncSetAttribute(paged_q8_kernel<D, DT, CODE, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return CLIS_ERR_CUDA;
    if (after_schedule) {
        if (launch_pdl(paged_q8_kernel<D, DT, CODE, RT>, dim3(grid), kDecodeThreads, smem, stream, p, z) != cudaSuccess)
            return CLIS_ERR_CUDA;
    } else {
        paged_q8_kernel<D, DT, CODE, RT><<<grid, kDecodeThreads, smem, stream>>>(p, z);
        if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    }
    return launch_join<D, DT>(p, stream) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

template <int D, int DT, int CODE>
clis_status_t launch_rows(const DecodeParams &p, const QuantArgs &z, int row_tiles, int grid, bool after_schedule, cudaStream_t stream)
{
    if (row_tiles == 1) return launch_impl<D, DT, CODE, 1>(p, z, grid, after_schedule, stream);
    if (row_tiles == 2) return launch_impl<D, DT, CODE, 2>(p, z, grid, after_schedule, stream);
    return launch_impl<D, DT, CODE, 4>(p, z, grid, after_schedule, stream);
}

template <int D>
clis_status_t launch_types(const DecodeParams &p, const QuantArgs &z, int row_tiles, int grid, bool after_schedule, cudaStream_t stream)
{
    const bool half = p.a.dtype == CLIS_DT_FP16;
    if (z.code == CLIS_CODE_INT8)
        return half ? launch_rows<D, 1, CLIS_CODE_INT8>(p, z, row_tiles, grid, after_schedule, stream)
                    : launch_rows<D, 0, CLIS_CODE_INT8>(p, z, row_tiles, grid, after_schedule, stream);
    return half ? launch_rows<D, 1, CLIS_CODE_E4M3>(p, z, row_tiles, grid, after_schedule, stream)
                : launch_rows<D, 0, CLIS_CODE_E4M3>(p, z, row_tiles, grid, after_schedule, stream);
}

}  // namespace

int paged_q8_row_tiles(int64_t max_q, int g)
{
    // Rows of the largest sequence if it is small; else those of single tokens.
    constexpr int most = 64;
    const int64_t rows = max_q <= most && max_q * g <= most ? max_q * g : g;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= most ? 4 : 0;
}

size_t paged_q8_workspace(int d, int row_tiles, int nsm)
{
    if (row_tiles == 0) return 0;
    return parts_workspace(2 * static_cast<size_t>(nsm) * kDecodeWarps / row_tiles, 16 * static_cast<size_t>(row_tiles), d);
}

clis_status_t launch_paged_q8(const PagedArgs &a, const QuantArgs &z, int row_tiles, bool strict, bool after_schedule,
                              void *workspace, int nsm, cudaStream_t stream)
{
    const int grid = 2 * nsm;  // two blocks fit an SM
    DecodeParams p;
    p.a = a;
    p.g = a.H / a.Hkv;
    p.least = 2;
    p.strict = strict;
    place_parts(p, static_cast<size_t>(grid) * kDecodeWarps / row_tiles, 16 * static_cast<size_t>(row_tiles), workspace);
    return a.d == 128 ? launch_types<128>(p, z, row_tiles, grid, after_schedule, stream)
                      : launch_types<64>(p, z, row_tiles, grid, after_schedule, stream);
}

clis_status_t read_q8_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_q8_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_q8_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_q8_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
