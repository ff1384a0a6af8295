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
// slots: turning 8 KB of codes into fp16 pairs alone takes a warp some 320 instructions.
//
//  * Work, runs and joins: as in paged_decode.cu.  A warp works alone, on 8, 16 or (d = 64)
//    24 query rows, NT = 1, 2 or 3 column tiles; a sequence of more rows (drafted tokens,
//    small chunks) is several items that read the same keys, one after the other, mostly from L2.  From 16
//    rows on what a warp does per unit is the time (850 instructions at NT = 2, two warps per
//    scheduler).  Larger tiles spill registers: 16, 32 and 64 rows of the 64 requests below 231, 460
//    and 920 us with tiles of 16; 413 and 783 with 32 of int8, but 526 and 979 of E4M3.  Teams of
//    four warps that convert a unit together into fp16 tiles in shared memory took 607 and 798.
//    Where the tables hold little, a block takes an item, each warp a quarter of its units, and
//    joins it in shared memory: no second launch.
//  * The products are taken transposed, S^T = KC Q^T and O^T += VC^T W^T: codes are the
//    16-row operand, query rows the 8-column one.  A single token's g query heads fill
//    4 or 8 of 8 places instead of 16, which halves the products, the weights and the
//    registers of O.  W^T comes out of S^T's registers by one 8 x 8 transposition each.
//  * int8 to fp16: the byte with its sign bit flipped is put below 0x64, which reads
//    1024 + 128 + code, and 1152 is subtracted: exact, and the byte permutation does
//    the transposition of V's pairs on the way.  E4M3 has its own instruction.
//  * The contraction over d takes the elements in the order in which a thread's
//    16-byte load of codes holds them; q's fragments are laid out the same way.
//  * Loads: a warp fetches its stages by TMA, page by page (a unit is 8 KB of
//    codes), the scales by 4-byte copies that arrive on the same barrier.  With 16-byte
//    copies by all lanes the addresses alone were a sixth of all instructions.
//  * q is scaled by a power of two per row so that its largest magnitude is between
//    2^15 and 2^16 (at most 65,504 in fp16 and 65,280 in bf16) and goes into fp16: exact for
//    fp16 values, which are never scaled down, and for bf16 values down to 2^-32 of the row's largest.
//    Scores of such rows are up to 2^32, and K's scales in bf16 up to 2^121: where rows were scaled up, a
//    power of two common to a warp's rows is taken off the scales as they are read (two or four
//    multiplications a lane and unit) and goes into the rows' factors, so that nothing overflows but a score.
//  * The weights of V carry vs_j, whose range has nothing to do with the softmax's: with
//    p_ij = 2^(x_ij - m_i) for the row sum, w_ij = p_ij vs_j 2^(e_i), where e_i follows the
//    largest p vs of the row: it stands at 2^7 when it is set, and e_i is lowered (and O with
//    it) when it has outgrown 2^15.  When m_i is raised, e_i goes along, so that w stays what
//    it was.  w is rounded to fp16 as the matrix instructions take it (off by up to 2^-11,
//    and by 2^-32 of the row's largest below that).
//
// 64 requests of 1,000 to 16,000 keys (8 key/value heads of d = 128, int8, 1.23 GB): 202 to 209 us
// with the join for 4 query heads a key (89% of the measured copy rate; 254 with 16-row products
// of all heads and 16-byte copies), 215 to 231 for 16 rows.  Drafted tokens, 20 or more rows a
// sequence: 41 us where the bytes alone would take 10.5: a warp spends 2.1 us on a unit.
#include <cuda_fp16.h>

#include "paged_warp.cuh"

namespace clis {

__device__ unsigned int g_q8_error_word = 0;

namespace {

constexpr float kTau = 8.0f;
// Exponents of V's weights.  Scales are 2^-109 (the smallest rows that a write keeps, in E4M3) to
// 2^121: 2^7 over them, and the powers and their inverses are ordinary fp32 numbers.
constexpr float kMostExp = 118.f, kLeastExp = -118.f;
constexpr unsigned kErrLoad = 1u << 0;  // a wait for a stage gave up (the forward kernel's producer bit)

template <int D, int NT>
struct QCfg {
    static constexpr int TK = 4096 / D;             // keys per unit: 8 KB of codes
    static constexpr int BLOCKS = NT == 1 ? 3 : 2;  // of an SM (registers)
    static constexpr int NST = NT == 1 ? 2 : 3;     // stages of a warp
    static constexpr int HALF = TK * D;             // bytes of K (or V) of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int SCALE = 2 * TK;            // floats of a stage: K's, V's
    static constexpr int TR = 8 * NT;               // query rows of an item
    static constexpr int SCALES = NST * SCALE * 4 + 16;  // bytes of a warp, and what K's are multiplied by
    static constexpr int PER_WARP = NST * STAGE + SCALES;
    static constexpr int SMEM = kDecodeWarps * PER_WARP + 1024;
};

// Place of a 16-byte chunk of a row of codes in its stage, as TMA's 128- and 64-byte swizzles
// leave it.  ldmatrix (8 rows, one chunk) touches all banks once, K's 16-byte loads of
// four threads per row twice at d = 128.
template <int D>
__device__ __forceinline__ uint32_t at_row(int row, int chunk)
{
    return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ float lds32(uint32_t at)
{
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}

__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
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

// An fp16 pair of E4M3 values with 448 in the place of NaN.
__device__ __forceinline__ uint32_t no_nan(uint32_t u)
{
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x5F005F00u));
    return r;
}

// Whether a word of E4M3 codes holds a NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan(uint32_t w)
{
    const uint32_t y = (w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu;
    return ((y - 0x01010101u) & ~y & 0x80808080u) != 0;
}

// The transpose of an 8 x 8 matrix of 16-bit values held by a warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// A warp's stages, and the fetching of units into them.
template <int D, int NST, int TR>
struct Loader {
    static constexpr int TK = 4096 / D, KPL = TK / 32;  // keys per lane of the scales (of one page: it has at least 8)
    Pos<TK, TR> ld;
    uint32_t ring, scales, full;  // shared addresses: stages, their scales, their barriers
    uint64_t pol;
    uint32_t loads;
    int stage, page, box_shift;

    // Whether the lane has a TMA box of the unit at hand, and its page.  What the table holds
    // is looked at when it is used (any number can stand there, so none can say that there
    // is no key).
    __device__ __forceinline__ bool has_box(int lane) const
    {
        return ld.left > 0 && lane < (TK >> box_shift) && ld.j * TK + (lane << box_shift) < ld.q.kv;
    }
    __device__ __forceinline__ void look_up(const PagedArgs &a, int lane)
    {
        page = has_box(lane) ? __ldg(a.block_table + ld.s * a.bt_s + ((ld.j * TK + (lane << box_shift)) >> a.page_shift)) : -1;
    }
    // The next unit of the run into the next stage, which has been read.
    __device__ __forceinline__ void step(const CUtensorMap *tm_k, const CUtensorMap *tm_v, const DecodeParams &p, const QuantArgs &z,
                                         int lane, unsigned int &bad)
    {
        const PagedArgs &a = p.a;
        if (ld.left == 0) return;
        const bool has = has_box(lane);
        if (has && (page < 0 || page >= a.num_pages)) {
            bad |= CLIS_PAGED_INDEX_BIT;
            page = static_cast<int>(a.num_pages);  // out of the map: its keys read as zeros
        }
        const uint32_t bar = full + 8 * stage;
        const int live = __popc(__ballot_sync(~0u, has)), key0 = ld.j * TK;
        if (lane == 0) mbar_arrive_expect_tx(bar, live * 2 * (D << box_shift));
        __syncwarp();
        if (has) {
            const uint32_t dst = ring + stage * (2 * TK * D) + lane * (D << box_shift);
            const int row = (key0 + (lane << box_shift)) & ((1 << a.page_shift) - 1);
            tma_load_4d_hint(dst, tm_k, bar, 0, row, ld.h, page, pol);
            tma_load_4d_hint(dst + TK * D, tm_v, bar, 0, row, ld.h, page, pol);
        }
        const int pg = __shfl_sync(~0u, page, (lane * KPL) >> box_shift);
#pragma unroll
        for (int i = 0; i < KPL; i++) {
            const int key = key0 + lane * KPL + i;
            const bool ok = key < ld.q.kv && pg < a.num_pages;
            const int64_t pi = ok ? pg : 0;
            const int in = ok ? key & ((1 << a.page_shift) - 1) : 0;
            const uint32_t to = scales + (stage * (2 * TK) + lane * KPL + i) * 4;
            cp_async4(to, z.ks + pi * z.ks_sp + ld.h * z.ks_sh + in * z.ks_sn, ok ? 4 : 0);
            cp_async4(to + TK * 4, z.vs + pi * z.vs_sp + ld.h * z.vs_sh + in * z.vs_sn, ok ? 4 : 0);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        ++loads;
        if (++stage == NST) stage = 0;
        ld.left--;
        if (++ld.j == ld.units && ld.left > 0) ld.next_item(a, p.g, p.limit);
        look_up(a, lane);
    }
    // A wait gave up: the copies in flight end before the block does (or are given up too).
    __device__ __forceinline__ void drain(uint32_t done)
    {
        for (uint32_t k = done; k < loads; k++) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(full + 8 * (k % NST), (k / NST) & 1) && globaltimer_ns() - t0 < 200000000ull) {
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
};

// The query rows of a warp: rows row0 + 8 nt + r of the item.  A thread loads row
// 8 nt + lane / 4 and keeps what belongs to the columns 2 (lane % 4), + 1 of its products.
template <int D, int NT>
struct Rows {
    uint32_t qf[NT][D / 16][2];
    float2 cs[NT];   // scale_log2 over the powers of two that q's row and K's scales were multiplied by
    float2 m[NT], l[NT], low[NT];  // low: what the last addition to l gained by rounding
    float2 e[NT], f[NT];           // the weights of V: exponent, and 2^exponent
    float o[D / 16][NT][4];        // d = 16 i + 2 (lane / 4) of two rows, then d + 1 of them

    // Word w of thread t holds elements 16 t + 4 w .. (w < 4) or 64 + 16 t + 4 (w - 4) .. of d,
    // as the loads of codes do.  s_down: shared address of what K's scales are to be multiplied by.
    template <int DT>
    __device__ __forceinline__ void load(const DecodeParams &p, const SeqLen &q, int head, int row0, int lane, uint32_t s_down)
    {
        const PagedArgs &a = p.a;
        const int R = q.n * p.g, r4 = lane >> 2, t4 = lane & 3;
        int exps[NT], least = 1000, most = -1000;  // of the rows' powers of two
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int row = row0 + nt * 8 + r4;
            const bool ok = row < R;
            const int tok = ok ? row / p.g : 0, hd = head * p.g + (ok ? row - tok * p.g : 0);
            const uint16_t *src = a.q + static_cast<int64_t>(q.q0 + tok) * a.q_st + hd * a.q_sh;
#pragma unroll
            for (int w = 0; w < D / 16; w += 2) {
                const uint4 v = ok ? __ldg(reinterpret_cast<const uint4 *>(src + t4 * 16 + (w >> 2) * 64 + (w & 3) * 4)) : make_uint4(0, 0, 0, 0);
                qf[nt][w][0] = v.x;
                qf[nt][w][1] = v.y;
                qf[nt][w + 1][0] = v.z;
                qf[nt][w + 1][1] = v.w;
            }
            uint32_t top = 0;  // the row's largest magnitude: bits of non-negative floats are ordered
#pragma unroll
            for (int w = 0; w < D / 16; w++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    top = max(top, __float_as_uint(elem_lo<DT>(qf[nt][w][h])) & 0x7FFFFFFFu);
                    top = max(top, __float_as_uint(elem_hi<DT>(qf[nt][w][h])) & 0x7FFFFFFFu);
                }
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // (a row of zeros or with something non-finite is taken as it is)
            const bool plain = top == 0 || top >= 0x7F800000u;
            const int ex = plain ? 0 : min(15 - (static_cast<int>(top >> 23) - 127), 126);
            const float by = exp2_int(ex);
            exps[nt] = plain ? -1000 : ex;
            if (!plain) {
                least = min(least, ex);
                most = max(most, ex);
            }
#pragma unroll
            for (int w = 0; w < D / 16; w++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    qf[nt][w][h] = pack2<1>(elem_lo<DT>(qf[nt][w][h]) * by, elem_hi<DT>(qf[nt][w][h]) * by);
            m[nt] = e[nt] = make_float2(-INFINITY, -INFINITY);
            l[nt] = low[nt] = f[nt] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < D / 16; i++) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
        // Off K's scales: what the smallest row was scaled up by, but no more than leaves those of
        // the largest row's scores above 2^-28.
        least = __reduce_min_sync(~0u, least);
        most = __reduce_max_sync(~0u, most);
        const int down = max(0, min(most, least + 90));
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const float s1 = exps[nt] == -1000 ? a.scale_log2 : a.scale_log2 * exp2_int(down - exps[nt]);
            cs[nt] = make_float2(__shfl_sync(~0u, s1, t4 * 8), __shfl_sync(~0u, s1, t4 * 8 + 4));
        }
        __syncwarp();
        if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_down), "f"(exp2_int(-down)) : "memory");
        __syncwarp();
    }

    // Keys that row 8 nt + 2 (lane % 4) + h sees.
    static __device__ __forceinline__ int limit(const DecodeParams &p, const SeqLen &q, int row0, int nt, int h, int lane)
    {
        const int r = row0 + nt * 8 + 2 * (lane & 3) + h;
        return r < q.n * p.g ? visible_keys(q.n, q.kv, r / p.g, p.a.causal) : 0;
    }

    // Products of a unit's codes, s[km][nt][0], [1]: key 16 km + lane / 4 and two rows, [2], [3]:
    // 8 keys on, into the weights of V's codes, wf: two keys' of row lane / 4.
    // sS: the unit's scales; down: what K's are multiplied by.
    // EDGE: some row does not see some key.  (A constant: as a condition at each score it
    // was a branch there.)
    template <bool EDGE, int KM>
    __device__ __forceinline__ void weights(const DecodeParams &p, const SeqLen &q, int row0, float (&s)[KM][NT][4], uint32_t sS, float down,
                                            int key0, int lane, uint32_t (&wf)[KM][NT][2])
    {
        constexpr int TK = KM * 16;
        const int r4 = lane >> 2;
        if (EDGE) {  // (before the scales, which may be no numbers: below)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int lim = limit(p, q, row0, nt, h, lane);
#pragma unroll
                    for (int km = 0; km < KM; km++)
#pragma unroll
                        for (int b = 0; b < 2; b++)
                            if (key0 + km * 16 + b * 8 + r4 >= lim) s[km][nt][2 * b + h] = -INFINITY;
                }
        }
        float vs[KM][2];
        float2 mx[NT];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) mx[nt] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int km = 0; km < KM; km++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int kr = km * 16 + h * 8 + r4;
                const float ks = lds32(sS + kr * 4) * down;
                vs[km][h] = lds32(sS + (TK + kr) * 4);
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float2 x = fmul2(make_float2(s[km][nt][2 * h], s[km][nt][2 * h + 1]), make_float2(ks, ks));
                    if (EDGE) {
                        if (s[km][nt][2 * h] == -INFINITY) x.x = -INFINITY;
                        if (s[km][nt][2 * h + 1] == -INFINITY) x.y = -INFINITY;
                    }
                    s[km][nt][2 * h] = x.x;
                    s[km][nt][2 * h + 1] = x.y;
                    mx[nt].x = fmaxf(mx[nt].x, x.x);
                    mx[nt].y = fmaxf(mx[nt].y, x.y);
                }
            }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            mx[nt] = fmul2(mx[nt], cs[nt]);
            grow |= mx[nt].x > m[nt].x + kTau || mx[nt].y > m[nt].y + kTau;
        }
        if (__any_sync(~0u, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                raise(mx[nt].x, m[nt].x, l[nt].x, low[nt].x, e[nt].x, f[nt].x);
                raise(mx[nt].y, m[nt].y, l[nt].y, low[nt].y, e[nt].y, f[nt].y);
            }
        }
        // p, its sum, and p times V's scale
        grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const float2 ns = make_float2(m[nt].x == -INFINITY ? 0.f : -m[nt].x, m[nt].y == -INFINITY ? 0.f : -m[nt].y);
            float2 sum = make_float2(0.f, 0.f), tx = sum;
#pragma unroll
            for (int km = 0; km < KM; km++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float2 x = ffma2(make_float2(s[km][nt][2 * h], s[km][nt][2 * h + 1]), cs[nt], ns);
                    const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    sum = fadd2(sum, pp);
                    float2 t = fmul2(pp, make_float2(vs[km][h], vs[km][h]));
                    if (EDGE) {  // (a scale that is no number must not reach a row that does not see its key)
                        if (s[km][nt][2 * h] == -INFINITY) t.x = 0.f;
                        if (s[km][nt][2 * h + 1] == -INFINITY) t.y = 0.f;
                    }
                    s[km][nt][2 * h] = t.x;
                    s[km][nt][2 * h + 1] = t.y;
                    tx.x = fmaxf(tx.x, t.x);
                    tx.y = fmaxf(tx.y, t.y);
                }
            // Compensated: a run may be many thousands of units, each far below the sum.
            const float2 minus = make_float2(-1.f, -1.f);
            const float2 y = ffma2(low[nt], minus, sum), t = fadd2(l[nt], y);
            low[nt] = ffma2(y, minus, ffma2(l[nt], minus, t));
            l[nt] = t;
            mx[nt] = tx;
            const float2 g = fmul2(tx, f[nt]);
            grow |= g.x > 32768.f || g.y > 32768.f || (e[nt].x == -INFINITY && tx.x > 0.f) || (e[nt].y == -INFINITY && tx.y > 0.f) ||
                    e[nt].x > kMostExp || e[nt].y > kMostExp;
        }
        if (__any_sync(~0u, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                lower(mx[nt].x, e[nt].x, f[nt].x, nt, 0);
                lower(mx[nt].y, e[nt].y, f[nt].y, nt, 1);
            }
        }
#pragma unroll
        for (int km = 0; km < KM; km++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float2 w = fmul2(make_float2(s[km][nt][2 * h], s[km][nt][2 * h + 1]), f[nt]);
                    wf[km][nt][h] = transposed(pack2<1>(w.x, w.y));
                }
    }

    // The largest over the lanes that share a row.
    static __device__ __forceinline__ float row_max(float v)
    {
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
        return fmaxf(v, __shfl_xor_sync(~0u, v, 16));
    }

    static __device__ __forceinline__ void raise(float v, float &m, float &l, float &low, float &e, float &f)
    {
        v = row_max(v);
        if (!(v > m + kTau)) return;
        const float al = ex2_approx(m - v);
        l *= al;
        low *= al;
        if (m != -INFINITY) {  // w stays what it was
            e += v - m;
            f = ex2_approx(fminf(e, kMostExp));
        }
        m = v;
    }

    __device__ __forceinline__ void lower(float v, float &e, float &f, int nt, int h)
    {
        v = row_max(v);
        const bool none = e == -INFINITY;
        float to = fminf(e, kMostExp);
        if (v > 0.f && (none || v * ex2_approx(to) > 32768.f)) {
            const int x = static_cast<int>(__float_as_uint(v) >> 23) - 127;
            to = fmaxf(kLeastExp, fminf(kMostExp, static_cast<float>(7 - x)));
        }
        if (to == e) return;
        const float al = none ? 0.f : ex2_approx(to - e);
        e = to;
        f = ex2_approx(to);
#pragma unroll
        for (int i = 0; i < D / 16; i++) {
            o[i][nt][h] *= al;
            o[i][nt][2 + h] *= al;
        }
    }

    // The item's rows, final (slot < 0) or partial.  nan_from >= 0: E4M3 codes of V that are NaN and
    // lie at keys [nan_from, nan_to) took part as numbers; rows that see them become NaN.
    template <int DT>
    __device__ __forceinline__ void write(const DecodeParams &p, const QuantArgs &z, const SeqLen &q, int s, int head, int row0, int64_t slot,
                                          float *part_o, float2 *part_ml, int nan_from, int nan_to, int lane)
    {
        const PagedArgs &a = p.a;
        const int R = q.n * p.g, r4 = lane >> 2, c2 = 2 * (lane & 3);
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int row = row0 + nt * 8 + c2 + h;
                float sum = h ? l[nt].y : l[nt].x;
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                if (row >= R) continue;
                const int tok = row / p.g, hd = head * p.g + (row - tok * p.g);
                if (nan_from >= 0) {
                    const int see = min(limit(p, q, row0, nt, h, lane), nan_to);
#pragma unroll 1
                    for (int key = nan_from; key < see; key++) {
                        const int pg = __ldg(a.block_table + s * a.bt_s + (key >> a.page_shift));
                        if (pg < 0 || pg >= a.num_pages) continue;
                        const uint8_t *v = z.vc + static_cast<int64_t>(pg) * a.vc_sp + head * a.vc_sh +
                                           static_cast<int64_t>(key & ((1 << a.page_shift) - 1)) * a.vc_sn + 2 * r4;
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            const uint32_t u = __ldg(reinterpret_cast<const unsigned short *>(v + i * 16));
                            if ((u & 0x7Fu) == 0x7Fu) o[i][nt][h] = NAN;
                            if (((u >> 8) & 0x7Fu) == 0x7Fu) o[i][nt][2 + h] = NAN;
                        }
                    }
                }
                const float mm = h ? m[nt].y : m[nt].x, ee = h ? e[nt].y : e[nt].x;
                const float back = ee == -INFINITY ? 0.f : ex2_approx(-ee);  // (O is 0 then)
                if (slot < 0) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    uint16_t *dst = a.o + static_cast<int64_t>(q.q0 + tok) * a.o_st + hd * a.o_sh + 2 * r4;
#pragma unroll
                    for (int i = 0; i < D / 16; i++)  // (zeros for a row that sees no key)
                        *reinterpret_cast<uint32_t *>(dst + i * 16) =
                            sum == 0.f ? 0u : pack2<DT>(o[i][nt][h] * inv * back, o[i][nt][2 + h] * inv * back);
                    if (r4 == 0 && a.lse2) a.lse2[static_cast<int64_t>(q.q0 + tok) * a.H + hd] = sum == 0.f ? -INFINITY : mm + log2f(sum);
                } else {
                    float *dst = part_o + (slot * p.rows_max + row - row0) * D + 2 * r4;
#pragma unroll
                    for (int i = 0; i < D / 16; i++)
                        *reinterpret_cast<float2 *>(dst + i * 16) = make_float2(o[i][nt][h] * back, o[i][nt][2 + h] * back);
                    if (r4 == 0) part_ml[slot * p.rows_max + row - row0] = make_float2(mm, sum);
                }
            }
    }
};

// Item blockIdx.x of the batch, if it has as many (all threads take part; ends with a
// barrier): item s_rel[0] of sequence s_seq[0].
template <int TR>
__device__ __forceinline__ bool block_item(const DecodeParams &p, uint64_t *s_sum, int *s_seq, uint64_t *s_rel, unsigned int &bad)
{
    const PagedArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.S + kDecodeThreads - 1) / kDecodeThreads;
    const int sb = min(a.S, tid * per), se = min(a.S, sb + per);
    auto items = [&](const SeqLen &q) { return is_decode(q, p.g, p.limit) ? a.Hkv * ceil_div(q.n * p.g, TR) : 0; };
    int n = 0;
    for (int s = sb; s < se; s++) {
        const SeqLen q = seq_len(a, s);
        if (q.bad || (p.strict && q.n > 0 && !is_decode(q, p.g, p.limit))) bad |= CLIS_PAGED_LENGTH_BIT;
        n += items(q);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = incl - n, all = 0;
    for (int i = 0; i < kDecodeWarps; i++) {
        if (i < warp) before += static_cast<int>(s_sum[i]);
        all += static_cast<int>(s_sum[i]);
    }
    int rel = static_cast<int>(blockIdx.x) - before;
    if (rel >= 0 && rel < n)
        for (int s = sb; s < se; s++) {
            const int k = items(seq_len(a, s));
            if (rel < k) {
                s_seq[0] = s;
                s_rel[0] = rel;
                break;
            }
            rel -= k;
        }
    __syncthreads();
    return static_cast<int>(blockIdx.x) < all;
}

// The output rows of an item from its warps' parts, in the order of the keys.
template <int D, int DT, int TR>
__device__ __forceinline__ void join_quarters(const DecodeParams &p, const SeqLen &q, int head, int row0, const float *sO, const float2 *s_ml)
{
    constexpr int V = D / 32;
    const PagedArgs &a = p.a;
    const int lane = threadIdx.x & 31, rows = min(TR, q.n * p.g - row0);
    for (int r = threadIdx.x >> 5; r < rows; r += kDecodeWarps) {
        float M = -INFINITY, l = 0.f, o[V];
#pragma unroll
        for (int i = 0; i < kDecodeWarps; i++) M = fmaxf(M, s_ml[i * TR + r].x);
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = 0.f;
#pragma unroll
        for (int i = 0; i < kDecodeWarps; i++) {
            const float2 ml = s_ml[i * TR + r];
            if (ml.y == 0.f) continue;  // a part none of whose keys the row sees
            const float w = ex2_approx(ml.x - M);
            l = fmaf(w, ml.y, l);
#pragma unroll
            for (int e = 0; e < V; e++) o[e] = fmaf(w, sO[(i * TR + r) * D + lane * V + e], o[e]);
        }
        const int tok = (row0 + r) / p.g, hd = head * p.g + (row0 + r - tok * p.g);
        const float inv = 1.f / l;
        uint16_t *dst = a.o + static_cast<int64_t>(q.q0 + tok) * a.o_st + hd * a.o_sh + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2)  // (zeros for a row that sees no key)
            *reinterpret_cast<uint32_t *>(dst + e) = l == 0.f ? 0u : pack2<DT>(o[e] * inv, o[e + 1] * inv);
        if (lane == 0 && a.lse2) a.lse2[static_cast<int64_t>(q.q0 + tok) * a.H + hd] = l == 0.f ? -INFINITY : M + log2f(l);
    }
}

template <int D, int DT, int CODE, int NT>
__global__ void __launch_bounds__(kDecodeThreads, QCfg<D, NT>::BLOCKS)
    paged_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeParams p,
                    const QuantArgs z, const int box_shift)
{
    using C = QCfg<D, NT>;
    constexpr int TK = C::TK, KM = TK / 16;  // key tiles of 16
    const PagedArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_sum[kDecodeWarps], s_rel[kDecodeWarps];
    __shared__ int s_seq[kDecodeWarps];
    __shared__ __align__(8) uint64_t s_full[kDecodeWarps * C::NST];
    __shared__ int s_abort;
    __shared__ float2 s_ml[kDecodeWarps * C::TR];  // (one)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned int bad = 0;
    pdl_launch();
    if (tid == 0) {
        for (int i = 0; i < kDecodeWarps * C::NST; i++) mbar_init(smem_u32(&s_full[i]), 33);  // TMA's bytes, and 32 lanes' scales
        s_abort = 0;
        fence_mbar_init();
    }
    const int c = warp * gridDim.x + blockIdx.x;  // this worker
    Runs runs{};
    uint64_t u1 = 0;
    bool mine = true;
    Pos<TK, C::TR> cur;
    if (p.one) {
        mine = block_item<C::TR>(p, s_sum, s_seq, s_rel, bad);
    } else {
        runs = block_runs<TK, kDecodeWarps, C::TR>(p, s_sum, s_seq, s_rel, bad);
        if (lane == 0) p.meta[c] = make_int4(0, 0, 0, 0);
        mine = c < runs.nb;
    }
    if (bad && blockIdx.x == 0) atomicOr(&g_q8_error_word, bad);
    bad = 0;
    if (!mine) {  // nothing for this warp (U = 0 included)
        pdl_wait();
        return;
    }
    if (p.one) {  // a quarter of the item's units
        cur.set(a, s_seq[0], p.g);
        const int item = static_cast<int>(s_rel[0]);
        cur.h = item / cur.tiles;
        cur.tile = item - cur.h * cur.tiles;
        cur.j = cur.units * warp / kDecodeWarps;
        cur.left = cur.units * (warp + 1) / kDecodeWarps - cur.j;
    } else {
        u1 = decode_cut(runs.U, runs.nb, c + 1);
        cur.set(a, s_seq[warp], p.g);
        const int item = static_cast<int>(div64(s_rel[warp], cur.units));
        cur.h = item / cur.tiles;
        cur.tile = item - cur.h * cur.tiles;
        cur.j = static_cast<int>(s_rel[warp] - static_cast<uint64_t>(item) * cur.units);
        cur.left = static_cast<uint32_t>(u1 - decode_cut(runs.U, runs.nb, c));
    }
    const SeqLen q0 = cur.q;  // (one)
    const int head0 = cur.h, row00 = cur.tile * C::TR;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    Loader<D, C::NST, C::TR> load;
    load.ld = cur;
    load.ring = base + warp * C::NST * C::STAGE;
    load.scales = base + kDecodeWarps * C::NST * C::STAGE + warp * C::SCALES;
    const uint32_t s_down = load.scales + C::SCALES - 16;
    load.full = smem_u32(&s_full[warp * C::NST]);
    load.pol = policy_evict_first();
    load.loads = load.stage = 0;
    load.box_shift = box_shift;
    load.look_up(a, lane);
#pragma unroll 1
    for (int i = 0; i < C::NST - 1; i++) load.step(&tm_k, &tm_v, p, z, lane, bad);

    const int r4 = lane >> 2, t4 = lane & 3;
    uint32_t done = 0, phase = 0;  // units read
    int stage = 0;
    bool fine = true, some = false;
    float *const sO = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));  // (one: the stages, all read by then)
    Rows<D, NT> w;
    while (fine && cur.left > 0) {
        // ---- one item, units j0 .. j1 - 1 of it
        const int j0 = cur.j;
        const int j1 = static_cast<int>(min(static_cast<uint32_t>(cur.units), j0 + cur.left));
        const int kv = cur.q.kv, row0 = cur.tile * C::TR;
        const int lim0 = visible_keys(cur.q.n, kv, row0 / p.g, a.causal);  // keys that every row sees
        w.template load<DT>(p, cur.q, cur.h, row0, lane, s_down);
        bool dirty = false;
#pragma unroll 1
        for (int j = j0; j < j1; j++) {
            __syncwarp();
            load.step(&tm_k, &tm_v, p, z, lane, bad);  // into the stage that the previous unit has been read from
            if (!mbar_wait_warp(load.full + 8 * stage, phase, &s_abort, &g_q8_error_word, kErrLoad)) {
                fine = false;
                break;
            }
            ++done;
            const int key0 = j * TK;
            const uint32_t sK = load.ring + stage * C::STAGE, sV = sK + C::HALF;
            const uint32_t sS = load.scales + stage * C::SCALE * 4;
            if (++stage == C::NST) {
                stage = 0;
                phase ^= 1;
            }
            if (key0 >= kv) continue;
            // S^T = KC Q^T: TK keys x 8 rows per column tile
            float s[KM][NT][4];
#pragma unroll
            for (int km = 0; km < KM; km++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++) s[km][nt][0] = s[km][nt][1] = s[km][nt][2] = s[km][nt][3] = 0.f;
#pragma unroll
            for (int hh = 0; hh < D / 64; hh++)
#pragma unroll
                for (int k0 = 0; k0 < KM; k0 += 2) {
                    uint4 kw[2][2];
#pragma unroll
                    for (int i = 0; i < 2; i++)
#pragma unroll
                        for (int h = 0; h < 2; h++) kw[i][h] = lds128(sK + at_row<D>((k0 + i) * 16 + h * 8 + r4, hh * 4 + t4));
#pragma unroll
                    for (int x = 0; x < 4; x++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            uint32_t f[4];
                            unpack<CODE, false>(x == 0 ? kw[i][0].x : x == 1 ? kw[i][0].y : x == 2 ? kw[i][0].z : kw[i][0].w, f[0], f[2]);
                            unpack<CODE, false>(x == 0 ? kw[i][1].x : x == 1 ? kw[i][1].y : x == 2 ? kw[i][1].z : kw[i][1].w, f[1], f[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma16816<1>(s[k0 + i][nt], f, w.qf[nt][hh * 4 + x][0], w.qf[nt][hh * 4 + x][1]);
                        }
                }
            const bool edge = key0 + TK > lim0;  // some row does not see some key
            uint32_t wf[KM][NT][2];
            const float down = lds32(s_down);
            if (edge) w.template weights<true, KM>(p, cur.q, row0, s, sS, down, key0, lane, wf);
            else w.template weights<false, KM>(p, cur.q, row0, s, sS, down, key0, lane, wf);
            // O^T += VC^T W^T: a transposed load gives 32 keys of 16 columns, in each word the
            // codes of two neighbouring columns and two neighbouring keys.
            auto pv = [&](bool clean) {
#pragma unroll
                for (int k0 = 0; k0 < KM; k0 += 2)
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        uint32_t vw[4], f[2][4];
                        ldsm4_t(sV + at_row<D>(k0 * 16 + lane, i), vw);
#pragma unroll
                        for (int e = 0; e < 4; e++) unpack<CODE, true>(vw[e], f[e >> 1][2 * (e & 1)], f[e >> 1][2 * (e & 1) + 1]);
                        if (CODE != CLIS_CODE_INT8 && clean)
#pragma unroll
                            for (int e = 0; e < 8; e++) f[e >> 2][e & 3] = no_nan(f[e >> 2][e & 3]);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            mma16816<1>(w.o[i][nt], f[0], wf[k0][nt][0], wf[k0][nt][1]);
                            mma16816<1>(w.o[i][nt], f[1], wf[k0 + 1][nt][0], wf[k0 + 1][nt][1]);
                        }
                    }
            };
            // Where a key is masked for some rows, or the stage's rows behind the last key hold
            // whatever was there, a NaN code must not reach the output as 0 * NaN: it takes part as a
            // number, and the rows that see it get a NaN at the end.  (Codes behind the last key do not
            // count: with them 19 short requests whose pages held such codes took 73 us, now 17.)
            if (CODE != CLIS_CODE_INT8 && edge) {
#pragma unroll 1
                for (int i = lane; i < C::HALF / 16 && key0 + i / (D / 16) < kv; i += 32) {
                    const uint4 u = lds128(sV + i * 16);
                    dirty |= has_nan(u.x) || has_nan(u.y) || has_nan(u.z) || has_nan(u.w);
                }
                pv(true);
            } else {
                pv(false);
            }
        }
        if (!fine) break;
        const bool any_dirty = CODE != CLIS_CODE_INT8 && __any_sync(~0u, dirty);
        const bool whole = j0 == 0 && j1 == cur.units;
        const int nan_from = any_dirty ? max(lim0 / TK * TK, j0 * TK) : -1;
        if (p.one) {
            __syncthreads();
            w.template write<DT>(p, z, cur.q, cur.s, cur.h, row0, warp, sO, s_ml, nan_from, j1 * TK, lane);
            some = true;
            break;
        }
        w.template write<DT>(p, z, cur.q, cur.s, cur.h, row0, whole ? -1 : 2 * static_cast<int64_t>(c) + (j0 == 0 ? 1 : 0), p.part_o,
                             p.part_ml, nan_from, j1 * TK, lane);
        if (!whole && j0 == 0 && lane == 0)
            p.meta[c] = make_int4(item_parts(runs, c, u1 - cur.left + cur.units - 1), cur.q.q0, cur.q.n | row0 << 16, cur.h);
        cur.left -= j1 - j0;
        cur.j = j1;
        if (cur.left > 0) cur.next_item(a, p.g, p.limit);
    }
    if (!fine) load.drain(done);
    if (bad) atomicOr(&g_q8_error_word, bad);
    if (p.one) {
        if (!some) {
            __syncthreads();
            if (lane < C::TR) s_ml[warp * C::TR + lane] = make_float2(-INFINITY, 0.f);
        }
        __syncthreads();
        join_quarters<D, DT, C::TR>(p, q0, head0, row00, sO, s_ml);
    }
    pdl_wait();
}

bool encode_codes(CUtensorMap *map, const uint8_t *base, const PagedArgs &a, int64_t sp, int64_t sh, int64_t sn, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(1) << a.page_shift, static_cast<cuuint64_t>(a.Hkv),
                                static_cast<cuuint64_t>(a.num_pages)};
    // (a stride of a size-1 dimension is never used; it gets a canonical value)
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(sn), static_cast<cuuint64_t>(a.Hkv == 1 ? a.d : sh),
                                   static_cast<cuuint64_t>(a.num_pages == 1 ? a.d : sp)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(a.d), static_cast<cuuint32_t>(box_rows), 1, 1}, step[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, a.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Column tiles of 8 query rows that a warp takes.  Three only at d = 64 (at d = 128 they spill
// registers: 20 rows 168 us instead of 141 with two tiles of 16), where a tile of 24 rows costs 1.25 times
// one of 16: 20 rows over 64 requests 88 us, 40 166; with two they are 2 and 3 tiles, with four
// (registers spilled) 132 and 245.  25 to 32 rows fill two tiles of 16.
int column_tiles(int d, int rows) { return rows <= 8 ? 1 : d == 64 && rows > 16 && (rows <= 24 || rows > 32) ? 3 : 2; }

// Blocks of the form without a second launch, or 0: where the GPU holds a block for each item that
// the batch can have, and the tables no more than 16 units of each, or 32 where runs would not be
// much shorter (64 items).  (d = 128, 4 query heads a key, 8 key/value heads, runs and join against a block
// per item: one request of 300 keys 12.4 and 10.4 us, of 60 12.5 and 7.4, 40 of 480 22.8 and 15.1, 8 of
// 900 18.4 and 16.6, one of 900 16.3 and 16.2, 8 of 1,900 22.1 and 24.9; d = 64: one of 900 14.9 and
// 11.1, of 1,900, 30 units, 13.7 and 16.6.)
int64_t one_item_blocks(const PagedArgs &a, int rows, int nsm)
{
    const int nt = column_tiles(a.d, rows), tk = 4096 / a.d;
    const int64_t items = static_cast<int64_t>(a.S) * a.Hkv * ((rows + 8 * nt - 1) / (8 * nt));
    const int64_t units = ((static_cast<int64_t>(a.width) << a.page_shift) + tk - 1) / tk;
    return items <= (nt == 1 ? QCfg<128, 1>::BLOCKS : QCfg<128, 2>::BLOCKS) * nsm && units <= (items >= 64 ? 32 : 16) ? items : 0;
}

template <int D, int DT, int CODE, int NT>
clis_status_t launch_impl(int rows, const PagedArgs &a, const QuantArgs &z, bool strict, bool after_schedule, void *workspace,
                          int nsm, cudaStream_t stream)
{
    using C = QCfg<D, NT>;
    const auto kernel = paged_q8_kernel<D, DT, CODE, NT>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return CLIS_ERR_CUDA;
    const int64_t items = one_item_blocks(a, rows, nsm);
    const int grid = items > 0 ? static_cast<int>(items) : C::BLOCKS * nsm;
    DecodeParams p;
    p.a = a;
    p.one = items > 0;
    p.g = a.H / a.Hkv;
    p.least = 2;
    p.strict = strict;
    place_parts(p, static_cast<size_t>(grid) * kDecodeWarps, C::TR, workspace);
    p.limit = rows;
    int box_shift = 0;
    while ((1 << box_shift) < C::TK && box_shift < a.page_shift) box_shift++;
    CUtensorMap mk, mv;
    if (!encode_codes(&mk, z.kc, a, a.kc_sp, a.kc_sh, a.kc_sn, 1 << box_shift) ||
        !encode_codes(&mv, z.vc, a, a.vc_sp, a.vc_sh, a.vc_sn, 1 << box_shift))
        return CLIS_ERR_CUDA;
    if (after_schedule) {
        if (launch_pdl(kernel, dim3(grid), kDecodeThreads, C::SMEM, stream, mk, mv, p, z, box_shift) != cudaSuccess) return CLIS_ERR_CUDA;
    } else {
        kernel<<<grid, kDecodeThreads, C::SMEM, stream>>>(mk, mv, p, z, box_shift);
        if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    }
    if (p.one) return CLIS_OK;
    return launch_join<D, DT>(p, stream) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

template <int D, int DT, int CODE, typename... A>
clis_status_t launch_rows(int rows, const A &...args)
{
    const int nt = column_tiles(D, rows);
    if (nt == 1) return launch_impl<D, DT, CODE, 1>(rows, args...);
    if constexpr (D == 64)
        if (nt == 3) return launch_impl<D, DT, CODE, 3>(rows, args...);
    return launch_impl<D, DT, CODE, 2>(rows, args...);
}

template <int D, typename... A>
clis_status_t launch_types(bool half, bool int8, int rows, const A &...args)
{
    if (int8) return half ? launch_rows<D, 1, CLIS_CODE_INT8>(rows, args...) : launch_rows<D, 0, CLIS_CODE_INT8>(rows, args...);
    return half ? launch_rows<D, 1, CLIS_CODE_E4M3>(rows, args...) : launch_rows<D, 0, CLIS_CODE_E4M3>(rows, args...);
}

}  // namespace

int paged_q8_rows(const PagedArgs &a, int64_t max_q, int nsm)
{
    // Rows of the largest sequence if it is small; else those of single tokens.  Small: up to 64
    // rows; up to 2048 where the tables can hold no more than 17 units (d = 64, where the chunk
    // kernel costs half: 6) for each of 1,216 workers.  (The chunk kernel with what it needs takes 40
    // to 55 us at least.  d = 128: 80 rows over 16,080 keys of 8 heads, 16.5 units, 51 us here
    // against 68; 160 rows of 4 x 4,040 keys, 16.7, 43 against 56; 2,048 rows over 712 keys, 19.4, 69
    // against 54.  d = 64: 160 rows, 5.9, 35 against 42; 2,048 rows, 6.8, 48 against 41.  Up to 64 rows, 8
    // heads, here against there: 64 requests of 1,000 to 16,000 keys, int8, d = 128, 20, 32 and 64 rows 418,
    // 427 and 831 against 1,011, 998 and 1,001, E4M3 876 for 64 against 993; d = 64 174, 260 and 472 against 625,
    // 609 and 611.  17 of 562 to 9,001 keys 85, 89 and 158 against 217; 8 of 1,875 to 30,000 113, 113 and 208
    // against 287; 64 of 125 to 2,000 90, 97 and 168 against 194, and only at d = 64, 64 rows, it is 143
    // against 135, E4M3 173 against 137.)
    const int g = a.H / a.Hkv, tile = a.d == 64 ? 24 : 16, keys = 4096 / a.d;
    const int64_t rows = max_q <= 2048 ? max_q * g : 2049;
    if (rows <= 64) return static_cast<int>(rows);
    const int64_t items = static_cast<int64_t>(a.S) * a.Hkv * ((rows + tile - 1) / tile);
    const int64_t units = ((static_cast<int64_t>(a.width) << a.page_shift) + keys - 1) / keys * items;
    if (rows <= 2048 && units <= static_cast<int64_t>(a.d == 64 ? 6 : 17) * nsm * 2 * kDecodeWarps) return static_cast<int>(rows);
    return g <= 64 ? g : 0;
}

size_t paged_q8_workspace(int d, int rows, int nsm)
{
    if (rows == 0) return 0;
    const int nt = column_tiles(d, rows);
    const int of_sm = kDecodeWarps * (nt == 1 ? QCfg<128, 1>::BLOCKS : QCfg<128, 2>::BLOCKS);  // (the same for both widths)
    static_assert(QCfg<64, 3>::BLOCKS == QCfg<128, 2>::BLOCKS, "one number of blocks");
    return parts_workspace(static_cast<size_t>(of_sm) * nsm, 8 * nt, d);
}

clis_status_t launch_paged_q8(const PagedArgs &a, const QuantArgs &z, int rows, bool strict, bool after_schedule,
                              void *workspace, int nsm, cudaStream_t stream)
{
    const bool half = a.dtype == CLIS_DT_FP16, int8 = z.code == CLIS_CODE_INT8;
    return a.d == 128 ? launch_types<128>(half, int8, rows, a, z, strict, after_schedule, workspace, nsm, stream)
                      : launch_types<64>(half, int8, rows, a, z, strict, after_schedule, workspace, nsm, stream);
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
