// paged_api.cu -- C entry points of rotary positions and of the paged
// key/value cache: argument checks on the host, then one launcher each.
#include <cmath>
#include <cstdint>

#include "clis_internal.h"
#include "paged_internal.h"

namespace {

constexpr int64_t kMaxN = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
// Keys of a sequence: a block works on at most one item's at a time, 1.5 us per 128
// of them (0.8 s), while other warps wait for it with a limit of 2 s.  Every warp follows
// every item, so no wait spans more than one.
constexpr int64_t kMaxKeys = int64_t(1) << 26;
constexpr int64_t kMaxSeqs = 16384;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides in elements of rows of 16-bit values: multiples of 16 bytes, below
// 2^38 (2^39 bytes; tensor maps take 2^40).
clis_status_t check_strides(std::initializer_list<int64_t> ss)
{
    for (int64_t s : ss)
        if (s < 0) return CLIS_ERR_INVALID_ARG;
    for (int64_t s : ss)
        if (s & 7) return CLIS_ERR_MISALIGNED;
    for (int64_t s : ss)
        if (s >= (int64_t(1) << 38)) return CLIS_ERR_UNSUPPORTED;
    return CLIS_OK;
}

// Whether a written tensor gives each of its rows of d elements a place of its
// own.  Sorted by stride, each dimension has to step over all of the faster ones.
bool overlapping(int64_t d, const int64_t (*dims)[2], int n)
{
    int64_t size[3], stride[3];
    int m = 0;
    for (int i = 0; i < n; i++) {
        if (dims[i][0] == 0) return false;  // nothing is written
        if (dims[i][0] > 1) {
            size[m] = dims[i][0];
            stride[m++] = dims[i][1];
        }
    }
    for (int i = 0; i < m; i++)
        for (int j = i + 1; j < m; j++)
            if (stride[j] < stride[i]) {
                const int64_t t = stride[i], u = size[i];
                stride[i] = stride[j];
                size[i] = size[j];
                stride[j] = t;
                size[j] = u;
            }
    int64_t span = d;  // elements from a block's first to behind its last
    for (int i = 0; i < m; i++) {
        if (stride[i] < span) return true;
        span += (size[i] - 1) * stride[i];
    }
    return false;
}

clis_status_t check_rope(const clis_rope_t *r, bool with_k_out)
{
    if (r->B < 0 || r->Hq < 0 || r->Hk < 0 || r->N < 0) return CLIS_ERR_INVALID_ARG;
    if (r->axes < 1 || r->axes > 4 || (r->interleaved != 0 && r->interleaved != 1) ||
        (r->inverse != 0 && r->inverse != 1))
        return CLIS_ERR_INVALID_ARG;
    if (r->dtype != CLIS_DT_BF16 && r->dtype != CLIS_DT_FP16) return CLIS_ERR_INVALID_ARG;
    if (r->d != 64 && r->d != 128) return CLIS_ERR_UNSUPPORTED;
    if (r->pairs < 8 || r->pairs > r->d / 2) return CLIS_ERR_INVALID_ARG;
    if (r->pairs & 7) return CLIS_ERR_UNSUPPORTED;
    if (r->Hq > 65536 || r->Hk > 65536 || r->B > kMaxTokens || r->N > kMaxTokens || r->B * r->N > kMaxTokens / 8)
        return CLIS_ERR_UNSUPPORTED;
    clis_status_t st = check_strides({r->q_sb, r->q_sh, r->q_sn, r->k_sb, r->k_sh, r->k_sn, r->qo_sb, r->qo_sh, r->qo_sn});
    if (st != CLIS_OK) return st;
    if (with_k_out && (st = check_strides({r->ko_sb, r->ko_sh, r->ko_sn})) != CLIS_OK) return st;
    const int64_t qd[3][2] = {{r->B, r->qo_sb}, {r->Hq, r->qo_sh}, {r->N, r->qo_sn}};
    const int64_t kd[3][2] = {{r->B, r->ko_sb}, {r->Hk, r->ko_sh}, {r->N, r->ko_sn}};
    if (overlapping(r->d, qd, 3) || (with_k_out && overlapping(r->d, kd, 3))) return CLIS_ERR_INVALID_ARG;
    return CLIS_OK;
}

// log2 of the page size, or -1.
int page_shift(int64_t page)
{
    for (int s = 3; s <= 16; s++)
        if (page == int64_t(1) << s) return s;
    return -1;
}

clis_status_t check_table(const clis_paged_t *p)
{
    if (p->S < 0 || p->T < 0 || p->width < 1 || p->num_pages < 1 || p->bt_ss < 0 || p->page_size < 1)
        return CLIS_ERR_INVALID_ARG;
    if (page_shift(p->page_size) < 0 || p->S > kMaxSeqs || p->T > kMaxTokens || p->num_pages > kMaxN) return CLIS_ERR_UNSUPPORTED;
    if (p->width > kMaxKeys / p->page_size || p->bt_ss >= (int64_t(1) << 38)) return CLIS_ERR_UNSUPPORTED;
    return CLIS_OK;
}

clis_status_t check_cache(const clis_paged_t *p, bool written)
{
    clis_status_t st = check_table(p);
    if (st != CLIS_OK) return st;
    if (p->H < 1 || p->Hkv < 1) return CLIS_ERR_INVALID_ARG;
    if (p->dtype != CLIS_DT_BF16 && p->dtype != CLIS_DT_FP16) return CLIS_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return CLIS_ERR_UNSUPPORTED;
    if (p->H > 65536 || p->H % p->Hkv) return p->H % p->Hkv ? CLIS_ERR_INVALID_ARG : CLIS_ERR_UNSUPPORTED;
    if ((st = check_strides({p->kc_sp, p->kc_sh, p->kc_sn, p->vc_sp, p->vc_sh, p->vc_sn})) != CLIS_OK) return st;
    if (p->kc_sn < p->d || p->vc_sn < p->d) return CLIS_ERR_INVALID_ARG;
    const int64_t kd[3][2] = {{p->num_pages, p->kc_sp}, {p->Hkv, p->kc_sh}, {p->page_size, p->kc_sn}};
    const int64_t vd[3][2] = {{p->num_pages, p->vc_sp}, {p->Hkv, p->vc_sh}, {p->page_size, p->vc_sn}};
    if (written && (overlapping(p->d, kd, 3) || overlapping(p->d, vd, 3))) return CLIS_ERR_INVALID_ARG;
    return CLIS_OK;
}

// Everything of the attention call but its pointers.
clis_status_t check_attn(const clis_paged_t *p, int64_t max_q)
{
    clis_status_t st = check_cache(p, false);
    if (st != CLIS_OK) return st;
    if (max_q < 1) return CLIS_ERR_INVALID_ARG;
    if (p->H / p->Hkv > clis::kChunkRows) return CLIS_ERR_UNSUPPORTED;
    if ((st = check_strides({p->q_st, p->q_sh, p->o_st, p->o_sh})) != CLIS_OK) return st;
    if (p->q_st < p->d) return CLIS_ERR_INVALID_ARG;
    const int64_t od[2][2] = {{p->T, p->o_st}, {p->H, p->o_sh}};
    if (overlapping(p->d, od, 2)) return CLIS_ERR_INVALID_ARG;
    // What the tables can hold, in the smallest of units (S Hkv is below 2^30, a row's keys
    // are at most 2^26).
    const uint64_t per = static_cast<uint64_t>(p->width) * p->page_size / clis::decode_keys(128);
    if (per > 0 && static_cast<uint64_t>(p->S) * p->Hkv > clis::kMaxUnits / per) return CLIS_ERR_UNSUPPORTED;
    const int64_t tpc = clis::chunk_tokens(static_cast<int>(p->H / p->Hkv));
    if (static_cast<double>(p->Hkv) * (static_cast<double>(p->T) / tpc + p->S + 1) >= 1.0e9) return CLIS_ERR_UNSUPPORTED;
    return CLIS_OK;
}

clis::PagedArgs attn_args(const clis_paged_t *p)
{
    clis::PagedArgs a{};
    a.q_st = p->q_st;
    a.q_sh = p->q_sh;
    a.o_st = p->o_st;
    a.o_sh = p->o_sh;
    a.kc_sp = p->kc_sp;
    a.kc_sh = p->kc_sh;
    a.kc_sn = p->kc_sn;
    a.vc_sp = p->vc_sp;
    a.vc_sh = p->vc_sh;
    a.vc_sn = p->vc_sn;
    a.bt_s = p->bt_ss;
    a.num_pages = p->num_pages;
    a.S = static_cast<int>(p->S);
    a.T = static_cast<int>(p->T);
    a.H = static_cast<int>(p->H);
    a.Hkv = static_cast<int>(p->Hkv);
    a.d = static_cast<int>(p->d);
    a.dtype = static_cast<int>(p->dtype);
    a.page_shift = page_shift(p->page_size);
    a.width = static_cast<int>(p->width);
    return a;
}

struct Split {
    int row_tiles;  // of the decode kernel, 0: not launched
    bool chunk;     // the chunk kernel is launched
};

Split split_of(const clis_paged_t *p, int64_t max_q, int nsm)
{
    const int g = static_cast<int>(p->H / p->Hkv);
    const int64_t mq = max_q < p->T ? max_q : p->T;
    Split s;
    s.row_tiles = clis::paged_decode_row_tiles(mq, g, static_cast<int>(p->d));
    s.chunk = mq * g > 16 * s.row_tiles;
    // A batch with chunks leaves its single tokens to the chunk kernel too where they
    // are few items (sequence, key/value head): an item costs that kernel some 5 us of
    // one SM, the decode kernel's launches cost the batch 25 us.  (8 key/value heads,
    // one chunk: 12 sequences of up to 8,000 keys 98 us against 127 with both, 64 of
    // 16,000 362 against 384; 100 of 600 104 against 80, 300 of 300 206 against 102.)
    // At d = 64 a key tile has half the bytes but takes almost as long, so the total
    // length counts too (24 sequences of up to 8,000 keys 84 us against 94, 40 119
    // against 112, 64 of 16,000 260 against 219): at most 96 tiles per SM by what the
    // block table can hold, which the host knows.
    // S counts sequences without a token too, which the host cannot tell apart: 3 chunks and
    // 9 single tokens take 92 us with 12 or 64 rows in the table, 132 with 256.  All of
    // these have 8 key/value heads.
    const int64_t items = p->S * p->Hkv;
    const int64_t per = (p->width * p->page_size + clis::kChunkKeys - 1) / clis::kChunkKeys;
    if (s.chunk && items <= 4 * nsm && (p->d == 128 || items * per <= 96 * nsm)) s.row_tiles = 0;
    return s;
}

bool sm_count(int *n)
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

clis::RotArgs rot_args(const clis_rope_t *r)
{
    clis::RotArgs a{};
    a.q_sb = r->q_sb;
    a.q_sh = r->q_sh;
    a.q_sn = r->q_sn;
    a.k_sb = r->k_sb;
    a.k_sh = r->k_sh;
    a.k_sn = r->k_sn;
    a.qo_sb = r->qo_sb;
    a.qo_sh = r->qo_sh;
    a.qo_sn = r->qo_sn;
    a.ko_sb = r->ko_sb;
    a.ko_sh = r->ko_sh;
    a.ko_sn = r->ko_sn;
    a.p_sb = r->p_sb;
    a.p_sn = r->p_sn;
    a.p_sa = r->p_sa;
    a.B = static_cast<int>(r->B);
    a.Hq = static_cast<int>(r->Hq);
    a.Hk = static_cast<int>(r->Hk);
    a.N = static_cast<int>(r->N);
    a.d = static_cast<int>(r->d);
    a.pairs = static_cast<int>(r->pairs);
    a.axes = static_cast<int>(r->axes);
    a.interleaved = static_cast<int>(r->interleaved);
    a.inverse = static_cast<int>(r->inverse);
    a.dtype = static_cast<int>(r->dtype);
    return a;
}

}  // namespace

extern "C" {

clis_status_t clis_rope(const clis_rope_t *desc, const void *q, const void *k, void *q_out, void *k_out,
                        const int32_t *positions, const double *inv_freq, const int32_t *axis, clis_stream_t stream)
{
    if (!desc) return CLIS_ERR_INVALID_ARG;
    const clis_status_t st = check_rope(desc, true);
    if (st != CLIS_OK) return st;
    if (desc->B * desc->N == 0 || desc->Hq + desc->Hk == 0) return CLIS_OK;
    if ((desc->Hq > 0 && (!q || !q_out)) || (desc->Hk > 0 && (!k || !k_out)) || !positions || !inv_freq || !axis)
        return CLIS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8) || !aligned(axis, 4))
        return CLIS_ERR_MISALIGNED;
    clis::RotArgs a = rot_args(desc);
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.qo = static_cast<uint16_t *>(q_out);
    a.ko = static_cast<uint16_t *>(k_out);
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.axis = axis;
    return clis::launch_rot(a, reinterpret_cast<cudaStream_t>(stream));
}

clis_status_t clis_paged_plan(const clis_paged_t *desc, const int32_t *ctx_len, const int32_t *new_len,
                              int32_t *block_table, int32_t *ring, int64_t ring_size, const int64_t *state_in,
                              int64_t *state_out, int32_t *cu_q, int32_t *kv_len, int64_t *slots, int32_t *positions,
                              clis_stream_t stream)
{
    if (!desc) return CLIS_ERR_INVALID_ARG;
    const clis_status_t st = check_table(desc);
    if (st != CLIS_OK) return st;
    if (desc->S > 1 && desc->bt_ss < desc->width) return CLIS_ERR_INVALID_ARG;  // rows are written
    if (ring_size < 1) return CLIS_ERR_INVALID_ARG;
    if (ring_size > kMaxN) return CLIS_ERR_UNSUPPORTED;
    if (!ring || !state_in || !state_out || !cu_q || state_in == state_out) return CLIS_ERR_INVALID_ARG;
    if (desc->S > 0 && (!ctx_len || !new_len || !block_table || !kv_len)) return CLIS_ERR_INVALID_ARG;
    if (desc->T > 0 && (!slots || !positions)) return CLIS_ERR_INVALID_ARG;
    if (!aligned(ctx_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) || !aligned(ring, 4) ||
        !aligned(state_in, 8) || !aligned(state_out, 8) || !aligned(cu_q, 4) || !aligned(kv_len, 4) ||
        !aligned(slots, 8) || !aligned(positions, 4))
        return CLIS_ERR_MISALIGNED;
    clis::PlanArgs a{};
    a.ctx_len = ctx_len;
    a.new_len = new_len;
    a.block_table = block_table;
    a.bt_s = desc->bt_ss;
    a.ring = ring;
    a.ring_size = ring_size;
    a.state_in = state_in;
    a.state_out = state_out;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.slots = slots;
    a.pos = positions;
    a.S = static_cast<int>(desc->S);
    a.T = static_cast<int>(desc->T);
    a.width = static_cast<int>(desc->width);
    a.page_shift = page_shift(desc->page_size);
    a.num_pages = desc->num_pages;
    return clis::launch_paged_plan(a, reinterpret_cast<cudaStream_t>(stream));
}

clis_status_t clis_paged_append(const clis_paged_t *desc, const clis_rope_t *rope, const void *q, const void *k,
                                const void *v, int64_t v_st, int64_t v_sh, void *q_out, void *k_cache, void *v_cache,
                                const int64_t *slots, const int32_t *positions, const double *inv_freq,
                                const int32_t *axis, clis_stream_t stream)
{
    if (!desc || !rope) return CLIS_ERR_INVALID_ARG;
    clis_status_t st = check_cache(desc, true);
    if (st != CLIS_OK) return st;
    clis_rope_t r = *rope;
    const bool turn = r.pairs != 0;
    if (!turn) {  // the rotation's other fields are not read then
        r.pairs = 8;
        r.axes = 1;
        r.interleaved = r.inverse = 0;
        r.Hq = 0;
        r.q_sb = r.q_sh = r.q_sn = r.qo_sb = r.qo_sh = r.qo_sn = 0;
        if (q) return CLIS_ERR_INVALID_ARG;
    }
    r.ko_sb = r.ko_sh = r.ko_sn = 0;
    if (r.B != 1 || r.N != desc->T || r.Hk != desc->Hkv || r.d != desc->d || r.dtype != desc->dtype || r.inverse ||
        (r.Hq != 0 && r.Hq != desc->H))
        return CLIS_ERR_INVALID_ARG;
    if ((st = check_rope(&r, false)) != CLIS_OK) return st;
    if ((st = check_strides({v_st, v_sh})) != CLIS_OK) return st;
    if (desc->T == 0) return CLIS_OK;
    if (!k || !v || !k_cache || !v_cache || !slots || (r.Hq > 0 && (!q || !q_out))) return CLIS_ERR_INVALID_ARG;
    if (turn && (!positions || !inv_freq || !axis)) return CLIS_ERR_INVALID_ARG;
    if ((r.Hq > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8) || !aligned(axis, 4))
        return CLIS_ERR_MISALIGNED;
    clis::RotArgs a = rot_args(&r);
    if (!turn) a.pairs = 0;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.v_sn = v_st;
    a.v_sh = v_sh;
    a.qo = static_cast<uint16_t *>(q_out);
    a.ko = static_cast<uint16_t *>(k_cache);
    a.ko_sb = desc->kc_sp;
    a.ko_sh = desc->kc_sh;
    a.ko_sn = desc->kc_sn;
    a.vo = static_cast<uint16_t *>(v_cache);
    a.vo_sb = desc->vc_sp;
    a.vo_sh = desc->vc_sh;
    a.vo_sn = desc->vc_sn;
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.axis = axis;
    a.slots = slots;
    a.num_slots = desc->num_pages * desc->page_size;
    a.page_shift = page_shift(desc->page_size);
    return clis::launch_rot(a, reinterpret_cast<cudaStream_t>(stream));
}

clis_status_t clis_attn_paged_workspace_size(const clis_paged_t *desc, int64_t max_q, size_t *bytes)
{
    if (!desc || !bytes) return CLIS_ERR_INVALID_ARG;
    const clis_status_t st = check_attn(desc, max_q);
    if (st != CLIS_OK) return st;
    *bytes = 0;
    if (desc->S == 0 || desc->T == 0) return CLIS_OK;
    int nsm = 0;
    if (!sm_count(&nsm)) return CLIS_ERR_CUDA;
    const Split s = split_of(desc, max_q, nsm);
    *bytes = clis::paged_decode_workspace(static_cast<int>(desc->d), s.row_tiles, nsm) +
             (s.chunk ? clis::paged_chunk_workspace(attn_args(desc), nsm) : 0);
    return CLIS_OK;
}

clis_status_t clis_attn_fwd_paged(const clis_paged_t *desc, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_table, const int32_t *cu_q, const int32_t *kv_len, void *o,
                                  float *lse2, int64_t max_q, float scale_log2, int causal, void *workspace,
                                  size_t ws_bytes, clis_stream_t stream)
{
    if (!desc) return CLIS_ERR_INVALID_ARG;
    const clis_status_t st = check_attn(desc, max_q);
    if (st != CLIS_OK) return st;
    if (!std::isfinite(scale_log2) || !(scale_log2 > 0.f)) return CLIS_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return CLIS_ERR_INVALID_ARG;
    if (desc->S == 0 || desc->T == 0) return CLIS_OK;
    if (!q || !k_cache || !v_cache || !block_table || !cu_q || !kv_len || !o) return CLIS_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
        !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(lse2, 4))
        return CLIS_ERR_MISALIGNED;
    int nsm = 0;
    if (!sm_count(&nsm)) return CLIS_ERR_CUDA;
    const Split s = split_of(desc, max_q, nsm);
    clis::PagedArgs a = attn_args(desc);
    const size_t dec = clis::paged_decode_workspace(a.d, s.row_tiles, nsm);
    const size_t need = dec + (s.chunk ? clis::paged_chunk_workspace(a, nsm) : 0);
    if (need > 0 && (!workspace || ws_bytes < need)) return CLIS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CLIS_ERR_MISALIGNED;
    a.q = static_cast<const uint16_t *>(q);
    a.kc = static_cast<const uint16_t *>(k_cache);
    a.vc = static_cast<const uint16_t *>(v_cache);
    a.o = static_cast<uint16_t *>(o);
    a.lse2 = lse2;
    a.block_table = block_table;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.scale_log2 = scale_log2;
    a.causal = causal;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    void *cws = static_cast<char *>(workspace) + dec;
    clis_status_t e = CLIS_OK;
    if (s.chunk) e = clis::launch_paged_chunk_schedule(a, 16 * s.row_tiles, cws, nsm, cs);
    if (e == CLIS_OK && s.row_tiles > 0)
        e = clis::launch_paged_decode(a, s.row_tiles, !s.chunk, s.chunk, workspace, nsm, cs);
    if (e == CLIS_OK && s.chunk) e = clis::launch_paged_chunk(a, 16 * s.row_tiles, cws, nsm, cs);
    return e;
}

}  // extern "C"
