// paged_sched.h -- who computes what in attention over a paged cache: plain
// integer arithmetic, shared by the kernels and by a CPU test (it compiles with
// nvcc and with an ordinary C++ compiler).
//
// A sequence brings n new tokens and g query heads per key/value head: n * g
// query rows that read the same keys.  Sequences of few rows go to the decode
// kernel (bound by the cache's bytes), the others to the chunk kernel (bound by
// the tensor cores).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CLIS_HD __host__ __device__ __forceinline__
#else
#define CLIS_HD inline
#endif

namespace clis {

CLIS_HD int imin(int a, int b) { return a < b ? a : b; }
CLIS_HD int imax(int a, int b) { return a > b ? a : b; }
CLIS_HD int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One sequence of the batch, its lengths brought into the range of the buffers:
// cu_q into [0, T], kv_len into what a block-table row can hold.
struct SeqLen {
    int q0, n, kv;
    bool bad;  // a length had to be changed
};

CLIS_HD SeqLen clip_seq(int q0, int q1, int kv, int T, int kv_cap)
{
    SeqLen s;
    s.q0 = imin(imax(q0, 0), T);
    const int e = imin(imax(q1, s.q0), T);
    s.n = e - s.q0;
    s.kv = imin(imax(kv, 0), kv_cap);
    s.bad = s.q0 != q0 || e != q1 || s.kv != kv;
    return s;
}

// Keys that new token t (0-based) of the sequence sees: 0 .. visible - 1.
CLIS_HD int visible_keys(int n, int kv, int t, bool causal)
{
    return causal ? imin(kv, imax(kv - n + t + 1, 0)) : kv;
}

// ------------------------------------------------------------ decode kernel
//
// Items are (sequence, key/value head), sequence-major; an item costs one unit
// per kDecodeKeys keys (at least one: its output must be written).  The units
// of all items, laid end to end, are cut into as many equal runs as there are
// blocks, so ragged batches balance to one unit, and an item that crosses a cut
// is joined from partial results afterwards.
constexpr int kDecodeKeys = 64;

CLIS_HD bool is_decode(const SeqLen &s, int g, int rows_max)
{
    // (n * g fits: both are below 2^31 and n is compared first)
    return s.n > 0 && s.n <= rows_max && s.n * g <= rows_max;
}

CLIS_HD int decode_units(const SeqLen &s) { return imax(1, ceil_div(s.kv, kDecodeKeys)); }

// Blocks that take part, for U units: every run holds at least `least` units.
CLIS_HD int decode_blocks(uint32_t U, int grid, int least)
{
    const uint32_t want = (U + least - 1) / least;
    return want < static_cast<uint32_t>(grid) ? static_cast<int>(want) : grid;
}

CLIS_HD uint32_t decode_cut(uint32_t U, int blocks, int c)
{
    return static_cast<uint32_t>(static_cast<uint64_t>(U) * static_cast<uint32_t>(c) / static_cast<uint32_t>(blocks));
}

// ------------------------------------------------------------- chunk kernel
//
// A row tile is up to 128 query rows: tpt = 128 / g tokens of all g heads.  A
// work tile is two row tiles of one (sequence, key/value head) against a range
// of 128-key tiles.  When there are too few work tiles to fill the GPU the
// keys of each are split into `parts` ranges, joined afterwards.
constexpr int kChunkRows = 128;
constexpr int kChunkKeys = 128;

struct __attribute__((aligned(16))) ChunkTile {
    int q0, n, kv, s;        // the sequence
    int h, tok0, start, n_kv;  // head, first token, first key tile, key tiles
    int parts, part, nt, masked;  // row tiles in use; masked: an empty range (no key of it counts)
};

CLIS_HD int chunk_tokens(int g) { return 2 * (kChunkRows / g); }  // tokens per work tile
CLIS_HD int chunk_q_tiles(int n, int g) { return ceil_div(n, chunk_tokens(g)); }

// Key tiles of work tile qt, at least one (its output must be written).
CLIS_HD int chunk_cost(const SeqLen &s, int g, int qt, bool causal)
{
    const int last = imin(s.n, (qt + 1) * chunk_tokens(g)) - 1;
    return imax(1, ceil_div(visible_keys(s.n, s.kv, last, causal), kChunkKeys));
}

CLIS_HD int chunk_max_cost(const SeqLen &s) { return imax(1, ceil_div(s.kv, kChunkKeys)); }

// Key tiles a part should have: `total` tiles of work in `items` work tiles, for
// `slots` places; with enough work tiles nothing is split.
CLIS_HD int chunk_part_len(uint64_t total, uint64_t items, int slots, int least)
{
    if (items >= static_cast<uint64_t>(slots)) return 1 << 30;
    const uint64_t len = (total + slots - 1) / slots;
    return len < static_cast<uint64_t>(least) ? least : static_cast<int>(len > (1u << 30) ? (1u << 30) : len);
}

CLIS_HD int chunk_parts(const SeqLen &s, int part_len) { return ceil_div(chunk_max_cost(s), part_len); }

// Tile r (0-based) of sequence s: head-major, then part, then query tile, so that
// tiles that read the same keys run side by side.
CLIS_HD ChunkTile chunk_tile(const SeqLen &s, int seq, int g, int parts, int r, bool causal)
{
    ChunkTile t;
    const int nqt = chunk_q_tiles(s.n, g);
    t.q0 = s.q0;
    t.n = s.n;
    t.kv = s.kv;
    t.s = seq;
    t.h = r / (nqt * parts);
    const int rem = r - t.h * nqt * parts;
    t.part = rem / nqt;
    const int qt = rem - t.part * nqt;
    t.parts = parts;
    t.tok0 = qt * chunk_tokens(g);
    t.nt = s.n - t.tok0 > kChunkRows / g ? 2 : 1;
    const int cost = chunk_cost(s, g, qt, causal);
    t.start = static_cast<int>(static_cast<int64_t>(cost) * t.part / parts);
    const int end = static_cast<int>(static_cast<int64_t>(cost) * (t.part + 1) / parts);
    t.n_kv = end - t.start;
    t.masked = 0;
    if (t.n_kv == 0) {  // an empty part still takes its place: one tile, none of whose keys counts
        t.n_kv = 1;
        t.masked = 1;
        if (t.start >= cost) t.start = cost - 1;
    }
    return t;
}

// First key tile of the work tile that some of its rows see only in part: from
// there on masked places lie among the keys.
CLIS_HD int chunk_first_masked(const ChunkTile &t, bool causal)
{
    const int full = t.masked ? 0 : visible_keys(t.n, t.kv, t.tok0, causal);
    return full / kChunkKeys;
}

}  // namespace clis
