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

// How far the shift of a row's weights 2^(x - shift) stands below the row's maximum
// (dt: 0 bf16, 1 fp16), in powers of two.  fp16 holds 2^-24 to 65504: with the shift at
// the maximum, many weights below 2^-25 of the largest vanish although the row sum counts
// them (262,143 of 2^-25.5 are 0.5% of a row).  The maximum may outgrow the shift by 2^8
// before it is raised; 2^7 more still fit, and weights down to 2^-32 count.
CLIS_HD constexpr float weight_room(int dt) { return dt ? 7.f : 0.f; }

// ------------------------------------------------------------ decode kernel
//
// Items are (sequence, key/value head), sequence-major; an item costs one unit
// per decode_keys(d) keys (at least one: its output must be written).  The units
// of all items, laid end to end, are cut into as many equal runs as there are
// workers (warps), so ragged batches balance to one unit, and an item that crosses
// a cut is joined from partial results afterwards.
CLIS_HD constexpr int decode_keys(int d) { return d == 128 ? 16 : 32; }  // the same bytes

CLIS_HD bool is_decode(const SeqLen &s, int g, int rows_max)
{
    // (n * g fits: both are below 2^31 and n is compared first)
    return s.n > 0 && s.n <= rows_max && s.n * g <= rows_max;
}

CLIS_HD int decode_units(const SeqLen &s, int keys) { return imax(1, ceil_div(s.kv, keys)); }

// 64-bit division is slow on the GPU, and units and costs are mostly below 2^32.
CLIS_HD uint64_t div64(uint64_t a, uint64_t b)
{
    return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Units of a batch, at most (the entry point checks what its tables can hold): a
// worker's run then counts in 32 bits on any GPU of more than 16 SMs (8 workers each).
constexpr uint64_t kMaxUnits = uint64_t(1) << 39;

// Workers that take part, for U units.
CLIS_HD int decode_workers(uint64_t U, int grid, int least)
{
    const uint64_t want = div64(U + least - 1, least);
    return want < static_cast<uint64_t>(grid) ? static_cast<int>(want) : grid;
}

CLIS_HD uint64_t decode_cut(uint64_t U, int blocks, int c)  // (U c: below 2^39 times the workers)
{
    return div64(U * static_cast<uint32_t>(c), static_cast<uint32_t>(blocks));
}

// ------------------------------------------------------------- chunk kernel
//
// A row tile is up to 128 query rows: 128 / g tokens of all g heads.  An item is
// two row tiles of one (sequence, key/value head) against the keys they see, in
// tiles of 128.  Items in order (sequence, head, query tile) are laid end to end,
// each as long as its cost, and cut into equal runs, one per block; an item that
// crosses a cut is joined from the blocks' partial results.
//
// Cost of a key tile: 3 with two row tiles (1.45 us), 2 with one (two key tiles are
// worked on at a time, but their bytes come no faster), and per item what loading
// Q, filling the pipeline and writing the output take (about 4.5 us).
constexpr int kChunkRows = 128;
constexpr int kChunkKeys = 128;
constexpr int kChunkOverhead = 9;

struct __attribute__((aligned(16))) ChunkItem {
    int q0, n, kv, s;        // the sequence
    int h, tok0, n_kv, nt;   // head, first token, key tiles, row tiles in use
    uint64_t first;          // cost of the items before it
    uint64_t pad;
};

CLIS_HD int chunk_tokens(int g) { return 2 * (kChunkRows / g); }  // tokens per item
CLIS_HD int chunk_q_tiles(int n, int g) { return ceil_div(n, chunk_tokens(g)); }

// Items of a sequence (those of up to rows_small rows are the decode kernel's).
CLIS_HD int chunk_items(const SeqLen &s, int g, int rows_small, int Hkv)
{
    return s.n == 0 || is_decode(s, g, rows_small) ? 0 : Hkv * chunk_q_tiles(s.n, g);
}

// Places of the list of items: what sequences of T tokens in all need at most (each
// rounds its query tiles up).
CLIS_HD int64_t chunk_list(int T, int S, int g, int Hkv)
{
    return static_cast<int64_t>(Hkv) * (T / chunk_tokens(g) + static_cast<int64_t>(S) + 1);
}

// Place of the list for the item behind `before` others.  Prefix sums that fall let
// sequences share rows, and then more items follow than there are places: those are left
// out (a sequence's first place is then the list's end).
CLIS_HD int chunk_place(uint64_t before, int64_t list)
{
    return static_cast<int>(before < static_cast<uint64_t>(list) ? before : static_cast<uint64_t>(list));
}

// Item r (0-based) of sequence seq; at least one key tile (its output must be written).
CLIS_HD ChunkItem chunk_item(const SeqLen &s, int seq, int g, int r, bool causal)
{
    ChunkItem t;
    const int nqt = chunk_q_tiles(s.n, g);
    t.q0 = s.q0;
    t.n = s.n;
    t.kv = s.kv;
    t.s = seq;
    t.h = r / nqt;
    t.tok0 = (r - t.h * nqt) * chunk_tokens(g);
    const int last = imin(s.n, t.tok0 + chunk_tokens(g)) - 1;
    t.n_kv = imax(1, ceil_div(visible_keys(s.n, s.kv, last, causal), kChunkKeys));
    t.nt = s.n - t.tok0 > kChunkRows / g ? 2 : 1;
    t.first = 0;
    t.pad = 0;
    return t;
}

CLIS_HD uint64_t chunk_cost(int n_kv, int nt) { return kChunkOverhead + static_cast<uint64_t>(n_kv) * (nt + 1); }

// Blocks that take part, for a total cost of U: every run is `least` or longer (if
// U is), which must be at least a key tile's cost, so that no run within an item
// is without a key tile of it.
CLIS_HD int chunk_blocks(uint64_t U, int grid, int least)
{
    const uint64_t want = U / least;
    return want >= static_cast<uint64_t>(grid) ? grid : want > 0 ? static_cast<int>(want) : U > 0 ? 1 : 0;
}

// The cuts: run c is [cut(c), cut(c + 1)), cut(c) = floor(U c / blocks).
struct ChunkCuts {
    uint64_t run;  // U / blocks
    uint32_t rem, blocks;
    CLIS_HD uint64_t cut(int c) const { return run * c + rem * static_cast<uint32_t>(c) / blocks; }  // rem c < blocks^2
};

CLIS_HD ChunkCuts chunk_cuts(uint64_t U, int blocks)
{
    ChunkCuts k;
    k.blocks = blocks > 0 ? blocks : 1;
    k.run = div64(U, k.blocks);
    k.rem = static_cast<uint32_t>(U - k.run * k.blocks);
    return k;
}

// Block whose run holds place x < U.
CLIS_HD int chunk_block_of(const ChunkCuts &k, uint64_t x)
{
    const uint64_t g = k.run > 0 ? div64(x, k.run) : x;
    int c = static_cast<int>(g < k.blocks ? g : k.blocks - 1);
    while (c > 0 && k.cut(c) > x) c--;
    while (c + 1 < static_cast<int>(k.blocks) && k.cut(c + 1) <= x) c++;
    return c;
}

// Key tile that place x (0 .. cost) of an item falls on.
CLIS_HD int chunk_tile_of(uint64_t x, int n_kv, int nt)
{
    if (x <= kChunkOverhead) return 0;
    const uint64_t t = static_cast<uint32_t>(x - kChunkOverhead) / static_cast<uint32_t>(nt + 1);  // (a cost is below 2^32)
    return t < static_cast<uint64_t>(n_kv) ? static_cast<int>(t) : n_kv;
}

// Key tiles [t0, t1) of an item that the run [lo, hi) takes.
struct ChunkRange {
    int t0, t1;
};

CLIS_HD ChunkRange chunk_range(const ChunkItem &t, uint64_t lo, uint64_t hi)
{
    ChunkRange r;
    r.t0 = lo > t.first ? chunk_tile_of(lo - t.first, t.n_kv, t.nt) : 0;
    r.t1 = hi > t.first ? chunk_tile_of(hi - t.first, t.n_kv, t.nt) : 0;
    return r;
}

// Blocks among which the item is shared out: the first with a key tile of it, and
// how many.
struct ChunkOwners {
    int c, count;
};

CLIS_HD ChunkOwners chunk_owners(const ChunkItem &t, const ChunkCuts &k)
{
    int c = chunk_block_of(k, t.first);
    while (c + 1 < static_cast<int>(k.blocks) && chunk_range(t, k.cut(c), k.cut(c + 1)).t1 == 0) c++;
    ChunkOwners o;
    o.c = c;
    o.count = chunk_block_of(k, t.first + chunk_cost(t.n_kv, t.nt) - 1) - c + 1;
    return o;
}

// First key tile of the item that some of its rows see only in part: from there
// on masked places lie among the keys.
CLIS_HD int chunk_first_masked(const ChunkItem &t, bool causal)
{
    return visible_keys(t.n, t.kv, t.tok0, causal) / kChunkKeys;
}

}  // namespace clis
