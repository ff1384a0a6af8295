"""The division of work of attention over a paged cache (csrc/paged_sched.h), on the CPU: every key
of every row is computed exactly once, no index leaves its buffer, whatever the lengths."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "certified_fixed_stabilizer_gb300", "csrc", "paged_sched.h")

HARNESS = r"""
#include <vector>
#include "%s"
using namespace clis;
// 0: sound; else the number of the broken property.
static int decode(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_max, int Hkv, int grid, int least, int keys)
{
    std::vector<int> units;   // per item
    for (int s = 0; s < S; s++) {
        SeqLen q = clip_seq(cu[s], cu[s + 1], kv[s], T, cap);
        if (q.n < 0 || q.q0 < 0 || q.q0 + q.n > T || q.kv < 0 || q.kv > cap) return 1;
        if (!is_decode(q, g, rows_max)) continue;
        if ((long long)q.n * g > rows_max) return 2;
        if ((long long)decode_units(q, keys) * keys < q.kv) return 3;
        for (int h = 0; h < Hkv; h++) units.push_back(decode_units(q, keys));
    }
    unsigned U = 0;
    for (int u : units) U += u;
    int nb = decode_workers(U, grid, least);
    if (nb > grid || (U > 0 && nb < 1) || (U == 0 && nb != 0)) return 4;
    unsigned at = 0;
    for (int c = 0; c < nb; c++) {
        unsigned a = decode_cut(U, nb, c), b = decode_cut(U, nb, c + 1);
        if (a != at || b <= a) return 5;     // runs follow one another, none is empty
        at = b;
    }
    return at == U ? 0 : 6;
}
static int chunk(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_small, int Hkv, int grid, int least,
                 int causal, long long max_items)
{
    std::vector<ChunkItem> items;
    unsigned long long U = 0;
    for (int s = 0; s < S; s++) {
        SeqLen q = clip_seq(cu[s], cu[s + 1], kv[s], T, cap);
        if (q.n == 0 || is_decode(q, g, rows_small)) continue;
        int nqt = chunk_q_tiles(q.n, g), tpt = kChunkRows / g;
        std::vector<char> row(q.n, 0);
        for (int r = 0; r < Hkv * nqt; r++) {
            ChunkItem t = chunk_item(q, s, g, r, causal);
            if (t.h != r / nqt || t.tok0 != (r % nqt) * 2 * tpt || t.tok0 >= q.n || t.n_kv < 1) return 13;
            if (t.nt != (q.n - t.tok0 > tpt ? 2 : 1)) return 15;
            if ((long long)(t.n_kv - 1) * kChunkKeys >= (q.kv > 0 ? q.kv : 1)) return 17;  // a tile without keys
            int first = chunk_first_masked(t, causal);
            for (int i = 0; i < 2 * tpt && t.tok0 + i < q.n; i++) {
                if (t.h == 0) row[t.tok0 + i]++;
                int lim = visible_keys(q.n, q.kv, t.tok0 + i, causal);
                if (lim < 0 || lim > q.kv) return 20;
                if (lim > (long long)t.n_kv * kChunkKeys) return 21;  // a visible key beyond the item
                if ((long long)first * kChunkKeys > lim) return 22;    // a tile before `first` is masked in part
            }
            t.first = U;
            U += chunk_cost(t.n_kv, t.nt);
            items.push_back(t);
        }
        for (int i = 0; i < q.n; i++)
            if (row[i] != 1) return 24;
    }
    if ((long long)items.size() > max_items) return 11;
    int nb = chunk_blocks(U, grid, least);
    if (nb > grid || (U > 0) != (nb > 0)) return 12;
    ChunkCuts cuts = chunk_cuts(U, nb);
    std::vector<int> first(nb, -1), starts(nb, -1);
    for (size_t i = 0; i < items.size(); i++) {   // as the schedule kernel finds them
        const ChunkItem &t = items[i];
        unsigned long long end = t.first + chunk_cost(t.n_kv, t.nt);
        int c = chunk_block_of(cuts, t.first);
        if (cuts.cut(c) < t.first) c++;
        for (; c < nb && cuts.cut(c) < end; c++) {
            if (first[c] != -1) return 26;
            first[c] = i;
        }
        ChunkOwners o = chunk_owners(t, cuts);
        if (o.c < 0 || o.count < 1 || o.c + o.count > nb) return 27;
        if (o.count > 1) {
            if (starts[o.c] != -1) return 28;     // two unfinished items started by one block
            starts[o.c] = i;
        }
    }
    std::vector<int> next(items.size(), 0), parts(items.size(), 0), begun(items.size(), -1), last(items.size(), -1);
    for (int c = 0; c < nb; c++) {
        unsigned long long lo = cuts.cut(c), hi = cuts.cut(c + 1);
        if (hi <= lo || (c == 0 && lo) || (c == nb - 1 && hi != U) || first[c] < 0) return 29;
        int go = 0, start = 0;
        for (size_t i = first[c]; i < items.size() && items[i].first < hi; i++) {
            ChunkRange r = chunk_range(items[i], lo, hi);
            if (r.t1 <= r.t0) continue;
            if (r.t0 != next[i] || r.t1 > items[i].n_kv) return 19;
            next[i] = r.t1;
            parts[i]++;
            if (begun[i] < 0) begun[i] = c;
            else if (last[i] != c - 1) return 30;  // parts lie in consecutive blocks
            last[i] = c;
            if (r.t0 > 0) go++;                                   // place 2 c
            else if (r.t1 < items[i].n_kv) start++;                // place 2 c + 1
        }
        if (go > 1 || start > 1) return 31;        // one place of each kind per block
    }
    for (size_t i = 0; i < items.size(); i++) {
        if (next[i] != items[i].n_kv) return 23;
        ChunkOwners o = chunk_owners(items[i], cuts);
        if (o.c != begun[i] || o.count != parts[i]) return 32;
    }
    int many = 0;
    for (int n : parts) many += n > 2;
    if (many > (grid - 1) / 2 + 1) return 33;      // items joined by the join kernel: its list and its grid
    return 0;
}
extern "C" int check_decode(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_max, int Hkv, int grid, int least, int keys)
{ return decode(S, cu, kv, T, cap, g, rows_max, Hkv, grid, least, keys); }
extern "C" int check_chunk(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_small, int Hkv, int grid, int least,
                           int causal, long long max_items)
{ return chunk(S, cu, kv, T, cap, g, rows_small, Hkv, grid, least, causal, max_items); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("sched")
    src = d / "h.cpp"
    src.write_text(HARNESS.replace("%s", HEADER, 1))
    so = d / "h.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.check_chunk.argtypes = [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int)] * 2 + [ctypes.c_int] * 8 + [ctypes.c_longlong]
    return L


def ints(v):
    return (ctypes.c_int * len(v))(*v)


def check(lib, ctx, new, g, Hkv, causal=1, sms=152, cap=None, cu=None, kv=None):
    S, T = len(ctx), sum(new)
    cu = cu or [sum(new[:i]) for i in range(S + 1)]
    kv = kv or [c + n for c, n in zip(ctx, new)]
    cap = cap or max(kv + [1])
    for rows in (0, 16, 32):
        if rows:
            for least in (1, 4):
                for keys in (16, 32):
                    assert lib.check_decode(S, ints(cu), ints(kv), T, cap, g, rows, Hkv, 2 * sms, least, keys) == 0
        tokens = 2 * (128 // g)
        items = Hkv * (T // tokens + S + 1)
        for least in (4, 16):
            assert lib.check_chunk(S, ints(cu), ints(kv), T, cap, g, rows, Hkv, sms, least, causal, items) == 0


def test_random_batches(lib):
    rng = random.Random(5)
    for _ in range(300):
        S = rng.randint(1, 12)
        ctx = [rng.choice([0, 0, 1, rng.randint(0, 300), rng.randint(0, 20000)]) for _ in range(S)]
        new = [rng.choice([0, 1, 1, rng.randint(1, 8), rng.randint(1, 300), rng.randint(1, 2000)]) for _ in range(S)]
        check(lib, ctx, new, rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 33, 64, 128]), rng.choice([1, 2, 8]), rng.randint(0, 1),
              rng.choice([1, 4, 152]))


def test_sizes_at_the_edges(lib):
    for ctx, new in (([0], [0]), ([0], [1]), ([127], [1]), ([128], [1]), ([0], [128]), ([0], [129]), ([0], [256]),
                     ([63], [1]), ([64], [1]), ([2 ** 29], [1]), ([2 ** 29], [300])):
        for g in (1, 3, 8, 128):
            for causal in (0, 1):
                check(lib, ctx, new, g, 2, causal)


def test_lengths_out_of_range(lib):
    """Prefix sums that fall, exceed T or are negative, lengths beyond the block table: brought into range."""
    check(lib, [0, 0, 0], [5, 5, 5], 4, 2, cu=[0, 10 ** 6, -3, 2 ** 31 - 1], kv=[-1, 2 ** 31 - 1, 50], cap=640)
    check(lib, [0, 0], [200, 200], 1, 1, cu=[300, 100, 2 ** 31 - 1], kv=[2 ** 31 - 1, -2 ** 31], cap=1 << 20)


def test_rows_without_keys(lib):
    """Fewer keys than new tokens: the first tokens see none."""
    for n, kv in ((1, 0), (200, 0), (300, 100), (300, 299)):
        check(lib, [0], [n], 4, 2, kv=[kv])


LISTING = r"""
#include <vector>
#include "%s"
using namespace clis;
// The list of items as the schedule kernel writes it, and what its places hold; 0: sound.
extern "C" int check_list(int S, const int *cu, int T, int g, int rows_small, int Hkv, long long *dropped)
{
    const long long list = chunk_list(T, S, g, Hkv);
    std::vector<int> first(S + 1);
    unsigned long long run = 0;
    for (int s = 0; s < S; s++) {
        first[s] = chunk_place(run, list);
        run += chunk_items(clip_seq(cu[s], cu[s + 1], 100, T, 4096), g, rows_small, Hkv);
    }
    const int W = first[S] = chunk_place(run, list);
    *dropped = (long long)run - W;
    if (W < 0 || W > list) return 1;                       // written behind the list
    for (int i = 0, s = 0; i < W; i++) {
        while (s < S && first[s + 1] <= i) s++;
        if (s >= S || first[s] > i) return 2;              // no sequence has this item
        const SeqLen q = clip_seq(cu[s], cu[s + 1], 100, T, 4096);
        const int r = i - first[s];
        if (r >= chunk_items(q, g, rows_small, Hkv)) return 3;
        const ChunkItem t = chunk_item(q, s, g, r, true);
        if (t.h < 0 || t.h >= Hkv || t.tok0 >= q.n || t.q0 + t.tok0 >= T) return 4;
    }
    return 0;
}
"""


def test_prefix_sums_that_fall_fit_the_list(tmp_path):
    """Prefix sums that fall let sequences share rows: every second one may have all of T.  The list of items has
    places for T rows in all; what does not fit is left out."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, so = tmp_path / "l.cpp", tmp_path / "l.so"
    src.write_text(LISTING.replace("%s", HEADER, 1))
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    rng = random.Random(8)
    for S, T, Hkv in ((64, 2048, 8), (3, 15, 2), (16384, 300, 1), (1000, 999, 3), (2, 1 << 20, 16)):
        for g in (1, 4, 7, 128):
            for rows in (0, 16, 32):
                for cu in ([T * (s % 2) for s in range(S + 1)], [rng.randint(-9, T + 9) for _ in range(S + 1)],
                           sorted(rng.randint(0, T) for _ in range(S + 1))):
                    dropped = ctypes.c_longlong(-1)
                    assert L.check_list(S, ints(cu), T, g, rows, Hkv, ctypes.byref(dropped)) == 0
                    if cu == sorted(cu):
                        assert dropped.value == 0            # sound prefix sums always fit
    L.check_list(64, ints([2048 * (s % 2) for s in range(65)]), 2048, 4, 16, 8, ctypes.byref(dropped))
    assert dropped.value > 7000                              # (8,192 items for 776 places)


MANY_UNITS = r"""
#include "%s"
using namespace clis;
extern "C" int check_units(unsigned long long U, int workers)
{
    const int nb = decode_workers(U, workers, 2);
    if (nb < 1 || nb > workers) return 1;
    uint64_t at = 0;
    for (int c = 0; c < nb; c++) {
        const uint64_t a = decode_cut(U, nb, c), b = decode_cut(U, nb, c + 1);
        if (a != at || b <= a) return 2;
        if (b - a > 0xFFFFFFFFull) return 3;   // a run counts in 32 bits
        at = b;
    }
    return at == U ? 0 : 4;
}
extern "C" unsigned long long max_units() { return kMaxUnits; }
"""


def test_units_past_32_bits(tmp_path):
    """What the documented sizes can add up to is shared out without wrapping round."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, so = tmp_path / "u.cpp", tmp_path / "u.so"
    src.write_text(MANY_UNITS.replace("%s", HEADER, 1))
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.check_units.argtypes = [ctypes.c_ulonglong, ctypes.c_int]
    L.max_units.restype = ctypes.c_ulonglong
    assert L.max_units() >= 16384 * 8 * (2 ** 26 // 16)
    for workers in (8 * 17, 8 * 152):
        for U in (1, 2, 2433, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 5 * 10 ** 9, 2 ** 39 - 1, 2 ** 39):
            assert L.check_units(U, workers) == 0, (U, workers)
