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
static int decode(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_max, int Hkv, int grid, int least)
{
    std::vector<int> units;   // per item
    for (int s = 0; s < S; s++) {
        SeqLen q = clip_seq(cu[s], cu[s + 1], kv[s], T, cap);
        if (q.n < 0 || q.q0 < 0 || q.q0 + q.n > T || q.kv < 0 || q.kv > cap) return 1;
        if (!is_decode(q, g, rows_max)) continue;
        if ((long long)q.n * g > rows_max) return 2;
        if ((long long)decode_units(q) * kDecodeKeys < q.kv) return 3;
        for (int h = 0; h < Hkv; h++) units.push_back(decode_units(q));
    }
    unsigned U = 0;
    for (int u : units) U += u;
    int nb = decode_blocks(U, grid, least);
    if (nb > grid || (U > 0 && nb < 1) || (U == 0 && nb != 0)) return 4;
    unsigned at = 0;
    for (int c = 0; c < nb; c++) {
        unsigned a = decode_cut(U, nb, c), b = decode_cut(U, nb, c + 1);
        if (a != at || b <= a) return 5;     // runs follow one another, none is empty
        at = b;
    }
    return at == U ? 0 : 6;
}
static int chunk(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_small, int Hkv, int places, int least,
                 int causal, long long max_items, long long max_parts)
{
    unsigned long long total = 0, items = 0;
    for (int s = 0; s < S; s++) {
        SeqLen q = clip_seq(cu[s], cu[s + 1], kv[s], T, cap);
        if (q.n == 0 || is_decode(q, g, rows_small)) continue;
        unsigned long long it = (unsigned long long)Hkv * chunk_q_tiles(q.n, g);
        items += it;
        total += it * chunk_max_cost(q);
    }
    if ((long long)items > max_items) return 11;
    int len = chunk_part_len(total, items, places, least);
    long long W = 0, shared = 0;
    for (int s = 0; s < S; s++) {
        SeqLen q = clip_seq(cu[s], cu[s + 1], kv[s], T, cap);
        if (q.n == 0 || is_decode(q, g, rows_small)) continue;
        int parts = chunk_parts(q, len), nqt = chunk_q_tiles(q.n, g), tpt = kChunkRows / g;
        // key tiles seen: [head][query tile], counted
        std::vector<int> next(Hkv * nqt, 0);
        std::vector<char> row(q.n, 0);
        for (int r = 0; r < Hkv * nqt * parts; r++, W++) {
            ChunkTile t = chunk_tile(q, s, g, parts, r, causal);
            if (parts > 1) { shared++; if (W >= max_parts) return 12; }
            if (t.h < 0 || t.h >= Hkv || t.part < 0 || t.part >= parts || t.tok0 < 0 || t.tok0 >= q.n) return 13;
            if (t.n_kv < 1 || t.start < 0) return 14;
            int qt = t.tok0 / (2 * tpt);
            if (t.nt != (q.n - t.tok0 > tpt ? 2 : 1)) return 15;
            int cost = chunk_cost(q, g, qt, causal);
            if (t.start + t.n_kv > cost) return 16;
            if ((long long)(cost - 1) * kChunkKeys >= (q.kv > 0 ? q.kv : 1)) return 17;
            // r's place among the parts of its work tile: later parts lie nqt tiles apart
            if (r != (t.h * parts + t.part) * nqt + qt) return 18;
            if (!t.masked) {
                if (next[t.h * nqt + qt] != t.start) return 19;
                next[t.h * nqt + qt] += t.n_kv;
            }
            int first = chunk_first_masked(t, causal);
            for (int i = 0; i < 2 * tpt; i++) {
                int tok = t.tok0 + i;
                if (tok >= q.n) break;
                if (t.h == 0 && t.part == 0) row[tok]++;
                int lim = visible_keys(q.n, q.kv, tok, causal);
                if (lim < 0 || lim > q.kv) return 20;
                if (lim > cost * kChunkKeys) return 21;          // a visible key beyond the work tile
                if (!t.masked && first * kChunkKeys > lim) return 22;  // a tile before `first` is masked in part
            }
        }
        for (int h = 0; h < Hkv; h++)
            for (int qt = 0; qt < nqt; qt++)
                if (next[h * nqt + qt] != chunk_cost(q, g, qt, causal)) return 23;
        for (int i = 0; i < q.n; i++)
            if (row[i] != 1) return 24;
    }
    if (W > max_items + max_parts) return 25;
    return 0;
}
extern "C" int check_decode(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_max, int Hkv, int grid, int least)
{ return decode(S, cu, kv, T, cap, g, rows_max, Hkv, grid, least); }
extern "C" int check_chunk(int S, const int *cu, const int *kv, int T, int cap, int g, int rows_small, int Hkv, int places, int least,
                           int causal, long long max_items, long long max_parts)
{ return chunk(S, cu, kv, T, cap, g, rows_small, Hkv, places, least, causal, max_items, max_parts); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("sched")
    src = d / "h.cpp"
    src.write_text(HARNESS % HEADER)
    so = d / "h.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.check_chunk.argtypes = [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int)] * 2 + [ctypes.c_int] * 8 + [ctypes.c_longlong] * 2
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
                assert lib.check_decode(S, ints(cu), ints(kv), T, cap, g, rows, Hkv, 2 * sms, least) == 0
        tokens = 2 * (128 // g)
        items = Hkv * (T // tokens + S + 1)
        places = 2 * sms
        parts = places + min(items, places)
        assert lib.check_chunk(S, ints(cu), ints(kv), T, cap, g, rows, Hkv, places, 4, causal, items, parts) == 0


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
