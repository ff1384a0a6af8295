// reorder.cu -- the beams' states after a selection: beam w of a request goes on from
// beam parent[w].  Keys and values that both share stay where they are: the new beam's
// block-table row names the same pages.  Only the last page of a row is written to again,
// so where it is partly filled and several beams go on from one, all but the first
// get a page of their own with a copy of its rows.  Pages that no beam of the request
// names any more go back to the ring of free pages.
//
// A page is shared only among the beams of a request, and at the same place of their
// rows, so whether a page is still named is seen in one column of the request's rows: no
// reference counts, and everything follows from prefix sums over the requests.
//
// Bound: launch latency, then the tables (read and written once) and the rows copied.
// Two launches: the first (a block per request) writes the tables, the list of copies
// and the list of pages that go back, the second copies rows and appends to the ring.
// 8 requests of 4 beams 12 us, two dependent launches; 64 of 8 beams, 4 layers in 8 bits (81 MB
// moved) 33 us: the copies are short runs (a head's rows of one page, 2 to 8 KB), four pieces a
// lane in flight; eight, with fewer blocks an SM, took 38.
#include <cuda_runtime.h>

#include "clis_internal.h"
#include "paged_internal.h"

namespace clis {

__device__ unsigned int g_reorder_error_word = 0;

namespace {

constexpr int kTableThreads = 512, kTableWarps = kTableThreads / 32;
constexpr int kCopyThreads = 256, kCopyWarps = kCopyThreads / 32;

struct ReorderParams {
    ReorderArgs a;
    int tile;     // columns of the tables that a block holds at a time
    int2 *count;  // [R] {pages taken, pages that go back}
    int4 *copy;   // [R * W] {from, to, rows} of the copies, those of all requests in order
    int *back;    // [R][W * width] pages that go back
};

// Whether row i wants a page for a copy: an earlier beam of its request goes on from the same
// one, whose last page is not full.  No row of a request with a number out of range does.
__device__ __forceinline__ bool wants(const ReorderArgs &a, int i)
{
    const int cap = a.width << a.page_shift, mask = (1 << a.page_shift) - 1;
    const int g0 = i - i % a.W, mine = __ldg(a.parent + i);
    bool bad = false, again = false;
#pragma unroll 4
    for (int v = 0; v < a.W; v++) {
        const int p = __ldg(a.parent + g0 + v), n = __ldg(a.lens + g0 + v);
        bad |= n < 0 || n > cap || p >= a.W;
        again |= p == mine && g0 + v < i;
    }
    return !bad && again && mine >= 0 && (__ldg(a.lens + g0 + mine) & mask) != 0;
}

__device__ __forceinline__ long long warp_sum(long long x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

__global__ void __launch_bounds__(kTableThreads) reorder_table_kernel(const ReorderParams p)
{
    const ReorderArgs &a = p.a;
    extern __shared__ int s_tab[];  // [W][tile] old entries
    __shared__ long long s_sum[kTableWarps];
    __shared__ int s_scan[kTableWarps];
    __shared__ int s_src[kMaxBeams], s_len[kMaxBeams], s_have[kMaxBeams], s_pages[kMaxBeams];
    __shared__ int s_copy[kMaxBeams], s_fresh[kMaxBeams];  // place in the list of copies (-1: none), page
    __shared__ bool s_kept[kMaxBeams], s_again[kMaxBeams];
    __shared__ int s_rows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x, W = a.W;
    const int mask = (1 << a.page_shift) - 1;
    unsigned int bad = 0;
    pdl_launch();

    // ---- pages that the requests before this one take, and this one's rows
    const int64_t row0 = static_cast<int64_t>(g) * W;
    const int64_t head = a.state_in[0], held = a.state_in[1] - head, F = a.ring_size;
    long long before = 0;
    for (int i = tid; i < static_cast<int>(row0); i += kTableThreads) before += wants(a, i);
    before = warp_sum(before);
    if (lane == 0) s_sum[warp] = before;
    int parent = -1, n = 0;
    bool wrong = false;
    if (tid < W) {  // a thread per beam
        parent = __ldg(a.parent + row0 + tid);
        n = __ldg(a.lens + row0 + tid);
        s_src[tid] = parent;
        s_len[tid] = n;
        const int cap = a.width << a.page_shift, ok = min(max(n, 0), cap);
        if (n != ok) bad |= CLIS_PAGED_LENGTH_BIT;
        if (parent >= W) bad |= CLIS_PAGED_INDEX_BIT;
        wrong = bad != 0;
        s_have[tid] = (ok >> a.page_shift) + ((ok & mask) ? 1 : 0);
        s_kept[tid] = false;
    }
    wrong = __syncthreads_or(wrong);
    before = 0;
    for (int i = 0; i < kTableWarps; i++) before += s_sum[i];
    bool again = false;
    if (tid < W && !wrong && parent >= 0 && (s_len[parent] & mask) != 0)
        for (int v = 0; v < tid; v++) again |= s_src[v] == parent;
    const int need = __syncthreads_count(again);
    const bool sane = held >= 0 && held <= F;
    const bool done = !wrong && (need == 0 || (sane && before + need <= held));
    if (tid == 0) {
        if (!sane || (!wrong && !done)) bad |= CLIS_PAGED_POOL_BIT;
        a.done[g] = done;
        p.count[g].x = done ? need : 0;
        s_rows = 0;
    }
    if (tid < W) {
        s_again[tid] = again && done;
        if (!done) {  // the request stays as it was: its rows whole, whatever their lengths say
            s_src[tid] = tid;
            s_have[tid] = a.width;
        }
    }
    __syncthreads();
    if (tid < W) {
        atomicMax(&s_rows, s_have[tid]);
        const int src = s_src[tid], len = src < 0 ? 0 : s_len[src];
        a.lens_out[row0 + tid] = len;
        s_pages[tid] = src < 0 ? 0 : s_have[src];
        if (src >= 0) s_kept[src] = true;  // (several threads write the same)
        s_copy[tid] = -1;
        if (s_again[tid]) {
            long long i = before;
            for (int v = 0; v < tid; v++) i += s_again[v];
            // (i is below the number of pages that the ring holds)
            const int page = __ldg(a.ring + (((head % F) + F) % F + i) % F);
            if (page < 0 || page >= a.num_pages) bad |= CLIS_PAGED_INDEX_BIT;
            s_fresh[tid] = page;
            s_copy[tid] = static_cast<int>(i);
            p.copy[i] = make_int4(-1, page, len & mask, 0);  // (the page to copy from: below)
        }
    }
    __syncthreads();

    // ---- the tables, a tile of columns at a time
    int base = 0;  // pages that went back in the columns before
    for (int c0 = 0; c0 < a.width; c0 += p.tile) {
        const int cols = min(p.tile, a.width - c0);
        if (c0 < s_rows) {
            for (int w = warp; w < W; w += kTableWarps)
                for (int c = lane; c < cols; c += 32)
                    s_tab[w * p.tile + c] = c0 + c < s_have[w] ? a.table_in[(row0 + w) * a.bt_s + c0 + c] : -1;
        }
        __syncthreads();
        // (a thread has at most one column: tile <= kTableThreads)
        const int c = tid, col = c0 + c;
        // Beams whose page of this column goes back, each page once: no beam that somebody goes on
        // from names it, nor an earlier one.
        uint64_t gone = 0;
        int mine = 0;
        if (c < cols) {
            if (done && c0 < s_rows)
                for (int w = 0; w < W; w++) {
                    if (s_kept[w] || col >= s_have[w]) continue;
                    const int page = s_tab[w * p.tile + c];
                    bool stays = false;
#pragma unroll 4
                    for (int v = 0; v < W; v++)
                        stays |= v != w && col < s_have[v] && (s_kept[v] || v < w) && s_tab[v * p.tile + c] == page;
                    gone |= static_cast<uint64_t>(!stays) << w;
                }
            mine = __popcll(gone);
            for (int w = 0; w < W; w++) {
                int page = -1;
                if (col < s_pages[w]) {
                    page = s_tab[s_src[w] * p.tile + c];
                    if (col == s_pages[w] - 1 && s_copy[w] >= 0) {
                        p.copy[s_copy[w]].x = page;
                        page = s_fresh[w];
                    }
                }
                a.table_out[(row0 + w) * a.bo_s + col] = page;
            }
        }
        // Their places in the list: by column, then by beam.
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int at = base + incl - mine;
        for (int i = 0; i < kTableWarps; i++) {
            if (i < warp) at += s_scan[i];
            base += s_scan[i];
        }
        for (; gone; gone &= gone - 1) {
            const int page = s_tab[(__ffsll(gone) - 1) * p.tile + c];
            if (page < 0 || page >= a.num_pages) bad |= CLIS_PAGED_INDEX_BIT;
            p.back[static_cast<int64_t>(g) * W * a.width + at++] = page;
        }
        __syncthreads();  // (the tile is loaded again)
    }
    if (tid == 0) p.count[g].y = base;
    if (bad) atomicOr(&g_reorder_error_word, bad);
}

// Sum of the counts of the requests before g (both of them), over the block.
__device__ __forceinline__ longlong2 counts_before(const ReorderParams &p, int g, long long (*s)[2])
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long x = 0, y = 0;
    for (int i = tid; i < g; i += kCopyThreads) {
        const int2 c = p.count[i];
        x += c.x;
        y += c.y;
    }
    x = warp_sum(x);
    y = warp_sum(y);
    __syncthreads();
    if (lane == 0) {
        s[warp][0] = x;
        s[warp][1] = y;
    }
    __syncthreads();
    longlong2 r = make_longlong2(0, 0);
    for (int i = 0; i < kCopyWarps; i++) {
        r.x += s[i][0];
        r.y += s[i][1];
    }
    return r;
}

// The first `rows` rows of all heads of a page, by a block: a warp per head, four pieces a
// lane in flight.
template <typename T>
__device__ __forceinline__ void copy_rows(const uint8_t *from, uint8_t *to, const clis_pages_t &x, int rows, int tid)
{
    const uint32_t per = static_cast<uint32_t>(x.row_bytes) / sizeof(T), one = rows * per;
    const bool dense = x.sn == x.row_bytes;  // rows follow each other
    constexpr int B = 4;
    for (int h = tid >> 5; h < x.heads; h += kCopyWarps) {
        const int64_t head = h * x.sh;
        for (uint32_t i0 = tid & 31; i0 < one; i0 += B * 32) {
            T v[B];
            int64_t at[B];
#pragma unroll
            for (int b = 0; b < B; b++) {
                const uint32_t i = i0 + b * 32;
                if (i >= one) continue;
                const uint32_t r = dense ? 0 : i / per;
                at[b] = head + r * x.sn + (i - r * per) * sizeof(T);
                v[b] = *reinterpret_cast<const T *>(from + at[b]);
            }
#pragma unroll
            for (int b = 0; b < B; b++)
                if (i0 + b * 32 < one) *reinterpret_cast<T *>(to + at[b]) = v[b];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads, 4) reorder_copy_kernel(const ReorderParams p)
{
    const ReorderArgs &a = p.a;
    __shared__ long long s_sum[kCopyWarps][2];
    const int tid = threadIdx.x;
    unsigned int bad = 0;
    pdl_wait();
    const longlong2 all = counts_before(p, a.R, s_sum);
    const int64_t head = a.state_in[0], tail = a.state_in[1], F = a.ring_size;
    const int64_t held = tail - head, avail = held < 0 || held > F ? 0 : held;
    if (blockIdx.x == 0 && tid == 0) {
        a.state_out[0] = head + all.x;
        a.state_out[1] = tail + min(static_cast<int64_t>(all.y), F - avail);
    }
    // Pages that go back follow the ring's tail.
    const int64_t tm = ((tail % F) + F) % F;
    for (int g = blockIdx.x; g < a.R; g += gridDim.x) {
        const int n = p.count[g].y;
        const long long first = counts_before(p, g, s_sum).y;
        for (int i = tid; i < n; i += kCopyThreads) {
            if (avail + first + i >= F) bad |= CLIS_PAGED_POOL_BIT;
            else a.ring[(tm + first + i) % F] = p.back[static_cast<int64_t>(g) * a.W * a.width + i];
        }
    }
    // Copies: (page, tensor, layer) by blocks.
    uint32_t layers = 0;
    for (int t = 0; t < a.tensors; t++) layers += static_cast<uint32_t>(a.t[t].layers);
    const uint64_t units = static_cast<uint64_t>(all.x) * layers;
    for (uint64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint64_t which = div64(u, layers);
        const int4 c = p.copy[which];
        int l = static_cast<int>(u - which * layers), t = 0;
        while (l >= a.t[t].layers) l -= static_cast<int>(a.t[t++].layers);
        if (c.x < 0 || c.x >= a.num_pages || c.y < 0 || c.y >= a.num_pages) {
            bad |= CLIS_PAGED_INDEX_BIT;
            continue;
        }
        const clis_pages_t &x = a.t[t];
        const uint8_t *from = static_cast<const uint8_t *>(x.base) + l * x.sl + c.x * x.sp;
        uint8_t *to = static_cast<uint8_t *>(x.base) + l * x.sl + c.y * x.sp;
        if (a.vec[t]) copy_rows<uint4>(from, to, x, c.z, tid);
        else copy_rows<uint32_t>(from, to, x, c.z, tid);
    }
    if (bad) atomicOr(&g_reorder_error_word, bad);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t reorder_workspace(const ReorderArgs &a)
{
    const size_t rows = static_cast<size_t>(a.R) * a.W;
    return up256(a.R * sizeof(int2)) + up256(rows * sizeof(int4)) + up256(rows * a.width * sizeof(int));
}

clis_status_t launch_reorder(const ReorderArgs &a, void *workspace, int nsm, cudaStream_t stream)
{
    ReorderParams p;
    p.a = a;
    p.tile = kTableThreads;
    while (p.tile * a.W * sizeof(int) > 40 * 1024) p.tile /= 2;
    char *w = static_cast<char *>(workspace);
    p.count = reinterpret_cast<int2 *>(w);
    w += up256(a.R * sizeof(int2));
    p.copy = reinterpret_cast<int4 *>(w);
    w += up256(static_cast<size_t>(a.R) * a.W * sizeof(int4));
    p.back = reinterpret_cast<int *>(w);
    reorder_table_kernel<<<a.R, kTableThreads, p.tile * a.W * sizeof(int), stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CLIS_ERR_CUDA;
    // (blocks without a copy or a request of their own end at once)
    return launch_pdl(reorder_copy_kernel, dim3(8 * nsm), kCopyThreads, 0, stream, p) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t read_reorder_error(uint32_t *code)
{
    return cudaMemcpyFromSymbol(code, g_reorder_error_word, sizeof *code) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

clis_status_t clear_reorder_error()
{
    const unsigned int z = 0;
    return cudaMemcpyToSymbol(g_reorder_error_word, &z, sizeof z) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
}

}  // namespace clis
