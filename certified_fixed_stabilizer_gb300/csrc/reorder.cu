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

// What a request wants: pages for copies, and whether its inputs make sense.
struct Wish {
    int need;
    unsigned int bad;
};

__device__ __forceinline__ Wish wish_of(const ReorderArgs &a, int g)
{
    Wish r = {0, 0u};
    const int cap = a.width << a.page_shift, mask = (1 << a.page_shift) - 1;
    const int32_t *parent = a.parent + static_cast<int64_t>(g) * a.W, *lens = a.lens + static_cast<int64_t>(g) * a.W;
    unsigned long long seen = 0;  // beams that some beam has gone on from
    for (int w = 0; w < a.W; w++) {
        const int p = __ldg(parent + w), n = __ldg(lens + w);
        if (n < 0 || n > cap) r.bad |= CLIS_PAGED_LENGTH_BIT;
        if (p >= a.W) r.bad |= CLIS_PAGED_INDEX_BIT;
        if (p < 0 || p >= a.W) continue;
        if ((seen >> p & 1) && (__ldg(lens + p) & mask)) r.need++;
        seen |= 1ull << p;
    }
    if (r.bad) r.need = 0;
    return r;
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
    __shared__ int s_done, s_rows;
    __shared__ long long s_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x, W = a.W;
    const int mask = (1 << a.page_shift) - 1;
    unsigned int bad = 0;
    pdl_launch();

    // ---- pages that the requests before this one take
    long long before = 0;
    for (int i = tid; i < g; i += kTableThreads) before += wish_of(a, i).need;
    before = warp_sum(before);
    if (lane == 0) s_sum[warp] = before;
    __syncthreads();
    const int64_t head = a.state_in[0], held = a.state_in[1] - head, F = a.ring_size;
    if (tid == 0) {
        before = 0;
        for (int i = 0; i < kTableWarps; i++) before += s_sum[i];
        const Wish mine = wish_of(a, g);
        const bool sane = held >= 0 && held <= F;
        s_done = !mine.bad && (mine.need == 0 || (sane && before + mine.need <= held));
        if (!sane || (!mine.bad && !s_done)) bad |= CLIS_PAGED_POOL_BIT;
        bad |= mine.bad;
        s_before = before;
        s_rows = 0;
        a.done[g] = s_done;
        p.count[g].x = s_done ? mine.need : 0;
    }
    __syncthreads();
    // A thread per beam: whom it goes on from, and whether it needs a copy.
    const int64_t row0 = static_cast<int64_t>(g) * W;
    int src = -1, len = 0;
    if (tid < W) {
        const int n = __ldg(a.lens + row0 + tid), ok = min(max(n, 0), a.width << a.page_shift);
        s_len[tid] = n;
        s_have[tid] = (ok >> a.page_shift) + ((ok & mask) ? 1 : 0);
        atomicMax(&s_rows, s_have[tid]);
        src = s_done ? __ldg(a.parent + row0 + tid) : tid;
        s_src[tid] = src;
        s_kept[tid] = false;
    }
    __syncthreads();
    if (tid < W) {
        len = src < 0 ? 0 : s_len[src];
        a.lens_out[row0 + tid] = len;
        s_pages[tid] = src < 0 ? 0 : s_have[src];
        bool again = false;
        for (int v = 0; v < tid; v++) again |= s_src[v] == src;
        if (src >= 0) s_kept[src] = true;  // (several threads write the same)
        s_again[tid] = again && src >= 0 && (len & mask) != 0 && s_done;
    }
    __syncthreads();
    if (tid < W) {
        s_copy[tid] = -1;
        if (s_again[tid]) {
            long long i = s_before;
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
    const bool done = s_done != 0;
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
        auto gone = [&](int w) -> bool {  // beam w's page of this column goes back, and beam w says so
            if (s_kept[w] || col >= s_have[w]) return false;
            const int page = s_tab[w * p.tile + c];
            for (int v = 0; v < W; v++)
                if (v != w && col < s_have[v] && s_tab[v * p.tile + c] == page && (s_kept[v] || v < w)) return false;
            return true;
        };
        int mine = 0;
        if (c < cols) {
            if (done && c0 < s_rows)
                for (int w = 0; w < W; w++) mine += gone(w);
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
        if (mine > 0)
            for (int w = 0; w < W; w++)
                if (gone(w)) {
                    const int page = s_tab[w * p.tile + c];
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

__global__ void __launch_bounds__(kCopyThreads) reorder_copy_kernel(const ReorderParams p)
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
    int64_t layers = 0;
    for (int t = 0; t < a.tensors; t++) layers += a.t[t].layers;
    for (int64_t u = blockIdx.x; u < all.x * layers; u += gridDim.x) {
        const int4 c = p.copy[u / layers];
        int l = static_cast<int>(u % layers), t = 0;
        while (l >= a.t[t].layers) l -= static_cast<int>(a.t[t++].layers);
        if (c.x < 0 || c.x >= a.num_pages || c.y < 0 || c.y >= a.num_pages) {
            bad |= CLIS_PAGED_INDEX_BIT;
            continue;
        }
        const clis_pages_t &x = a.t[t];
        const uint8_t *from = static_cast<const uint8_t *>(x.base) + l * x.sl + c.x * x.sp;
        uint8_t *to = static_cast<uint8_t *>(x.base) + l * x.sl + c.y * x.sp;
        const bool vec = a.vec[t] != 0;
        const int size = vec ? 16 : 4, per = static_cast<int>(x.row_bytes) / size, one = c.z * per;
        const int total = static_cast<int>(x.heads) * one;
        for (int i = tid; i < total; i += kCopyThreads) {
            const int h = i / one, e = i - h * one, r = e / per;
            const int64_t at = h * x.sh + r * x.sn + (e - r * per) * size;
            if (vec) *reinterpret_cast<uint4 *>(to + at) = *reinterpret_cast<const uint4 *>(from + at);
            else *reinterpret_cast<uint32_t *>(to + at) = *reinterpret_cast<const uint32_t *>(from + at);
        }
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
    return launch_pdl(reorder_copy_kernel, dim3(4 * nsm), kCopyThreads, 0, stream, p) == cudaSuccess ? CLIS_OK : CLIS_ERR_CUDA;
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
