// paged_internal.h -- declarations shared by the C-ABI layer and the kernels
// around a paged key/value cache: rotary positions, the write into the cache,
// the plan of a serving step, and attention over the cache.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/clis.h"
#include "paged_sched.h"

namespace clis {

// ------------------------------------------------- rotary positions, append

struct RotArgs {
    // Heads 0..Hq-1 are q's, then Hk of k, then (append) Hk of v, which is
    // copied as it is.  With `slots`, k's and v's destinations are the caches:
    // their sb, sh, sn are the page, head and in-page row strides.
    const uint16_t *q, *k, *v;
    uint16_t *qo, *ko, *vo;
    int64_t q_sb, q_sh, q_sn, k_sb, k_sh, k_sn, v_sh, v_sn;
    int64_t qo_sb, qo_sh, qo_sn, ko_sb, ko_sh, ko_sn, vo_sb, vo_sh, vo_sn;
    const int32_t *pos;
    int64_t p_sb, p_sn, p_sa;
    const double *inv_freq;
    const int32_t *axis;
    const int64_t *slots;  // nullptr: plain rotation
    int64_t num_slots;     // pages * page size
    int page_shift;        // log2 of the page size
    int B, Hq, Hk, N, d;
    int pairs, axes;
    int interleaved, inverse;
    int dtype;
};

clis_status_t launch_rot(const RotArgs &a, cudaStream_t stream);

// --------------------------------------------------------------------- plan

struct PlanArgs {
    const int32_t *ctx_len, *new_len;
    int32_t *block_table;
    int64_t bt_s;
    int32_t *ring;
    int64_t ring_size;
    const int64_t *state_in;
    int64_t *state_out;
    int32_t *cu_q, *kv_len;
    int64_t *slots;
    int32_t *pos;
    int S, T, width, page_shift;
    int64_t num_pages;
};

clis_status_t launch_paged_plan(const PlanArgs &a, cudaStream_t stream);

// ---------------------------------------------------------------- attention

struct PagedArgs {
    const uint16_t *q, *kc, *vc;
    uint16_t *o;
    float *lse2;
    const int32_t *block_table, *cu_q, *kv_len;
    int64_t q_st, q_sh, o_st, o_sh, kc_sp, kc_sh, kc_sn, vc_sp, vc_sh, vc_sn, bt_s;
    int64_t num_pages;
    int S, T, H, Hkv, d, dtype, page_shift, width;
    float scale_log2;
    int causal;
};

#ifdef __CUDACC__
// Programmatic dependent launch.  A kernel launched by launch_pdl may start while
// the kernel before it in the stream still runs; pdl_wait returns once that
// kernel has ended and its writes are visible.  Every kernel of a chain calls it,
// so the end of one implies the end of all before it.  pdl_launch lets the next
// kernel be set up (it changes nothing for correctness).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

// Row tiles (of 16 rows) per sequence that the decode kernel is built for, when
// no sequence has more than max_q new tokens: 1, 2 (d = 64), or 0 (not used).
int paged_decode_row_tiles(int64_t max_q, int g, int d);
size_t paged_decode_workspace(int d, int row_tiles, int nsm);
// strict: no chunk kernel follows, a sequence of more rows is an error.
// after_schedule: launched behind launch_paged_chunk_schedule, whose results it
// does not read.
clis_status_t launch_paged_decode(const PagedArgs &a, int row_tiles, bool strict, bool after_schedule, void *workspace,
                                  int nsm, cudaStream_t stream);
size_t paged_chunk_workspace(const PagedArgs &a, int nsm);
// Sequences of at most rows_small query rows are left to the decode kernel.
// Schedule first, then (with rows_small > 0) the decode kernel, then the chunk kernel:
// each of these kernels but the first may be set up while the one before it
// still runs, and waits for it before it reads its results.
clis_status_t launch_paged_chunk_schedule(const PagedArgs &a, int rows_small, void *workspace, int nsm,
                                          cudaStream_t stream);
clis_status_t launch_paged_chunk(const PagedArgs &a, int rows_small, void *workspace, int nsm, cudaStream_t stream);

// Device error words of these kernels (CLIS_PAGED_* bits and wait bits), one
// per translation unit; read after a device synchronisation.
clis_status_t read_rot_error(uint32_t *code);
clis_status_t clear_rot_error();
clis_status_t read_plan_error(uint32_t *code);
clis_status_t clear_plan_error();
clis_status_t read_decode_error(uint32_t *code);
clis_status_t clear_decode_error();
clis_status_t read_chunk_error(uint32_t *code);
clis_status_t clear_chunk_error();

}  // namespace clis
