/*
 * clis.h -- C ABI of the CLiS attention library (libclis.so), sm_103a.
 *
 * CLiS ("CLiS: Plug-and-Play Attention Acceleration for Video Diffusion on
 * TPUs via Certified Stabilization", Tsai et al., 2026) fixes one softmax
 * stabiliser per query row before the KV loop, so the fused attention kernel
 * needs no running row maximum and no accumulator rescaling.  A per-head
 * certificate (Algorithm 1) proves that doing so cannot overflow; heads that
 * fail certification run standard online softmax instead (abstract).
 *
 * Conventions shared by every entry point:
 *  - Tensors are bf16 (or fp16, shape->dtype) in layout [B, H, N, d] with
 *    element strides given in clis_shape_t; the d dimension is contiguous.
 *  - Device pointers must be 16-byte aligned and every stride (n, h, b) a
 *    multiple of 8 elements (16 bytes); otherwise CLIS_ERR_MISALIGNED.
 *  - d must be 64 or 128 (CLIS_ERR_UNSUPPORTED otherwise).
 *  - The caller owns every buffer.  The library allocates no device memory;
 *    scratch space is passed in as `workspace`.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and never synchronise the host.  The returned status
 *    covers argument checks and launch errors only: on any argument error
 *    nothing is launched.  Faults found inside a kernel (a pipeline wait
 *    that exceeded its time limit) are recorded in a device-side error word
 *    read by clis_get_device_error().
 *  - All results are deterministic: every floating-point sum has a fixed
 *    order.  (The one place that adds through memory, the KV-chunk merge of
 *    certified heads, adds one value per accumulator element per launch, so
 *    the order is the launch order.  The certification combines partial
 *    maxima with atomic max operations, which are exact in any order.)
 */
#ifndef CLIS_H
#define CLIS_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CLIS_API __attribute__((visibility("default")))
#else
#define CLIS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque CUDA stream handle, ABI-compatible with cudaStream_t. */
typedef struct CUstream_st *clis_stream_t;

typedef enum {
    CLIS_OK = 0,
    CLIS_ERR_INVALID_ARG = 1,  /* null pointer, negative/zero size, bad enum or dtype, non-finite or <= 0 scale */
    CLIS_ERR_UNSUPPORTED = 2,  /* head dim not in {64, 128}, causal with Nq != Nk, sizes beyond int32 */
    CLIS_ERR_MISALIGNED = 3,   /* pointer not 16-byte aligned or stride not a multiple of 8 elements */
    CLIS_ERR_WORKSPACE = 4,    /* workspace null or smaller than clis_certify_workspace_size() */
    CLIS_ERR_CUDA = 5,         /* a CUDA runtime/driver call or a kernel launch failed */
    CLIS_ERR_TIMEOUT = 6,      /* a kernel pipeline wait exceeded its limit (device error word) */
    CLIS_ERR_DATA = 7          /* device data (lengths, page numbers, slots) out of range (device error word) */
} clis_status_t;

/* Floating-point formats whose exp2 overflow limits Figure 3 tabulates (FP16,
 * BF16, FP32).  U_exp and U_acc of Algorithm 1 step 7 are those limits for
 * the format holding exp2 outputs and for the accumulator format. */
typedef enum { CLIS_FMT_FP16 = 0, CLIS_FMT_BF16 = 1, CLIS_FMT_FP32 = 2 } clis_fmt_t;

/* Which softmax the attention kernel runs per head:
 *  CLIS_AUTO              certified heads use the fixed stabiliser, the rest
 *                         fall back to online softmax (the fallback the
 *                         abstract describes for heads that fail);
 *  CLIS_ONLINE            every head uses online softmax that rescales the
 *                         accumulator after every KV block (the baseline);
 *  CLIS_CERTIFIED_FORCED  every head uses the fixed stabiliser, ignoring the
 *                         flags (benchmarks and tests only: output of a head
 *                         that did not certify is then unspecified);
 *  CLIS_ONLINE_LAZY       every head uses online softmax that rescales only
 *                         when a row maximum grows by more than 8 (exp2 units),
 *                         the FlashAttention-4-style baseline the paper adapts
 *                         as "FA4-style (row)" (Tables 5 and 8); needs no
 *                         certificate. */
typedef enum {
    CLIS_AUTO = 0,
    CLIS_ONLINE = 1,
    CLIS_CERTIFIED_FORCED = 2,
    CLIS_ONLINE_LAZY = 3
} clis_variant_t;

/* Element type of Q, K, V and O (all four share it).  The attention kernel
 * feeds P to the tensor cores in the same type, so with FP16 data the exp2
 * outputs are FP16 (Figure 3: U_exp = 15.9993): certify FP16 data with
 * exp_fmt = CLIS_FMT_FP16.  As a safeguard, in CLIS_AUTO an FP16 head takes the
 * fixed-stabiliser path only if its certificate also satisfies
 * B_h <= min(15, C); otherwise it runs online softmax. */
typedef enum { CLIS_DT_BF16 = 0, CLIS_DT_FP16 = 1 } clis_dtype_t;

/* Problem shape and element strides (elements, not bytes).  K and V share
 * Nk; Q and O share Nq.  O strides are ignored by clis_certify.  dtype is a
 * clis_dtype_t (0 = BF16, the zero-initialised default).
 *
 * Strides are non-negative, n-strides at least d.  A head or batch stride of
 * 0 on K and V makes the heads (or batches) read one K/V head: grouped-query
 * and multi-query attention map onto it by folding the key/value heads into
 * the batch (B' = B * H_kv, H' = query heads per key/value head, K and V
 * head stride 0, batch stride one K/V head).  Each query head is then
 * certified against the shared keys and values like any other head.  Strides
 * of anything written must not make two elements share an address: an O (or,
 * in the backward, dQ, dK, dV) head stride of 0 with H > 1 or batch stride of
 * 0 with B > 1 is CLIS_ERR_INVALID_ARG, with one exception: the backward
 * writes dK and dV with the K and V strides, and when K and V are broadcast
 * over the heads together (both head strides 0) it sums the gradients of all
 * H query heads into each dK and dV row and writes it once. */
typedef struct {
    int64_t B, H, Nq, Nk, d;
    int64_t q_sb, q_sh, q_sn;
    int64_t k_sb, k_sh, k_sn;
    int64_t v_sb, v_sh, v_sn;
    int64_t o_sb, o_sh, o_sn;
    int64_t dtype;
} clis_shape_t;

/* Per-head certificate, Algorithm 1 (one per (b, h) pair, index b*H + h).
 *  certified  1 if every input of the head is finite and B_h <= C
 *  G          step 5: ceil(log2 max(1, max |V|))
 *  A          step 6: ceil(log2 Nk) + G
 *  C          step 7: min(floor(U_exp), ceil(U_acc - A) - 1)
 *  reason     0 certified, 1 B_h > C, 2 a non-finite value in Q, K or V
 *             (then G = A = C = 0 and B_h = +inf)
 *  B_h        step 4 with BoundUp(q, kappa) = scale_log2 * ||q||_2 * kappa,
 *             rounded upward (exp2-argument units)
 *  kappa      step 3: an upper bound on max_r ||k_r - kbar||_2 computed
 *             with upward rounding about the kbar returned by clis_certify
 *  qmax       an upper bound on max_r ||q_r||_2 */
typedef struct {
    int32_t certified, G, A, C, reason;
    float B_h, kappa, qmax;
} clis_head_cert_t;

/* Bytes of device workspace clis_certify needs for this shape.
 * Host-only; never touches the GPU.  Errors: CLIS_ERR_INVALID_ARG for a
 * null argument or a negative size. */
CLIS_API clis_status_t clis_certify_workspace_size(const clis_shape_t *shape, size_t *bytes);

/* Certification pre-pass, Algorithm 1 steps 1-7 plus the decision, for all
 * B*H heads (Algorithm 1 certifies one dense attention head; here every
 * (b, h) pair is one such head).  The decision after step 7 is lost from the
 * text; it is read here as: every input finite and B_h <= C.
 *   q, k, v     device bf16 [B,H,Nq,d] / [B,H,Nk,d] / [B,H,Nk,d]
 *   scale_log2  softmax scale times log2(e) (> 0, finite); scores enter
 *               exp2 as scale_log2 * q.k
 *   exp_fmt     format that holds exp2 outputs (U_exp); the attention
 *               kernel feeds P to the tensor cores as BF16
 *   acc_fmt     accumulator format (U_acc); the kernel accumulates in FP32
 *   kbar        device fp32 out [B*H, d]: step 1 key mean, round-to-nearest
 *   certs       device out [B*H]
 *   mu          optional device fp32 out [B*H*Nq] (index (b*H + h)*Nq + i):
 *               the per-row stabilisers mu_i = scale_log2 * (q_i . kbar) that
 *               the certified path fixes before the KV loop (Figure 5(a));
 *               pass it to clis_attn_fwd so the kernel need not recompute
 *               them.  NULL = skip.
 *   workspace   device scratch of at least clis_certify_workspace_size()
 *               bytes, 256-byte aligned; contents need no initialisation
 * Launches four kernels on `stream`.  Nk must be >= 1; Nq may be 0. */
CLIS_API clis_status_t clis_certify(const clis_shape_t *shape, const void *q, const void *k,
                           const void *v, float scale_log2, clis_fmt_t exp_fmt,
                           clis_fmt_t acc_fmt, float *kbar, clis_head_cert_t *certs,
                           float *mu, void *workspace, size_t ws_bytes, clis_stream_t stream);

/* Size in bytes of the scratch buffer that clis_certify_noalloc uses instead
 * of a caller workspace (a fixed array inside the library). */
#define CLIS_NOALLOC_SCRATCH_BYTES (4u << 20)

/* clis_certify for callers that must not allocate device memory.  The paper
 * has no counterpart to this entry point: it exists for code that runs where
 * cudaMalloc is off limits -- a plugin or custom operator inside another
 * runtime that owns all device memory and hands out no workspace, a serving
 * loop whose memory was planned up front, or any caller for whom an
 * allocation would synchronise the device or break the host's accounting.
 *
 * Same arguments and results as clis_certify minus the workspace: the
 * scratch lives in one library-owned device array of
 * CLIS_NOALLOC_SCRATCH_BYTES, which every GPU that loads the library keeps
 * until the process exits.  The caller still provides q, k, v, kbar and
 * certs.  Nothing is allocated or freed, by this call or by any routine it
 * uses.
 *   - The first call on a device (with that device current) does the set-up:
 *     it looks up the array's device address with cudaGetSymbolAddress (which
 *     allocates nothing).  Make that first call before any stream capture on
 *     that device.  Later calls made outside capture repeat the lookup in the
 *     current context, so a device reset or another context gets its own
 *     address; a call made while `stream` is being captured does no lookup and
 *     uses the address of the last lookup in the same context (CLIS_ERR_CUDA
 *     if there was none).
 *   - All calls share the one array and it keeps what the last call left in
 *     it.  The kernels overwrite every scratch word they read, so nothing
 *     needs clearing between calls, but calls that overlap on the GPU (two
 *     streams, two host threads) race on it: serialise them.
 *   - Arguments are checked first, with the statuses of clis_certify.  Then
 *     shapes whose clis_certify_workspace_size() exceeds
 *     CLIS_NOALLOC_SCRATCH_BYTES return CLIS_ERR_WORKSPACE before anything
 *     is launched (about B*H*ceil(Nk/1024)*d*4 bytes; B*H = 40 heads of
 *     75,600 keys at d = 128 need 1.6 MB).
 *   - CLIS_ERR_CUDA if the address lookup fails. */
CLIS_API clis_status_t clis_certify_noalloc(const clis_shape_t *shape, const void *q, const void *k,
                                   const void *v, float scale_log2, clis_fmt_t exp_fmt,
                                   clis_fmt_t acc_fmt, float *kbar, clis_head_cert_t *certs,
                                   float *mu, clis_stream_t stream);

/* Fused attention forward O = softmax(scale * Q K^T) V (abstract and
 * Figure 5(a): with mu_i fixed before the KV loop, the loop needs no running
 * maximum and no rescaling).  One persistent kernel; each 256-row query block of a
 * head runs either
 *   - the certified path: mu_i = scale_log2 * (q_i . kbar) fixed before the
 *     KV loop, p_ij = exp2(scale_log2 * s_ij - mu_i), no row maximum, no
 *     rescaling; or
 *   - the online path: running row maximum and accumulator rescaling.
 *   o       device bf16 out [B,H,Nq,d] (strides from shape)
 *   lse2    optional device fp32 out [B*H*Nq] (contiguous, index
 *           (b*H + h)*Nq + i): log2 sum_j exp2(scale_log2 * s_ij); NULL = skip
 *   kbar, certs  outputs of clis_certify (may be NULL for CLIS_ONLINE and
 *           CLIS_ONLINE_LAZY)
 *   mu      optional per-row stabilisers from clis_certify (NULL: the kernel
 *           computes mu_i from q_i and kbar itself)
 *   causal  0 or 1; 1 requires Nq == Nk (key j visible to query i iff j <= i)
 * Nq == 0 or B*H == 0 launches nothing and returns CLIS_OK. */
CLIS_API clis_status_t clis_attn_fwd(const clis_shape_t *shape, const void *q, const void *k,
                            const void *v, void *o, float *lse2, const float *kbar,
                            const clis_head_cert_t *certs, const float *mu, float scale_log2,
                            int causal, clis_variant_t variant, clis_stream_t stream);

/* The forward for Q, K, V and O held in host memory (the abstract's
 * plug-and-play use: the attention call of a model whose tensors live on the
 * host).  Per group of consecutive heads: copy Q, K, V to the device, run
 * clis_certify (variants CLIS_AUTO and CLIS_CERTIFIED_FORCED; exp2 format of
 * the data type, FP32 accumulation) and clis_attn_fwd with its stabilisers,
 * copy O back.  The copies of one group overlap the kernels of others: copies
 * in on one stream of the plan, the kernels of even and odd groups on two
 * more, copies out on a fourth.  Each head is computed alone by the kernels
 * of clis_certify and clis_attn_fwd, so k-bar and the certificates equal
 * theirs on the whole tensors bit for bit; O may differ from their O by
 * rounding, because the attention kernel sweeps the keys of some work tiles
 * in reverse order depending on where the tile falls in its launch.
 *
 * clis_host_plan_create: a plan for one shape on the current device: its
 *   four streams and per-group events.  shape is as for clis_attn_fwd, but
 *   Q, K, V and O must be dense (n-stride d, head stride N*d, batch stride
 *   H*N*d, free when B = 1; CLIS_ERR_UNSUPPORTED otherwise); causal as for
 *   clis_attn_fwd; groups = number of head groups, 0 = about one group per
 *   2 TFLOP of attention work, at least 8 and at most B*H.  Argument errors
 *   as for clis_attn_fwd; CLIS_ERR_CUDA if a stream or event cannot be made.
 * clis_host_plan_workspace_size: bytes of device workspace every call with
 *   the plan needs: staging for Q, K, V and O of every head, k-bar,
 *   certificates and stabilisers, and two certification scratch areas (0 when
 *   B*H = 0 or Nq = 0).
 * clis_attention_host: one forward with the plan.
 *   q, k, v, o  host memory, any alignment; o is written.  Page-locked memory
 *               (cudaHostAlloc, cudaHostRegister) lets the copies run
 *               asynchronously; with pageable memory the CUDA runtime stages
 *               each copy and the call returns only after its copies ran.
 *   scale_log2, variant  as for clis_attn_fwd
 *   workspace   device memory of clis_host_plan_workspace_size() bytes,
 *               256-byte aligned, the same for every call with the plan.  Once
 *               the call is complete, its first B*H*d floats hold k-bar and the
 *               B*H certificates start at the next multiple of 256 bytes
 *               (certified variants).
 *   stream      the copies in follow the work queued on it before the call
 *   The call is queued, not waited for.  Calls with one plan must come from
 *   one host thread at a time (the plan records its events in each call).  Consecutive calls with one plan
 *   overlap: a call's copies of a group start once the previous call's
 *   kernels on that group have run, and its kernels once the previous call's
 *   copy out of that group has.  Must be called on the plan's device
 *   (CLIS_ERR_INVALID_ARG otherwise).  Errors: the argument checks of
 *   clis_attn_fwd, CLIS_ERR_WORKSPACE, CLIS_ERR_MISALIGNED for the
 *   workspace, all before anything is queued; CLIS_ERR_CUDA when a copy or
 *   launch fails, after which clis_host_plan_wait still covers everything the
 *   call queued.  B*H = 0 or Nq = 0 returns CLIS_OK and queues nothing.
 * clis_host_plan_wait: makes `stream` wait for the last copy out of the most
 *   recent call with the plan (nothing if there was none): o of that call and
 *   of every earlier one is complete once `stream` passes this point.
 * clis_host_plan_destroy: releases the plan (NULL is a no-op); work already
 *   queued still runs, and the CUDA runtime frees the streams and events
 *   after it.  The workspace may be reused or freed once that work is done. */
typedef struct clis_host_plan_s clis_host_plan_t;
CLIS_API clis_status_t clis_host_plan_create(const clis_shape_t *shape, int causal, int groups,
                                             clis_host_plan_t **plan);
CLIS_API clis_status_t clis_host_plan_workspace_size(const clis_host_plan_t *plan, size_t *bytes);
CLIS_API clis_status_t clis_attention_host(clis_host_plan_t *plan, const void *q, const void *k,
                                           const void *v, void *o, float scale_log2,
                                           clis_variant_t variant, void *workspace, size_t ws_bytes,
                                           clis_stream_t stream);
CLIS_API clis_status_t clis_host_plan_wait(clis_host_plan_t *plan, clis_stream_t stream);
CLIS_API clis_status_t clis_host_plan_destroy(clis_host_plan_t *plan);

/* FP8 P.V path.  Figure 3 tabulates exp2 limits per format; one step below
 * FP16 is E4M3 (largest finite value 448, so U_exp = log2 448 and the budget
 * is floor(U_exp) = 8).  One tcgen05.mma of kind::f8f6f4 takes both operands
 * in 8 bits, so P in E4M3 needs V in E4M3 too.  A head takes this path when it
 * certifies (clis_certify, BF16/FP32 formats) and also B_h <= min(8, C) and
 * G <= 8 (max |V| <= 256 fits E4M3) -- these make E4M3 safe -- and, for
 * accuracy, Nk >= 4096; every other head runs exactly as in clis_attn_fwd
 * (certified BF16 path or online softmax).  The row sum stays the fp32 sum of
 * the unrounded exp2 outputs.  Accuracy: V's E4M3 rounding (up to 2^-4
 * relative per entry) averages over the keys, so on diffuse heads the mean
 * output error is about 0.033 / sqrt(Nk) (2e-4 at 32,760 keys, 1.4e-3 at 513)
 * and the largest about ten times the BF16 path's; sharp heads (B_h above 8)
 * never qualify.
 *
 * clis_v_e4m3_size: bytes of the E4M3 V^T buffer, B*H*d*pitch with pitch =
 *   Nk rounded up to 16.
 * clis_v_to_e4m3: writes V^T [b*H + h][c][j] = E4M3(V[b, h, j, c]) (round to
 *   nearest even, saturating at +-448; bytes from Nk to the pitch are 0).
 *   BF16 V only (CLIS_ERR_UNSUPPORTED for FP16); vt8 16-byte aligned.
 * clis_attn_fwd_fp8pv: clis_attn_fwd (no mask) for d = 128 and BF16 data
 *   (CLIS_ERR_UNSUPPORTED otherwise) that also takes vt8 from clis_v_to_e4m3
 *   of the same v.  variant: CLIS_AUTO (the rule above) or
 *   CLIS_CERTIFIED_FORCED (every head on the FP8 P.V path whatever its
 *   certificate or length: benchmarks and tests only); other variants
 *   CLIS_ERR_INVALID_ARG. */
CLIS_API clis_status_t clis_v_e4m3_size(const clis_shape_t *shape, size_t *bytes);
CLIS_API clis_status_t clis_v_to_e4m3(const clis_shape_t *shape, const void *v, void *vt8, clis_stream_t stream);
CLIS_API clis_status_t clis_attn_fwd_fp8pv(const clis_shape_t *shape, const void *q, const void *k,
                                           const void *v, const void *vt8, void *o, float *lse2,
                                           const float *kbar, const clis_head_cert_t *certs, const float *mu,
                                           float scale_log2, clis_variant_t variant, clis_stream_t stream);

/* The ring-step form (clis_attn_fwd_chunk, no mask) with the FP8 P.V path:
 * vt8 is clis_v_to_e4m3 of the chunk's v (k and v point at the chunk, shape->Nk
 * its length); a head takes E4M3 by the rule above, with Nk the chunk's
 * length.  Certified heads still merge by plain addition.  Other arguments
 * and errors as clis_attn_fwd_chunk and clis_attn_fwd_fp8pv. */
CLIS_API clis_status_t clis_attn_fwd_chunk_fp8pv(const clis_shape_t *shape, const void *q, const void *k,
                                                 const void *v, const void *vt8, float *o_acc, float *l_acc,
                                                 float *m_acc, const float *kbar, const clis_head_cert_t *certs,
                                                 const float *mu, float scale_log2, int first,
                                                 clis_variant_t variant, clis_stream_t stream);

/* Per-prefix certificates for causal attention: clis_certify plus one flag per
 * block of 256 query rows.  The pages certify causal heads with the head's
 * bound (Table 3) and state no finer rule; this entry point is a finer reading
 * of the same Cauchy-Schwarz bound.  A causal row i sees keys 0..i only, so
 * for query block b (rows 256b .. 256b + 255) every exp2 argument is bounded
 * by B_b = scale_log2 * max_{i in b} ||q_i|| * max_{j <= 256b + 255}
 * ||k_j - kbar|| (rounded upward as B_h is), and the block is safe when the
 * head's inputs are finite and B_b <= C, the head's budget.  A certified head
 * has every block certified; a head that fails can still certify the blocks
 * whose prefixes exclude its large keys.
 *   tile_certs  device uint8 out [B*H][ceil(Nq / 256)]: 1 = the block may take
 *               the fixed stabiliser in clis_attn_fwd_tiles
 *   (other arguments as for clis_certify; Nq must equal Nk)
 * Errors as for clis_certify; CLIS_ERR_INVALID_ARG for a null tile_certs,
 * CLIS_ERR_UNSUPPORTED if Nq != Nk. */
CLIS_API clis_status_t clis_certify_tiles(const clis_shape_t *shape, const void *q, const void *k,
                                          const void *v, float scale_log2, clis_fmt_t exp_fmt,
                                          clis_fmt_t acc_fmt, float *kbar, clis_head_cert_t *certs,
                                          float *mu, uint8_t *tile_certs, void *workspace,
                                          size_t ws_bytes, clis_stream_t stream);

/* clis_attn_fwd for causal attention (causal = 1, variant = CLIS_AUTO) that
 * also takes the per-prefix certificates of clis_certify_tiles: a query block
 * of a head that failed certification as a whole still takes the fixed
 * stabiliser when its block flag is set (for FP16 data only if the head's
 * budget C <= 15).  Errors as for clis_attn_fwd; CLIS_ERR_INVALID_ARG for a
 * null tile_certs, causal = 0 or another variant. */
CLIS_API clis_status_t clis_attn_fwd_tiles(const clis_shape_t *shape, const void *q, const void *k,
                                           const void *v, void *o, float *lse2, const float *kbar,
                                           const clis_head_cert_t *certs, const uint8_t *tile_certs,
                                           const float *mu, float scale_log2, int causal,
                                           clis_variant_t variant, clis_stream_t stream);

/* One KV chunk of a ring / context-parallel attention step (paper: Table 7,
 * the ring and 2D-ring columns, and Figure 6, one ring attention step).  The
 * keys and values of a head are split into chunks that arrive one at a time;
 * each call runs the fused kernel over one chunk (shape->Nk = its length, k and
 * v point at it) and merges the chunk's partial result into fp32 accumulators
 * kept by the caller (contiguous, index (b*H + h)*Nq + i):
 *   o_acc [B*H*Nq*d]  sum_j 2^(x_ij - m_i) v_j over the keys merged so far
 *   l_acc [B*H*Nq]    sum_j 2^(x_ij - m_i)
 *   m_acc [B*H*Nq]    the shift m_i (exp2 units), x_ij = scale_log2 * q_i . k_j
 * first = 1 overwrites the accumulators (first chunk), 0 merges.  A certified
 * head's shift is its fixed stabiliser mu_i in every chunk, so its partials
 * add with no exponentials, no rescaling and no read of the accumulators
 * (in-memory vector adds); other heads read the accumulators and merge by
 * rescaling to the larger maximum.  Calls on one set of accumulators must
 * be ordered (one stream, or events between streams).  kbar, certs (and mu, optional) must come from
 * clis_certify over the whole key sequence (for a ring: the k-bar partials and norm maxima of all
 * chunks reduced before the first step).  Non-causal (clis_attn_fwd_chunk_causal is the causal
 * form); shape->o_* ignored.
 * Errors as clis_attn_fwd. */
CLIS_API clis_status_t clis_attn_fwd_chunk(const clis_shape_t *shape, const void *q, const void *k,
                                  const void *v, float *o_acc, float *l_acc, float *m_acc,
                                  const float *kbar, const clis_head_cert_t *certs,
                                  const float *mu, float scale_log2, int first,
                                  clis_variant_t variant, clis_stream_t stream);

/* Causal form of clis_attn_fwd_chunk (Table 7's ring columns and Figure 6's
 * ring step, for the causal training setting of Table 3): the chunk holds keys
 * key_offset .. key_offset + shape->Nk - 1 of the head (k and v point at the
 * chunk's first key), q all shape->Nq query rows, and query i sees chunk key j
 * iff key_offset + j <= i.  Rows before key_offset see none of the chunk's
 * keys and their accumulators are left untouched; query blocks of 256 rows that
 * end before key_offset are not computed at all.  The partials merge as in
 * clis_attn_fwd_chunk: a certified row's shift is its fixed mu_i in every chunk,
 * so its partial is added with no rescaling, in any chunk order.
 *   key_offset  >= 0, with key_offset + shape->Nk <= shape->Nq
 *               (CLIS_ERR_UNSUPPORTED otherwise)
 *   first       1 overwrites the accumulators of every row: only the chunk
 *               with key_offset = 0 may be first (CLIS_ERR_INVALID_ARG
 *               otherwise); the other chunks follow in any order
 *   tile_certs  optional per-prefix certificates from clis_certify_tiles over
 *               the whole sequence (NULL: per-head flags only); a query block
 *               whose flag is set takes the fixed stabiliser in every chunk
 *               (CLIS_AUTO only; CLIS_ERR_INVALID_ARG with another variant)
 *   kbar, certs, mu  from clis_certify (or clis_certify_tiles) over the whole
 *               sequence
 * Other arguments and errors as clis_attn_fwd_chunk. */
CLIS_API clis_status_t clis_attn_fwd_chunk_causal(const clis_shape_t *shape, const void *q, const void *k,
                                                  const void *v, float *o_acc, float *l_acc, float *m_acc,
                                                  const float *kbar, const clis_head_cert_t *certs,
                                                  const uint8_t *tile_certs, const float *mu, float scale_log2,
                                                  int64_t key_offset, int first, clis_variant_t variant,
                                                  clis_stream_t stream);

/* After the last chunk: o = o_acc / l_acc (bf16, strides shape->o_*) and, if
 * lse2 is not NULL, lse2 = m_acc + log2(l_acc). */
CLIS_API clis_status_t clis_attn_chunk_finalize(const clis_shape_t *shape, const float *o_acc,
                                       const float *l_acc, const float *m_acc, void *o,
                                       float *lse2, clis_stream_t stream);

/* Workspace bytes for clis_attn_bwd: one fp32 per query row (B*H*Nq, the
 * row dots D_i), rounded up to 256.  CLIS_ERR_INVALID_ARG for a NULL or
 * invalid shape. */
CLIS_API clis_status_t clis_attn_bwd_workspace_size(const clis_shape_t *shape, size_t *bytes);

/* Attention backward: dQ, dK, dV of L = sum(dout * O) for O = softmax(scale *
 * Q K^T) V, scale = scale_log2 * ln 2.  The paper's causal LLM training
 * results (Table 3) run a backward pass but the paper gives none; this is the
 * plain chain rule through softmax, driven by the forward's row statistic:
 *   P_ij = exp2(scale_log2 * s_ij - lse2_i),  D_i = dout_i . o_i,
 *   dS_ij = P_ij (dout_i . v_j - D_i),
 *   dV_j = sum_i P_ij dout_i,  dK_j = scale sum_i dS_ij q_i,  dQ_i = scale sum_j dS_ij k_j.
 * lse2 is fixed per row, whichever forward path produced it, so the
 * backward has no running maximum and no rescaling.
 *   q, k, v   the forward's inputs (device, shape->dtype)
 *   o         the forward's output and dout its gradient, both with strides
 *             shape->o_*
 *   lse2      device fp32 [B*H*Nq], from clis_attn_fwd (or
 *             clis_attn_chunk_finalize) with the same q, k, scale_log2, causal
 *   dq, dk, dv  device outputs, same dtype; dq has strides shape->q_*, dk
 *             shape->k_*, dv shape->v_*.  Every element is written once
 *             (deterministic: no atomics).
 *   workspace device buffer of at least clis_attn_bwd_workspace_size() bytes,
 *             16-byte aligned (CLIS_ERR_WORKSPACE otherwise)
 *   causal    0 or 1; 1 requires Nq == Nk
 * Nq == 0 writes dK = dV = 0.  Errors as clis_attn_fwd. */
CLIS_API clis_status_t clis_attn_bwd(const clis_shape_t *shape, const void *q, const void *k,
                                     const void *v, const void *o, const void *dout,
                                     const float *lse2, void *dq, void *dk, void *dv,
                                     float scale_log2, int causal, void *workspace,
                                     size_t ws_bytes, clis_stream_t stream);

/* Rotary positions with up to four axes (text: one; images and video: height
 * and width, or time, height and width) for q and k, before clis_certify and the
 * attention calls.  The paper rotates q and k of its video models before the
 * path it describes; here it is one launch over both tensors.  Pair p of a row
 * turns by the angle a = position[b, n, axis[p]] * inv_freq[p]:
 *   (y0, y1) = (x0 cos a - x1 sin a, x1 cos a + x0 sin a),
 * p < pairs; pairs are elements (p, p + pairs) of a row, or (2p, 2p + 1) when
 * interleaved; elements from 2 * pairs on are copied.  inverse = 1 turns back:
 * the gradient of the rotation.  Angles are exact to fp32 for positions of any
 * size and sign; products are rounded once, to the data type.
 *   B, Hq, Hk, N, d   q [B, Hq, N, d], k [B, Hk, N, d]; d 64 or 128; B * N up to 2^27
 *   pairs             a multiple of 8, 8 .. d / 2
 *   axes              1 .. 4
 *   q_s*, k_s*        strides of q and k (may be 0: broadcast); qo_s*, ko_s* of
 *                     the outputs, which must not alias
 *   p_sb, p_sn, p_sa  strides of positions (int32), any */
typedef struct {
    int64_t B, Hq, Hk, N, d;
    int64_t pairs, axes, interleaved, inverse;
    int64_t q_sb, q_sh, q_sn, k_sb, k_sh, k_sn;
    int64_t qo_sb, qo_sh, qo_sn, ko_sb, ko_sh, ko_sn;
    int64_t p_sb, p_sn, p_sa;
    int64_t dtype;
} clis_rope_t;

/*   q, k        device inputs (k may be NULL when Hk = 0)
 *   q_out, k_out  device outputs; the input itself with its own strides is
 *               allowed (in place), any other overlap is not
 *   positions   device int32
 *   inv_freq    device double [pairs], finite, radians per position
 *   axis        device int32 [pairs], 0 .. axes - 1 (another value turns nothing
 *               and sets CLIS_PAGED_INDEX_BIT in the device error word)
 * Empty tensors launch nothing.  Errors as for clis_attn_fwd. */
CLIS_API clis_status_t clis_rope(const clis_rope_t *desc, const void *q, const void *k, void *q_out, void *k_out,
                                 const int32_t *positions, const double *inv_freq, const int32_t *axis,
                                 clis_stream_t stream);

/* A paged key/value cache and a batch of sequences that use it.
 *
 * The cache is k_cache, v_cache [num_pages, Hkv, page_size, d] with strides kc_s*
 * and vc_s* (d contiguous; a [num_pages, page_size, Hkv, d] cache is the same
 * with other strides).  Key j of sequence s lies in page block_table[s * bt_ss +
 * j / page_size], row j % page_size.  New tokens of all sequences are packed:
 * those of sequence s are rows cu_q[s] .. cu_q[s + 1] - 1 of q [T, H, d].
 *   S          sequences, at most 16384
 *   T          rows of q, k, v, o (rows from cu_q[S] on belong to no sequence)
 *   H, Hkv     query and key/value heads, H a multiple of Hkv, H / Hkv <= 128
 *   d          64 or 128
 *   page_size  a power of two, 8 .. 65536
 *   width      block-table columns; width * page_size (keys of a sequence, at
 *              most) up to 2^26
 * Attention also wants S * Hkv * width * page_size up to 2^43 (16,384 sequences of
 * 2^26 keys and 8 heads) and Hkv * (S + 1 + T / t) below 10^9, with the 2 * (128 / (H /
 * Hkv)) tokens t of a work item.
 * Lengths, tables, slots and page numbers live on the device, so one captured
 * graph serves every step; what is out of range there is not followed: it sets
 * a bit in the device error word (CLIS_PAGED_*) and reads as zeros, is not
 * written, or is brought into range. */
typedef struct {
    int64_t S, T, H, Hkv, d;
    int64_t page_size, num_pages, width;
    int64_t q_st, q_sh, o_st, o_sh;
    int64_t kc_sp, kc_sh, kc_sn, vc_sp, vc_sh, vc_sn;
    int64_t bt_ss;
    int64_t dtype;
} clis_paged_t;

/* Bits of the device error word: a page number, slot or axis out of range; the
 * ring of free pages ran out (or its counters contradict its size); a length
 * out of range. */
#define CLIS_PAGED_INDEX_BIT (1u << 16)
#define CLIS_PAGED_POOL_BIT (1u << 17)
#define CLIS_PAGED_LENGTH_BIT (1u << 18)

/* Plan of a step from the lengths of its sequences, all on the device: pages
 * for the new tokens, block tables, slots and positions.
 *   S, T, width, bt_ss, page_size, num_pages  as in clis_paged_t (no other
 *                field is read)
 *   ctx_len      int32 [S]: tokens of each sequence that are in the cache
 *   new_len      int32 [S]: tokens that this step adds; negative: the sequence
 *                is finished and gives its pages back
 *   block_table  int32 in/out: its first ceil(ctx / page_size) columns of a row
 *                are read, the following ones that the step needs are written
 *   ring         int32 [ring_size] in/out: free pages, those from state_in[0] (head)
 *                up to state_in[1] (tail), both counted without end and taken
 *                modulo ring_size; ring_size >= num_pages holds every page.
 *                Pages are taken from the head on in the order of the sequences,
 *                pages given back are written from the tail on.
 *   state_in, state_out  int64 [2]: head and tail before and after; different
 *                memory
 *   cu_q         int32 out [S + 1]: prefix sums of the new tokens
 *   kv_len       int32 out [S]: ctx + new (0 for a finished sequence; ctx for one
 *                that cannot be served)
 *   slots        int64 out [T]: page * page_size + row of each new token in
 *                packed order; -1 for rows behind the last and of sequences that
 *                cannot be served
 *   positions    int32 out [T]: the token's place in its sequence (0 behind the last)
 * A sequence for which the ring has too few pages (CLIS_PAGED_POOL_BIT) or the batch
 * too few rows (CLIS_PAGED_LENGTH_BIT) stays as it was: it takes no page and none of
 * its new tokens gets a slot, nor do those of later sequences that need a page.  Their
 * rows of this step mean nothing; their tokens can be brought again in a later one.
 * A sequence whose tokens the block-table row cannot hold (ctx + new beyond width *
 * page_size, or ctx out of range: CLIS_PAGED_LENGTH_BIT) stays as it was too, and no
 * other sequence is concerned: cu_q counts its rows as given.
 * Outputs must not overlap each other or the inputs.  The same inputs give the
 * same outputs bit for bit.  One launch.  Errors: CLIS_ERR_INVALID_ARG (null
 * pointers, sizes, state_out == state_in), CLIS_ERR_UNSUPPORTED (S > 16384, T
 * beyond 2^30), CLIS_ERR_MISALIGNED. */
CLIS_API clis_status_t clis_paged_plan(const clis_paged_t *desc, const int32_t *ctx_len, const int32_t *new_len,
                                       int32_t *block_table, int32_t *ring, int64_t ring_size, const int64_t *state_in,
                                       int64_t *state_out, int32_t *cu_q, int32_t *kv_len, int64_t *slots,
                                       int32_t *positions, clis_stream_t stream);

/* The same where rows share pages, as clis_paged_reorder leaves them: rows r * beams .. r * beams
 * + beams - 1 of the table are the beams of request r.  A finished row gives back the pages that
 * no row of its request names any more that goes on or is finished before it; clis_paged_plan
 * (beams = 1) would give a shared page back once for each row.
 *   beams        rows of a request, or of several (a multiple of its beams will do): S is a
 *                multiple of it (CLIS_ERR_INVALID_ARG otherwise) */
CLIS_API clis_status_t clis_paged_plan_beams(const clis_paged_t *desc, int64_t beams, const int32_t *ctx_len,
                                             const int32_t *new_len, int32_t *block_table, int32_t *ring,
                                             int64_t ring_size, const int64_t *state_in, int64_t *state_out,
                                             int32_t *cu_q, int32_t *kv_len, int64_t *slots, int32_t *positions,
                                             clis_stream_t stream);

/* New keys and values into the cache, rotated on the way, and q rotated beside
 * them, in one launch.  T up to 2^27.
 *   rope       desc for the rotation: N = T, B = 1, Hq = H (0: no q), Hk = Hkv, d,
 *              strides of q, q_out, k and positions (ko_s* are ignored: k goes to
 *              the cache); dtype as in desc; inverse must be 0
 *   v_st, v_sh strides of v [T, Hkv, d]
 *   slots      device int64 [T]: row t goes to page slots[t] / page_size, row
 *              slots[t] % page_size; negative: nowhere (padding).  Slots >= 0
 *              must be distinct; for equal ones it is not specified which row's
 *              pieces stay.
 *   positions, inv_freq, axis  as for clis_rope; pairs = 0: no rotation, and the
 *              three may be NULL (then q must be NULL too)
 * q_out may be q (in place); the caches must not overlap q, k or v. */
CLIS_API clis_status_t clis_paged_append(const clis_paged_t *desc, const clis_rope_t *rope, const void *q, const void *k,
                                         const void *v, int64_t v_st, int64_t v_sh, void *q_out, void *k_cache,
                                         void *v_cache, const int64_t *slots, const int32_t *positions,
                                         const double *inv_freq, const int32_t *axis, clis_stream_t stream);

/* Workspace bytes of clis_attn_fwd_paged for this shape and max_q (on the
 * current device: it depends on the number of SMs). */
CLIS_API clis_status_t clis_attn_paged_workspace_size(const clis_paged_t *desc, int64_t max_q, size_t *bytes);

/* Attention of the new tokens of every sequence over its cached keys (the new
 * tokens' own among them: append first).  The n = cu_q[s + 1] - cu_q[s] new
 * tokens are the last of the kv_len[s] tokens:
 *   o_i = sum_j 2^(x_ij) v_j / sum_j 2^(x_ij),  x_ij = scale_log2 * q_i . k_j,
 * over the keys j < kv_len[s] of head h / (H / Hkv) and, if causal, j <= kv_len[s] - n
 * + i.  Any mix of single tokens, drafted tokens and long chunks is one call:
 * sequences of few rows (n * H / Hkv up to 16, or 32) run a kernel bound by the
 * cache's bytes, the others one bound by the tensor cores (which takes them all
 * where the batch is small).  The softmax is
 * online with a lazily raised shift, as CLIS_ONLINE_LAZY: a certificate would
 * have to read all keys first, which for a few query rows is the whole cost.
 * Scores, row sums and outputs are held in fp32; the weights 2^(x_ij - shift) are rounded
 * to the data type before they multiply v, as the dense calls do it: off by up to 2^-8
 * of each in bf16, 2^-11 in fp16 (there at least 2^-32 of the row's largest).
 *   q          device [T, H, d] (q_st, q_sh)
 *   k_cache, v_cache, block_table, cu_q (int32 [S + 1], from 0 on, not falling),
 *              kv_len (int32 [S]): see clis_paged_t
 *   o          device out [T, H, d] (o_st, o_sh; must not alias).  Rows that
 *              belong to no sequence are left as they are; a row that sees no
 *              key becomes 0 (lse2: -inf).
 *   lse2       optional device fp32 out [T * H], index t * H + h
 *   max_q      no sequence has more new tokens than this (T is always valid); a
 *              sequence that does may be left out, with CLIS_PAGED_LENGTH_BIT
 *   workspace  device scratch of clis_attn_paged_workspace_size() bytes, 256-byte
 *              aligned; contents need no initialisation; not shared by calls that
 *              may run at the same time
 * What pages hold behind the last key has no effect, whatever it is, nor have
 * non-finite keys or values on rows that do not see them.  Results do not
 * depend on timing: reruns agree bit for bit.  S = 0 or T = 0 launches nothing.
 * Errors as for clis_attn_fwd; CLIS_ERR_WORKSPACE. */
CLIS_API clis_status_t clis_attn_fwd_paged(const clis_paged_t *desc, const void *q, const void *k_cache,
                                           const void *v_cache, const int32_t *block_table, const int32_t *cu_q,
                                           const int32_t *kv_len, void *o, float *lse2, int64_t max_q, float scale_log2,
                                           int causal, void *workspace, size_t ws_bytes, clis_stream_t stream);

/* The same cache in 8 bits.  A row (one token and key/value head of K or of V) is d
 * codes of one byte and one fp32 scale; its values are code * scale.  The codes lie in
 * k_codes, v_codes [num_pages, Hkv, page_size, d] with the strides kc_s*, vc_s* of
 * clis_paged_t (here bytes, multiples of 16), the scales in k_scale, v_scale [num_pages,
 * Hkv, page_size] with strides of their own.  dtype is that of q, k, v and outputs.
 * Scales are zero or positive. */
typedef enum { CLIS_CODE_INT8 = 0, CLIS_CODE_E4M3 = 1 } clis_code_t;

typedef struct {
    int64_t code;                 /* clis_code_t */
    int64_t ks_sp, ks_sh, ks_sn;  /* strides of k_scale: page, head, row (any, >= 0) */
    int64_t vs_sp, vs_sh, vs_sn;
} clis_quant_t;

/* clis_paged_append into a cache of codes.  k is rotated in fp32 and not rounded
 * before it is quantised.  Each row's scale is its largest magnitude over 127 (int8) or
 * 448 (E4M3), and a value's code the nearest one to value / scale (ties to even), so a
 * value is off by at most half a step: scale / 2 in int8; in E4M3 2^-4 of the value, or
 * scale * 2^-10 below scale * 2^-6.  A row below 2^-100 becomes zeros; one that holds a value that
 * is not finite gets the scale NaN and reads back as NaN throughout.  Other arguments
 * and errors as for clis_paged_append; rows of scales must not overlap. */
CLIS_API clis_status_t clis_paged_append_q8(const clis_paged_t *desc, const clis_quant_t *quant, const clis_rope_t *rope,
                                            const void *q, const void *k, const void *v, int64_t v_st, int64_t v_sh,
                                            void *q_out, void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                                            const int64_t *slots, const int32_t *positions, const double *inv_freq,
                                            const int32_t *axis, clis_stream_t stream);

/* Cached keys and values as 16-bit rows again: rows cu[s] .. cu[s + 1] - 1 of k_out and
 * v_out are tokens start[s], start[s] + 1, ... of sequence s.
 *   desc        S, T (rows of the outputs), Hkv, d, page_size, num_pages, width, kc_s*,
 *               vc_s*, bt_ss, dtype; T up to 2^27
 *   quant       NULL: a cache of 16-bit values, which are copied (scales may be NULL);
 *               else codes: code * scale, rounded to fp32 and then to the data type
 *   cu          device int32 [S + 1], from 0 on, not falling
 *   start       device int32 [S], or NULL (0)
 *   k_out, v_out  device [T, Hkv, d], strides k_st, k_sh, v_st, v_sh; must not overlap
 *               the cache or each other
 * Rows that belong to no sequence are left as they are.  Tokens outside of a
 * block-table row (CLIS_PAGED_LENGTH_BIT) and those of pages out of range
 * (CLIS_PAGED_INDEX_BIT) read as zeros.  One launch.  Errors as for clis_attn_fwd. */
CLIS_API clis_status_t clis_paged_read(const clis_paged_t *desc, const clis_quant_t *quant, const void *k_cache,
                                       const void *v_cache, const float *k_scale, const float *v_scale,
                                       const int32_t *block_table, const int32_t *cu, const int32_t *start, void *k_out,
                                       int64_t k_st, int64_t k_sh, void *v_out, int64_t v_st, int64_t v_sh,
                                       clis_stream_t stream);

/* clis_attn_fwd_paged over a cache of codes: x_ij = scale_log2 * q_i . k_j and o_i with the
 * values code * scale.  Where max_q allows for no more than 64 query rows of a sequence
 * (max_q * H / Hkv; single and drafted tokens), or the tables can hold little enough to go
 * with them, one kernel (and a second one that joins what it split, unless the tables are
 * small) does it all, bound by the codes' bytes: codes are exact in its
 * products, the weights times V's scale are rounded to fp16 (off by up to 2^-11 of each, at
 * least 2^-32 of the row's largest), q is exact in fp16, and in bf16 where it is within 2^-32 of
 * its row's largest value.  Else that kernel serves single tokens, and the other sequences (all of them
 * where the tables can hold no more than 16 MB of codes) are unpacked to 16 bits first (K's
 * codes, exact, its scales applied to the scores; V's values, rounded as clis_paged_read does)
 * and run the chunk kernel of clis_attn_fwd_paged; the workspace then holds a 16-bit copy
 * of as many pages as the tables have places (S * width) or the cache has (one layer's), whichever
 * is less.
 * A NaN code of E4M3 stands for NaN.  Masked places, padding, reruns and errors as for
 * clis_attn_fwd_paged. */
CLIS_API clis_status_t clis_attn_paged_q8_workspace_size(const clis_paged_t *desc, const clis_quant_t *quant, int64_t max_q,
                                                         size_t *bytes);
CLIS_API clis_status_t clis_attn_fwd_paged_q8(const clis_paged_t *desc, const clis_quant_t *quant, const void *q,
                                              const void *k_codes, const void *v_codes, const float *k_scale,
                                              const float *v_scale, const int32_t *block_table, const int32_t *cu_q,
                                              const int32_t *kv_len, void *o, float *lse2, int64_t max_q,
                                              float scale_log2, int causal, void *workspace, size_t ws_bytes,
                                              clis_stream_t stream);

/* Selection of a beam search.  Of the W * V continuations (beam w, token v) of each
 * request the K best by
 *   scores[r, w] + logits[r, w, v] - log sum_u e^(logits[r, w, u]),
 * best first, ties to the lowest w * V + v.  A continuation whose value is not finite is
 * none (a masked token, -inf; every token of a beam whose score is -inf, or whose logits
 * hold a NaN or +inf); where fewer than K are left, the places behind get the score
 * -inf, parent -1 and token -1.
 *   R, W, V, K   R * W up to 65535, W and K up to 64, W * V up to 2^31 - 1
 *   dtype        0 bf16, 1 fp16 (clis_dtype_t), 2 fp32
 *   l_sr, l_sw   strides of the logits in elements, any >= 0 (rows need no alignment
 *                beyond their type's)
 *   logits       device [R, W, V], tokens contiguous
 *   scores       device fp32 [R, W]
 *   out_scores, parent, token  device fp32, int32, int32 [R, K]
 *   workspace    device scratch of clis_beam_workspace_size() bytes (on the current
 *                device), 256-byte aligned; not shared by calls that may run at the same time
 * Values are compared to 48 bits, with logarithms off by at most 4e-6 (up to 2^18 tokens; measured
 * 3e-7).  So the order is that of the logits within a beam (those that differ by less than the 48
 * bits tie), and between beams that of values further apart than the logarithms' errors; beams of
 * equal logits have equal logarithms.  Reruns agree bit for bit.  Errors as for clis_attn_fwd; CLIS_ERR_WORKSPACE. */
typedef struct {
    int64_t R, W, V, K;
    int64_t dtype;
    int64_t l_sr, l_sw;
} clis_beam_t;

CLIS_API clis_status_t clis_beam_workspace_size(const clis_beam_t *desc, size_t *bytes);
CLIS_API clis_status_t clis_beam_select(const clis_beam_t *desc, const void *logits, const float *scores,
                                        float *out_scores, int32_t *parent, int32_t *token, void *workspace,
                                        size_t ws_bytes, clis_stream_t stream);

/* The beams' block tables after a selection: row g * W + w (beam w of request g) goes on
 * from row g * W + parent[g, w]; a negative parent ends the row.  Rows share pages: the
 * new row names the pages of the one it goes on from, except that where a partly filled last
 * page is gone on from more than once, all but the first (lowest w) get a page of
 * the ring with a copy of its rows.  Pages that no row of the request names any more go
 * back to the ring.  So the last page of a row is never shared unless it is full, and
 * clis_paged_plan and clis_paged_append go on as ever; a beam's row that shares pages is ended
 * here, or by a negative new_len of clis_paged_plan_beams (not of clis_paged_plan, which does not
 * know that other rows name its pages).
 *   groups, beams  requests and W (up to 64); groups * beams up to 16384
 *   width, page_size, num_pages  as in clis_paged_t
 *   bt_ss, bo_ss   strides of rows of block_table and new_table
 *   lens         device int32 [groups * beams]: tokens of each row
 *   parent       device int32 [groups, beams], below beams
 *   block_table, new_table  device int32 [groups * beams, width]; new_table may be
 *                block_table itself (same stride), no other overlap.  Columns
 *                behind a row's pages become -1.
 *   ring, ring_size, state_in, state_out  as for clis_paged_plan: pages are taken from the
 *                head on in the order of requests and beams, pages that go back
 *                follow the tail in the order of requests, columns and beams
 *   lens_out     device int32 [groups * beams]: tokens of the new rows; not lens or parent itself
 *   done         device int32 [groups]: 0 for a request that stays as it was (whole rows of its
 *                table, and its lens): the ring has too few pages for it and those before
 *                (CLIS_PAGED_POOL_BIT), a parent is out of range (CLIS_PAGED_INDEX_BIT) or a
 *                length (CLIS_PAGED_LENGTH_BIT)
 *   tensors, n   host array of the caches (values, codes, scales of K and V; up to 8) whose
 *                rows are copied
 *   workspace    device scratch of clis_paged_reorder_workspace_size() bytes, 256-byte
 *                aligned; not shared by calls that may run at the same time
 * Pages may be shared only within a request and in the same column, as this call makes
 * them.  Two launches; reruns agree bit for bit.  Errors as for clis_paged_plan;
 * CLIS_ERR_WORKSPACE. */
typedef struct {
    int64_t groups, beams, width, page_size, num_pages;
    int64_t bt_ss, bo_ss;
} clis_reorder_t;

/* One tensor of a cache, all layers: row r of page p, head h, layer l lies at base + l * sl + p *
 * sp + h * sh + r * sn (bytes) and has row_bytes bytes; all multiples of 4. */
typedef struct {
    void *base;
    int64_t layers, heads, row_bytes;
    int64_t sl, sp, sh, sn;
} clis_pages_t;

CLIS_API clis_status_t clis_paged_reorder_workspace_size(const clis_reorder_t *desc, size_t *bytes);
CLIS_API clis_status_t clis_paged_reorder(const clis_reorder_t *desc, const int32_t *lens, const int32_t *parent,
                                          const int32_t *block_table, int32_t *new_table, int32_t *ring,
                                          int64_t ring_size, const int64_t *state_in, int64_t *state_out,
                                          int32_t *lens_out, int32_t *done, const clis_pages_t *tensors, int64_t n,
                                          void *workspace, size_t ws_bytes, clis_stream_t stream);

/* Static description of a status code (never NULL). */
CLIS_API const char *clis_status_string(clis_status_t status);

/* Reads the device error word of the current device (synchronises the
 * device).  *code = 0 when no kernel recorded a fault; otherwise bit flags of
 * the pipeline waits that timed out and CLIS_PAGED_* bits.  Returns
 * CLIS_ERR_DATA if *code holds CLIS_PAGED_* bits alone, CLIS_ERR_TIMEOUT if it
 * holds others, CLIS_ERR_CUDA if the read failed. */
CLIS_API clis_status_t clis_get_device_error(uint32_t *code);

/* Resets the device error word of the current device to 0 (synchronous). */
CLIS_API clis_status_t clis_clear_device_error(void);

/* Self-test of the kernels' bounded waits (no counterpart in the paper).
 * Launches one small kernel whose single wait is on a barrier that nothing
 * ever arrives on, with a limit of limit_us microseconds (1..1,000,000): the
 * wait gives up, records CLIS_WAIT_SELFTEST_BIT in the device error word and
 * the kernel returns, leaving the context usable.  Read the word with
 * clis_get_device_error() and reset it with clis_clear_device_error(). */
#define CLIS_WAIT_SELFTEST_BIT (1u << 8)
CLIS_API clis_status_t clis_debug_wait_selftest(uint32_t limit_us, clis_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CLIS_H */
