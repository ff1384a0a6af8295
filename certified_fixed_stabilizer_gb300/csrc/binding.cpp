// binding.cpp -- torch tensors into the calls around a paged key/value cache
// and beam search over it (include/clis.h): argument checks, output allocation, the current stream, one
// call of the library each, and the rotation's autograd node.
//
// These calls are made once or more per layer and token, and at a few tokens the
// kernels take a few microseconds: marshalled in Python a call took 25 to 36 us of
// host time, here 4 to 9.  Everything that computes is in libclis.so.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/clis.h"

namespace {

using at::Tensor;

PyObject *g_error_class = nullptr;  // clis.ClisError(function, status)

struct StatusError : std::runtime_error {
    const char *fn;
    int status;
    StatusError(const char *f, int s)
        : std::runtime_error(std::string(f) + " failed: " + clis_status_string(static_cast<clis_status_t>(s))), fn(f),
          status(s)
    {
    }
};

void ok(const char *fn, clis_status_t st)
{
    if (st != CLIS_OK) throw StatusError(fn, st);
}

// The tensor's device made current for the call, and the stream: the given one or
// the device's current one.  What a call with a given stream allocates belongs to
// that stream: a block of the current stream's may still be in use there by work
// that was queued before its last tensor was dropped.
struct Place {
    c10::cuda::CUDAGuard guard;
    c10::cuda::CUDAStream current;
    c10::cuda::OptionalCUDAStreamGuard given;
    clis_stream_t stream;
    Place(const Tensor &t, std::optional<uintptr_t> raw)
        : guard(t.device()), current(c10::cuda::getCurrentCUDAStream(t.device().index())),
          stream(reinterpret_cast<clis_stream_t>(raw ? *raw : reinterpret_cast<uintptr_t>(current.stream())))
    {
        if (raw && reinterpret_cast<cudaStream_t>(*raw) != current.stream())
            given.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*raw), t.device().index()));
    }
    // A result, which the caller may read on the current stream and drop.
    Tensor result(Tensor t) const
    {
        if (given.current_stream()) t.record_stream(current);
        return t;
    }
};

bool elem(const Tensor &t) { return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf; }
int64_t dtype_of(const Tensor &t) { return t.scalar_type() == at::kHalf ? CLIS_DT_FP16 : CLIS_DT_BF16; }

void check_ints(const Tensor &t, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev, const char *name)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.device() == dev && t.is_contiguous(), name,
                      " must be a contiguous ", type, " tensor ", shape, " on the same device");
}

void check_table(const Tensor &positions, const Tensor &inv_freq, const Tensor &axis, const at::Device &dev)
{
    TORCH_CHECK_VALUE(positions.scalar_type() == at::kInt, "positions must be int32");
    TORCH_CHECK_VALUE(inv_freq.scalar_type() == at::kDouble && inv_freq.dim() == 1 && inv_freq.is_contiguous(),
                      "inv_freq must be a contiguous float64 tensor [pairs]");
    TORCH_CHECK_VALUE(axis.scalar_type() == at::kInt && axis.sizes() == inv_freq.sizes() && axis.is_contiguous(),
                      "axis must be a contiguous int32 tensor [pairs]");
    TORCH_CHECK_VALUE(positions.device() == dev && inv_freq.device() == dev && axis.device() == dev,
                      "positions, inv_freq and axis must be on the device of q");
}

void check_like(const Tensor &t, const Tensor &like, const char *name)
{
    TORCH_CHECK_VALUE(t.sizes() == like.sizes() && t.scalar_type() == like.scalar_type() && t.device() == like.device() &&
                          t.stride(-1) == 1,
                      name, " must have its input's shape, dtype and device and a contiguous last dimension");
}

// Stride of a dimension; one of size 1 is never stepped over, and torch leaves
// anything in its stride: it gets the row length, which passes every check.
int64_t st(const Tensor &t, int64_t i) { return t.size(i) == 1 ? t.size(t.dim() - 1) : t.stride(i); }

// New tensors straight from the CUDA allocator (the dispatcher on the way to it costs
// as much again).
Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Device &dev)
{
    return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}

Tensor empty_as(const Tensor &t) { return empty(t.sizes(), t.scalar_type(), t.device()); }

// -------------------------------------------------------------------- rotary

struct Rotated {
    Tensor q, k;  // k undefined without k
};

Rotated rope(const Tensor &q, const std::optional<Tensor> &k, const Tensor &positions, const Tensor &inv_freq,
             const Tensor &axis, bool interleaved, bool inverse, std::optional<Tensor> q_out, std::optional<Tensor> k_out,
             std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(q.is_cuda() && q.dim() == 4 && elem(q) && q.stride(3) == 1,
                      "q must be a bfloat16 or float16 device tensor [B, H, N, d] with a contiguous last dimension");
    const int64_t B = q.size(0), N = q.size(2);
    const bool shared = positions.dim() == 2;
    TORCH_CHECK_VALUE((shared || positions.dim() == 3) && positions.size(-2) == N &&
                          (shared || positions.size(0) == 1 || positions.size(0) == B),
                      "positions must be [B, N, axes] or [N, axes]");
    check_table(positions, inv_freq, axis, q.device());
    if (k)
        TORCH_CHECK_VALUE(k->dim() == 4 && k->scalar_type() == q.scalar_type() && k->device() == q.device() &&
                              k->stride(3) == 1 && k->size(0) == B && k->size(2) == N && k->size(3) == q.size(3),
                          "k must match q in all but its number of heads");
    Place at_(q, raw);
    Rotated r;
    r.q = q_out ? *q_out : at_.result(empty_as(q));
    if (q_out) check_like(r.q, q, "q_out");
    if (k) {
        r.k = k_out ? *k_out : at_.result(empty_as(*k));
        if (k_out) check_like(r.k, *k, "k_out");
    }
    clis_rope_t d = {};
    d.B = B;
    d.Hq = q.size(1);
    d.Hk = k ? k->size(1) : 0;
    d.N = N;
    d.d = q.size(3);
    d.pairs = inv_freq.numel();
    d.axes = positions.size(-1);
    d.interleaved = interleaved;
    d.inverse = inverse;
    d.q_sb = st(q, 0), d.q_sh = st(q, 1), d.q_sn = st(q, 2);
    d.qo_sb = st(r.q, 0), d.qo_sh = st(r.q, 1), d.qo_sn = st(r.q, 2);
    if (k) {
        d.k_sb = st(*k, 0), d.k_sh = st(*k, 1), d.k_sn = st(*k, 2);
        d.ko_sb = st(r.k, 0), d.ko_sh = st(r.k, 1), d.ko_sn = st(r.k, 2);
    }
    d.p_sb = shared || positions.size(0) == 1 ? 0 : positions.stride(0);
    d.p_sn = positions.stride(-2), d.p_sa = positions.stride(-1);
    d.dtype = dtype_of(q);
    ok("clis_rope", clis_rope(&d, q.data_ptr(), k ? k->data_ptr() : nullptr, r.q.data_ptr(), k ? r.k.data_ptr() : nullptr,
                              static_cast<const int32_t *>(positions.data_ptr()),
                              static_cast<const double *>(inv_freq.data_ptr()),
                              static_cast<const int32_t *>(axis.data_ptr()), at_.stream));
    return r;
}

// The rotation as an autograd node: its gradient is the rotation back, itself
// differentiable.  The angles carry no gradient; an inv_freq that wants one is refused.
struct RopeNode : torch::autograd::Function<RopeNode> {
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext *ctx, const Tensor &q,
                                                  const std::optional<Tensor> &k, const Tensor &positions,
                                                  const Tensor &inv_freq, const Tensor &axis, bool interleaved,
                                                  bool inverse)
    {
        ctx->save_for_backward({positions, inv_freq, axis});
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["inverse"] = inverse;
        ctx->set_materialize_grads(false);
        Rotated r = rope(q, k, positions, inv_freq, axis, interleaved, inverse, std::nullopt, std::nullopt, std::nullopt);
        if (!k) return {r.q};
        return {r.q, r.k};
    }

    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx,
                                                   torch::autograd::variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const bool interleaved = ctx->saved_data["interleaved"].toBool(), inverse = ctx->saved_data["inverse"].toBool();
        torch::autograd::variable_list out(7);
        std::vector<std::pair<int, Tensor>> need;
        for (size_t i = 0; i < grads.size(); i++) {
            if (!grads[i].defined() || !ctx->needs_input_grad(i)) continue;
            // Gradients come in any layout: expanded, or a contiguous piece at an odd offset.
            Tensor g = grads[i].contiguous();
            if (reinterpret_cast<uintptr_t>(g.data_ptr()) & 15) g = g.clone();
            need.emplace_back(static_cast<int>(i), g);
        }
        if (need.empty()) return out;
        const std::optional<Tensor> second = need.size() > 1 ? std::optional<Tensor>(need[1].second) : std::nullopt;
        if (at::GradMode::is_enabled()) {
            auto back = RopeNode::apply(need[0].second, second, saved[0], saved[1], saved[2], interleaved, !inverse);
            for (size_t i = 0; i < need.size(); i++) out[need[i].first] = back[i];
        } else {
            Rotated r = rope(need[0].second, second, saved[0], saved[1], saved[2], interleaved, !inverse, std::nullopt,
                             std::nullopt, std::nullopt);
            out[need[0].first] = r.q;
            if (second) out[need[1].first] = r.k;
        }
        return out;
    }
};

// ---------------------------------------------------------------------- plan

std::vector<Tensor> plan(const Tensor &ctx_len, const Tensor &new_len, const Tensor &table, const Tensor &ring,
                         const Tensor &ring_state, int64_t page_size, int64_t T, std::optional<int64_t> num_pages,
                         int64_t beams, std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(ctx_len.is_cuda() && ctx_len.dim() == 1, "ctx_len must be an int32 device tensor [S]");
    const at::Device dev = ctx_len.device();
    const int64_t S = ctx_len.size(0);
    check_ints(ctx_len, at::kInt, ctx_len.sizes(), dev, "ctx_len");
    check_ints(new_len, at::kInt, ctx_len.sizes(), dev, "new_len");
    check_ints(ring_state, at::kLong, {2}, dev, "ring_state");
    TORCH_CHECK_VALUE(ring.dim() == 1, "ring must be an int32 tensor [ring size]");
    check_ints(ring, at::kInt, ring.sizes(), dev, "ring");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.device() == dev && table.size(0) == S &&
                          table.stride(1) == 1,
                      "block_table must be an int32 tensor [S, width] with contiguous rows on the same device");
    TORCH_CHECK_VALUE(T >= 0, "num_tokens must not be negative");
    TORCH_CHECK_VALUE(beams > 0 && S % beams == 0, "the sequences must be requests of `beams` rows each");
    Place at_(ctx_len, raw);
    Tensor cu = empty({S + 1}, at::kInt, dev), kv = empty({S}, at::kInt, dev), slots = empty({T}, at::kLong, dev),
           pos = empty({T}, at::kInt, dev), state = empty({2}, at::kLong, dev);
    clis_paged_t d = {};
    d.S = S;
    d.T = T;
    d.page_size = page_size;
    d.num_pages = num_pages ? *num_pages : ring.size(0);
    d.width = table.size(1);
    d.bt_ss = S > 1 ? table.stride(0) : table.size(1);
    auto i32 = [](const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); };
    auto i64 = [](const Tensor &t) { return static_cast<int64_t *>(t.data_ptr()); };
    ok(beams == 1 ? "clis_paged_plan" : "clis_paged_plan_beams",
       clis_paged_plan_beams(&d, beams, i32(ctx_len), i32(new_len), i32(table), i32(ring), ring.size(0), i64(ring_state),
                             i64(state), i32(cu), i32(kv), i64(slots), i32(pos), at_.stream));
    return {at_.result(cu), at_.result(kv), at_.result(slots), at_.result(pos), at_.result(state)};
}

// --------------------------------------------------------- cache and attention

bool is_codes(const Tensor &t) { return t.scalar_type() == at::kChar || t.scalar_type() == at::kFloat8_e4m3fn; }

// The caches' part of the descriptor.
clis_paged_t cache_desc(const Tensor &kc, const Tensor &vc)
{
    TORCH_CHECK_VALUE(kc.dim() == 4 && kc.sizes() == vc.sizes() && kc.scalar_type() == vc.scalar_type() &&
                          kc.device() == vc.device(),
                      "k_cache and v_cache must be [pages, H_kv, page_size, d], of one dtype and on one device");
    TORCH_CHECK_VALUE(kc.stride(3) == 1 && vc.stride(3) == 1, "the caches must have a contiguous last dimension");
    clis_paged_t d = {};
    d.d = kc.size(3);
    d.Hkv = kc.size(1);
    d.page_size = kc.size(2);
    d.num_pages = kc.size(0);
    d.width = 1;
    d.kc_sp = st(kc, 0), d.kc_sh = st(kc, 1), d.kc_sn = st(kc, 2);
    d.vc_sp = st(vc, 0), d.vc_sh = st(vc, 1), d.vc_sn = st(vc, 2);
    return d;
}

// The caches beside q, k or v; with scales they hold codes.
clis_paged_t cache_desc(const Tensor &kc, const Tensor &vc, const Tensor &like, bool codes)
{
    TORCH_CHECK_VALUE(kc.dim() == 4 && kc.sizes() == vc.sizes() && kc.size(3) == like.size(2),
                      "k_cache and v_cache must be [pages, H_kv, page_size, d]");
    if (codes) {
        TORCH_CHECK_VALUE(is_codes(kc) && kc.scalar_type() == vc.scalar_type(),
                          "caches with scales must be int8 or float8_e4m3fn");
    } else {
        TORCH_CHECK_VALUE(kc.scalar_type() == like.scalar_type() && vc.scalar_type() == like.scalar_type(),
                          "the caches must have the dtype of q, k and v", is_codes(kc) ? " (codes need k_scale and v_scale)" : "");
    }
    TORCH_CHECK_VALUE(kc.device() == like.device() && vc.device() == like.device(),
                      "the caches must be on the device of q, k and v");
    clis_paged_t d = cache_desc(kc, vc);
    d.T = like.size(0);
    d.dtype = dtype_of(like);
    return d;
}

// The scales of a cache of codes.
clis_quant_t quant_desc(const Tensor &kc, const std::optional<Tensor> &ks, const std::optional<Tensor> &vs)
{
    clis_quant_t z = {};
    TORCH_CHECK_VALUE(ks.has_value() == vs.has_value(), "k_scale and v_scale belong together");
    if (!ks) return z;
    for (const Tensor *t : {&*ks, &*vs})
        TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->device() == kc.device() && t->sizes() == kc.sizes().slice(0, 3),
                          "k_scale and v_scale must be float32 [pages, H_kv, page_size] on the caches' device");
    z.code = kc.scalar_type() == at::kChar ? CLIS_CODE_INT8 : CLIS_CODE_E4M3;
    auto step = [](const Tensor &t, int64_t i) { return t.size(i) == 1 ? 1 : t.stride(i); };
    z.ks_sp = step(*ks, 0), z.ks_sh = step(*ks, 1), z.ks_sn = step(*ks, 2);
    z.vs_sp = step(*vs, 0), z.vs_sh = step(*vs, 1), z.vs_sn = step(*vs, 2);
    return z;
}

float *floats(const std::optional<Tensor> &t) { return t ? static_cast<float *>(t->data_ptr()) : nullptr; }

std::optional<Tensor> append(const Tensor &k, const Tensor &v, const Tensor &kc, const Tensor &vc, const Tensor &slots,
                             const std::optional<Tensor> &q, const std::optional<Tensor> &positions,
                             const std::optional<Tensor> &inv_freq, const std::optional<Tensor> &axis, bool interleaved,
                             std::optional<Tensor> q_out, const std::optional<Tensor> &ks, const std::optional<Tensor> &vs,
                             std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(k.is_cuda() && k.dim() == 3 && elem(k) && k.stride(2) == 1,
                      "k must be a bfloat16 or float16 device tensor [T, H_kv, d] with a contiguous last dimension");
    const int64_t T = k.size(0), Hk = k.size(1), d = k.size(2);
    TORCH_CHECK_VALUE(v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && v.device() == k.device() &&
                          v.stride(2) == 1,
                      "v must match k");
    clis_paged_t desc = cache_desc(kc, vc, k, ks.has_value());
    const clis_quant_t z = quant_desc(kc, ks, vs);
    TORCH_CHECK_VALUE(desc.Hkv == Hk, "the caches must have k's number of heads");
    check_ints(slots, at::kLong, {T}, k.device(), "slots");
    Place at_(k, raw);
    desc.H = Hk;
    clis_rope_t r = {};
    r.B = 1;
    r.Hk = Hk;
    r.N = T;
    r.d = d;
    r.dtype = desc.dtype;
    r.k_sh = st(k, 1), r.k_sn = st(k, 0);
    if (q) {
        TORCH_CHECK_VALUE(positions.has_value(), "q is rotated: positions are needed");
        TORCH_CHECK_VALUE(q->dim() == 3 && q->size(0) == T && q->size(2) == d && q->scalar_type() == k.scalar_type() &&
                              q->device() == k.device() && q->stride(2) == 1,
                          "q must match k in all but its number of heads");
        desc.H = r.Hq = q->size(1);
        if (q_out) check_like(*q_out, *q, "q_out");
        else q_out = at_.result(empty_as(*q));
        r.q_sh = st(*q, 1), r.q_sn = st(*q, 0);
        r.qo_sh = st(*q_out, 1), r.qo_sn = st(*q_out, 0);
    }
    if (positions) {
        TORCH_CHECK_VALUE((positions->dim() == 1 || positions->dim() == 2) && positions->size(0) == T,
                          "positions must be [T, axes] or [T]");
        TORCH_CHECK_VALUE(inv_freq && axis, "positions need inv_freq and axis");
        check_table(*positions, *inv_freq, *axis, k.device());
        r.pairs = inv_freq->numel();
        TORCH_CHECK_VALUE(r.pairs > 0, "inv_freq is empty");
        r.axes = positions->dim() == 2 ? positions->size(1) : 1;
        r.interleaved = interleaved;
        r.p_sn = positions->stride(0);
        r.p_sa = positions->dim() == 2 ? positions->stride(1) : 0;
    }
    const void *qp = q ? q->data_ptr() : nullptr;
    void *qo = q ? q_out->data_ptr() : nullptr;
    const auto *sl = static_cast<const int64_t *>(slots.data_ptr());
    const auto *pos = positions ? static_cast<const int32_t *>(positions->data_ptr()) : nullptr;
    const auto *inv = positions ? static_cast<const double *>(inv_freq->data_ptr()) : nullptr;
    const auto *ax = positions ? static_cast<const int32_t *>(axis->data_ptr()) : nullptr;
    if (ks)
        ok("clis_paged_append_q8",
           clis_paged_append_q8(&desc, &z, &r, qp, k.data_ptr(), v.data_ptr(), st(v, 0), st(v, 1), qo, kc.data_ptr(), vc.data_ptr(),
                                floats(ks), floats(vs), sl, pos, inv, ax, at_.stream));
    else
        ok("clis_paged_append", clis_paged_append(&desc, &r, qp, k.data_ptr(), v.data_ptr(), st(v, 0), st(v, 1), qo, kc.data_ptr(),
                                                  vc.data_ptr(), sl, pos, inv, ax, at_.stream));
    return q ? q_out : std::nullopt;
}

// with_lse: lse2 is allocated if it is not given.
std::vector<Tensor> attention(const Tensor &q, const Tensor &kc, const Tensor &vc, const Tensor &table, const Tensor &cu,
                              const Tensor &kv, int64_t max_q, double scale_log2, bool causal, std::optional<Tensor> out,
                              std::optional<Tensor> lse2, bool with_lse, std::optional<Tensor> workspace,
                              const std::optional<Tensor> &ks, const std::optional<Tensor> &vs, std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(q.is_cuda() && q.dim() == 3 && elem(q) && q.stride(2) == 1,
                      "q must be a bfloat16 or float16 device tensor [T, H, d] with a contiguous last dimension");
    const at::Device dev = q.device();
    clis_paged_t d = cache_desc(kc, vc, q, ks.has_value());
    const clis_quant_t z = quant_desc(kc, ks, vs);
    d.H = q.size(1);
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.device() == dev && table.stride(1) == 1,
                      "block_table must be an int32 tensor [S, width] with contiguous rows on the device of q");
    d.S = table.size(0);
    d.width = table.size(1);
    d.bt_ss = d.S > 1 ? table.stride(0) : 0;
    check_ints(cu, at::kInt, {d.S + 1}, dev, "cu_q");
    check_ints(kv, at::kInt, {d.S}, dev, "kv_len");
    if (lse2) check_ints(*lse2, at::kFloat, {d.T, d.H}, dev, "lse2");
    Place at_(q, raw);
    if (out) check_like(*out, q, "out");
    else out = at_.result(empty_as(q));
    if (with_lse && !lse2) lse2 = at_.result(empty({d.T, d.H}, at::kFloat, dev));
    d.q_st = st(q, 0), d.q_sh = st(q, 1);
    d.o_st = st(*out, 0), d.o_sh = st(*out, 1);
    size_t need = 0;
    if (ks) ok("clis_attn_paged_q8_workspace_size", clis_attn_paged_q8_workspace_size(&d, &z, max_q, &need));
    else ok("clis_attn_paged_workspace_size", clis_attn_paged_workspace_size(&d, max_q, &need));
    if (!workspace) workspace = empty({static_cast<int64_t>(need)}, at::kByte, dev);
    TORCH_CHECK_VALUE(workspace->device() == dev && workspace->is_contiguous(),
                      "the workspace must be contiguous and on the device of q");
    const auto *tb = static_cast<const int32_t *>(table.data_ptr()), *cq = static_cast<const int32_t *>(cu.data_ptr()),
               *kl = static_cast<const int32_t *>(kv.data_ptr());
    if (ks)
        ok("clis_attn_fwd_paged_q8",
           clis_attn_fwd_paged_q8(&d, &z, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), floats(ks), floats(vs), tb, cq, kl,
                                  out->data_ptr(), floats(lse2), max_q, static_cast<float>(scale_log2), causal,
                                  workspace->data_ptr(), workspace->nbytes(), at_.stream));
    else
        ok("clis_attn_fwd_paged",
           clis_attn_fwd_paged(&d, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), tb, cq, kl, out->data_ptr(), floats(lse2), max_q,
                               static_cast<float>(scale_log2), causal, workspace->data_ptr(), workspace->nbytes(), at_.stream));
    return {*out, lse2 ? *lse2 : Tensor()};
}

// Cached tokens as rows [T, Hkv, d]; type: of the rows, that of the caches without scales.
std::vector<Tensor> read(const Tensor &kc, const Tensor &vc, const Tensor &table, const Tensor &cu, int64_t T,
                         const std::optional<Tensor> &start, const std::optional<Tensor> &ks, const std::optional<Tensor> &vs,
                         bool half, std::optional<Tensor> k_out, std::optional<Tensor> v_out, std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(kc.is_cuda(), "k_cache must be a device tensor [pages, H_kv, page_size, d]");
    const at::Device dev = kc.device();
    clis_paged_t d = cache_desc(kc, vc);
    const clis_quant_t z = quant_desc(kc, ks, vs);
    TORCH_CHECK_VALUE(ks ? is_codes(kc) : elem(kc), ks ? "caches with scales must be int8 or float8_e4m3fn"
                                                      : "caches without scales must be bfloat16 or float16");
    const at::ScalarType type = ks ? (half ? at::kHalf : at::kBFloat16) : kc.scalar_type();
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.device() == dev && table.stride(1) == 1,
                      "block_table must be an int32 tensor [S, width] with contiguous rows on the caches' device");
    TORCH_CHECK_VALUE(T >= 0, "num_tokens must not be negative");
    d.S = table.size(0);
    d.T = T;
    d.H = d.Hkv;
    d.width = table.size(1);
    d.bt_ss = d.S > 1 ? table.stride(0) : 0;
    d.dtype = type == at::kHalf ? CLIS_DT_FP16 : CLIS_DT_BF16;
    check_ints(cu, at::kInt, {d.S + 1}, dev, "cu");
    if (start) check_ints(*start, at::kInt, {d.S}, dev, "start");
    Place at_(kc, raw);
    for (auto *t : {&k_out, &v_out}) {
        if (!*t) *t = at_.result(empty({T, d.Hkv, d.d}, type, dev));
        const Tensor &x = **t;
        TORCH_CHECK_VALUE(x.dim() == 3 && x.size(0) == T && x.size(1) == d.Hkv && x.size(2) == d.d && x.scalar_type() == type &&
                              x.device() == dev && x.stride(2) == 1,
                          "k_out and v_out must be [num_tokens, H_kv, d] of the rows' dtype with a contiguous last dimension");
    }
    ok("clis_paged_read",
       clis_paged_read(&d, ks ? &z : nullptr, kc.data_ptr(), vc.data_ptr(), floats(ks), floats(vs),
                       static_cast<const int32_t *>(table.data_ptr()), static_cast<const int32_t *>(cu.data_ptr()),
                       start ? static_cast<const int32_t *>(start->data_ptr()) : nullptr, k_out->data_ptr(), st(*k_out, 0),
                       st(*k_out, 1), v_out->data_ptr(), st(*v_out, 0), st(*v_out, 1), at_.stream));
    return {*k_out, *v_out};
}

// --------------------------------------------------------------- beam search

std::vector<Tensor> beam(const Tensor &logits, const Tensor &scores, int64_t K, std::optional<Tensor> workspace,
                         std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(logits.is_cuda() && logits.dim() == 3 && (elem(logits) || logits.scalar_type() == at::kFloat) &&
                          (logits.size(2) < 2 || logits.stride(2) == 1),
                      "logits must be a bfloat16, float16 or float32 device tensor [R, W, V] with a contiguous last dimension");
    const at::Device dev = logits.device();
    const int64_t R = logits.size(0), W = logits.size(1);
    TORCH_CHECK_VALUE(R == 0 || (W > 0 && logits.size(2) > 0), "logits must have beams and tokens");
    check_ints(scores, at::kFloat, {R, W}, dev, "scores");
    TORCH_CHECK_VALUE(K > 0, "num must be positive");
    Place at_(logits, raw);
    Tensor best = at_.result(empty({R, K}, at::kFloat, dev)), parent = at_.result(empty({R, K}, at::kInt, dev)),
           token = at_.result(empty({R, K}, at::kInt, dev));
    if (R > 0) {
        clis_beam_t d = {};
        d.R = R, d.W = W, d.V = logits.size(2), d.K = K;
        d.dtype = logits.scalar_type() == at::kFloat ? 2 : dtype_of(logits);
        d.l_sr = R == 1 ? 0 : logits.stride(0), d.l_sw = W == 1 ? 0 : logits.stride(1);
        size_t need = 0;
        ok("clis_beam_workspace_size", clis_beam_workspace_size(&d, &need));
        if (!workspace) workspace = empty({static_cast<int64_t>(need)}, at::kByte, dev);
        TORCH_CHECK_VALUE(workspace->device() == dev && workspace->is_contiguous(),
                          "the workspace must be contiguous and on the device of the logits");
        ok("clis_beam_select",
           clis_beam_select(&d, logits.data_ptr(), static_cast<const float *>(scores.data_ptr()), static_cast<float *>(best.data_ptr()),
                            static_cast<int32_t *>(parent.data_ptr()), static_cast<int32_t *>(token.data_ptr()),
                            workspace->data_ptr(), workspace->nbytes(), at_.stream));
    }
    return {best, parent, token};
}

// A cache tensor [layers, pages, H_kv, page_size, d], or scales without the last
// dimension; both also without the first.
clis_pages_t pages_desc(const Tensor &t, int64_t tail, int64_t pages, int64_t page_size, const at::Device &dev)
{
    const int64_t n = t.dim(), first = n - 3 - tail;
    TORCH_CHECK_VALUE(t.device() == dev && (first == 0 || first == 1) && t.size(first) == pages && t.size(first + 2) == page_size &&
                          (tail == 0 || t.stride(n - 1) == 1),
                      "caches must be [layers, pages, H_kv, page_size, d] or [pages, H_kv, page_size, d], scales the same without "
                      "d, all of one size of pages on the device of the block table");
    const int64_t e = t.element_size();
    auto step = [&](int64_t i) { return (t.size(i) == 1 ? (tail ? t.size(n - 1) : 1) : t.stride(i)) * e; };
    clis_pages_t p = {};
    p.base = t.data_ptr();
    p.layers = first ? t.size(0) : 1;
    p.heads = t.size(first + 1);
    p.row_bytes = (tail ? t.size(n - 1) : 1) * e;
    p.sl = first ? step(0) : 0;
    p.sp = step(first), p.sh = step(first + 1), p.sn = step(first + 2);
    return p;
}

std::vector<Tensor> reorder(const Tensor &lens, const Tensor &parent, const Tensor &table, const Tensor &ring,
                            const Tensor &ring_state, const std::vector<Tensor> &caches, const std::vector<Tensor> &scales,
                            int64_t page_size, std::optional<Tensor> out, std::optional<Tensor> workspace,
                            std::optional<uintptr_t> raw)
{
    TORCH_CHECK_VALUE(parent.is_cuda() && parent.dim() == 2, "parent must be an int32 device tensor [requests, beams]");
    const at::Device dev = parent.device();
    const int64_t R = parent.size(0), W = parent.size(1), S = R * W;
    TORCH_CHECK_VALUE(W > 0, "parent must have beams");
    check_ints(parent, at::kInt, {R, W}, dev, "parent");
    check_ints(lens, at::kInt, {S}, dev, "lens");
    check_ints(ring_state, at::kLong, {2}, dev, "ring_state");
    TORCH_CHECK_VALUE(ring.dim() == 1, "ring must be an int32 tensor [ring size]");
    check_ints(ring, at::kInt, ring.sizes(), dev, "ring");
    for (const Tensor *t : {&table, out ? &*out : &table})
        TORCH_CHECK_VALUE(t->dim() == 2 && t->scalar_type() == at::kInt && t->device() == dev && t->size(0) == S &&
                              t->size(1) == table.size(1) && t->stride(1) == 1,
                          "block_table and out must be int32 [requests * beams, width] with contiguous rows on one device");
    clis_reorder_t d = {};
    d.groups = R, d.beams = W, d.width = table.size(1), d.num_pages = ring.size(0);
    std::vector<clis_pages_t> tensors;
    for (const auto *list : {&caches, &scales})
        for (const Tensor &t : *list) {
            const int64_t tail = list == &caches ? 1 : 0;
            TORCH_CHECK_VALUE(t.dim() == 3 + tail || t.dim() == 4 + tail, list == &caches ? "a cache must have 4 or 5 dimensions"
                                                                                         : "scales must have 3 or 4 dimensions");
            if (tensors.empty()) {
                d.num_pages = t.size(t.dim() - 3 - tail);
                page_size = t.size(t.dim() - 1 - tail);
            }
            tensors.push_back(pages_desc(t, tail, d.num_pages, page_size, dev));
        }
    d.page_size = page_size;
    d.bt_ss = S > 1 ? table.stride(0) : table.size(1);
    Place at_(parent, raw);
    if (!out) out = at_.result(empty(table.sizes(), at::kInt, dev));
    d.bo_ss = S > 1 ? out->stride(0) : out->size(1);
    Tensor lens_out = at_.result(empty({S}, at::kInt, dev)), state = at_.result(empty({2}, at::kLong, dev)),
           done = at_.result(empty({R}, at::kInt, dev));
    size_t need = 0;
    ok("clis_paged_reorder_workspace_size", clis_paged_reorder_workspace_size(&d, &need));
    if (!workspace) workspace = empty({static_cast<int64_t>(need)}, at::kByte, dev);
    TORCH_CHECK_VALUE(workspace->device() == dev && workspace->is_contiguous(),
                      "the workspace must be contiguous and on the device of parent");
    auto i32 = [](const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); };
    auto i64 = [](const Tensor &t) { return static_cast<int64_t *>(t.data_ptr()); };
    ok("clis_paged_reorder",
       clis_paged_reorder(&d, i32(lens), i32(parent), i32(table), i32(*out), i32(ring), ring.size(0), i64(ring_state), i64(state),
                          i32(lens_out), i32(done), tensors.data(), static_cast<int64_t>(tensors.size()), workspace->data_ptr(),
                          workspace->nbytes(), at_.stream));
    return {*out, lens_out, state, done};
}

// -------------------------------------------------------------- Python objects

Tensor tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

std::optional<Tensor> maybe(PyObject *o, const char *name)
{
    if (o == Py_None) return std::nullopt;
    return tensor(o, name);
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

std::optional<int64_t> maybe_int(PyObject *o)
{
    if (o == Py_None) return std::nullopt;
    return integer(o);
}

std::optional<uintptr_t> stream_of(PyObject *o)
{
    if (o == Py_None) return std::nullopt;
    return static_cast<uintptr_t>(integer(o));
}

PyObject *wrap(const std::vector<Tensor> &v)
{
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(v.size()));
    if (!t) throw python_error();
    for (size_t i = 0; i < v.size(); i++) {
        PyObject *o;
        if (v[i].defined()) {
            o = THPVariable_Wrap(v[i]);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        PyTuple_SET_ITEM(t, static_cast<Py_ssize_t>(i), o);
    }
    return t;
}

// A library status becomes clis.ClisError; C++ exceptions become Python's.
template <typename F>
PyObject *call(Py_ssize_t got, Py_ssize_t want, const F &f)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(got == want, "wrong number of arguments");
    try {
        return f();
    } catch (const StatusError &e) {
        if (g_error_class) {
            PyObject *x = PyObject_CallFunction(g_error_class, "si", e.fn, e.status);
            if (x) {
                PyErr_SetObject(g_error_class, x);
                Py_DECREF(x);
            }
        } else {
            PyErr_SetString(PyExc_RuntimeError, e.what());
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *py_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 10, [&] {
        const Rotated r = rope(tensor(a[0], "q"), maybe(a[1], "k"), tensor(a[2], "positions"), tensor(a[3], "inv_freq"),
                               tensor(a[4], "axis"), truth(a[5]), truth(a[6]), maybe(a[7], "q_out"), maybe(a[8], "k_out"),
                               stream_of(a[9]));
        return wrap({r.q, r.k});
    });
}

PyObject *py_rope_autograd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 6, [&] {
        const Tensor inv_freq = tensor(a[3], "inv_freq");
        TORCH_CHECK_VALUE(!(inv_freq.requires_grad() && at::GradMode::is_enabled()),
                          "inv_freq gets no gradient from the rotation: detach it");
        auto r = RopeNode::apply(tensor(a[0], "q"), maybe(a[1], "k"), tensor(a[2], "positions"), inv_freq,
                                 tensor(a[4], "axis"), truth(a[5]), false);
        return wrap({r[0], r.size() > 1 ? r[1] : Tensor()});
    });
}

PyObject *py_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 10, [&] {
        return wrap(plan(tensor(a[0], "ctx_len"), tensor(a[1], "new_len"), tensor(a[2], "block_table"), tensor(a[3], "ring"),
                         tensor(a[4], "ring_state"), integer(a[5]), integer(a[6]), maybe_int(a[7]), integer(a[8]), stream_of(a[9])));
    });
}

PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 14, [&]() -> PyObject * {
        const auto q = append(tensor(a[0], "k"), tensor(a[1], "v"), tensor(a[2], "k_cache"), tensor(a[3], "v_cache"),
                              tensor(a[4], "slots"), maybe(a[5], "q"), maybe(a[6], "positions"), maybe(a[7], "inv_freq"),
                              maybe(a[8], "axis"), truth(a[9]), maybe(a[10], "q_out"), maybe(a[11], "k_scale"),
                              maybe(a[12], "v_scale"), stream_of(a[13]));
        if (q) return THPVariable_Wrap(*q);
        Py_RETURN_NONE;
    });
}

PyObject *py_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 16, [&] {
        return wrap(attention(tensor(a[0], "q"), tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor(a[3], "block_table"),
                              tensor(a[4], "cu_q"), tensor(a[5], "kv_len"), integer(a[6]), real(a[7]), truth(a[8]),
                              maybe(a[9], "out"), maybe(a[10], "lse2"), truth(a[11]), maybe(a[12], "workspace"),
                              maybe(a[13], "k_scale"), maybe(a[14], "v_scale"), stream_of(a[15])));
    });
}

PyObject *py_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 12, [&] {
        return wrap(read(tensor(a[0], "k_cache"), tensor(a[1], "v_cache"), tensor(a[2], "block_table"), tensor(a[3], "cu"),
                         integer(a[4]), maybe(a[5], "start"), maybe(a[6], "k_scale"), maybe(a[7], "v_scale"), truth(a[8]),
                         maybe(a[9], "k_out"), maybe(a[10], "v_out"), stream_of(a[11])));
    });
}

std::vector<Tensor> tensors(PyObject *o, const char *name)
{
    std::vector<Tensor> v;
    PyObject *seq = PySequence_Fast(o, name);
    if (!seq) throw python_error();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    for (Py_ssize_t i = 0; i < n; i++) {
        PyObject *x = PySequence_Fast_GET_ITEM(seq, i);
        if (!THPVariable_Check(x)) {
            Py_DECREF(seq);
            TORCH_CHECK_TYPE(false, name, " must hold tensors");
        }
        v.push_back(THPVariable_Unpack(x));
    }
    Py_DECREF(seq);
    return v;
}

PyObject *py_beam(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 5, [&] {
        return wrap(beam(tensor(a[0], "logits"), tensor(a[1], "scores"), integer(a[2]), maybe(a[3], "workspace"), stream_of(a[4])));
    });
}

PyObject *py_reorder(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 11, [&] {
        return wrap(reorder(tensor(a[0], "lens"), tensor(a[1], "parent"), tensor(a[2], "block_table"), tensor(a[3], "ring"),
                            tensor(a[4], "ring_state"), tensors(a[5], "caches"), tensors(a[6], "scales"), integer(a[7]),
                            maybe(a[8], "out"), maybe(a[9], "workspace"), stream_of(a[10])));
    });
}

PyObject *py_set_error_class(PyObject *, PyObject *c)
{
    Py_INCREF(c);
    Py_XDECREF(g_error_class);
    g_error_class = c;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_rope)), METH_FASTCALL, nullptr},
    {"rope_autograd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_rope_autograd)), METH_FASTCALL, nullptr},
    {"paged_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_plan)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_append)), METH_FASTCALL, nullptr},
    {"attention_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_attention)), METH_FASTCALL, nullptr},
    {"paged_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_read)), METH_FASTCALL, nullptr},
    {"beam_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_beam)), METH_FASTCALL, nullptr},
    {"paged_reorder", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_reorder)), METH_FASTCALL, nullptr},
    {"set_error_class", py_set_error_class, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_clis_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__clis_torch() { return PyModule_Create(&g_module); }
