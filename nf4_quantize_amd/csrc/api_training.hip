// api_training.hip - the extern "C" entry points of the training-step operators
// (AdamW, the residual norms, the token embedding): host-side validation and
// dispatch. Declarations and contracts are in include/nf4.h.
//
// Every argument is checked before any HIP call; a rejected call launches
// nothing and returns its status. The library allocates nothing.
#include <math.h>

#include "training_internal.h"

#define NF4_API extern "C" __attribute__((visibility("default")))

using namespace nf4;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 37;
constexpr int64_t kMaxEntry = int64_t(1) << 33;  // keeps an entry's grid below 2^31 threads
constexpr int64_t kMaxDim = 32768;               // a row in a workgroup's registers
constexpr int64_t kMaxTokens = int64_t(1) << 28;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_dtype(int32_t d) { return d == NF4_F32 || d == NF4_BF16; }
nf4_status launch_status(hipError_t e) { return e == hipSuccess ? NF4_OK : NF4_ERR_LAUNCH; }
hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

// The list of an optimizer call: sizes, and the gradients' pointers.
nf4_status check_grads(const nf4_adamw_entry *e, int32_t count) {
    if (count < 0) return NF4_ERR_SIZE;
    if (count > 0 && !e) return NF4_ERR_NULL;
    for (int32_t i = 0; i < count; ++i) {
        if (e[i].n < 0 || e[i].n > kMaxEntry) return NF4_ERR_SIZE;
        if (e[i].n == 0) continue;
        if (!e[i].grad) return NF4_ERR_NULL;
        if (!aligned(e[i].grad, 16)) return NF4_ERR_ALIGN;
    }
    return NF4_OK;
}

nf4_status check_workspace(size_t need, const void *ws, size_t bytes) {
    if (need == 0) return NF4_OK;
    if (!ws || bytes < need) return NF4_ERR_WORKSPACE;
    return aligned(ws, 256) ? NF4_OK : NF4_ERR_ALIGN;
}

}  // namespace

NF4_API size_t nf4_grad_norm_workspace_size(const nf4_adamw_entry *entries, int32_t count) {
    if (count < 0 || (count > 0 && !entries)) return (size_t)-1;
    for (int32_t i = 0; i < count; ++i)
        if (entries[i].n < 0 || entries[i].n > kMaxEntry) return (size_t)-1;
    return grad_norm_workspace(entries, count);
}

NF4_API nf4_status nf4_grad_norm(const nf4_adamw_entry *entries, int32_t count, int32_t grad_dtype, float *norm,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    nf4_status st = check_grads(entries, count);
    if (st != NF4_OK) return st;
    if (!is_dtype(grad_dtype)) return NF4_ERR_UNSUPPORTED;
    if (!norm) return NF4_ERR_NULL;
    if (!aligned(norm, 4)) return NF4_ERR_ALIGN;
    if ((st = check_workspace(grad_norm_workspace(entries, count), workspace, workspace_bytes)) != NF4_OK) return st;
    return launch_status(launch_grad_norm(entries, count, static_cast<nf4_dtype>(grad_dtype), norm, workspace,
                                          stream_of(stream)));
}

NF4_API size_t nf4_adamw_workspace_size(int32_t count) { return count < 0 ? (size_t)-1 : adamw_workspace(count); }

namespace {

nf4_status adamw(const nf4_adamw_entry *entries, int32_t count, int32_t w_dtype, int32_t grad_dtype, int32_t moments,
                 const nf4_adamw_config *config, float *norm, bool own_norm, void *workspace, size_t workspace_bytes,
                 void *stream) {
    nf4_status st = check_grads(entries, count);
    if (st != NF4_OK) return st;
    if (!config) return NF4_ERR_NULL;
    if (!is_dtype(w_dtype) || !is_dtype(grad_dtype)) return NF4_ERR_UNSUPPORTED;
    if (moments != NF4_MOMENTS_8 && moments != NF4_MOMENTS_32) return NF4_ERR_UNSUPPORTED;
    const nf4_adamw_config &c = *config;
    if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0) || !(c.eps >= 0.0f) ||
        c.step < 1 || isnan(c.max_norm))
        return NF4_ERR_SIZE;
    if ((c.max_norm > 0.0f || own_norm) && !norm) return NF4_ERR_NULL;
    if (norm && !aligned(norm, 4)) return NF4_ERR_ALIGN;
    const bool eight = moments == NF4_MOMENTS_8;
    for (int32_t i = 0; i < count; ++i) {
        const nf4_adamw_entry &e = entries[i];
        if (e.n == 0) continue;
        if (!isfinite(e.lr) || !isfinite(e.weight_decay)) return NF4_ERR_SIZE;
        if (!e.w || !e.m || !e.v || (eight && (!e.m_scale || !e.v_scale))) return NF4_ERR_NULL;
        if (e.master && w_dtype != NF4_BF16) return NF4_ERR_UNSUPPORTED;
        if (!aligned(e.w, 16) || !aligned(e.m, 16) || !aligned(e.v, 16) || (e.master && !aligned(e.master, 16)))
            return NF4_ERR_ALIGN;
        if (eight && (!aligned(e.m_scale, 4) || !aligned(e.v_scale, 4))) return NF4_ERR_ALIGN;
    }
    size_t need = adamw_workspace(count);
    if (own_norm && grad_norm_workspace(entries, count) > need) need = grad_norm_workspace(entries, count);
    if ((st = check_workspace(need, workspace, workspace_bytes)) != NF4_OK) return st;
    return launch_status(launch_adamw(entries, count, static_cast<nf4_dtype>(w_dtype),
                                      static_cast<nf4_dtype>(grad_dtype), eight, c, norm, own_norm, workspace,
                                      stream_of(stream)));
}

}  // namespace

NF4_API nf4_status nf4_adamw_step(const nf4_adamw_entry *entries, int32_t count, int32_t w_dtype, int32_t grad_dtype,
                                  int32_t moments, const nf4_adamw_config *config, const float *grad_norm,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    return adamw(entries, count, w_dtype, grad_dtype, moments, config, const_cast<float *>(grad_norm), false, workspace,
                 workspace_bytes, stream);  // read only
}

NF4_API nf4_status nf4_adamw_clip_step(const nf4_adamw_entry *entries, int32_t count, int32_t w_dtype,
                                       int32_t grad_dtype, int32_t moments, const nf4_adamw_config *config,
                                       float *grad_norm, void *workspace, size_t workspace_bytes, void *stream) {
    return adamw(entries, count, w_dtype, grad_dtype, moments, config, grad_norm, true, workspace, workspace_bytes,
                 stream);
}

namespace {

nf4_status check_norm_shape(const nf4_residual_norm_shape *sh) {
    if (!sh) return NF4_ERR_NULL;
    if (sh->rows < 0 || sh->dim < 1 || sh->dim > kMaxDim || sh->rows > kMaxElems / sh->dim) return NF4_ERR_SIZE;
    if (!is_dtype(sh->dtype) || !is_dtype(sh->res_dtype) || !is_dtype(sh->w_dtype)) return NF4_ERR_UNSUPPORTED;
    if (sh->res_dtype != sh->dtype && sh->res_dtype != NF4_F32) return NF4_ERR_UNSUPPORTED;
    if (sh->gate_kind < NF4_GATE_NONE || sh->gate_kind > NF4_GATE_TOKEN) return NF4_ERR_UNSUPPORTED;
    if (!(sh->eps >= 0.0f) || !isfinite(sh->alpha) || !isfinite(sh->w_offset)) return NF4_ERR_SIZE;
    return NF4_OK;
}

}  // namespace

NF4_API nf4_status nf4_residual_norm_forward(const nf4_residual_norm_shape *shape, const void *y, const void *h,
                                             const void *w_post, const void *gate, const void *w_pre, void *h_out,
                                             void *x_out, float *rstd_post, float *rstd_pre, void *stream) {
    const nf4_status st = check_norm_shape(shape);
    if (st != NF4_OK) return st;
    if (shape->rows == 0) return NF4_OK;
    if (!h || !w_pre || !x_out || (y && !h_out)) return NF4_ERR_NULL;
    if (y && shape->gate_kind != NF4_GATE_NONE && !gate) return NF4_ERR_NULL;
    for (const void *p : {y, h, w_post, gate, w_pre, static_cast<const void *>(h_out), static_cast<const void *>(x_out)})
        if (!aligned(p, 16)) return NF4_ERR_ALIGN;
    if (!aligned(rstd_post, 4) || !aligned(rstd_pre, 4)) return NF4_ERR_ALIGN;
    ResidualNormIn in{};
    in.y = y, in.h = h, in.w_post = y ? w_post : nullptr, in.gate = gate, in.w_pre = w_pre;
    ResidualNormOut out{};
    out.h = h_out, out.x = x_out, out.rstd_post = rstd_post, out.rstd_pre = rstd_pre;
    return launch_status(launch_residual_norm_forward(*shape, in, out, stream_of(stream)));
}

NF4_API size_t nf4_residual_norm_backward_workspace_size(const nf4_residual_norm_shape *shape) {
    return check_norm_shape(shape) == NF4_OK ? residual_norm_workspace(*shape, true) : (size_t)-1;
}

NF4_API nf4_status nf4_residual_norm_backward(const nf4_residual_norm_shape *shape, const void *dx, const void *dh_out,
                                              const void *y, const void *h_out, const void *w_post, const void *gate,
                                              const void *w_pre, const float *rstd_post, const float *rstd_pre,
                                              void *dy, void *dh, void *dgate, void *dw_pre, void *dw_post,
                                              void *workspace, size_t workspace_bytes, void *stream) {
    nf4_status st = check_norm_shape(shape);
    if (st != NF4_OK) return st;
    const bool channel = shape->gate_kind == NF4_GATE_CHANNEL;
    const bool has_y = y || shape->rows == 0;  // no rows: nothing says whether there was a y
    const bool sums = dw_pre || (has_y && (dw_post || (channel && dgate)));
    if (shape->rows > 0) {
        if (!h_out || !w_pre || !rstd_pre) return NF4_ERR_NULL;
        if (y && shape->gate_kind != NF4_GATE_NONE && !gate) return NF4_ERR_NULL;
        if (y && w_post && !rstd_post) return NF4_ERR_NULL;
    }
    if (has_y && ((dw_post && !w_post) || (dgate && shape->gate_kind == NF4_GATE_NONE))) return NF4_ERR_NULL;
    for (const void *p : {dx, dh_out, y, h_out, w_post, gate, w_pre, static_cast<const void *>(dy),
                          static_cast<const void *>(dh), static_cast<const void *>(dgate),
                          static_cast<const void *>(dw_pre), static_cast<const void *>(dw_post)})
        if (!aligned(p, 16)) return NF4_ERR_ALIGN;
    if (!aligned(rstd_post, 4) || !aligned(rstd_pre, 4)) return NF4_ERR_ALIGN;
    if ((st = check_workspace(residual_norm_workspace(*shape, sums), workspace, workspace_bytes)) != NF4_OK) return st;
    if (shape->rows == 0 && !sums) return NF4_OK;
    ResidualNormIn in{};
    in.dx = dx, in.dh_out = dh_out, in.y = y, in.h = h_out, in.w_post = y ? w_post : nullptr, in.gate = gate;
    in.w_pre = w_pre, in.rstd_post = rstd_post, in.rstd_pre = rstd_pre;
    ResidualNormOut out{};
    out.dy = dy, out.dh = dh, out.dgate = has_y ? dgate : nullptr;
    out.dw_pre = dw_pre, out.dw_post = has_y ? dw_post : nullptr;
    return launch_status(launch_residual_norm_backward(*shape, in, out, workspace, stream_of(stream)));
}

namespace {

nf4_status check_tokens(int32_t id_dtype, int64_t tokens, int64_t vocab, int64_t dim) {
    if (id_dtype != NF4_I32 && id_dtype != NF4_I64) return NF4_ERR_UNSUPPORTED;
    if (tokens < 0 || tokens > kMaxTokens || vocab < 1 || vocab > kMaxTokens || dim < 1) return NF4_ERR_SIZE;
    if (dim > (int64_t(1) << 30) || vocab > kMaxElems / dim || tokens > kMaxElems / dim) return NF4_ERR_SIZE;
    return NF4_OK;
}

}  // namespace

NF4_API nf4_status nf4_embedding_forward(const void *ids, int32_t id_dtype, int64_t tokens, const void *table,
                                         int32_t dtype, int64_t vocab, int64_t dim, float scale, void *out,
                                         int32_t out_dtype, void *stream) {
    const nf4_status st = check_tokens(id_dtype, tokens, vocab, dim);
    if (st != NF4_OK) return st;
    if (!is_dtype(dtype) || !is_dtype(out_dtype)) return NF4_ERR_UNSUPPORTED;
    if (tokens == 0) return NF4_OK;
    if (!ids || !table || !out) return NF4_ERR_NULL;
    if (!aligned(ids, id_dtype == NF4_I64 ? 8 : 4) || !aligned(table, 16) || !aligned(out, 16)) return NF4_ERR_ALIGN;
    return launch_status(launch_embedding_forward(ids, id_dtype == NF4_I64, tokens, table,
                                                  static_cast<nf4_dtype>(dtype), vocab, dim, scale, out,
                                                  static_cast<nf4_dtype>(out_dtype), stream_of(stream)));
}

NF4_API nf4_status nf4_embedding_forward_packed(const void *ids, int32_t id_dtype, int64_t tokens,
                                                const nf4_weight *table, float scale, void *out, int32_t out_dtype,
                                                void *stream) {
    if (!table) return NF4_ERR_NULL;
    const nf4_status st = check_tokens(id_dtype, tokens, table->n_out, table->k_in);
    if (st != NF4_OK) return st;
    if (table->k_in % kBlock != 0) return NF4_ERR_SIZE;
    if (!is_dtype(out_dtype) || table->blocksize != kBlock) return NF4_ERR_UNSUPPORTED;
    const bool dq = table->absmax_q != nullptr || table->absmax_scale != nullptr;
    if (dq && table->dq_blocksize != kDqBlock) return NF4_ERR_UNSUPPORTED;
    if (tokens == 0) return NF4_OK;
    if (!ids || !out || !table->codes) return NF4_ERR_NULL;
    if (dq && (!table->absmax_q || !table->absmax_scale)) return NF4_ERR_NULL;
    if (!dq && !table->absmax) return NF4_ERR_NULL;
    if (!aligned(ids, id_dtype == NF4_I64 ? 8 : 4) || !aligned(table->codes, 16) || !aligned(out, 16))
        return NF4_ERR_ALIGN;
    if (!aligned(table->absmax, 4) || !aligned(table->absmax_q, 4) || !aligned(table->absmax_scale, 4))
        return NF4_ERR_ALIGN;
    nf4_weight w = *table;
    if (dq) w.absmax = nullptr;
    return launch_status(launch_embedding_packed(ids, id_dtype == NF4_I64, tokens, w, scale, out,
                                                 static_cast<nf4_dtype>(out_dtype), stream_of(stream)));
}

NF4_API size_t nf4_embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t dim) {
    if (check_tokens(NF4_I64, tokens, vocab, dim) != NF4_OK) return (size_t)-1;
    return embedding_backward_workspace(tokens, vocab, dim);
}

NF4_API nf4_status nf4_embedding_backward(const void *ids, int32_t id_dtype, int64_t tokens, const void *dy,
                                          int32_t dtype, int64_t vocab, int64_t dim, float scale, int64_t padding_id,
                                          void *grad, int32_t grad_dtype, int32_t accumulate, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    nf4_status st = check_tokens(id_dtype, tokens, vocab, dim);
    if (st != NF4_OK) return st;
    if (!is_dtype(dtype) || !is_dtype(grad_dtype)) return NF4_ERR_UNSUPPORTED;
    if (!grad || (tokens > 0 && (!ids || !dy))) return NF4_ERR_NULL;
    if (!aligned(ids, id_dtype == NF4_I64 ? 8 : 4) || !aligned(dy, 16) || !aligned(grad, 16)) return NF4_ERR_ALIGN;
    if ((st = check_workspace(embedding_backward_workspace(tokens, vocab, dim), workspace, workspace_bytes)) != NF4_OK)
        return st;
    return launch_status(launch_embedding_backward(ids, id_dtype == NF4_I64, tokens, dy,
                                                   static_cast<nf4_dtype>(dtype), vocab, dim, scale, padding_id, grad,
                                                   static_cast<nf4_dtype>(grad_dtype), accumulate != 0, workspace,
                                                   stream_of(stream)));
}
