// Host side of the losses of language models: argument checks, then the
// launches on the caller's stream.  Nothing here waits for the GPU or allocates.
#include <hip/hip_runtime.h>

#include <cmath>

#include "loss_internal.h"

using namespace gnms;

namespace {

nms_status hip_status(hipError_t e) { return e == hipSuccess ? NMS_OK : NMS_HIP_ERROR; }

bool known(nms_dtype t) { return t == NMS_F32 || t == NMS_F16 || t == NMS_BF16; }

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A matrix of rows whose elements are contiguous: rows must not overlap.
nms_status check_matrix(const void *p, nms_dtype t, int64_t rows, int64_t columns,
                        int64_t stride) {
    if (p == nullptr || !aligned(p, t == NMS_F32 ? 4 : 2)) return NMS_INVALID_ARG;
    if (rows > 1 && stride < columns) return NMS_INVALID_ARG;
    return NMS_OK;
}

nms_status check_sizes(nms_dtype dtype, int64_t rows, int64_t vocab) {
    if (!known(dtype) || rows < 0 || vocab < 1) return NMS_INVALID_ARG;
    if (rows > NMS_MAX_ROWS || vocab > NMS_MAX_VOCAB) return NMS_TOO_LARGE;
    return NMS_OK;
}

nms_status check_workspace(const void *workspace, size_t bytes, size_t needed) {
    if (workspace == nullptr || !aligned(workspace, 256)) return NMS_INVALID_ARG;
    return bytes < needed ? NMS_WORKSPACE_TOO_SMALL : NMS_OK;
}

// What all calls on rows of logits check; grad_logits null: not wanted.
nms_status check_rows(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                      int64_t row_stride, const int32_t *tokens, const void *grad_logits,
                      int64_t grad_stride) {
    if (rows == 0) return NMS_OK;
    nms_status st = check_matrix(logits, dtype, rows, vocab, row_stride);
    if (st == NMS_OK && grad_logits)
        st = check_matrix(grad_logits, dtype, rows, vocab, grad_stride);
    if (st == NMS_OK && tokens == nullptr) st = NMS_INVALID_ARG;
    return st;
}

nms_status check_preference(const nms_preference_options *o, int64_t pairs,
                            const int64_t *offsets) {
    if (o == nullptr || pairs < 1) return NMS_INVALID_ARG;
    if (pairs > NMS_MAX_PAIRS) return NMS_TOO_LARGE;
    if (o->kind != NMS_PREFERENCE_SIGMOID && o->kind != NMS_PREFERENCE_HINGE &&
        o->kind != NMS_PREFERENCE_SQUARED)
        return NMS_INVALID_ARG;
    if (!(o->beta > 0.0f) || !std::isfinite(o->beta) || !std::isfinite(o->margin) ||
        !(o->smoothing >= 0.0f) || o->smoothing > 0.5f ||
        (o->smoothing != 0.0f && o->kind != NMS_PREFERENCE_SIGMOID))
        return NMS_INVALID_ARG;
    if (offsets == nullptr || !aligned(offsets, 8)) return NMS_INVALID_ARG;
    return NMS_OK;
}

PreferenceArgs preference_args(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, const int32_t *tokens, const int64_t *offsets,
                               int64_t pairs, const float *weights,
                               const nms_preference_options &o, const float *grad_loss,
                               void *grad_logits, int64_t grad_stride, void *workspace) {
    PreferenceArgs a = {};
    a.in = {logits, dtype, rows, (int)vocab, row_stride, tokens, nullptr, nullptr};
    a.offsets = offsets;
    a.pairs = pairs;
    a.weights = weights;
    a.weight = (float)(1.0 / (double)pairs);
    a.beta = o.beta;
    a.smoothing = o.smoothing;
    a.margin = o.margin;
    a.kind = o.kind;
    a.average = o.average != 0;
    a.grad_loss = grad_loss;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    a.workspace = workspace;
    return a;
}

}  // namespace

extern "C" {

nms_status nms_loss_workspace_size(int64_t rows, int64_t vocab, int64_t pairs, size_t *bytes) {
    if (bytes == nullptr) return NMS_INVALID_ARG;
    *bytes = 0;
    const nms_status st = check_sizes(NMS_F32, rows, vocab);
    if (st != NMS_OK) return st;
    if (pairs < 0) return NMS_INVALID_ARG;
    if (pairs > NMS_MAX_PAIRS) return NMS_TOO_LARGE;
    *bytes = loss_workspace_bytes(rows, (int)vocab, pairs);
    return NMS_OK;
}

nms_status nms_token_logprobs(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                              int64_t row_stride, const int32_t *tokens, const float *temperature,
                              float *logprobs, float *entropies, void *workspace,
                              size_t workspace_bytes, void *stream) {
    nms_status st = check_sizes(dtype, rows, vocab);
    if (st != NMS_OK) return st;
    if (rows == 0) return NMS_OK;
    st = check_rows(logits, dtype, rows, vocab, row_stride, tokens, nullptr, 0);
    if (st != NMS_OK) return st;
    if (logprobs == nullptr) return NMS_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, loss_workspace_bytes(rows, (int)vocab, 0));
    if (st != NMS_OK) return st;
    LossArgs a = {};
    a.in = {logits, dtype, rows, (int)vocab, row_stride, tokens, temperature, nullptr};
    a.kind = LOSS_LOGPROBS;
    a.logprobs = logprobs;
    a.entropies = entropies;
    a.entropy = entropies != nullptr;
    a.workspace = workspace;
    return hip_status(launch_loss(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_token_logprobs_backward(const void *logits, nms_dtype dtype, int64_t rows,
                                       int64_t vocab, int64_t row_stride, const int32_t *tokens,
                                       const float *temperature, const float *grad_logprobs,
                                       const float *grad_entropies, void *grad_logits,
                                       int64_t grad_stride, void *workspace,
                                       size_t workspace_bytes, void *stream) {
    nms_status st = check_sizes(dtype, rows, vocab);
    if (st != NMS_OK) return st;
    if (rows == 0) return NMS_OK;
    if (grad_logprobs == nullptr || grad_logits == nullptr) return NMS_INVALID_ARG;
    st = check_rows(logits, dtype, rows, vocab, row_stride, tokens, grad_logits, grad_stride);
    if (st != NMS_OK) return st;
    st = check_workspace(workspace, workspace_bytes, loss_workspace_bytes(rows, (int)vocab, 0));
    if (st != NMS_OK) return st;
    LossArgs a = {};
    a.in = {logits, dtype, rows, (int)vocab, row_stride, tokens, temperature, nullptr};
    a.kind = LOSS_GIVEN;
    a.grad_logprobs = grad_logprobs;
    a.grad_entropies = grad_entropies;
    a.entropy = grad_entropies != nullptr;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    a.workspace = workspace;
    return hip_status(launch_loss(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_policy_loss(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                           int64_t row_stride, const int32_t *tokens, const float *old_logprobs,
                           const float *advantages, const float *weights,
                           const float *ref_logprobs, const float *temperature,
                           const nms_policy_options *options, const float *grad_loss, float *loss,
                           float *logprobs, float *entropies, void *grad_logits,
                           int64_t grad_stride, void *workspace, size_t workspace_bytes,
                           void *stream) {
    nms_status st = check_sizes(dtype, rows, vocab);
    if (st != NMS_OK) return st;
    if (options == nullptr) return NMS_INVALID_ARG;
    const nms_policy_options &o = *options;
    if (!(o.clip_low >= 0.0f && o.clip_low <= 1.0f && o.clip_high >= 0.0f) ||
        !std::isfinite(o.clip_high) || !(o.kl >= 0.0f) || !std::isfinite(o.kl) ||
        !std::isfinite(o.entropy))
        return NMS_INVALID_ARG;
    if (rows > 0) {
        // (the arrays of an empty batch have no address)
        st = check_rows(logits, dtype, rows, vocab, row_stride, tokens, grad_logits, grad_stride);
        if (st != NMS_OK) return st;
        if (old_logprobs == nullptr || advantages == nullptr ||
            (o.kl != 0.0f && ref_logprobs == nullptr) ||
            (loss == nullptr && logprobs == nullptr && entropies == nullptr &&
             grad_logits == nullptr))
            return NMS_INVALID_ARG;
    }
    st = check_workspace(workspace, workspace_bytes, loss_workspace_bytes(rows, (int)vocab, 0));
    if (st != NMS_OK) return st;
    LossArgs a = {};
    a.in = {logits, dtype, rows, (int)vocab, row_stride, tokens, temperature, weights};
    a.kind = LOSS_POLICY;
    a.old_logprobs = old_logprobs;
    a.advantages = advantages;
    a.ref_logprobs = o.kl != 0.0f ? ref_logprobs : nullptr;
    a.clip_low = (float)(1.0 - (double)o.clip_low);
    a.clip_high = (float)(1.0 + (double)o.clip_high);
    a.kl = o.kl;
    a.bonus = o.entropy;
    a.weight = rows > 0 ? (float)(1.0 / (double)rows) : 0.0f;
    a.grad_loss = grad_loss;
    a.loss = loss;
    a.logprobs = logprobs;
    a.entropies = entropies;
    a.entropy = entropies != nullptr || o.entropy != 0.0f;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    a.workspace = workspace;
    return hip_status(launch_loss(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_preference_loss(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, const int32_t *tokens, const int64_t *offsets,
                               int64_t pairs, const float *ref_logprobs, const float *weights,
                               const nms_preference_options *options, const float *grad_loss,
                               float *loss, float *logprobs, float *margins, void *grad_logits,
                               int64_t grad_stride, void *workspace, size_t workspace_bytes,
                               void *stream) {
    nms_status st = check_sizes(dtype, rows, vocab);
    if (st == NMS_OK) st = check_preference(options, pairs, offsets);
    if (st == NMS_OK)
        st = check_rows(logits, dtype, rows, vocab, row_stride, tokens, grad_logits, grad_stride);
    if (st != NMS_OK) return st;
    if (loss == nullptr || logprobs == nullptr || margins == nullptr) return NMS_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes,
                         loss_workspace_bytes(rows, (int)vocab, pairs));
    if (st != NMS_OK) return st;
    PreferenceArgs a = preference_args(logits, dtype, rows, vocab, row_stride, tokens, offsets,
                                       pairs, weights, *options, grad_loss, grad_logits,
                                       grad_stride, workspace);
    a.ref_logprobs = ref_logprobs;
    a.loss = loss;
    a.logprobs = logprobs;
    a.margins = margins;
    return hip_status(launch_preference(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_preference_loss_backward(const void *logits, nms_dtype dtype, int64_t rows,
                                        int64_t vocab, int64_t row_stride, const int32_t *tokens,
                                        const int64_t *offsets, int64_t pairs,
                                        const float *weights,
                                        const nms_preference_options *options,
                                        const float *margins, const float *grad_loss,
                                        void *grad_logits, int64_t grad_stride, void *workspace,
                                        size_t workspace_bytes, void *stream) {
    nms_status st = check_sizes(dtype, rows, vocab);
    if (st == NMS_OK) st = check_preference(options, pairs, offsets);
    if (st != NMS_OK) return st;
    if (rows == 0) return NMS_OK;
    if (grad_logits == nullptr || margins == nullptr) return NMS_INVALID_ARG;
    st = check_rows(logits, dtype, rows, vocab, row_stride, tokens, grad_logits, grad_stride);
    if (st != NMS_OK) return st;
    st = check_workspace(workspace, workspace_bytes,
                         loss_workspace_bytes(rows, (int)vocab, pairs));
    if (st != NMS_OK) return st;
    PreferenceArgs a = preference_args(logits, dtype, rows, vocab, row_stride, tokens, offsets,
                                       pairs, weights, *options, grad_loss, grad_logits,
                                       grad_stride, workspace);
    a.known_margins = margins;
    return hip_status(launch_preference(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_balance_workspace_size(int64_t tokens, int64_t experts, int64_t sequences,
                                      int top_k, size_t *bytes) {
    if (bytes == nullptr) return NMS_INVALID_ARG;
    *bytes = 0;
    if (tokens < 0 || experts < 1 || sequences < 1 || top_k < 0 || top_k > NMS_ROUTE_MAX_TOP_K)
        return NMS_INVALID_ARG;
    if (experts > NMS_ROUTE_MAX_EXPERTS || tokens > NMS_ROUTE_MAX_TOKENS ||
        sequences > NMS_MAX_SEQUENCES)
        return NMS_TOO_LARGE;
    *bytes = balance_workspace_bytes(tokens, (int)experts, sequences, top_k);
    return NMS_OK;
}

nms_status nms_balance_loss(const void *logits, nms_dtype dtype, int64_t tokens, int64_t experts,
                            int64_t row_stride, const int32_t *ids, const uint8_t *live,
                            const int64_t *offsets, int64_t sequences,
                            const nms_balance_options *options, const float *grad_loss,
                            float *loss, int32_t *counts, void *grad_logits, int64_t grad_stride,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (options == nullptr || !known(dtype)) return NMS_INVALID_ARG;
    const nms_balance_options &o = *options;
    size_t needed = 0;
    nms_status st = nms_balance_workspace_size(tokens, experts, sequences, o.top_k, &needed);
    if (st != NMS_OK) return st;
    if ((o.score != NMS_ROUTE_SOFTMAX && o.score != NMS_ROUTE_SIGMOID) ||
        !std::isfinite(o.balance) || !std::isfinite(o.z))
        return NMS_INVALID_ARG;
    if (offsets == nullptr ? sequences != 1 : !aligned(offsets, 8)) return NMS_INVALID_ARG;
    if (tokens > 0) {
        st = check_matrix(logits, dtype, tokens, experts, row_stride);
        if (st == NMS_OK && grad_logits)
            st = check_matrix(grad_logits, dtype, tokens, experts, grad_stride);
        if (st != NMS_OK) return st;
    }
    // without ids the kernels read the counts, those of an empty batch too
    if (ids == nullptr && counts == nullptr) return NMS_INVALID_ARG;
    if (loss == nullptr && counts == nullptr && grad_logits == nullptr) return NMS_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, needed);
    if (st != NMS_OK) return st;
    const BalanceArgs a = {logits,     dtype,     tokens,  (int)experts, row_stride, ids,
                           o.top_k,    live,      offsets, sequences,    o.score,    o.balance,
                           o.z,        grad_loss, loss,    counts,       grad_logits, grad_stride,
                           workspace};
    return hip_status(launch_balance(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
