// Host side of the selection operators: argument checks, then the launches on
// the caller's stream.  Nothing here waits for the GPU or allocates.
#include <hip/hip_runtime.h>

#include <cmath>

#include "select_internal.h"

using namespace gnms;

namespace {

nms_status hip_status(hipError_t e) { return e == hipSuccess ? NMS_OK : NMS_HIP_ERROR; }

bool known(nms_dtype t) { return t == NMS_F32 || t == NMS_F16 || t == NMS_BF16; }

size_t size_of(nms_dtype t) { return t == NMS_F32 ? 4 : 2; }

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A matrix of rows whose elements are contiguous: rows must not overlap.
nms_status check_matrix(const void *p, nms_dtype t, int64_t rows, int64_t columns,
                        int64_t stride) {
    if (p == nullptr || !aligned(p, size_of(t))) return NMS_INVALID_ARG;
    if (rows > 1 && stride < columns) return NMS_INVALID_ARG;
    return NMS_OK;
}

nms_status check_route(nms_dtype dtype, int64_t tokens, int64_t experts,
                       const nms_route_options *o) {
    if (o == nullptr || !known(dtype) || tokens < 0 || experts < 1) return NMS_INVALID_ARG;
    if (experts > NMS_ROUTE_MAX_EXPERTS || tokens > NMS_ROUTE_MAX_TOKENS) return NMS_TOO_LARGE;
    if (o->score != NMS_ROUTE_SOFTMAX && o->score != NMS_ROUTE_SIGMOID) return NMS_INVALID_ARG;
    if (o->top_k < 1 || o->top_k > NMS_ROUTE_MAX_TOP_K || !std::isfinite(o->scale))
        return NMS_INVALID_ARG;
    return NMS_OK;
}

nms_status check_rules(const nms_logit_rules &u, int64_t rows, int64_t vocab) {
    if (u.history != nullptr) {
        if (u.history_len == nullptr || u.history_capacity < 0 ||
            u.history_stride < u.history_capacity)
            return NMS_INVALID_ARG;
        if (u.history_capacity > NMS_MAX_HISTORY) return NMS_TOO_LARGE;
    } else if (u.history_len != nullptr || u.prompt_len != nullptr) {
        return NMS_INVALID_ARG;
    }
    // (the entries of an empty batch have no address)
    if (u.bias_count < 0 || (u.bias_count > 0 && u.bias_stride < u.bias_count) ||
        (u.bias_count > 0 && rows > 0 && (!u.bias_ids || !u.bias_values)))
        return NMS_INVALID_ARG;
    if (u.bias_count > NMS_MAX_BIASES) return NMS_TOO_LARGE;
    if (u.allowed != nullptr) {
        if (u.allowed_count < 0 || u.allowed_stride < (vocab + 63) / 64 || !aligned(u.allowed, 8))
            return NMS_INVALID_ARG;
    } else if (u.allowed_rows != nullptr) {
        return NMS_INVALID_ARG;
    }
    return NMS_OK;
}

nms_status check_logits(nms_dtype dtype, int64_t rows, int64_t vocab) {
    if (!known(dtype) || rows < 0 || vocab < 1) return NMS_INVALID_ARG;
    if (rows > NMS_MAX_ROWS || vocab > NMS_MAX_VOCAB) return NMS_TOO_LARGE;
    return NMS_OK;
}

nms_logit_rules rules_or_none(const nms_logit_rules *u) {
    nms_logit_rules r = {};
    if (u != nullptr) {
        r = *u;
        if (r.history == nullptr) r.history_capacity = 0;
    }
    return r;
}

}  // namespace

extern "C" {

nms_status nms_route_experts(const void *logits, nms_dtype dtype, int64_t tokens, int64_t experts,
                             int64_t row_stride, const float *bias, const uint8_t *live,
                             const nms_route_options *options, int32_t *ids, float *weights,
                             int32_t *counts, void *stream) {
    nms_status st = check_route(dtype, tokens, experts, options);
    if (st != NMS_OK) return st;
    const nms_route_options &o = *options;
    if (o.groups < 1 || experts % o.groups != 0 || o.kept_groups < 1 || o.kept_groups > o.groups ||
        (o.group_top != 1 && o.group_top != 2) ||
        o.top_k > o.kept_groups * (experts / o.groups))
        return NMS_INVALID_ARG;
    if (tokens > 0) {
        st = check_matrix(logits, dtype, tokens, experts, row_stride);
        if (st != NMS_OK) return st;
        if (ids == nullptr || weights == nullptr) return NMS_INVALID_ARG;
    }
    const RouteArgs a = {logits, dtype, tokens, (int)experts, row_stride, bias,
                         live,   o,     ids,    weights,      counts};
    return hip_status(launch_route(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_route_experts_backward(const void *logits, nms_dtype dtype, int64_t tokens,
                                      int64_t experts, int64_t row_stride, const int32_t *ids,
                                      const float *grad_weights, const nms_route_options *options,
                                      void *grad_logits, int64_t grad_stride, void *stream) {
    nms_status st = check_route(dtype, tokens, experts, options);
    if (st != NMS_OK) return st;
    if (tokens == 0) return NMS_OK;
    st = check_matrix(logits, dtype, tokens, experts, row_stride);
    if (st == NMS_OK) st = check_matrix(grad_logits, dtype, tokens, experts, grad_stride);
    if (st != NMS_OK) return st;
    if (ids == nullptr || grad_weights == nullptr) return NMS_INVALID_ARG;
    const RouteBackArgs a = {logits, dtype,        tokens,   (int)experts, row_stride,
                             ids,    grad_weights, *options, grad_logits,  grad_stride};
    return hip_status(launch_route_back(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_adjust_logits(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                             int64_t row_stride, const nms_logit_rules *rules, void *out,
                             int64_t out_stride, void *stream) {
    nms_status st = check_logits(dtype, rows, vocab);
    if (st != NMS_OK) return st;
    if (rules == nullptr) return NMS_INVALID_ARG;
    st = check_rules(*rules, rows, vocab);
    if (st != NMS_OK) return st;
    if (rows == 0) return NMS_OK;
    st = check_matrix(logits, dtype, rows, vocab, row_stride);
    if (st == NMS_OK) st = check_matrix(out, dtype, rows, vocab, out_stride);
    if (st != NMS_OK) return st;
    const AdjustArgs a = {logits, dtype, rows, (int)vocab, row_stride, rules_or_none(rules), out,
                          out_stride};
    return hip_status(launch_adjust(a, static_cast<hipStream_t>(stream)));
}

nms_status nms_pick_workspace_size(int64_t rows, int64_t vocab, int max_top_k, size_t *bytes) {
    if (bytes == nullptr) return NMS_INVALID_ARG;
    *bytes = 0;
    const nms_status st = check_logits(NMS_F32, rows, vocab);
    if (st != NMS_OK) return st;
    if (max_top_k < 1 || max_top_k > NMS_MAX_TOP_K) return NMS_INVALID_ARG;
    *bytes = pick_workspace_bytes(rows, (int)vocab, max_top_k);
    return NMS_OK;
}

nms_status nms_pick_tokens(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                           int64_t row_stride, const nms_logit_rules *rules, const float *uniform,
                           const float *temperature, const int32_t *top_k, const float *top_p,
                           const float *min_p, int max_top_k, int32_t *ids, float *logprobs,
                           void *workspace, size_t workspace_bytes, void *stream) {
    nms_status st = check_logits(dtype, rows, vocab);
    if (st != NMS_OK) return st;
    if (max_top_k < 1 || max_top_k > NMS_MAX_TOP_K) return NMS_INVALID_ARG;
    if (rules != nullptr) {
        st = check_rules(*rules, rows, vocab);
        if (st != NMS_OK) return st;
    }
    if (rows == 0) return NMS_OK;
    st = check_matrix(logits, dtype, rows, vocab, row_stride);
    if (st != NMS_OK) return st;
    if (uniform == nullptr || ids == nullptr || logprobs == nullptr || workspace == nullptr ||
        !aligned(workspace, 256))
        return NMS_INVALID_ARG;
    if (workspace_bytes < pick_workspace_bytes(rows, (int)vocab, max_top_k))
        return NMS_WORKSPACE_TOO_SMALL;
    const PickArgs a = {logits,  dtype, rows,  (int)vocab, row_stride, rules_or_none(rules),
                        uniform, temperature, top_k, top_p, min_p, max_top_k, ids, logprobs,
                        workspace};
    return hip_status(launch_pick(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
