// Shared by the losses of language models (loss.hip, balance.hip) and their
// host side (loss_api.cpp): their arguments and their workspace.
#pragma once

#include "select_internal.h"

namespace gnms {

// Rows of logits with one token each.  A row counts where its token is in the
// vocabulary and its weight is not 0.
struct LossRows {
    const void *logits;
    int dtype;
    int64_t rows;
    int vocab;
    int64_t row_stride;
    const int32_t *tokens;
    const float *temperature;  // null: 1
    const float *weights;      // null: 1 (of the policy loss)
};

// What the rows' results become.
enum LossKind { LOSS_LOGPROBS, LOSS_GIVEN, LOSS_POLICY };

struct LossArgs {
    LossRows in;
    int kind;
    // LOSS_GIVEN: the gradients of the log probabilities and of the entropies
    const float *grad_logprobs, *grad_entropies;
    // LOSS_POLICY
    const float *old_logprobs, *advantages, *ref_logprobs;
    float clip_low, clip_high, kl, bonus, weight;
    const float *grad_loss;  // null: 1
    // outputs, each null where it is not wanted
    float *logprobs, *entropies, *loss;
    bool entropy;  // the rows' entropies are needed
    void *grad_logits;
    int64_t grad_stride;
    void *workspace;
};

struct PreferenceArgs {
    LossRows in;
    const int64_t *offsets;
    int64_t pairs;
    const float *ref_logprobs, *weights;  // of sequences; of pairs
    float weight;                         // of a pair where weights is null
    float beta, smoothing, margin;
    int kind;
    bool average;
    const float *grad_loss;
    float *loss, *logprobs, *margins;
    const float *known_margins;  // of the forward call, where only the gradient is wanted
    void *grad_logits;
    int64_t grad_stride;
    void *workspace;
};

struct BalanceArgs {
    const void *logits;
    int dtype;
    int64_t tokens;
    int experts;
    int64_t row_stride;
    const int32_t *ids;  // null: counts are given
    int top_k;
    const uint8_t *live;
    const int64_t *offsets;  // null: one sequence
    int64_t sequences;
    int score;
    float balance, z;
    const float *grad_loss;
    float *loss;
    int32_t *counts;
    void *grad_logits;
    int64_t grad_stride;
    void *workspace;
};

size_t loss_workspace_bytes(int64_t rows, int vocab, int64_t pairs);
hipError_t launch_loss(const LossArgs &a, hipStream_t stream);
hipError_t launch_preference(const PreferenceArgs &a, hipStream_t stream);
size_t balance_workspace_bytes(int64_t tokens, int experts, int64_t sequences, int top_k);
hipError_t launch_balance(const BalanceArgs &a, hipStream_t stream);

// Sums n terms in a fixed order into one float, by one workgroup.
void launch_total(const double *terms, int64_t n, float *out, hipStream_t stream);

}  // namespace gnms
