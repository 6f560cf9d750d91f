// The rules on a slice of a row of logits, shared by nms_adjust_logits and
// nms_pick_tokens.
//
// One word of LDS per token of the slice gathers what the history and the
// bias list say about it: how often it was generated (20 bits), whether it
// was seen at all, and the place of its last bias entry plus one (11 bits).
// The slice's logits are then read once.
#pragma once

#include "select_internal.h"

namespace gnms {

constexpr uint32_t RULE_COUNT = (1u << 20) - 1u;
constexpr uint32_t RULE_SEEN = 1u << 20;
constexpr int RULE_BIAS_SHIFT = 21;
static_assert(NMS_MAX_HISTORY == RULE_COUNT, "a count fits its field");
static_assert(NMS_MAX_BIASES < (1 << (32 - RULE_BIAS_SHIFT)), "a place fits its field");

// What one row's rules are, read once per workgroup.
struct RowRules {
    float repetition, presence, frequency;
    int length, prompt;            // of the history, both within its capacity
    const uint64_t *allowed;       // the row's mask words, or null: all allowed
    bool none_allowed;             // the row names a mask that does not exist
    bool words;                    // the history or the bias list has entries
};

__device__ __forceinline__ RowRules row_rules(const nms_logit_rules &u, int64_t row) {
    RowRules r;
    r.repetition = u.repetition ? u.repetition[row] : 1.0f;
    r.presence = u.presence ? u.presence[row] : 0.0f;
    r.frequency = u.frequency ? u.frequency[row] : 0.0f;
    r.length = 0;
    r.prompt = 0;
    if (u.history) {
        const int cap = (int)u.history_capacity;
        r.length = min(max(u.history_len[row], 0), cap);
        r.prompt = u.prompt_len ? min(max(u.prompt_len[row], 0), r.length) : 0;
    }
    r.allowed = nullptr;
    r.none_allowed = false;
    if (u.allowed) {
        const int64_t at = u.allowed_rows ? (int64_t)u.allowed_rows[row] : row;
        if (at >= u.allowed_count) r.none_allowed = true;
        else if (at >= 0) r.allowed = u.allowed + at * u.allowed_stride;
    }
    r.words = r.length > 0 || u.bias_count > 0;
    return r;
}

// Fills word[0..size) for the tokens lo..lo+size-1 of the row.  Every thread
// of the workgroup calls it; it ends with a barrier.
__device__ __forceinline__ void gather_rules(const nms_logit_rules &u, const RowRules &r,
                                             int64_t row, int lo, int size, uint32_t *word,
                                             int tid, int threads) {
    if (!r.words) return;
    for (int i = tid; i < size; i += threads) word[i] = 0;
    __syncthreads();
    if (u.bias_count > 0) {
        const int32_t *ids = u.bias_ids + row * u.bias_stride;
        for (int i = tid; i < (int)u.bias_count; i += threads) {
            const unsigned at = (unsigned)ids[i] - (unsigned)lo;
            if (ids[i] >= 0 && at < (unsigned)size)
                atomicMax(&word[at], (uint32_t)(i + 1) << RULE_BIAS_SHIFT);
        }
        __syncthreads();
    }
    const int32_t *history = u.history + row * u.history_stride;
    for (int i = tid; i < r.length; i += threads) {
        const int v = history[i];
        const unsigned at = (unsigned)v - (unsigned)lo;
        if (v >= 0 && at < (unsigned)size) {
            atomicOr(&word[at], RULE_SEEN);
            if (i >= r.prompt) atomicAdd(&word[at], 1u);
        }
    }
    __syncthreads();
}

// The adjusted value of one token.  Every operation is one binary32
// operation (this file is compiled without contraction).
__device__ __forceinline__ float adjusted(const nms_logit_rules &u, const RowRules &r, int64_t row,
                                          float z, uint32_t word, int token) {
    if (word != 0u) {
        if (word & RULE_SEEN) z = z > 0.0f ? z / r.repetition : z * r.repetition;
        const uint32_t count = word & RULE_COUNT;
        if (count > 0u) {
            z = z - r.frequency * (float)count;
            z = z - r.presence;
        }
        const uint32_t place = word >> RULE_BIAS_SHIFT;
        if (place > 0u) z = z + u.bias_values[row * u.bias_stride + place - 1];
    }
    if (r.none_allowed) return NEG_INF;
    if (r.allowed && !((r.allowed[token >> 6] >> (token & 63)) & 1ull)) return NEG_INF;
    return z;
}

}  // namespace gnms
