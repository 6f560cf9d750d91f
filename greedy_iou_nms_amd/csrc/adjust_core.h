// The rules on a slice of a row of logits, shared by nms_adjust_logits and
// nms_pick_tokens.
//
// One word of LDS per token of the slice.  First the words gather what the
// history and the bias list say: the place of the token's last bias entry
// (11 bits, stored as 2047 - place so that no entry reads as all ones), a bit
// for "seen in the prompt" and 20 bits of "how often generated".  Then the
// touched words are replaced by the token's adjusted value, one thread per
// touched token, and the slice is streamed once: an untouched word is a NaN
// that no adjusted value is, so a token costs one compare and one select,
// however many tokens the history touches.  (Adjusting while streaming costs
// a division and four more operations for every token of a wave that holds
// one touched token, and with a history of a few thousand tokens every wave
// does.)
#pragma once

#include "select_internal.h"

namespace gnms {

constexpr int RULE_BIAS_SHIFT = 21;
constexpr uint32_t RULE_SEEN = 1u << 20;
constexpr uint32_t RULE_COUNT = RULE_SEEN - 1u;
constexpr uint32_t RULE_TOUCHED = RULE_SEEN | RULE_COUNT;  // by the history
constexpr uint32_t RULE_NO_BIAS = 2047u;
constexpr uint32_t UNTOUCHED = RULE_NO_BIAS << RULE_BIAS_SHIFT;  // a NaN
static_assert(NMS_MAX_HISTORY == RULE_COUNT, "a count fits its field");
static_assert(NMS_MAX_BIASES <= (int)RULE_NO_BIAS, "a place fits its field");

// What one row's rules are, read once per workgroup.
struct RowRules {
    float repetition, presence, frequency;
    int length, prompt;        // of the history, both within its capacity
    const uint8_t *allowed;    // the row's mask, a byte per 8 tokens; null: none
    bool none_allowed;         // the row names a mask that does not exist
    bool words;                // the history or the bias list has entries
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
        else if (at >= 0) r.allowed = reinterpret_cast<const uint8_t *>(u.allowed + at * u.allowed_stride);
    }
    r.words = r.length > 0 || u.bias_count > 0;
    return r;
}

// Where the word of a slice's token lies: threads read the words of eight
// neighbouring tokens as two quarters, and a wave's quarters lie side by side
// (eight neighbouring words per lane would put every other lane on the same
// LDS banks).
template <int SLICE>
__device__ __forceinline__ unsigned slot(unsigned at) {
    return ((at >> 2) & 1u) * (SLICE / 2) + (at >> 3) * 4 + (at & 3u);
}

// The adjusted value of a touched token, but for its mask.  Every operation
// is one binary32 operation (compiled without contraction).
__device__ __forceinline__ uint32_t replaced(const nms_logit_rules &u, const RowRules &r,
                                             int64_t row, float z, uint32_t word) {
    if (word & RULE_TOUCHED) z = z > 0.0f ? z / r.repetition : z * r.repetition;
    const uint32_t count = word & RULE_COUNT;
    if (count > 0u) {
        z = z - r.frequency * (float)count;
        z = z - r.presence;
    }
    const uint32_t place = RULE_NO_BIAS - (word >> RULE_BIAS_SHIFT);
    if (place > 0u) z = z + u.bias_values[row * u.bias_stride + place - 1];
    // one NaN for all, which is not UNTOUCHED
    return z != z ? 0x7fc00000u : __float_as_uint(z);
}

// Fills word[0..SLICE) for the tokens lo..lo+size-1 of the row: UNTOUCHED, or
// the adjusted value's bits.  Every thread of the workgroup calls it, and it
// ends with a barrier.  in: the slice's logits.
template <typename T, int THREADS, int SLICE>
__device__ __forceinline__ void slice_rules(const nms_logit_rules &u, const RowRules &r,
                                            int64_t row, int lo, int size, const T *in,
                                            uint32_t *word) {
    const int tid = threadIdx.x;
    const uint4 none = make_uint4(UNTOUCHED, UNTOUCHED, UNTOUCHED, UNTOUCHED);
    for (int i = tid; i < SLICE / 4; i += THREADS) reinterpret_cast<uint4 *>(word)[i] = none;
    __syncthreads();
    const int32_t *bias_ids = u.bias_ids + row * u.bias_stride;
    if (u.bias_count > 0) {
        for (int i = tid; i < (int)u.bias_count; i += THREADS) {
            const unsigned at = (unsigned)bias_ids[i] - (unsigned)lo;
            if (at < (unsigned)size)
                atomicMin(&word[slot<SLICE>(at)], (RULE_NO_BIAS - (uint32_t)(i + 1))
                                                      << RULE_BIAS_SHIFT);
        }
        __syncthreads();
    }
    // The thread whose access is the first to a token adjusts it; which
    // thread that is makes no difference to the value.  Up to 64 entries per
    // thread are remembered in a bit each.
    const int32_t *history = u.history + row * u.history_stride;
    const bool remember = r.length <= 64 * THREADS;
    uint64_t owned = 0;
    for (int i0 = 0; i0 < r.length; i0 += 4 * THREADS) {
        int v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * THREADS + tid;
            v[q] = i < r.length ? history[i] : -1;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned at = (unsigned)v[q] - (unsigned)lo;
            if (at < (unsigned)size) {
                uint32_t *w = &word[slot<SLICE>(at)];
                const uint32_t old = i0 + q * THREADS + tid < r.prompt ? atomicOr(w, RULE_SEEN)
                                                                       : atomicAdd(w, 1u);
                if ((old & RULE_TOUCHED) == 0u && remember)
                    owned |= 1ull << (i0 / THREADS + q);
            }
        }
    }
    __syncthreads();
    if (remember) {
        // tokens that only the bias list touches: decided for every entry
        // before any word is replaced
        constexpr int MOST = (NMS_MAX_BIASES + THREADS - 1) / THREADS;
        uint32_t biased[MOST];
#pragma unroll
        for (int q = 0; q < MOST; ++q) {
            const int i = q * THREADS + tid;
            biased[q] = UNTOUCHED;
            if (i < (int)u.bias_count) {
                const unsigned at = (unsigned)bias_ids[i] - (unsigned)lo;
                if (at < (unsigned)size) {
                    const uint32_t w = word[slot<SLICE>(at)];
                    if ((w & RULE_TOUCHED) == 0u &&
                        w >> RULE_BIAS_SHIFT == RULE_NO_BIAS - (uint32_t)(i + 1))
                        biased[q] = w;
                }
            }
        }
        if (u.bias_count > 0) __syncthreads();
#pragma unroll
        for (int q = 0; q < MOST; ++q)
            if (biased[q] != UNTOUCHED) {
                const unsigned at = (unsigned)bias_ids[q * THREADS + tid] - (unsigned)lo;
                word[slot<SLICE>(at)] = replaced(u, r, row, to_f32(in[at]), biased[q]);
            }
        while (owned != 0ull) {
            const int q = __builtin_ctzll(owned);
            owned &= owned - 1ull;
            const unsigned at = (unsigned)history[q * THREADS + tid] - (unsigned)lo;
            uint32_t *w = &word[slot<SLICE>(at)];
            *w = replaced(u, r, row, to_f32(in[at]), *w);
        }
    } else {
        // a history this long touches a good part of the slice: every thread
        // looks through tokens of its own
        for (int i = tid; i < size; i += THREADS) {
            uint32_t *w = &word[slot<SLICE>(i)];
            if (*w != UNTOUCHED) *w = replaced(u, r, row, to_f32(in[i]), *w);
        }
    }
    __syncthreads();
}

// Eight neighbouring logits from any element-aligned address.
template <typename T>
struct Eight {
    T v[8];
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, int left, float *z) {
    if (left >= 8) {
        Eight<T> e;
        __builtin_memcpy(&e, p, sizeof(e));
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = to_f32(e.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = j < left ? to_f32(p[j]) : NEG_INF;
    }
}

// The adjusted values of the eight tokens at..at+7 of the slice (at a
// multiple of 8); those past the slice are -infinity.
template <typename T, int SLICE>
__device__ __forceinline__ void adjusted8(const RowRules &r, int lo, int size, int at, const T *in,
                                          const uint32_t *word, float *z) {
    load8(in + at, size - at, z);
    if (r.words) {
        uint32_t w[8];
        __builtin_memcpy(w, word + at / 2, 16);
        __builtin_memcpy(w + 4, word + SLICE / 2 + at / 2, 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = w[j] == UNTOUCHED ? z[j] : __uint_as_float(w[j]);
    }
    if (r.allowed) {
        const uint32_t bits = at < size ? r.allowed[(lo + at) >> 3] : 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (bits >> j) & 1u ? z[j] : NEG_INF;
    } else if (r.none_allowed) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = NEG_INF;
    }
}

}  // namespace gnms
