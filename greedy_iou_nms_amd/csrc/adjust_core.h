// The rules on a slice of a row of logits, shared by nms_adjust_logits and
// nms_pick_tokens.
//
// One word of LDS per token of the slice gathers what the history and the
// bias list say about it: the place of its last bias entry (11 bits, stored
// as 2047 - place so that no entry reads as all ones), a bit for "seen in the
// prompt" and 20 bits of "how often generated".  Then every thread looks at
// the words of its own tokens, eight neighbours at a time, and replaces each
// touched word by the token's adjusted value: as many rounds as the wave's
// fullest lane has touched tokens, not eight times the division and the four
// operations behind it.  An untouched word is a NaN that no adjusted value
// is, so that a token then costs one compare and one select.
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

// array[row], or what stands for an array that is not given.  The load is
// made either way, from `any` if need be, so that all of a row's parameters
// are in flight together: behind a branch each they cost a round trip each,
// 1.6 us before a slice of 16384 tokens could begin.
template <typename V>
__device__ __forceinline__ V parameter(const V *array, int64_t row, V otherwise, const void *any) {
    const V v = *(array ? array + row : static_cast<const V *>(any));
    return array ? v : otherwise;
}

// Four bytes that may be read, whatever they hold: the aligned word with the
// logits' first element.
__device__ __forceinline__ const void *readable(const void *logits) {
    return reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(logits) & ~(uintptr_t)3);
}

__device__ __forceinline__ RowRules row_rules(const nms_logit_rules &u, int64_t row,
                                              const void *any) {
    RowRules r;
    r.repetition = parameter(u.repetition, row, 1.0f, any);
    r.presence = parameter(u.presence, row, 0.0f, any);
    r.frequency = parameter(u.frequency, row, 0.0f, any);
    const int length = parameter(u.history_len, row, 0, any);
    const int prompt = parameter(u.prompt_len, row, 0, any);
    const int64_t at = parameter(u.allowed_rows, row, (int)row, any);
    r.length = min(max(length, 0), (int)u.history_capacity);
    r.prompt = min(max(prompt, 0), r.length);
    r.none_allowed = u.allowed && at >= u.allowed_count;
    r.allowed = u.allowed && at >= 0 && !r.none_allowed
                    ? reinterpret_cast<const uint8_t *>(u.allowed + at * u.allowed_stride)
                    : nullptr;
    r.words = r.length > 0 || u.bias_count > 0;
    return r;
}

// A thread's first entries of the history, which it loads before it knows
// how many are in use.
constexpr int EARLY = 4;
struct EarlyHistory {
    int v[EARLY];
};

template <int THREADS>
__device__ __forceinline__ EarlyHistory early_history(const nms_logit_rules &u, int64_t row) {
    EarlyHistory e;
    const int32_t *history = u.history + row * u.history_stride;
#pragma unroll
    for (int q = 0; q < EARLY; ++q) {
        const int i = q * THREADS + (int)threadIdx.x;
        e.v[q] = i < (int)u.history_capacity ? history[i] : -1;
    }
    return e;
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

// Gathers the rules of the tokens lo..lo+size-1 of the row in word[0..SLICE).
// Every thread of the workgroup calls it, and it ends with a barrier.
template <int THREADS, int SLICE>
__device__ __forceinline__ void slice_rules(const nms_logit_rules &u, const RowRules &r,
                                            int64_t row, int lo, int size,
                                            const EarlyHistory &early, uint32_t *word) {
    const int tid = threadIdx.x;
    const uint4 none = make_uint4(UNTOUCHED, UNTOUCHED, UNTOUCHED, UNTOUCHED);
    for (int i = tid; i < SLICE / 4; i += THREADS) reinterpret_cast<uint4 *>(word)[i] = none;
    __syncthreads();
    if (u.bias_count > 0) {
        const int32_t *ids = u.bias_ids + row * u.bias_stride;
        for (int i = tid; i < (int)u.bias_count; i += THREADS) {
            const unsigned at = (unsigned)ids[i] - (unsigned)lo;
            if (at < (unsigned)size)
                atomicMin(&word[slot<SLICE>(at)], (RULE_NO_BIAS - (uint32_t)(i + 1))
                                                      << RULE_BIAS_SHIFT);
        }
        __syncthreads();
    }
    auto count = [&](int i, int v) {
        const unsigned at = (unsigned)v - (unsigned)lo;
        if (i < r.length && at < (unsigned)size) {
            uint32_t *w = &word[slot<SLICE>(at)];
            if (i < r.prompt) atomicOr(w, RULE_SEEN);
            else atomicAdd(w, 1u);
        }
    };
#pragma unroll
    for (int q = 0; q < EARLY; ++q) count(q * THREADS + tid, early.v[q]);
    const int32_t *history = u.history + row * u.history_stride;
    for (int i0 = EARLY * THREADS; i0 < r.length; i0 += EARLY * THREADS) {
        int v[EARLY];
#pragma unroll
        for (int q = 0; q < EARLY; ++q) {
            const int i = i0 + q * THREADS + tid;
            v[q] = i < r.length ? history[i] : -1;
        }
#pragma unroll
        for (int q = 0; q < EARLY; ++q) count(i0 + q * THREADS + tid, v[q]);
    }
    __syncthreads();
}

// Eight neighbouring logits from any element-aligned address.
template <typename T>
struct Eight {
    T v[8];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p, int left) {
    Eight<T> e;
    if (left >= 8) {
        __builtin_memcpy(&e, p, sizeof(e));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = j < left ? p[j] : from_f32<T>(NEG_INF);
    }
    return e;
}

// The adjusted values of the eight tokens at..at+7 of the slice (at a
// multiple of 8) from their logits, which start at in; those past the slice
// are -infinity.
template <typename T, int SLICE>
__device__ __forceinline__ void adjusted8(const nms_logit_rules &u, const RowRules &r, int64_t row,
                                          int lo, int size, int at, const T *in,
                                          const Eight<T> &logits, uint32_t *word, float *z) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = to_f32(logits.v[j]);
    if (r.words) {
        uint32_t w[8];
        uint4 *w0 = reinterpret_cast<uint4 *>(word + at / 2);
        uint4 *w1 = reinterpret_cast<uint4 *>(word + SLICE / 2 + at / 2);
        __builtin_memcpy(w, w0, 16);
        __builtin_memcpy(w + 4, w1, 16);
        uint32_t touched = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) touched |= w[j] == UNTOUCHED ? 0u : 1u << j;
        if (touched != 0u) {
            do {
                const int j = __builtin_ctz(touched);
                touched &= touched - 1u;
                uint32_t *x = word + (j >> 2) * (SLICE / 2) + at / 2 + (j & 3);
                *x = replaced(u, r, row, to_f32(in[at + j]), *x);
            } while (touched != 0u);
            __builtin_memcpy(w, w0, 16);
            __builtin_memcpy(w + 4, w1, 16);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = w[j] == UNTOUCHED ? z[j] : __uint_as_float(w[j]);
    }
    if (r.allowed) {
        const int bits = at < size ? r.allowed[(lo + at) >> 3] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t keep = (uint32_t)((int)((uint32_t)bits << (31 - j)) >> 31);
            z[j] = __uint_as_float((__float_as_uint(z[j]) & keep) | (0xff800000u & ~keep));
        }
    } else if (r.none_allowed) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = NEG_INF;
    }
}

}  // namespace gnms
