// The rules on a slice of a row of logits, shared by nms_adjust_logits and
// nms_pick_tokens.
//
// One word of LDS per token of the slice gathers what the history and the
// bias list say about it: how often it was generated (20 bits) and the place
// of its last bias entry plus one (11 bits); one bit per token says whether it
// is in the history, another whether it is in the bias list.  Then every thread looks
// through the bits of its own tokens, replaces the words of those touched by
// their adjusted values, and selects between these and the logits.  That is
// as many rounds as the wave's fullest lane has touched tokens, where
// adjusting in line costs every token of a wave with one touched token the
// division and the four operations behind it.
#pragma once

#include "select_internal.h"

namespace gnms {

constexpr uint32_t RULE_COUNT = (1u << 20) - 1u;
constexpr int RULE_BIAS_SHIFT = 21;
static_assert(NMS_MAX_HISTORY == RULE_COUNT, "a count fits its field");
static_assert(NMS_MAX_BIASES < (1 << (32 - RULE_BIAS_SHIFT)), "a place fits its field");

// What one row's rules are, read once per workgroup.
struct RowRules {
    float repetition, presence, frequency;
    int length, prompt;        // of the history, both within its capacity
    bool masked;               // the row has a mask,
    const uint8_t *allowed;    // a byte per 8 tokens; null: no token is allowed
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
    r.masked = u.allowed && at >= 0;
    r.allowed = r.masked && at < u.allowed_count
                    ? reinterpret_cast<const uint8_t *>(u.allowed + at * u.allowed_stride)
                    : nullptr;
    r.words = r.length > 0 || u.bias_count > 0;
    return r;
}

// Four neighbouring entries of a history.
struct FourTokens {
    int v[4];
};

// A wave's next 256 entries from base on, four per lane; -1 from limit on.
__device__ __forceinline__ FourTokens load4(const int32_t *history, int base, int limit) {
    FourTokens f;
    const int i = base + 4 * (int)(threadIdx.x & 63);
    if (base + 256 <= limit) {  // the same for the whole wave
        __builtin_memcpy(&f, history + i, sizeof(f));
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) f.v[c] = i + c < limit ? history[i + c] : -1;
    }
    return f;
}

// The first of a wave's entries, in the first round.
__device__ __forceinline__ int wave_entry() {
    return __builtin_amdgcn_readfirstlane(4 * (int)(threadIdx.x & ~63u));
}

// Where the word of a slice's token lies: threads read the words of eight
// neighbouring tokens as two quarters of four, and every other eight lanes have
// theirs exchanged (a wave's first quarters, 32 bytes apart, would else lie on
// half of the LDS banks).
__device__ __forceinline__ unsigned slot(unsigned at) {
    return at ^ (at >> 4 & 4u);
}

// The adjusted value of a touched token, but for its mask.  Every operation
// is one binary32 operation (compiled without contraction).
__device__ __forceinline__ float replaced(const nms_logit_rules &u, const RowRules &r, int64_t row,
                                          float z, bool seen, uint32_t word) {
    if (seen) z = z > 0.0f ? z / r.repetition : z * r.repetition;
    const uint32_t count = word & RULE_COUNT;
    if (count > 0u) {
        z = z - r.frequency * (float)count;
        z = z - r.presence;
    }
    const uint32_t place = word >> RULE_BIAS_SHIFT;
    if (place > 0u) z = z + u.bias_values[row * u.bias_stride + place - 1];
    return z;
}

// What a slice's rules are gathered in: a word per token, and the bits of
// those in the history and of those in the bias list.
template <int SLICE>
struct alignas(16) RuleSpace {
    uint32_t seen[SLICE / 32], listed[SLICE / 32], word[SLICE];
};

// Gathers the rules of the tokens lo..lo+size-1 of the row.  early: the first
// entries, load4 up to the capacity.  Every thread of the workgroup calls it,
// and it ends with a barrier.
template <int THREADS, int SLICE>
__device__ __forceinline__ void slice_rules(const nms_logit_rules &u, const RowRules &r,
                                            int64_t row, int lo, int size,
                                            const FourTokens &early, RuleSpace<SLICE> &x) {
    const int tid = threadIdx.x;
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < SLICE / 4 / THREADS; ++i)
        reinterpret_cast<uint4 *>(x.word)[i * THREADS + tid] = none;
    for (int i = tid; i < SLICE / 32; i += THREADS) x.seen[i] = x.listed[i] = 0;
    // entries two loads ahead of those that are counted
    constexpr int STEP = 4 * THREADS, DEEP = 2;
    const int32_t *history = u.history + row * u.history_stride;
    const int first = wave_entry();
    FourTokens next[DEEP];
    auto load = [&](int base) {
#pragma unroll
        for (int q = 0; q < DEEP; ++q) next[q] = load4(history, base + q * STEP, r.length);
    };
    if (first + STEP < r.length) load(first + STEP);
    __syncthreads();
    if (u.bias_count > 0) {
        const int32_t *ids = u.bias_ids + row * u.bias_stride;
        for (int i = tid; i < (int)u.bias_count; i += THREADS) {
            const unsigned at = (unsigned)ids[i] - (unsigned)lo;
            if (at < (unsigned)size) {
                atomicMax(&x.word[slot(at)], (uint32_t)(i + 1) << RULE_BIAS_SHIFT);
                atomicOr(&x.listed[at >> 5], 1u << (at & 31u));
            }
        }
        __syncthreads();
    }
    // a token of the prompt is counted 0 times
    auto count = [&](int base, const FourTokens &f) {
        const int i = base + 4 * (tid & 63);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const unsigned at = (unsigned)f.v[c] - (unsigned)lo;
            if (at < (unsigned)size) {
                atomicAdd(&x.word[slot(at)], i >= r.prompt - c ? 1u : 0u);
                atomicOr(&x.seen[at >> 5], 1u << (at & 31u));
            }
        }
    };
    if (first < r.length) {
        FourTokens f = early;
        if (first + 256 > r.length) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (first + 4 * (tid & 63) + c >= r.length) f.v[c] = -1;
        }
        count(first, f);
    }
    for (int base = first + STEP; base < r.length; base += DEEP * STEP) {
        FourTokens now[DEEP];
#pragma unroll
        for (int q = 0; q < DEEP; ++q) now[q] = next[q];
        if (base + DEEP * STEP < r.length) load(base + DEEP * STEP);
#pragma unroll
        for (int q = 0; q < DEEP; ++q)
            if (base + q * STEP < r.length) count(base + q * STEP, now[q]);
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

// A thread's VALUES tokens of the slice, in groups of eight neighbours: value
// j is the slice's token at(j).
template <int THREADS>
__device__ __forceinline__ int token_at(int j) {
    return 8 * ((j >> 3) * THREADS + (int)threadIdx.x) + (j & 7);
}

// What a thread reads of its tokens, in flight while the rules are gathered.
template <typename T, int THREADS, int VALUES>
struct Raw {
    Eight<T> logits[VALUES / 8];
    uint32_t allowed[VALUES / 8];
    __device__ __forceinline__ Raw(const RowRules &r, int lo, int size, const T *in) {
#pragma unroll
        for (int g = 0; g < VALUES / 8; ++g) {
            const int at = token_at<THREADS>(8 * g);
            logits[g] = load8(in + at, size - at);
            allowed[g] = r.allowed && at < size ? r.allowed[(lo + at) >> 3] : 0u;
        }
    }
};

// The adjusted values of the thread's tokens, whose logits start at in; those
// past the slice are -infinity.
template <typename T, int THREADS, int VALUES>
__device__ __forceinline__ void adjusted(const nms_logit_rules &u, const RowRules &r, int64_t row,
                                         const T *in, const Raw<T, THREADS, VALUES> &raw,
                                         RuleSpace<THREADS * VALUES> &x, float *z) {
    uint32_t *word = x.word;
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < VALUES; ++j) z[j] = to_f32(raw.logits[j / 8].v[j % 8]);
    // m is -1 or 0: a or b
    auto select = [](int m, float a, float b) {
        return __uint_as_float((__float_as_uint(a) & (uint32_t)m) |
                               (__float_as_uint(b) & ~(uint32_t)m));
    };
    auto bit_of = [](uint32_t bits, int j) { return (int)(bits << (31 - j)) >> 31; };
    if (r.words) {
        uint32_t seen = 0, listed = 0;
#pragma unroll
        for (int g = 0; g < VALUES / 8; ++g) {
            const int at = g * THREADS + tid;
            seen |= (uint32_t)reinterpret_cast<const uint8_t *>(x.seen)[at] << (8 * g);
            listed |= (uint32_t)reinterpret_cast<const uint8_t *>(x.listed)[at] << (8 * g);
        }
        const uint32_t touched = seen | listed;
        if (touched != 0u) {
            uint32_t left = touched;
            do {
                const int j = __builtin_ctz(left), at = token_at<THREADS>(j);
                left &= left - 1u;
                uint32_t *w = word + slot((unsigned)at);
                *w = __float_as_uint(
                    replaced(u, r, row, to_f32(in[at]), (seen >> j & 1u) != 0u, *w));
            } while (left != 0u);
#pragma unroll
            for (int q = 0; q < VALUES / 4; ++q) {
                float w[4];
                __builtin_memcpy(w, word + slot((unsigned)token_at<THREADS>(4 * q)), 16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    z[4 * q + j] = select(bit_of(touched, 4 * q + j), w[j], z[4 * q + j]);
            }
        }
    }
    if (r.masked) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            z[j] = select(bit_of(raw.allowed[j / 8], j % 8), z[j], NEG_INF);
    }
}

}  // namespace gnms
