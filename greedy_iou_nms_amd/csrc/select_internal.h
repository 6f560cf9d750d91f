// Shared by the selection operators (route.hip, logits.hip, pick.hip) and
// their host side (select_api.cpp): element types, order-preserving keys and
// wave reductions.
#pragma once

#include <hip/hip_runtime.h>

#include "greedy_nms.h"

namespace gnms {

// ------------------------------------------------------------ element types

using half_t = _Float16;
using bf16_t = __bf16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(half_t v) { return (float)v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return (float)v; }

// One rounding to nearest even, from the float32 value.
template <typename T>
__device__ __forceinline__ T from_f32(float v) { return (T)v; }

constexpr float NEG_INF = -__builtin_inff();

// --------------------------------------------------------------------- keys

// Unsigned key whose order is the order of the float (-0 folded onto +0),
// always above 0 for a finite value or +infinity; 0 for -infinity and NaN,
// which no selection takes.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > NEG_INF)) return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// ---------------------------------------------------------- wave reductions

// Orders this wave's LDS accesses before and after it (LDS executes a wave's
// accesses in order; the fence holds the compiler to that order).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// ----------------------------------------------------------------- launches

struct RouteArgs {
    const void *logits;
    int dtype;
    int64_t tokens;
    int experts;
    int64_t row_stride;
    const float *bias;
    const uint8_t *live;
    nms_route_options opt;
    int32_t *ids;
    float *weights;
    int32_t *counts;
};

struct RouteBackArgs {
    const void *logits;
    int dtype;
    int64_t tokens;
    int experts;
    int64_t row_stride;
    const int32_t *ids;
    const float *grad_weights;
    nms_route_options opt;
    void *grad_logits;
    int64_t grad_stride;
};

hipError_t launch_route(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream);

struct AdjustArgs {
    const void *logits;
    int dtype;
    int64_t rows;
    int vocab;
    int64_t row_stride;
    nms_logit_rules rules;
    void *out;
    int64_t out_stride;
};

struct PickArgs {
    const void *logits;
    int dtype;
    int64_t rows;
    int vocab;
    int64_t row_stride;
    nms_logit_rules rules;
    const float *uniform, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int max_top_k;
    int32_t *ids;
    float *logprobs;
    void *workspace;
};

hipError_t launch_adjust(const AdjustArgs &a, hipStream_t stream);
size_t pick_workspace_bytes(int64_t rows, int vocab, int max_top_k);
hipError_t launch_pick(const PickArgs &a, hipStream_t stream);

}  // namespace gnms
