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

// One step of a reduction over the wave in DPP moves: every lane combines
// with a lane before it, in six steps lane 63 has combined with all.  `none`
// is the value that changes nothing.
#define GNMS_DPP_STEPS(STEP) STEP(0x111, 0xf) STEP(0x112, 0xf) STEP(0x114, 0xf) \
    STEP(0x118, 0xf) STEP(0x142, 0xa) STEP(0x143, 0xc)

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int none, int v) {
    return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float v) {
    return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(none), __float_as_uint(v)));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double none, double v) {
    const uint64_t n = (uint64_t)__double_as_longlong(none), x = (uint64_t)__double_as_longlong(v);
    const uint64_t lo = dpp<CTRL, ROWS>((uint32_t)n, (uint32_t)x);
    const uint64_t hi = dpp<CTRL, ROWS>((uint32_t)(n >> 32), (uint32_t)(x >> 32));
    return __longlong_as_double((long long)(hi << 32 | lo));
}

__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }
__device__ __forceinline__ float last_lane(float v) {
    return __uint_as_float(last_lane(__float_as_uint(v)));
}
__device__ __forceinline__ double last_lane(double v) {
    const uint64_t x = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)last_lane((uint32_t)(x >> 32)) << 32 |
                                            last_lane((uint32_t)x)));
}

// Inclusive sums over the lanes.
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
#define GNMS_STEP(CTRL, ROWS) v += dpp<CTRL, ROWS>((V)0, v);
    GNMS_DPP_STEPS(GNMS_STEP)
#undef GNMS_STEP
    return v;
}

// The reductions' results are the same in every lane.
template <typename V>
__device__ __forceinline__ V wave_sum(V v) { return last_lane(wave_scan(v)); }

// The order of floats as that of signed integers (and back): integer steps
// are one instruction each, where every float maximum costs two more that
// quieten its inputs.  No NaN.
__device__ __forceinline__ int ordered(float v) {
    const int i = __float_as_int(v);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

__device__ __forceinline__ int wave_max(int v) {
#define GNMS_STEP(CTRL, ROWS) v = max(v, dpp<CTRL, ROWS>((int)0x80000000, v));
    GNMS_DPP_STEPS(GNMS_STEP)
#undef GNMS_STEP
    return last_lane(v);
}
__device__ __forceinline__ int wave_min(int v) {
#define GNMS_STEP(CTRL, ROWS) v = min(v, dpp<CTRL, ROWS>(0x7fffffff, v));
    GNMS_DPP_STEPS(GNMS_STEP)
#undef GNMS_STEP
    return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) { return unordered(wave_max(ordered(v))); }
__device__ __forceinline__ float wave_min(float v) { return unordered(wave_min(ordered(v))); }

// ------------------------------------------------- reductions within a wave

// A DPP move that reaches every lane (permutations and mirrors within 16
// lanes), which the compiler can make part of the instruction that uses it.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ int moved(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __int_as_float(moved<CTRL>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const uint64_t x = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)moved<CTRL>((uint32_t)(x >> 32)) << 32 |
                                            moved<CTRL>((uint32_t)x)));
}

constexpr int XOR1 = 0xB1, XOR2 = 0x4E;            // quads permuted
constexpr int MIRROR8 = 0x141, MIRROR16 = 0x140;   // lanes in reverse order
constexpr int ROTATE = 0x120;                      // + n: by n lanes within 16

// Combines with every lane of the aligned N lanes; the result is in all of
// them.  Mirrors serve as butterfly steps once the halves agree.
template <int N, typename V, typename F>
__device__ __forceinline__ V all_lanes(V v, F f) {
    if (N >= 2) v = f(v, moved<XOR1>(v));
    if (N >= 4) v = f(v, moved<XOR2>(v));
    if (N >= 8) v = f(v, moved<MIRROR8>(v));
    if (N >= 16) v = f(v, moved<MIRROR16>(v));
    if (N >= 32) v = f(v, __shfl_xor(v, 16));
    if (N >= 64) v = f(v, __shfl_xor(v, 32));
    return v;
}
template <int N, typename V>
__device__ __forceinline__ V all_max(V v) {
    return all_lanes<N>(v, [](V a, V b) { return a > b ? a : b; });
}
template <int N, typename V>
__device__ __forceinline__ V all_min(V v) {
    return all_lanes<N>(v, [](V a, V b) { return a < b ? a : b; });
}
template <int N, typename V>
__device__ __forceinline__ V all_sum(V v) {
    return all_lanes<N>(v, [](V a, V b) { return a + b; });
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
