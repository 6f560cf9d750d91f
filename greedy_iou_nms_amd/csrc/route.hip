// Routing of tokens to experts, and its gradient.
//
// Forward.  s = softmax(z) or sigmoid(z), c = s + bias; an expert whose logit
// or c is NaN or -infinity cannot be chosen.  With groups, the kept groups are
// those with the largest sums of their best one or two c.  The chosen experts
// come in descending c (in descending z where there is no bias), ties to the
// lower index.  The choice is a comparison of real numbers, made as in
// binary64: of 16384 tokens with 256 experts about one has two candidates
// closer than a float32 sigmoid's error.
//
// Two forms.  quick_kernel makes the choice on 32-bit keys, 22 bits of the
// value's distance from the token's largest and 10 bits of the index, so that
// a comparison, a sort step and a maximum over lanes are one or two
// instructions each.  It knows how far a key may be off; where candidates or
// groups are closer than that (in about one token of 500, where scores have no
// ties), it orders these few from binary64 scores.  exact_kernel does all in
// binary64, a wave per token, for shapes that the first form does not hold.
#include "select_internal.h"

namespace gnms {
namespace {

constexpr int RT = 256;  // threads per workgroup
constexpr int RWAVES = RT / 64;
constexpr double LOWEST = -__builtin_inf();

// ---------------------------------------- reductions over 4 .. 64 lanes

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

// ------------------------------------------------------------ exact scores

// exp(x) to 2^-40 of its value: 2^n from the exponent, a Taylor polynomial of
// degree 11 on [-ln 2 / 2, ln 2 / 2] (its remainder is below
// 0.3466^12 / 12! = 6e-15).  The library's exp takes four times as many
// instructions for the last 12 bits, which no float32 weight shows.
__device__ __forceinline__ double exp_of(double x) {
    x = fmin(fmax(x, -800.0), 800.0);
    const double n = rint(x * 1.4426950408889634);
    double f = __builtin_fma(n, -0.6931471805599453, x);
    f = __builtin_fma(n, -2.3190468138462996e-17, f);
    double p = 1.0 / 39916800;
    p = __builtin_fma(p, f, 1.0 / 3628800);
    p = __builtin_fma(p, f, 1.0 / 362880);
    p = __builtin_fma(p, f, 1.0 / 40320);
    p = __builtin_fma(p, f, 1.0 / 5040);
    p = __builtin_fma(p, f, 1.0 / 720);
    p = __builtin_fma(p, f, 1.0 / 120);
    p = __builtin_fma(p, f, 1.0 / 24);
    p = __builtin_fma(p, f, 1.0 / 6);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / x for x from 1e-290, to 2^-50; 0 from 1e300 on.
__device__ __forceinline__ double inverse_of(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    return x < 1.0e300 ? r : 0.0;
}

// exp(z - top), 1 at z = top (infinite ones too); no branches.
template <typename EXP>
__device__ __forceinline__ double exp_below(float z, float top, EXP e) {
    const double d = (double)z - (double)top;
    return e(z == top ? 0.0 : d);
}

// ------------------------------------------------- one token, in binary64

// What a wave needs of LDS for it.
struct ExactSpace {
    double c[NMS_ROUTE_MAX_EXPERTS];
    uint8_t kept[NMS_ROUTE_MAX_EXPERTS];
};

// The largest value above -infinity that the lanes know, and the lowest place
// that has it; place -1 if there is none.
__device__ __forceinline__ void wave_best(double &v, int &at) {
#pragma unroll 1
    for (int d = 32; d > 0; d >>= 1) {
        const double v2 = __shfl_xor(v, d);
        const int at2 = __shfl_xor(at, d);
        if (at2 >= 0 && (at < 0 || v2 > v || (v2 == v && at2 < at))) {
            v = v2;
            at = at2;
        }
    }
}

// Chooses the experts of token t: lane i gets the i-th one's index, or -1.
// Every loop is over LDS and rolled, so that it takes few registers.
template <typename T>
__device__ __forceinline__ int exact_token(const RouteArgs &a, int64_t t, ExactSpace &x) {
    const int lane = threadIdx.x & 63;
    const int E = a.experts, G = a.opt.groups, size = E / G;
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX;
    float top = NEG_INF;
    double sum = 0.0;
    wave_fence();
    if (softmax) {
#pragma unroll 1
        for (int e = lane; e < E; e += 64) top = fmaxf(top, to_f32(row[e]));
        top = wave_max(top > NEG_INF ? top : NEG_INF);
#pragma unroll 1
        for (int e = lane; e < E; e += 64) {
            const float z = to_f32(row[e]);
            if (z > NEG_INF) sum += exp_below(z, top, [](double v) { return exp(v); });
        }
        sum = wave_sum(sum);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
        const float z = to_f32(row[e]);
        double c = LOWEST;
        if (z > NEG_INF) {
            c = softmax ? exp_below(z, top, [](double v) { return exp(v); }) / sum
                        : 1.0 / (1.0 + exp(-(double)z));
            if (a.bias != nullptr) c += (double)a.bias[e];
            if (!(c > LOWEST)) c = LOWEST;
        }
        x.c[e] = c;
    }
    if (G > 1) {
#pragma unroll 1
        for (int g = lane; g < G; g += 64) x.kept[g] = 0;
        wave_fence();
#pragma unroll 1
        for (int i = 0; i < a.opt.kept_groups; ++i) {
            // the groups' scores anew each time: nothing is kept of them
            double v = LOWEST;
            int at = -1;
#pragma unroll 1
            for (int g = lane; g < G; g += 64) {
                double b0 = LOWEST, b1 = LOWEST;
#pragma unroll 1
                for (int j = 0; j < size; ++j) {
                    const double w = x.c[g * size + j];
                    b1 = w > b0 ? b0 : w > b1 ? w : b1;
                    b0 = w > b0 ? w : b0;
                }
                if (a.opt.group_top == 2 && b1 > LOWEST) b0 += b1;
                if (x.kept[g] == 0 && b0 > v) {
                    v = b0;
                    at = g;
                }
            }
            wave_best(v, at);
            if (at < 0) break;
            if (lane == 0) x.kept[at] = 1;
            wave_fence();
        }
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (x.kept[e / size] == 0) x.c[e] = LOWEST;
    }
    // without a bias the order is the logits'
    if (a.bias == nullptr) {
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (x.c[e] > LOWEST) x.c[e] = (double)to_f32(row[e]);
    }
    int mine = -1;
#pragma unroll 1
    for (int i = 0; i < a.opt.top_k; ++i) {
        double v = LOWEST;
        int at = -1;
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (x.c[e] > v) {
                v = x.c[e];
                at = e;
            }
        wave_best(v, at);
        if (at < 0) break;
        if (lane == (at & 63)) x.c[at] = LOWEST;
        if (lane == i) mine = at;
    }
    wave_fence();
    return mine;
}

// The weights of a token's chosen experts and what is written of them.  The
// token's LANES lanes call it together; lane i has the i-th expert (or -1).
// sum: of exp(z - top) over the whole row where the softmax needs it.
template <typename T, int LANES>
__device__ __forceinline__ void write_token(const RouteArgs &a, int64_t t, bool write, int place,
                                            int id, float top, double sum) {
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    const float z = id >= 0 ? to_f32(row[id]) : NEG_INF;
    const auto e = [](double v) { return exp_of(v); };
    double w = 0.0;
    if (a.opt.score == NMS_ROUTE_SOFTMAX) {
        // renormalised: the softmax over the chosen logits, the same quotient,
        // which holds where every chosen probability is below binary64's range
        if (a.opt.renormalise) top = unordered(all_max<LANES>(ordered(z)));
        w = id >= 0 ? exp_below(z, top, e) : 0.0;
        if (a.opt.renormalise) sum = all_sum<LANES>(w);
    } else {
        w = id >= 0 ? 1.0 / (1.0 + e(-(double)z)) : 0.0;
        sum = a.opt.renormalise ? all_sum<LANES>(w) : 1.0;
    }
    // a quotient where the inverse is out of range, and only there: the other
    // tokens of the wave must not round differently for it
    const bool in_range = sum > 1.0e-290;
    double share = in_range ? w * inverse_of(sum) : 0.0;
    if (__builtin_expect(!in_range && sum > 0.0, 0)) share = w / sum;
    w = share;
    if (write && place < a.opt.top_k) {
        a.ids[t * a.opt.top_k + place] = id;
        a.weights[t * a.opt.top_k + place] = (float)(w * (double)a.opt.scale);
    }
}

// The softmax sum of a row by the whole wave.
template <typename T>
__device__ __forceinline__ void row_sum(const RouteArgs &a, int64_t t, float &top, double &sum) {
    const int lane = threadIdx.x & 63;
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    top = NEG_INF;
    sum = 0.0;
    for (int e = lane; e < a.experts; e += 64) top = fmaxf(top, to_f32(row[e]));
    top = wave_max(top > NEG_INF ? top : NEG_INF);
    for (int e = lane; e < a.experts; e += 64) {
        const float z = to_f32(row[e]);
        if (z > NEG_INF) sum += exp_below(z, top, [](double v) { return exp_of(v); });
    }
    sum = wave_sum(sum);
}

// The first workgroup clears the counts, which count_kernel adds to.
__device__ __forceinline__ void clear_counts(const RouteArgs &a) {
    if (a.counts != nullptr && blockIdx.x == 0)
        for (int e = threadIdx.x; e < a.experts; e += RT) a.counts[e] = 0;
}

// Or, where the launch is one workgroup, counts the experts of all tokens,
// whose ids it has written itself.
__device__ __forceinline__ void count_here(const RouteArgs &a) {
    __syncthreads();
    const int n = (int)a.tokens * a.opt.top_k;
    for (int i = threadIdx.x; i < n; i += RT) {
        const int id = a.ids[i];
        if (id >= 0) atomicAdd(a.counts + id, 1);
    }
}

template <typename T>
__global__ __launch_bounds__(RT) void exact_kernel(RouteArgs a) {
    __shared__ ExactSpace space[RWAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * RWAVES + wave;
    clear_counts(a);
    if (t >= a.tokens) return;  // no barrier follows
    const bool live = a.live == nullptr || a.live[t] != 0;
    const int id = live ? exact_token<T>(a, t, space[wave]) : -1;
    float top = 0.0f;
    double sum = 1.0;
    if (a.opt.score == NMS_ROUTE_SOFTMAX && !a.opt.renormalise) row_sum<T>(a, t, top, sum);
    write_token<T, 64>(a, t, true, lane, id, top, sum);
}

// -------------------------------------------------------------- quick form

// Batcher's merge exchange, descending.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t *key) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

constexpr uint32_t INDEX_BITS = 10, INDEX_MASK = (1u << INDEX_BITS) - 1u;
constexpr uint32_t Q_TOP = (1u << 22) - 1u;
static_assert(NMS_ROUTE_MAX_EXPERTS <= (int)INDEX_MASK + 1, "an index fits its field");

__device__ __forceinline__ uint32_t with_index(uint32_t q, int e) {
    return q << INDEX_BITS | (INDEX_MASK - (uint32_t)e);
}

// A whole number from a float at most Q_TOP; 0 below 1 and for a NaN, as
// v_cvt_u32_f32 gives (C leaves it open).
__device__ __forceinline__ uint32_t saturated(float q) {
    uint32_t r;
    asm("v_cvt_u32_f32 %0, %1" : "=v"(r) : "v"(q));
    return r;
}

// The 16-bit types' order in 16 bits (-0 folded onto +0), 0 for -infinity and
// NaN.
template <typename T>
__device__ __forceinline__ uint32_t short_key(T v) {
    uint16_t u;
    __builtin_memcpy(&u, &v, 2);
    if (u == 0x8000u) u = 0;
    const uint32_t k = (u & 0x8000u) ? (uint16_t)~u : (uint32_t)(u | 0x8000u);
    return to_f32(v) > NEG_INF ? k : 0u;
}

// The score of one expert of a token as binary64 has it: to the last places,
// or groups whose sums are equal, as 1 / (1 + exp(-z)) + 1 / (1 + exp(z)) is for
// every z, would come in the order of the errors.  (16384 tokens of 256 experts
// take the same 9.6 us with exp_of, and 34 if all their scores are equal; a
// sigmoid is above 0 down to -709.78, where inverse_of is out of range.)
__device__ __forceinline__ double exact_score(bool softmax, float z, float top, double share,
                                              float bias) {
    const double s = softmax ? exp_below(z, top, [](double v) { return exp(v); }) * share
                             : 1.0 / (1.0 + exp(-(double)z));
    return s + (double)bias;
}

// The choice of quick_kernel for a wave's tokens, from binary64 scores: lane i
// of a token gets its i-th expert, or -1.  z: the lane's logits, -infinity where
// there is none; bias: the lane's, or 0.
template <int LANES, int VALUES>
__device__ __forceinline__ int choose_exactly(const RouteArgs &a, const float *z,
                                              const float *bias, float top, double sum,
                                              int e0, int group_lanes) {
    const int lane = threadIdx.x & 63, sub = lane % LANES;
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX, biased = a.bias != nullptr;
    const double share = inverse_of(sum);
    double r[VALUES];  // what the experts are ordered by
    double b0 = LOWEST, b1 = LOWEST;
#pragma unroll
    for (int j = 0; j < VALUES; ++j) {
        double c = exact_score(softmax, z[j], top, share, bias[j]);
        if (!(z[j] > NEG_INF && c > LOWEST)) c = LOWEST;
        b1 = c > b0 ? b0 : c > b1 ? c : b1;
        b0 = c > b0 ? c : b0;
        r[j] = biased || c == LOWEST ? c : (double)z[j];
    }
    if (a.opt.groups > 1) {
        auto merge = [&](double o0, double o1) {
            b1 = fmax(fmin(b0, o0), fmax(b1, o1));
            b0 = fmax(b0, o0);
        };
        if (group_lanes >= 2) merge(moved<XOR1>(b0), moved<XOR1>(b1));
        if (group_lanes >= 4) merge(moved<XOR2>(b0), moved<XOR2>(b1));
        if (group_lanes >= 8) merge(moved<MIRROR8>(b0), moved<MIRROR8>(b1));
        if (group_lanes >= 16) merge(moved<MIRROR16>(b0), moved<MIRROR16>(b1));
        if (group_lanes >= 32) merge(__shfl_xor(b0, 16), __shfl_xor(b1, 16));
        const double score = a.opt.group_top == 2 && b1 > LOWEST ? b0 + b1 : b0;
        int before = 0;
        for (int o = group_lanes; o < LANES; o += group_lanes) {
            const int from = (sub + o) % LANES;
            const double other = __shfl(score, lane - sub + from);
            before += other > score || (other == score && from < sub) ? 1 : 0;
        }
        if (before >= a.opt.kept_groups) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) r[j] = LOWEST;
        }
    }
    int mine = -1;
#pragma unroll 1
    for (int i = 0; i < a.opt.top_k; ++i) {
        double v = r[0];
        int at = e0;
#pragma unroll
        for (int j = 1; j < VALUES; ++j)
            if (r[j] > v) {
                v = r[j];
                at = e0 + j;
            }
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) {
            const double v2 = __shfl_xor(v, d);
            const int at2 = __shfl_xor(at, d);
            const bool take = v2 > v || (v2 == v && at2 < at);
            v = take ? v2 : v;
            at = take ? at2 : at;
        }
        if (sub == i && v > LOWEST) mine = at;
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            if (v > LOWEST && r[j] == v && at == e0 + j) r[j] = LOWEST;
    }
    return mine;
}

// LANES lanes share a token, VALUES experts each.  A group of experts (all of
// them, where there are none) has group_lanes lanes, a power of two, the last
// of which may have places that are empty.  top_k is at most LANES.
//
// A token's row is read once, in one load per lane, and everything after it
// stays in registers: what bounds a large call is the instructions (Batcher's
// sort per lane, then top_k maxima over the lanes, each of which moves all
// VALUES keys up), and that its 4096 waves are one fill of the GPU, so that
// reading and computing hardly overlap.  16384 tokens of 256 float32 experts in
// 8 groups, top 8: 11 us, 9.6 in a graph, where reading them takes 2.4 at a
// copy's 7.4 TB/s from cache; 5003 of 60 float16 experts, top 4: 4.3 us; a
// decode step of 8 tokens 3.6 us, all of it latency.  16 lanes rather than a
// wave per token leave four tokens' steps to share each instruction.
template <typename T, int LANES, int VALUES>
__global__ __launch_bounds__(RT, 4) void quick_kernel(RouteArgs a, int group_lanes) {
    constexpr int TOKENS = 64 / LANES;  // per wave
    const int lane = threadIdx.x & 63, sub = lane % LANES;
    const int64_t t = ((int64_t)blockIdx.x * RWAVES + (threadIdx.x >> 6)) * TOKENS + lane / LANES;
    const bool inside = t < a.tokens;
    const int64_t tok = inside ? t : a.tokens - 1;
    const bool live = inside && (a.live == nullptr || a.live[tok] != 0);
    const int E = a.experts, k = a.opt.top_k, size = E / a.opt.groups;
    // the lane's experts: e0 .. limit - 1, at most VALUES of them
    const int g = sub / group_lanes, e0 = g * size + sub % group_lanes * VALUES;
    const int limit = g < a.opt.groups ? (g + 1) * size : 0;
    const T *row = static_cast<const T *>(a.logits) + tok * a.row_stride;
    clear_counts(a);

    // the lane's logits, -infinity in empty places
    T raw[VALUES];
    if (e0 + VALUES <= limit) {
        __builtin_memcpy(raw, row + e0, sizeof(raw));
    } else {
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            raw[j] = e0 + j < limit ? row[e0 + j] : from_f32<T>(NEG_INF);
    }
    float z[VALUES], top = NEG_INF;
#pragma unroll
    for (int j = 0; j < VALUES; ++j) z[j] = to_f32(raw[j]);
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX;
    const bool grouped = a.opt.groups > 1, scored = a.bias != nullptr || grouped;
    const bool whole = softmax && (scored || !a.opt.renormalise);
    // the largest logit, where scores or keys are relative to it
    const bool relative = whole || (!scored && sizeof(T) == 4);
    if (relative) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            z[j] = z[j] > NEG_INF ? z[j] : NEG_INF;
            top = fmaxf(top, z[j]);
        }
        top = unordered(all_max<LANES>(ordered(top)));
    }

    // the softmax sum, which the weights need to 2^-24 and better
    double sum = 1.0;
    if (whole) {
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            sum += exp_below(z[j], top, [](double v) { return exp_of(v); });
        sum = all_sum<LANES>(sum);
    }

    // Keys.  margin: two candidates whose q differ by no more may be in either
    // order, unless they are equal; negative: the keys are exact.
    uint32_t key[VALUES];
    float bias[VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) bias[j] = 0.0f;
    int margin = 0;
    bool bad = false;  // the token has to be chosen exactly
    if (scored) {
        // c in float32: a sigmoid or a softmax share is off by less than
        // 3 * 2^-23, and its sum with a bias by |c| 2^-24 more; the scale is
        // 2^22, and q is rounded twice
        if (a.bias != nullptr) {
            if (e0 + VALUES <= limit) {
                __builtin_memcpy(bias, a.bias + e0, sizeof(bias));
            } else {
#pragma unroll
                for (int j = 0; j < VALUES; ++j) bias[j] = e0 + j < limit ? a.bias[e0 + j] : 0.0f;
            }
        }
        float c[VALUES], c_top = NEG_INF;
        if (softmax) {
            const float share = (float)inverse_of(sum);
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                c[j] = __builtin_amdgcn_exp2f((z[j] - top) * 1.44269504f) * share;
        } else {
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                c[j] = __builtin_amdgcn_rcpf(1.0f +
                                             __builtin_amdgcn_exp2f(z[j] * -1.44269504f));
        }
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            c[j] = z[j] > NEG_INF ? c[j] + bias[j] : NEG_INF;
            c_top = fmaxf(c_top, c[j]);
        }
        c_top = unordered(all_max<LANES>(ordered(c_top)));
        bad = !(fabsf(c_top) < 64.0f) || (softmax && !(fabsf(top) < 3.0e38f));
        margin = 8 + (int)fabsf(bad ? 0.0f : c_top);
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            key[j] = with_index(saturated(__builtin_fmaf(c[j] - c_top, 4194304.0f, (float)Q_TOP)),
                                e0 + j);
        if (c_top == NEG_INF) bad = false;
    } else if (sizeof(T) == 2) {
        margin = -1;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            key[j] = with_index(short_key(raw[j]), e0 + j);
        }
    } else {
        // z down to 64 below the top, monotone: only equal q are open
        bad = !(fabsf(top) < 3.0e38f) && top != NEG_INF;
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            key[j] = with_index(saturated(__builtin_fmaf(z[j] - top, 65536.0f, (float)Q_TOP)),
                                e0 + j);
    }
    sort_keys<VALUES>(key);

    if (grouped) {
        // The best two of each group, over its lanes; then how many groups
        // have a larger sum, equal ones ordered by their number.
        uint32_t b0 = key[0], b1 = VALUES > 1 ? key[VALUES > 1 ? 1 : 0] : 0u;
        auto merge = [&](uint32_t o0, uint32_t o1) {
            b1 = max(min(b0, o0), max(b1, o1));
            b0 = max(b0, o0);
        };
        if (group_lanes >= 2) merge(moved<XOR1>(b0), moved<XOR1>(b1));
        if (group_lanes >= 4) merge(moved<XOR2>(b0), moved<XOR2>(b1));
        if (group_lanes >= 8) merge(moved<MIRROR8>(b0), moved<MIRROR8>(b1));
        if (group_lanes >= 16) merge(moved<MIRROR16>(b0), moved<MIRROR16>(b1));
        if (group_lanes >= 32) merge(__shfl_xor(b0, 16), __shfl_xor(b1, 16));
        const bool group = g < a.opt.groups;
        const bool two = a.opt.group_top == 2;
        const uint32_t q0 = b0 >> INDEX_BITS, q1 = b1 >> INDEX_BITS;
        // a group with one expert where others sum two, or one that reaches
        // the keys' end
        if (group && two && q0 != 0u && q1 == 0u) bad = true;
        const uint32_t score = group ? q0 + (two ? q1 : 0u) : 0u;
        const uint32_t ranked = score << 6 | (uint32_t)(63 - g);
        int larger = 0;
        if (LANES == 16) {
#define GNMS_ROTATE(N) \
    if (((N) & (group_lanes - 1)) == 0) larger += moved<ROTATE + N>(ranked) > ranked ? 1 : 0;
            GNMS_ROTATE(1) GNMS_ROTATE(2) GNMS_ROTATE(3) GNMS_ROTATE(4) GNMS_ROTATE(5)
            GNMS_ROTATE(6) GNMS_ROTATE(7) GNMS_ROTATE(8) GNMS_ROTATE(9) GNMS_ROTATE(10)
            GNMS_ROTATE(11) GNMS_ROTATE(12) GNMS_ROTATE(13) GNMS_ROTATE(14) GNMS_ROTATE(15)
#undef GNMS_ROTATE
        } else {
            for (int o = group_lanes; o < LANES; o += group_lanes)
                larger += __shfl(ranked, (lane + o) & 63) > ranked ? 1 : 0;
        }
        bool kept = score > 0u && larger < a.opt.kept_groups;
        // how close the choice of the groups was
        const uint32_t least = all_min<LANES>(kept ? score : 0xffffffffu);
        const uint32_t most = all_max<LANES>(kept ? 0u : score);
        const bool near_groups = least - most <= (uint32_t)(2 * margin);
        if (__ballot(near_groups) != 0ull) {
            // the groups' sums in binary64; a third expert that may be among
            // a group's best two leaves it to choose_exactly
            const double share = inverse_of(sum);
            auto exact_of = [&](uint32_t m) -> double {
                const int e = (int)(INDEX_MASK - (m & INDEX_MASK));
                if (m <= INDEX_MASK) return LOWEST;
                return exact_score(softmax, to_f32(row[e]), top, share,
                                   a.bias != nullptr ? a.bias[e] : 0.0f);
            };
            const double s0 = exact_of(b0), s1 = two ? exact_of(b1) : 0.0;
            const double exact = group ? s0 + s1 : LOWEST;
            bool third = false;
            const uint32_t lowest = (two ? q1 : q0) - min(two ? q1 : q0, (uint32_t)margin);
#pragma unroll
            for (int j = 0; j < 3 && j < VALUES; ++j)
                third |= key[j] != b0 && !(two && key[j] == b1) &&
                         (key[j] >> INDEX_BITS) >= lowest && lowest > 0u;
            int before = 0;
            for (int o = group_lanes; o < LANES; o += group_lanes) {
                const int from = (sub + o) % LANES;
                const double other = __shfl(exact, lane - sub + from);
                before += other > exact || (other == exact && from < sub) ? 1 : 0;
            }
            if (near_groups) {
                kept = score > 0u && before < a.opt.kept_groups;
                if (group && (third || lowest == 0u)) bad = true;
            }
        }
        if (!kept) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) key[j] = 0u;
        }
    }

    // The largest key of all lanes, top_k times; the lane that has it moves
    // its next one up.  Keys without a value are below 2^INDEX_BITS.
    uint32_t mine = 0u, last = 0u;
    bool close = false;
    auto next = [&]() -> uint32_t {
        const uint32_t m = all_max<LANES>(key[0]);
        if (key[0] == m) {
#pragma unroll
            for (int j = 0; j + 1 < VALUES; ++j) key[j] = key[j + 1];
            key[VALUES - 1] = 0u;
        }
        return m <= INDEX_MASK ? 0u : m;
    };
    // whether m, which comes after last, may belong before it
    auto near_last = [&](uint32_t m) {
        return m != 0u && (int)((last >> INDEX_BITS) - (m >> INDEX_BITS)) <= margin;
    };
    for (int i = 0; i < k; ++i) {
        const uint32_t m = next();
        close |= i > 0 && near_last(m);
        if (sub == i) mine = m;
        last = m;
    }
    // those that may belong among them: near the last, or near one that is
    int candidates = k;
    if (margin >= 0) {
        uint32_t m = next();
        bool open = near_last(m);
        while (__ballot(open) != 0ull) {
            if (open) {
                close = true;
                if (candidates == LANES) bad = true;  // no lane to hold it
                else if (sub == candidates) mine = m;
                candidates = min(candidates + 1, LANES);
                last = m;
            }
            m = next();
            open = open && !bad && near_last(m);
        }
    }
    // Nothing left, or nearly at the keys' end: there is no further eligible
    // expert, or one below what keys reach.
    const bool at_end = margin >= 0 && (int)(last >> INDEX_BITS) <= margin;
    if (__ballot(at_end) != 0ull) {
        bool low = false;
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            low |= z[j] > NEG_INF && bias[j] > NEG_INF;
        if (at_end && low) bad = true;
    }
    int id = mine != 0u ? (int)(INDEX_MASK - (mine & INDEX_MASK)) : -1;
    if (margin >= 0 && __ballot(close) != 0ull) {
        // the candidates' order in binary64, equal ones by their index
        const int e = mine != 0u ? id : INDEX_MASK + 1 + sub;
        double v = LOWEST;
        if (mine != 0u) {
            const float ze = to_f32(row[e]);
            v = a.bias != nullptr
                    ? exact_score(softmax, ze, top, inverse_of(sum), a.bias[e])
                    : (double)ze;
        }
        int before = 0;
        for (int o = 0; o < LANES; ++o) {
            const double other = __shfl(v, lane - sub + o);
            const int other_e = __shfl(e, lane - sub + o);
            before += other > v || (other == v && other_e < e) ? 1 : 0;
        }
        // every lane's place is another's
        const int sorted = __builtin_amdgcn_ds_permute((lane - sub + before) * 4, e);
        if (close) id = sorted <= (int)INDEX_MASK ? sorted : -1;
    }
    if (sub >= k) id = -1;
    if (margin >= 0) bad = all_max<LANES>((int)(live && bad)) != 0;  // any lane of the token
    else bad = false;
    if (__ballot(bad) != 0ull) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = z[j] > NEG_INF ? z[j] : NEG_INF;
        const int exact = choose_exactly<LANES, VALUES>(a, z, bias, top, sum, e0, group_lanes);
        if (bad) id = exact;
    }
    write_token<T, LANES>(a, tok, inside, sub, live ? id : -1, top, sum);
    if (a.counts != nullptr && gridDim.x == 1) count_here(a);
}

// Adds the experts of ids[0..n) to the counts; a single workgroup writes them.
// A launch of its own: 2 to 4 us on the GPU behind quick_kernel (131072 ids of
// 256 experts 2.7 us) and 3.3 us of the caller's time.  Routing all tokens in
// one workgroup that counts them itself saves 2.5 us of an eager call of 64
// tokens and 64 experts, but takes 6.2 us in a graph where the two launches
// take 4.9, and 20 for 7 at 128 tokens of 256 experts.
constexpr int CT = 1024, COUNTED = 4096;  // threads; ids per workgroup
__global__ __launch_bounds__(CT) void count_kernel(const int32_t *ids, int64_t n, int experts,
                                                   int32_t *counts) {
    __shared__ int32_t hist[NMS_ROUTE_MAX_EXPERTS];
    hist[threadIdx.x] = 0;
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * (4 * CT);
    for (int64_t i = 4 * ((int64_t)blockIdx.x * CT + threadIdx.x); i < n; i += step) {
        int id[4];
        if (i + 4 <= n) {
            __builtin_memcpy(id, ids + i, sizeof(id));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) id[j] = i + j < n ? ids[i + j] : -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (id[j] >= 0) atomicAdd(&hist[id[j]], 1);
    }
    __syncthreads();
    const int e = threadIdx.x, c = hist[e];
    if (e < experts) {
        if (gridDim.x == 1) counts[e] = c;
        else if (c != 0) atomicAdd(&counts[e], c);
    }
}
static_assert(CT == NMS_ROUTE_MAX_EXPERTS, "a thread per expert");

// ---------------------------------------------------------------- gradient

// Gradient of the weights in the logits, given the chosen experts.
//   softmax, not renormalised  w_i = scale p_i:
//       dz_j = p_j (scale g_j [j chosen] - sum_i scale g_i p_i)
//   softmax, renormalised      q = softmax over the chosen logits, w = scale q:
//       dz_j = q_j scale (g_j - sum_i g_i q_i), 0 for the others
//   sigmoid                    w_i = scale s_i / D, D = 1 or sum of chosen s:
//       dz_j = scale (g_j - [renormalised] sum_i g_i s_i / D) / D s_j (1 - s_j)
// Only the first needs the whole row.  LANES lanes share a token, VALUES
// experts each; the chosen experts' terms go to their places through LDS, all
// at once, or one after another where an index comes twice, so that it adds up
// in a fixed order.  32768 tokens of 128 bfloat16 experts, plain softmax: 7.2
// us (renormalised 5.6, in a graph), of which 3.8 are instructions (283 per wave
// of four tokens; every lane has places for 64 / LANES chosen experts, whatever
// top_k is) and 2.6 would be the reading and writing alone (19 MB at a copy's
// 7.4 TB/s from cache); one term after another took 8.9, the library's
// exponential 8.7.
template <typename T, int LANES, int VALUES>
__global__ __launch_bounds__(RT) void back_kernel(RouteBackArgs a) {
    constexpr int TOKENS = 64 / LANES;            // per wave
    constexpr int CHOSEN = NMS_ROUTE_MAX_TOP_K / LANES;  // per lane, at most
    __shared__ float place[RWAVES * TOKENS][LANES * VALUES];
    const int lane = threadIdx.x & 63, sub = lane % LANES;
    const int mine = (threadIdx.x >> 6) * TOKENS + lane / LANES;
    const int64_t t = (int64_t)blockIdx.x * (RWAVES * TOKENS) + mine;
    const bool inside = t < a.tokens;
    const int64_t tok = inside ? t : a.tokens - 1;
    const int E = a.experts, k = a.opt.top_k, e0 = sub * VALUES;
    const T *row = static_cast<const T *>(a.logits) + tok * a.row_stride;
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX;
    const bool whole = softmax && !a.opt.renormalise;

    float z[VALUES];
    if (whole) {
        T raw[VALUES];
        if (e0 + VALUES <= E) {
            __builtin_memcpy(raw, row + e0, sizeof(raw));
        } else {
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                raw[j] = e0 + j < E ? row[e0 + j] : from_f32<T>(NEG_INF);
        }
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = to_f32(raw[j]);
    }
    int id[CHOSEN];
    float g[CHOSEN], zc[CHOSEN];
#pragma unroll
    for (int q = 0; q < CHOSEN; ++q) {
        const int i = q * LANES + sub;
        id[q] = -1;
        g[q] = 0.0f;
        zc[q] = NEG_INF;
        if (i < k) {
            const int e = a.ids[tok * k + i];
            if ((unsigned)e < (unsigned)E) {
                id[q] = e;
                g[q] = a.grad_weights[tok * k + i] * a.opt.scale;
                const float v = to_f32(row[e]);
                zc[q] = v > NEG_INF ? v : NEG_INF;
            }
        }
    }
    // LDS executes a wave's accesses in order
#pragma unroll
    for (int j = 0; j < VALUES; ++j) place[mine][e0 + j] = 0.0f;

    // exp(v - top) by the exponential instruction: the product with log2 e is
    // rounded to 2^-24 of itself, as the difference is
    constexpr float LOG2E = 1.44269504f;
    const auto share = [](float v, float top) {
        return v == top ? 1.0f : __builtin_amdgcn_exp2f((v - top) * LOG2E);
    };
    float top = NEG_INF, total = 0.0f, inner = 0.0f, s[CHOSEN], d[CHOSEN];
    if (softmax) {
        if (whole) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) top = fmaxf(top, z[j]);
        } else {
#pragma unroll
            for (int q = 0; q < CHOSEN; ++q) top = fmaxf(top, zc[q]);
        }
        top = unordered(all_max<LANES>(ordered(top)));
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q) s[q] = zc[q] == NEG_INF ? 0.0f : share(zc[q], top);
        if (whole) {
            // a NaN or an infinite top shows in the sum, which is 1 at least
            // else; then every term is looked at
            const float base = fabsf(top) < __builtin_inff() ? top : 0.0f;
            float p[VALUES];
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                p[j] = __builtin_amdgcn_exp2f((z[j] - base) * LOG2E);
                total += p[j];
            }
            total = all_sum<LANES>(total);
            if (__ballot(!(total < 3.0e38f)) != 0ull) {
                total = 0.0f;
#pragma unroll
                for (int j = 0; j < VALUES; ++j) {
                    p[j] = z[j] > NEG_INF ? share(z[j], top) : 0.0f;
                    total += p[j];
                }
                total = all_sum<LANES>(total);
            }
#pragma unroll
            for (int j = 0; j < VALUES; ++j) z[j] = p[j];
        } else {
#pragma unroll
            for (int q = 0; q < CHOSEN; ++q) total += s[q];
            total = all_sum<LANES>(total);
        }
        const float inverse = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q) {
            s[q] *= inverse;
            inner += g[q] * s[q];
        }
        inner = all_sum<LANES>(inner);
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q) d[q] = whole ? g[q] : s[q] * (g[q] - inner);
        if (whole) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) z[j] *= inverse;
        }
    } else {
        // shares of the chosen scores' sum, each score divided by exp(m) first,
        // m = min(largest chosen logit, 0): below -88 a score itself is under
        // float32's range, its share and its gradient are not.  From -709.78
        // down a score is 0 in binary64 too, and so are the forward's weights.
        float m = 0.0f;
        if (a.opt.renormalise) {
#pragma unroll
            for (int q = 0; q < CHOSEN; ++q) top = fmaxf(top, zc[q]);
            m = fminf(unordered(all_max<LANES>(ordered(top))), 0.0f);
        }
        float weighted = 0.0f, rest[CHOSEN];  // rest: 1 - score
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q) {
            rest[q] = 1.0f / (1.0f + expf(zc[q]));
            s[q] = zc[q] <= -709.78271f ? 0.0f
                   : zc[q] > 0.0f       ? 1.0f / (1.0f + expf(-zc[q]))
                                        : expf(zc[q] - m) * rest[q];
            total += s[q];
            weighted += g[q] * s[q];
        }
        if (a.opt.renormalise) {
            total = all_sum<LANES>(total);
            weighted = all_sum<LANES>(weighted);
            inner = total > 0.0f ? weighted / total : 0.0f;
        } else {
            total = 1.0f;
        }
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q)
            d[q] = total > 0.0f ? (g[q] - inner) * (s[q] / total) * rest[q] : 0.0f;
    }
    // Every chosen place keeps the number of one term that goes there: where
    // each term finds its own, no index comes twice.
    bool twice = false;
    wave_fence();
#pragma unroll
    for (int q = 0; q < CHOSEN; ++q)
        if (id[q] >= 0) place[mine][id[q]] = (float)(q * LANES + sub);
    wave_fence();
#pragma unroll
    for (int q = 0; q < CHOSEN; ++q)
        if (id[q] >= 0) twice |= place[mine][id[q]] != (float)(q * LANES + sub);
    wave_fence();
    const bool in_turn = __ballot(twice) != 0ull;
#pragma unroll
    for (int q = 0; q < CHOSEN; ++q)
        if (id[q] >= 0) place[mine][id[q]] = in_turn ? 0.0f : d[q];
    if (in_turn) {
#pragma unroll
        for (int q = 0; q < CHOSEN; ++q)
            for (int l = 0; l < LANES && q * LANES + l < k; ++l) {
                wave_fence();
                if (sub == l && id[q] >= 0) place[mine][id[q]] += d[q];
            }
    }
    wave_fence();
    if (!inside) return;
    T out[VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) {
        const float ds = place[mine][e0 + j];
        out[j] = from_f32<T>(whole ? z[j] * (ds - inner) : ds);
    }
    T *to = static_cast<T *>(a.grad_logits) + t * a.grad_stride + e0;
    if (e0 + VALUES <= E) {
        __builtin_memcpy(to, out, sizeof(out));
    } else {
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            if (e0 + j < E) to[j] = out[j];
    }
}

// ----------------------------------------------------------------- launches

// Each returns whether the launch has counted the experts.
template <typename T, int LANES, int VALUES>
bool run_quick(const RouteArgs &a, int group_lanes, hipStream_t stream) {
    constexpr int per = RWAVES * (64 / LANES);
    const unsigned grid = (unsigned)((a.tokens + per - 1) / per);
    quick_kernel<T, LANES, VALUES><<<grid, RT, 0, stream>>>(a, group_lanes);
    return grid == 1;
}

// Whether quick_kernel<., lanes, values> holds the shape, and over how many
// lanes a group lies.
bool holds(const RouteArgs &a, int lanes, int values, int *group_lanes) {
    if (a.experts > lanes * values || a.opt.top_k > lanes) return false;
    *group_lanes = lanes;
    if (a.opt.groups == 1) return true;
    int n = 1;
    while (n * values < a.experts / a.opt.groups) n *= 2;
    *group_lanes = n;
    return a.opt.groups * n <= lanes;
}

// The fewest lanes and places that hold the shape; binary64 throughout where
// groups are more than lanes.  8192 tokens of float32 with top 8, in a graph: 256
// experts 7.0 us, 384 19.5, 512 18.4 and 1024 17.9 (the last three a wave per
// token, 384 with 40 of 64 lanes empty); 512 in 64 groups 35 us; in 512 groups,
// which only exact_kernel holds, 1363 us, and 539 for 128 tokens.
template <typename T>
bool run_route(const RouteArgs &a, hipStream_t stream) {
    int g = 1;
    if (holds(a, 16, 4, &g)) return run_quick<T, 16, 4>(a, g, stream);
    if (holds(a, 16, 8, &g)) return run_quick<T, 16, 8>(a, g, stream);
    if (holds(a, 16, 16, &g)) return run_quick<T, 16, 16>(a, g, stream);
    if (holds(a, 64, 4, &g)) return run_quick<T, 64, 4>(a, g, stream);
    if (holds(a, 64, 16, &g)) return run_quick<T, 64, 16>(a, g, stream);
    exact_kernel<T><<<(unsigned)((a.tokens + RWAVES - 1) / RWAVES), RT, 0, stream>>>(a);
    return false;
}

template <typename T, int LANES, int VALUES>
void run_back(const RouteBackArgs &a, hipStream_t stream) {
    constexpr int per = RWAVES * (64 / LANES);
    back_kernel<T, LANES, VALUES><<<(unsigned)((a.tokens + per - 1) / per), RT, 0, stream>>>(a);
}

// 8192 float32 tokens, top 8, softmax over all: 256 experts 7.1 us, 384 10.8, 512
// 13.2, 1024 20.1.
template <typename T>
void run_back(const RouteBackArgs &a, hipStream_t stream) {
    if (a.experts <= 64) run_back<T, 16, 4>(a, stream);
    else if (a.experts <= 128) run_back<T, 16, 8>(a, stream);
    else if (a.experts <= 256) run_back<T, 16, 16>(a, stream);
    else run_back<T, 64, 16>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    bool counted = false;
    if (a.tokens > 0) {
        if (a.dtype == NMS_F32) counted = run_route<float>(a, stream);
        else if (a.dtype == NMS_F16) counted = run_route<half_t>(a, stream);
        else counted = run_route<bf16_t>(a, stream);
    }
    if (a.counts != nullptr && !counted) {
        const int64_t n = a.tokens * a.opt.top_k, groups = (n + COUNTED - 1) / COUNTED;
        count_kernel<<<(unsigned)(groups < 1 ? 1 : groups > 256 ? 256 : groups), CT, 0, stream>>>(
            a.ids, n, a.experts, a.counts);
    }
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream) {
    if (a.dtype == NMS_F32) run_back<float>(a, stream);
    else if (a.dtype == NMS_F16) run_back<half_t>(a, stream);
    else run_back<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
