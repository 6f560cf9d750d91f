// Routing of tokens to experts, and its gradient.
//
// Forward.  s = softmax(z) or sigmoid(z) in binary64, c = s + bias; an expert
// whose logit or c is NaN or -infinity cannot be chosen.  With groups, the
// kept groups are those with the largest sums of their best one or two c.
// The chosen experts come in descending c (in descending logit when there is
// no bias, which is the same order before rounding), ties to the lower index.
// Binary64 because the choice is a comparison: a float32 sigmoid is off by a
// few 2^-24, and of 16384 tokens with 256 experts about one has two
// candidates closer than that.
#include "select_internal.h"

namespace gnms {
namespace {

constexpr int RT = 256;  // threads per workgroup, one wave per token
constexpr int RWAVES = RT / 64;
constexpr int MAX_VALUES = NMS_ROUTE_MAX_EXPERTS / 64;  // experts per lane

constexpr double LOWEST = -__builtin_inf();

template <typename T>
__global__ __launch_bounds__(RT) void route_kernel(RouteArgs a) {
    __shared__ double group_c[RWAVES][NMS_ROUTE_MAX_EXPERTS];
    __shared__ uint8_t group_kept[RWAVES][NMS_ROUTE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * RWAVES + wave;
    // every wave of the workgroup reaches its end by itself (no barrier)
    if (t >= a.tokens) return;
    const int E = a.experts, k = a.opt.top_k;
    int32_t *ids = a.ids + t * k;
    float *weights = a.weights + t * k;
    if (a.live != nullptr && a.live[t] == 0) {
        if (lane < k) {
            ids[lane] = -1;
            weights[lane] = 0.0f;
        }
        return;
    }
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    float z[MAX_VALUES];
    float m = NEG_INF;
#pragma unroll
    for (int j = 0; j < MAX_VALUES; ++j) {
        const int e = 64 * j + lane;
        float v = e < E ? to_f32(row[e]) : NEG_INF;
        if (!(v > NEG_INF)) v = NEG_INF;
        z[j] = v;
        m = fmaxf(m, v);
    }
    double s[MAX_VALUES], c[MAX_VALUES], r[MAX_VALUES];
    double total = 0.0;
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX;
    if (softmax) {
        m = wave_max(m);
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) {
            s[j] = z[j] == NEG_INF ? 0.0 : z[j] == m ? 1.0 : exp((double)z[j] - (double)m);
            total += s[j];
        }
        total = wave_sum(total);
    }
#pragma unroll
    for (int j = 0; j < MAX_VALUES; ++j) {
        const int e = 64 * j + lane;
        s[j] = z[j] == NEG_INF ? 0.0 : softmax ? s[j] / total : 1.0 / (1.0 + exp(-(double)z[j]));
        c[j] = z[j] == NEG_INF ? LOWEST : s[j] + (a.bias ? (double)a.bias[e] : 0.0);
        if (!(c[j] > LOWEST)) c[j] = LOWEST;
        r[j] = a.bias == nullptr && c[j] > LOWEST ? (double)z[j] : c[j];
    }
    if (a.opt.groups > 1) {
        const int G = a.opt.groups, size = E / G;
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j)
            if (64 * j + lane < E) group_c[wave][64 * j + lane] = c[j];
        wave_fence();
        double best[MAX_VALUES];
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) {
            const int g = 64 * j + lane;
            double b0 = LOWEST, b1 = LOWEST;
            if (g < G)
                for (int i = 0; i < size; ++i) {
                    const double v = group_c[wave][g * size + i];
                    b1 = v > b0 ? b0 : v > b1 ? v : b1;
                    b0 = v > b0 ? v : b0;
                }
            best[j] = a.opt.group_top == 2 && b1 > LOWEST ? b0 + b1 : b0;
        }
        for (int g = lane; g < G; g += 64) group_kept[wave][g] = 0;
        wave_fence();
        for (int i = 0; i < a.opt.kept_groups; ++i) {
            double v = LOWEST;
            int at = -1;
#pragma unroll
            for (int j = 0; j < MAX_VALUES; ++j)
                if (best[j] > v) {
                    v = best[j];
                    at = 64 * j + lane;
                }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) {
                const double v2 = __shfl_xor(v, d);
                const int at2 = __shfl_xor(at, d);
                if (v2 > v || (v2 == v && at2 >= 0 && at2 < at)) {
                    v = v2;
                    at = at2;
                }
            }
            if (at < 0) break;
#pragma unroll
            for (int j = 0; j < MAX_VALUES; ++j)
                if (at == 64 * j + lane) {
                    best[j] = LOWEST;
                    group_kept[wave][at] = 1;
                }
        }
        wave_fence();
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) {
            const int e = 64 * j + lane;
            if (e < E && group_kept[wave][e / size] == 0) r[j] = LOWEST;
        }
    }
    int my_id = -1;
    float my_z = NEG_INF;
    double my_s = 0.0;
    for (int i = 0; i < k; ++i) {
        double v = LOWEST;
        int at = -1;
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j)
            if (r[j] > v) {
                v = r[j];
                at = 64 * j + lane;
            }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const double v2 = __shfl_xor(v, d);
            const int at2 = __shfl_xor(at, d);
            if (v2 > v || (v2 == v && at2 >= 0 && (at < 0 || at2 < at))) {
                v = v2;
                at = at2;
            }
        }
        if (at < 0) break;
        double sv = 0.0;
        float zv = 0.0f;
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j)
            if (at == 64 * j + lane) {
                r[j] = LOWEST;
                sv = s[j];
                zv = z[j];
            }
        sv = __shfl(sv, at & 63);
        zv = __shfl(zv, at & 63);
        if (lane == i) {
            my_id = at;
            my_s = sv;
            my_z = zv;
        }
    }
    if (a.opt.renormalise) {
        if (softmax) {
            // the softmax over the chosen logits: the same quotient, and it
            // holds where every chosen probability is below binary64's range
            const float zm = wave_max(my_z);
            my_s = my_id < 0 ? 0.0 : my_z == zm ? 1.0 : exp((double)my_z - (double)zm);
        }
        const double sum = wave_sum(my_s);
        my_s = sum > 0.0 ? my_s / sum : 0.0;
    }
    if (lane < k) {
        ids[lane] = my_id;
        weights[lane] = (float)(my_s * (double)a.opt.scale);
        if (a.counts != nullptr && my_id >= 0) atomicAdd(a.counts + my_id, 1);
    }
}

__global__ void zero_counts_kernel(int32_t *counts, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) counts[i] = 0;
}

// Gradient of the weights in the logits, given the chosen experts.
//   softmax, not renormalised  w_i = scale p_i:
//       dz_j = p_j (scale g_j [j chosen] - sum_i scale g_i p_i)
//   softmax, renormalised      q = softmax over the chosen logits, w = scale q:
//       dz_j = q_j scale (g_j - sum_i g_i q_i), 0 for the others
//   sigmoid                    w_i = scale s_i / D, D = 1 or sum of chosen s:
//       dz_j = scale (g_j - [renormalised] sum_i g_i s_i / D) / D s_j (1 - s_j)
template <typename T>
__global__ __launch_bounds__(RT) void route_back_kernel(RouteBackArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * RWAVES + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const int E = a.experts, k = a.opt.top_k;
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    T *out = static_cast<T *>(a.grad_logits) + t * a.grad_stride;
    int id = -1;
    float g = 0.0f, zc = NEG_INF;
    if (lane < k) {
        id = a.ids[t * k + lane];
        if ((unsigned)id >= (unsigned)E) id = -1;
        if (id >= 0) {
            g = a.grad_weights[t * k + lane] * a.opt.scale;
            zc = to_f32(row[id]);
        }
    }
    const bool softmax = a.opt.score == NMS_ROUTE_SOFTMAX;
    float z[MAX_VALUES], p[MAX_VALUES];
    float inner = 0.0f, d = 0.0f;
    bool whole = softmax && !a.opt.renormalise;
    if (whole) {
        float m = NEG_INF, total = 0.0f;
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) {
            const int e = 64 * j + lane;
            float v = e < E ? to_f32(row[e]) : NEG_INF;
            if (!(v > NEG_INF)) v = NEG_INF;
            z[j] = v;
            m = fmaxf(m, v);
        }
        m = wave_max(m);
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) {
            p[j] = z[j] == NEG_INF ? 0.0f : z[j] == m ? 1.0f : expf(z[j] - m);
            total += p[j];
        }
        total = wave_sum(total);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j) p[j] *= inv;
        const float pc = !(zc > NEG_INF) ? 0.0f : (zc == m ? 1.0f : expf(zc - m)) * inv;
        inner = wave_sum(g * pc);
        d = g;
    } else if (softmax) {
        if (!(zc > NEG_INF)) zc = NEG_INF;
        const float m = wave_max(zc);
        float q = zc == NEG_INF ? 0.0f : zc == m ? 1.0f : expf(zc - m);
        const float total = wave_sum(q);
        q = total > 0.0f ? q / total : 0.0f;
        d = q * (g - wave_sum(g * q));
    } else {
        // a NaN or -infinity logit is never chosen by the forward pass
        const float s = !(zc > NEG_INF) ? 0.0f : 1.0f / (1.0f + expf(-zc));
        const float slope = !(zc > NEG_INF) ? 0.0f : s / (1.0f + expf(zc));
        if (a.opt.renormalise) {
            const float total = wave_sum(s);
            const float mean = total > 0.0f ? wave_sum(g * s) / total : 0.0f;
            d = total > 0.0f ? (g - mean) / total * slope : 0.0f;
        } else {
            d = g * slope;
        }
    }
    float ds[MAX_VALUES];
#pragma unroll
    for (int j = 0; j < MAX_VALUES; ++j) ds[j] = 0.0f;
    for (int i = 0; i < k; ++i) {
        const int at = __shfl(id, i);
        const float v = __shfl(d, i);
#pragma unroll
        for (int j = 0; j < MAX_VALUES; ++j)
            if (at == 64 * j + lane) ds[j] += v;
    }
#pragma unroll
    for (int j = 0; j < MAX_VALUES; ++j) {
        const int e = 64 * j + lane;
        if (e < E) out[e] = from_f32<T>(whole ? p[j] * (ds[j] - inner) : ds[j]);
    }
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    if (a.counts != nullptr)
        zero_counts_kernel<<<(a.experts + 255) / 256, 256, 0, stream>>>(a.counts, a.experts);
    if (a.tokens > 0) {
        const unsigned grid = (unsigned)((a.tokens + RWAVES - 1) / RWAVES);
        if (a.dtype == NMS_F32) route_kernel<float><<<grid, RT, 0, stream>>>(a);
        else if (a.dtype == NMS_F16) route_kernel<half_t><<<grid, RT, 0, stream>>>(a);
        else route_kernel<bf16_t><<<grid, RT, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.tokens + RWAVES - 1) / RWAVES);
    if (a.dtype == NMS_F32) route_back_kernel<float><<<grid, RT, 0, stream>>>(a);
    else if (a.dtype == NMS_F16) route_back_kernel<half_t><<<grid, RT, 0, stream>>>(a);
    else route_back_kernel<bf16_t><<<grid, RT, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gnms
