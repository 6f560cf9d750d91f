// The balance loss of routing, and the loss on the size of its logits, with
// their gradient.
//
// With c_qe how many tokens of sequence q chose expert e, n_q its tokens, s a
// token's scores divided by their sum, and
//     a_qe = balance E c_qe / (S n_q sum_e c_qe)
// the loss is a sum over tokens, sum_e a_qe s_e + z / N lse^2: the counts have
// no gradient, so that once they are known one pass over the logits gives the
// loss and its gradient,
//     softmax:  dz_j = s_j (a_j - sum a s)
//     sigmoid:  dz_j = s_j (1 - sigmoid_j) (a_j - sum a s)
//     both:     + 2 z / N lse softmax_j.
#include "loss_internal.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr float LOG2E = 1.44269504f;
constexpr int CT = 1024;  // threads that count
constexpr int MAX_PARTS = 64, PART_IDS = 32768;

// The counts of each part of a sequence and of the whole (as they go into the
// factors), its tokens, the factors a, the sequence of each token, the terms.
struct BalanceSpace {
    int32_t *parts, *part_tokens, *tokens, *owner;
    float *factors;
    double *terms;
    int64_t blocks;
};

constexpr size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

// Parts of a sequence that are counted apart.  Sequences are as long as they
// are: the number goes by their mean length.
int parts_of(int64_t tokens, int64_t sequences, int top_k) {
    const int64_t ids = tokens * (top_k < 1 ? 1 : top_k) / (sequences < 1 ? 1 : sequences);
    const int64_t n = (ids + PART_IDS - 1) / PART_IDS;
    return n < 1 ? 1 : n > MAX_PARTS ? MAX_PARTS : (int)n;
}

constexpr int MT = 256;  // threads of the main pass

int lanes_of(int experts) {
    return experts <= 64 ? 8 : experts <= 128 ? 16 : experts <= 256 ? 32 : 64;
}

int64_t blocks_of(int64_t tokens, int experts) {
    const int64_t per = MT / lanes_of(experts);
    return (tokens + per - 1) / per;
}

size_t lay_out(int64_t tokens, int experts, int64_t sequences, int top_k, void *at,
               BalanceSpace *s) {
    const int parts = parts_of(tokens, sequences, top_k);
    const int64_t blocks = blocks_of(tokens, experts);
    const size_t cells = (size_t)sequences * experts;
    size_t n = 0;
    auto take = [&](size_t bytes) {
        const size_t from = n;
        n += round_up(bytes);
        return static_cast<char *>(at) + (at ? from : 0);
    };
    char *counted = take(parts > 1 ? parts * cells * sizeof(int32_t) : 0);
    char *part_tokens = take((size_t)parts * sequences * sizeof(int32_t));
    char *seq = take((size_t)sequences * sizeof(int32_t));
    char *owner = take((size_t)tokens * sizeof(int32_t));
    char *factors = take(cells * sizeof(float));
    char *terms = take((size_t)blocks * sizeof(double));
    if (s)
        *s = {reinterpret_cast<int32_t *>(counted), reinterpret_cast<int32_t *>(part_tokens),
              reinterpret_cast<int32_t *>(seq),     reinterpret_cast<int32_t *>(owner),
              reinterpret_cast<float *>(factors),   reinterpret_cast<double *>(terms), blocks};
    return n;
}

__device__ __forceinline__ int block_total(int v, int *shared) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    int sum = 0;
    for (int q = 0; q < (int)blockDim.x / 64; ++q) sum += shared[q];
    return sum;
}

// Where a sequence starts: the largest offset up to its own, within the
// tokens, so that the sequences never overlap.
__device__ __forceinline__ int start_of(const BalanceArgs &a, int64_t q, int *shared) {
    if (a.offsets == nullptr) return q == 0 ? 0 : (int)a.tokens;
    int64_t top = 0;
    for (int64_t i = threadIdx.x; i <= q; i += blockDim.x) top = max(top, a.offsets[i]);
    int v = wave_max((int)min(top, a.tokens));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 64; ++w) v = max(v, shared[w]);
    return v;
}

// a_qe of the thread's expert from its count, whose sum over the experts all
// threads know.
__device__ __forceinline__ void write_factor(const BalanceArgs &a, const BalanceSpace &s, int64_t q,
                                             int count, int64_t all, int tokens) {
    const int e = threadIdx.x;
    if (e >= a.experts) return;
    const double per = (double)a.sequences * (double)tokens * (double)all;
    s.factors[q * a.experts + e] =
        all > 0 && tokens > 0 ? (float)((double)a.balance * a.experts * (double)count / per) : 0.0f;
}

// The sum of counts that are given may pass 31 bits.
__device__ __forceinline__ int64_t block_total64(int64_t v, double *shared) {
    double d = wave_sum((double)v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = d;
    __syncthreads();
    d = 0.0;
    for (int q = 0; q < (int)blockDim.x / 64; ++q) d += shared[q];
    return (int64_t)d;
}

// A workgroup per (sequence, part): the part's counts and tokens, and which
// sequence its tokens are of.  Alone, it writes the sequence's factors too.
__global__ __launch_bounds__(CT) void count_kernel(BalanceArgs a, BalanceSpace s, int parts) {
    __shared__ int hist[NMS_ROUTE_MAX_EXPERTS];
    __shared__ int shared[CT / 64];
    __shared__ double wide[CT / 64];
    const int64_t q = blockIdx.x;
    const int part = blockIdx.y, tid = threadIdx.x;
    hist[tid] = 0;
    const int begin = start_of(a, q, shared), end = start_of(a, q + 1, shared);
    __syncthreads();
    const int size = (end - begin + parts - 1) / parts;
    const int from = min(begin + part * size, end), to = min(from + size, end);
    int used = 0;
    for (int t = from + tid; t < to; t += CT) {
        const bool live = a.live == nullptr || a.live[t] != 0;
        used += live;
        s.owner[t] = live ? (int)q : -1;
    }
    // the tokens of no sequence
    if (q == 0 && part == 0)
        for (int t = tid; t < begin; t += CT) s.owner[t] = -1;
    if (q == a.sequences - 1 && part == 0)
        for (int64_t t = end + tid; t < a.tokens; t += CT) s.owner[t] = -1;
    if (a.ids) {
        const int64_t last = (int64_t)to * a.top_k;
        for (int64_t i = (int64_t)from * a.top_k + tid; i < last; i += CT) {
            const int id = a.ids[i];
            if ((unsigned)id < (unsigned)a.experts &&
                (a.live == nullptr || a.live[i / a.top_k] != 0))
                atomicAdd(&hist[id], 1);
        }
    }
    const int tokens = block_total(used, shared);
    __syncthreads();
    if (parts > 1) {
        if (tid < a.experts && a.ids)
            s.parts[((int64_t)q * parts + part) * a.experts + tid] = hist[tid];
        if (tid == 0) s.part_tokens[q * parts + part] = tokens;
        return;
    }
    int count = 0;
    if (tid < a.experts) {
        count = a.ids ? hist[tid] : max(a.counts[q * a.experts + tid], 0);
        if (a.ids && a.counts) a.counts[q * a.experts + tid] = count;
    }
    write_factor(a, s, q, count, block_total64(count, wide), tokens);
    if (tid == 0) s.tokens[q] = tokens;
}

// A workgroup per sequence: its counts and factors from those of its parts.
__global__ __launch_bounds__(CT) void join_kernel(BalanceArgs a, BalanceSpace s, int parts) {
    __shared__ double wide[CT / 64];
    const int64_t q = blockIdx.x;
    const int tid = threadIdx.x;
    int tokens = 0, count = 0;
    for (int p = 0; p < parts; ++p) tokens += s.part_tokens[q * parts + p];
    if (tid < a.experts) {
        if (a.ids) {
            for (int p = 0; p < parts; ++p) count += s.parts[(q * parts + p) * a.experts + tid];
            if (a.counts) a.counts[q * a.experts + tid] = count;
        } else {
            count = max(a.counts[q * a.experts + tid], 0);
        }
    }
    write_factor(a, s, q, count, block_total64(count, wide), tokens);
    if (tid == 0) s.tokens[q] = tokens;
}

// LANES lanes per token, VALUES experts each.
template <typename T, int LANES, int VALUES>
__global__ __launch_bounds__(MT) void balance_kernel(BalanceArgs a, BalanceSpace s) {
    __shared__ double shared[MT / 64];
    constexpr int TOKENS = MT / LANES;
    const int sub = threadIdx.x % LANES, E = a.experts, e0 = sub * VALUES;
    const int64_t t = (int64_t)blockIdx.x * TOKENS + threadIdx.x / LANES;
    const bool inside = t < a.tokens;
    const int owner = inside ? s.owner[t] : -1;
    const bool softmax = a.score == NMS_ROUTE_SOFTMAX;
    float per = 0.0f;  // z / N
    if (a.z != 0.0f) {
        int64_t all = 0;
        for (int64_t q = threadIdx.x & 63; q < a.sequences; q += 64) all += s.tokens[q];
        const double n = wave_sum((double)all);
        per = n > 0.0 ? (float)((double)a.z / n) : 0.0f;
    }
    float z[VALUES], f[VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) {
        z[j] = NEG_INF;
        f[j] = 0.0f;
    }
    if (owner >= 0) {
        const T *row = static_cast<const T *>(a.logits) + t * a.row_stride + e0;
        const float *from = s.factors + (int64_t)owner * E + e0;
        if (e0 + VALUES <= E) {
            T raw[VALUES];
            __builtin_memcpy(raw, row, sizeof(raw));
            __builtin_memcpy(f, from, sizeof(f));
#pragma unroll
            for (int j = 0; j < VALUES; ++j) z[j] = to_f32(raw[j]);
        } else {
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (e0 + j < E) {
                    z[j] = to_f32(row[j]);
                    f[j] = from[j];
                }
        }
    }
    float top = NEG_INF;
#pragma unroll
    for (int j = 0; j < VALUES; ++j) top = fmaxf(top, z[j]);
    top = unordered(all_max<LANES>(ordered(top)));
    const float base = top == NEG_INF ? 0.0f : top;
    float x[VALUES], sum = 0.0f;
    if (softmax || per != 0.0f) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            x[j] = __builtin_amdgcn_exp2f((z[j] - base) * LOG2E);
            sum += x[j];
        }
        sum = all_sum<LANES>(sum);
    }
    const float inverse = sum != 0.0f ? 1.0f / sum : 0.0f;
    float d[VALUES], inner = 0.0f;
    if (softmax) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) inner += f[j] * x[j];
        inner = all_sum<LANES>(inner) * inverse;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) d[j] = x[j] * inverse * (f[j] - inner);
    } else {
        // shares of the scores' sum, each score divided by exp(m) first,
        // m = min(largest logit, 0): below -88 a score itself is under
        // float32's range, its share is not
        const float m = fminf(base, 0.0f);
        float total = 0.0f, rest[VALUES];  // rest: 1 - score
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            // one exponential of what is not above 0
            const float low = __builtin_amdgcn_exp2f(-fabsf(z[j]) * LOG2E);
            const float part = 1.0f / (1.0f + low);
            const bool up = z[j] > 0.0f;
            rest[j] = up ? low * part : part;
            const float score =
                up ? part : __builtin_amdgcn_exp2f((z[j] - m) * LOG2E) * part;
            d[j] = z[j] == z[j] ? score : z[j];
            total += d[j];
        }
        total = all_sum<LANES>(total);
        const float under = total != 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) inner += f[j] * d[j];
        inner = all_sum<LANES>(inner) * under;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) d[j] = d[j] * under * rest[j] * (f[j] - inner);
    }
    float term = inner;
    if (per != 0.0f && sum != 0.0f) {
        const float lse = base + logf(sum);
        term += per * lse * lse;
        const float more = 2.0f * per * lse * inverse;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) d[j] += more * x[j];
    }
    if (a.grad_logits && inside) {
        const float up = a.grad_loss ? a.grad_loss[0] : 1.0f;
        T out[VALUES];
#pragma unroll
        for (int j = 0; j < VALUES; ++j) out[j] = from_f32<T>(owner >= 0 ? d[j] * up : 0.0f);
        T *to = static_cast<T *>(a.grad_logits) + t * a.grad_stride + e0;
        if (e0 + VALUES <= E) {
            __builtin_memcpy(to, out, sizeof(out));
        } else {
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (e0 + j < E) to[j] = out[j];
        }
    }
    if (a.loss == nullptr) return;
    const double mine = wave_sum(sub == 0 && owner >= 0 ? (double)term : 0.0);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int q = 0; q < MT / 64; ++q) all += shared[q];
        s.terms[blockIdx.x] = all;
    }
}

template <typename T>
void run(const BalanceArgs &a, const BalanceSpace &s, hipStream_t stream) {
    const unsigned n = (unsigned)s.blocks;
    const int E = a.experts;
    if (E <= 64) balance_kernel<T, 8, 8><<<n, MT, 0, stream>>>(a, s);
    else if (E <= 128) balance_kernel<T, 16, 8><<<n, MT, 0, stream>>>(a, s);
    else if (E <= 256) balance_kernel<T, 32, 8><<<n, MT, 0, stream>>>(a, s);
    else if (E <= 512) balance_kernel<T, 64, 8><<<n, MT, 0, stream>>>(a, s);
    else balance_kernel<T, 64, 16><<<n, MT, 0, stream>>>(a, s);
}

}  // namespace

size_t balance_workspace_bytes(int64_t tokens, int experts, int64_t sequences, int top_k) {
    return lay_out(tokens, experts, sequences, top_k, nullptr, nullptr) + 256;
}

hipError_t launch_balance(const BalanceArgs &a, hipStream_t stream) {
    BalanceSpace s;
    lay_out(a.tokens, a.experts, a.sequences, a.top_k, a.workspace, &s);
    const int parts = parts_of(a.tokens, a.sequences, a.top_k);
    count_kernel<<<dim3((unsigned)a.sequences, (unsigned)parts), CT, 0, stream>>>(a, s, parts);
    if (parts > 1) join_kernel<<<(unsigned)a.sequences, CT, 0, stream>>>(a, s, parts);
    if (a.tokens > 0 && (a.loss || a.grad_logits)) {
        if (a.dtype == NMS_F32) run<float>(a, s, stream);
        else if (a.dtype == NMS_F16) run<half_t>(a, s, stream);
        else run<bf16_t>(a, s, stream);
    }
    if (a.loss) launch_total(s.terms, a.tokens > 0 ? s.blocks : 0, a.loss, stream);
    return hipGetLastError();
}

}  // namespace gnms
