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
// What bounds it: up to some ten thousand tokens the kernels, one after another, and
// the caller's time are about as long.  Three or four launches (3.3 us each), three
// outputs and the binding take the caller 18 to 21 us; of the kernels, at 16384 x 256
// float32 in 16 sequences (19.4 us a call), counting takes 6.8 to 8.0 us (a workgroup
// for each sequence, five trips to memory one after another), the pass 10.9 to 12.4 us
// for 33 MB (345 vector instructions for a wave's two tokens) and the sum 1.8 to 3.8.
// Scores, their sums over a token's experts and the gradient are in float32, by one
// term of log2(e): with x the distance to the largest logit, a share is off by
// (4 x + 2) 2^-24 of it by its exponential and by 22 more at most by the sum (16
// experts in a lane, 6 joins), and by an ulp where a sigmoid takes its inverse by one
// instruction; no difference of nearly equal numbers makes more of that.  Sums over
// tokens are in binary64.
#include "loss_internal.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr float LOG2E = 1.44269504f;
constexpr int CT = 1024;  // threads that count
constexpr int MAX_PARTS = 64, PART_IDS = 8192;

// The counts of each part of a sequence, the tokens of the parts and of the
// whole, the sequence of each token, or where there is only one its first token
// and the one behind its last, the factors a, the terms.
struct BalanceSpace {
    int32_t *parts, *part_tokens, *tokens, *owner, *range;
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

// Tokens that a group of lanes takes in turn, their logits loaded together: 131072 x
// 128 float32 43.1 us with four, 44.3 with one; of fewer tokens it makes no odds.
int turns_of(int64_t tokens, int experts) {
    return tokens * lanes_of(experts) >= (int64_t)4096 * MT ? 4 : 1;
}

int64_t blocks_of(int64_t tokens, int experts) {
    const int64_t per = (int64_t)MT / lanes_of(experts) * turns_of(tokens, experts);
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
    char *range = take(2 * sizeof(int32_t));
    char *owner = take(sequences > 1 ? (size_t)tokens * sizeof(int32_t) : 0);
    char *factors = take(cells * sizeof(float));
    char *terms = take((size_t)blocks * sizeof(double));
    if (s)
        *s = {reinterpret_cast<int32_t *>(counted), reinterpret_cast<int32_t *>(part_tokens),
              reinterpret_cast<int32_t *>(seq),     reinterpret_cast<int32_t *>(owner),
              reinterpret_cast<int32_t *>(range),   reinterpret_cast<float *>(factors),
              reinterpret_cast<double *>(terms),    blocks};
    return n;
}

// -------------------------------------------------------- counts and factors

// Two sums over the workgroup, the same in every thread.  (Counts that are
// given may add up to more than 31 bits.)
struct Totals {
    int tokens;
    double counts;
};
__device__ __forceinline__ Totals totals_of(int tokens, int count, Totals *shared) {
    Totals t = {wave_sum(tokens), wave_sum((double)count)};
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = t;
    __syncthreads();
    t = {0, 0.0};
    for (int q = 0; q < CT / 64; ++q) {
        t.tokens += shared[q].tokens;
        t.counts += shared[q].counts;
    }
    return t;
}

// Where sequence q starts and ends: the largest offset up to its own, within
// the tokens, so that the sequences never overlap.
__device__ __forceinline__ void bounds_of(const BalanceArgs &a, int64_t q, int *shared, int &begin,
                                          int &end) {
    begin = 0;
    end = (int)a.tokens;
    if (a.offsets == nullptr) return;
    const int64_t next = a.offsets[q + 1];
    int64_t top = 0;
    for (int64_t i = threadIdx.x; i <= q; i += CT) top = max(top, a.offsets[i]);
    const int v = wave_max((int)min(top, a.tokens));
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < CT / 64; ++w) begin = max(begin, shared[w]);
    end = max(begin, (int)min(max(next, (int64_t)0), a.tokens));
}

// Adds the experts of the tokens from `from` to `to` to the counts in LDS, a
// thread per token; returns how many of these count.
__device__ __forceinline__ int count_tokens(const BalanceArgs &a, int from, int to, int q,
                                            int32_t *owner, int *hist) {
    int used = 0;
    for (int t = from + (int)threadIdx.x; t < to; t += CT) {
        const bool live = a.live == nullptr || a.live[t] != 0;
        used += live;
        if (owner) owner[t] = live ? q : -1;
        if (!live || a.ids == nullptr) continue;
        const int32_t *ids = a.ids + (int64_t)t * a.top_k;
        for (int i = 0; i < a.top_k; i += 4) {
            int id[4] = {-1, -1, -1, -1};
            if (i + 4 <= a.top_k) {
                __builtin_memcpy(id, ids + i, sizeof(id));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i + j < a.top_k) id[j] = ids[i + j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((unsigned)id[j] < (unsigned)a.experts) atomicAdd(&hist[id[j]], 1);
        }
    }
    return used;
}

// a_qe from an expert's count.
__device__ __forceinline__ float factor_of(const BalanceArgs &a, int count, const Totals &t) {
    const double per = (double)a.sequences * (double)t.tokens * t.counts;
    return per > 0.0 ? (float)((double)a.balance * a.experts * (double)count / per) : 0.0f;
}

__device__ __forceinline__ void write_sequence(const BalanceArgs &a, const BalanceSpace &s,
                                               int64_t q, int count, const Totals &t) {
    const int e = threadIdx.x;
    if (e == 0) s.tokens[q] = t.tokens;
    if (e < a.experts) s.factors[q * a.experts + e] = factor_of(a, count, t);
}

// A workgroup per (sequence, part): the part's counts and tokens, and which
// sequence its tokens are of.  Alone, it writes the sequence's factors too.
__global__ __launch_bounds__(CT) void count_kernel(BalanceArgs a, BalanceSpace s, int parts) {
    __shared__ int hist[NMS_ROUTE_MAX_EXPERTS];
    __shared__ int places[CT / 64];
    __shared__ Totals sums[CT / 64];
    const int64_t q = blockIdx.x;
    const int part = blockIdx.y, tid = threadIdx.x;
    hist[tid] = 0;
    int begin, end;
    bounds_of(a, q, places, begin, end);
    __syncthreads();
    const int size = (end - begin + parts - 1) / parts;
    const int from = min(begin + part * size, end), to = min(from + size, end);
    const bool several = a.sequences > 1;
    const int used = count_tokens(a, from, to, (int)q, several ? s.owner : nullptr, hist);
    // the tokens of no sequence
    if (several && q == 0 && part == 0)
        for (int t = tid; t < begin; t += CT) s.owner[t] = -1;
    if (several && q == a.sequences - 1 && part == 0)
        for (int64_t t = end + tid; t < a.tokens; t += CT) s.owner[t] = -1;
    if (!several && tid == 0 && part == 0) {
        s.range[0] = begin;
        s.range[1] = end;
    }
    __syncthreads();
    int count = 0;
    if (tid < a.experts) {
        if (a.ids) count = hist[tid];
        else if (parts == 1) count = max(a.counts[q * a.experts + tid], 0);
    }
    const Totals t = totals_of(used, count, sums);
    if (parts > 1) {
        if (tid < a.experts && a.ids) s.parts[(q * parts + part) * a.experts + tid] = count;
        if (tid == 0) s.part_tokens[q * parts + part] = t.tokens;
        return;
    }
    if (tid < a.experts && a.ids && a.counts) a.counts[q * a.experts + tid] = count;
    write_sequence(a, s, q, count, t);
}

// A workgroup per sequence: its counts and factors from those of its parts.
__global__ __launch_bounds__(CT) void join_kernel(BalanceArgs a, BalanceSpace s, int parts) {
    __shared__ Totals sums[CT / 64];
    const int64_t q = blockIdx.x;
    const int tid = threadIdx.x;
    int count = 0;
    if (tid < a.experts) {
        if (a.ids) {
#pragma unroll 8
            for (int p = 0; p < parts; ++p) count += s.parts[(q * parts + p) * a.experts + tid];
            if (a.counts) a.counts[q * a.experts + tid] = count;
        } else {
            count = max(a.counts[q * a.experts + tid], 0);
        }
    }
    write_sequence(a, s, q, count,
                   totals_of(tid < parts ? s.part_tokens[q * parts + tid] : 0, count, sums));
}

// ------------------------------------------------------- loss and gradient

// z / N, for the number N of tokens that count.
__device__ __forceinline__ float share_of(float z, double n) {
    return n > 0.0 ? (float)((double)z / n) : 0.0f;
}

// A token's part of the loss and its gradient (in place of its logits) on LANES
// lanes, VALUES experts each: z its logits (-infinity past the last), f its
// sequence's factors, per: z / N.
template <int LANES, int VALUES>
__device__ __forceinline__ float token_loss(float (&z)[VALUES], const float (&f)[VALUES],
                                            bool softmax, float per) {
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
    float inner = 0.0f;
    if (softmax) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) inner += f[j] * x[j];
        inner = all_sum<LANES>(inner) * inverse;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = x[j] * inverse * (f[j] - inner);
    } else {
        // shares of the scores' sum, each score divided by exp(m) first,
        // m = min(largest logit, 0): below -88 a score itself is under
        // float32's range, its share is not
        const float m = fminf(base, 0.0f);
        const bool under_0 = __ballot(m < 0.0f) != 0ull;
        float total = 0.0f, rest[VALUES];  // rest: 1 - score
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            // (the inverse by one instruction, off by up to an ulp)
            float low = __builtin_amdgcn_exp2f(-fabsf(z[j]) * LOG2E);
            const float part = __builtin_amdgcn_rcpf(1.0f + low);
            const bool up = z[j] > 0.0f;
            rest[j] = up ? low * part : part;
            if (under_0) low = __builtin_amdgcn_exp2f((z[j] - m) * LOG2E);
            z[j] = (up ? 1.0f : low) * part;
            total += z[j];
        }
        total = all_sum<LANES>(total);
        const float under = total != 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) inner += f[j] * z[j];
        inner = all_sum<LANES>(inner) * under;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = z[j] * under * rest[j] * (f[j] - inner);
    }
    if (per != 0.0f && sum != 0.0f) {
        const float lse = base + logf(sum);
        const float more = 2.0f * per * lse * inverse;
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] += more * x[j];
        inner += per * lse * lse;
    }
    return inner;
}

template <typename T, int VALUES>
struct Raw {
    T v[VALUES];
};

template <typename T, int VALUES>
__device__ __forceinline__ Raw<T, VALUES> load_raw(const T *row, int left, bool there) {
    Raw<T, VALUES> r;
    if (there && left >= VALUES) {
        __builtin_memcpy(&r, row, sizeof(r));
    } else {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) r.v[j] = there && j < left ? row[j] : from_f32<T>(NEG_INF);
    }
    return r;
}

template <typename T, int VALUES>
__device__ __forceinline__ void store_gradient(T *to, int left, const float (&d)[VALUES], float up) {
    T out[VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) out[j] = from_f32<T>(d[j] * up);
    if (left >= VALUES) {
        __builtin_memcpy(to, out, sizeof(out));
    } else {
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            if (j < left) to[j] = out[j];
    }
}

// LANES lanes per token, VALUES experts each, TURNS tokens one after another.
template <typename T, int LANES, int VALUES, int TURNS>
__global__ __launch_bounds__(MT) void balance_kernel(BalanceArgs a, BalanceSpace s) {
    __shared__ double shared[MT / 64];
    constexpr int GROUPS = MT / LANES;
    const int sub = threadIdx.x % LANES, E = a.experts, e0 = sub * VALUES, left = E - e0;
    const int64_t first = (int64_t)blockIdx.x * (GROUPS * TURNS) + threadIdx.x / LANES;
    const T *logits = static_cast<const T *>(a.logits) + e0;
    T *out = static_cast<T *>(a.grad_logits) + e0;
    int owner[TURNS];
    Raw<T, VALUES> raw[TURNS];
    // (loaded whether the token counts or not, which another load says)
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int64_t t = first + i * GROUPS;
        raw[i] = load_raw<T, VALUES>(logits + t * a.row_stride, left, t < a.tokens);
    }
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int64_t t = first + i * GROUPS;
        owner[i] = -1;
        if (t < a.tokens) {
            if (a.sequences > 1) owner[i] = s.owner[t];
            else if (t >= s.range[0] && t < s.range[1] && (!a.live || a.live[t])) owner[i] = 0;
        }
    }
    float per = 0.0f;
    if (a.z != 0.0f) {
        int64_t all = 0;
        for (int64_t q = threadIdx.x & 63; q < a.sequences; q += 64) all += s.tokens[q];
        per = share_of(a.z, wave_sum((double)all));
    }
    const float up = a.grad_loss ? a.grad_loss[0] : 1.0f;
    double term = 0.0;
    float f[VALUES];
    int held = -1;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int64_t t = first + i * GROUPS;
        if (i == 0 || (a.sequences > 1 && owner[i] != held)) {
            const float *from = s.factors + (int64_t)max(owner[i], 0) * E + e0;
            if (left >= VALUES) {
                __builtin_memcpy(f, from, sizeof(f));
            } else {
#pragma unroll
                for (int j = 0; j < VALUES; ++j) f[j] = j < left ? from[j] : 0.0f;
            }
            held = owner[i];
        }
        float z[VALUES];
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = owner[i] >= 0 ? to_f32(raw[i].v[j]) : NEG_INF;
        const float mine = token_loss<LANES, VALUES>(z, f, a.score == NMS_ROUTE_SOFTMAX, per);
        if (sub == 0) term += (double)mine;
        if (a.grad_logits && t < a.tokens)
            store_gradient<T, VALUES>(out + t * a.grad_stride, left, z, owner[i] >= 0 ? up : 0.0f);
    }
    if (a.loss == nullptr) return;
    term = wave_sum(term);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int q = 0; q < MT / 64; ++q) all += shared[q];
        s.terms[blockIdx.x] = all;
    }
}

// All of a small call in one workgroup, which saves two launches: 512 x 64 in 13.0
// us of the caller's time for 18.4, though in a graph it takes 9.0 for 8.0 (16 x 64
// 4.9 for 7.1); 1024 x 64 would take 14.2 for 8.5.
template <typename T, int LANES, int VALUES>
__global__ __launch_bounds__(CT) void small_kernel(BalanceArgs a) {
    __shared__ int hist[NMS_ROUTE_MAX_EXPERTS];
    __shared__ int places[CT / 64];
    __shared__ Totals sums[CT / 64];
    __shared__ float factors[NMS_ROUTE_MAX_EXPERTS];
    __shared__ double shared[CT / 64];
    constexpr int GROUPS = CT / LANES;
    const int tid = threadIdx.x, sub = tid % LANES, E = a.experts, e0 = sub * VALUES, left = E - e0;
    hist[tid] = 0;
    int begin, end;
    bounds_of(a, 0, places, begin, end);
    __syncthreads();
    const int used = count_tokens(a, begin, end, 0, nullptr, hist);
    __syncthreads();
    const int count = tid >= E ? 0 : a.ids ? hist[tid] : max(a.counts[tid], 0);
    const Totals sum = totals_of(used, count, sums);
    if (tid < E && a.ids && a.counts) a.counts[tid] = count;
    factors[tid] = tid < E ? factor_of(a, count, sum) : 0.0f;
    __syncthreads();
    const float per = a.z != 0.0f ? share_of(a.z, (double)sum.tokens) : 0.0f;
    const float up = a.grad_loss ? a.grad_loss[0] : 1.0f;
    float f[VALUES];
#pragma unroll
    for (int j = 0; j < VALUES; ++j) f[j] = j < left ? factors[e0 + j] : 0.0f;
    double term = 0.0;
    for (int from = 0; from < (int)a.tokens; from += GROUPS) {
        const int t = from + tid / LANES;
        const bool counts = t >= begin && t < end && (a.live == nullptr || a.live[t] != 0);
        const Raw<T, VALUES> raw = load_raw<T, VALUES>(
            static_cast<const T *>(a.logits) + t * a.row_stride + e0, left, counts);
        float z[VALUES];
#pragma unroll
        for (int j = 0; j < VALUES; ++j) z[j] = to_f32(raw.v[j]);
        const float mine = token_loss<LANES, VALUES>(z, f, a.score == NMS_ROUTE_SOFTMAX, per);
        if (sub == 0) term += (double)mine;
        if (a.grad_logits && t < a.tokens)
            store_gradient<T, VALUES>(static_cast<T *>(a.grad_logits) + t * a.grad_stride + e0,
                                      left, z, counts ? up : 0.0f);
    }
    term = wave_sum(term);
    if ((tid & 63) == 0) shared[tid >> 6] = term;
    __syncthreads();
    if (tid == 0 && a.loss) {
        double all = 0.0;
        for (int q = 0; q < CT / 64; ++q) all += shared[q];
        a.loss[0] = (float)all;
    }
}

// ----------------------------------------------------------------- launches

template <typename T, int LANES, int VALUES>
void launch(const BalanceArgs &a, const BalanceSpace &s, bool small, hipStream_t stream) {
    const unsigned n = (unsigned)s.blocks;
    if (small) small_kernel<T, LANES, VALUES><<<1, CT, 0, stream>>>(a);
    else if (turns_of(a.tokens, a.experts) == 1)
        balance_kernel<T, LANES, VALUES, 1><<<n, MT, 0, stream>>>(a, s);
    else
        balance_kernel<T, LANES, VALUES, 4><<<n, MT, 0, stream>>>(a, s);
}

template <typename T>
void run(const BalanceArgs &a, const BalanceSpace &s, bool small, hipStream_t stream) {
    const int E = a.experts;
    if (E <= 64) launch<T, 8, 8>(a, s, small, stream);
    else if (E <= 128) launch<T, 16, 8>(a, s, small, stream);
    else if (E <= 256) launch<T, 32, 8>(a, s, small, stream);
    else if (E <= 512) launch<T, 64, 8>(a, s, small, stream);
    else launch<T, 64, 16>(a, s, small, stream);
}

void run(const BalanceArgs &a, const BalanceSpace &s, bool small, hipStream_t stream) {
    if (a.dtype == NMS_F32) run<float>(a, s, small, stream);
    else if (a.dtype == NMS_F16) run<half_t>(a, s, small, stream);
    else run<bf16_t>(a, s, small, stream);
}

}  // namespace

size_t balance_workspace_bytes(int64_t tokens, int experts, int64_t sequences, int top_k) {
    return lay_out(tokens, experts, sequences, top_k, nullptr, nullptr) + 256;
}

hipError_t launch_balance(const BalanceArgs &a, hipStream_t stream) {
    BalanceSpace s;
    lay_out(a.tokens, a.experts, a.sequences, a.top_k, a.workspace, &s);
    if (a.sequences == 1 && a.tokens * lanes_of(a.experts) <= 4 * CT) {
        run(a, s, true, stream);
        return hipGetLastError();
    }
    const int parts = parts_of(a.tokens, a.sequences, a.top_k);
    count_kernel<<<dim3((unsigned)a.sequences, (unsigned)parts), CT, 0, stream>>>(a, s, parts);
    if (parts > 1) join_kernel<<<(unsigned)a.sequences, CT, 0, stream>>>(a, s, parts);
    if (a.tokens > 0 && (a.loss || a.grad_logits)) run(a, s, false, stream);
    if (a.loss) launch_total(s.terms, a.tokens > 0 ? s.blocks : 0, a.loss, stream);
    return hipGetLastError();
}

}  // namespace gnms
