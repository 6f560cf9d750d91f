// Log probabilities of given tokens and the losses made of them, with their
// gradients in the logits.
//
// With t a row's temperature, k = log2(e) / t, m the row's largest logit and
//     u_j = (z_j - m) k,  e_j = 2^u_j,  s = sum e_j,  w = sum u_j e_j:
//     log probability  (z_token - m) / t - log s
//     entropy          log s - ln 2 w / s
// and, where alpha and eta are the gradients in these two,
//     dz_j = e_j (P + Q u_j) + [j = token] alpha / t,
//     P = -(alpha + eta (entropy - log s)) / (s t),  Q = -eta ln 2 / (s t).
// So a row is read once for its (m, s, w), which join by rescaling, and once
// more for its gradient.
#include "loss_internal.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr float LOG2E = 1.44269504f;
constexpr double LN2 = 0.693147180559945309;

// -------------------------------------------------------------------- rows

// A slice's largest logit, sum of exponentials and weighted sum.  m may be
// -infinity (no logit above it); then s and w are 0, or NaN where one was NaN.
// at: the logit of the row's token, which a gradient in place of the logits
// overwrites.
struct Part {
    float m, s, w, at;
};

// Sixteen bytes of neighbouring elements.
template <typename T>
struct Pack {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
};

template <typename T>
__device__ __forceinline__ Pack<T> load_pack(const T *p, int left) {
    Pack<T> e;
    if (left >= Pack<T>::N) {
        __builtin_memcpy(&e, p, sizeof(e));
    } else {
#pragma unroll
        for (int j = 0; j < Pack<T>::N; ++j) e.v[j] = j < left ? p[j] : from_f32<T>(NEG_INF);
    }
    return e;
}

// What a row's logits are multiplied by, and 1 / t.  A temperature of 0 or
// below (or NaN) stands for 1; one beyond what its inverse holds takes the
// largest or smallest that float32 has, so that the largest logit keeps 2^0
// and -infinity stays out.
__device__ __forceinline__ void temperature_of(const LossRows &r, int64_t row, float &k,
                                               float &inverse) {
    float t = r.temperature ? r.temperature[row] : 1.0f;
    if (!(t > 0.0f)) t = 1.0f;
    k = fminf(fmaxf(LOG2E / t, 1.4012985e-45f), 3.4028235e38f);
    inverse = fminf(1.0f / t, 3.4028235e38f);
}

__device__ __forceinline__ bool counts_for(const LossRows &r, int64_t row, int &token) {
    token = r.tokens[row];
    return (unsigned)token < (unsigned)r.vocab && (!r.weights || r.weights[row] != 0.0f);
}

// The difference to a largest logit that may be -infinity.
__device__ __forceinline__ float base_of(float m) { return m == NEG_INF ? 0.0f : m; }

__device__ __forceinline__ float exp2_of(float u) { return __builtin_amdgcn_exp2f(u); }

// u as a factor of an exponential that is 0 from -150 down
__device__ __forceinline__ float factor(float u) { return fmaxf(u, -200.0f); }

// p becomes that of the logits of p and q.
template <bool ENTROPY>
__device__ __forceinline__ void join(Part &p, float m, float s, float w, float k) {
    const float top = fmaxf(p.m, m);
    const float a = p.m == NEG_INF ? 0.0f : (p.m - top) * k, b = m == NEG_INF ? 0.0f : (m - top) * k;
    const float fa = exp2_of(a), fb = exp2_of(b);
    if (ENTROPY) p.w = (p.w + factor(a) * p.s) * fa + (w + factor(b) * s) * fb;
    p.s = p.s * fa + s * fb;
    p.m = top;
}

// The join over the wave's lanes, the same in all of them.
template <bool ENTROPY>
__device__ __forceinline__ Part join_wave(Part p, float k) {
    const float top = wave_max(p.m);
    const float d = p.m == NEG_INF ? 0.0f : (p.m - top) * k;
    const float f = exp2_of(d);
    if (ENTROPY) p.w = wave_sum((p.w + factor(d) * p.s) * f);
    p.s = wave_sum(p.s * f);
    p.m = top;
    return p;
}

// ---------------------------------------------------------------- results

// One row's results; alpha and eta: the gradients in its log probability and
// entropy, times that of the loss; term: its part of the loss.
struct RowResult {
    float logprob, entropy, alpha, eta;
    double exact, term;
};

template <bool ENTROPY>
__device__ __forceinline__ RowResult result_of(const LossArgs &a, int64_t row, bool counts,
                                               const Part &p, float inverse, double &log_s) {
    RowResult r = {};
    log_s = 0.0;
    if (!counts) return r;
    // in binary64: sums over rows are made of these
    log_s = log((double)p.s);
    r.exact = p.s == 0.0f    ? (double)NEG_INF
              : p.at == NEG_INF ? (double)NEG_INF - log_s
                                : ((double)p.at - (double)p.m) * (double)inverse - log_s;
    r.logprob = (float)r.exact;
    if (ENTROPY) r.entropy = p.s == 0.0f ? 0.0f : (float)(log_s - LN2 * (double)p.w / (double)p.s);
    if (a.kind == LOSS_GIVEN) {
        r.alpha = a.grad_logprobs[row];
        if (ENTROPY) r.eta = a.grad_entropies[row];
    } else if (a.kind == LOSS_POLICY) {
        const float weight = a.in.weights ? a.in.weights[row] : a.weight;
        const float up = a.grad_loss ? a.grad_loss[0] : 1.0f;
        const float advantage = a.advantages[row];
        const float ratio = expf((float)(r.exact - (double)a.old_logprobs[row]));
        float each = 0.0f, slope = 0.0f;
        if (advantage != 0.0f) {
            const float free = ratio * advantage;
            const float held = fminf(fmaxf(ratio, a.clip_low), a.clip_high) * advantage;
            each = -fminf(free, held);
            slope = free <= held ? -free : 0.0f;
            if (ratio != ratio || advantage != advantage) each = slope = ratio * advantage;
        }
        if (a.ref_logprobs) {
            // exp(q) - q - 1, in binary64: it is small where q is
            const double q = (double)a.ref_logprobs[row] - r.exact;
            const double more = expm1(q);
            each += a.kl * (float)(more - q);
            slope -= a.kl * (float)more;
        }
        if (ENTROPY) each -= a.bonus * r.entropy;
        r.term = (double)weight * (double)each;
        r.alpha = up * weight * slope;
        r.eta = -up * weight * a.bonus;
    }
    return r;
}

template <bool ENTROPY>
__device__ __forceinline__ void write_result(const LossArgs &a, int64_t row, const RowResult &r,
                                             double *exact, double *terms) {
    if (a.logprobs) a.logprobs[row] = r.logprob;
    if (ENTROPY && a.entropies) a.entropies[row] = r.entropy;
    if (exact) exact[row] = r.exact;
    if (terms) terms[row] = r.term;
}

// --------------------------------------------------------------- workspace

// parts: rows x slices; terms: of the loss, one per row or pair; of a
// preference loss also exact, the rows' log probabilities in binary64, and
// alpha, the gradients in these.
struct LossSpace {
    Part *parts;
    double *terms, *exact;
    float *alpha;
};

constexpr size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int THREADS = 256, WAVES = THREADS / 64;
constexpr int MAX_SLICES = 64;

// Slices of a row: enough workgroups for the GPU where rows are few.
__host__ __device__ inline int slices_of(int64_t rows, int vocab) {
    int64_t n = (2048 + rows - 1) / (rows < 1 ? 1 : rows);
    const int64_t most = (vocab + 4095) / 4096;
    if (n > most) n = most;
    if (n > MAX_SLICES) n = MAX_SLICES;
    return n < 1 ? 1 : (int)n;
}

__host__ __device__ inline int slice_size(int vocab, int slices) {
    return ((vocab + slices - 1) / slices + 7) & ~7;
}

size_t lay_out(int64_t rows, int vocab, int64_t pairs, void *at, LossSpace *s) {
    const size_t parts = round_up((size_t)rows * slices_of(rows, vocab) * sizeof(Part));
    const size_t terms = round_up((size_t)(pairs > 0 ? pairs : rows) * sizeof(double));
    const size_t exact = pairs > 0 ? round_up((size_t)rows * sizeof(double)) : 0;
    const size_t alpha = pairs > 0 ? round_up((size_t)rows * sizeof(float)) : 0;
    char *p = static_cast<char *>(at);
    if (s) {
        s->parts = reinterpret_cast<Part *>(p);
        s->terms = reinterpret_cast<double *>(p + parts);
        s->exact = reinterpret_cast<double *>(p + parts + terms);
        s->alpha = reinterpret_cast<float *>(p + parts + terms + exact);
    }
    return parts + terms + exact + alpha;
}

// ----------------------------------------------------------------- kernels

// A workgroup per (row, slice): the slice's part, and where it is the row's
// only one the row's results.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void part_kernel(LossArgs a, LossSpace space, int slices,
                                                       bool finish) {
    constexpr int N = Pack<T>::N, UNROLL = 4, STEP = THREADS * N * UNROLL;
    __shared__ Part shared[WAVES];
    const int64_t row = blockIdx.x;
    int token;
    const bool counts = counts_for(a.in, row, token);
    const T *z = static_cast<const T *>(a.in.logits) + row * a.in.row_stride;
    float k, inverse;
    temperature_of(a.in, row, k, inverse);
    Part p = {NEG_INF, 0.0f, 0.0f, 0.0f};
    if (counts) {
        const int size = slice_size(a.in.vocab, slices);
        const int lo = (int)blockIdx.y * size;
        const int end = min(lo + size, a.in.vocab);
        for (int at = lo; at < end; at += STEP) {
            Pack<T> e[UNROLL];
#pragma unroll
            for (int q = 0; q < UNROLL; ++q) {
                const int i = at + (q * THREADS + (int)threadIdx.x) * N;
                e[q] = load_pack(z + i, end - i);
            }
            float top = p.m;
#pragma unroll
            for (int q = 0; q < UNROLL; ++q)
#pragma unroll
                for (int j = 0; j < N; ++j) top = fmaxf(top, to_f32(e[q].v[j]));
            const float base = base_of(top);
            const float d = p.m == NEG_INF ? 0.0f : (p.m - base) * k, f = exp2_of(d);
            if (ENTROPY) p.w = (p.w + factor(d) * p.s) * f;
            p.s *= f;
            p.m = top;
#pragma unroll
            for (int q = 0; q < UNROLL; ++q)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float u = (to_f32(e[q].v[j]) - base) * k;
                    const float x = exp2_of(u);
                    p.s += x;
                    if (ENTROPY) p.w = fmaf(factor(u), x, p.w);
                }
        }
        p = join_wave<ENTROPY>(p, k);
    }
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = p;
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int q = 1; q < WAVES; ++q)
        join<ENTROPY>(p, shared[q].m, shared[q].s, shared[q].w, k);
    p.at = counts ? to_f32(z[token]) : 0.0f;
    space.parts[row * slices + blockIdx.y] = p;
    if (finish) {
        double log_s;
        const RowResult r = result_of<ENTROPY>(a, row, counts, p, inverse, log_s);
        write_result<ENTROPY>(a, row, r, space.exact, space.terms);
    }
}

// A row's part from those of its slices, the same in every lane.
template <bool ENTROPY>
__device__ __forceinline__ Part row_part(const LossSpace &space, int64_t row, int slices, float k) {
    const int lane = threadIdx.x & 63;
    Part p = {NEG_INF, 0.0f, 0.0f, 0.0f};
    if (lane < slices) p = space.parts[row * slices + lane];
    const float at = __shfl(p.at, 0);
    p = slices > 1 ? join_wave<ENTROPY>(p, k)
                   : Part{__shfl(p.m, 0), __shfl(p.s, 0), __shfl(p.w, 0), 0.0f};
    p.at = at;
    return p;
}

// A wave per row: its results from its slices' parts.
template <bool ENTROPY>
__global__ __launch_bounds__(THREADS) void finish_kernel(LossArgs a, LossSpace space, int slices) {
    const int64_t row = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    if (row >= a.in.rows) return;
    int token;
    const bool counts = counts_for(a.in, row, token);
    float k, inverse;
    temperature_of(a.in, row, k, inverse);
    const Part p = row_part<ENTROPY>(space, row, slices, k);
    double log_s;
    const RowResult r = result_of<ENTROPY>(a, row, counts, p, inverse, log_s);
    if ((threadIdx.x & 63) == 0) write_result<ENTROPY>(a, row, r, space.exact, space.terms);
}

// A workgroup per (row, slice): the gradient in its logits; the first of a
// row writes the row's results.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void gradient_kernel(LossArgs a, LossSpace space,
                                                           int part_slices, int slices,
                                                           bool results) {
    constexpr int N = Pack<T>::N;
    const int64_t row = blockIdx.x;
    int token;
    const bool counts = counts_for(a.in, row, token);
    float k, inverse;
    temperature_of(a.in, row, k, inverse);
    const T *z = static_cast<const T *>(a.in.logits) + row * a.in.row_stride;
    T *dz = static_cast<T *>(a.grad_logits) + row * a.grad_stride;
    const int size = slice_size(a.in.vocab, slices);
    const int lo = (int)blockIdx.y * size;
    const int end = min(lo + size, a.in.vocab);
    const Part p = row_part<ENTROPY>(space, row, part_slices, k);
    double log_s;
    const RowResult r = result_of<ENTROPY>(a, row, counts, p, inverse, log_s);
    if (results && blockIdx.y == 0 && threadIdx.x == 0)
        write_result<ENTROPY>(a, row, r, nullptr, space.terms);
    // (a row without a gradient in its results has none, whatever it holds)
    const bool any = counts && p.s != 0.0f && (r.alpha != 0.0f || r.eta != 0.0f);
    const float base = base_of(p.m);
    const float per = any ? inverse / p.s : 0.0f;
    const float P = ENTROPY ? -(r.alpha + r.eta * (float)((double)r.entropy - log_s)) * per
                            : -r.alpha * per;
    const float Q = ENTROPY ? -r.eta * (float)LN2 * per : 0.0f;
    const float more = any ? r.alpha * inverse : 0.0f;
    for (int i = lo + (int)threadIdx.x * N; i < end; i += THREADS * N) {
        Pack<T> e = {};
        if (any) {
            e = load_pack(z + i, end - i);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float u = (to_f32(e.v[j]) - base) * k;
                const float x = exp2_of(u);
                float d = ENTROPY ? x * fmaf(Q, factor(u), P) : x * P;
                if (i + j == token) d += more;
                e.v[j] = from_f32<T>(d);
            }
        }
        if (end - i >= N) {
            __builtin_memcpy(dz + i, &e, sizeof(e));
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < end - i) dz[i + j] = e.v[j];
        }
    }
}

// ---------------------------------------------------------- sums of a loss

constexpr int TOTAL_THREADS = 1024;

// The sum over the workgroup, in a fixed order, the same in every thread.
__device__ __forceinline__ double block_sum(double v, double *shared) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    double sum = 0.0;
    for (int q = 0; q < (int)blockDim.x / 64; ++q) sum += shared[q];
    return sum;
}

__global__ __launch_bounds__(TOTAL_THREADS) void total_kernel(const double *terms, int64_t n,
                                                              float *out) {
    __shared__ double shared[TOTAL_THREADS / 64];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += TOTAL_THREADS) sum += terms[i];
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) out[0] = (float)sum;
}

// -------------------------------------------------------------- preference

// Where a sequence starts: the largest offset up to its own, within the rows,
// so that the sequences never overlap.
__device__ __forceinline__ int64_t start_of(const int64_t *offsets, int64_t q, int64_t rows,
                                            double *shared) {
    int64_t top = 0;
    for (int64_t i = threadIdx.x; i <= q; i += blockDim.x) top = max(top, offsets[i]);
    top = min(top, rows);
    int v = wave_max((int)top);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = (double)v;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 64; ++w) v = max(v, (int)shared[w]);
    return v;
}

// A workgroup per pair: the log probabilities of its sequences, its loss, and
// the gradient in the log probability of each of their rows.
__global__ __launch_bounds__(TOTAL_THREADS) void pair_kernel(PreferenceArgs a, LossSpace space) {
    __shared__ double shared[TOTAL_THREADS / 64];
    const int64_t pair = blockIdx.x;
    int64_t begin[2], end[2];
    double sum[2], n[2];
    for (int side = 0; side < 2; ++side) {
        const int64_t q = side * a.pairs + pair;
        begin[side] = start_of(a.offsets, q, a.in.rows, shared);
        end[side] = start_of(a.offsets, q + 1, a.in.rows, shared);
        double total = 0.0, used = 0.0;
        for (int64_t i = begin[side] + threadIdx.x; i < end[side]; i += TOTAL_THREADS) {
            const bool counts = (unsigned)a.in.tokens[i] < (unsigned)a.in.vocab;
            if (counts) used += 1.0;
            if (counts && a.known_margins == nullptr) total += space.exact[i];
        }
        n[side] = a.average ? fmax(block_sum(used, shared), 1.0) : 1.0;
        sum[side] = a.known_margins == nullptr ? block_sum(total, shared) / n[side] : 0.0;
    }
    double h;
    if (a.known_margins) {
        h = (double)a.known_margins[pair];
    } else {
        double rel[2];
        for (int side = 0; side < 2; ++side)
            rel[side] = sum[side] -
                        (a.ref_logprobs ? (double)a.ref_logprobs[side * a.pairs + pair] : 0.0);
        h = (double)a.beta * (rel[0] - rel[1]) - (double)a.margin;
    }
    const double weight = a.weights ? (double)a.weights[pair] : (double)a.weight;
    const double beta = (double)a.beta, smooth = (double)a.smoothing;
    double each, slope;
    if (a.kind == NMS_PREFERENCE_SIGMOID) {
        // log(1 + exp(-h)) and log(1 + exp(h)), one of which is near 0
        const double rest = log1p(exp(-fabs(h)));
        const double up = rest + fmax(-h, 0.0), down = rest + fmax(h, 0.0);
        each = (1.0 - smooth) * up + (smooth > 0.0 ? smooth * down : 0.0);
        slope = smooth * exp(-up) - (1.0 - smooth) * exp(-down);
        if (h != h) each = slope = h;
    } else if (a.kind == NMS_PREFERENCE_HINGE) {
        each = h < 1.0 ? 1.0 - h : h - h;
        slope = h < 1.0 ? -1.0 : h - h;
        if (h > 1.0) each = slope = 0.0;
    } else {
        each = (h - 0.5) / beta * ((h - 0.5) / beta);
        slope = 2.0 * (h - 0.5) / (beta * beta);
    }
    if (weight == 0.0) each = slope = 0.0;
    if (threadIdx.x == 0) {
        space.terms[pair] = weight * each;
        if (a.logprobs) {
            a.logprobs[pair] = (float)sum[0];
            a.logprobs[a.pairs + pair] = (float)sum[1];
        }
        if (a.margins) a.margins[pair] = (float)h;
    }
    if (a.grad_logits == nullptr) return;
    const double up = a.grad_loss ? (double)a.grad_loss[0] : 1.0;
    for (int side = 0; side < 2; ++side) {
        const float alpha = (float)((side ? -1.0 : 1.0) * up * weight * slope * beta / n[side]);
        for (int64_t i = begin[side] + threadIdx.x; i < end[side]; i += TOTAL_THREADS)
            space.alpha[i] = alpha;
    }
    // the rows of no sequence
    if (pair == 0) {
        for (int64_t i = threadIdx.x; i < begin[0]; i += TOTAL_THREADS) space.alpha[i] = 0.0f;
    }
    if (pair == a.pairs - 1) {
        for (int64_t i = end[1] + threadIdx.x; i < a.in.rows; i += TOTAL_THREADS)
            space.alpha[i] = 0.0f;
    }
}

// ----------------------------------------------------------------- launches

// Parts of all rows; their results too where nothing else is to follow.
template <typename T, bool ENTROPY>
void run_parts(const LossArgs &a, const LossSpace &s, int slices, bool results,
               hipStream_t stream) {
    const bool finish = results && slices == 1;
    part_kernel<T, ENTROPY><<<dim3((unsigned)a.in.rows, (unsigned)slices), THREADS, 0, stream>>>(
        a, s, slices, finish);
    if (results && !finish)
        finish_kernel<ENTROPY>
            <<<(unsigned)((a.in.rows + WAVES - 1) / WAVES), THREADS, 0, stream>>>(a, s, slices);
}

template <typename T, bool ENTROPY>
void run_gradient(const LossArgs &a, const LossSpace &s, int slices, bool results,
                  hipStream_t stream) {
    gradient_kernel<T, ENTROPY>
        <<<dim3((unsigned)a.in.rows, (unsigned)slices), THREADS, 0, stream>>>(a, s, slices, slices,
                                                                               results);
}

template <typename T, bool ENTROPY>
void run(const LossArgs &a, hipStream_t stream) {
    LossSpace s;
    lay_out(a.in.rows, a.in.vocab, 0, a.workspace, &s);
    s.exact = nullptr;
    const int slices = slices_of(a.in.rows, a.in.vocab);
    const bool gradient = a.grad_logits != nullptr;
    if (a.loss == nullptr) s.terms = nullptr;
    run_parts<T, ENTROPY>(a, s, slices, !gradient, stream);
    if (gradient)
        run_gradient<T, ENTROPY>(a, s, slices, a.logprobs || a.entropies || a.loss, stream);
}

template <typename T>
void choose(const LossArgs &a, hipStream_t stream) {
    if (a.entropy) run<T, true>(a, stream);
    else run<T, false>(a, stream);
}

template <typename T>
void run_preference(const PreferenceArgs &a, hipStream_t stream) {
    LossSpace s;
    lay_out(a.in.rows, a.in.vocab, a.pairs, a.workspace, &s);
    const int slices = slices_of(a.in.rows, a.in.vocab);
    LossArgs rows = {};
    rows.in = a.in;
    rows.kind = LOSS_LOGPROBS;
    LossSpace first = s;
    first.terms = nullptr;
    if (a.in.rows > 0) run_parts<T, false>(rows, first, slices, a.known_margins == nullptr, stream);
    pair_kernel<<<(unsigned)a.pairs, TOTAL_THREADS, 0, stream>>>(a, s);
    if (a.loss) launch_total(s.terms, a.pairs, a.loss, stream);
    if (a.grad_logits && a.in.rows > 0) {
        rows.kind = LOSS_GIVEN;
        rows.grad_logprobs = s.alpha;
        rows.grad_logits = a.grad_logits;
        rows.grad_stride = a.grad_stride;
        run_gradient<T, false>(rows, first, slices, false, stream);
    }
}

}  // namespace

size_t loss_workspace_bytes(int64_t rows, int vocab, int64_t pairs) {
    return lay_out(rows, vocab, pairs, nullptr, nullptr) + 256;
}

void launch_total(const double *terms, int64_t n, float *out, hipStream_t stream) {
    total_kernel<<<1, TOTAL_THREADS, 0, stream>>>(terms, n, out);
}

hipError_t launch_loss(const LossArgs &a, hipStream_t stream) {
    if (a.in.rows > 0) {
        if (a.in.dtype == NMS_F32) choose<float>(a, stream);
        else if (a.in.dtype == NMS_F16) choose<half_t>(a, stream);
        else choose<bf16_t>(a, stream);
    }
    if (a.loss) {
        LossSpace s;
        lay_out(a.in.rows, a.in.vocab, 0, a.workspace, &s);
        launch_total(s.terms, a.in.rows, a.loss, stream);
    }
    return hipGetLastError();
}

hipError_t launch_preference(const PreferenceArgs &a, hipStream_t stream) {
    if (a.in.dtype == NMS_F32) run_preference<float>(a, stream);
    else if (a.in.dtype == NMS_F16) run_preference<half_t>(a, stream);
    else run_preference<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
