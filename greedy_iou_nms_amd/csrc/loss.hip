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
// So a row is looked through for its (m, s, w), which join by rescaling, and then
// for its gradient.  Memory is the bound: 16.2 vector instructions an element for
// both, by counters, are 60 % of the vector units' time where rows are read and
// written at a copy's rate (with entropies 10.5 for the sums, 81 % where rows are
// only read).
// Hence
//   * row_kernel, a workgroup that holds a row in its registers in between: logits
//     are read once and the gradient is written once, 4096 x 131072 bfloat16 in 385
//     to 413 us for 2.04 GB, where a copy takes 393;
//   * part_kernel and gradient_kernel, which read a row twice: where a loss needs
//     all rows before any gradient (preference), where the rows are few and a row is
//     shared by workgroups, and, the first alone, for results of long rows (4097 x
//     131072 with entropies 190 us, 5.6 TB/s).
#include "loss_internal.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr double LN2 = 0.693147180559945309;

// -------------------------------------------------------------------- rows

// The largest logit m of a part of a row, the sum s of the exponentials and the
// weighted sum w.  m may be -infinity (no logit above it); then s and w are 0,
// or NaN where one was NaN.  s is a sum in binary64 of float32 exponentials:
// where the largest logit, 1 of the sum, is the token's, log s is what the others
// add to 1, and float32 loses 2^-25 with each (of log probabilities around -0.01
// 6e-6 of the value for 6e-8).  With the other steps to that end it cost 389 -> 395
// us for a policy step of 4096 x 131072, and with entropies of 1003 x 150001 186 ->
// 195.
// at: the logit of the row's token, which a gradient in place of the logits
// overwrites.
struct Part {
    double s, w;
    float m, at;
};

// Sixteen bytes of neighbouring elements, as words: as elements of 16 bits they
// would take a register each.
template <typename T>
struct Pack {
    static constexpr int N = 16 / sizeof(T);
    uint32_t w[4];
};

__device__ __forceinline__ float element(const Pack<float> &e, int j) {
    return __uint_as_float(e.w[j]);
}
__device__ __forceinline__ float element(const Pack<bf16_t> &e, int j) {
    const uint32_t w = e.w[j / 2];
    return __uint_as_float(j % 2 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float element(const Pack<half_t> &e, int j) {
    const uint32_t w = e.w[j / 2];
    return (float)__builtin_bit_cast(half_t, (uint16_t)(j % 2 ? w >> 16 : w));
}

__device__ __forceinline__ void set_elements(Pack<float> &e, const float *v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e.w[j] = __float_as_uint(v[j]);
}
template <typename T>
__device__ __forceinline__ void set_elements(Pack<T> &e, const float *v) {
    typedef T Two __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < 4; ++j)
        e.w[j] = __builtin_bit_cast(uint32_t, (Two){(T)v[2 * j], (T)v[2 * j + 1]});
}

typedef uint32_t Words __attribute__((ext_vector_type(4), may_alias));
typedef uint32_t LooseWords __attribute__((ext_vector_type(4), aligned(2), may_alias));

// The pack at an aligned address, or one of -infinity.  STREAM: it is not read
// again, and does not stay in the caches.
template <bool STREAM, typename T>
__device__ __forceinline__ Pack<T> load_pack(const T *p, bool there) {
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u
                          : __is_same(T, half_t) ? 0xfc00fc00u : 0xff80ff80u;
    Words w = {none, none, none, none};
    if (there) {
        const Words *from = reinterpret_cast<const Words *>(p);
        w = STREAM ? __builtin_nontemporal_load(from) : *from;
    }
    return {{w.x, w.y, w.z, w.w}};
}

// To any element's address.  STREAM: it does not stay in the caches, where it
// would take the place of logits that are still to be read.
template <bool STREAM, typename T>
__device__ __forceinline__ void store_pack(T *p, const Pack<T> &e) {
    const LooseWords w = {e.w[0], e.w[1], e.w[2], e.w[3]};
    LooseWords *to = reinterpret_cast<LooseWords *>(p);
    if (STREAM) __builtin_nontemporal_store(w, to);
    else *to = w;
}

// log2(e) / t as a sum, whose second term keeps sums over many rows unbiased
// (the first alone is off by up to 2^-23 of u, 2^-26 at a temperature of 1, in one
// direction for all rows), and 1 / t, in binary64: for t below 2^-128 float32 does
// not hold it.  The second term is above 0, so that -infinity times it is -infinity.
struct Scale {
    float hi, lo;
    double inverse;
};

// A temperature of 0 or below (or NaN) stands for 1; a scale beyond float32
// takes the largest or smallest that float32 has, so that the largest logit keeps
// 2^0 and -infinity stays out.
__device__ __forceinline__ Scale scale_of(const LossRows &r, int64_t row) {
    constexpr double LOG2E = 1.4426950408889634;
    constexpr float ONE = 1.44269502f, REST = (float)(LOG2E - (double)ONE);
    static_assert((double)ONE < LOG2E, "the rest is above 0");
    float t = r.temperature ? r.temperature[row] : 1.0f;
    if (!(t > 0.0f) || t == 1.0f) return {ONE, REST, 1.0};
    constexpr float LEAST = 1.4012985e-45f, MOST = 3.4028235e38f;
    const double k = LOG2E / (double)t;
    float hi = fminf(fmaxf((float)k, LEAST), MOST);
    // the next float below where it was rounded up
    if ((double)hi > k && hi > LEAST) hi = __uint_as_float(__float_as_uint(hi) - 1u);
    float lo = fmaxf((float)(k - (double)hi), LEAST);
    if (hi == MOST) lo = LEAST;
    return {hi, lo, k * LN2};
}

// A row's logits: a body of whole packs at aligned addresses, and the elements
// before and behind it, fewer than two packs, which threads take one each.  (Packs
// at odd elements of 16 bits took 20 % longer: 4096 x 131073 float16 255 us for
// 211 read, 541 for 440 read and written; and branches for a pack that is not
// whole, at each pack that a thread holds, made 256 x 32000 27.7 us for 25.6 as the
// kernel was then; now it takes 11.3.)
template <typename T>
struct Row {
    const T *z;       // the body
    int size;         // of the body
    int head, edges;  // elements before it; before and behind it
    int token;        // its place from the body on
    __device__ __forceinline__ Row(const LossRows &r, int64_t row, int of) {
        constexpr int N = Pack<T>::N;
        z = static_cast<const T *>(r.logits) + row * r.row_stride;
        const int past = (int)(reinterpret_cast<uintptr_t>(z) & 15) / (int)sizeof(T);
        head = min((N - past) & (N - 1), r.vocab);
        z += head;
        size = (r.vocab - head) & ~(N - 1);
        edges = r.vocab - size;
        token = of - head;
    }
    __device__ __forceinline__ float at_token() const { return to_f32(z[token]); }
    __device__ __forceinline__ int edge(int j) const { return j < head ? j - head : size + j - head; }
    // the part of the thread's element at the edges, or an empty one
    __device__ __forceinline__ Part first(bool mine) const {
        Part p = {0.0, 0.0, NEG_INF, 0.0f};
        if (mine && (int)threadIdx.x < edges) {
            const float v = to_f32(z[edge(threadIdx.x)]);
            if (v != NEG_INF) p.s = 1.0 + (double)(v - v);  // NaN of NaN and infinity
            if (v == v) p.m = v;
        }
        return p;
    }
};

// The difference to a largest logit that may be -infinity.
__device__ __forceinline__ float base_of(float m) { return m == NEG_INF ? 0.0f : m; }

__device__ __forceinline__ float exp2_of(float u) { return __builtin_amdgcn_exp2f(u); }

// The maximum of three in one instruction, without quietening them first.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
    return d;
}

// The natural logarithm of a sum that is 0, NaN or from 2^-100 to 2^100: with
// s = 2^n v, v from sqrt(1/2) to sqrt(2) and f = (v - 1) / (v + 1), n ln 2 +
// 2 (f + f^3 / 3 + ... + f^15 / 15); the remainder is below 2 f^17 / 17 =
// 1.2e-14.  The library's takes three times the instructions for the last bits,
// which show where rows are short.
__device__ __forceinline__ double inverse_of(double v) {
    const double y = __builtin_amdgcn_rcp(v);
    const double z = y * __builtin_fma(-v, y, 2.0);
    return z * __builtin_fma(-v, z, 2.0);
}
__device__ __forceinline__ double log_of(double s) {
    const int n = __builtin_amdgcn_frexp_exp(s);
    const double half = __builtin_amdgcn_frexp_mant(s);  // 1/2 .. 1
    const bool low = half < 0.70710678118654752;
    const double v = low ? half + half : half;
    const double f = (v - 1.0) * inverse_of(v + 1.0), g = f * f;
    double p = 2.0 / 15;
    p = __builtin_fma(p, g, 2.0 / 13);
    p = __builtin_fma(p, g, 2.0 / 11);
    p = __builtin_fma(p, g, 2.0 / 9);
    p = __builtin_fma(p, g, 2.0 / 7);
    p = __builtin_fma(p, g, 2.0 / 5);
    p = __builtin_fma(p, g, 2.0 / 3);
    p = __builtin_fma(p, g, 2.0);
    const double y = __builtin_fma((double)(low ? n - 1 : n), LN2, f * p);
    return s > 0.0 ? y : s == 0.0 ? (double)NEG_INF : s;
}

// float16 two at a time, converted at the end
template <int K>
__device__ __forceinline__ float largest_half(float top, const Pack<half_t> *e) {
    Pack<half_t> most = e[0];
#pragma unroll
    for (int q = 0; q < K; ++q)
#pragma unroll
        for (int i = q == 0 ? 1 : 0; i < 4; ++i)
            asm("v_pk_max_f16 %0, %0, %1" : "+v"(most.w[0]) : "v"(e[q].w[i]));
    return max3(top, element(most, 0), element(most, 1));
}

// The largest of some packs' elements and `top`.
template <typename T, int K>
__device__ __forceinline__ float largest(float top, const Pack<T> *e) {
    if constexpr (__is_same(T, half_t)) return largest_half<K>(top, e);
#pragma unroll
    for (int q = 0; q < K; ++q)
#pragma unroll
        for (int j = 0; j < Pack<T>::N; j += 2)
            top = max3(top, element(e[q], j), element(e[q], j + 1));
    return top;
}

// An element less a base, rounded once.
template <typename T>
__device__ __forceinline__ float less(const Pack<T> &e, int j, float base) {
    return element(e, j) - base;
}
// of float16 in one instruction, with its conversion
__device__ __forceinline__ float less(const Pack<half_t> &e, int j, float base) {
    float d;
    if (j % 2)
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
            : "=v"(d) : "v"(e.w[j / 2]), "v"(base));
    else
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[0,0,0] op_sel_hi:[1,0,0]"
            : "=v"(d) : "v"(e.w[j / 2]), "v"(base));
    return d;
}

// v x for an exponential x: 0 where x is, whatever v (x's exponent of -infinity, a
// slope beyond float32), by the multiplication whose product with 0 is 0.  What the
// exponential has just made may be read after a wait only, which the compiler puts
// before its own instructions and not here.
__device__ __forceinline__ float times_exponential(float v, float x) {
    float d;
    asm("s_nop 0\n\tv_mul_legacy_f32 %0, %1, %2" : "=v"(d) : "v"(v), "v"(x));
    return d;
}

// u as a factor of an exponential that is 0 from -150 down
__device__ __forceinline__ float factor(float u) { return fmaxf(u, -200.0f); }

// u of a logit less the largest one.  (With entropies by k.hi alone: w is at hand
// then, and corrects the sum at the end.)
template <bool ENTROPY>
__device__ __forceinline__ float scaled(float d, const Scale &k) {
    return ENTROPY ? d * k.hi : fmaf(d, k.hi, d * k.lo);
}

// What a part's sums are multiplied by, and w's are shifted by, when its
// largest logit becomes top.
struct Shift {
    double by;
    float u;
};
template <bool ENTROPY>
__device__ __forceinline__ Shift shift_to(float m, float top, const Scale &k) {
    const float u = m == NEG_INF ? 0.0f : scaled<ENTROPY>(m - top, k);
    return {(double)exp2_of(u), factor(u)};
}

// The sum of K values by halves.
template <int K>
__device__ __forceinline__ float sum_of(const float *v) {
    float x[K];
#pragma unroll
    for (int j = 0; j < K; ++j) x[j] = v[j];
#pragma unroll
    for (int h = K / 2; h > 0; h /= 2)
#pragma unroll
        for (int j = 0; j < h; ++j) x[j] += x[j + h];
    return x[0];
}

// A thread's next K packs.
template <typename T, bool ENTROPY, int K>
__device__ __forceinline__ void add_packs(Part &p, const Pack<T> *e, const Scale &k) {
    constexpr int N = Pack<T>::N;
    const float top = largest<T, K>(p.m, e);
    const float base = base_of(top);
    const Shift f = shift_to<ENTROPY>(p.m, base, k);
    float w[K];
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < K; ++q) {
        float x[N], y[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float d = less(e[q], j, base);
            const float u = scaled<ENTROPY>(d, k);
            x[j] = exp2_of(u);
            if (ENTROPY) y[j] = times_exponential(u, x[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) sum += (double)x[j];
        if (ENTROPY) w[q] = sum_of<N>(y);
    }
    if (ENTROPY) p.w = (p.w + (double)f.u * p.s) * f.by + (double)sum_of<K>(w);
    p.s = p.s * f.by + sum;
    p.m = top;
}

// The join over the wave's lanes, the same in all of them.
template <bool ENTROPY>
__device__ __forceinline__ Part join_wave(Part p, const Scale &k) {
    const float top = wave_max(p.m);
    const Shift f = shift_to<ENTROPY>(p.m, top, k);
    if (ENTROPY) p.w = wave_sum((p.w + (double)f.u * p.s) * f.by);
    p.s = wave_sum(p.s * f.by);
    p.m = top;
    return p;
}

// The join over a workgroup of WAVES waves, the same in every lane.
template <bool ENTROPY, int WAVES>
__device__ __forceinline__ Part join_group(Part p, const Scale &k, Part *shared) {
    p = join_wave<ENTROPY>(p, k);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = p;
    __syncthreads();
    const int lane = threadIdx.x & 63;
    p = {0.0, 0.0, NEG_INF, 0.0f};
    if (lane < WAVES) p = shared[lane];
    return join_wave<ENTROPY>(p, k);
}

// ---------------------------------------------------------------- results

// What comes with a row besides its logits, read before them, and whether it
// counts.
struct RowGiven {
    int token;
    bool counts;
    float weight, old, advantage, ref, up;  // LOSS_POLICY
    float alpha, eta;                       // LOSS_GIVEN
};

// array[row], or what stands for an array that is not given.  The load is made
// either way, of the row's token in its place, so that all of them are in flight
// together: behind a branch each, or behind the token, they cost a round trip
// each.
__device__ __forceinline__ float parameter(const float *array, int64_t row, float otherwise,
                                           const void *any) {
    const float v = *(array ? array + row : static_cast<const float *>(any));
    return array ? v : otherwise;
}

template <bool ENTROPY>
__device__ __forceinline__ RowGiven given_of(const LossArgs &a, int64_t row) {
    RowGiven r = {};
    const void *any = a.in.tokens + row;
    r.token = a.in.tokens[row];
    r.weight = parameter(a.in.weights, row, a.weight, any);
    r.old = parameter(a.old_logprobs, row, 0.0f, any);
    r.advantage = parameter(a.advantages, row, 0.0f, any);
    r.ref = parameter(a.ref_logprobs, row, 0.0f, any);
    r.up = parameter(a.grad_loss, 0, 1.0f, any);
    r.alpha = parameter(a.grad_logprobs, row, 0.0f, any);
    r.eta = ENTROPY ? parameter(a.grad_entropies, row, 0.0f, any) : 0.0f;
    r.counts = (unsigned)r.token < (unsigned)a.in.vocab;
    if (!r.counts) r.token = -1;  // places are reckoned from it
    if (a.in.weights) r.counts &= r.weight != 0.0f;
    // (a row without a gradient in its results has none, whatever it holds)
    if (a.kind == LOSS_GIVEN) r.counts &= r.alpha != 0.0f || r.eta != 0.0f;
    return r;
}

// exp(q) - 1 - q, where more is exp(q) - 1: near 0 by its series q^2 / 2 (1 + q / 3
// (1 + q / 4 (...))), whose remainder at 1/2 is 2 q^8 / 10! = 2e-9 of it.  The
// difference would be off by 2^-23 / q of its value, and below 0 at times.
__device__ __forceinline__ float past_linear(float q, float more) {
    if (!(fabsf(q) < 0.5f)) return more - q;
    float p = 1.0f;
#pragma unroll
    for (int n = 9; n >= 3; --n) p = fmaf(q * (1.0f / n), p, 1.0f);
    return 0.5f * q * q * p;
}

// One row's results; alpha and eta: the gradients in its log probability and
// entropy, times that of the loss; term: its part of the loss.
struct RowResult {
    float logprob, entropy, alpha, eta;
    double exact, term, log_s;
};

template <bool ENTROPY>
__device__ __forceinline__ RowResult result_of(const LossArgs &a, const RowGiven &given,
                                               const Part &p, const Scale &k) {
    RowResult r = {};
    if (!given.counts) return r;
    // in binary64: sums over rows are made of these
    // (with entropies the exponentials are those of k.hi alone: one of k.hi + k.lo is
    // (1 + ln 2 u k.lo / k.hi) times that, and w is the sum of u times that)
    r.log_s = log_of(ENTROPY ? p.s + LN2 * (double)(k.lo / k.hi) * p.w : p.s);
    r.exact = p.s == 0.0        ? (double)NEG_INF
              : p.at == NEG_INF ? (double)NEG_INF - r.log_s
                                : ((double)p.at - (double)p.m) * k.inverse - r.log_s;
    r.logprob = (float)r.exact;
    if (ENTROPY)
        r.entropy = p.s == 0.0 ? 0.0f : (float)(r.log_s - LN2 * p.w * inverse_of(p.s));
    r.alpha = given.alpha;
    r.eta = given.eta;
    if (a.kind == LOSS_POLICY) {
        const float advantage = given.advantage;
        const float ratio = expf((float)(r.exact - (double)given.old));
        float each = 0.0f, slope = 0.0f;
        if (advantage != 0.0f) {
            const float free = ratio * advantage;
            const float held = fminf(fmaxf(ratio, a.clip_low), a.clip_high) * advantage;
            each = -fminf(free, held);
            slope = free <= held ? -free : 0.0f;
            if (ratio != ratio || advantage != advantage) each = slope = ratio * advantage;
        }
        if (a.ref_logprobs) {
            const float q = (float)((double)given.ref - r.exact);
            const float more = expm1f(q);
            each += a.kl * past_linear(q, more);
            slope -= a.kl * more;
        }
        if (ENTROPY) each -= a.bonus * r.entropy;
        r.term = (double)given.weight * (double)each;
        r.alpha = given.up * given.weight * slope;
        r.eta = -given.up * given.weight * a.bonus;
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

// Slices of a row: two workgroups for each compute unit where rows are few (64 x
// 131072 bfloat16: log probabilities 8.8 us, 11.1 with eight).
inline int slices_of(int64_t rows, int vocab) {
    int64_t n = 512 / (rows < 1 ? 1 : rows);
    const int64_t most = (vocab + 4095) / 4096;
    if (n > most) n = most;
    if (n > MAX_SLICES) n = MAX_SLICES;
    return n < 1 ? 1 : (int)n;
}

__device__ inline int slice_size(int vocab, int slices) {
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

// ---------------------------------------------------------------- gradient

// What makes a row's gradient: dz_j = e_j (P + Q u_j), but for the token's, which
// is made in binary64: where its probability is near 1, it is a difference of
// nearly equal ones.  any: the gradient is not 0.  (A whole word: the bytes behind
// a smaller one were copied through LDS at the thread's number, for which every
// workgroup read the launch's packet in host memory: those of 256 x 32000 started
// over 13 us.)
struct Slope {
    float base, k, P, Q, token;
    int any;
};

template <bool ENTROPY>
__device__ __forceinline__ Slope slope_of(const RowResult &r, const Part &p, const Scale &k,
                                          bool counts) {
    Slope g;
    g.any = counts && p.s != 0.0 && (r.alpha != 0.0f || r.eta != 0.0f);
    g.base = base_of(p.m);
    g.k = k.hi;
    const double per = k.inverse * inverse_of(p.s);
    const double eta = ENTROPY ? (double)r.eta : 0.0;
    const double P = -((double)r.alpha + eta * ((double)r.entropy - r.log_s)) * per;
    const double Q = -eta * LN2 * per;
    const float u = factor((p.at - g.base) * g.k);
    // (of NaN every element's exponential is made NaN: 0 would give 0 in a product
    // with entropies)
    if (P != P || Q != Q) g.base = __uint_as_float(0x7fc00000u);
    g.P = (float)P;
    // (P may be beyond float32, and the gradient then is; but not Q, whose product
    // with the largest logit's exponent of 0 would be NaN)
    constexpr double MOST = 3.4028235e38f;
    g.Q = fabs(Q) < 1e300 ? (float)fmin(fmax(Q, -MOST), MOST) : (float)Q;
    g.token = (float)((double)r.alpha * k.inverse +
                      (double)exp2_of(u) * (P + Q * (double)u));
    return g;
}

// The gradient of one logit that is not the token's, from it less the base: 0
// where its exponential is, also by a P that float32 does not hold.  (u is by k.hi
// alone, which is off by less than 2^-23 of u, 2^-26 at a temperature of 1: about
// what the difference and the product are rounded by.  The second term would be an
// instruction more for each element.)
template <bool ENTROPY>
__device__ __forceinline__ float gradient_of(float less, const Slope &g) {
    const float u = less * g.k;
    const float x = exp2_of(u);
    return times_exponential(ENTROPY ? fmaf(g.Q, u, g.P) : g.P, x);
}

// A pack of logits becomes its gradient, but for what the token's has more.
template <typename T, bool ENTROPY>
__device__ __forceinline__ void to_gradient(Pack<T> &e, const Slope &g) {
    constexpr int N = Pack<T>::N;
    float d[N];
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] = gradient_of<ENTROPY>(less(e, j, g.base), g);
    set_elements(e, d);
}

// As one store of its own, by bytes: it may follow one of a pack to the same place.
template <typename T>
__device__ __forceinline__ void store_one(T *p, float v) {
    const T t = from_f32<T>(v);
    __builtin_memcpy(p, &t, sizeof(t));
}

// The gradients of the elements at the edges, one by each thread.
template <typename T, bool ENTROPY>
__device__ __forceinline__ void write_edges(const Row<T> &r, T *dz, const Slope &g) {
    if ((int)threadIdx.x >= r.edges) return;
    const int i = r.edge(threadIdx.x);
    float d = 0.0f;
    if (g.any) {
        d = i == r.token ? g.token : gradient_of<ENTROPY>(to_f32(r.z[i]) - g.base, g);
    }
    store_one(dz + i, d);
}

// The token's gradient, over what its pack's thread has written there.
template <typename T>
__device__ __forceinline__ void write_token(const Row<T> &r, T *dz, const Slope &g, int lo, int end,
                                            int group) {
    if (r.token >= lo && r.token < end &&
        (int)threadIdx.x == (r.token - lo) / Pack<T>::N % group)
        store_one(dz + r.token, g.token);
}

// ---------------------------------------------------------- sums of a loss

constexpr int TOTAL_THREADS = 1024;

// The sum of n terms by a workgroup of GROUP threads, in a fixed order.
template <int GROUP>
__device__ __forceinline__ void write_total(const double *terms, int64_t n, float *out) {
    __shared__ double shared[GROUP / 64];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += GROUP) sum += terms[i];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int q = 1; q < GROUP / 64; ++q) sum += shared[q];
    out[0] = (float)sum;
}

__global__ __launch_bounds__(TOTAL_THREADS) void total_kernel(const double *terms, int64_t n,
                                                              float *out) {
    write_total<TOTAL_THREADS>(terms, n, out);
}

// ----------------------------------------------------------------- kernels

// A workgroup per (row, slice): the slice's part, and where it is the row's
// only one the row's results.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void part_kernel(LossArgs a, LossSpace space, int slices,
                                                       bool finish) {
    constexpr int N = Pack<T>::N, UNROLL = 32 / N, STEP = THREADS * 32;
    __shared__ Part shared[WAVES];
    const int64_t row = blockIdx.x;
    const RowGiven given = given_of<ENTROPY>(a, row);
    const Scale k = scale_of(a.in, row);
    Part p = {0.0, 0.0, NEG_INF, 0.0f};
    if (given.counts) {
        const Row<T> r(a.in, row, given.token);
        const float at_token = r.at_token();
        const int size = slice_size(r.size, slices);
        const int lo = (int)blockIdx.y * size;
        const int end = min(lo + size, r.size);
        p = r.first(blockIdx.y == 0);
        for (int at = lo; at < end; at += STEP) {
            Pack<T> e[UNROLL];
#pragma unroll
            for (int q = 0; q < UNROLL; ++q) {
                const int i = at + (q * THREADS + (int)threadIdx.x) * N;
                e[q] = load_pack<false>(r.z + i, i < end);
            }
            add_packs<T, ENTROPY, UNROLL>(p, e, k);
        }
        p = join_group<ENTROPY, WAVES>(p, k, shared);
        p.at = at_token;
    }
    if (threadIdx.x != 0) return;
    space.parts[row * slices + blockIdx.y] = p;
    if (finish)
        write_result<ENTROPY>(a, row, result_of<ENTROPY>(a, given, p, k), space.exact,
                              space.terms);
}

// A row's part from those of its slices, the same in every lane.
template <bool ENTROPY>
__device__ __forceinline__ Part row_part(const LossSpace &space, int64_t row, int slices,
                                         const Scale &k) {
    const int lane = threadIdx.x & 63;
    if (slices == 1) return space.parts[row];
    Part p = {0.0, 0.0, NEG_INF, 0.0f};
    if (lane < slices) p = space.parts[row * slices + lane];
    const float at = __shfl(p.at, 0);
    p = join_wave<ENTROPY>(p, k);
    p.at = at;
    return p;
}

// A wave per row: its results from its slices' parts.
template <bool ENTROPY>
__global__ __launch_bounds__(THREADS) void finish_kernel(LossArgs a, LossSpace space, int slices) {
    const int64_t row = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    if (row >= a.in.rows) return;
    const RowGiven given = given_of<ENTROPY>(a, row);
    const Scale k = scale_of(a.in, row);
    const Part p = row_part<ENTROPY>(space, row, slices, k);
    const RowResult r = result_of<ENTROPY>(a, given, p, k);
    if ((threadIdx.x & 63) == 0) write_result<ENTROPY>(a, row, r, space.exact, space.terms);
}

// A workgroup per (row, slice): the gradient in its logits; the first of a
// row writes the row's results.  With `pairs`, workgroups behind the rows' add up
// the terms of so many pairs, which would be a launch of its own else.
template <typename T, bool ENTROPY, bool STREAM>
__global__ __launch_bounds__(THREADS) void gradient_kernel(LossArgs a, LossSpace space,
                                                           int part_slices, int slices,
                                                           bool results, int64_t pairs) {
    constexpr int N = Pack<T>::N;
    if ((int64_t)blockIdx.x >= a.in.rows) {
        if (blockIdx.y == 0) write_total<THREADS>(space.terms, pairs, a.loss);
        return;
    }
    // the rows that were read last are still in the last cache
    const int64_t row = a.in.rows - 1 - blockIdx.x;
    const RowGiven given = given_of<ENTROPY>(a, row);
    const Scale k = scale_of(a.in, row);
    const Row<T> r(a.in, row, given.token);
    T *dz = static_cast<T *>(a.grad_logits) + row * a.grad_stride + r.head;
    const int size = slice_size(r.size, slices);
    const int lo = (int)blockIdx.y * size;
    const int end = min(lo + size, r.size);
    Slope g = {};
    if (given.counts || results) {
        const Part p = row_part<ENTROPY>(space, row, part_slices, k);
        const RowResult result = result_of<ENTROPY>(a, given, p, k);
        if (results && blockIdx.y == 0 && threadIdx.x == 0)
            write_result<ENTROPY>(a, row, result, nullptr, space.terms);
        g = slope_of<ENTROPY>(result, p, k, given.counts);
    }
    if (blockIdx.y == 0) write_edges<T, ENTROPY>(r, dz, g);
    constexpr int SPAN = THREADS * N, UNROLL = 4;
    for (int i = lo + (int)threadIdx.x * N; i < end; i += UNROLL * SPAN) {
        Pack<T> e[UNROLL] = {};
        if (g.any) {
#pragma unroll
            for (int q = 0; q < UNROLL; ++q)
                e[q] = load_pack<STREAM>(r.z + i + q * SPAN, i + q * SPAN < end);
#pragma unroll
            for (int q = 0; q < UNROLL; ++q) to_gradient<T, ENTROPY>(e[q], g);
        }
#pragma unroll
        for (int q = 0; q < UNROLL; ++q)
            if (i + q * SPAN < end) store_pack<STREAM>(dz + i + q * SPAN, e[q]);
    }
    if (g.any) write_token<T>(r, dz, g, lo, end, THREADS);
}

// Waves of a vector unit: as many as leave the registers that the packs and a
// chunk of 16 exponentials need (with entropies also 16 products; chunks of 8
// of them take fewer, but 224 us for 215 at 4096 x 65536 float16).
constexpr int waves_of(bool entropy, int held) {
    return held <= 4 ? 8 - 2 * entropy : held <= 8 ? 6 - entropy : 4;
}

// A workgroup per row: its results and, with GRADIENT, its gradient.  The first
// HELD packs of each thread stay in registers between the two, the others are
// read again.  All of them are asked for at once: a row's time is one trip to
// memory, its two passes of instructions and its results, which other rows of the
// compute unit fill.
template <typename T, bool ENTROPY, bool GRADIENT, bool STREAM, int GROUP, int HELD>
__global__ __launch_bounds__(GROUP, waves_of(ENTROPY, HELD)) void row_kernel(LossArgs a,
                                                                             LossSpace space) {
    constexpr int N = Pack<T>::N, UNROLL = 16 / N, SPAN = GROUP * N;
    constexpr int CHUNK = HELD < UNROLL ? HELD : UNROLL;
    static_assert(HELD % CHUNK == 0, "whole chunks");
    __shared__ Part shared[GROUP / 64];
    __shared__ Slope slope;
    // the rows that were read or written last are still in the last cache
    const int64_t row = GRADIENT ? (int64_t)gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int first = (int)threadIdx.x * N;
    const RowGiven given = given_of<ENTROPY>(a, row);
    const Row<T> r(a.in, row, given.token);
    const int V = r.size;
    T *dz = static_cast<T *>(a.grad_logits) + row * a.grad_stride + r.head;
    Pack<T> held[HELD];
    Slope g = {};
    if (given.counts) {
        const float at_token = r.at_token();
#pragma unroll
        for (int c = 0; c < HELD; c += CHUNK)
            if (c == 0 || c * SPAN < V) {
#pragma unroll
                for (int q = c; q < c + CHUNK; ++q)
                    held[q] = load_pack<STREAM>(r.z + q * SPAN + first, q * SPAN + first < V);
            }
        const Scale k = scale_of(a.in, row);
        Part p = r.first(true);
#pragma unroll
        for (int c = 0; c < HELD; c += CHUNK)
            if (c == 0 || c * SPAN < V) add_packs<T, ENTROPY, CHUNK>(p, held + c, k);
        for (int i = HELD * SPAN + first; i < V; i += UNROLL * SPAN) {
            Pack<T> e[UNROLL];
#pragma unroll
            for (int q = 0; q < UNROLL; ++q)
                e[q] = load_pack<false>(r.z + i + q * SPAN, i + q * SPAN < V);
            add_packs<T, ENTROPY, UNROLL>(p, e, k);
        }
        p = GROUP == 64 ? join_wave<ENTROPY>(p, k) : join_group<ENTROPY, GROUP / 64>(p, k, shared);
        p.at = at_token;
        if (threadIdx.x < 64) {
            const RowResult result = result_of<ENTROPY>(a, given, p, k);
            g = slope_of<ENTROPY>(result, p, k, true);
            if (threadIdx.x == 0) {
                write_result<ENTROPY>(a, row, result, space.exact, space.terms);
                if (!GRADIENT && space.parts) space.parts[row] = p;
                if (GRADIENT && GROUP > 64) slope = g;
            }
        }
        if (GRADIENT && GROUP > 64) {
            __syncthreads();
            g = slope;
        }
    } else if (threadIdx.x == 0) {
        write_result<ENTROPY>(a, row, RowResult{}, space.exact, space.terms);
        if (!GRADIENT && space.parts) space.parts[row] = {0.0, 0.0, NEG_INF, 0.0f};
    }
    if (!GRADIENT) return;
    write_edges<T, ENTROPY>(r, dz, g);
    if (!g.any) {
        for (int i = first; i < V; i += SPAN) store_pack<STREAM>(dz + i, Pack<T>{});
        return;
    }
#pragma unroll
    for (int q = 0; q < HELD; ++q) {
        const int i = q * SPAN + first;
        if (q == 0 || q * SPAN < V) {
            to_gradient<T, ENTROPY>(held[q], g);
            if (i < V) store_pack<STREAM>(dz + i, held[q]);
        }
    }
    for (int i = HELD * SPAN + first; i < V; i += SPAN) {
        Pack<T> e = load_pack<STREAM>(r.z + i, true);
        to_gradient<T, ENTROPY>(e, g);
        store_pack<STREAM>(dz + i, e);
    }
    write_token<T>(r, dz, g, 0, V, GROUP);
}

// -------------------------------------------------------------- preference

// What the waves of a pair's workgroup tell each other.
struct PairShared {
    int top[TOTAL_THREADS / 64][2];
    double sum[TOTAL_THREADS / 64][2], used[TOTAL_THREADS / 64][2];
    float alpha[2];
};

// A workgroup per pair: the log probabilities of its sequences, its loss, and
// the gradient in the log probability of each of their rows.
__global__ __launch_bounds__(TOTAL_THREADS) void pair_kernel(PreferenceArgs a, LossSpace space) {
    __shared__ PairShared shared;
    constexpr int WAVES = TOTAL_THREADS / 64;
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t pair = blockIdx.x, other = a.pairs + pair;
    const bool forward = a.known_margins == nullptr;
    // A sequence starts at the largest offset up to its own, within the rows, so
    // that the sequences never overlap.
    const int64_t next[2] = {a.offsets[pair + 1], a.offsets[other + 1]};
    int64_t top[2] = {0, 0};
    for (int64_t i = tid; i <= other; i += TOTAL_THREADS) {
        const int64_t at = a.offsets[i];
        if (i <= pair) top[0] = max(top[0], at);
        top[1] = max(top[1], at);
    }
    for (int side = 0; side < 2; ++side) {
        const int v = wave_max((int)min(top[side], a.in.rows));
        if ((tid & 63) == 0) shared.top[wave][side] = v;
    }
    __syncthreads();
    int begin[2] = {0, 0}, end[2];
    for (int side = 0; side < 2; ++side) {
        for (int w = 0; w < WAVES; ++w) begin[side] = max(begin[side], shared.top[w][side]);
        end[side] = max(begin[side], (int)min(max(next[side], (int64_t)0), a.in.rows));
    }
    for (int side = 0; side < 2; ++side) {
        double sum = 0.0, used = 0.0;
        for (int i = begin[side] + tid; i < end[side]; i += TOTAL_THREADS) {
            const bool counts = (unsigned)a.in.tokens[i] < (unsigned)a.in.vocab;
            if (counts) used += 1.0;
            if (counts && forward) sum += space.exact[i];
        }
        sum = wave_sum(sum);
        used = wave_sum(used);
        if ((tid & 63) == 0) {
            shared.sum[wave][side] = sum;
            shared.used[wave][side] = used;
        }
    }
    __syncthreads();
    if (tid == 0) {
        double l[2], n[2];
        for (int side = 0; side < 2; ++side) {
            double sum = 0.0, used = 0.0;
            for (int w = 0; w < WAVES; ++w) {
                sum += shared.sum[w][side];
                used += shared.used[w][side];
            }
            n[side] = a.average ? fmax(used, 1.0) : 1.0;
            l[side] = sum / n[side];
        }
        double h;
        if (forward) {
            const float *ref = a.ref_logprobs;
            const double first = l[0] - (ref ? (double)ref[pair] : 0.0);
            const double second = l[1] - (ref ? (double)ref[other] : 0.0);
            h = (double)a.beta * (first - second) - (double)a.margin;
        } else {
            h = (double)a.known_margins[pair];
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
        space.terms[pair] = weight * each;
        if (a.logprobs) {
            a.logprobs[pair] = (float)l[0];
            a.logprobs[other] = (float)l[1];
        }
        if (a.margins) a.margins[pair] = (float)h;
        const double up = a.grad_loss ? (double)a.grad_loss[0] : 1.0;
        const double by = slope == 0.0 ? 0.0 : up * weight * slope * beta;
        shared.alpha[0] = (float)(by / n[0]);
        shared.alpha[1] = (float)(-by / n[1]);
    }
    if (a.grad_logits == nullptr) return;
    __syncthreads();
    for (int side = 0; side < 2; ++side)
        for (int i = begin[side] + tid; i < end[side]; i += TOTAL_THREADS)
            space.alpha[i] = shared.alpha[side];
    // the rows of no sequence
    if (pair == 0)
        for (int i = tid; i < begin[0]; i += TOTAL_THREADS) space.alpha[i] = 0.0f;
    if (pair == a.pairs - 1)
        for (int64_t i = end[1] + tid; i < a.in.rows; i += TOTAL_THREADS) space.alpha[i] = 0.0f;
}

// ----------------------------------------------------------------- launches

int64_t row_bytes(const LossRows &in) {
    return (int64_t)in.vocab * (in.dtype == NMS_F32 ? 4 : 2);
}

// Whether a workgroup takes a whole row and holds it, for results alone.  Rows
// up to 64 KB: 64 x 32000 bfloat16 5.2 us, 6.3 by slices in two launches; 16384 x
// 2000 14 us, 42 by a workgroup of 256 that reads on.  Up to 128 KB from 64 rows
// on: 256 x 65536 10.0 us, 12.6 by slices (one row: 6.6 and 5.3).  Longer rows
// take all registers of a compute unit, so that reading one row waits for the
// one before: 4096 x 131072 218 us, 200 by workgroups of 256 that read on.
bool held_for_results(const LossRows &in) {
    return row_bytes(in) <= 65536 || (row_bytes(in) <= 131072 && in.rows >= 64);
}

// For the gradient, which slices read a second time: policy loss of 256 x 131072
// bfloat16 30.7 us, 39.4 by slices; of 4096 x 131072 401 and 559.  Few long rows
// leave the GPU empty: 16 x 131072 19.8 and 10.3, 64 x 131072 22.6 and 17.0, 96
// even; 16 x 65536 12.4 and 9.0, 64 x 65536 13.8 and 15.8.
bool held_for_gradient(const LossRows &in) {
    return row_bytes(in) <= 65536 || in.rows >= (row_bytes(in) <= 131072 ? 64 : 96);
}

// Threads and packs by the row's size; what 1024 threads do not hold (of rows
// above 256 KB) is read a second time.  Rows of 4000 bfloat16 took 48 us for
// 16384 with 128 threads, 60 with 64 and 53 with 256; of 32000 101 us for 4096 with
// 512, 109 with 256; of 65536 201 with 1024 of 8 packs, 219 with 1024 of 16.
template <typename T, bool ENTROPY, bool GRADIENT, bool STREAM>
void launch_rows(const LossArgs &a, const LossSpace &s, hipStream_t stream) {
    const unsigned n = (unsigned)a.in.rows;
    const int64_t bytes = row_bytes(a.in);
    if (bytes <= 4096)
        row_kernel<T, ENTROPY, GRADIENT, STREAM, 64, 4><<<n, 64, 0, stream>>>(a, s);
    else if (bytes <= 16384)
        row_kernel<T, ENTROPY, GRADIENT, STREAM, 128, 8><<<n, 128, 0, stream>>>(a, s);
    else if (bytes <= 65536)
        row_kernel<T, ENTROPY, GRADIENT, STREAM, 512, 8><<<n, 512, 0, stream>>>(a, s);
    else if (bytes <= 131072)
        row_kernel<T, ENTROPY, GRADIENT, STREAM, 1024, 8><<<n, 1024, 0, stream>>>(a, s);
    else if constexpr (GRADIENT)
        row_kernel<T, ENTROPY, GRADIENT, STREAM, 1024, 16><<<n, 1024, 0, stream>>>(a, s);
}

// Logits of more bytes than this pass the caches when they are read for the last
// time, and so does their gradient.  What was read of them before, or is yet
// to be, stays there: preference loss of 8192 x 32000 bfloat16 189 us, 248
// without, of 4001 x 131072 507 and 574; policy loss of 4096 x 131072 389 and
// 399, of 3000 x 32000 (183 MB) 66 and 80, but of 1024 x 32000 31 and 28.  Below,
// whatever comes next finds the gradient in the caches; where logits are read
// twice (2048 x 32000, 125 MB: 63 and 73 us) they are streamed earlier.
constexpr int64_t STREAMED_ONCE = (int64_t)160 << 20, STREAMED_TWICE = (int64_t)96 << 20;

template <typename T, bool ENTROPY>
void run_rows(const LossArgs &a, const LossSpace &s, hipStream_t stream) {
    if (a.in.rows * row_bytes(a.in) > STREAMED_ONCE)
        launch_rows<T, ENTROPY, true, true>(a, s, stream);
    else
        launch_rows<T, ENTROPY, true, false>(a, s, stream);
}

// The parts of all rows, and with `results` their results.  Returns the number
// of parts of a row.
template <typename T, bool ENTROPY>
int run_parts(const LossArgs &a, const LossSpace &s, bool results, hipStream_t stream) {
    if (held_for_results(a.in)) {
        launch_rows<T, ENTROPY, false, false>(a, s, stream);
        return 1;
    }
    const int slices = slices_of(a.in.rows, a.in.vocab);
    const bool finish = results && slices == 1;
    part_kernel<T, ENTROPY><<<dim3((unsigned)a.in.rows, (unsigned)slices), THREADS, 0, stream>>>(
        a, s, slices, finish);
    if (results && !finish)
        finish_kernel<ENTROPY>
            <<<(unsigned)((a.in.rows + WAVES - 1) / WAVES), THREADS, 0, stream>>>(a, s, slices);
    return slices;
}

// The gradient from the parts; pairs: of those whose terms make a.loss.
template <typename T, bool ENTROPY>
void run_gradient(const LossArgs &a, const LossSpace &s, int parts, bool results, int64_t pairs,
                  hipStream_t stream) {
    const int slices = slices_of(a.in.rows, a.in.vocab);
    const dim3 grid((unsigned)(a.in.rows + (pairs > 0)), (unsigned)slices);
    if (a.in.rows * row_bytes(a.in) > STREAMED_TWICE)
        gradient_kernel<T, ENTROPY, true>
            <<<grid, THREADS, 0, stream>>>(a, s, parts, slices, results, pairs);
    else
        gradient_kernel<T, ENTROPY, false>
            <<<grid, THREADS, 0, stream>>>(a, s, parts, slices, results, pairs);
}

template <typename T, bool ENTROPY>
void run(const LossArgs &a, hipStream_t stream) {
    LossSpace s;
    lay_out(a.in.rows, a.in.vocab, 0, a.workspace, &s);
    s.exact = nullptr;
    if (a.loss == nullptr) s.terms = nullptr;
    if (a.grad_logits == nullptr) {
        run_parts<T, ENTROPY>(a, s, true, stream);
    } else if (held_for_gradient(a.in)) {
        run_rows<T, ENTROPY>(a, s, stream);
    } else {
        const int parts = run_parts<T, ENTROPY>(a, s, false, stream);
        run_gradient<T, ENTROPY>(a, s, parts, a.logprobs || a.entropies || a.loss, 0, stream);
    }
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
    LossArgs rows = {};
    rows.in = a.in;
    rows.kind = LOSS_LOGPROBS;
    LossSpace of_rows = s;
    of_rows.terms = nullptr;
    const bool forward = a.known_margins == nullptr, some = a.in.rows > 0;
    int parts = 1;
    if (forward && some) parts = run_parts<T, false>(rows, of_rows, true, stream);
    pair_kernel<<<(unsigned)a.pairs, TOTAL_THREADS, 0, stream>>>(a, s);
    if (a.grad_logits == nullptr || !some) {
        if (forward) launch_total(s.terms, a.pairs, a.loss, stream);
        return;
    }
    rows.kind = LOSS_GIVEN;
    rows.grad_logprobs = s.alpha;
    rows.grad_logits = a.grad_logits;
    rows.grad_stride = a.grad_stride;
    if (forward) {
        rows.loss = a.loss;
        run_gradient<T, false>(rows, s, parts, false, a.pairs, stream);
    } else {
        of_rows.exact = nullptr;
        if (held_for_gradient(a.in)) {
            run_rows<T, false>(rows, of_rows, stream);
        } else {
            parts = run_parts<T, false>(rows, of_rows, false, stream);
            run_gradient<T, false>(rows, of_rows, parts, false, 0, stream);
        }
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
