// Picking the next token of every row from its adjusted logits.
//
// Two launches.  slice_kernel: one workgroup per (row, slice of the
// vocabulary) adjusts the slice once (adjust_core.h), keeps its values in
// registers, and writes those among which its largest max_top_k are, with the
// slice's part of the softmax sum (a maximum and a sum relative to it).
// join_kernel: one workgroup per row takes the largest max_top_k of all
// slices, sorts them, and draws.
//
// A candidate is a 64-bit word: the order-preserving key of its value above,
// the complement of its token below, so that the words of a row are all
// different and their descending order is the order of the definition (equal
// values by ascending token).  0 is no candidate.
#include "adjust_core.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr int JT = 1024;     // threads of the join
constexpr int JCAP = 2 * JT; // candidates that the join sorts
constexpr int BINS = 512;    // of the histograms that bound the k-th value
static_assert(NMS_MAX_TOP_K <= JT, "a candidate per thread once they are sorted");

struct Part {
    float top;       // the slice's largest value
    float edge;      // no candidate of the slice is below
    uint32_t count;  // candidates written
    double sum;      // of exp((value - top) / temperature)
};

// Candidates a slice may write: more than max_top_k, because the bound that
// they are above is below the max_top_k-th value (or equal to it).
__host__ __device__ constexpr int slice_cap(int k) { return k + k / 2 + 16; }

__device__ __forceinline__ uint64_t candidate(float z, int token) {
    const uint32_t k = order_key(z);
    return k == 0u ? 0ull : ((uint64_t)k << 32) | (uint32_t)~token;
}

// The temperature of the softmax: greedy rows (0, or anything not above it)
// use 1.
__device__ __forceinline__ float warmth(const float *temperature, int64_t row) {
    const float t = temperature ? temperature[row] : 1.0f;
    return t > 0.0f ? t : 1.0f;
}

// z - top, with the limit 0 at z = top = +infinity.
__device__ __forceinline__ double below_top(float z, float top) {
    return z == top ? 0.0 : (double)z - (double)top;
}

// The bin of v in [lo, hi], monotone in v: lo in bin 0, hi at most in the
// last.
struct Bins {
    float lo, scale;
    __device__ __forceinline__ Bins(float lo_, float hi, int bins) : lo(lo_) {
        const float width = hi - lo_;
        scale = width > 0.0f ? (float)bins / width : 0.0f;
        if (!(scale < 3.0e38f)) scale = 3.0e38f;
    }
    __device__ __forceinline__ int of(float v, int bins) const {
        // v = lo gives 0 whatever the scale; an overflow ends in the last bin
        return (int)fminf((v - lo) * scale, (float)(bins - 1));
    }
};

// The highest bin at or above which there are at least `need` entries, and
// -1 if there are fewer in all.  One wave; hist has 64 * PER bins.
template <int PER>
__device__ __forceinline__ int bin_of_rank(const uint32_t *hist, uint32_t need) {
    const int lane = threadIdx.x & 63;
    uint32_t c[PER], s = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = hist[lane * PER + i];
        s += c[i];
    }
    // entries in this lane's bins and above: an inclusive sum from the top
    uint32_t above = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_down(above, d);
        if (lane + d < 64) above += v;
    }
    const uint64_t enough = __ballot(above >= need);
    if (enough == 0ull) return -1;
    const int at = 63 - __builtin_clzll(enough);
    int bin = -1;
    uint32_t sum = above - s;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
        sum += c[i];
        if (bin < 0 && sum >= need) bin = lane * PER + i;
    }
    return __shfl(bin, at);
}

// ------------------------------------------------------------------- slices

// VALUES per thread in groups of eight neighbouring tokens; GROUP of them
// share an entry in the histogram (their largest).
template <typename T, int THREADS, int VALUES, int GROUP>
__global__ __launch_bounds__(THREADS) void slice_kernel(PickArgs a, int slices, Part *parts,
                                                        uint64_t *found) {
    constexpr int SLICE = THREADS * VALUES;
    constexpr int WAVES = THREADS / 64;
    __shared__ uint32_t word[SLICE];
    __shared__ uint32_t hist[BINS], low[BINS];
    __shared__ float wave_top[WAVES], wave_low[WAVES];
    __shared__ float wave_sums[WAVES];
    __shared__ uint32_t bound_key, taken, chosen[2];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t row = blockIdx.x / slices;
    const int lo = (int)(blockIdx.x % slices) * SLICE;
    const int size = min(SLICE, a.vocab - lo);
    const RowRules r = row_rules(a.rules, row);
    const float c = fminf(1.4426950408889634f / warmth(a.temperature, row), 3.0e38f);
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + lo;
    for (int i = tid; i < BINS; i += THREADS) {
        hist[i] = 0;
        low[i] = 0xffffffffu;
    }
    if (tid == 0) taken = 0;
    if (r.words) slice_rules<T, THREADS, SLICE>(a.rules, r, row, lo, size, in, word);
    float z[VALUES];
#pragma unroll
    for (int g = 0; g < VALUES / 8; ++g)
        adjusted8<T, SLICE>(r, lo, size, 8 * (g * THREADS + tid), in, word, z + 8 * g);
    // v_max drops a NaN
    float m[VALUES / GROUP], top = NEG_INF, least = __builtin_inff();
#pragma unroll
    for (int g = 0; g < VALUES / GROUP; ++g) {
        m[g] = z[g * GROUP];
        if (!(m[g] > NEG_INF)) m[g] = NEG_INF;
#pragma unroll
        for (int j = 1; j < GROUP; ++j) m[g] = fmaxf(m[g], z[g * GROUP + j]);
        top = fmaxf(top, m[g]);
        if (m[g] > NEG_INF) least = fminf(least, m[g]);
    }
    top = wave_max(top);
    least = -wave_max(-least);
    // the softmax sum, relative to the wave's largest value
    float sum = 0.0f;
    if (top == __builtin_inff()) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) sum += z[j] == top ? 1.0f : 0.0f;
    } else if (top > NEG_INF) {
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            const float e = __builtin_amdgcn_exp2f((z[j] - top) * c);
            sum += z[j] > NEG_INF ? e : 0.0f;
        }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) {
        wave_top[wave] = top;
        wave_low[wave] = least;
        wave_sums[wave] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        top = fmaxf(top, wave_top[w]);
        least = fminf(least, wave_low[w]);
    }
    const int k = a.max_top_k, cap = slice_cap(k);
    const Bins bins(least, top, BINS);
#pragma unroll
    for (int g = 0; g < VALUES / GROUP; ++g)
        if (m[g] > NEG_INF) {
            const int b = bins.of(m[g], BINS);
            atomicAdd(&hist[b], 1u);
            atomicMin(&low[b], order_key(m[g]));
        }
    __syncthreads();
    if (wave == 0) {
        const int b = bin_of_rank<BINS / 64>(hist, (uint32_t)k);
        // fewer groups than k: every value is a candidate
        if (tid == 0) bound_key = b < 0 ? 1u : low[b];
    }
    __syncthreads();
    // at least k values (or all there are) lie at the bound or above
    const uint32_t bound = bound_key;
    float edge = bound <= 1u ? -3.402823466e38f : key_value(bound);
    uint64_t *to = found + (int64_t)blockIdx.x * cap;
#pragma unroll
    for (int j = 0; j < VALUES; ++j)
        if (z[j] >= edge) {
            const uint32_t at = atomicAdd(&taken, 1u);
            if (at < (uint32_t)cap)
                to[at] = candidate(z[j], lo + 8 * ((j / 8) * THREADS + tid) + j % 8);
        }
    __syncthreads();
    if (taken > (uint32_t)cap) {
        // Equal values, or a spread that the bins do not resolve: the k-th
        // largest word, digit by digit from the top, and exactly k of them.
        uint64_t prefix = 0, mask = 0;
        uint32_t left = (uint32_t)k;
        for (int shift = 56; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += THREADS) hist[i] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                const uint64_t w = candidate(z[j], lo + 8 * ((j / 8) * THREADS + tid) + j % 8);
                if (w != 0 && (w & mask) == prefix) atomicAdd(&hist[(w >> shift) & 255], 1u);
            }
            __syncthreads();
            if (wave == 0) {
                const int d = bin_of_rank<4>(hist, left);
                uint32_t over = 0;
                for (int i = d + 1 + (tid & 63); i < 256; i += 64) over += hist[i];
                over = wave_sum(over);
                if (tid == 0) {
                    chosen[0] = (uint32_t)d;
                    chosen[1] = left - over;
                }
            }
            if (tid == 0) taken = 0;
            __syncthreads();
            prefix |= (uint64_t)chosen[0] << shift;
            mask |= 255ull << shift;
            left = chosen[1];
        }
#pragma unroll
        for (int j = 0; j < VALUES; ++j) {
            const uint64_t w = candidate(z[j], lo + 8 * ((j / 8) * THREADS + tid) + j % 8);
            if (w >= prefix) to[atomicAdd(&taken, 1u)] = w;
        }
        edge = key_value((uint32_t)(prefix >> 32));
        __syncthreads();
    }
    if (tid == 0) {
        double all = 0.0;
        for (int w = 0; w < WAVES; ++w)
            if (wave_top[w] > NEG_INF)
                all += (double)wave_sums[w] *
                       (wave_top[w] == top ? 1.0
                                           : (double)__builtin_amdgcn_exp2f((wave_top[w] - top) * c));
        parts[blockIdx.x] = Part{top, edge, taken, all};
    }
}

// --------------------------------------------------------------------- join

// Descending sort of E * JT words over the workgroup, word t + JT * e in
// thread t; only the first `n` (a power of two, 64 at least) take part.  Steps
// within a wave are shuffles, between waves they go through LDS.
template <int E>
__device__ __forceinline__ void sort_words(uint64_t *v, int n, uint64_t *lds) {
    const int tid = threadIdx.x;
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            if (E == 2 && step == JT) {
                const uint64_t x = v[0], y = v[E - 1];
                v[0] = x > y ? x : y;
                v[E - 1] = x > y ? y : x;
                continue;
            }
            uint64_t other[E];
            if (step >= 64) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) lds[tid + JT * e] = v[e];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) other[e] = lds[(tid ^ step) + JT * e];
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) other[e] = __shfl_xor((unsigned long long)v[e], step);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = tid + JT * e;
                // the larger word goes to the lower place in a descending run
                const bool larger = ((i & size) == 0) == ((i & step) == 0);
                if ((other[e] > v[e]) == larger) v[e] = other[e];
            }
        }
}

__global__ __launch_bounds__(JT) void join_kernel(PickArgs a, int slices, const Part *parts,
                                                  const uint64_t *found) {
    constexpr int WAVES = JT / 64;
    constexpr int HELD = 12;  // pieces of 64 candidates that a wave keeps in registers
    __shared__ uint64_t list[JCAP];
    __shared__ double scan[JT];
    __shared__ uint32_t hist[JT];
    __shared__ double wave_d[WAVES];
    __shared__ float wave_f[3][WAVES];
    __shared__ int wave_i[4][WAVES];
    __shared__ uint32_t taken, chosen[2];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int kmax = a.max_top_k, cap = slice_cap(kmax);
    parts += row * slices;
    found += row * slices * cap;
    // The slices' candidates in pieces of 64, one piece per wave at a time: a
    // wave's first pieces are loaded once, further ones (many slices of many
    // candidates) again for every pass over them.  A place past a slice's
    // count is read but not used.
    const int pieces = (cap + 63) / 64, total = slices * pieces;
    auto load = [&](int p) -> uint64_t {
        if (p >= total) return 0;
        const int s = p / pieces, i = (p - s * pieces) * 64 + lane;
        const uint32_t count = parts[s].count;
        const uint64_t w = i < cap ? found[(int64_t)s * cap + i] : 0ull;
        return (uint32_t)i < count ? w : 0ull;
    };
    uint64_t held[HELD];
#pragma unroll
    for (int q = 0; q < HELD; ++q) held[q] = load(q * WAVES + wave);
    auto each = [&](auto f) {
#pragma unroll
        for (int q = 0; q < HELD; ++q)
            if (held[q] != 0) f(held[q]);
        for (int p = HELD * WAVES + wave; p < total; p += WAVES) {
            const uint64_t w = load(p);
            if (w != 0) f(w);
        }
    };
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const float warm = warmth(a.temperature, row);
    // The row's largest value; a bound that its max_top_k-th value is not
    // below (any slice's with so many candidates), or one below them all.
    float top = NEG_INF, edge = NEG_INF, least = __builtin_inff();
    for (int s = tid; s < slices; s += JT) {
        const Part x = parts[s];
        top = fmaxf(top, x.top);
        if (x.count >= (uint32_t)kmax) edge = fmaxf(edge, x.edge);
        if (x.count > 0) least = fminf(least, x.edge);
    }
    top = wave_max(top);
    edge = wave_max(edge);
    least = -wave_max(-least);
    if (lane == 0) {
        wave_f[0][wave] = top;
        wave_f[1][wave] = edge;
        wave_f[2][wave] = least;
    }
    hist[tid] = 0;
    if (tid == 0) taken = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        top = fmaxf(top, wave_f[0][w]);
        edge = fmaxf(edge, wave_f[1][w]);
        least = fminf(least, wave_f[2][w]);
    }
    if (!(top > NEG_INF)) {
        if (tid == 0) {
            a.ids[row] = -1;
            a.logprobs[row] = NEG_INF;
        }
        return;
    }
    if (!(edge > NEG_INF)) edge = least;
    // the candidates at the bound or above, as far as the list holds them
    each([&](uint64_t w) {
        if (key_value((uint32_t)(w >> 32)) >= edge) {
            const uint32_t at = atomicAdd(&taken, 1u);
            if (at < (uint32_t)JCAP) list[at] = w;
        }
    });
    __syncthreads();
    if (taken > (uint32_t)JCAP) {
        // too many: a closer bound, from a histogram between it and the top
        const Bins bins(edge, top, JT);
        each([&](uint64_t w) {
            const float v = key_value((uint32_t)(w >> 32));
            if (v >= edge) atomicAdd(&hist[bins.of(v, JT)], 1u);
        });
        __syncthreads();
        if (wave == 0) {
            const int b = bin_of_rank<JT / 64>(hist, (uint32_t)kmax);
            uint32_t inside = 0;
            for (int i = b + lane; i < JT; i += 64) inside += hist[i];
            inside = wave_sum(inside);
            if (lane == 0) {
                chosen[0] = (uint32_t)b;
                chosen[1] = inside;
                taken = 0;
            }
        }
        __syncthreads();
        const int b = (int)chosen[0];
        if (chosen[1] <= (uint32_t)JCAP) {
            each([&](uint64_t w) {
                const float v = key_value((uint32_t)(w >> 32));
                if (v >= edge && bins.of(v, JT) >= b) list[atomicAdd(&taken, 1u)] = w;
            });
        } else {
            // as in the slices: the k-th largest word, digit by digit
            uint64_t prefix = 0, mask = 0;
            uint32_t left = (uint32_t)kmax;
            for (int shift = 56; shift >= 0; shift -= 8) {
                __syncthreads();
                if (tid < 256) hist[tid] = 0;
                __syncthreads();
                each([&](uint64_t w) {
                    if ((w & mask) == prefix) atomicAdd(&hist[(w >> shift) & 255], 1u);
                });
                __syncthreads();
                if (wave == 0) {
                    const int d = bin_of_rank<4>(hist, left);
                    uint32_t over = 0;
                    for (int i = d + 1 + lane; i < 256; i += 64) over += hist[i];
                    over = wave_sum(over);
                    if (lane == 0) {
                        chosen[0] = (uint32_t)d;
                        chosen[1] = left - over;
                    }
                }
                __syncthreads();
                prefix |= (uint64_t)chosen[0] << shift;
                mask |= 255ull << shift;
                left = chosen[1];
            }
            each([&](uint64_t w) {
                if (w >= prefix) list[atomicAdd(&taken, 1u)] = w;
            });
        }
        __syncthreads();
    }
    const int listed = (int)taken;
    uint64_t v[2];
    v[0] = tid < listed ? list[tid] : 0ull;
    v[1] = JT + tid < listed ? list[JT + tid] : 0ull;
    if (listed > JT) {
        sort_words<2>(v, JCAP, list);
    } else {
        int p = 64;
        while (p < listed) p <<= 1;
        sort_words<1>(v, p, list);
    }
    const uint64_t mine = v[0];

    int k = a.top_k ? a.top_k[row] : kmax;
    k = min(max(k, 1), kmax);
    const bool there = tid < k && mine != 0;
    const float z = key_value((uint32_t)(mine >> 32));
    const double w = there ? exp(below_top(z, top) / (double)warm) : 0.0;
    // running sums of the candidates' weights
    double cum = w;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(cum, d);
        if (lane >= d) cum += up;
    }
    // the softmax sum over the whole vocabulary, relative to the top
    double sum = 0.0;
    for (int s = tid; s < slices; s += JT)
        if (parts[s].top > NEG_INF)
            sum += parts[s].sum * exp(below_top(parts[s].top, top) / (double)warm);
    sum = wave_sum(sum);
    __syncthreads();
    if (lane == 63) wave_d[wave] = cum;
    if (lane == 0) scan[wave] = sum;
    __syncthreads();
    double all = 0.0, before = 0.0;
    sum = 0.0;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) {
        if (x == wave) before = all;
        all += wave_d[x];
        sum += scan[x];
    }
    cum += before;
    const double top_p = a.top_p ? (double)a.top_p[row] : 1.0;
    const double min_p = a.min_p ? (double)a.min_p[row] : 0.0;
    const int in_k = __popcll(__ballot(there));
    const int in_p = __popcll(__ballot(there && cum < top_p * all));
    const int in_m = __popcll(__ballot(there && w >= min_p));
    __syncthreads();
    scan[tid] = cum;
    if (lane == 0) {
        wave_i[0][wave] = in_k;
        wave_i[1][wave] = in_p;
        wave_i[2][wave] = in_m;
    }
    __syncthreads();
    int count = 0, short_n = 1, large_n = 0;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) {
        count += wave_i[0][x];
        short_n += wave_i[1][x];
        large_n += wave_i[2][x];
    }
    const int keep = max(1, min(min(short_n, large_n), count));
    const double bound = (double)a.uniform[row] * scan[keep - 1];
    const int passed = __popcll(__ballot(tid < keep && cum <= bound));
    if (lane == 0) wave_i[3][wave] = passed;
    __syncthreads();
    int j = 0;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) j += wave_i[3][x];
    j = t > 0.0f ? min(j, keep - 1) : 0;
    if (tid == j) {
        a.ids[row] = (int32_t)~(uint32_t)mine;
        a.logprobs[row] = (float)(below_top(z, top) / (double)warm - log(sum));
    }
}

// Whether a row is split into slices of 16384 tokens, or of 2048 so that
// small batches fill the GPU.
bool wide_slices(int64_t rows, int vocab) { return rows * ((vocab + 16383) / 16384) >= 256; }

int slices_of(int64_t rows, int vocab) {
    const int slice = wide_slices(rows, vocab) ? 16384 : 2048;
    return (vocab + slice - 1) / slice;
}

size_t parts_bytes(int64_t rows, int slices) {
    return ((size_t)rows * slices * sizeof(Part) + 255) / 256 * 256;
}

template <typename T, int THREADS, int VALUES, int GROUP>
void run_slices(const PickArgs &a, int slices, Part *parts, uint64_t *found, hipStream_t stream) {
    slice_kernel<T, THREADS, VALUES, GROUP>
        <<<(unsigned)(a.rows * slices), THREADS, 0, stream>>>(a, slices, parts, found);
}

template <typename T>
void run(const PickArgs &a, hipStream_t stream) {
    const int slices = slices_of(a.rows, a.vocab);
    Part *parts = static_cast<Part *>(a.workspace);
    uint64_t *found = reinterpret_cast<uint64_t *>(static_cast<char *>(a.workspace) +
                                                   parts_bytes(a.rows, slices));
    // Groups of the histogram: at least four for each of max_top_k, so that
    // the k-th largest group bounds the k-th value closely (of values without
    // order about 1.15 k lie above it).
    if (wide_slices(a.rows, a.vocab)) {
        if (a.max_top_k <= 256) run_slices<T, 1024, 16, 16>(a, slices, parts, found, stream);
        else run_slices<T, 1024, 16, 4>(a, slices, parts, found, stream);
    } else {
        if (a.max_top_k <= 64) run_slices<T, 256, 8, 8>(a, slices, parts, found, stream);
        else run_slices<T, 256, 8, 1>(a, slices, parts, found, stream);
    }
    join_kernel<<<(unsigned)a.rows, JT, 0, stream>>>(a, slices, parts, found);
}

}  // namespace

size_t pick_workspace_bytes(int64_t rows, int vocab, int max_top_k) {
    const int slices = slices_of(rows, vocab);
    return parts_bytes(rows, slices) + (size_t)rows * slices * slice_cap(max_top_k) * 8;
}

hipError_t launch_pick(const PickArgs &a, hipStream_t stream) {
    if (a.dtype == NMS_F32) run<float>(a, stream);
    else if (a.dtype == NMS_F16) run<half_t>(a, stream);
    else run<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
