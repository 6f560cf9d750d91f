// Picking the next token of every row from its adjusted logits.
//
// Two steps.  slice_kernel: one workgroup per (row, slice of the
// vocabulary) adjusts the slice once (adjust_core.h), keeps its values in
// registers, and writes those among which its largest max_top_k are, with the
// slice's part of the softmax sum (a maximum and a sum relative to it).
// join_kernel: one workgroup per row takes the largest max_top_k of all
// slices, sorts them, and draws.  whole_kernel does both in one launch.
//
// A candidate is a 64-bit word: the order-preserving key of its value above,
// the complement of its token below, so that the words of a row are all
// different and their descending order is the order of the definition (equal
// values by ascending token).  0 is no candidate.
#include "adjust_core.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr int BINS = 512;         // of a slice's histogram
// Values from here down, masks by a type's lowest value or by -10000, do not
// count for a slice's bound: its bins would begin there and hold all others in
// one.  (A slice with too few values above it takes the long way.)  64 rows of
// 131072 with 90 % of the tokens at -10000 take 16 us so, and 32 with them
// (50 candidates; without any masked 16).
constexpr float MASKED = -4096.0f;
constexpr int JOIN_BINS = 1024;   // of the join's
constexpr int JOIN_HELD = 12;     // pieces of 64 candidates that a wave of it holds
constexpr int CROWDED = 64;       // most candidates of a bin that it ranks one by one

// What a slice says about itself.  edge[i]: at least max_top_k / 2^i (rounded
// up) of its values are not below; -infinity if it has fewer.
constexpr int EDGES = 4;
struct Part {
    float top;       // the slice's largest value
    uint32_t count;  // candidates written
    double sum;      // of exp((value - top) / temperature)
    float edge[EDGES];
    float least;     // no candidate is below
    float pad;
};

// Candidates a slice may write: more than max_top_k, because the bound that
// they are above is below the max_top_k-th value (or equal to it).
__host__ __device__ constexpr int slice_cap(int k) { return k + k / 2 + 16; }

// The word of a value above -infinity.
__device__ __forceinline__ uint64_t candidate_of(float z, int token) {
    const int u = __float_as_int(z + 0.0f);
    return (uint64_t)(uint32_t)(u ^ ((u >> 31) | (int)0x80000000)) << 32 | (uint32_t)~token;
}

// The largest of four, in two instructions: fmaxf takes two more to quieten its
// operands.  A NaN may go through.
__device__ __forceinline__ float max4(float a, float b, float c, float d) {
    float m;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
    asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(m), "v"(d));
    return m;
}

// The temperature of the softmax: greedy rows (0, or anything not above it)
// use 1.
__device__ __forceinline__ float warmth(float t) { return t > 0.0f ? t : 1.0f; }

// z - top, with the limit 0 at z = top = +infinity, and finite, so that an
// infinite temperature makes every quotient 0.  In binary64: two float32 values
// may lie further apart than float32 reaches.
__device__ __forceinline__ double below_top(float z, float top) {
    return z == top ? 0.0 : fmax((double)z - (double)top, -1.7976931348623157e308);
}

// The bin of v in [lo, hi], monotone in v: lo in bin 0, hi at most in the
// last.
struct Bins {
    float lo, scale;
    __device__ __forceinline__ Bins(float lo_, float hi, int bins) : lo(lo_) {
        const float width = hi - lo_;
        scale = width > 0.0f ? (float)bins * __builtin_amdgcn_rcpf(width) : 0.0f;
        if (!(scale < 3.0e38f)) scale = 3.0e38f;
    }
    __device__ __forceinline__ int of(float v, int bins) const {
        // v = lo gives 0 whatever the scale; an overflow ends in the last bin
        return (int)fminf((v - lo) * scale, (float)(bins - 1));
    }
    // Not above any value of bin b or higher, and not far below (-1: below
    // every value).  v in such a bin has (v - lo) * scale >= b after two
    // roundings, of 2^-24 each; the subtracted parts cover these and the
    // roundings here.
    __device__ __forceinline__ float edge(int b) const {
        if (b <= 0 || !(scale > 0.0f)) return b < 0 || !(lo > -3.4e38f) ? -3.402823466e38f : lo;
        const float up = (float)b / scale;
        return fmaxf(lo, (lo + up) - (fabsf(lo) + up) * 0x1p-20f);
    }
};

// A wave's view of a histogram of 64 * PER bins from the top.
template <int PER>
struct Ranks {
    uint32_t c[PER], s, above;
    __device__ __forceinline__ explicit Ranks(const uint32_t *hist) : s(0) {
        const int lane = threadIdx.x & 63;
        // lane 0 has the highest bins
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = hist[64 * PER - 1 - lane * PER - i];
            s += c[i];
        }
        above = wave_scan(s);
    }
    // The highest bin at or above which there are at least `need` entries,
    // and -1 if there are fewer in all.
    __device__ __forceinline__ int bin(uint32_t need) const {
        const int lane = threadIdx.x & 63;
        const uint64_t enough = __ballot(above >= need);
        if (enough == 0ull) return -1;
        int at = -1;
        uint32_t sum = above - s;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            sum += c[i];
            if (at < 0 && sum >= need) at = 64 * PER - 1 - lane * PER - i;
        }
        return __builtin_amdgcn_readlane(at, __builtin_ctzll(enough));
    }
};

// One more in hist[bin] for every lane that is in.  The lanes that agree with
// the first one add once for all: equal values would else queue for a bin.
// Called by whole waves.
__device__ __forceinline__ void count_bin(uint32_t *hist, bool in, uint32_t bin) {
    const uint64_t all = __ballot(in);
    if (all == 0ull) return;
    const int leader = __builtin_ctzll(all);
    const uint32_t its = (uint32_t)__builtin_amdgcn_readlane((int)bin, leader);
    const uint64_t same = __ballot(in && bin == its);
    if ((int)(threadIdx.x & 63) == leader) atomicAdd(&hist[its], (uint32_t)__popcll(same));
    else if (in && bin != its) atomicAdd(&hist[bin], 1u);
}

// One digit of a k-th largest word: chosen[0] is the digit of the word that
// is `left`-th largest among those counted in hist[0..256), chosen[1] its rank
// among those with this digit.  One wave.
__device__ __forceinline__ void digit_of_rank(const uint32_t *hist, uint32_t left,
                                              uint32_t *chosen) {
    const int lane = threadIdx.x & 63;
    const int d = Ranks<4>(hist).bin(left);
    uint32_t over = 0;
    for (int i = d + 1 + lane; i < 256; i += 64) over += hist[i];
    over = wave_sum(over);
    if (lane == 0) {
        chosen[0] = (uint32_t)d;
        chosen[1] = left - over;
    }
}

// ------------------------------------------------------------------- slices

// VALUES per thread in groups of eight neighbouring tokens; GROUP of them
// share an entry in the histogram (their largest).  FIRST is for max_top_k = 1:
// the slice's first largest token, without a histogram (1.1 us of a slice's
// 4.8 where little else runs).
template <int THREADS, int VALUES>
struct SliceSpace {  // in LDS
    RuleSpace<THREADS * VALUES> rules;  // their words then hold the values
    uint32_t hist[BINS];
    float wave_top[THREADS / 64], wave_sums[THREADS / 64];
    float bound[EDGES];
    unsigned long long greatest;
    int highest, lowest;  // as ordered()
    uint32_t taken, chosen[3];
};

// The candidates of a slice whose bound lets too many through (equal values,
// masks of the type's lowest value, largest values side by side): of the values
// in x.rules.word those among which the k largest are, at most cap.  Their keys
// are between low and high; each round counts all keys of the range in BINS
// parts and goes on in the part with the k-th, until what lies at or above it
// fits, or it is a single key, four rounds at most.  Then its first tokens are
// taken, so many as are missing.  Returns how many it wrote; x.chosen[0] is the
// smallest one's key.  64 rows of 131072 with 50 candidates take 47 us where
// all but 40 tokens have the type's lowest value, and 29 where the rows are
// sorted (16 at random); a radix selection of the 64-bit words took 245 and 91.
template <int THREADS, int VALUES>
__device__ __forceinline__ uint32_t narrowed(SliceSpace<THREADS, VALUES> &x, uint32_t low,
                                             uint32_t high, int k, int cap, int lo,
                                             uint64_t *found) {
    constexpr int WAVES = THREADS / 64, PARTS = VALUES / 8;
    static_assert(PARTS * WAVES <= 64 && BINS == 512, "a lane per total, nine bits per round");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t *word = x.rules.word;
    // f(j, key) with the keys of the thread's tokens
    auto each = [&](auto f) {
#pragma unroll 1
        for (int q = 0; q < VALUES / 4; ++q) {
            float v[4];
            __builtin_memcpy(v, word + slot((unsigned)token_at<THREADS>(4 * q)), 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) f(4 * q + c, order_key(v[c]));
        }
    };
    uint32_t range = high - low, above = 0;
    bool single = range == 0u, fits = false;
    if (single && tid == 0) x.chosen[0] = low;
    while (!single && !fits) {
        const int shift = max(0, 23 - __clz(range | 1u));
        for (int i = tid; i < BINS; i += THREADS) x.hist[i] = 0;
        __syncthreads();
        each([&](int, uint32_t key) {
            const uint32_t d = key - low;
            count_bin(x.hist, d <= range, d >> shift);
        });
        __syncthreads();
        if (wave == 0) {
            const int b = Ranks<BINS / 64>(x.hist).bin((uint32_t)k - above);
            uint32_t over = 0;
            for (int i = b + 1 + lane; i < BINS; i += 64) over += x.hist[i];
            over = wave_sum(over);
            if (lane == 0) {
                x.chosen[0] = low + ((uint32_t)b << shift);
                x.chosen[1] = above + over;
                x.chosen[2] = x.hist[b];
                x.taken = 0;  // (read by all before the first barrier here)
            }
        }
        __syncthreads();
        low = x.chosen[0];
        above = x.chosen[1];
        range = (1u << shift) - 1u;
        single = shift == 0;
        fits = above + x.chosen[2] <= (uint32_t)cap;
    }
    uint32_t equal = 0;  // bit j: the key is low, and not all of them are taken
    each([&](int j, uint32_t key) {
        if (key > low || (fits && key == low))
            found[atomicAdd(&x.taken, 1u)] =
                (uint64_t)key << 32 | (uint32_t)~(lo + token_at<THREADS>(j));
        if (!fits && key == low) equal |= 1u << j;
    });
    if (!fits) {
        // their ranks in the order of the tokens: by part, wave, lane and place
        uint32_t rank[PARTS];
#pragma unroll
        for (int g = 0; g < PARTS; ++g) {
            const uint32_t n = (uint32_t)__popc(equal >> (8 * g) & 255u);
            const uint32_t through = wave_scan(n);
            rank[g] = through - n;
            if (lane == 63) x.hist[g * WAVES + wave] = through;
        }
        __syncthreads();
        const uint32_t total = lane < PARTS * WAVES ? x.hist[lane] : 0u;
        const uint32_t before = wave_scan(total) - total;
        const uint32_t missing = (uint32_t)k - above;
#pragma unroll
        for (int g = 0; g < PARTS; ++g) {
            uint32_t r = rank[g] + (uint32_t)__builtin_amdgcn_readlane((int)before,
                                                                       g * WAVES + wave);
            for (uint32_t bits = equal >> (8 * g) & 255u; bits != 0u && r < missing;
                 bits &= bits - 1u, ++r)
                found[above + r] =
                    (uint64_t)low << 32 |
                    (uint32_t)~(lo + token_at<THREADS>(8 * g + __builtin_ctz(bits)));
        }
    }
    __syncthreads();
    return fits ? x.taken : (uint32_t)k;
}

// Instructions bound it: a wave (1024 tokens) issues 230 for the values, the
// maximum and the softmax sum, 115 more to find 50 candidates, 210 to find
// 1000, 150 for a history of 4096, 20 for biases and 25 for a mask.  256 rows
// of 131072 bfloat16 logits with all of these take 47.7 us, 35 of them issuing,
// where reading the 72 MB takes 10 to 14 (a copy's 7.5 TB/s from cache, 5.1 from
// HBM); 64 rows of 100003 float32 logits with 50 candidates 12.4 us (reading:
// 3.5 to 5).
template <typename T, int THREADS, int VALUES, int GROUP, bool FIRST>
__device__ __forceinline__ void slice(const PickArgs &a, Part *parts, uint64_t *found,
                                      SliceSpace<THREADS, VALUES> &x) {
    constexpr int SLICE = THREADS * VALUES;
    constexpr int WAVES = THREADS / 64;
    uint32_t *word = x.rules.word, *hist = x.hist;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    static_assert(WAVES >= EDGES, "a wave for each bound");
    const int64_t row = blockIdx.x;
    const int64_t part = row * gridDim.y + blockIdx.y;
    const int lo = (int)blockIdx.y * SLICE;
    const int size = min(SLICE, a.vocab - lo);
    // a thread's first entries, before it knows how many are in use
    const FourTokens early = load4(a.rules.history + row * a.rules.history_stride,
                                   wave_entry(), (int)a.rules.history_capacity);
    const RowRules r = row_rules(a.rules, row, a.uniform);
    const float warm = warmth(parameter(a.temperature, row, 1.0f, a.uniform));
    const float c = fminf(1.4426950408889634f / warm, 3.0e38f);
    // exp((z - top) / t) where c, or a product with it, may be out of range
    auto share = [&](float v, float most) {
        return __builtin_amdgcn_exp2f(
            (float)(below_top(v, most) * (1.4426950408889634 / (double)warm)));
    };
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + lo;
    const Raw<T, THREADS, VALUES> raw(r, lo, size, in);
    for (int i = tid; i < BINS; i += THREADS) hist[i] = 0;
    if (tid == 0) {
        x.taken = 0;
        x.greatest = 0;
        x.highest = ordered(NEG_INF);
        x.lowest = ordered(__builtin_inff());
    }
    if (r.words) slice_rules<THREADS, SLICE>(a.rules, r, row, lo, size, early, x.rules);
    else __syncthreads();
    float z[VALUES];
    adjusted<T, THREADS, VALUES>(a.rules, r, row, in, raw, x.rules, z);
    // The groups' largest values and the wave's, and the softmax sum relative
    // to that: exp2(z c - top c), one multiply-add and one exponential a value,
    // where the rounding of top c is a factor of all terms and is taken out of
    // the sum.  A NaN, an infinite top, a c of 0 or a product of 2^24 and more
    // show in the sum or in what is taken out; then, and where c does not reach
    // (temperatures below 4.8e-39), the values are gone over again, with a NaN
    // made -infinity and each difference taken by itself.
    float m[VALUES / GROUP], top, sum;
    for (bool again = false;; again = true) {
        if (again) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) z[j] = z[j] > NEG_INF ? z[j] : NEG_INF;
        }
        top = NEG_INF;
#pragma unroll
        for (int g = 0; g < VALUES / GROUP; ++g) {
            m[g] = z[g * GROUP];
            if (GROUP >= 4) {
#pragma unroll
                for (int j = 0; j < GROUP; j += 4) {
                    const float *v = z + g * GROUP + j;
                    const float w = max4(v[0], v[1], v[2], v[3]);
                    m[g] = j == 0 ? w : fmaxf(m[g], w);
                }
            } else {
#pragma unroll
                for (int j = 1; j < GROUP; ++j) m[g] = fmaxf(m[g], z[g * GROUP + j]);
            }
            top = fmaxf(top, m[g]);
        }
        top = wave_max(top);
        sum = 0.0f;
        if (!again) {
            const float hi = top * c, rest = __builtin_fmaf(top, c, -hi);
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                sum += __builtin_amdgcn_exp2f(__builtin_fmaf(z[j], c, -hi));
            sum = wave_sum(sum) * __builtin_amdgcn_exp2f(-rest);
            if (__builtin_amdgcn_readfirstlane(sum < 3.0e38f && fabsf(rest) <= 1.0f &&
                                               c < 3.0e38f))
                break;
        } else {
#pragma unroll
            for (int j = 0; j < VALUES; ++j)
                if (z[j] > NEG_INF) sum += share(z[j], top);
            sum = wave_sum(sum);
            break;
        }
    }
    if (!FIRST) {
#pragma unroll
        for (int q = 0; q < VALUES / 4; ++q)
            // a copy that can be read by a number of its place
            __builtin_memcpy(word + slot((unsigned)token_at<THREADS>(4 * q)),
                             z + 4 * q, 16);
    }
    int least = ordered(__builtin_inff());
#pragma unroll
    for (int g = 0; g < VALUES / GROUP; ++g)
        if (m[g] > MASKED) least = min(least, ordered(m[g]));
    least = wave_min(least);
    if ((tid & 63) == 0) {
        x.wave_top[wave] = top;
        x.wave_sums[wave] = sum;
        atomicMax(&x.highest, ordered(top));
        atomicMin(&x.lowest, least);
    }
    __syncthreads();
    top = unordered(x.highest);
    const int k = a.max_top_k, cap = slice_cap(k);
    found += part * cap;
    // the slice's softmax sum from its waves', and what else it says; wave 0
    auto finish = [&](uint32_t count, float e0, float e1, float e2, float e3, float least_found) {
        const float wt = tid < WAVES ? x.wave_top[tid & (WAVES - 1)] : NEG_INF;
        double all = 0.0;
        if (wt > NEG_INF)
            all = (double)x.wave_sums[tid & (WAVES - 1)] * (double)share(wt, top);
        all = wave_sum(all);
        if (tid == 0) parts[part] = Part{top, count, all, {e0, e1, e2, e3}, least_found, 0.0f};
    };
    if (FIRST) {
        int mine = 0x7fffffff;
#pragma unroll
        for (int j = VALUES - 1; j >= 0; --j)
            if (z[j] == top) mine = lo + token_at<THREADS>(j);
        // one lane for its wave: many may have it
        if (top > NEG_INF && __ballot(mine != 0x7fffffff) != 0ull) {
            mine = wave_min(mine);
            if ((tid & 63) == 0)
                atomicMax(&x.greatest, (unsigned long long)candidate_of(top, mine));
        }
        __syncthreads();
        if (tid == 0) found[0] = x.greatest;
        if (wave == 0) finish(top > NEG_INF ? 1u : 0u, top, top, top, top, top);
        return;
    }
    const Bins bins(unordered(x.lowest), top, BINS);
#pragma unroll
    for (int g = 0; g < VALUES / GROUP; ++g)
        if (m[g] > MASKED) atomicAdd(&hist[bins.of(m[g], BINS)], 1u);
    __syncthreads();
    if (wave < EDGES) {
        // a wave per bound
        const int b = Ranks<BINS / 64>(hist).bin((uint32_t)(k + (1 << wave) - 1) >> wave);
        if ((tid & 63) == 0) x.bound[wave] = b < 0 ? NEG_INF : bins.edge(b);
    }
    if (tid == 0) x.lowest = ordered(__builtin_inff());
    __syncthreads();
    // at least k values lie at the bound or above; without one, all values
    // are candidates
    const float first = x.bound[0];
    float edge = fminf(fmaxf(first, -3.402823466e38f), 3.402823466e38f);
    constexpr float ZERO_EDGE = -1.0e-38f;
    if (edge == 0.0f) edge = ZERO_EDGE;  // so that -0 is not below it
    // bit j: z[j] >= edge, the sign of a difference that is no NaN
    uint32_t hits = 0;
#pragma unroll
    for (int j = VALUES - 1; j >= 0; --j)
        hits = __builtin_amdgcn_alignbit(hits, __float_as_uint(z[j] - edge), 31);
    hits = ~hits & (uint32_t)((1ull << VALUES) - 1);
    const uint32_t mine = (uint32_t)__popc(hits);
    const uint32_t through = wave_scan(mine);
    const uint32_t wave_hits = last_lane(through);
    uint32_t to = 0;
    if ((tid & 63) == 0) to = atomicAdd(&x.taken, wave_hits);
    to = __builtin_amdgcn_readfirstlane(to);
    if (to >= (uint32_t)cap) hits = 0;  // too many: they are found anew below
    to += through - mine;
    while (hits != 0u) {
        const int j = __builtin_ctz(hits), at = token_at<THREADS>(j);
        hits &= hits - 1u;
        // (what the last wave has too many goes to the last place)
        found[min(to++, (uint32_t)cap - 1u)] =
            candidate_of(__uint_as_float(word[slot((unsigned)at)]), lo + at);
    }
    if (first == NEG_INF) {
        // the smallest of them, which the join's bins begin at
        float low = __builtin_inff();
#pragma unroll
        for (int j = 0; j < VALUES; ++j)
            if (z[j] > NEG_INF) low = fminf(low, z[j]);
        low = wave_min(low);
        if ((tid & 63) == 0) atomicMin(&x.lowest, ordered(low));
    }
    __syncthreads();
    if (first == NEG_INF) edge = unordered(x.lowest);
    uint32_t count = x.taken;
    if (count > (uint32_t)cap) {
        count = narrowed<THREADS, VALUES>(x, order_key(edge == ZERO_EDGE ? 0.0f : edge),
                                          order_key(top), k, cap, lo, found);
        edge = key_value(x.chosen[0]);
    }
    if (wave == 0) finish(count, first, x.bound[1], x.bound[2], x.bound[3], edge);
}

template <typename T, int THREADS, int VALUES, int GROUP, bool FIRST>
__global__ __launch_bounds__(THREADS, 8) void slice_kernel(PickArgs a, Part *parts,
                                                           uint64_t *found) {
    __shared__ SliceSpace<THREADS, VALUES> space;
    slice<T, THREADS, VALUES, GROUP, FIRST>(a, parts, found, space);
}

// --------------------------------------------------------------------- join

// Descending sort of one word per thread over the first n threads (n a power
// of two, 64 at least; the others' words must be 0).  Steps within a wave are
// shuffles, between waves they go through LDS.
__device__ __forceinline__ uint64_t sort_words(uint64_t v, int n, uint64_t *lds) {
    const int tid = threadIdx.x;
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            uint64_t other;
            if (step >= 64) {
                __syncthreads();
                lds[tid] = v;
                __syncthreads();
                other = lds[tid ^ step];
            } else {
                other = __shfl_xor((unsigned long long)v, step);
            }
            // the larger word goes to the lower place in a descending run
            const bool larger = ((tid & size) == 0) == ((tid & step) == 0);
            if ((other > v) == larger) v = other;
        }
    return v;
}

// The row's largest value, its softmax sum relative to that, and a bound that
// its kmax-th value is not below, or failing that one that no candidate is
// below.  2^i slices with kmax / 2^i values each at a bound or above make a
// bound, so it is the 2^i-th largest of the slices' edge[i]: with eight slices
// of like values their eighth lets about kmax candidates through where one
// slice's own kmax-th would let eight times as many.  One wave; a lane has the
// part of slice `lane` already.
struct RowParts {
    float top, edge;
    double sum;
};

__device__ __forceinline__ RowParts join_parts(const Part *parts, int slices, const Part &first,
                                               float warm) {
    const int lane = threadIdx.x & 63;
    RowParts r;
    r.top = first.top;
    float least = first.count > 0 ? first.least : __builtin_inff(), best = first.edge[0];
    for (int s = 64 + lane; s < slices; s += 64) {
        r.top = fmaxf(r.top, parts[s].top);
        if (parts[s].count > 0) least = fminf(least, parts[s].least);
        best = fmaxf(best, parts[s].edge[0]);
    }
    r.top = wave_max(r.top);
    r.sum = first.top > NEG_INF ? first.sum * exp(below_top(first.top, r.top) / (double)warm) : 0.0;
    for (int s = 64 + lane; s < slices; s += 64)
        if (parts[s].top > NEG_INF)
            r.sum += parts[s].sum * exp(below_top(parts[s].top, r.top) / (double)warm);
    r.sum = wave_sum(r.sum);
    r.edge = wave_max(best);
    if (slices > 1) {
        const int level = slices >= 8 ? 3 : slices >= 4 ? 2 : 1;
        const float e1 = first.edge[1], e2 = first.edge[2], e3 = first.edge[3];
        float e = level == 3 ? e3 : level == 2 ? e2 : e1;
        float m = NEG_INF;
        for (int i = 0; i < 1 << level; ++i) {
            m = wave_max(e);
            if (lane == __builtin_ctzll(__ballot(e == m))) e = NEG_INF;
        }
        r.edge = fmaxf(r.edge, m);
    }
    if (!(r.edge > NEG_INF)) r.edge = wave_min(least);
    return r;
}

// The part of slice `lane`, or an empty one.
__device__ __forceinline__ Part lane_part(const Part *parts, int slices) {
    const int lane = threadIdx.x & 63;
    Part p = parts[min(lane, slices - 1)];
    if (lane >= slices) {
        p.top = NEG_INF;
        p.count = 0;
#pragma unroll
        for (int i = 0; i < EDGES; ++i) p.edge[i] = NEG_INF;
    }
    return p;
}

template <int THREADS>
struct JoinSpace {  // in LDS
    uint64_t list[THREADS + CROWDED + 4], sorted[THREADS];
    // per bin: its count of held candidates, then its first place; its count
    // of the rest, then the next place of the rest; and its end
    uint32_t hist[JOIN_BINS], rest[JOIN_BINS], ends[JOIN_BINS];
    RowParts whole;
    double wave_d[4], kept;
    uint32_t wave_u[THREADS / 64];
    int wave_i[3][4];
    uint32_t taken, crowded, inside, chosen[2];
};

// Latency bounds it, a chain of loads, seven barriers and the exponentials:
// 6.6 us for 64 rows with 50 candidates, of which 1.8 are the loads and 1 the
// slices' sums.  256 rows with 1000 candidates of each of 8 slices take 15.4
// us, 5 of them to read the 19 MB of candidates.
template <int THREADS>
__device__ __forceinline__ void join(const PickArgs &a, int64_t row, int slices, uint32_t inverse,
                                     const Part *parts, const uint64_t *found,
                                     JoinSpace<THREADS> &x) {
    constexpr int WAVES = THREADS / 64;
    constexpr int HELD = JOIN_HELD;
    constexpr int PER = JOIN_BINS / THREADS;  // bins per thread
    constexpr int DRAW = THREADS / 256;       // candidates per thread that draws
    constexpr int LIST = THREADS + CROWDED;
    uint64_t *list = x.list, *sorted = x.sorted;
    uint32_t *hist = x.hist, *rest = x.rest, *ends = x.ends;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kmax = a.max_top_k, cap = slice_cap(kmax);
    parts += row * slices;
    found += row * slices * cap;
    const Part first = lane_part(parts, slices);
    // The slices' candidates in pieces of 64, one piece per wave at a time: a
    // wave's first pieces are loaded once, further ones (many slices of many
    // candidates) again for every pass over them.  Loads are made without a
    // branch, from a place that exists, so that all are in flight together;
    // what lies past a slice's count is read but not used.
    const int pieces = (cap + 63) / 64, total = slices * pieces;
    auto load = [&](int p) -> uint64_t {
        const int q = min(p, total - 1);
        // q / pieces: exact for q < 2^21 and pieces < 2^6
        const int s = inverse == 0u ? q : (int)__umulhi((uint32_t)q, inverse);
        const int i = (q - s * pieces) * 64 + lane;
        const uint64_t w = found[(int64_t)s * cap + min(i, cap - 1)];
        return p < total && (uint32_t)i < parts[s].count ? w : 0ull;
    };
    uint64_t held[HELD];
#pragma unroll
    for (int q = 0; q < HELD; ++q) held[q] = load(q * WAVES + wave);
    // f is called with every candidate, and with 0 in their places' rest
    auto each_rest = [&](auto f) {
        for (int p = HELD * WAVES + wave; p < total; p += WAVES) f(load(p));
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int q = 0; q < HELD; ++q)
            if (q * WAVES < total) f(held[q]);
        each_rest(f);
    };
    // the row's parameters, in flight with the candidates
    const float t = parameter(a.temperature, row, 1.0f, a.uniform);
    const float warm = warmth(t);
    const double top_p = (double)parameter(a.top_p, row, 1.0f, a.uniform);
    const double min_p = (double)parameter(a.min_p, row, 0.0f, a.uniform);
    const double uniform = (double)a.uniform[row];
    const int k = min(max(parameter(a.top_k, row, kmax, a.uniform), 1), kmax);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        hist[i * THREADS + tid] = 0;
        rest[i * THREADS + tid] = 0;
    }
    if (tid == 0) {
        x.taken = 0;
        x.crowded = 0;
    }
    sorted[tid] = 0;
    for (int i = tid; i < LIST; i += THREADS) list[i] = 0;
    if (wave == 0) {
        const RowParts r = join_parts(parts, slices, first, warm);
        if (lane == 0) x.whole = r;
    }
    __syncthreads();
    const float top = x.whole.top, edge = x.whole.edge;
    if (!(top > NEG_INF)) {
        if (tid == 0) {
            a.ids[row] = -1;
            a.logprobs[row] = NEG_INF;
        }
        return;
    }
    // Counting sort by bins between the bound and the top, then by rank
    // within a bin; bins that start at rank kmax or later are left out.  A held
    // candidate keeps the number it arrived with.
    const Bins bins(edge, top, JOIN_BINS);
    auto value = [](uint64_t w) { return key_value((uint32_t)(w >> 32)); };
    uint32_t arrival[HELD];
#pragma unroll
    for (int q = 0; q < HELD; ++q) {
        uint32_t n = 0;
        if (held[q] != 0 && value(held[q]) >= edge)
            n = atomicAdd(&hist[bins.of(value(held[q]), JOIN_BINS)], 1u);
        arrival[q] = n;
    }
    each_rest([&](uint64_t w) {
        if (w != 0 && value(w) >= edge) atomicAdd(&rest[bins.of(value(w), JOIN_BINS)], 1u);
    });
    __syncthreads();
    // bins in descending order: thread i has those from JOIN_BINS - 1 - i * PER
    uint32_t held_count[PER], all_count[PER], bin_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = JOIN_BINS - 1 - tid * PER - i;
        held_count[i] = hist[b];
        all_count[i] = held_count[i] + rest[b];
        bin_sum += all_count[i];
    }
    uint32_t start = wave_scan(bin_sum);
    if (lane == 63) x.wave_u[wave] = start;
    __syncthreads();
    start -= bin_sum;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) start += w < wave ? x.wave_u[w] : 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = JOIN_BINS - 1 - tid * PER - i;
        hist[b] = start;
        rest[b] = start + held_count[i];
        if (start < (uint32_t)kmax && all_count[i] > (uint32_t)CROWDED) x.crowded = 1;
        start += all_count[i];
        ends[b] = start;
    }
    if (tid == THREADS - 1) x.inside = start;
    __syncthreads();
    if (x.crowded == 0) {
        // a bin that starts before kmax ends before LIST
#pragma unroll
        for (int q = 0; q < HELD; ++q)
            if (held[q] != 0 && value(held[q]) >= edge) {
                const uint32_t at = hist[bins.of(value(held[q]), JOIN_BINS)];
                if (at < (uint32_t)kmax) list[at + arrival[q]] = held[q];
            }
        each_rest([&](uint64_t w) {
            if (w != 0 && value(w) >= edge) {
                const int b = bins.of(value(w), JOIN_BINS);
                if (hist[b] < (uint32_t)kmax) list[atomicAdd(&rest[b], 1u)] = w;
            }
        });
        __syncthreads();
        for (int i = tid; i < LIST; i += THREADS) {
            const uint64_t w = list[i];
            if (w == 0) break;
            const int b = bins.of(value(w), JOIN_BINS);
            uint32_t rank = hist[b];
            // four at a time, of which the last may lie past the bin
            for (uint32_t y = rank, last = ends[b]; y < last; y += 4)
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
                    rank += list[y + c] > w && y + c < last ? 1u : 0u;
            if (rank < (uint32_t)THREADS) sorted[rank] = w;
        }
    } else {
        // Many values that are equal or nearly so: the kmax-th largest word,
        // digit by digit, and a sort of those from there up.
        uint64_t prefix = 0, mask = 0;
        uint32_t left = (uint32_t)kmax;
        if (x.inside <= (uint32_t)kmax) {
            prefix = 1;
        } else {
            for (int shift = 56; shift >= 0; shift -= 8) {
                __syncthreads();
                if (tid < 256) hist[tid] = 0;
                __syncthreads();
                each([&](uint64_t w) {
                    count_bin(hist, w != 0 && (w & mask) == prefix, (uint32_t)(w >> shift) & 255u);
                });
                __syncthreads();
                if (wave == 0) digit_of_rank(hist, left, x.chosen);
                __syncthreads();
                prefix |= (uint64_t)x.chosen[0] << shift;
                mask |= 255ull << shift;
                left = x.chosen[1];
            }
        }
        each([&](uint64_t w) {
            if (w >= prefix && value(w) >= edge) list[atomicAdd(&x.taken, 1u)] = w;
        });
        __syncthreads();
        int p = 64;
        while (p < (int)x.taken) p <<= 1;
        const uint64_t mine = sort_words(list[tid], p, list);
        sorted[tid] = mine;
    }
    __syncthreads();

    // The draw: four waves, or the first alone if it holds all candidates.
    const bool single = kmax <= 64 * DRAW;
    if (wave >= (single ? 1 : 4)) return;
    uint64_t mine[DRAW];
    bool there[DRAW];
    double w[DRAW], cum[DRAW], run = 0.0;
    int in_k = 0, in_m = 0;
#pragma unroll
    for (int i = 0; i < DRAW; ++i) {
        mine[i] = sorted[tid * DRAW + i];
        there[i] = tid * DRAW + i < k && mine[i] != 0;
        w[i] = there[i] ? exp(below_top(value(mine[i]), top) / (double)warm) : 0.0;
        run += w[i];
        cum[i] = run;
        in_k += __popcll(__ballot(there[i]));
        in_m += __popcll(__ballot(there[i] && w[i] >= min_p));
    }
    // running sums of the candidates' weights
    const double through = wave_scan(run);
    double before = through - run, all = last_lane(through);
    if (!single) {
        if (lane == 0) {
            x.wave_d[wave] = all;
            x.wave_i[0][wave] = in_k;
            x.wave_i[1][wave] = in_m;
        }
        __syncthreads();
        all = 0.0;
        in_k = in_m = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (y < wave) before += x.wave_d[y];
            all += x.wave_d[y];
            in_k += x.wave_i[0][y];
            in_m += x.wave_i[1][y];
        }
    }
    // how many come before the sum reaches top_p of all
    int in_p = 0;
#pragma unroll
    for (int i = 0; i < DRAW; ++i) {
        cum[i] += before;
        in_p += __popcll(__ballot(there[i] && cum[i] < top_p * all));
    }
    if (!single) {
        if (lane == 0) x.wave_i[2][wave] = in_p;
        __syncthreads();
        in_p = x.wave_i[2][0] + x.wave_i[2][1] + x.wave_i[2][2] + x.wave_i[2][3];
    }
    const int keep = max(1, min(min(in_p + 1, in_m), in_k));
#pragma unroll
    for (int i = 0; i < DRAW; ++i)
        if (tid * DRAW + i == keep - 1) x.kept = cum[i];
    if (single) wave_fence();
    else __syncthreads();
    const double bound = uniform * x.kept;
    int j = 0;
#pragma unroll
    for (int i = 0; i < DRAW; ++i)
        j += __popcll(__ballot(tid * DRAW + i < keep && cum[i] <= bound));
    if (!single) {
        if (lane == 0) x.wave_i[0][wave] = j;
        __syncthreads();
        j = x.wave_i[0][0] + x.wave_i[0][1] + x.wave_i[0][2] + x.wave_i[0][3];
    }
    j = t > 0.0f ? min(j, keep - 1) : 0;
#pragma unroll
    for (int i = 0; i < DRAW; ++i)
        if (tid * DRAW + i == j) {
            a.ids[row] = (int32_t)~(uint32_t)mine[i];
            a.logprobs[row] = (float)(below_top(value(mine[i]), top) / (double)warm -
                                      log(x.whole.sum));
        }
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void join_kernel(PickArgs a, int slices, uint32_t inverse,
                                                       const Part *parts, const uint64_t *found) {
    __shared__ JoinSpace<THREADS> space;
    join<THREADS>(a, blockIdx.x, slices, inverse, parts, found, space);
}

// max_top_k = 1: the largest of the slices' best words; one wave per row.
__device__ __forceinline__ void join_first(const PickArgs &a, int64_t row, int slices,
                                           const Part *parts, const uint64_t *found) {
    const int lane = threadIdx.x & 63;
    const int cap = slice_cap(1);
    parts += row * slices;
    found += row * slices * cap;
    const Part first = lane_part(parts, slices);
    uint64_t best = lane < slices ? found[lane * cap] : 0ull;
    const float warm = warmth(parameter(a.temperature, row, 1.0f, a.uniform));
    if (first.count == 0) best = 0;
    for (int s = 64 + lane; s < slices; s += 64) {
        const uint64_t w = found[s * cap];
        if (parts[s].count > 0 && w > best) best = w;
    }
    const RowParts r = join_parts(parts, slices, first, warm);
    // the high words' largest, then the low words' largest among those
    const uint32_t high = (uint32_t)wave_max((int)((uint32_t)(best >> 32) ^ 0x80000000u)) ^ 0x80000000u;
    const uint32_t low = (uint32_t)(best >> 32) == high ? (uint32_t)best : 0u;
    const uint32_t token = ~((uint32_t)wave_max((int)(low ^ 0x80000000u)) ^ 0x80000000u);
    if (lane == 0) {
        a.ids[row] = high != 0u ? (int32_t)token : -1;
        a.logprobs[row] = high != 0u ? (float)-log(r.sum) : NEG_INF;
    }
}

constexpr int FT = 256;
__global__ __launch_bounds__(FT) void first_kernel(PickArgs a, int slices, const Part *parts,
                                                   const uint64_t *found) {
    const int64_t row = (int64_t)blockIdx.x * (FT / 64) + (threadIdx.x >> 6);
    if (row < a.rows) join_first(a, row, slices, parts, found);
}

// ------------------------------------------------------ both in one launch

// A row of one slice: its workgroup joins what it has found.  (A row of several
// slices could be joined by the workgroup that ends last; the fences at device
// scope that this takes made 14.5 us of what two launches do in 7.1, at 16
// slices of one row.)
template <typename T, int VALUES, int GROUP, bool FIRST>
__global__ __launch_bounds__(1024, 4) void whole_kernel(PickArgs a, uint32_t inverse, Part *parts,
                                                        uint64_t *found) {
    __shared__ union {
        SliceSpace<1024, VALUES> slice;
        JoinSpace<1024> join;
    } space;
    slice<T, 1024, VALUES, GROUP, FIRST>(a, parts, found, space.slice);
    __syncthreads();
    if (!FIRST) join<1024>(a, blockIdx.x, 1, inverse, parts, found, space.join);
    else if (threadIdx.x < 64) join_first(a, blockIdx.x, 1, parts, found);
}

// How a row is split.  Not at all, in one launch, while no more than one
// workgroup of 1024 threads is wanted per CU.  Bfloat16 rows, us a call, eager /
// in a graph, in one launch and in two:
//   rows x tokens, candidates            one launch      two
//   1 x 32000, 1                         9.5 / 6.7       11.7 / 7.1
//   1 x 32000, 1, a history of 200       9.8 / 8.4       12.4 / 8.0
//   1 x 32000, 50, a history of 200      13.8 / 13.8     12.8 / 12.4
//   64 x 32000, 50, a history of 200     14.7 / 14.7     13.8 / 13.2
//   256 x 8000, 50, a history of 200     12.5 / 12.4     13.4 / 12.8
//   256 x 32000, 1000, a history of 200  18.1 / 18.1     21.9 / 21.7
//   300 x 32000, 50, a history of 200    28.4 / 28.4     21.1 / 20.4
//   600 x 8000, 50, a history of 200     30.3 / 30.4     19.4 / 19.2
// (What the first form loses by with 50 candidates in few rows is less than
// what it gains with one or with many.)
// Else in slices of 16384 tokens, or of 8192 where the vocabulary has no more
// (300 rows of 8000 with 50 candidates: 13.5 us, and 15.1 in one of 16384).
// Slices of 8192 have twice the candidates to join and every slice reads the
// whole history: 17 rows of 131072 with 1000 candidates take 31 us in them and
// 20.7 in slices of 16384, 256 rows 73 and 46 (86 and 55 with a history of
// 4096); one row with 50 candidates 14.2 and 13.2.  512 threads with 32 tokens
// each made 65 us where 16384 by 1024 threads made 59.
constexpr int WHOLE_MOST = 32768;

bool whole(int64_t rows, int vocab) { return vocab <= WHOLE_MOST && rows <= 256; }

int slice_of(int vocab) { return vocab <= 8192 ? 8192 : 16384; }

int slices_of(int64_t rows, int vocab) {
    return whole(rows, vocab) ? 1 : (vocab + slice_of(vocab) - 1) / slice_of(vocab);
}

// The workspace: a part per slice, then the candidates.
size_t parts_bytes(int64_t rows, int slices) {
    return ((size_t)rows * slices * sizeof(Part) + 255) / 256 * 256;
}

template <typename T, int THREADS, int VALUES, int GROUP, bool FIRST = false>
void run_slices(const PickArgs &a, int slices, Part *parts, uint64_t *found, hipStream_t stream) {
    const dim3 grid((unsigned)a.rows, (unsigned)slices);
    slice_kernel<T, THREADS, VALUES, GROUP, FIRST>
        <<<grid, THREADS, 0, stream>>>(a, parts, found);
}

template <typename T, int VALUES, int GROUP, bool FIRST = false>
void run_whole(const PickArgs &a, uint32_t inverse, Part *parts, uint64_t *found,
               hipStream_t stream) {
    whole_kernel<T, VALUES, GROUP, FIRST>
        <<<(unsigned)a.rows, 1024, 0, stream>>>(a, inverse, parts, found);
}

template <typename T>
void run(const PickArgs &a, hipStream_t stream) {
    const bool one = whole(a.rows, a.vocab), wide = slice_of(a.vocab) == 16384;
    const int slices = slices_of(a.rows, a.vocab), k = a.max_top_k;
    Part *parts = static_cast<Part *>(a.workspace);
    uint64_t *found = reinterpret_cast<uint64_t *>(static_cast<char *>(a.workspace) +
                                                   parts_bytes(a.rows, slices));
    const int pieces = (slice_cap(k) + 63) / 64;
    const uint32_t inverse = pieces == 1 ? 0u : (uint32_t)(((1ull << 32) + pieces - 1) / pieces);
    if (k == 1 && !one) {
        if (wide) run_slices<T, 1024, 16, 16, true>(a, slices, parts, found, stream);
        else run_slices<T, 1024, 8, 8, true>(a, slices, parts, found, stream);
        first_kernel<<<(unsigned)((a.rows + FT / 64 - 1) / (FT / 64)), FT, 0, stream>>>(
            a, slices, parts, found);
        return;
    }
    // Groups of the histogram: at least four for each of max_top_k, so that
    // the k-th largest group bounds the k-th value closely (of values without
    // order about 1.15 k lie above it).
    if (one) {
        if (a.vocab <= 8192) {
            if (k == 1) run_whole<T, 8, 8, true>(a, inverse, parts, found, stream);
            else if (k <= 256) run_whole<T, 8, 8>(a, inverse, parts, found, stream);
            else run_whole<T, 8, 2>(a, inverse, parts, found, stream);
        } else if (a.vocab <= 16384) {
            if (k == 1) run_whole<T, 16, 16, true>(a, inverse, parts, found, stream);
            else if (k <= 256) run_whole<T, 16, 16>(a, inverse, parts, found, stream);
            else run_whole<T, 16, 4>(a, inverse, parts, found, stream);
        } else {
            if (k == 1) run_whole<T, 32, 32, true>(a, inverse, parts, found, stream);
            else if (k <= 256) run_whole<T, 32, 32>(a, inverse, parts, found, stream);
            else run_whole<T, 32, 8>(a, inverse, parts, found, stream);
        }
        return;
    }
    if (wide) {
        if (k <= 256) run_slices<T, 1024, 16, 16>(a, slices, parts, found, stream);
        else run_slices<T, 1024, 16, 4>(a, slices, parts, found, stream);
    } else {
        if (k <= 256) run_slices<T, 1024, 8, 8>(a, slices, parts, found, stream);
        else run_slices<T, 1024, 8, 2>(a, slices, parts, found, stream);
    }
    // a join of four waves where they hold all candidates
    if (k <= 256 && slices * pieces <= 4 * JOIN_HELD)
        join_kernel<256><<<(unsigned)a.rows, 256, 0, stream>>>(a, slices, inverse, parts, found);
    else
        join_kernel<1024><<<(unsigned)a.rows, 1024, 0, stream>>>(a, slices, inverse, parts, found);
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
