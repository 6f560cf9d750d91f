// Picking the next token of every row from its adjusted logits.
//
// Two launches.  slice_kernel: one workgroup per (row, slice of the
// vocabulary) adjusts the slice, keeps its values in registers, and writes
// its largest max_top_k candidates and the slice's part of the softmax sum.
// join_kernel: one workgroup per row sorts the slices' candidates and draws.
//
// A candidate is a 64-bit word: the order-preserving key of its value above,
// the complement of its token below, so that the words of a row are all
// different and their descending order is the order of the definition (equal
// values by ascending token).  0 is no candidate.
#include "adjust_core.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr int PT = 1024;          // threads per workgroup
constexpr int PV = 16;            // values per thread
constexpr int SLICE = PT * PV;    // tokens per workgroup
constexpr int PWAVES = PT / 64;
static_assert(NMS_MAX_TOP_K <= PT, "one candidate per thread in the join");

struct Part {
    float top;   // the slice's largest value
    float pad;
    double sum;  // of exp((value - top) / temperature)
};

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

// z - top, with the limit 0 at z = top = +infinity; in the type of its use:
// float32 in the slices' sums, binary64 where a draw is decided.
template <typename V>
__device__ __forceinline__ V below_top(float z, float top) {
    return z == top ? (V)0 : (V)z - (V)top;
}

template <typename V>
__device__ __forceinline__ V block_sum(V v, V *scratch) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    V s = scratch[0];
    for (int w = 1; w < PWAVES; ++w) s += scratch[w];
    __syncthreads();
    return s;
}

__device__ __forceinline__ float block_max(float v, float *scratch) {
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = scratch[0];
    for (int w = 1; w < PWAVES; ++w) s = fmaxf(s, scratch[w]);
    __syncthreads();
    return s;
}

template <typename T>
__global__ __launch_bounds__(PT) void slice_kernel(PickArgs a, int slices, Part *parts,
                                                   uint64_t *found) {
    extern __shared__ uint32_t word[];
    __shared__ double dsum[PWAVES];
    __shared__ float fmaxs[PWAVES];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t chosen[2];  // the digit, and how many are left to find
    __shared__ uint32_t taken;
    const int64_t row = blockIdx.x / slices;
    const int lo = (int)(blockIdx.x % slices) * SLICE;
    const int size = min(SLICE, a.vocab - lo);
    const RowRules r = row_rules(a.rules, row);
    gather_rules(a.rules, r, row, lo, size, word, threadIdx.x, PT);
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + lo;
    float z[PV];
    float top = NEG_INF;
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        const int i = PT * j + threadIdx.x;
        z[j] = NEG_INF;
        if (i < size) {
            const float v = adjusted(a.rules, r, row, to_f32(in[i]), r.words ? word[i] : 0u,
                                     lo + i);
            if (v > NEG_INF) z[j] = v;
        }
        top = fmaxf(top, z[j]);
    }
    top = block_max(top, fmaxs);
    const float warm = warmth(a.temperature, row);
    double sum = 0.0;
    int eligible = 0;
#pragma unroll
    for (int j = 0; j < PV; ++j)
        if (z[j] > NEG_INF) {
            sum += (double)expf(below_top<float>(z[j], top) / warm);
            ++eligible;
        }
    sum = block_sum(sum, dsum);
    if (threadIdx.x == 0) parts[blockIdx.x] = Part{top, 0.0f, sum};

    // the k-th largest candidate, digit by digit from the top
    const int k = a.max_top_k;
    uint64_t prefix = 0, mask = 0;
    uint32_t left = (uint32_t)k;
    if (threadIdx.x == 0) taken = 0;
    eligible = block_sum(eligible, reinterpret_cast<int *>(fmaxs));
    if (eligible > k) {
        for (int shift = 56; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const uint64_t c = candidate(z[j], lo + PT * j + (int)threadIdx.x);
                if (c != 0 && (c & mask) == prefix) atomicAdd(&hist[(c >> shift) & 255], 1u);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t need = left;
                int d = 255;
                while (d > 0 && hist[d] < need) need -= hist[d--];
                chosen[0] = (uint32_t)d;
                chosen[1] = need;
            }
            __syncthreads();
            prefix |= (uint64_t)chosen[0] << shift;
            mask |= 255ull << shift;
            left = chosen[1];
            __syncthreads();
        }
    } else {
        __syncthreads();
        prefix = 1;
    }
    uint64_t *to = found + (int64_t)blockIdx.x * k;
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        const uint64_t c = candidate(z[j], lo + PT * j + (int)threadIdx.x);
        if (c >= prefix) {
            const uint32_t at = atomicAdd(&taken, 1u);
            if (at < (uint32_t)k) to[at] = c;
        }
    }
    __syncthreads();
    for (uint32_t i = taken + threadIdx.x; i < (uint32_t)k; i += PT) to[i] = 0;
}

// Descending bitonic sort of 2 * PT words.
__device__ __forceinline__ void sort_words(uint64_t *w) {
    for (int size = 2; size <= 2 * PT; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            const int i = 2 * threadIdx.x - (threadIdx.x & (step - 1));
            const bool down = (i & size) == 0;
            const uint64_t x = w[i], y = w[i + step];
            if ((x < y) == down) {
                w[i] = y;
                w[i + step] = x;
            }
            __syncthreads();
        }
}

__global__ __launch_bounds__(PT) void join_kernel(PickArgs a, int slices, const Part *parts,
                                                  const uint64_t *found) {
    __shared__ uint64_t best[2 * PT];
    __shared__ double scan[PT];
    __shared__ double dsum[PWAVES];
    __shared__ int isum[PWAVES];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    parts += row * slices;
    found += row * slices * a.max_top_k;
    const int64_t n = (int64_t)slices * a.max_top_k;
    best[tid] = 0;
    for (int64_t lo = 0; lo < n; lo += PT) {
        best[PT + tid] = lo + tid < n ? found[lo + tid] : 0;
        __syncthreads();
        sort_words(best);
    }
    const uint64_t first = best[0], mine = best[tid];
    if (first == 0) {
        if (tid == 0) {
            a.ids[row] = -1;
            a.logprobs[row] = NEG_INF;
        }
        return;
    }
    const float top = key_value((uint32_t)(first >> 32));
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const float warm = warmth(a.temperature, row);
    int k = a.top_k ? a.top_k[row] : a.max_top_k;
    k = min(max(k, 1), a.max_top_k);
    const bool there = tid < k && mine != 0;
    const float z = key_value((uint32_t)(mine >> 32));
    const double w = there ? exp(below_top<double>(z, top) / (double)warm) : 0.0;
    // running sums of the candidates' weights
    scan[tid] = w;
    __syncthreads();
    for (int d = 1; d < PT; d <<= 1) {
        const double v = tid >= d ? scan[tid - d] : 0.0;
        __syncthreads();
        scan[tid] += v;
        __syncthreads();
    }
    const double cum = scan[tid], all = scan[PT - 1];
    const double top_p = a.top_p ? (double)a.top_p[row] : 1.0;
    const double min_p = a.min_p ? (double)a.min_p[row] : 0.0;
    const int count = block_sum((int)there, isum);
    const int short_n = block_sum((int)(there && cum < top_p * all), isum) + 1;
    const int large_n = block_sum((int)(there && w >= min_p), isum);
    const int keep = max(1, min(min(short_n, large_n), count));
    const double bound = (double)a.uniform[row] * scan[keep - 1];
    int j = block_sum((int)(tid < keep && cum <= bound), isum);
    j = t > 0.0f ? min(j, keep - 1) : 0;
    // the softmax sum over the whole vocabulary, relative to the top
    double part = 0.0;
    for (int s = tid; s < slices; s += PT)
        if (parts[s].top > NEG_INF)
            part += parts[s].sum * exp(below_top<double>(parts[s].top, top) / (double)warm);
    const double sum = block_sum(part, dsum);
    if (tid == j) {
        a.ids[row] = (int32_t)~(uint32_t)mine;
        a.logprobs[row] = (float)(below_top<double>(z, top) / (double)warm - log(sum));
    }
}

size_t parts_bytes(int64_t rows, int slices) {
    return ((size_t)rows * slices * sizeof(Part) + 255) / 256 * 256;
}

template <typename T>
void run(const PickArgs &a, hipStream_t stream) {
    const int slices = (a.vocab + SLICE - 1) / SLICE;
    Part *parts = static_cast<Part *>(a.workspace);
    uint64_t *found = reinterpret_cast<uint64_t *>(static_cast<char *>(a.workspace) +
                                                   parts_bytes(a.rows, slices));
    slice_kernel<T><<<(unsigned)(a.rows * slices), PT, SLICE * 4, stream>>>(a, slices, parts,
                                                                            found);
    join_kernel<<<(unsigned)a.rows, PT, 0, stream>>>(a, slices, parts, found);
}

}  // namespace

size_t pick_workspace_bytes(int64_t rows, int vocab, int max_top_k) {
    const int slices = (vocab + SLICE - 1) / SLICE;
    return parts_bytes(rows, slices) + (size_t)rows * slices * max_top_k * 8;
}

hipError_t launch_pick(const PickArgs &a, hipStream_t stream) {
    if (a.dtype == NMS_F32) run<float>(a, stream);
    else if (a.dtype == NMS_F16) run<half_t>(a, stream);
    else run<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
