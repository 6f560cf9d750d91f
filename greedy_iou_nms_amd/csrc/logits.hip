// Penalties for repeated tokens, biases and grammar masks on logits: one
// workgroup per slice of a row, which adjusts the tokens that the rules touch
// in LDS and streams the slice once (adjust_core.h).  256 rows of 131072
// bfloat16 logits with 2048 history entries take 30 us for 138 MB, 4.6 TB/s: a
// copy from HBM reaches 5.1 to 5.4, one of this size that stays in the last
// cache 8.2, so that gathering the rules before the stream shows too; 4 rows of
// 32000 take 4.4 us, which is latency.
#include "adjust_core.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

template <typename T, int THREADS, int VALUES>
__global__ __launch_bounds__(THREADS, 8) void adjust_kernel(AdjustArgs a) {
    constexpr int SLICE = THREADS * VALUES;
    __shared__ RuleSpace<SLICE> rules;
    const int64_t row = blockIdx.x;
    const int lo = (int)blockIdx.y * SLICE;
    const int size = min(SLICE, a.vocab - lo);
    // a thread's first entries, before it knows how many are in use
    const FourTokens early = load4(a.rules.history + row * a.rules.history_stride,
                                   wave_entry(), (int)a.rules.history_capacity);
    const RowRules r = row_rules(a.rules, row, readable(a.logits));
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + lo;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + lo;
    const Raw<T, THREADS, VALUES> raw(r, lo, size, in);
    if (r.words) slice_rules<THREADS, SLICE>(a.rules, r, row, lo, size, early, rules);
    float z[VALUES];
    adjusted<T, THREADS, VALUES>(a.rules, r, row, in, raw, rules, z);
#pragma unroll
    for (int g = 0; g < VALUES / 8; ++g) {
        const int at = token_at<THREADS>(8 * g);
        if (size - at >= 8) {
            Eight<T> e;
#pragma unroll
            for (int j = 0; j < 8; ++j) e.v[j] = from_f32<T>(z[8 * g + j]);
            __builtin_memcpy(out + at, &e, sizeof(e));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at + j < size) out[at + j] = from_f32<T>(z[8 * g + j]);
        }
    }
}

template <typename T, int THREADS, int VALUES>
void run(const AdjustArgs &a, hipStream_t stream) {
    constexpr int SLICE = THREADS * VALUES;
    const dim3 grid((unsigned)a.rows, (unsigned)((a.vocab + SLICE - 1) / SLICE));
    adjust_kernel<T, THREADS, VALUES><<<grid, THREADS, 0, stream>>>(a);
}

// Slices of 16384 tokens where they fill the GPU.  Else of 8192, with half the
// tokens per thread, or of 2048 with a quarter of the threads while those are
// few and no long history is read by each: 1 row of 131072 tokens takes 4.2 us
// in slices of 2048 and 4.7 of 8192, 31 rows 8.7 and 6.8.
template <typename T>
void choose(const AdjustArgs &a, hipStream_t stream) {
    const int64_t wide = a.rows * ((a.vocab + 16383) / 16384);
    const int64_t fine = a.rows * ((a.vocab + 8191) / 8192);
    if (wide >= 256) run<T, 1024, 16>(a, stream);
    else if (fine >= 64 || a.rules.history_capacity > 4096) run<T, 1024, 8>(a, stream);
    else run<T, 256, 8>(a, stream);
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs &a, hipStream_t stream) {
    if (a.dtype == NMS_F32) choose<float>(a, stream);
    else if (a.dtype == NMS_F16) choose<half_t>(a, stream);
    else choose<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
