// Penalties for repeated tokens, biases and grammar masks on logits.
#include "adjust_core.h"

#pragma clang fp contract(off)

namespace gnms {
namespace {

constexpr int AT = 1024;       // threads per workgroup
constexpr int SLICE = 16384;   // tokens per workgroup (64 KiB of LDS words)

template <typename T>
__global__ __launch_bounds__(AT) void adjust_kernel(AdjustArgs a, int slices) {
    extern __shared__ uint32_t word[];
    const int64_t row = blockIdx.x / slices;
    const int lo = (int)(blockIdx.x % slices) * SLICE;
    const int size = min(SLICE, a.vocab - lo);
    const RowRules r = row_rules(a.rules, row);
    gather_rules(a.rules, r, row, lo, size, word, threadIdx.x, AT);
    const T *in = static_cast<const T *>(a.logits) + row * a.row_stride + lo;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + lo;
    for (int i = threadIdx.x; i < size; i += AT)
        out[i] = from_f32<T>(adjusted(a.rules, r, row, to_f32(in[i]), r.words ? word[i] : 0u,
                                      lo + i));
}

template <typename T>
void run(const AdjustArgs &a, hipStream_t stream) {
    const int slices = (a.vocab + SLICE - 1) / SLICE;
    adjust_kernel<T><<<(unsigned)(a.rows * slices), AT, SLICE * 4, stream>>>(a, slices);
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs &a, hipStream_t stream) {
    if (a.dtype == NMS_F32) run<float>(a, stream);
    else if (a.dtype == NMS_F16) run<half_t>(a, stream);
    else run<bf16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace gnms
