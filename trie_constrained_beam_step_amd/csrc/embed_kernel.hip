// embed_kernel.hip -- rows of the embedding table for a step's tokens, and the
// table's gradient from those rows' gradient.
#include "device_common.h"
#include "gr.h"
#include "vocab.h"

namespace gr {
namespace {

__device__ __forceinline__ void store_elem(float* p, int64_t i, float v) { p[i] = v; }
// bf16 with round to nearest even; NaN stays NaN
__device__ __forceinline__ void store_elem(uint16_t* p, int64_t i, float v) {
    const uint32_t b = __float_as_uint(v);
    p[i] = (v != v) ? (uint16_t)((b >> 16) | 0x40) : (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

template <typename T>
__global__ __launch_bounds__(256) void embed_lookup_kernel(EmbedLookupArgs a) {
    const int64_t i = blockIdx.x;
    const int32_t t = a.tokens[i];
    const bool ok = t >= 0 && t < a.V;
    const T* w = (const T*)a.weight + (int64_t)(ok ? t : 0) * a.wstride;
    T* o = (T*)a.out + i * a.ostride;
    for (int d = threadIdx.x; d < a.D; d += 256) store_elem(o, d, ok ? load_elem(w, d) * a.scale : 0.0f);
}

// One workgroup per word walks all tokens.
template <typename T>
__global__ __launch_bounds__(256) void embed_backward_kernel(EmbedBackwardArgs a) {
    const int32_t v = blockIdx.x;
    T* o = (T*)a.gweight + (int64_t)v * a.wstride;
    for (int d0 = 0; d0 < a.D; d0 += 256) {
        const int d = d0 + threadIdx.x;
        float acc = 0.0f;
        bool any = false;
        for (int i = 0; i < a.n; ++i) {
            if (a.tokens[i] != v) continue;
            any = true;
            if (d < a.D) acc += load_elem((const T*)a.grad + (int64_t)i * a.gstride, d);
        }
        if (d >= a.D) continue;
        if (!a.accumulate) store_elem(o, d, acc * a.scale);
        else if (any) store_elem(o, d, fmaf(acc, a.scale, load_elem(o, d)));
    }
}

}  // namespace

hipError_t launch_embed_lookup(const EmbedLookupArgs& a, int dtype, hipStream_t st) {
    if (a.n == 0) return hipSuccess;
    if (dtype == GR_BF16) embed_lookup_kernel<uint16_t><<<dim3((unsigned)a.n), 256, 0, st>>>(a);
    else embed_lookup_kernel<float><<<dim3((unsigned)a.n), 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbedBackwardArgs& a, int dtype, hipStream_t st) {
    if (a.n == 0 && a.accumulate) return hipSuccess;
    if (dtype == GR_BF16) embed_backward_kernel<uint16_t><<<dim3((unsigned)a.V), 256, 0, st>>>(a);
    else embed_backward_kernel<float><<<dim3((unsigned)a.V), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace gr
