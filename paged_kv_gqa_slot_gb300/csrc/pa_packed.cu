// pa_packed.cu -- causal attention over packed prompts (pa_prefill_packed).
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// One warp a (token, query head): the keys one after another under a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) packed_row_kernel(const PackedArgs a) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int b = blockIdx.y;
    const int h = (int)(w % a.num_heads);
    const long long i = w / a.num_heads;
    const int c0 = a.cu_lens[b], c1 = a.cu_lens[b + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.num_tokens || c1 - c0 > a.max_len) {
        if (w == 0 && lane == 0) atomicOr(a.status, kDevOutOfRange);
        if (c0 < 0 || c1 < c0 || c1 > a.num_tokens) return;
    }
    if (i >= min(c1 - c0, a.max_len)) return;
    const int kvh = h / (a.num_heads / a.num_kv_heads);
    float q[E], o[E] = {};
    for (int e = 0; e < E; ++e)
        q[e] = __bfloat162float(a.q[(c0 + i) * a.q_stride + (long long)h * D + e * 32 + lane]) * a.scale;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j <= i; ++j) {
        float s = 0.f;
        for (int e = 0; e < E; ++e)
            s += q[e] * __bfloat162float(a.k[(long long)(c0 + j) * a.k_stride + (long long)kvh * D + e * 32 + lane]);
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = l * f + p;
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * f +
                   p * __bfloat162float(a.v[(long long)(c0 + j) * a.v_stride + (long long)kvh * D + e * 32 + lane]);
        m = mn;
    }
    for (int e = 0; e < E; ++e)
        a.out[((c0 + i) * a.num_heads + h) * D + e * 32 + lane] = __float2bfloat16_rn(o[e] / l);
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedArgs& a, cudaStream_t stream) {
    const long long warps = (long long)a.max_len * a.num_heads;
    const long long ctas = (warps + 3) / 4;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, a.batch);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.head_dim == 64 ? cudaLaunchKernelEx(&cfg, packed_row_kernel<64>, a)
                            : cudaLaunchKernelEx(&cfg, packed_row_kernel<128>, a);
}

}  // namespace pa
