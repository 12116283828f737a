// pa_linear.cu -- linear attention with a decay for each head: the form for single tokens
// (pa_linear_decode) and the recurrence over a chunk, token by token (pa_linear_prefill).
//
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t
//
// Decode moves 8 d^2 bytes of state a (sequence, kv head) for about 5 d^2 flops: bound by HBM.  A CTA
// holds one state (or a slice of its columns, when there are few) in registers: read once, updated,
// written once, and every query head of the group is multiplied against the registers.  2048 states from HBM take
// 36.5 us at d = 128, 6.2 TB/s, 12.0 at d = 64, 5.7 TB/s; 32 states 3.1 and 2.1 us inside a graph.
#include <algorithm>

#include "pa_internal.h"
#include "pa_step.cuh"

namespace pa {
namespace {

// Chunks up to this long go token by token, in fp32 throughout.  us of 6 and of 8 tokens against one chunk of
// pa_linear_tc.cu, a query head a state and (in brackets) four, inputs in L2 where they fit:
//   d = 128   32 states 8.6, 10.4 : 9.5 (16.8, 21.3 : 15.3)     512 20.4, 24.7 : 30.5 (38.4, 48.6 : 53.6)
//             152 9.0, 10.7 : 10.0 (17.2, 21.8 : 15.9)          2048 89.8, 106 : 103 (157, 196 : 185)
//   d = 64    32 states 5.9, 7.3 : 6.1 (11.8, 15.0 : 10.0)      512 8.8, 10.2 : 16.9 (15.6, 19.9 : 32.7)
//             152 6.2, 7.5 : 6.7 (11.9, 15.4 : 10.8)            2048 16.7, 20.0 : 50.9 (30.2, 44.4 : 107)
// Six is where the two cross for d = 128; groups of four with few states would change over at five, and at d = 64
// many states at 12 to 16 tokens.
constexpr int kFewTokens = 6;

// What a sequence's state slot says: its state (null: padding, zero rows) and whether it begins at zero.
__device__ __forceinline__ float* state_of(const LinearArgs& a, int b, int kvh, bool report) {
    const int slot = a.state_slots[b], d = a.rows.head_dim;
    if (slot >= a.num_slots && report) atomicOr(a.rows.status, kDevOutOfRange);
    if (slot < 0 || slot >= a.num_slots) return nullptr;
    return a.state + ((size_t)slot * a.rows.num_kv_heads + kvh) * d * d;
}

// One CTA a (sequence, kv head, slice of CW columns of S), 256 threads: thread (r, c) holds rows
// r, r + R, ... and the four columns 4c .. 4c+3 of S, so a warp reads whole 128-byte lines.
// (CTAs an SM that leave the registers to load all of the slice at once: one state of 32 heads 2.3 us against 2.5 without.)
template <int D, int CW>
__global__ void __launch_bounds__(256, D == CW ? (D == 128 ? 2 : 6) : 4) linear_decode_kernel(const LinearArgs a) {
    constexpr int C4 = CW / 4, R = 256 / C4, N = D / R;
    __shared__ float s_k[D], s_q[D];
    __shared__ float4 s_part[256];
    const int tid = threadIdx.x, c = tid % C4, r = tid / C4;
    const int kvh = blockIdx.x / (D / CW), col = (blockIdx.x % (D / CW)) * CW + 4 * c;
    const int b = blockIdx.y, g = a.rows.num_heads / a.rows.num_kv_heads;
    pdl_trigger();
    pdl_wait();
    const int len = a.seq_lens[b];
    float* st = state_of(a, b, kvh, tid == 0 && blockIdx.x == 0);
    const bool live = st && len > 0;
    __nv_bfloat16* out = a.rows.out + ((size_t)b * a.rows.num_heads + (size_t)kvh * g) * D;
    if (!live) {
        for (int i = tid; i < g * CW; i += 256)
            out[(size_t)(i / CW) * D + (blockIdx.x % (D / CW)) * CW + i % CW] = __float2bfloat16_rn(0.f);
        return;
    }
    float4 s[N];
    if (len > 1) {
#pragma unroll
        for (int n = 0; n < N; ++n) s[n] = *reinterpret_cast<const float4*>(st + (size_t)(r + n * R) * D + col);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) s[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < D) s_k[tid] = __bfloat162float(a.rows.k[b * a.rows.k_stride + (long long)kvh * D + tid]);
    const Decay decay(in_range(a.log_decay[kvh]), 1.f);
    const uint2 vv = *reinterpret_cast<const uint2*>(a.rows.v + b * a.rows.v_stride + (long long)kvh * D + col);
    const float v0 = bf16_lo(vv.x), v1 = bf16_hi(vv.x), v2 = bf16_lo(vv.y), v3 = bf16_hi(vv.y);
    __syncthreads();
    const float x = decay.x;
    if (decay.near) {  // (one loop that chooses in every term: 2048 states 42.1 us against 41.4)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float k = s_k[r + n * R];
            s[n].x = fmaf(k, v0, fmaf(s[n].x, x, s[n].x));
            s[n].y = fmaf(k, v1, fmaf(s[n].y, x, s[n].y));
            s[n].z = fmaf(k, v2, fmaf(s[n].z, x, s[n].z));
            s[n].w = fmaf(k, v3, fmaf(s[n].w, x, s[n].w));
            *reinterpret_cast<float4*>(st + (size_t)(r + n * R) * D + col) = s[n];
        }
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float k = s_k[r + n * R];
            s[n].x = fmaf(s[n].x, x, k * v0);
            s[n].y = fmaf(s[n].y, x, k * v1);
            s[n].z = fmaf(s[n].z, x, k * v2);
            s[n].w = fmaf(s[n].w, x, k * v3);
            *reinterpret_cast<float4*>(st + (size_t)(r + n * R) * D + col) = s[n];
        }
    }
    for (int h = 0; h < g; ++h) {
        if (tid < D)
            s_q[tid] = __bfloat162float(a.rows.q[b * a.rows.q_stride + (long long)(kvh * g + h) * D + tid]);
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float q = s_q[r + n * R];
            o.x = fmaf(q, s[n].x, o.x);
            o.y = fmaf(q, s[n].y, o.y);
            o.z = fmaf(q, s[n].z, o.z);
            o.w = fmaf(q, s[n].w, o.w);
        }
        s_part[tid] = o;
        __syncthreads();
        if (tid < CW) {
            const float* part = reinterpret_cast<const float*>(s_part);
            float sum = 0.f;
            for (int i = 0; i < R; ++i) sum += part[i * CW + tid];
            out[(size_t)h * D + col - 4 * c + tid] = __float2bfloat16_rn(sum * a.rows.scale);
        }
        __syncthreads();
    }
}

// The recurrence token by token: one CTA a (sequence, kv head), one thread a column of S, which it
// holds in registers, so that o needs no sum across threads.
template <int D>
__global__ void __launch_bounds__(D) linear_step_kernel(const LinearArgs a) {
    __shared__ __align__(16) float s_k[D], s_q[D];
    const int col = threadIdx.x, kvh = blockIdx.x, b = blockIdx.y;
    const PackedArgs& p = a.rows;
    const int g = p.num_heads / p.num_kv_heads;
    pdl_trigger();
    pdl_wait();
    const int c0 = p.cu_lens[b], c1 = p.cu_lens[b + 1], len = a.seq_lens[b];
    const bool report = col == 0 && kvh == 0;
    if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || len < c1 - c0) {
        if (report) atomicOr(p.status, kDevOutOfRange);
        return;
    }
    if (c1 - c0 > p.max_len && report) atomicOr(p.status, kDevOutOfRange);
    const int n = min(c1 - c0, p.max_len);
    if (n == 0) return;
    float* st = state_of(a, b, kvh, report);
    float s[D];
#pragma unroll
    for (int i = 0; i < D; ++i) s[i] = st && len > c1 - c0 ? st[(size_t)i * D + col] : 0.f;
    const Decay decay(in_range(a.log_decay[kvh]), 1.f);  // (before the loads of S: 2048 states x 6 tokens 92.7 us, behind them 91.8)
    for (int t = 0; t < n; ++t) {
        const long long row = c0 + t;
        __syncthreads();
        s_k[col] = __bfloat162float(p.k[row * p.k_stride + (long long)kvh * D + col]);
        const float v = __bfloat162float(p.v[row * p.v_stride + (long long)kvh * D + col]);
        __syncthreads();
        if (decay.near) {
#pragma unroll
            for (int i = 0; i < D; ++i) s[i] = fmaf(s_k[i], v, fmaf(s[i], decay.x, s[i]));
        } else {
#pragma unroll
            for (int i = 0; i < D; ++i) s[i] = fmaf(s[i], decay.x, s_k[i] * v);
        }
        for (int h = kvh * g; h < (kvh + 1) * g; ++h) {
            __syncthreads();
            s_q[col] = __bfloat162float(p.q[row * p.q_stride + (long long)h * D + col]);
            __syncthreads();
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < D; ++i) o = fmaf(s_q[i], s[i], o);
            p.out[((size_t)row * p.num_heads + h) * D + col] = __float2bfloat16_rn(st ? o * p.scale : 0.f);
        }
    }
    if (st) {
#pragma unroll
        for (int i = 0; i < D; ++i) st[(size_t)i * D + col] = s[i];
    }
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int threads, const LinearArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D>
cudaError_t decode(const LinearArgs& a, cudaStream_t stream) {
    const int kvh = a.rows.num_kv_heads;
    // Columns are split over CTAs while the states alone leave SMs idle.  us split and whole, in L2, a query head a state and
    // (in brackets) four:
    //   d = 128   8 states 2.0, 2.9 (3.1, 4.2)   32 2.8, 3.3 (4.1, 4.6)   128 4.0, 4.4 (5.6, 5.8)   152 3.9, 3.2 (5.6, 4.5)
    //   d = 64    8 states 1.8, 1.9 (3.0, 2.8)   32 2.0, 1.9 (3.3, 2.9)   128 2.9, 2.6 (4.9, 3.9)   152 2.2, 2.2 (3.7, 3.0)
    // (at d = 64 a state is small enough for one CTA: whole costs no more there, and up to 1.2 us less)
    const long long states = (long long)kvh * a.rows.batch;
    if (states < device_info().num_sms)
        return launch(linear_decode_kernel<D, D / 4>, dim3(kvh * 4, a.rows.batch), 256, a, stream);
    return launch(linear_decode_kernel<D, D>, dim3(kvh, a.rows.batch), 256, a, stream);
}

}  // namespace

cudaError_t launch_linear_decode(const LinearArgs& a, cudaStream_t stream) {
    return a.rows.head_dim == 64 ? decode<64>(a, stream) : decode<128>(a, stream);
}

size_t linear_workspace(int batch, int num_kv_heads, int head_dim, int max_chunk) {
    if (max_chunk <= kFewTokens) return 0;
    const int segments = linear_segments(batch, num_kv_heads, max_chunk);
    return segments == 1 ? 0 : (size_t)segments * batch * num_kv_heads * head_dim * head_dim * sizeof(float);
}

cudaError_t launch_linear_prefill(const LinearArgs& a, void* workspace, cudaStream_t stream) {
    if (a.max_chunk > kFewTokens) return launch_linear_prefill_tc(a, workspace, stream);
    const dim3 grid(a.rows.num_kv_heads, a.rows.batch);
    return a.rows.head_dim == 64 ? launch(linear_step_kernel<64>, grid, 64, a, stream)
                                 : launch(linear_step_kernel<128>, grid, 128, a, stream);
}

}  // namespace pa
