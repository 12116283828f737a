// pa_evict.cu -- eviction of a paged cache's blocks by accumulated attention weight.
//
// Per sequence, with nb = ceil(L / 16) blocks, e = max(0, nb - keep) leave: among the logical
// blocks [sink, nb - recent) the e with the lowest W_j = sum over kv heads of weights[h, j],
// the lowest index first among equals (a NaN counts as the lowest).  Table and weights rows
// close up in order, their freed tail becomes -1 and 0, and L shrinks by 16 e.  Whole blocks
// leave, so no K or V moves, the pool is only ever read by others, and a block that several
// sequences share is dropped from one table only.
//
// A few KB per sequence: latency is all there is.  One CTA per sequence sums the heads into
// order-preserving 32-bit keys in shared memory, finds the e-th smallest by four 8-bit radix
// passes, ranks ties and survivors with two block scans, and gathers through the resulting
// source list.  W_j is summed in 64 bits and rounded once, so it does not depend on the order
// of the heads.  Every source index is >= its destination and the gather runs in ascending
// tiles, each read before it is written, so outputs may be their inputs.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// float order as unsigned order; -0 as +0, NaN below everything
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum of v over the block's threads in order; `total` is the sum of all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();  // warp_sums may still be read from the call before
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int s = warp_sums[w];
        before += w < warp ? s : 0;
        total += s;
    }
    return before + incl - v;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ uint32_t src[];  // keys first, then the source index of every new entry
    __shared__ int hist[256];
    __shared__ int warp_sums[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int b = blockIdx.x, width = a.max_blocks, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int32_t* table = a.tables + (size_t)b * width;
    const float* weights = a.weights + (size_t)b * a.num_kv_heads * width;
    int L = a.seq_lens[b];
    if (L < 0 || L > width * kBlockSize) {
        if (tid == 0) atomicOr(a.status, kDevOutOfRange);
        L = L < 0 ? 0 : width * kBlockSize;
    }
    const int nb = (L + kBlockSize - 1) / kBlockSize;
    const int e = max(0, nb - a.keep);
    const int lo = a.sink, hi = nb - a.recent;  // candidates [lo, hi): at least e of them, as sink + recent <= keep

    // this thread's run of entries
    const int per = (width + kThreads - 1) / kThreads;
    const int j0 = min(width, tid * per), j1 = min(width, j0 + per);
    if (e > 0) {
        for (int j = lo + tid; j < hi; j += kThreads) {
            double w = 0.0;
            for (int h = 0; h < a.num_kv_heads; ++h) w += (double)weights[(size_t)h * width + j];
            src[j] = order_key((float)w);
        }
        // the e-th smallest key, a digit at a time: `prefix` its upper digits, `left` how many of
        // the keys that share them still leave
        uint32_t prefix = 0;
        int left = e;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kThreads) {
                const uint32_t key = src[j];
                if (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[key >> shift & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {
                int v[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += v[i] = hist[lane * 8 + i];
                int incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                int below = incl - sum;
                if (below < left && left <= incl) {  // the digit is one of this lane's
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (below < left && left <= below + v[i]) {
                            s_prefix = prefix | (uint32_t)(lane * 8 + i) << shift;
                            s_left = left - below;
                        }
                        below += v[i];
                    }
                }
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
        }
        // keys below `prefix` leave, and the first `left` equal to it
        int ties = 0;
        for (int j = j0; j < j1; ++j) ties += j >= lo && j < hi && src[j] == prefix;
        int total;
        int tie = block_scan(ties, warp_sums, total);
        int gone = 0;
        for (int j = j0; j < j1; ++j) {
            const bool cand = j >= lo && j < hi;
            const uint32_t key = cand ? src[j] : 0xffffffffu;
            const bool out = cand && (key < prefix || (key == prefix && tie < left));
            tie += cand && key == prefix;
            gone += out;
            src[j] = out ? 1u : 0u;
        }
        int before = block_scan(gone, warp_sums, total);
        // evicted entries in order; the survivors' source list is built in place: entry
        // j - before <= j, and no thread's run is overwritten before it is read (the sync below)
        uint32_t out_bits[(kEvictMaxBlocks / kThreads + 31) / 32];
#pragma unroll
        for (int i = 0; i < (int)(sizeof out_bits / 4); ++i) out_bits[i] = 0u;
        for (int j = j0; j < j1; ++j) {
            const int i = j - j0;
#pragma unroll
            for (int w = 0; w < (int)(sizeof out_bits / 4); ++w)
                if (i >> 5 == w) out_bits[w] |= src[j] << (i & 31);
        }
        __syncthreads();
        for (int j = j0; j < j1; ++j) {
            const int i = j - j0;
            uint32_t bits = 0;
#pragma unroll
            for (int w = 0; w < (int)(sizeof out_bits / 4); ++w)
                if (i >> 5 == w) bits = out_bits[w];
            if (bits >> (i & 31) & 1u) {
                a.evicted[(size_t)b * width + before] = table[j];
                ++before;
            } else {
                src[j - before] = j;
            }
        }
        __syncthreads();
    }
    for (int j = e + tid; j < width; j += kThreads) a.evicted[(size_t)b * width + j] = -1;
    if (tid == 0) {
        a.num_evicted[b] = e;
        a.seq_lens_out[b] = L - kBlockSize * e;
    }
    // close up: ascending tiles, read before written
    int32_t* table_out = a.tables_out + (size_t)b * width;
    float* weights_out = a.weights_out + (size_t)b * a.num_kv_heads * width;
    const bool in_place = a.tables_out == a.tables || a.weights_out == a.weights;
    for (int i0 = 0; i0 < width; i0 += kThreads) {
        const int i = i0 + tid;
        const bool in = i < width, kept = i < width - e;
        const int from = kept ? (e > 0 ? (int)src[i] : i) : 0;
        const int32_t id = kept ? table[from] : -1;
        for (int h0 = 0; h0 < a.num_kv_heads; h0 += 8) {
            float w[8];
#pragma unroll
            for (int h = 0; h < 8; ++h)
                w[h] = kept && h0 + h < a.num_kv_heads ? weights[(size_t)(h0 + h) * width + from] : 0.f;
            if (in_place) __syncthreads();
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (in && h0 + h < a.num_kv_heads) weights_out[(size_t)(h0 + h) * width + i] = w[h];
        }
        if (in) table_out[i] = id;
        if (in_place) __syncthreads();
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int batch, cudaStream_t stream) {
    static OncePerDevice configured;
    const cudaError_t e = configured.run([] {
        return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxBlocks * 4);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)a.max_blocks * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace pa
