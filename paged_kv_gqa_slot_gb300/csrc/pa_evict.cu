// pa_evict.cu -- eviction of a paged cache's blocks by accumulated attention weight.
//
// Per sequence, with nb = ceil(L / 16) blocks, e = max(0, nb - keep) leave: among the logical
// blocks [sink, nb - recent) the e with the lowest W_j = sum over kv heads of weights[h, j],
// the lowest index first among equals (a NaN counts as the lowest).  Table and weights rows
// close up in order, their freed tail becomes -1 and 0, and L shrinks by 16 e.  Whole blocks
// leave, so no K or V moves, the pool is only ever read by others, and a block that several
// sequences share is dropped from one table only.
//
// A few KB per sequence: latency is all there is.  One CTA per sequence copies its rows into
// shared memory (while they fit; else it reads them twice), sums the heads into
// order-preserving 32-bit keys, which its threads keep in registers, finds the e-th smallest by
// bisection -- two bits a round, a count and one barrier each, which beat radix histograms,
// whose shared-memory atomics pile up on the few exponents that weights have -- ranks ties and
// survivors with two block scans, and gathers through the resulting source list.  W_j is summed
// in 64 bits and rounded once, so it does not depend on the order of the heads.  Rows in shared
// memory are read whole before any output is written; the others are gathered in
// ascending tiles, each read before it is written, from sources at or past it: outputs may be
// their inputs.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kFewBlocks = 256;    // tables up to this width: 128 threads, else 1024
constexpr int kResident = 200 * 1024;  // bytes of rows and keys a CTA keeps in shared memory

// float order as unsigned order; -0 as +0, NaN below everything
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum of v over the block's threads in order.
template <int T>
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
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
    const int below = lane < warp ? warp_sums[lane] : 0;  // at most 32 warps
    return __reduce_add_sync(0xffffffffu, below) + incl - v;
}

template <int T>
__global__ void __launch_bounds__(T) evict_kernel(const __grid_constant__ EvictArgs a, int resident) {
    extern __shared__ uint32_t src[];  // keys, then the source index of every new entry
    __shared__ int warp_sums[32];
    __shared__ int counts[2][3];
    const int b = blockIdx.x, width = a.max_blocks, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int32_t* table = a.tables + (size_t)b * width;
    const float* weights = a.weights + (size_t)b * a.num_kv_heads * width;
    int L = a.seq_lens[b];
    if (resident) {
        float* rows = reinterpret_cast<float*>(src + width);
        int32_t* ids = reinterpret_cast<int32_t*>(rows + a.num_kv_heads * width);
        const int cells = a.num_kv_heads * width;
        int i = tid;
        for (; i + 7 * T < cells; i += 8 * T) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = weights[i + k * T];
#pragma unroll
            for (int k = 0; k < 8; ++k) rows[i + k * T] = v[k];
        }
        for (; i < cells; i += T) rows[i] = weights[i];
        for (int j = tid; j < width; j += T) ids[j] = table[j];
        weights = rows;
        table = ids;
    }
    if (tid < 6) (&counts[0][0])[tid] = 0;
    __syncthreads();
    if (L < 0 || L > width * kBlockSize) {
        if (tid == 0) atomicOr(a.status, kDevOutOfRange);
        L = L < 0 ? 0 : width * kBlockSize;
    }
    const int nb = (L + kBlockSize - 1) / kBlockSize;
    const int e = max(0, nb - a.keep);
    const int lo = a.sink, hi = nb - a.recent;  // candidates [lo, hi): at least e of them, as sink + recent <= keep

    if (e > 0) {
        for (int j = lo + tid; j < hi; j += T) {
            double w = 0.0;
#pragma unroll 8
            for (int h = 0; h < a.num_kv_heads; ++h) w += (double)weights[(size_t)h * width + j];
            src[j] = order_key((float)w);
        }
        __syncthreads();
        // The e-th smallest key T: the largest value with fewer than e keys below it, two bits at a
        // time.  `left` of the keys equal to it leave too.  A thread keeps up to 4 keys at hand.
        constexpr int kHand = 4;
        uint32_t hand[kHand];
#pragma unroll
        for (int i = 0; i < kHand; ++i) {
            const int j = lo + tid + i * T;
            hand[i] = j < hi ? src[j] : 0xffffffffu;  // counts as below no trial value
        }
        uint32_t prefix = 0;
        int below = 0;  // keys below prefix
        for (int shift = 30, round = 0; shift >= 0; shift -= 2, ++round) {
            // keys below prefix + 1, 2, 3 steps
            int c[3] = {0, 0, 0};
            const auto count = [&](uint32_t key) {
#pragma unroll
                for (int i = 0; i < 3; ++i) c[i] += key < (prefix | ((uint32_t)(i + 1) << shift));
            };
#pragma unroll
            for (int i = 0; i < kHand; ++i) count(hand[i]);
            for (int j = lo + tid + kHand * T; j < hi; j += T) count(src[j]);
            int* to = counts[round & 1];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int sum = __reduce_add_sync(0xffffffffu, c[i]);
                if ((tid & 31) == i && sum) atomicAdd(&to[i], sum);
            }
            __syncthreads();
            int digit = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (to[i] < e) {
                    digit = i + 1;
                    below = to[i];
                }
            prefix |= (uint32_t)digit << shift;
            if (tid < 3) counts[(round + 1) & 1][tid] = 0;
            __syncthreads();
        }
        const int left = e - below;
        // this thread's run of entries
        const int per = (width + T - 1) / T;
        const int j0 = min(width, tid * per), j1 = min(width, j0 + per);
        int ties = 0;
        for (int j = j0; j < j1; ++j) ties += j >= lo && j < hi && src[j] == prefix;
        int tie = block_scan<T>(ties, warp_sums);
        int gone = 0;
        for (int j = j0; j < j1; ++j) {
            const bool cand = j >= lo && j < hi;
            const uint32_t key = cand ? src[j] : 0xffffffffu;
            const bool out = cand && (key < prefix || (key == prefix && tie < left));
            tie += cand && key == prefix;
            gone += out;
            src[j] = out ? 1u : 0u;
        }
        int before = block_scan<T>(gone, warp_sums);
        // the survivors' source list, in place: entry j - before <= j, which may lie in another
        // thread's run, so the flags move to registers first
        uint32_t flags[(kEvictMaxBlocks / 1024 + 31) / 32] = {};
        for (int j = j0; j < j1; ++j) {
#pragma unroll
            for (int w = 0; w < (int)(sizeof flags / 4); ++w)
                if ((j - j0) >> 5 == w) flags[w] |= src[j] << ((j - j0) & 31);
        }
        __syncthreads();
        for (int j = j0; j < j1; ++j) {
            uint32_t bits = 0;
#pragma unroll
            for (int w = 0; w < (int)(sizeof flags / 4); ++w)
                if ((j - j0) >> 5 == w) bits = flags[w];
            if (bits >> ((j - j0) & 31) & 1u) {
                a.evicted[(size_t)b * width + before] = table[j];
                ++before;
            } else {
                src[j - before] = j;
            }
        }
        __syncthreads();
    }
    for (int j = e + tid; j < width; j += T) a.evicted[(size_t)b * width + j] = -1;
    if (tid == 0) {
        a.num_evicted[b] = e;
        a.seq_lens_out[b] = L - kBlockSize * e;
    }
    // close up
    int32_t* table_out = a.tables_out + (size_t)b * width;
    float* weights_out = a.weights_out + (size_t)b * a.num_kv_heads * width;
    const bool in_place = !resident && (a.tables_out == a.tables || a.weights_out == a.weights);
    for (int i0 = 0; i0 < width; i0 += T) {
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

template <int T>
cudaError_t launch(const EvictArgs& a, int batch, cudaStream_t stream) {
    static OncePerDevice configured;
    const cudaError_t e = configured.run([] {
        return cudaFuncSetAttribute(evict_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kResident);
    });
    if (e != cudaSuccess) return e;
    const long long all = (long long)a.max_blocks * (a.num_kv_heads + 2) * 4;
    const int resident = all <= kResident;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(batch);
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = resident ? (size_t)all : (size_t)a.max_blocks * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<T>, a, resident);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int batch, cudaStream_t stream) {
    return a.max_blocks <= kFewBlocks ? launch<128>(a, batch, stream) : launch<1024>(a, batch, stream);
}

}  // namespace pa
