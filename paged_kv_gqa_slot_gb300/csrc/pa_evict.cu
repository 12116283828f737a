// pa_evict.cu -- eviction of a paged cache's blocks by accumulated attention weight.
//
// Per sequence, with nb = ceil(L / 16) blocks, e = max(0, nb - keep) leave: among the logical
// blocks [sink, nb - recent) the e with the lowest W_j = sum over kv heads of weights[h, j],
// the lowest index first among equals (a NaN counts as the lowest).  Table and weights rows
// close up in order, their freed tail becomes -1 and 0, and L shrinks by 16 e.  Whole blocks
// leave, so no K or V moves, the pool is only ever read by others, and a block that several
// sequences share is dropped from one table only.
//
// A few KB per sequence: latency is all there is.  One CTA per sequence reads its rows once, summing
// the heads into order-preserving 32-bit keys on the way into shared memory (where the rows fit;
// else it reads them again for the copy), finds the e-th smallest key by four 8-bit radix passes,
// ranks ties and survivors with two block scans, and gathers through the resulting source list.  The
// weights of a sequence share a few exponents, so the lanes of a warp that hold the same digit
// count together before they add to a bin.  W_j is the sum in 64 bits rounded once; it is formed
// from fp32 sums and their exact errors (fp64 arithmetic, of which an SM does two operations a cycle,
// took half the kernel's time), and in fp64 only where these leave the rounding open.  Rows in
// shared memory are read whole before any output is written; the others are gathered in
// ascending tiles, each read before it is written, from sources at or past it: outputs may be
// their inputs.
//
// Measured on GB300, 8 kv heads: 64 sequences of 72 blocks 5.3 us, 16 of 2048 14.2 us, nearly all of it the
// latency of the radix passes' barriers and the scans (the bytes would take 0.1 and 0.4 us).
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kFewBlocks = 256;    // tables up to this width: 128 threads, else 512
constexpr int kResident = 200 * 1024;  // bytes of rows and keys a CTA keeps in shared memory

// float order as unsigned order; -0 as +0, NaN below everything
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __noinline__ float sum64(const float* col, int heads, int width) {
    double d = 0.0;
    for (int h = 0; h < heads; ++h) d += (double)col[(size_t)h * width];
    return (float)d;
}

// W_j of one entry: the sum over heads of col[h * width] in fp64, rounded once.  s + err is the sum but for the
// roundings of err itself: every addition's error, at most 2^-24 of (1 + 2^-10) s, is exact and added up on its own.
//  * All numbers are multiples of q, the step of fp32 at the smallest weight `least`, and so are s and err.
//    While err stays below 2^24 q >= least, it is exact, and so is fp64's sum: with least >= heads 2^-23 s, s + err
//    rounds to W_j.
//  * Otherwise err is off by at most heads^2 2^-48 (1 + 2^-9) s, and fp64's sum by at most heads 2^-53 s: where both
//    ends of that range round to the same number, it is W_j.
//  * The rest, negative weights, infinities and NaN are summed in fp64.
// (Without the first rule every table had entries on their way to fp64, as sums that lie in the middle of two
// numbers are common, and 16 x 2048 took 15.3 us.)
struct WeightSum {
    float s = 0.f, err = 0.f, least = INFINITY;
    __device__ __forceinline__ void add(float w, bool in) {  // w = 0 unless `in`
        const float t = s + w, z = t - s;
        err += (s - (t - z)) + (w - z);
        s = t;
        least = fminf(least, in ? w : INFINITY);
    }
    __device__ __forceinline__ float value(const float* col, int heads, int width) const {
        const float n = static_cast<float>(heads);
        if (s < INFINITY && least >= s * (n * 0x1p-23f)) return s + err;
        const float off = s * (n * n * 0x1p-47f), lo = s + (err - off), hi = s + (err + off);
        return s < INFINITY && least >= 0.f && lo == hi ? lo : sum64(col, heads, width);
    }
};

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
    __shared__ int hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int b = blockIdx.x, width = a.max_blocks, heads = a.num_kv_heads, tid = threadIdx.x;
    const int lane = tid & 31;
    pdl_trigger();
    pdl_wait();
    const int32_t* table = a.tables + (size_t)b * width;
    const float* weights = a.weights + (size_t)b * heads * width;
    int L = a.seq_lens[b];
    float* rows = reinterpret_cast<float*>(src + width);             // resident: the weights
    int32_t* ids = reinterpret_cast<int32_t*>(rows + heads * width);  // and the table
    for (int j = tid; j < width; j += T) {
        const int32_t id = resident ? table[j] : 0;
        WeightSum w;
        for (int h0 = 0; h0 < heads; h0 += 8) {
            float v[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) v[h] = h0 + h < heads ? weights[(size_t)(h0 + h) * width + j] : 0.f;
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                w.add(v[h], h0 + h < heads);
                if (resident && h0 + h < heads) rows[(h0 + h) * width + j] = v[h];
            }
        }
        src[j] = order_key(w.value(weights + j, heads, width));
        if (resident) ids[j] = id;
    }
    if (resident) {
        weights = rows;
        table = ids;
    }
    __syncthreads();
    if (L < 0 || L > width * kBlockSize) {
        if (tid == 0) atomicOr(a.status, kDevOutOfRange);
        L = L < 0 ? 0 : width * kBlockSize;
    }
    const int nb = (L + kBlockSize - 1) / kBlockSize;
    const int e = max(0, nb - a.keep);
    const int lo = a.sink, hi = nb - a.recent;  // candidates [lo, hi): at least e of them, as sink + recent <= keep

    if (e > 0) {
        // the e-th smallest key, a digit at a time: `prefix` its upper digits, `left` how many of the
        // keys that share them still leave
        uint32_t prefix = 0;
        int left = e;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += T) hist[i] = 0;
            __syncthreads();
            for (int j0 = lo; j0 < hi; j0 += T) {
                const int j = j0 + tid;
                const uint32_t key = j < hi ? src[j] : 0u;
                const bool in = j < hi && (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8));
                const unsigned peers = __match_any_sync(0xffffffffu, in ? (int)(key >> shift & 255u) : -1);
                if (in && lane == __ffs(peers) - 1) atomicAdd(&hist[key >> shift & 255u], __popc(peers));
            }
            __syncthreads();
            if (tid < 32) {
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
        uint32_t flags[(kEvictMaxBlocks / 512 + 31) / 32] = {};
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
    float* weights_out = a.weights_out + (size_t)b * heads * width;
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
    return a.max_blocks <= kFewBlocks ? launch<128>(a, batch, stream) : launch<512>(a, batch, stream);
}

}  // namespace pa
