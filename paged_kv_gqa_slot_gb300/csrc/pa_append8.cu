// pa_append8.cu -- new bf16 K/V rows quantised into an 8-bit pool through a slot mapping.
//
// A pool block's 16 rows of one kv head share one power-of-two scale 2^k (pa_kv8.cuh).  The rows
// a call writes into a block are consecutive entries of slot_mapping, and per (block, kv
// head, K or V):
//   * a row at offset 0 begins the block anew: k is the smallest exponent that holds the new
//     rows, and the bytes of the rows not written stay;
//   * otherwise k = max(k_old, the new rows' exponent), and if it grew the other rows' codes
//     are shifted by k_old - k and rounded again (exact but for e4m3's subnormals).
//
// One warp does one such unit, from the first of the block's entries.  It looks for these
// "first" entries in a window of slot_mapping: one entry a warp when there are few (a decode
// step, where every row goes to another block and latency counts), 16 entries when there are
// many (a prefill chunk, where 15 of 16 entries only continue a block).  The unit's new rows
// are read once, 16 bytes a lane, and stay in registers between the maximum and the rounding.
#include <algorithm>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

struct Append8Args {
    uint8_t* codes[2];  // K, V
    uint8_t* exps;
    const uint4* rows[2];
    const int64_t* slots;
    unsigned* status;
    long long pool_slots;
    int num_tokens, num_kv_heads, window;
};

// Largest finite magnitude of the 8 bf16 values of a chunk (NaN and infinities do not count).
__device__ __forceinline__ float chunk_amax(const uint4& v) {
    float m = 0.f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = fabsf(bf16_lo(w[i])), b = fabsf(bf16_hi(w[i]));
        m = fmaxf(m, a < INFINITY ? a : 0.f);
        m = fmaxf(m, b < INFINITY ? b : 0.f);
    }
    return m;
}

// 8 bf16 values times s, as 8 codes.
__device__ __forceinline__ uint2 chunk_codes(const uint4& v, float s) {
    auto word = [&](uint32_t a, uint32_t b) {
        return to_e4m3x2(bf16_lo(a) * s, bf16_hi(a) * s) | (to_e4m3x2(bf16_lo(b) * s, bf16_hi(b) * s) << 16);
    };
    return make_uint2(word(v.x, v.y), word(v.z, v.w));
}

// 4 codes times s, rounded again.
__device__ __forceinline__ uint32_t shift_codes(uint32_t w, float s) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(w & 0xffffu));
    const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(w >> 16));
    return to_e4m3x2(a.x * s, a.y * s) | (to_e4m3x2(b.x * s, b.y * s) << 16);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_append8_kernel(const __grid_constant__ Append8Args a) {
    constexpr int kLanes = D / 8;            // lanes of a row: 8 values each
    constexpr int kPar = 32 / kLanes;        // rows a warp handles at once
    constexpr int kSteps = kBlockSize / kPar;
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const int heads2 = 2 * a.num_kv_heads;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int head = static_cast<int>(unit % heads2);  // kv head, then K or V
    const int t0 = static_cast<int>(min((long long)a.num_tokens, unit / heads2 * a.window));
    const int t1 = static_cast<int>(min((long long)a.num_tokens, (long long)t0 + a.window));
    const int kvh = head >> 1, is_v = head & 1;

    for (int t = t0; t < t1; ++t) {
        const int64_t slot = __ldg(a.slots + t);
        if (slot < 0) continue;
        if (slot >= a.pool_slots) {
            if (head == 0 && lane == 0) atomicOr(a.status, kDevOutOfRange);
            continue;
        }
        const int64_t block = slot / kBlockSize;
        // the entry before this one that names a slot: of the same block, and this unit is done there
        auto in_pool = [&](int64_t s) { return s >= 0 && s < a.pool_slots; };
        bool first = true;
        for (int p = t - 1; p >= 0; p -= 32) {
            const int64_t s = p - lane >= 0 ? __ldg(a.slots + p - lane) : -1;
            const unsigned named = __ballot_sync(0xffffffffu, in_pool(s));
            if (!named) continue;
            const int64_t last = __shfl_sync(0xffffffffu, s, __ffs(named) - 1);
            first = last / kBlockSize != block;
            break;
        }
        if (!first) continue;
        // the block's entries: lane o keeps the token whose row goes to offset o (-1: none); of
        // entries with the same slot the last counts
        int token = -1;
        for (int p = t; p < a.num_tokens; p += 32) {
            const int64_t s = p + lane < a.num_tokens ? __ldg(a.slots + p + lane) : -1;
            const bool named = in_pool(s);
            const unsigned other = __ballot_sync(0xffffffffu, named && s / kBlockSize != block);
            unsigned mine = __ballot_sync(0xffffffffu, named && s / kBlockSize == block);
            if (other) mine &= (1u << (__ffs(other) - 1)) - 1;  // entries before the next block's
            while (mine) {
                const int src = __ffs(mine) - 1;
                mine &= mine - 1;
                const int off = static_cast<int>(__shfl_sync(0xffffffffu, s, src) % kBlockSize);
                if (lane == off) token = p + src;
            }
            if (other) break;
        }
        const unsigned written = __ballot_sync(0xffffffffu, token >= 0);
        const int sub = lane / kLanes, c = lane % kLanes;
        const size_t tile = (size_t)block * a.num_kv_heads + kvh;
        uint8_t* exp_at = a.exps + tile * 2 + is_v;
        uint8_t* rows = a.codes[is_v] + tile * kBlockSize * D;

        uint4 x[kSteps];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int src = __shfl_sync(0xffffffffu, token, i * kPar + sub);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (src >= 0) x[i] = __ldg(a.rows[is_v] + ((size_t)src * a.num_kv_heads + kvh) * kLanes + c);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) amax = fmaxf(amax, chunk_amax(x[i]));
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        int k = scale_exponent(amax);
        if (!(written & 1u)) {
            const int k_old = static_cast<int>(*exp_at) - kExpBias;
            if (k > k_old) {
                const float s = exp2_int(k_old - k);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int row = i * kPar + sub;
                    if (written >> row & 1u) continue;
                    uint2* at = reinterpret_cast<uint2*>(rows + row * D + c * 8);
                    const uint2 w = *at;
                    *at = make_uint2(shift_codes(w.x, s), shift_codes(w.y, s));
                }
            }
            k = max(k, k_old);
        }
        const float s = exp2_int(-k);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = i * kPar + sub;
            if (written >> row & 1u) *reinterpret_cast<uint2*>(rows + row * D + c * 8) = chunk_codes(x[i], s);
        }
        __syncwarp();  // every lane has read the old exponent
        if (lane == 0) *exp_at = static_cast<uint8_t>(k + kExpBias);
    }
}

}  // namespace

cudaError_t launch_kv_append8(const Pool8View& pool, const void* k_new, const void* v_new, const int64_t* slots,
                              int num_tokens, unsigned* status, cudaStream_t stream) {
    Append8Args a;
    a.codes[0] = pool.k;
    a.codes[1] = pool.v;
    a.exps = pool.exps;
    a.rows[0] = static_cast<const uint4*>(k_new);
    a.rows[1] = static_cast<const uint4*>(v_new);
    a.slots = slots;
    a.status = status;
    a.pool_slots = (long long)pool.num_blocks * kBlockSize;
    a.num_tokens = num_tokens;
    a.num_kv_heads = pool.num_kv_heads;
    const long long per_token = 2LL * pool.num_kv_heads;
    a.window = num_tokens * per_token > 16LL * 4 * device_info().num_sms ? kBlockSize : 1;
    const long long units = (num_tokens + a.window - 1) / a.window * per_token;
    const long long ctas = (units + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return pool.head_dim == 128 ? cudaLaunchKernelEx(&cfg, kv_append8_kernel<128>, a)
                                : cudaLaunchKernelEx(&cfg, kv_append8_kernel<64>, a);
}

}  // namespace pa
