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
//
// Measured on GB300, 8 kv heads of d 128: 64 rows of 64 sequences 3.0 us (a launch and the chain slot, row
// and exponent, store); 8 x 2043 rows 19.0 us, 79% of the copy bandwidth for their 101 MB.  What is left
// there is the rows in flight: 32 warps an SM of 4 KB each, waiting about half of the time.
#include <algorithm>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace pa {
namespace {


struct Append8Args {
    uint8_t* codes[2];  // K, V
    uint8_t* exps;
    const uint4* rows[2];
    const int64_t* slots;
    unsigned* status;
    long long pool_slots;
    int num_tokens, num_kv_heads, window;
};

// 8 bf16 values times s2, a pair of equal powers of two, as 8 codes.  The product is exact in bf16
// but for results below 2^-126, whose code is zero either way.
__device__ __forceinline__ uint2 chunk_codes(const uint4& v, __nv_bfloat162 s2) {
    const auto mul = [&](uint32_t w) {
        const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), s2);
        return *reinterpret_cast<const uint32_t*>(&p);
    };
    const uint32_t x = mul(v.x), y = mul(v.y), z = mul(v.z), w = mul(v.w);
    return make_uint2(to_e4m3x4(bf16_lo(x), bf16_hi(x), bf16_lo(y), bf16_hi(y)),
                      to_e4m3x4(bf16_lo(z), bf16_hi(z), bf16_lo(w), bf16_hi(w)));
}

// 4 codes times s, rounded again.
__device__ __forceinline__ uint32_t shift_codes(uint32_t w, float s) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = f16x2_to_float2(lo), b = f16x2_to_float2(hi);
    return to_e4m3x4(a.x * s, a.y * s, b.x * s, b.y * s);
}

// One unit: the blocks whose first entry lies in the window from t0 on, of one kv head's K or V.
// ent, before: this lane's of the 32 entries from t0 on, and of the 32 before them.
template <int D>
__device__ __forceinline__ void append_unit(const Append8Args& a, int t0, int head, int64_t ent, int64_t before,
                                            int* token_at) {
    constexpr int kLanes = D / 8;            // lanes of a row: 8 values each
    constexpr int kPar = 32 / kLanes;        // rows a warp handles at once
    constexpr int kSteps = kBlockSize / kPar;
    const int lane = threadIdx.x & 31;
    const int kvh = head >> 1, is_v = head & 1;
    const auto slot_at = [&](long long t) { return t >= 0 && t < a.num_tokens ? __ldg(a.slots + t) : -1; };
    const auto in_pool = [&](int64_t s) { return s >= 0 && s < a.pool_slots; };
    // an entry is its block's first if the one before it that names a slot is of another block
    const unsigned window = (1u << a.window) - 1u;
    if (ent >= a.pool_slots && head == 0 && window >> lane & 1u) atomicOr(a.status, kDevOutOfRange);
    const auto block_of = [](int64_t s) { return static_cast<int>(s >> 4); };  // of a slot in the pool
    static_assert(kBlockSize == 16, "block_of");
    const int block_of_ent = in_pool(ent) ? block_of(ent) : -1;
    const unsigned named = __ballot_sync(0xffffffffu, block_of_ent >= 0);
    if (!(named & window)) return;
    const unsigned lower = named & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, block_of_ent, lower ? 31 - __clz(lower) : 0);
    unsigned firsts = window & __ballot_sync(0xffffffffu, block_of_ent >= 0 && lower && prev != block_of_ent);
    {
        // the window's first named entry: look back past its start, farther if need be
        const int f = __ffs(named) - 1;
        const int block = __shfl_sync(0xffffffffu, block_of_ent, f);
        bool first = true;
        int64_t s = before;
        for (int p = t0 - 1; p >= 0; p -= 32) {
            const unsigned some = __ballot_sync(0xffffffffu, in_pool(s));
            if (some) {
                first = __shfl_sync(0xffffffffu, block_of(s), __ffs(some) - 1) != block;
                break;
            }
            s = slot_at((long long)p - 32 - lane);
        }
        if (first && f < a.window) firsts |= 1u << f;
    }

    for (; firsts; firsts &= firsts - 1) {
        const int f = __ffs(firsts) - 1;
        const int block = __shfl_sync(0xffffffffu, block_of_ent, f);
        // the block's entries, up to the first of another block: token_at[o] is the token whose row
        // goes to offset o (-1: none); of entries with the same slot the last counts
        if (lane < kBlockSize) token_at[lane] = -1;
        __syncwarp();
        unsigned other = named & (~0u << f) & __ballot_sync(0xffffffffu, block_of_ent != block);
        if (lane >= f && block_of_ent == block && lane < (other ? __ffs(other) - 1 : 32))
            atomicMax(&token_at[ent & 15], t0 + lane);
        for (long long p = (long long)t0 + 32; !other && p < a.num_tokens; p += 32) {
            const int64_t s = slot_at(p + lane);
            other = __ballot_sync(0xffffffffu, in_pool(s) && block_of(s) != block);
            if (in_pool(s) && lane < (other ? __ffs(other) - 1 : 32))
                atomicMax(&token_at[s & 15], static_cast<int>(p) + lane);
        }
        __syncwarp();
        const int token = lane < kBlockSize ? token_at[lane] : -1;
        const unsigned written = __ballot_sync(0xffffffffu, token >= 0);
        const int sub = lane / kLanes, c = lane % kLanes;
        const size_t tile = (size_t)block * a.num_kv_heads + kvh;
        uint8_t* exp_at = a.exps + tile * 2 + is_v;
        uint8_t* rows = a.codes[is_v] + tile * kBlockSize * D;

        uint4 x[kSteps];
        uint32_t mag = 0u;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int src = __shfl_sync(0xffffffffu, token, i * kPar + sub);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (src >= 0) x[i] = __ldg(a.rows[is_v] + ((size_t)src * a.num_kv_heads + kvh) * kLanes + c);
        }
        const int k_old = valid_exp(*exp_at) - kExpBias;  // as the reading kernels take it
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            mag = max_mag2(max_mag2(max_mag2(max_mag2(mag, x[i].x), x[i].y), x[i].z), x[i].w);
        mag = __reduce_max_sync(0xffffffffu, max(mag & 0xffffu, mag >> 16));
        if (mag >= 0x7f80u) {  // infinities and NaN do not count
            mag = 0u;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                mag = max_mag2(max_mag2(max_mag2(max_mag2(mag, finite2(x[i].x)), finite2(x[i].y)), finite2(x[i].z)),
                               finite2(x[i].w));
            mag = __reduce_max_sync(0xffffffffu, max(mag & 0xffffu, mag >> 16));
        }
        int k = scale_exponent(__uint_as_float(mag << 16));
        if (!(written & 1u)) {
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
        const __nv_bfloat162 s = __float2bfloat162_rn(exp2_int(-k));
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = i * kPar + sub;
            if (written >> row & 1u) *reinterpret_cast<uint2*>(rows + row * D + c * 8) = chunk_codes(x[i], s);
        }
        __syncwarp();  // every lane has read the old exponent
        if (lane == 0) *exp_at = static_cast<uint8_t>(k + kExpBias);
    }
}

template <int D, int kWarps, int kCtasPerSm>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) kv_append8_kernel(const __grid_constant__ Append8Args a) {
    __shared__ int tokens[kWarps][kBlockSize];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    pdl_trigger();
    pdl_wait();
    const int heads2 = 2 * a.num_kv_heads;
    const long long unit = (long long)blockIdx.x * kWarps + warp;
    const long long start = unit / heads2 * a.window;
    if (start >= a.num_tokens) return;
    const auto slot_at = [&](long long t) { return t >= 0 && t < a.num_tokens ? __ldg(a.slots + t) : -1; };
    append_unit<D>(a, (int)start, (int)(unit % heads2), slot_at(start + lane), slot_at(start - 1 - lane),
                   tokens[warp]);
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
    // Many units: eight warps a CTA, four CTAs an SM; else four warps a CTA, so that few units spread over
    // more SMs: 16k rows of 8 heads 19.0 us against 19.9, but 2k rows 4.75 against 4.40.
    const auto launch = [&](auto kern, int warps) {
        const long long ctas = (units + warps - 1) / warps;
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(warps * 32);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1] = {pdl_attribute()};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, a);
    };
    if (units >= 64LL * device_info().num_sms)
        return pool.head_dim == 128 ? launch(kv_append8_kernel<128, 8, 4>, 8) : launch(kv_append8_kernel<64, 8, 4>, 8);
    return pool.head_dim == 128 ? launch(kv_append8_kernel<128, 4, 7>, 4) : launch(kv_append8_kernel<64, 4, 7>, 4);
}

}  // namespace pa
