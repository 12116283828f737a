// pa_step.cuh -- device helpers of the packed prompts and of linear attention over chunks.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr float kLog2e = 1.44269504088896340736f;

// A head's log decay as given, in its range (a NaN is taken as the lower end).
__device__ __forceinline__ float in_range(float log_decay) { return fminf(fmaxf(log_decay, -1e4f), 0.f); }

// A state's decay over n tokens, a^n = e^(n log_decay).  A state decays again and again, so the rounding of a factor near
// one would add up (one token at a time with log decay -1e-5, after 4000 tokens: 1.5e-4 by a factor from exp2f, 2.7e-5
// by one rounded to nearest).  There x = a^n - 1, to its own last bits, and S a^n is S + S x.
struct Decay {
    float x;
    bool near;
    __device__ __forceinline__ Decay(float log_decay, float n) {
        const float t = log_decay * n;
        near = t > -0.5f;
        // e^t - 1 = t + t^2/2! + .. + t^9/9! + .., for t in (-1/2, 0] with what is left out below 2^-30 of it (without a
        // branch, which would hold up the loads around it)
        float p = 1.f / 362880.f;
        p = fmaf(p, t, 1.f / 40320.f);
        p = fmaf(p, t, 1.f / 5040.f);
        p = fmaf(p, t, 1.f / 720.f);
        p = fmaf(p, t, 1.f / 120.f);
        p = fmaf(p, t, 1.f / 24.f);
        p = fmaf(p, t, 1.f / 6.f);
        p = fmaf(p, t, 0.5f);
        x = near ? fmaf(p, t * t, t) : exp2f(t * kLog2e);
    }
};

// 4-D tiled load of a tile of packed rows (strided_map): heads from `head`, rows from `row`, column halves from
// `half`.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int head, int row, int half,
                                              uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(row), "r"(half), "r"(smem_u32(bar))
        : "memory");
}

// Nonzero if one of the eight bf16 values is a NaN or an infinity: all exponent bits set, which a carry out of
// them shows (0x0080 added to the masked exponent 0x7f80 gives 0x8000).
__device__ __forceinline__ uint32_t not_finite(const uint4& x) {
    const uint32_t a = (x.x & 0x7f807f80u) + 0x00800080u, b = (x.y & 0x7f807f80u) + 0x00800080u;
    const uint32_t c = (x.z & 0x7f807f80u) + 0x00800080u, d = (x.w & 0x7f807f80u) + 0x00800080u;
    return (a | b | c | d) & 0x80008000u;
}

// Eight words (sixteen bf16) to global memory, in one 32-byte store, a whole sector, where the address allows it.
__device__ __forceinline__ void store_32(void* dst, const uint32_t* w, bool wide) {
    if (!wide) {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Eight words from global memory, in one 32-byte load where the address allows it.
__device__ __forceinline__ void load_32(const void* src, uint32_t* w, bool wide) {
    if (!wide) {
        const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        return;
    }
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src)
                 : "memory");
}

// A warp takes over a block of the grid that has not started (clusterlaunchcontrol): its x coordinate in `id`.
// False: there is none left, and it may not be asked again; or the wait ran out (ok false).  `reply` and `next`
// (an mbarrier of count 1, its phase in `phase`) are shared memory of this use alone.
__device__ __forceinline__ bool take_block(uint4* reply, uint64_t* next, uint32_t& phase, unsigned& id, bool& ok) {
    if ((threadIdx.x & 31) == 0) {
        fence_proxy_async_smem();  // the reply before has been read
        mbar_arrive_expect_tx(next, 16);
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                smem_u32(reply)),
            "r"(smem_u32(next))
            : "memory");
    }
    __syncwarp();
    ok = __all_sync(0xffffffffu, mbar_wait(next, phase));
    phase ^= 1;
    if (!ok) return false;
    uint32_t got, x, y, z;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%4];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, r;\n\t}"
        : "=r"(got), "=r"(x), "=r"(y), "=r"(z)
        : "r"(smem_u32(reply))
        : "memory");
    __syncwarp();
    if (got) id = x;
    return got != 0;
}

// The pairs of tiles of a packed call, found by number: the pairs of the sequences are counted one after another, each
// sequence's longest first.  A warp looks at 32 sequences at a time, one a lane, and goes on from where it was, as blocks
// are mostly taken over in rising order.  Nothing promises that order: a pair that lies before is looked for from
// the first sequence on.
struct PairWalk {
    const PackedArgs& p;
    const int tokens;             // of a pair
    int b0 = 0;                   // first of the sequences looked at
    unsigned before = 0;          // pairs of those before them
    unsigned mine = 0, upto = 0;  // the lane's sequence: its pairs, and those up to its end from b0 on
    int row = 0, len = 0;         // its rows

    __device__ __forceinline__ PairWalk(const PackedArgs& args, int pair_tokens) : p(args), tokens(pair_tokens) { look_at(0); }

    // Sequence b's rows and pairs for the lane that asks.
    __device__ __forceinline__ void look(int b) {
        row = len = 0;
        mine = 0;
        if (b >= p.batch) return;
        const int c0 = p.cu_lens[b], c1 = p.cu_lens[b + 1];
        const bool off = c0 < 0 || c1 < c0 || c1 > p.num_tokens;
        if (off || c1 - c0 > p.max_len) atomicOr(p.status, kDevOutOfRange);
        row = c0;
        len = off ? 0 : min(c1 - c0, p.max_len);
        mine = (unsigned)((len + tokens - 1) / tokens);
    }
    __device__ __forceinline__ void look_at(int b) {
        const int lane = threadIdx.x & 31;
        b0 = b;
        look(b + lane);
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += up;
        }
    }
    // Looks at the sequence of pair `pair`, the same in every lane; false: it lies past the last.  (The roles of a CTA
    // share the instruction cache, so there is one place that looks: with another for the way back 16 prompts of 2000 tokens
    // at d = 64 took 98 us against 96.)
    __device__ __forceinline__ bool find(unsigned pair) {
        for (;;) {
            const unsigned all = __shfl_sync(0xffffffffu, upto, 31);
            const bool back = pair < before;
            if (!back) {
                if (pair < before + all) return true;
                if (b0 + 32 >= p.batch) return false;
            }
            before = back ? 0 : before + all;
            look_at(back ? 0 : b0 + 32);
        }
    }
    // Of the lane whose sequence it is, once it has been found.
    __device__ __forceinline__ bool owns(unsigned pair) const {
        return pair >= before + upto - mine && pair < before + upto;
    }
    __device__ __forceinline__ int first_token(unsigned pair) const { return (int)(before + upto - 1 - pair) * tokens; }
};

}  // namespace pa
