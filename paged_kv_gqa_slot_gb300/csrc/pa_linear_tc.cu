// pa_linear_tc.cu -- linear attention over chunks of tokens (pa_linear_prefill) on the 5th-generation
// tensor cores.
//
// The recurrence S_t = a S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t, taken 128 tokens at a time.  With S the
// state before a chunk of n tokens and i, j its rows,
//   o_i = scale ( sum_{j <= i} a^{i-j} <q_i, k_j> v_j  +  a^{i+1} q_i^T S )
//   S'  = a^n S + sum_j (a^{n-1-j} k_j) v_j^T
// that is four products on the tensor core: Q K^T, P V (P the weighted, masked scores), Q S and K~^T V
// (K~ the weighted keys).  The powers enter as 2^{(i-j) log2 a} <= 1, so nothing overflows however
// strong the decay.  A token moves (2 heads + 2 kv heads) d 2 bytes; per SM and 128 tokens of one head that is
// 128 KB, about 5900 cycles of HBM time at d = 128, against about 2600 of tensor core: HBM bounds
// it, as long as the chain of one chunk (Q K^T, K~, K~^T V, S) stays below.
//
// S stays in tensor memory in fp32 (lane: row of k, column: column of v).  Each chunk it is read once,
// written to shared memory as bf16 (the operand of Q S: one rounding, as the scores have) and back,
// multiplied by a^n, for K~^T V to add to.  K~ enters as two bf16 parts (2^-16 of every term), since what
// it adds stays in the state.
//
// Masked rows of P are zero, and 0 times a NaN or an infinity in V is NaN: V is looked over when it
// arrives, what is not finite becomes 0, and the first token it was seen at is noted per column; from
// that row on the column is NaN, and so is the state's.
//
// One CTA a (sequence, kv head), one an SM.  Warps: 0-3 P and the outputs (one row a thread), 4-7 the
// state (one row a thread), 8-11 K~, 12 MMA issue and tensor memory, 13 TMA loads of K and V, 14 of Q (one thread
// issues a copy in about half a microsecond), 15 the look at V.
#include <algorithm>
#include <climits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kChunk = 128;
constexpr int kThreads = 512;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kQLoadWarp = 14, kCleanWarp = 15;
constexpr int kHalf = kChunk * 128;  // [128 rows][64 columns] bf16
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMinLogDecay = -1e4f;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTile;        // two tiles; each becomes the high parts of K~ in place
    static constexpr int kOffLo = kOffK + 2 * kTile;   // the low parts
    static constexpr int kOffV = kOffLo + kTile;       // two tiles
    static constexpr int kOffS = kOffV + 2 * kTile;    // the state, bf16, D rows
    static constexpr int kOffBars = kOffS + D * 128 * kHalves;
    static constexpr int kOffBad = kOffBars + 256;     // [D] first token of a column with a value that is not finite
    static constexpr int kSmem = kOffBad + D * 4;
    // tensor memory: scores and P, P V, Q S, the state
    static constexpr uint32_t kColP = 0, kColO1 = 128, kColO2 = kColO1 + D, kColU = kColO2 + D;
    static constexpr int kTmemCols = 512;
};
static_assert(Layout<128>::kSmem <= 227 * 1024, "shared memory");

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_clean[2], q_full, q_empty;
    uint64_t s_full, p_full, o_full, o_empty;  // scores, P, outputs ready; outputs read
    uint64_t k_raw;                            // Q K^T of the chunk is done: K may become K~
    uint64_t kt_full, st_full, u_full;         // K~ ready; the state ready for the chunk; K~^T V done
    uint64_t drain;
    uint32_t tmem_base;
    int any_bad;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct TcArgs {
    LinearArgs l;
    int group;
    float scale;
};

// d = (a0 * b0, a1 * b1), each rounded to nearest even
__device__ __forceinline__ void mul_x2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Sixteen values as bf16, in one 32-byte store (a whole sector a thread) where the address allows it.
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float* o, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
    if (!wide) {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                             const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const __grid_constant__ TcArgs a) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kOffBars);
    int* bad = reinterpret_cast<int*>(smem + L::kOffBad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127;
    const PackedArgs& p = a.l.rows;
    const int kvh = (int)(blockIdx.x % (unsigned)p.num_kv_heads), b = (int)(blockIdx.x / (unsigned)p.num_kv_heads);
    pdl_wait();
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(p.status, kDevOutOfRange);
        return;
    }
    const bool report = kvh == 0 && threadIdx.x == 0;
    const int c0 = p.cu_lens[b], c1 = p.cu_lens[b + 1], total = a.l.seq_lens[b], slot = a.l.state_slots[b];
    if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || total < c1 - c0) {
        if (report) atomicOr(p.status, kDevOutOfRange);
        return;
    }
    const int len = min(c1 - c0, p.max_len);
    if (report && (c1 - c0 > p.max_len || (len > 0 && slot >= a.l.num_slots))) atomicOr(p.status, kDevOutOfRange);
    if (len == 0) return;
    const int g = a.group;
    if (slot < 0 || slot >= a.l.num_slots) {  // padding: zero rows
        const int per = g * D / 8;
        for (long long i = threadIdx.x; i < (long long)len * per; i += kThreads)
            *reinterpret_cast<uint4*>(p.out + ((size_t)(c0 + i / per) * p.num_heads + (size_t)kvh * g) * D + i % per * 8) =
                make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    float* state = a.l.state + ((size_t)slot * p.num_kv_heads + kvh) * D * D;
    const bool fresh = total == c1 - c0;
    const int chunks = (len + kChunk - 1) / kChunk;
    // log2 of the decay (a NaN is taken as the lower end)
    const float la = fminf(fmaxf(a.l.log_decay[kvh], kMinLogDecay), 0.f) * kLog2e;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 1);
            mbar_init(&bars->v_clean[s], 32);
        }
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_full, 128);
        mbar_init(&bars->o_full, 1);
        mbar_init(&bars->o_empty, 128);
        mbar_init(&bars->k_raw, 1);
        mbar_init(&bars->kt_full, 128);
        mbar_init(&bars->st_full, 128);
        mbar_init(&bars->u_full, 1);
        mbar_init(&bars->drain, 1);
        bars->any_bad = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < D) bad[threadIdx.x] = INT_MAX;
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    bool ok = true;

    if (warp == kLoadWarp || warp == kQLoadWarp) {
        // ---------------------------------------------------------------- TMA loads
        if (lane == 0 && warp == kLoadWarp) {
            auto load = [&](int off, const CUtensorMap* map, int c, uint64_t* full) {
                mbar_arrive_expect_tx(full, L::kTile);
                tma_load_rows(smem + off + (c & 1) * L::kTile, map, kvh, c0 + c * kChunk, 0, full);
            };
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            int ks = 0, vs = 0;  // copies issued
            for (int c = 0; c < chunks; ++c) {
                if (c >= 2) ok = mbar_wait(&bars->k_empty[c & 1], ((c >> 1) & 1) ^ 1);
                if (!ok) break;
                load(L::kOffK, &tm_k, c, &bars->k_full[c & 1]);
                ++ks;
                if (c >= 2) ok = mbar_wait(&bars->v_empty[c & 1], ((c >> 1) & 1) ^ 1);
                if (!ok) break;
                load(L::kOffV, &tm_v, c, &bars->v_full[c & 1]);
                ++vs;
            }
            // before the CTA may leave: every copy issued here has landed
            for (int i = max(0, ks - 2); i < ks; ++i)
                if (!mbar_wait(&bars->k_full[i & 1], (i >> 1) & 1)) ok = false;
            for (int i = max(0, vs - 2); i < vs; ++i)
                if (!mbar_wait(&bars->v_full[i & 1], (i >> 1) & 1)) ok = false;
        } else if (lane == 0) {
            prefetch_tensormap(&tm_q);
            int qs = 0;
            for (int c = 0; c < chunks && ok; ++c) {
                for (int h = 0; h < g; ++h) {
                    if (qs > 0) ok = mbar_wait(&bars->q_empty, (qs & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars->q_full, L::kTile);
                    tma_load_rows(smem + L::kOffQ, &tm_q, kvh * g + h, c0 + c * kChunk, 0, &bars->q_full);
                    ++qs;
                }
            }
            if (qs && !mbar_wait(&bars->q_full, (qs - 1) & 1)) ok = false;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idesc_s = tc_idesc_bf16(kChunk, kChunk, false);
        constexpr uint32_t idesc_o = tc_idesc_bf16(kChunk, D, true);
        constexpr uint32_t idesc_u = tc_idesc_bf16(kChunk, D, true) | (1u << 15);  // A MN-major too
        const uint64_t qd = smem_desc_sw128(smem_u32(smem + L::kOffQ), 0, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kOffK), 0, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + L::kOffV), kHalf, 1024);
        const uint64_t sd = smem_desc_sw128(smem_u32(smem + L::kOffS), D * 128, 1024);
        // K~^T as A: at d = 64 its rows 64 .. 127 are whatever lies behind the tile, in lanes that nobody reads
        const uint64_t hd0 = smem_desc_sw128(smem_u32(smem + L::kOffK), kHalf, 1024);
        const uint64_t ld = smem_desc_sw128(smem_u32(smem + L::kOffLo), kHalf, 1024);
        for (int c = 0; c < chunks && ok; ++c) {
            const uint64_t kslot = (uint64_t)(((c & 1) * L::kTile) >> 4), vd = vd0 + kslot;
            ok = mbar_wait_warp(&bars->k_full[c & 1], (c >> 1) & 1);
            for (int h = 0; h < g && ok; ++h) {
                const int i = c * g + h;
                ok = mbar_wait_warp(&bars->q_full, i & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                    tc_mma_ew(tmem + L::kColP, qd + off, kd0 + kslot + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                tc_commit_ew(&bars->s_full);
                if (h == g - 1) tc_commit_ew(&bars->k_raw);
                // Q S, once the state is in shared memory and the outputs before are read
                if (h == 0) ok = mbar_wait_warp(&bars->st_full, c & 1);
                if (ok && i > 0) ok = mbar_wait_warp(&bars->o_empty, (i - 1) & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_ew(tmem + L::kColO2, qd + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                              sd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, kk > 0 ? 1u : 0u);
                tc_commit_ew(&bars->q_empty);
                if (h == 0) ok = mbar_wait_warp(&bars->v_clean[c & 1], (c >> 1) & 1);
                if (ok) ok = mbar_wait_warp(&bars->p_full, i & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kChunk / 16; ++kk)
                    tc_mma_ts_ew(tmem + L::kColO1, tmem + L::kColP + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4),
                                 idesc_o, kk > 0 ? 1u : 0u);
                tc_commit_ew(&bars->o_full);
            }
            if (ok) ok = mbar_wait_warp(&bars->kt_full, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kChunk / 16; ++kk) {
                const uint64_t off = (uint64_t)((kk * 16 * 128) >> 4);
                tc_mma_ew(tmem + L::kColU, hd0 + kslot + off, vd + off, idesc_u, 1u);
                tc_mma_ew(tmem + L::kColU, ld + off, vd + off, idesc_u, 1u);
            }
            tc_commit_ew(&bars->u_full);
            tc_commit_ew(&bars->k_empty[c & 1]);
            tc_commit_ew(&bars->v_empty[c & 1]);
        }
        // every MMA this warp issued has finished before the tensor memory is released
        tc_commit_ew(&bars->drain);
        if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
    } else if (warp >= kCleanWarp) {
        // ---------------------------------------------------------------- V looked over
        for (int c = 0; c < chunks && ok; ++c) {
            const int n = min(kChunk, len - c * kChunk);
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[c & 1], (c >> 1) & 1));
            if (!ok) break;
            uint8_t* tile = smem + L::kOffV + (c & 1) * L::kTile;
            // a pass that only reads (its loads run ahead), and only where something was found the repair
            uint32_t seen = 0;
#pragma unroll 8
            for (int i = lane; i < L::kTile / 16; i += 32) seen |= not_finite(*reinterpret_cast<const uint4*>(tile + 16 * i));
            if (seen) {
                for (int i = lane; i < L::kTile / 16; i += 32) {
                    uint4* at = reinterpret_cast<uint4*>(tile + 16 * i);
                    if (!not_finite(*at)) continue;
                    const int half = i / (kHalf / 16), row = i / 8 % kChunk, col = half * 64 + ((i & 7) ^ (row & 7)) * 8;
                    for (int e = 0; e < 8; ++e) {
                        uint16_t* x = reinterpret_cast<uint16_t*>(at) + e;
                        if ((*x & 0x7f80u) != 0x7f80u) continue;
                        if (row < n) {
                            atomicMin(&bad[col + e], c * kChunk + row);
                            bars->any_bad = 1;
                        }
                        *x = 0;
                    }
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(&bars->v_clean[c & 1]);
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- K weighted: row r of the chunk
        for (int c = 0; c < chunks && ok; ++c) {
            const int n = min(kChunk, len - c * kChunk);
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_raw, c & 1));
            if (!ok) break;
            // k_raw also means that the products with the low parts of the chunk before are done
            const float w = r < n ? fast_exp2((float)(n - 1 - r) * la) : 0.f;
            uint8_t* hi = smem + L::kOffK + (c & 1) * L::kTile + r * 128;
            uint8_t* lo = smem + L::kOffLo + r * 128;
#pragma unroll 1
            for (int i0 = 0; i0 < D / 8; i0 += 4) {
                uint4 in[4];  // four loads in flight together
                const int base = (i0 >> 3) * kHalf;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    in[i] = *reinterpret_cast<const uint4*>(hi + base + ((((i0 & 7) + i) ^ (r & 7)) << 4));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int off = base + ((((i0 & 7) + i) ^ (r & 7)) << 4);
                    uint32_t x[4] = {in[i].x, in[i].y, in[i].z, in[i].w}, lw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // rows past the sequence's end are not its own: zero
                        float f0 = r < n ? bf16_lo(x[e]) : 0.f, f1 = r < n ? bf16_hi(x[e]) : 0.f;
                        mul_x2(f0, f1, f0, f1, w, w);
                        x[e] = pack_bf16x2(f0, f1);
                        lw[e] = pack_bf16x2(f0 - bf16_lo(x[e]), f1 - bf16_hi(x[e]));
                    }
                    *reinterpret_cast<uint4*>(hi + off) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4*>(lo + off) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars->kt_full);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- the state: row r of S
        const uint32_t tm_u = tmem + ((uint32_t)((warp & 3) * 32) << 16) + L::kColU;
        const bool mine = r < D;
        uint8_t* ss = smem + L::kOffS + r * 128;
        for (int c = 0; c < chunks && ok; ++c) {
            const int n = min(kChunk, len - c * kChunk);
            const float f = fast_exp2((float)n * la);
            if (c > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_full, (c - 1) & 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t u[32];
                if (c > 0) {
                    tmem_ld32(tm_u + x, u);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const uint4 v = mine && !fresh ? *reinterpret_cast<const uint4*>(state + (size_t)r * D + x + e)
                                                       : make_uint4(0u, 0u, 0u, 0u);
                        u[e] = v.x;
                        u[e + 1] = v.y;
                        u[e + 2] = v.z;
                        u[e + 3] = v.w;
                    }
                }
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = pack_bf16x2(__uint_as_float(u[e + 2 * q]), __uint_as_float(u[e + 2 * q + 1]));
                        const int chunk = (x + e) >> 3;
                        *reinterpret_cast<uint4*>(ss + (chunk >> 3) * (D * 128) + (((chunk & 7) ^ (r & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
                tmem_st32_nowait(tm_u + x, u);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            mbar_arrive(&bars->st_full);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_full, (chunks - 1) & 1));
        if (ok) {
            tc_fence_after();
            const bool any_bad = bars->any_bad != 0;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t u[32];
                tmem_ld32(tm_u + x, u);
                if (any_bad)
                    for (int e = 0; e < 32; ++e)
                        if (bad[x + e] < len) u[e] = 0x7fffffffu;
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(state + (size_t)r * D + x + e) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
                }
            }
        }
        tc_fence_before();
    } else {
        // ---------------------------------------------------------------- P and the outputs: row r of the chunk
        const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float lead = fast_exp2((float)(r + 1) * la) * a.scale, row = (float)r;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        for (int i = 0; i < chunks * g && ok; ++i) {
            const int c = i / g, h = i - c * g;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full, i & 1));
            if (!ok) break;
            tc_fence_after();
            // (loops over column blocks are not unrolled: the roles run at the same time, and their code has to
            // fit the instruction cache together; unrolled, a chunk took 8500 cycles instead of NNNN)
#pragma unroll 1
            for (int x = 0; x < kChunk; x += 32) {
                // (a warp's rows are r & ~31 .. + 31: to the right of the diagonal there are zeros)
                uint32_t w[16];
                if (x <= (r | 31)) {
                    const float base = row - (float)x;
                    uint32_t s[32];
                    tmem_ld32(tm + L::kColP + x, s);
                    // P goes over the first half of the scores: column x / 2 has been read
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float d0 = base - (float)e, d1 = base - (float)(e + 1);  // rows between j and i
                        float y0, y1;
                        mul_x2(y0, y1, d0, d1, la, la);
                        mul_x2(y0, y1, fast_exp2(y0), fast_exp2(y1), __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                        w[e / 2] = pack_bf16x2(d0 >= 0.f ? y0 : 0.f, d1 >= 0.f ? y1 : 0.f);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0u;
                }
                tmem_st8_nowait(tm + L::kColP + x / 2, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
                tmem_st8_nowait(tm + L::kColP + x / 2 + 8, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_full);
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full, i & 1));
            if (!ok) break;
            tc_fence_after();
            const int t = c * kChunk + r;
            const bool any_bad = bars->any_bad != 0;
            __nv_bfloat16* dst = p.out + ((size_t)(c0 + t) * p.num_heads + (size_t)kvh * g + h) * D;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t o1[32], o2[32];
                tmem_ld32_async(tm + L::kColO1 + x, o1);
                tmem_ld32_async(tm + L::kColO2 + x, o2);
                tmem_wait_ld(o1);
                tmem_wait_ld(o2);
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = fmaf(__uint_as_float(o2[e]), lead, __uint_as_float(o1[e]) * a.scale);
                if (any_bad)
                    for (int e = 0; e < 32; ++e)
                        if (t >= bad[x + e]) o[e] = __uint_as_float(0x7fffffffu);
                if (t < len) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) store16(dst + x + e, o + e, wide);
                }
            }
            tc_fence_before();
            mbar_arrive(&bars->o_empty);
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, kDevTimeout);
    __syncthreads();
    pdl_trigger();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int D>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
    static OncePerDevice configured;
    const cudaError_t e = configured.run([] {
        return cudaFuncSetAttribute(linear_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kSmem);
    });
    if (e != cudaSuccess) return e;
    const PackedArgs& p = a.rows;
    TcArgs t;
    t.l = a;
    t.group = p.num_heads / p.num_kv_heads;
    t.scale = p.scale;
    CUtensorMap q, k, v;
    if (!strided_map(&q, p.q, p.num_tokens, p.num_heads, D, p.q_stride, 1, kChunk, Layout<D>::kHalves) ||
        !strided_map(&k, p.k, p.num_tokens, p.num_kv_heads, D, p.k_stride, 1, kChunk, Layout<D>::kHalves) ||
        !strided_map(&v, p.v, p.num_tokens, p.num_kv_heads, D, p.v_stride, 1, kChunk, Layout<D>::kHalves))
        return cudaErrorInvalidValue;
    const long long ctas = (long long)p.batch * p.num_kv_heads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<D>, q, k, v, t);
}

}  // namespace

cudaError_t launch_linear_prefill_tc(const LinearArgs& a, cudaStream_t stream) {
    return a.rows.head_dim == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace pa
