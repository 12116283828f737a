// pa_packed.cu -- causal attention over packed prompts (pa_prefill_packed) on the 5th-generation
// tensor cores.
//
//   o_i = sum_{j <= i} softmax_j(scale <q_i, k_j>) v_j   within each sequence
//
// A query tile is 128 rows of (token, head) pairs: th heads of one kv head's group, 128 / th tokens, so
// the heads of a group share every K and V tile and the tile of a short prompt is well filled.  A
// CTA, one an SM, holds two neighbouring tiles and walks the keys in stages of 128:
//   S_t = Q_t K^T     tcgen05.mma M = N = 128, both operands from shared memory, S_t in tensor memory
//   softmax           one thread a row: P_t (bf16) over the first half of S_t
//   O_t += P_t V      tcgen05.mma M = 128, N = d, P_t from tensor memory
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (d each): all of it at d = 128.  While one tile's
// softmax runs, the tensor core works for the other; per tile and stage it is busy for 1024 cycles at
// d = 128 (two products of 128 x 128 x 128), which bounds the kernel at long prompts.  N = 128
// matters: with both operands in shared memory, 64-key products are bound by its bandwidth.
//
// Base of the softmax: a stage is taken against the row's current base; only a row's first stage, or
// one whose sum passes 2^16, takes the maximum, and O is rescaled where the maximum grew by more than
// 2^8.  P is rounded to bf16 and the normaliser sums the rounded values, so their rounding moves
// weight between keys but not its total.  Where few keys can dominate (a tile with a row of at most
// 128 keys, or |scale| sqrt(d) > 2) P enters as two bf16 parts, in the two halves of S_t.
//
// Masked keys have P = 0, and 0 times a NaN or an infinity in V is NaN.  So in the stages that hold a
// key masked for some row, two warps look V over before its product: what is not finite is replaced
// by 0, and the first token it was seen at noted per column; rows at or behind it get it back.
//
// Warps: 0-3 and 4-7 softmax of tiles 0 and 1, 8 MMA issue and tensor memory, 9 TMA loads, 10-11 V.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRows = 128;              // rows of a query tile (MMA M)
constexpr int kKeys = 128;              // keys a stage (MMA N of Q K^T)
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10;
constexpr int kThreads = 384;
constexpr int kHalf = kRows * 128;      // [128 rows][64 columns] bf16
constexpr float kRescaleThreshold = 8.f;
constexpr float kSpecSumLimit = 65536.f;
constexpr float kSplitScale = 2.f;      // |scale| sqrt(d) past this: P in two parts
constexpr int kFewKeys = 128;           // a tile with a row of at most this many keys: the same
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalf;      // a tile of Q, K or V
    static constexpr int kKSlots = 3, kVSlots = D == 64 ? 3 : 2;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + kKSlots * kTile;
    static constexpr int kOffBars = kOffV + kVSlots * kTile;
    static constexpr int kOffBad = kOffBars + 256;     // [3][D] first token of a NaN, +inf, -inf in a column of V
    static constexpr int kSmem = kOffBad + 3 * D * 4;
    static constexpr int kColsO = 2 * kKeys;           // tensor memory: S_0, S_1, O_0, O_1
    static constexpr int kTmemCols = 512;
};
static_assert(Layout<128>::kSmem <= 227 * 1024, "shared memory");

template <int D>
struct Bars {
    uint64_t q_full[2], k_full[Layout<D>::kKSlots], k_empty[Layout<D>::kKSlots], v_full[Layout<D>::kVSlots],
        v_empty[Layout<D>::kVSlots], v_clean[Layout<D>::kVSlots], s_full[2], p_full[2], o_final[2], drain;
    uint32_t tmem_base;
    int any_bad;
};
static_assert(sizeof(Bars<64>) <= 256 && sizeof(Bars<128>) <= 256, "barrier block");

struct TcArgs {
    PackedArgs p;
    int th, tpt;       // heads and tokens of a tile
    int subs;          // tiles' head groups: num_heads / th
    int pairs;         // tile pairs the grid holds a sequence
    int split_all;
    float scale_log2;  // scale * log2(e), signed
};

__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// (a0, a1) += the two bf16 values of a packed word, each widened exactly.
__device__ __forceinline__ void add_bf16x2(float& a0, float& a1, uint32_t w) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(w));
}

// The extreme visible score of a stage's quarter (32 keys, `lim` the last visible of them): the
// largest, or with kNeg (a negative scale) minus the smallest.
template <bool kAll, bool kNeg>
__device__ __forceinline__ float quarter_max(const uint32_t (&s)[32], int lim) {
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = kNeg ? -__uint_as_float(s[c + e]) : __uint_as_float(s[c + e]);
            if (!kAll) a[e] = c + e > lim ? -INFINITY : a[e];
        }
        m0 = fmax3(m0, a[0], a[1]);
        m1 = fmax3(m1, a[2], a[3]);
    }
    return fmaxf(m0, m1);
}

// P of a quarter against base -nbase, written over its 16 columns of tensor memory at `dst`, and the sum of the
// rounded values; with kSplit the rounding errors, rounded, at dst + 64, and their sum too.
template <bool kAll, bool kSplit>
__device__ __forceinline__ void quarter_p(const uint32_t (&s)[32], int lim, float sl, float nbase, uint32_t dst,
                                          float (&ls)[4]) {
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float x0, x1;
        fma_x2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl, sl, nbase, nbase);
        if (!kAll) {
            x0 = c > lim ? -INFINITY : x0;  // 2^-inf = 0
            x1 = c + 1 > lim ? -INFINITY : x1;
        }
        w[c / 2] = pack_bf16x2(fast_exp2(x0), fast_exp2(x1));
    }
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        add_bf16x2(ls[0], ls[1], w[i]);
        add_bf16x2(ls[2], ls[3], w[i + 1]);
    }
    tmem_st16_nowait(dst, w);
    if (kSplit) {
        uint32_t lo[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            fma_x2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl, sl, nbase, nbase);
            if (!kAll) {
                x0 = c > lim ? -INFINITY : x0;
                x1 = c + 1 > lim ? -INFINITY : x1;
            }
            lo[c / 2] = pack_bf16x2(fast_exp2(x0) - bf16_lo(w[c / 2]), fast_exp2(x1) - bf16_hi(w[c / 2]));
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            add_bf16x2(ls[0], ls[1], lo[i]);
            add_bf16x2(ls[2], ls[3], lo[i + 1]);
        }
        tmem_st16_nowait(dst + 64, lo);
    }
}

template <bool kAll, bool kSplit>
__device__ __forceinline__ float stage_p(const uint32_t (&s0)[32], const uint32_t (&s1)[32], const uint32_t (&s2)[32],
                                         const uint32_t (&s3)[32], int lim, float sl, float nbase, uint32_t dst) {
    float ls[4] = {0.f, 0.f, 0.f, 0.f};
    quarter_p<kAll, kSplit>(s0, lim, sl, nbase, dst, ls);
    quarter_p<kAll, kSplit>(s1, lim - 32, sl, nbase, dst + 16, ls);
    quarter_p<kAll, kSplit>(s2, lim - 64, sl, nbase, dst + 32, ls);
    quarter_p<kAll, kSplit>(s3, lim - 96, sl, nbase, dst + 48, ls);
    return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

template <bool kNeg>
__device__ __forceinline__ float stage_max(const uint32_t (&s0)[32], const uint32_t (&s1)[32], const uint32_t (&s2)[32],
                                           const uint32_t (&s3)[32], int lim, bool unmasked) {
    if (unmasked)
        return fmaxf(fmaxf(quarter_max<true, kNeg>(s0, lim), quarter_max<true, kNeg>(s1, lim)),
                     fmaxf(quarter_max<true, kNeg>(s2, lim), quarter_max<true, kNeg>(s3, lim)));
    return fmaxf(fmaxf(quarter_max<false, kNeg>(s0, lim), quarter_max<false, kNeg>(s1, lim - 32)),
                 fmaxf(quarter_max<false, kNeg>(s2, lim - 64), quarter_max<false, kNeg>(s3, lim - 96)));
}

// O (the row's D fp32 columns of tensor memory at `taddr`) *= f.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 8) {
        uint32_t o[8];
        tmem_ld8(taddr + c, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st8_nowait(taddr + c, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    }
    tmem_wait_st();
}

// The softmax of one tile's rows, stage by stage; `pos` the row's own key.  Returns false when a
// wait ran out.  tcgen05.ld / st are warp-collective, so every branch that leads to one is the warp's.
template <int D, bool kSplit>
__device__ __forceinline__ bool softmax_rows(Bars<D>* bars, int t, int n, int pos, float sl, uint32_t tm_s,
                                             uint32_t tm_o, float& l_out) {
    float m_used = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
        if (__any_sync(0xffffffffu, !mbar_wait(&bars->s_full[t], j & 1))) return false;
        tc_fence_after();
        const int lim = pos - j * kKeys;
        const bool unmasked = __all_sync(0xffffffffu, lim >= kKeys - 1);
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tmem_ld32_async(tm_s, s0);
        tmem_ld32_async(tm_s + 32, s1);
        tmem_ld32_async(tm_s + 64, s2);
        tmem_ld32_async(tm_s + 96, s3);
        tmem_wait_ld(s0);
        tmem_wait_ld(s1);
        tmem_wait_ld(s2);
        tmem_wait_ld(s3);
        float sum = 0.f;
        bool full = __any_sync(0xffffffffu, m_used == -INFINITY && lim >= 0);
        auto p = [&] {
            const float nbase = m_used == -INFINITY ? 0.f : -m_used;
            return unmasked ? stage_p<true, kSplit>(s0, s1, s2, s3, lim, sl, nbase, tm_s)
                            : stage_p<false, kSplit>(s0, s1, s2, s3, lim, sl, nbase, tm_s);
        };
        if (!full) {
            sum = p();
            full = __any_sync(0xffffffffu, !(sum <= kSpecSumLimit));
        }
        if (full) {
            const float mx = sl < 0.f ? stage_max<true>(s0, s1, s2, s3, lim, unmasked)
                                      : stage_max<false>(s0, s1, s2, s3, lim, unmasked);
            const float mxs = mx == -INFINITY ? -INFINITY : mx * fabsf(sl);  // log2 units
            const float m_new = fmaxf(m_used, mxs);
            const bool rebase = m_new > m_used + kRescaleThreshold;  // always for the first visible key
            // S_t(j) was issued after P_t V (j-1) and is complete, so O may be changed
            if (__any_sync(0xffffffffu, rebase && m_used != -INFINITY))
                scale_o<D>(tm_o, rebase && m_used != -INFINITY ? fast_exp2(m_used - m_new) : 1.f);
            if (rebase) {
                l *= m_used == -INFINITY ? 0.f : fast_exp2(m_used - m_new);
                m_used = m_new;
            }
            sum = p();
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[t]);
    }
    l_out = l;
    return true;
}

// The two-part form as a function of its own: its code stays out of the usual tile's way.
template <int D>
__device__ __noinline__ bool softmax_rows_split(Bars<D>* bars, int t, int n, int pos, float sl, uint32_t tm_s,
                                                uint32_t tm_o, float* l_out) {
    return softmax_rows<D, true>(bars, t, n, pos, sl, tm_s, tm_o, *l_out);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) packed_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                             const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const __grid_constant__ CUtensorMap tm_out,
                                                             const __grid_constant__ TcArgs a) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars<D>* bars = reinterpret_cast<Bars<D>*>(smem + L::kOffBars);
    int* bad = reinterpret_cast<int*>(smem + L::kOffBad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blockIdx.x = (rank * batch + b) * subs + sub: rank 0 holds every sequence's last (longest) pair
    const int sub = (int)(blockIdx.x % (unsigned)a.subs);
    const int rb = (int)(blockIdx.x / (unsigned)a.subs);
    const int b = rb % a.p.batch, rank = rb / a.p.batch;
    const int head0 = sub * a.th, kvh = head0 / (a.p.num_heads / a.p.num_kv_heads);
    pdl_wait();
    const bool report = rank == 0 && sub == 0 && threadIdx.x == 0;
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(a.p.status, kDevOutOfRange);
        return;
    }
    const int c0 = a.p.cu_lens[b], c1 = a.p.cu_lens[b + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.p.num_tokens) {
        if (report) atomicOr(a.p.status, kDevOutOfRange);
        return;
    }
    if (c1 - c0 > a.p.max_len && report) atomicOr(a.p.status, kDevOutOfRange);
    const int len = min(c1 - c0, a.p.max_len);
    const int pairs = (len + 2 * a.tpt - 1) / (2 * a.tpt);
    if (rank >= pairs) return;
    const int tok0 = (pairs - 1 - rank) * 2 * a.tpt;  // first token of tile 0
    int ntok[2], n[2];                                // tokens and stages of the two tiles
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        ntok[t] = max(0, min(a.tpt, len - tok0 - t * a.tpt));
        n[t] = ntok[t] > 0 ? (tok0 + t * a.tpt + ntok[t] + kKeys - 1) / kKeys : 0;
    }
    const int nst = max(n[0], n[1]);
    const int first_masked = (tok0 + 1) / kKeys;      // stages before it are visible to every row

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kKSlots; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < L::kVSlots; ++s) {
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 3);  // the products' commit, and the two warps that look V over
            mbar_init(&bars->v_clean[s], 64);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 128);
            mbar_init(&bars->o_final[t], 1);
        }
        mbar_init(&bars->drain, 1);
        bars->any_bad = 0;
        fence_mbar_init();
    }
    if (threadIdx.x >= kCleanWarp * 32)
        for (int i = threadIdx.x - kCleanWarp * 32; i < 3 * D; i += 64) bad[i] = INT_MAX;
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == kLoadWarp) {
        // ---------------------------------------------------------------- TMA loads, in the order of use
        if (lane == 0) {
            bool ok = true;
            const uint32_t q_bytes = (uint32_t)(a.tpt * a.th * 128 * L::kHalves);
            auto load_q = [&](int t) {
                mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
                // a copy a half: those of a box with fewer than 128 rows would lie closer than kHalf
                for (int h = 0; h < L::kHalves; ++h)
                    tma_load_rows(smem + L::kOffQ + t * L::kTile + h * kHalf, &tm_q, head0, c0 + tok0 + t * a.tpt, h,
                                  &bars->q_full[t]);
            };
            auto load = [&](int off, const CUtensorMap* map, int j, uint64_t* full) {
                mbar_arrive_expect_tx(full, L::kTile);
                tma_load_rows(smem + off, map, kvh, c0 + j * kKeys, 0, full);
            };
            prefetch_tensormap(&tm_q);
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            if (n[0] > 0) load_q(0);
            int k_issued = 0, v_issued = 0;
            for (int j = 0; j < nst && ok; ++j) {
                const int ks = j % L::kKSlots, vs = j % L::kVSlots;
                if (j >= L::kKSlots) ok = mbar_wait(&bars->k_empty[ks], ((j / L::kKSlots) & 1) ^ 1);
                if (!ok) break;
                load(L::kOffK + ks * L::kTile, &tm_k, j, &bars->k_full[ks]);
                ++k_issued;
                if (j == 0 && n[1] > 0) load_q(1);
                if (j >= L::kVSlots) ok = mbar_wait(&bars->v_empty[vs], ((j / L::kVSlots) & 1) ^ 1);
                if (!ok) break;
                load(L::kOffV + vs * L::kTile, &tm_v, j, &bars->v_full[vs]);
                ++v_issued;
            }
            // before the CTA may leave: every copy issued here has landed
            for (int t = 0; t < 2; ++t)
                if (n[t] > 0 && (t == 0 || k_issued > 0) && !mbar_wait(&bars->q_full[t], 0)) ok = false;
            for (int j = max(0, k_issued - L::kKSlots); j < k_issued; ++j)
                if (!mbar_wait(&bars->k_full[j % L::kKSlots], (j / L::kKSlots) & 1)) ok = false;
            for (int j = max(0, v_issued - L::kVSlots); j < v_issued; ++j)
                if (!mbar_wait(&bars->v_full[j % L::kVSlots], (j / L::kVSlots) & 1)) ok = false;
            if (!ok) atomicOr(a.p.status, kDevTimeout);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idesc_s = tc_idesc_bf16(kRows, kKeys, false);
        constexpr uint32_t idesc_o = tc_idesc_bf16(kRows, D, true);
        const uint64_t qd0 = smem_desc_sw128(smem_u32(smem + L::kOffQ), 0, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kOffK), 0, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + L::kOffV), kHalf, 1024);
        const bool split[2] = {a.split_all || tok0 + 1 <= kFewKeys, a.split_all || tok0 + a.tpt + 1 <= kFewKeys};
        auto issue_qk = [&](int t, int j) {
            const uint64_t qd = qd0 + (uint64_t)((t * L::kTile) >> 4);
            const uint64_t kd = kd0 + (uint64_t)(((j % L::kKSlots) * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                tc_mma_ew(tmem + t * kKeys, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
            }
            tc_commit_ew(&bars->s_full[t]);
        };
        auto issue_pv = [&](int t, int j) {
            const uint64_t vd = vd0 + (uint64_t)(((j % L::kVSlots) * L::kTile) >> 4);
            const uint32_t to = tmem + L::kColsO + t * D, tp = tmem + t * kKeys;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                tc_mma_ts_ew(to, tp + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
            if (split[t]) {  // the low parts of P, against the same V
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    tc_mma_ts_ew(to, tp + 64 + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, 1u);
            }
            if (j + 1 == n[t]) tc_commit_ew(&bars->o_final[t]);
        };
        bool ok = mbar_wait_warp(&bars->k_full[0], 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (n[t] == 0 || !ok) continue;
            ok = mbar_wait_warp(&bars->q_full[t], 0);
            if (!ok) continue;
            tc_fence_after();
            issue_qk(t, 0);
        }
        if (ok) tc_commit_ew(&bars->k_empty[0]);
        for (int j = 0; j < nst && ok; ++j) {
            // V(j) and K(j+1) are normally long in place, so they are waited for before P
            const int vs = j % L::kVSlots;
            ok = j < first_masked ? mbar_wait_warp(&bars->v_full[vs], (j / L::kVSlots) & 1)
                                  : mbar_wait_warp(&bars->v_clean[vs], ((j - first_masked) / L::kVSlots) & 1);
            if (ok && j + 1 < nst) ok = mbar_wait_warp(&bars->k_full[(j + 1) % L::kKSlots], ((j + 1) / L::kKSlots) & 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (j >= n[t] || !ok) continue;
                ok = mbar_wait_warp(&bars->p_full[t], j & 1);
                if (!ok) continue;
                tc_fence_after();
                issue_pv(t, j);
                if (j + 1 < n[t]) issue_qk(t, j + 1);  // S_t takes the place of P_t, after its product in issue order
            }
            if (!ok) break;
            tc_commit_ew(&bars->v_empty[vs]);
            if (j + 1 < nst) tc_commit_ew(&bars->k_empty[(j + 1) % L::kKSlots]);
        }
        // every MMA this warp issued has finished before the tensor memory is released
        tc_commit_ew(&bars->drain);
        if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
        if (!ok && lane == 0) atomicOr(a.p.status, kDevTimeout);
    } else if (warp >= kCleanWarp) {
        // ---------------------------------------------------------------- V of the stages with masked keys
        const int i0 = threadIdx.x - kCleanWarp * 32;
        bool ok = true;
        // every stage is followed, so that a barrier's phases cannot pass these warps by
        for (int j = 0; j < nst && ok; ++j) {
            const int vs = j % L::kVSlots;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[vs], (j / L::kVSlots) & 1));
            if (!ok) break;
            if (j < first_masked) {
                if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
                continue;
            }
            uint8_t* tile = smem + L::kOffV + vs * L::kTile;
            // a pass that only reads (its loads run ahead), and only where something was found the repair
            uint32_t seen = 0;
#pragma unroll 8
            for (int i = i0; i < L::kTile / 16; i += 64) seen |= not_finite(*reinterpret_cast<const uint4*>(tile + 16 * i));
            if (seen) {
                for (int i = i0; i < L::kTile / 16; i += 64) {
                    uint4* at = reinterpret_cast<uint4*>(tile + 16 * i);
                    if (!not_finite(*at)) continue;
                    const int half = i / (kHalf / 16), row = i / 8 % kRows, col = half * 64 + ((i & 7) ^ (row & 7)) * 8;
                    for (int e = 0; e < 8; ++e) {
                        uint16_t* x = reinterpret_cast<uint16_t*>(at) + e;
                        if ((*x & 0x7f80u) != 0x7f80u) continue;
                        const int what = (*x & 0x7fu) ? 0 : (*x & 0x8000u) ? 2 : 1;
                        atomicMin(&bad[what * D + col + e], j * kKeys + row);
                        *x = 0;
                    }
                }
                bars->any_bad = 1;
                fence_proxy_async_smem();
            }
            mbar_arrive(&bars->v_clean[vs]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
        }
        if (!ok && lane == 0) atomicOr(a.p.status, kDevTimeout);
    } else {
        // ---------------------------------------------------------------- softmax and epilogue, one row a thread
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int first = tok0 + t * a.tpt;                    // the tile's first token
        const int qi = r / a.th, hh = r - qi * a.th;
        const bool valid = qi < ntok[t];
        const int pos = valid ? first + qi : -1;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm_s = tmem + lanes + t * kKeys, tm_o = tmem + lanes + L::kColsO + t * D;
        if (n[t] > 0) {
            float l = 0.f;
            const bool two = a.split_all || first + 1 <= kFewKeys;
            bool ok = two ? softmax_rows_split<D>(bars, t, n[t], pos, a.scale_log2, tm_s, tm_o, &l)
                          : softmax_rows<D, false>(bars, t, n[t], pos, a.scale_log2, tm_s, tm_o, l);
            if (ok) ok = !__any_sync(0xffffffffu, !mbar_wait(&bars->o_final[t], 0));
            if (!ok) {
                if (lane == 0) atomicOr(a.p.status, kDevTimeout);
            } else {
                tc_fence_after();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const bool any_bad = bars->any_bad != 0;
                uint8_t* qs = smem + L::kOffQ + t * L::kTile;
                __nv_bfloat16* dst = a.p.out + ((size_t)(c0 + first + qi) * a.p.num_heads + head0 + hh) * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tm_o + c, o);
                    if (any_bad) {
                        for (int e = 0; e < 32; ++e) {
                            float x = __uint_as_float(o[e]);
                            if (pos >= bad[D + c + e]) x += INFINITY;
                            if (pos >= bad[2 * D + c + e]) x -= INFINITY;
                            if (pos >= bad[c + e]) x = NAN;
                            o[e] = __float_as_uint(x);
                        }
                    }
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 v;
                            v.x = pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                            v.y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                            v.z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                            v.w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                            *reinterpret_cast<uint4*>(dst + c + e) = v;
                        }
                    }
                }
                (void)qs;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    pdl_trigger();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Heads of a group that one tile holds: the largest divisor of the group up to 16.  (Few heads a tile make
// its token range long, which wastes the diagonal's stages; a divisor that does not divide 128 leaves
// up to 11 of the 128 rows empty.)
int tile_heads(int group) {
    for (int th = std::min(group, 16); th > 1; --th)
        if (group % th == 0) return th;
    return 1;
}

template <int D>
cudaError_t launch(const PackedArgs& a, cudaStream_t stream) {
    using L = Layout<D>;
    static OncePerDevice configured;
    const cudaError_t e = configured.run([] {
        return cudaFuncSetAttribute(packed_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kSmem);
    });
    if (e != cudaSuccess) return e;
    TcArgs t;
    t.p = a;
    t.th = tile_heads(a.num_heads / a.num_kv_heads);
    t.tpt = kRows / t.th;
    t.subs = a.num_heads / t.th;
    t.pairs = (a.max_len + 2 * t.tpt - 1) / (2 * t.tpt);
    t.scale_log2 = a.scale * kLog2e;
    t.split_all = std::fabs(a.scale) * std::sqrt((float)D) > kSplitScale;
    CUtensorMap q, k, v, out;
    if (!strided_map(&q, a.q, a.num_tokens, a.num_heads, D, a.q_stride, t.th, t.tpt, 1) ||
        !strided_map(&k, a.k, a.num_tokens, a.num_kv_heads, D, a.k_stride, 1, kKeys, L::kHalves) ||
        !strided_map(&v, a.v, a.num_tokens, a.num_kv_heads, D, a.v_stride, 1, kKeys, L::kHalves) ||
        !strided_map(&out, a.out, a.num_tokens, a.num_heads, D, (long long)a.num_heads * D, t.th, t.tpt, 1))
        return cudaErrorInvalidValue;
    const long long ctas = (long long)t.pairs * a.batch * t.subs;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, packed_kernel<D>, q, k, v, out, t);
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedArgs& a, cudaStream_t stream) {
    return a.head_dim == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace pa
