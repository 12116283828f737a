// pa_packed.cu -- causal attention over packed prompts (pa_prefill_packed) on the 5th-generation
// tensor cores.
//
//   o_i = sum_{j <= i} softmax_j(scale <q_i, k_j>) v_j   within each sequence
//
// A query tile is 128 rows of (token, head) pairs: th heads of one kv head's group, 128 / th tokens, so
// the heads of a group share every K and V tile and the tile of a short prompt is well filled.  An
// item is two neighbouring tiles of one sequence and head group; a CTA, one an SM, walks its keys in stages
// of 128:
//   S_t = Q_t K^T     tcgen05.mma M = N = 128, both operands from shared memory, S_t in tensor memory
//   softmax           one thread a row: P_t (bf16) over the first half of S_t
//   O_t += P_t V      tcgen05.mma M = 128, N = d, P_t from tensor memory
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (d each): all of it at d = 128.  While one tile's
// softmax runs, the tensor core works for the other; per tile and stage it is busy for 1024 cycles at
// d = 128 (two products of 128 x 128 x 128), which bounds the kernel at long prompts.  N = 128
// matters: with both operands in shared memory, 64-key products are bound by its bandwidth.
//
// A CTA takes item after item: once the copies of one are on their way it asks for a block of the grid that has
// not started (clusterlaunchcontrol), and the next item's Q, K and V arrive and its first scores are
// computed under the end of the one before.  Items go sequence by sequence, each sequence's longest first (longest
// first altogether was no faster: 7 prompts at d = 64 94 us against 92, 48 prompts 219 against 224).
//
// Base of the softmax: a stage is taken against the row's current base, 2^8 to begin with.  Only a stage whose sum passes
// 2^8 of it, or a row's first one whose sum is below 2^-16 of it, takes the maximum (at d = 128 so does any stage with a
// masked key); where that is 2^(1/2) above the base (a sum that passes has one at least twice it), or in a first stage far
// below it, the base moves there and O is rescaled.  (Kept until 2^8 above it in masked stages, for which the two need
// telling apart: 48 prompts 236 us against 207.)  So P stays below 2^8, as in the prefill over a pool, and sums of P V in
// fp32's range for V up to 2^100 and down to 2^-100.  (A row's first stage is the first in which a key has any
// weight: those before may hold scores of -inf alone.)  P is rounded to bf16 and the normaliser sums the
// rounded values, so their rounding moves weight between keys but not its total.  Where few keys can dominate (a
// tile with a row of at most 128 keys, or |scale| sqrt(d) > 2) P enters as two bf16 parts, in the two halves of S_t.
//
// Measured: 1 x 16384 tokens (16 / 2 heads of 128) 650 us, 1.69 PFLOP/s; 48 prompts of up to 1300 tokens (32 / 8 heads
// of 128) 213 us; 7 of up to 2200 (24 / 8 heads of 64) 82 us.  Long prompts are bound by the tensor core, d = 64 by the
// softmax, short prompts by what an item costs besides its stages and by masked stages, one of the 3.9 that an item of
// the 48 has: they read their scores twice, and work through quarters that no row of the warp sees.
// Also tried: two softmax threads a row (1 x 16384 969 us against 774 then), an issuing warp a tile (48 prompts 266
// us against 260), both tiles half a stage apart (no gain).
//
// Masked keys have P = 0, and 0 times a NaN or an infinity in V is NaN.  So in the stages that hold a
// key masked for some row, a warp looks V over before its product: what is not finite is replaced
// by 0, and the first token it was seen at noted per column; rows at or behind it get it back.
//
// Warps: 0-3 and 4-7 softmax and outputs of tiles 0 and 1, 8 MMA issue and tensor memory, 9 TMA loads, 10
// the look at V, 11 the items.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pa_internal.h"
#include "pa_step.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;              // rows of a query tile (MMA M)
constexpr int kKeys = 128;              // keys a stage (MMA N of Q K^T)
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10, kItemWarp = 11;
constexpr int kThreads = 384;
constexpr int kHalf = kRows * 128;      // [128 rows][64 columns] bf16
constexpr float kBase = 8.f;            // the base to begin with
constexpr float kRescaleThreshold = 0.5f;
constexpr float kSumMost = 256.f, kFirstSumLeast = 0x1p-16f;  // a stage's sum outside takes the maximum
constexpr float kFirstLeast = -8.f;     // a first maximum below it becomes the base
constexpr float kSplitScale = 2.f;      // |scale| sqrt(d) past this: P in two parts
constexpr int kFewKeys = 128;           // a tile with a row of at most this many keys: the same
constexpr int kNoRow = INT_MAX;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalf;      // a tile of Q, K or V
    static constexpr int kKSlots = 3, kVSlots = D == 64 ? 3 : 2;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + kKSlots * kTile;
    static constexpr int kOffBars = kOffV + kVSlots * kTile;
    static constexpr int kOffItem = kOffBars + 384;    // two items
    static constexpr int kOffBad = kOffItem + 128;     // [3][D] first token of a NaN, +inf, -inf in a column of V
    static constexpr int kSmem = kOffBad + 3 * D * 4;
    static constexpr int kColsO = 2 * kKeys;           // tensor memory: S_0, S_1, O_0, O_1
    static constexpr int kTmemCols = 512;
};
static_assert(Layout<128>::kSmem <= 227 * 1024, "shared memory");

// One item: two tiles of sequence rows [row, row + len), the first of them at token tok0.
struct Item {
    int row, len, tok0, head0, kvh;
    int none;     // there is none: the CTA is done
    int any_bad;  // a value of V in a stage with masked keys was not finite
};
static_assert(sizeof(Item) <= 64, "item");

// A barrier is waited for by the parity of its phase, so a phase may be over only once all who wait for the one before
// have seen that: behind each lies something that they do after their wait (a tile is loaded again after the commits,
// and the arrival of the warp that looks at V, that empty it; S_t, O_t and Q_t change hands in turn; an item's slot is
// written again after every warp has given it back).
template <int D>
struct Bars {
    uint64_t q_full[2], q_empty[2], k_full[Layout<D>::kKSlots], k_empty[Layout<D>::kKSlots], v_full[Layout<D>::kVSlots],
        v_empty[Layout<D>::kVSlots], v_clean[Layout<D>::kVSlots], s_full[2], p_full[2], o_full[2], o_empty[2];
    uint64_t item_full[2], item_empty[2], soon, next, drain;
    uint4 reply;  // of clusterlaunchcontrol
    uint32_t tmem_base;
};
static_assert(sizeof(Bars<64>) <= 384 && sizeof(Bars<128>) <= 384, "barrier block");

struct TcArgs {
    PackedArgs p;
    int th, tpt;       // heads and tokens of a tile
    int subs;          // tiles' head groups: num_heads / th
    int split_all;
    float scale_log2;  // scale * log2(e), signed
};

// (a0, a1) += the two bf16 values of a packed word, each widened exactly.
__device__ __forceinline__ void add_bf16x2(float& a0, float& a1, uint32_t w) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(w));
}

// The largest visible sgn * score of a quarter of a stage (32 keys, `lim` the last visible of them).
__device__ __forceinline__ float quarter_max(const uint32_t (&s)[32], int lim, float sgn) {
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = c + e > lim ? -INFINITY : __uint_as_float(s[c + e]) * sgn;
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
#pragma unroll
    for (int c0 = 0; c0 < 32; c0 += 16) {
        uint32_t w[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + 2 * i;
            float x0, x1;
            fma_x2(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl, sl, nbase, nbase);
            if (!kAll) {
                x0 = c > lim ? -INFINITY : x0;  // 2^-inf = 0
                x1 = c + 1 > lim ? -INFINITY : x1;
            }
            x0 = fast_exp2(x0);
            x1 = fast_exp2(x1);
            w[i] = pack_bf16x2(x0, x1);
            add_bf16x2(ls[0], ls[1], w[i]);
            if (kSplit) {
                lo[i] = pack_bf16x2(x0 - bf16_lo(w[i]), x1 - bf16_hi(w[i]));
                add_bf16x2(ls[2], ls[3], lo[i]);
            }
        }
        tmem_st8_nowait(dst + c0 / 2, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        if (kSplit) tmem_st8_nowait(dst + 64 + c0 / 2, lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]);
    }
}

// A quarter seen whole, its P as 16 words (quarter_p<true, false> without its stores).
__device__ __forceinline__ void quarter_w(const uint32_t (&s)[32], float sl, float nbase, uint32_t* w, float (&ls)[4]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x0, x1;
        fma_x2(x0, x1, __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]), sl, sl, nbase, nbase);
        w[i] = pack_bf16x2(fast_exp2(x0), fast_exp2(x1));
        add_bf16x2(ls[(i & 1) * 2], ls[(i & 1) * 2 + 1], w[i]);
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

// The softmax of one tile's rows, stage by stage (the first is number `sc` of the tile's); `pos` the row's own
// key, kNoRow for a row past the sequence's end or the tile's heads: nothing of it is masked, it has no say in
// what its warp does, and what it computes from whatever its Q holds is not stored.  (With all its keys masked its warp
// took every stage as a masked one: 6 x 4000 tokens, group 3 at d = 128, 601 us against 382.)  Returns false when a
// wait ran out.  tcgen05.ld / st are warp-collective, so every branch that leads to one is the warp's.
template <int D, bool kSplit>
__device__ __forceinline__ bool softmax_rows(Bars<D>* bars, int t, int sc, int n, int pos, float sl, uint32_t tm_s,
                                             uint32_t tm_o, float& l_out) {
    const bool there = pos != kNoRow, none = D == 64 && !__any_sync(0xffffffffu, there);
    float base = kBase, l = 0.f;  // P = 2^(score - base)
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++sc) {
        if (__any_sync(0xffffffffu, !mbar_wait(&bars->s_full[t], sc & 1))) return false;
        // No row of the warp's is anybody's: P is what it is.  (At d = 64, where the code is larger, this spares short
        // prompts the variant without masks: 256 x 48 tokens 58 us against 75.)
        if (D == 64 && none) {
            mbar_arrive(&bars->p_full[t]);
            continue;
        }
        tc_fence_after();
        const int lim = pos - j * kKeys;
        const bool unmasked = __all_sync(0xffffffffu, lim >= kKeys - 1);
        uint32_t s0[32], s1[32], s2[32], s3[32];
        float sum = 0.f;
        // At d = 128, where the tensor core is to be kept busy, the usual stage is taken in quarters and all others in
        // little code (the whole below for both: 48 prompts 226 us against 219, 1 x 16384 773 against 655).  At d = 64
        // the softmax bounds the kernel, and loads and P of a stage run on without a wait between them (as at d = 128:
        // 7 prompts 120 us against 92).
        if constexpr (D == 128) {
            bool done = false;
            if (!kSplit && unmasked) {
                // quarter by quarter, each loaded while the one before is worked on
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t w[32];
                tmem_ld32(tm_s, s0);
                tmem_ld32_async(tm_s + 32, s1);
                quarter_w(s0, sl, -base, w, ls);
                tmem_wait_ld(s1);
                tmem_ld32_async(tm_s + 64, s2);
                quarter_w(s1, sl, -base, w + 16, ls);
                tmem_st32_nowait(tm_s, w);
                tmem_wait_ld(s2);
                tmem_ld32_async(tm_s + 96, s3);
                quarter_w(s2, sl, -base, w, ls);
                tmem_wait_ld(s3);
                quarter_w(s3, sl, -base, w + 16, ls);
                tmem_st32_nowait(tm_s + 32, w);
                sum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
                done = true;
            }
            // a sum past 2^8, or a first one below 2^-16: once more against a new base
            if (done && __any_sync(0xffffffffu, there && (!(sum <= kSumMost) || (l == 0.f && sum < kFirstSumLeast)))) {
                tmem_wait_st();  // the scores that P went over
                tmem_st32_nowait(tm_s, s0);
                tmem_st32_nowait(tm_s + 32, s1);
                tmem_wait_st();
                done = false;
            }
            if (!done) {
                // the maximum first, so that P is written once
                const float sgn = sl < 0.f ? -1.f : 1.f;
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t s[32];
                    tmem_ld32(tm_s + c, s);
                    mx = fmaxf(mx, quarter_max(s, lim - c, sgn));
                }
                mx *= fabsf(sl);
                // (a maximum that is no number leaves the base: the row's result is none either)
                float f = 1.f;
                if (there && fabsf(mx) < INFINITY && (mx > base + kRescaleThreshold || (l == 0.f && mx < kFirstLeast))) {
                    f = l == 0.f ? 1.f : fast_exp2(base - mx);
                    base = mx;
                }
                // S_t(j) was issued after P_t V (j-1) and is complete, so O may be changed
                if (j > 0) {
                    if (__any_sync(0xffffffffu, f != 1.f)) scale_o<D>(tm_o, f);
                    l *= f;
                }
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                if (kSplit) {
                    tmem_ld32_async(tm_s, s0);
                    tmem_ld32_async(tm_s + 32, s1);
                    tmem_ld32_async(tm_s + 64, s2);
                    tmem_ld32_async(tm_s + 96, s3);
                    tmem_wait_ld(s0);
                    tmem_wait_ld(s1);
                    tmem_wait_ld(s2);
                    tmem_wait_ld(s3);
                    quarter_p<false, true>(s0, lim, sl, -base, tm_s, ls);
                    quarter_p<false, true>(s1, lim - 32, sl, -base, tm_s + 16, ls);
                    quarter_p<false, true>(s2, lim - 64, sl, -base, tm_s + 32, ls);
                    quarter_p<false, true>(s3, lim - 96, sl, -base, tm_s + 48, ls);
                } else {
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t s[32];
                        tmem_ld32(tm_s + c, s);
                        quarter_p<false, false>(s, lim - c, sl, -base, tm_s + c / 2, ls);
                    }
                }
                sum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
            }
        } else {
            tmem_ld32_async(tm_s, s0);
            tmem_ld32_async(tm_s + 32, s1);
            tmem_ld32_async(tm_s + 64, s2);
            tmem_ld32_async(tm_s + 96, s3);
            tmem_wait_ld(s0);
            tmem_wait_ld(s1);
            tmem_wait_ld(s2);
            tmem_wait_ld(s3);
            sum = unmasked ? stage_p<true, kSplit>(s0, s1, s2, s3, lim, sl, -base, tm_s)
                           : stage_p<false, kSplit>(s0, s1, s2, s3, lim, sl, -base, tm_s);
            // a sum past 2^8, or a first one below 2^-16: once more against a new base
            if (__any_sync(0xffffffffu, there && (!(sum <= kSumMost) || (l == 0.f && sum < kFirstSumLeast)))) {
                const float sgn = sl < 0.f ? -1.f : 1.f;
                const float m0 = fmaxf(quarter_max(s0, lim, sgn), quarter_max(s1, lim - 32, sgn));
                const float m1 = fmaxf(quarter_max(s2, lim - 64, sgn), quarter_max(s3, lim - 96, sgn));
                const float mx = fabsf(sl) * fmaxf(m0, m1);
                // (a maximum that is no number leaves the base: the row's result is none either)
                float f = 1.f;
                if (there && fabsf(mx) < INFINITY && (l == 0.f || mx > base + kRescaleThreshold)) {
                    f = l == 0.f ? 1.f : fast_exp2(base - mx);
                    base = mx;
                }
                // S_t(j) was issued after P_t V (j-1) and is complete, so O may be changed
                if (j > 0) {
                    if (__any_sync(0xffffffffu, f != 1.f)) scale_o<D>(tm_o, f);
                    l *= f;
                }
                sum = unmasked ? stage_p<true, kSplit>(s0, s1, s2, s3, lim, sl, -base, tm_s)
                               : stage_p<false, kSplit>(s0, s1, s2, s3, lim, sl, -base, tm_s);
            }
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[t]);
    }
    l_out = l;
    return true;
}

// Tokens and key stages of an item's tiles.
struct Tiles {
    int ntok[2], n[2], nst, first_masked;
    // (through shuffles, so that the compiler knows them, and all that follows from them, to be the warp's)
    __device__ __forceinline__ Tiles(const Item* it, int tpt) {
        const int len = __shfl_sync(0xffffffffu, it->len, 0), tok0 = __shfl_sync(0xffffffffu, it->tok0, 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            ntok[t] = max(0, min(tpt, len - tok0 - t * tpt));
            n[t] = ntok[t] > 0 ? (tok0 + t * tpt + ntok[t] + kKeys - 1) / kKeys : 0;
        }
        nst = max(n[0], n[1]);
        first_masked = (tok0 + 1) / kKeys;  // stages before it are visible to every row
    }
};

// The items as one warp sees them, in order; next() waits for one and done() gives it back.
template <int D>
struct Items {
    Bars<D>* bars;
    uint8_t* slots;
    int n = 0;
    __device__ __forceinline__ Item* next(bool& ok) {
        ok = __all_sync(0xffffffffu, ok);
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->item_full[n & 1], (n >> 1) & 1));
        Item* it = reinterpret_cast<Item*>(slots + (n & 1) * 64);
        return ok && !it->none ? it : nullptr;
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->item_empty[n & 1]);
        ++n;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) packed_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                             const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const __grid_constant__ TcArgs a) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars<D>* bars = reinterpret_cast<Bars<D>*>(smem + L::kOffBars);
    int* bad = reinterpret_cast<int*>(smem + L::kOffBad);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(a.p.status, kDevOutOfRange);
        return;
    }
    if (threadIdx.x == kItemWarp * 32) {
        for (int s = 0; s < L::kKSlots; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < L::kVSlots; ++s) {
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 2);  // the products' commit, and the warp that looks V over
            mbar_init(&bars->v_clean[s], 32);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->q_empty[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 128);
            mbar_init(&bars->o_full[t], 1);
            mbar_init(&bars->o_empty[t], 128);
            mbar_init(&bars->item_full[t], 1);
            mbar_init(&bars->item_empty[t], kItemWarp);  // every other warp
        }
        mbar_init(&bars->soon, 1);
        mbar_init(&bars->next, 1);
        mbar_init(&bars->drain, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    pdl_wait();
    bool ok = true;
    Items<D> items{bars, smem + L::kOffItem};

    // registers: 256 softmax threads of 200 and 128 others of 96 are fewer than the 384 x 168 of the launch
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == kItemWarp) {
            // ---------------------------------------------------------------- the items
            // id = pair * subs + sub
            unsigned id = blockIdx.x;
            uint32_t phase = 0;
            PairWalk walk(a.p, 2 * a.tpt);
            bool reports = id == 0;
            for (int n = 0; ok; ++n) {
                bool there = true;
                if (n > 0) {  // the last copies of the item before are on their way, and a slot is free
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->soon, (n - 1) & 1));
                    if (ok && n > 1)
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->item_empty[n & 1], ((n >> 1) & 1) ^ 1));
                    if (ok) there = take_block(&bars->reply, &bars->next, phase, id, ok);
                }
                Item* it = reinterpret_cast<Item*>(smem + L::kOffItem + (n & 1) * 64);
                while (ok && there) {  // (the grid has blocks past the last pair; they may come before others)
                    reports |= id == 0;
                    const unsigned pair = id / (unsigned)a.subs, sub = id % (unsigned)a.subs;
                    if (walk.find(pair)) {
                        if (walk.owns(pair)) {  // one lane
                            it->row = walk.row;
                            it->len = walk.len;
                            it->tok0 = walk.first_token(pair);
                            it->head0 = (int)sub * a.th;
                            it->kvh = it->head0 / (a.p.num_heads / a.p.num_kv_heads);
                            it->none = 0;
                            it->any_bad = 0;
                        }
                        break;
                    }
                    there = take_block(&bars->reply, &bars->next, phase, id, ok);
                }
                if (!ok) break;
                if (!there && lane == 0) it->none = 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->item_full[n & 1]);
                if (!there) break;
            }
            // (sequences behind the last pair that anybody took are looked at for their offsets, too)
            if (reports)
                for (int b = walk.b0 + 32; b < a.p.batch; b += 32) walk.look(b + lane);
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- TMA loads, in the order of use
            const uint32_t q_bytes = (uint32_t)(a.tpt * a.th * 128 * L::kHalves);
            int kc = 0, vc = 0, q0 = 0, q1 = 0;  // copies issued
            for (const Item* it; (it = items.next(ok)); items.done()) {
                const Tiles w(it, a.tpt);
                if (lane == 0) {
                    const int base = it->row, tok0 = it->tok0, head0 = it->head0, kvh = it->kvh;
                    auto load_q = [&](int t, int& qc) {
                        if (qc > 0 && ok) ok = mbar_wait(&bars->q_empty[t], (qc & 1) ^ 1);
                        if (!ok) return;
                        mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
                        // a copy a half: those of a box with fewer than 128 rows would lie closer than kHalf
                        for (int h = 0; h < L::kHalves; ++h)
                            tma_load_rows(smem + L::kOffQ + t * L::kTile + h * kHalf, &tm_q, head0,
                                          base + tok0 + t * a.tpt, h,
                                          &bars->q_full[t]);
                        ++qc;
                    };
                    load_q(0, q0);
                    for (int j = 0; j < w.nst && ok; ++j) {
                        const int ks = kc % L::kKSlots, vs = vc % L::kVSlots;
                        if (kc >= L::kKSlots) ok = mbar_wait(&bars->k_empty[ks], ((kc / L::kKSlots) & 1) ^ 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars->k_full[ks], L::kTile);
                        tma_load_rows(smem + L::kOffK + ks * L::kTile, &tm_k, kvh, base + j * kKeys, 0,
                                      &bars->k_full[ks]);
                        ++kc;
                        if (j == 0 && w.n[1] > 0) load_q(1, q1);
                        if (ok && vc >= L::kVSlots) ok = mbar_wait(&bars->v_empty[vs], ((vc / L::kVSlots) & 1) ^ 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars->v_full[vs], L::kTile);
                        tma_load_rows(smem + L::kOffV + vs * L::kTile, &tm_v, kvh, base + j * kKeys, 0,
                                      &bars->v_full[vs]);
                        ++vc;
                    }
                    mbar_arrive(&bars->soon);
                }
                __syncwarp();
            }
            if (lane == 0) {  // before the CTA may leave: every copy issued here has landed
                if (q0 && !mbar_wait(&bars->q_full[0], (q0 - 1) & 1)) ok = false;
                if (q1 && !mbar_wait(&bars->q_full[1], (q1 - 1) & 1)) ok = false;
                for (int j = max(0, kc - L::kKSlots); j < kc; ++j)
                    if (!mbar_wait(&bars->k_full[j % L::kKSlots], (j / L::kKSlots) & 1)) ok = false;
                for (int j = max(0, vc - L::kVSlots); j < vc; ++j)
                    if (!mbar_wait(&bars->v_full[j % L::kVSlots], (j / L::kVSlots) & 1)) ok = false;
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- MMA issue
            constexpr uint32_t idesc_s = tc_idesc_bf16(kRows, kKeys, false);
            constexpr uint32_t idesc_o = tc_idesc_bf16(kRows, D, true);
            const uint64_t qd0 = smem_desc_sw128(smem_u32(smem + L::kOffQ), 0, 1024);
            const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kOffK), 0, 1024);
            const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + L::kOffV), kHalf, 1024);
            int kc = 0, vc = 0;                    // stages so far
            int sc[2] = {0, 0}, ic[2] = {0, 0};    // the tiles' own stages and items so far
            uint32_t cleaned = 0;                  // parity of each slot's looks so far
            for (const Item* it; (it = items.next(ok)); items.done()) {
                const Tiles w(it, a.tpt);
                const int tok0 = __shfl_sync(0xffffffffu, it->tok0, 0);
                const bool split[2] = {a.split_all || tok0 + 1 <= kFewKeys,
                                       a.split_all || tok0 + a.tpt + 1 <= kFewKeys};
                auto issue_qk = [&](int t, int j) {  // stage j of the item, in K slot (kc + j) % slots
                    const uint64_t qd = qd0 + (uint64_t)((t * L::kTile) >> 4);
                    const uint64_t kd = kd0 + (uint64_t)((((kc + j) % L::kKSlots) * L::kTile) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                        tc_mma_ew(tmem + t * kKeys, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    tc_commit_ew(&bars->s_full[t]);
                    if (j + 1 == w.n[t]) tc_commit_ew(&bars->q_empty[t]);
                };
                auto issue_pv = [&](int t, int j) {
                    const uint64_t vd = vd0 + (uint64_t)((((vc + j) % L::kVSlots) * L::kTile) >> 4);
                    const uint32_t to = tmem + L::kColsO + t * D, tp = tmem + t * kKeys;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc_mma_ts_ew(to, tp + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o,
                                     (j > 0 || kk > 0) ? 1u : 0u);
                    if (split[t]) {  // the low parts of P, against the same V
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            tc_mma_ts_ew(to, tp + 64 + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, 1u);
                    }
                    if (j + 1 == w.n[t]) tc_commit_ew(&bars->o_full[t]);
                };
                ok = mbar_wait_warp(&bars->k_full[kc % L::kKSlots], (kc / L::kKSlots) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (w.n[t] == 0 || !ok) continue;
                    ok = mbar_wait_warp(&bars->q_full[t], ic[t] & 1);
                    if (!ok) continue;
                    tc_fence_after();
                    issue_qk(t, 0);
                }
                if (ok) tc_commit_ew(&bars->k_empty[kc % L::kKSlots]);
#pragma unroll 1
                for (int j = 0; j < w.nst && ok; ++j) {
                    // V(j) and K(j+1) are normally long in place, so they are waited for before P
                    const int vs = (vc + j) % L::kVSlots, ks = (kc + j + 1) % L::kKSlots;
                    if (j < w.first_masked) {
                        ok = mbar_wait_warp(&bars->v_full[vs], ((vc + j) / L::kVSlots) & 1);
                    } else {
                        ok = mbar_wait_warp(&bars->v_clean[vs], (cleaned >> vs) & 1);
                        cleaned ^= 1u << vs;
                    }
                    if (ok && j + 1 < w.nst) ok = mbar_wait_warp(&bars->k_full[ks], ((kc + j + 1) / L::kKSlots) & 1);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j >= w.n[t] || !ok) continue;
                        ok = mbar_wait_warp(&bars->p_full[t], (sc[t] + j) & 1);
                        // the outputs of the tile's item before have been read
                        if (ok && j == 0 && ic[t] > 0) ok = mbar_wait_warp(&bars->o_empty[t], (ic[t] - 1) & 1);
                        if (!ok) continue;
                        tc_fence_after();
                        issue_pv(t, j);
                        // S_t takes the place of P_t, after its product in issue order
                        if (j + 1 < w.n[t]) issue_qk(t, j + 1);
                    }
                    if (!ok) break;
                    tc_commit_ew(&bars->v_empty[vs]);
                    if (j + 1 < w.nst) tc_commit_ew(&bars->k_empty[ks]);
                }
                kc += w.nst;
                vc += w.nst;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    sc[t] += w.n[t];
                    ic[t] += w.n[t] > 0;
                }
            }
            // every MMA this warp issued has finished before the tensor memory is released
            tc_commit_ew(&bars->drain);
            if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
        } else if (warp == kCleanWarp) {
            // ---------------------------------------------------------------- V of the stages with masked keys
            int vc = 0;
            for (Item* it; (it = items.next(ok)); items.done()) {
                const Tiles w(it, a.tpt);
                // every stage is followed, so that a barrier's phases cannot pass this warp by
                for (int j = 0; j < w.nst && ok; ++j, ++vc) {
                    const int vs = vc % L::kVSlots;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[vs], (vc / L::kVSlots) & 1));
                    if (!ok) break;
                    if (j >= w.first_masked) {
                        uint8_t* tile = smem + L::kOffV + vs * L::kTile;
                        // a pass that only reads (its loads run ahead), and only where something was found the repair
                        uint32_t seen = 0;
#pragma unroll 8
                        for (int i = lane; i < L::kTile / 16; i += 32)
                            seen |= not_finite(*reinterpret_cast<const uint4*>(tile + 16 * i));
                        if (__any_sync(0xffffffffu, seen != 0)) {
                            if (!it->any_bad) {  // the notes of the item before have been read
                                if (items.n > 0)
                                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->item_empty[(items.n - 1) & 1],
                                                                           ((items.n - 1) >> 1) & 1));
                                if (!ok) break;
                                for (int i = lane; i < 3 * D; i += 32) bad[i] = INT_MAX;
                                __syncwarp();
                                if (lane == 0) it->any_bad = 1;
                                __syncwarp();
                            }
#pragma unroll 1
                            for (int i = lane; i < L::kTile / 16; i += 32) {
                                const int half = i / (kHalf / 16), row = i / 8 % kRows;
                                const int col = half * 64 + ((i & 7) ^ (row & 7)) * 8;
#pragma unroll 1
                                for (int e = 0; e < 8; ++e) {
                                    uint16_t* x = reinterpret_cast<uint16_t*>(tile + 16 * i) + e;
                                    if ((*x & 0x7f80u) != 0x7f80u) continue;
                                    const int what = (*x & 0x7fu) ? 0 : (*x & 0x8000u) ? 2 : 1;
                                    atomicMin(&bad[what * D + col + e], j * kKeys + row);
                                    *x = 0;
                                }
                            }
                            fence_proxy_async_smem();
                        }
                        mbar_arrive(&bars->v_clean[vs]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax and outputs, one row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int qi = r / a.th, hh = r - qi * a.th;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm_s = tmem + lanes + t * kKeys, tm_o = tmem + lanes + L::kColsO + t * D;
        const bool wide = (reinterpret_cast<uintptr_t>(a.p.out) & 31u) == 0;
        int sc = 0, ic = 0;  // the tile's stages and items so far
        for (const Item* it; (it = items.next(ok)); items.done()) {
            const int first = it->tok0 + t * a.tpt;  // the tile's first token
            const int ntok = max(0, min(a.tpt, it->len - first));
            if (ntok == 0) continue;
            const int n = (first + ntok + kKeys - 1) / kKeys;
            const bool valid = qi < ntok;
            const int pos = valid ? first + qi : kNoRow;
            float l = 0.f;
            if (a.split_all || first + 1 <= kFewKeys)
                ok = softmax_rows<D, true>(bars, t, sc, n, pos, a.scale_log2, tm_s, tm_o, l);
            else
                ok = softmax_rows<D, false>(bars, t, sc, n, pos, a.scale_log2, tm_s, tm_o, l);
            sc += n;
            if (ok) ok = !__any_sync(0xffffffffu, !mbar_wait(&bars->o_full[t], ic & 1));
            ++ic;
            if (!ok) continue;
            tc_fence_after();
            const float inv = 1.f / l;  // (l = 0 where every score is -inf: 0 / 0, a NaN as the definition has it)
            const bool any_bad = it->any_bad != 0;
            __nv_bfloat16* dst = a.p.out + ((size_t)(it->row + first + qi) * a.p.num_heads + it->head0 + hh) * D;
            // Two neighbouring lanes store 64 bytes of one row together, then of the other's: half the lines a
            // store touches.
            const bool odd = lane & 1;
            const unsigned long long at = valid ? reinterpret_cast<unsigned long long>(dst) : 0;
            auto row_of = [&](int from) {
                const unsigned long long row = __shfl_sync(0xffffffffu, at, from);
                return row ? reinterpret_cast<__nv_bfloat16*>(row) + (odd ? 16 : 0) : nullptr;
            };
            __nv_bfloat16* even_row = row_of(lane & ~1);
            __nv_bfloat16* odd_row = row_of(lane | 1);
            uint32_t o[32];
            tmem_ld32(tm_o, o);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                if (c + 32 < D) tmem_ld32_async(tm_o + c + 32, o);  // on their way while these are stored
                uint32_t first[8], second[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[8 + e], 1);
                    first[e] = odd ? got : v[e];
                    second[e] = odd ? v[8 + e] : got;
                }
                if (even_row) store_32(even_row + c, first, wide);
                if (odd_row) store_32(odd_row + c, second, wide);
                if (c + 32 < D) tmem_wait_ld(o);
                if (c + 64 == D) {
                    tc_fence_before();
                    mbar_arrive(&bars->o_empty[t]);
                }
            }
            __syncwarp();
            if (any_bad && valid) {
#pragma unroll 1
                for (int c = 0; c < D; ++c) {
                    float x = __bfloat162float(dst[c]);
                    if (pos >= bad[D + c]) x += INFINITY;
                    if (pos >= bad[2 * D + c]) x -= INFINITY;
                    if (pos >= bad[c]) x = NAN;
                    if (!isfinite(x)) dst[c] = __float2bfloat16_rn(x);
                }
            }
        }
        tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(a.p.status, kDevTimeout);
    __syncthreads();
    pdl_trigger();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// What the warp of the items finds for each of `pairs`: [row, length, first token], or -1s past the last pair.
__global__ void __launch_bounds__(32) pairs_kernel(const PackedArgs p, int tokens, const int32_t* pairs, int n, int32_t* out) {
    PairWalk walk(p, tokens);
    for (int i = 0; i < n; ++i) {
        const unsigned pair = (unsigned)pairs[i];
        if (!walk.find(pair)) {
            if (threadIdx.x < 3) out[3 * i + threadIdx.x] = -1;
        } else if (walk.owns(pair)) {
            out[3 * i] = walk.row;
            out[3 * i + 1] = walk.len;
            out[3 * i + 2] = walk.first_token(pair);
        }
    }
}

// Heads of a group that one tile holds: the largest divisor of the group up to 16, as few heads a tile make its token
// range long and leave more of it empty (group 4: 187 prompts of up to 128 tokens 90 us with 4 heads a tile, 97
// with 2, 173 with 1; 6 of up to 4000 483, 495, 511).  One that does not divide 128 leaves rows empty and
// has its token ranges begin anywhere, so the power of two goes before it where it is more than half as large
// (group 24, 8 against 12: 34 prompts of up to 700 tokens 63 us against 72, 256 of up to 48 45 against 43; but group
// 12, 4 against 12: 64 against 71, 53 against 40).
int tile_heads(int group) {
    int most = std::min(group, 16), two = 1;
    while (group % most != 0) --most;
    while (two < 16 && group % (2 * two) == 0) two *= 2;
    return 2 * two > most ? two : most;
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
    t.scale_log2 = a.scale * kLog2e;
    t.split_all = std::fabs(a.scale) * std::sqrt((float)D) > kSplitScale;
    CUtensorMap q, k, v;
    if (!strided_map(&q, a.q, a.num_tokens, a.num_heads, D, a.q_stride, t.th, t.tpt, 1) ||
        !strided_map(&k, a.k, a.num_tokens, a.num_kv_heads, D, a.k_stride, 1, kKeys, L::kHalves) ||
        !strided_map(&v, a.v, a.num_tokens, a.num_kv_heads, D, a.v_stride, 1, kKeys, L::kHalves))
        return cudaErrorInvalidValue;
    // an upper bound of the pairs that sequences of num_tokens rows in all, and of max_len each, can have
    const long long two = 2 * t.tpt;
    const long long pairs =
        std::min((a.num_tokens + a.batch * (two - 1)) / two, a.batch * ((a.max_len + two - 1) / two));
    const long long ctas = std::max(1LL, pairs) * t.subs;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, packed_kernel<D>, q, k, v, t);
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedArgs& a, cudaStream_t stream) {
    return a.head_dim == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

cudaError_t launch_selftest_pairs(const PackedArgs& a, int pair_tokens, const int32_t* pairs, int n, int32_t* out,
                                  cudaStream_t stream) {
    pairs_kernel<<<1, 32, 0, stream>>>(a, pair_tokens, pairs, n, out);
    return cudaGetLastError();
}

}  // namespace pa
