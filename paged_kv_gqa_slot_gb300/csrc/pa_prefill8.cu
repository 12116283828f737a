// pa_prefill8.cu -- chunked prefill over an 8-bit pool (pa_kv8.cuh) on the 5th-generation tensor
// cores.
//
// Query i of sequence s's chunk of C_s tokens sits at position L_s - C_s + i and attends causally
// to keys 0 .. that position.  The (query, head of the group) pairs of a (sequence, kv head)
// are the rows r = i g + h of its query tiles, 128 to a tile, whatever g is.  One CTA an SM
// holds two tiles (one where that leaves SMs empty), which share every K and V it widens, and
// the CTAs with the most keys launch first.
//
// Arithmetic: f16 operands and fp32 sums, as in pa_decode_lanes.cu.  A code is an f16 number, so K and V
// widen with one conversion per two codes and no multiplication; q is brought to a maximum in
// [2^14, 2^15) per row by a power of two.  The scales live in the softmax: with kK, kV the
// exponents of a key's block, s the raw product and f = log2(e) scale 2^(eq + kK),
//     u = 2^(s f + kV - base),   O += u codeV,   l += u 2^(-kV - 7) (or 2^(s f - base - 7): stage_terms),
// base some log2 units below the row's maximum of s f + kV.  u is rounded to f16: 11 bits down to 2^-14, fewer
// below, zero below 2^-25.  So the base lies kHeadroom units below a maximum that stands alone, kFlatHeadroom
// below one that has others beside it.
//
// Per stage of 64 keys (four pool blocks):
//   warps 10-15  three for K, three for V, take every third pair of blocks: codes come by a bulk copy a
//                block into the warp's own raw slots, kAhead pairs ahead, and are widened into the
//                128-byte swizzled layout of the MMA operands (rows past the sequence's end as zeros).
//                Pairs, because the waits, the fence and the hand-over cost as much as the widening:
//                block by block the warps needed 1500 cycles a block and bounded the kernel.
//   warps 8, 9   one per tile: S[128 x 64] = Q K^T into one of two 64-column buffers and
//                O[128 x D] += u V with u from tensor memory; per stage u V(j), then S(j + 2), which
//                reuses u(j)'s buffer.  Tile 1 starts half a stage behind.  The warp index comes from a
//                shuffle, so that descriptors and barrier addresses live in uniform registers: with
//                them in every thread's, an instruction took 80 cycles to issue, and a stage 1750.
//   warps 0-7    softmax, one row a thread: reads S, writes u over it.  The base is set by a row's
//                first visible stage and moves only when a stage's sum passes kSumLimit (f16 ends at
//                2^16), then by the maximum, if that is more than 2^9 above; O is rescaled in
//                tensor memory by all rows of a warp together.  (The maximum in every stage instead
//                cost 6 us of 52.)
// Before, they stage their rows of q by coalesced asynchronous copies and normalise them in place (rows
// loaded by the threads that own them took 4000 cycles more).  At the end all warps normalise O, stage
// the rows in the free Q buffer and store them coalesced.
//
// Measured on GB300 (32 q / 8 kv heads, d 128), the bf16 pool's kernel on the same dequantised values in
// brackets: 8 x 256 over 768 cached tokens 38.3 us (34.5), over 3840 110 (111), 1 x 256 over 768 16.4
// (14.9), 8 x 1024 over 1024 178 (167): 0.75 us a stage of two tiles, 1450 cycles, of which the matrix
// pipe needs 1280 (Q K^T reads Q and K from shared memory for 768, u V runs for 512), and about
// 8 us a CTA outside its stages: loads that wait for one another (lengths, table, codes) and q 4.5,
// output 2.5.  So a chunk over a short prefix is slower than from a bf16 pool, by up to an eighth, and one over a
// long prefix as fast.  At d 64 8 x 256 over 768 takes 30.4 us (125), over 3840 95.5 (513).
// Of these, keeping far scales exact cost 0.5 us of the 38.3, keeping later keys' NaNs apart 0.7.
// Tried and not kept: Q in tensor memory, which would bring the pipe to 1024 cycles but leaves room for
// one score buffer a tile, so that its softmax and its instructions take turns; stages of 128 keys with one
// buffer; two threads a row (these three and one tile a CTA were measured at 51 to 75 us, before uniform warp
// indices, paired conversion and coalesced loads of q); codes loaded into registers a pair ahead (115 us for
// 8 x 256 + 3840 became 118); one call site of the two softmax attempts (121 us against 108).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                 // MMA M: rows of a query tile
constexpr int kKeys = 64;                  // keys of a stage
constexpr int kParts = kKeys / kBlockSize;  // pool blocks of a stage
constexpr int kKStages = 3, kVStages = 3;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kMmaWarps = 2, kCvtWarp = 10, kCvtWarps = 6;
constexpr int kAhead = 2;                  // pairs of blocks a converter warp has in hand or in flight
constexpr int kThreads = 512;
constexpr int kTmemCols = 512;             // per tile: two 64-column score buffers, then O
constexpr uint32_t kTmemTile = 256;
constexpr uint32_t kTmemS = 0, kTmemO = 128;
constexpr float kSumLimit = 61440.f;      // a stage sum of u past this takes the maximum path
// Log2 units a maximum must exceed the base by to move it: 64 keys under it sum to less than 2^(6 + 9), so a row whose
// sum is past the limit moves.
constexpr float kRebase = 9.f;
static_assert(kKeys * 512 < kSumLimit, "a row past the limit moves its base");
// A maximum is alone if no other block of the stage comes within 2^-kAlone of it.  The units that the base
// lies below a maximum are lost above it, and where K's scales differ from block to block (by 2^0.7 in
// the standard deviation), 7 for every row took 5% of the stages to the maximum path, and 8 x 256 over
// 768 39.5 us; with 2 beside others it is 0.5%, as with none.
constexpr float kAlone = 6.f, kFlatHeadroom = 2.f;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct Pre8 {
    static constexpr int kHalves = D / 64;            // 64-column (128-byte) pieces of a row
    static constexpr int kQHalf = kRows * 128;
    static constexpr int kQTile = kHalves * kQHalf;
    static constexpr int kKVHalf = kKeys * 128;
    static constexpr int kStage = kHalves * kKVHalf;  // K or V of a stage
    static constexpr int kUnit = kBlockSize * D;      // codes of one block's K or V
    static constexpr int kOffK = 2 * kQTile;
    static constexpr int kOffV = kOffK + kKStages * kStage;
    static constexpr int kOffRaw = kOffV + kVStages * kStage;
    static constexpr int kOffBars = kOffRaw + kCvtWarps * kAhead * 2 * kUnit;
    static constexpr int kOffInv = kOffBars + 512;     // [2][128] 2^-7 / l, then whether every wait ended, and whether kOffNan names a key
    static constexpr int kOffNan = kOffInv + 2 * kRows * 4 + 16;  // [D] first key with a NaN in V's column d (see Converter)
    static constexpr int kSmem = kOffNan + D * 4;
    static constexpr int kLoads = kBlockSize * D / 512;  // 16-byte pieces of a block a lane takes
};
static_assert(Pre8<128>::kSmem <= 227 * 1024, "shared memory of a CTA");

struct Bars8 {
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t raw_full[kCvtWarps][kAhead];
    uint64_t q_full, s_full[2][2], p_full[2][2], o_done[2], o_final[2], drain;  // [tile][buffer]
    uint32_t tmem_base;
};
static_assert(sizeof(Bars8) <= 512, "barrier block");

// Division by a number that is known at launch, for any 32-bit x (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): a division proper is a chain of 30 instructions, and
// half a dozen stand before a CTA's first load.
struct Divisor {
    unsigned d, m, s1, s2;
    explicit Divisor(unsigned by = 1) : d(by) {
        unsigned l = 0;
        while ((1ull << l) < d) ++l;
        m = static_cast<unsigned>((((1ull << l) - d) << 32) / d + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ int div(int x) const {
        const unsigned u = static_cast<unsigned>(x), h = __umulhi(m, u);
        return static_cast<int>((h + ((u - h) >> s1)) >> s2);
    }
    __device__ __forceinline__ int mod(int x, int quotient) const { return x - quotient * static_cast<int>(d); }
};

struct Pre8Args {
    const __nv_bfloat16* q;
    const uint8_t *k, *v;
    const uint16_t* exps;  // K in the low byte
    const int32_t *block_tables, *seq_lens, *cu_q_lens;
    __nv_bfloat16* out;
    unsigned* status;
    Divisor by_group, by_batch, by_heads;
    int max_blocks, num_heads, num_kv_heads, num_blocks, group, batch;
    int ctas_per_pair;   // CTAs the grid holds per (sequence, kv head)
    int tiles_per_cta;   // 1 or 2
    float scale_log2;
};

constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    return tc_idesc_bf16(kRows, n, b_mn_major) & ~((1u << 7) | (1u << 10));  // f16 A and B
}

// 16 bytes into shared memory, zeros unless `in`.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// `bytes` contiguous bytes into shared memory, completing on `bar` (all multiples of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Converter warp w: of K (the first half of the warps) or V, every kSide-th pair of blocks, whose codes
// come into the warp's own raw slots by a bulk copy each, kAhead pairs ahead.
// A NaN of V in a key that only some rows see stays out of the product, where it would reach all of them (NaN
// times u = 0 is NaN): the key goes on record for its column, and the epilogue sets the column in the rows that see it.
template <int D>
struct Converter {
    using P = Pre8<D>;
    static constexpr int kSide = kCvtWarps / 2, kPairs = kParts / 2;
    uint8_t* smem;
    Bars8* bars;
    const Pre8Args& a;
    const int32_t* bt;
    const uint8_t* pool;  // of this warp's side, at its kv head
    int L, nst, nblk, w, lane, all_see, first;  // all_see: the last key that every row sees
    bool is_v;
    int next_id;  // lanes 0 and 1: of the pair to be fetched next

    __device__ __forceinline__ Converter(uint8_t* smem_, Bars8* bars_, const Pre8Args& a_, const int32_t* bt_, int kvh,
                                         int L_, int nst_, int nblk_, int w_, int lane_, int all_see_)
        : smem(smem_), bars(bars_), a(a_), bt(bt_), L(L_), nst(nst_), nblk(nblk_), w(w_), lane(lane_),
          all_see(all_see_) {
        is_v = w >= kSide;
        first = is_v ? w - kSide : w;
        pool = (is_v ? a.v : a.k) + (size_t)kvh * P::kUnit;
    }
    __device__ __forceinline__ uint32_t raw(int n) const {
        return smem_u32(smem + P::kOffRaw) + (w * kAhead + n % kAhead) * (2 * P::kUnit);
    }
    // the warp's n-th pair: start its copies, and load the next one's table entries
    __device__ __forceinline__ void issue(int n) {
        const int blk = 2 * (first + n * kSide) + lane, left = nblk - (blk - lane);
        if (left <= 0) return;
        uint64_t* bar = &bars->raw_full[w][n % kAhead];
        if (lane == 0) mbar_arrive_expect_tx(bar, left > 1 ? 2 * P::kUnit : P::kUnit);
        __syncwarp();
        if (lane < 2 && lane < left) {
            int id = next_id;
            if (id < 0 || id >= a.num_blocks) {
                atomicOr(a.status, kDevOutOfRange);
                id = 0;  // read inside the pool; the status word reports the bad id
            }
            bulk_load(raw(n) + lane * P::kUnit, pool + (size_t)id * a.num_kv_heads * P::kUnit, P::kUnit, bar);
            if (blk + 2 * kSide < nblk) next_id = __ldg(bt + blk + 2 * kSide);
        }
    }
    // The n-th pair's codes in its raw slot: NaNs of keys that only some rows see become zeros and go on record.
    // (Every lane reads and writes the pieces that it then widens.)
    __device__ __forceinline__ void scrub(int n, int pair) {
        const auto at = [&](int i) { return reinterpret_cast<uint32_t*>(smem + P::kOffRaw + (w * kAhead + n % kAhead) * (2 * P::kUnit) + lane * 16 + i * 512); };
        uint32_t some = 0u;
#pragma unroll
        for (int i = 0; i < 2 * P::kLoads; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(at(i));
            some |= nan_bits(v.x) | nan_bits(v.y) | nan_bits(v.z) | nan_bits(v.w);
        }
        if (!(some & 0x80808080u)) return;
        int* first_nan = reinterpret_cast<int*>(smem + P::kOffNan);
#pragma unroll 1
        for (int i = 0; i < 2 * P::kLoads * 4; ++i) {
            const int piece = (i >> 2) * 32 + lane, key = pair * 2 * kBlockSize + piece / (D / 16);
            const int d = piece % (D / 16) * 16 + (i & 3) * 4;
            uint32_t* word = at(i >> 2) + (i & 3);
            const uint32_t nan = nan_codes(*word);
            if (!nan || key <= all_see || key >= L) continue;
            *word &= ~nan;
            for (int j = 0; j < 4; ++j)
                if (nan >> (8 * j) & 1u) atomicMin(first_nan + d + j, key);
            *(reinterpret_cast<int*>(smem + P::kOffInv) + 2 * kRows + 1) = 1;
        }
    }
    __device__ __forceinline__ void start() {
        if (lane < kAhead) mbar_init(&bars->raw_full[w][lane], 1);
        fence_mbar_init();
        __syncwarp();
        next_id = lane < 2 && 2 * first + lane < nblk ? __ldg(bt + 2 * first + lane) : -1;
        for (int n = 0; n < kAhead; ++n) issue(n);
    }
    __device__ __forceinline__ void run() {
        static_assert(kKStages == kVStages, "one slot rule for both sides");
        bool ok = true;
        int n = 0;
        uint64_t *full = is_v ? bars->v_full : bars->k_full, *empty = is_v ? bars->v_empty : bars->k_empty;
        uint8_t* slots = smem + (is_v ? P::kOffV : P::kOffK);
        // rows from here on are zeros: past the blocks the CTA needs, and V past the sequence's end (u is 0
        // there, but 0 times NaN is NaN)
        const int end = is_v ? min(L, nblk * kBlockSize) : nblk * kBlockSize;
        const auto one = [&](int pair, auto masked) {
            const int stage = pair / kPairs, slot = stage % kKStages;
            uint4 codes[2 * P::kLoads];
            if (2 * pair < nblk) {
                ok = mbar_wait_warp(&bars->raw_full[w][n % kAhead], (n / kAhead) & 1);
                if (!ok) return;
                if constexpr (decltype(masked)::value) scrub(n, pair);
            }
#pragma unroll
            for (int i = 0; i < 2 * P::kLoads; ++i)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(codes[i].x), "=r"(codes[i].y), "=r"(codes[i].z), "=r"(codes[i].w)
                             : "r"(raw(n) + lane * 16 + i * 512)
                             : "memory");
            if ((pair + 1) * 2 * kBlockSize > end) {
#pragma unroll
                for (int i = 0; i < 2 * P::kLoads; ++i)
                    if (pair * 2 * kBlockSize + (i * 32 + lane) / (D / 16) >= end) codes[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (stage >= kKStages) ok = mbar_wait_warp(&empty[slot], ((stage / kKStages) & 1) ^ 1);
            if (!ok) return;
            uint8_t* dst = slots + slot * P::kStage + pair % kPairs * (2 * kBlockSize * 128);
#pragma unroll
            for (int i = 0; i < 2 * P::kLoads; ++i) {
                // 16 codes: the 16-byte chunks ch, ch + 1 of column half h; lanes of the second half
                // store them in the other order, so that the lanes of one row hit different banks
                const int piece = i * 32 + lane, row = piece / (D / 16), c = piece % (D / 16);
                const int h = c >> 2, ch = (c & 3) * 2;
                uint4 lo, hi;
                e4m3x4_to_f16x4(codes[i].x, lo.x, lo.y);
                e4m3x4_to_f16x4(codes[i].y, lo.z, lo.w);
                e4m3x4_to_f16x4(codes[i].z, hi.x, hi.y);
                e4m3x4_to_f16x4(codes[i].w, hi.z, hi.w);
                uint8_t* at = dst + h * P::kKVHalf;
                *reinterpret_cast<uint4*>(at + swz128(row, ch + h)) = h ? hi : lo;
                *reinterpret_cast<uint4*>(at + swz128(row, ch + 1 - h)) = h ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[slot]);
            issue(n + kAhead);  // over the codes, which every lane has read
            ++n;
        };
        // pairs of keys that every row sees, then the others (in one loop with a branch the scrubbing made every
        // pair slower: 8 x 256 over 768 38.7 us against 38.4)
        const int clear = is_v ? min((all_see + 1) / (2 * kBlockSize), nst * kPairs) : nst * kPairs;
        int pair = first;
        for (; pair < clear && ok; pair += kSide) one(pair, std::false_type{});
        for (; pair < nst * kPairs && ok; pair += kSide) one(pair, std::true_type{});
        if (!ok) {
            // a wait ran out: the copies in flight must still land before their memory is used again
            for (int i = n; i < n + kAhead; ++i)
                if (2 * (first + i * kSide) < nblk) mbar_wait_warp(&bars->raw_full[w][i % kAhead], (i / kAhead) & 1);
            if (lane == 0) atomicOr(a.status, kDevTimeout);
        }
    }
};

// The scales of a block as the softmax takes them, from its word of exponents (K in the low byte):
// the factor qf 2^kK on s, kV, and 2^(-kV - 7).
__device__ __forceinline__ float k_factor(int e, float qf) { return qf * __int_as_float((e & 255) << 23); }
__device__ __forceinline__ float v_exponent(int e) { return static_cast<float>((e >> 8) - kExpBias); }
__device__ __forceinline__ float v_unscale(int e) {
    return __int_as_float((2 * kExpBias - kHeadroom - (e >> 8)) << 23);
}

// Largest s f + kV of the stage's visible keys c <= lim (all of them with kAll); second: that of the other blocks.
template <bool kAll>
__device__ __forceinline__ float stage_max(const uint32_t (&s)[2][32], int lim, const int (&ew)[kParts], float qf,
                                           float& second) {
    float best = -INFINITY;
    second = -INFINITY;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int c = i * 16; c < i * 16 + 16; c += 4) {
            float x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[t] = __uint_as_float(s[(c + t) >> 5][(c + t) & 31]);
                if (!kAll) x[t] = c + t > lim ? -INFINITY : x[t];
            }
            m0 = fmax3(m0, x[0], x[1]);
            m1 = fmax3(m1, x[2], x[3]);
        }
        float m = fmaxf(m0, m1);
        m = m == -INFINITY ? m : fmaf(m, k_factor(ew[i], qf), v_exponent(ew[i]));
        second = fmaxf(second, fminf(best, m));
        best = fmaxf(best, m);
    }
    return best;
}

// u of the stage, 2^(s f + kV + nbase), as f16 pairs into the 32 columns at `dst`; returns their plain
// sum, and lsum gets the sum of u 2^(-kV - 7).
template <bool kAll>
__device__ __forceinline__ float stage_u(const uint32_t (&s)[2][32], int lim, const int (&ew)[kParts], float qf,
                                         float nbase, uint32_t dst, float& lsum) {
    float all = 0.f;
    lsum = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const float f = k_factor(ew[i], qf), off = v_exponent(ew[i]) + nbase;
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        uint32_t pw[8];
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
            const int c = i * 16 + t;
            float x0, x1;
            fma_x2(x0, x1, __uint_as_float(s[c >> 5][c & 31]), __uint_as_float(s[c >> 5][(c & 31) + 1]), f, f, off, off);
            if (!kAll) {
                x0 = c > lim ? -INFINITY : x0;  // 2^-inf = 0
                x1 = c + 1 > lim ? -INFINITY : x1;
            }
            const float u0 = fast_exp2(x0), u1 = fast_exp2(x1);
            if (t & 2)
                add_x2(a2, a3, u0, u1);
            else
                add_x2(a0, a1, u0, u1);
            pw[t / 2] = pack_f16x2(u0, u1);
        }
        const float sum = (a0 + a1) + (a2 + a3);
        all += sum;
        lsum = fmaf(sum, v_unscale(ew[i]), lsum);
        tmem_st8_nowait(dst + 8 * i, pw[0], pw[1], pw[2], pw[3], pw[4], pw[5], pw[6], pw[7]);
    }
    return all;
}

// The stage's sum of 2^(s f + nbase), the normaliser's terms, each by an exponential of its own (far_scale),
// in two steps, so that it ends with fp32's subnormals.
__device__ __forceinline__ float stage_terms(const uint32_t (&s)[2][32], int lim, const int (&ew)[kParts], float qf,
                                             float nbase) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kKeys; ++c) {
        const float x = fmaf(__uint_as_float(s[c >> 5][c & 31]), k_factor(ew[c >> 4], qf), nbase);
        const float h = fast_exp2(c > lim ? -INFINITY : 0.5f * x);
        sum = fmaf(h, h, sum);
    }
    return sum;
}

// The row's D fp32 columns of O at `taddr` times f, eight at a time.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 8) {
        uint32_t o[8];
        tmem_ld8(taddr + c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st8_nowait(taddr + c, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    }
    tmem_wait_st();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill8_kernel(const __grid_constant__ Pre8Args a) {
    using P = Pre8<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars8* bars = reinterpret_cast<Bars8*>(smem + P::kOffBars);
    float* row_inv = reinterpret_cast<float*>(smem + P::kOffInv);
    int* all_ok = reinterpret_cast<int*>(row_inv + 2 * kRows);
    int* some_nan = all_ok + 1;
    int* first_nan = reinterpret_cast<int*>(smem + P::kOffNan);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    // blockIdx.x = (rank * batch + b) * num_kv_heads + kvh: rank 0 is every chunk's last CTA
    const int rb = a.by_heads.div((int)blockIdx.x), kvh = a.by_heads.mod((int)blockIdx.x, rb);
    const int rank = a.by_batch.div(rb), b = a.by_batch.mod(rb, rank);
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(a.status, kDevOutOfRange);
        return;
    }
    // The set-up waits for nothing of another kernel's.
    if (warp == kMmaWarp + 1 && lane == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bars->k_full[s], kParts / 2);
            mbar_init(&bars->k_empty[s], kMmaWarps);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&bars->v_full[s], kParts / 2);
            mbar_init(&bars->v_empty[s], kMmaWarps);
        }
        mbar_init(&bars->q_full, kSoftmaxWarps);
        for (int t = 0; t < 2; ++t) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars->s_full[t][i], 1);
                mbar_init(&bars->p_full[t][i], kRows / 32);
            }
            mbar_init(&bars->o_done[t], 1);
            mbar_init(&bars->o_final[t], 1);
        }
        mbar_init(&bars->drain, kMmaWarps);
        *all_ok = 1;
        *some_nan = 0;
        fence_mbar_init();
    }
    if (warp >= kCvtWarp && threadIdx.x - kCvtWarp * 32 < D) first_nan[threadIdx.x - kCvtWarp * 32] = 0x7fffffff;
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    pdl_wait();
    const int g = a.group;
    const int q0 = a.cu_q_lens[b];
    const int C = a.cu_q_lens[b + 1] - q0;
    const int L = a.seq_lens[b];
    const auto leave = [&] {
        if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    };
    if (C < 0 || L < C || L > a.max_blocks * kBlockSize) {
        if (threadIdx.x == 0 && rank == 0 && kvh == 0) atomicOr(a.status, kDevOutOfRange);
        return leave();
    }
    const long long rows = (long long)C * g;
    const int cta_rows = a.tiles_per_cta * kRows;
    const long long need = (rows + cta_rows - 1) >> (a.tiles_per_cta == 2 ? 8 : 7);
    // a chunk longer than max_chunk: the grid covers its first rows, the rest is reported
    if (rank == 0 && kvh == 0 && threadIdx.x == 0 && need > a.ctas_per_pair) atomicOr(a.status, kDevOutOfRange);
    const int covered = (int)min(need, (long long)a.ctas_per_pair);
    if (rank >= covered) return leave();
    const int row0 = (covered - 1 - rank) * cta_rows;
    // rows of either tile, and its stages: up to the key its last query sees
    const int live = (int)min((long long)cta_rows, rows - row0);
    const auto live_of = [&](int t) { return max(0, min(kRows, live - t * kRows)); };
    const auto keys_of = [&](int t) {
        const int n = live_of(t);
        return n ? L - C + a.by_group.div(row0 + t * kRows + n - 1) + 1 : 0;
    };
    const int keys0 = keys_of(0), keys1 = keys_of(1), nkeys = max(keys0, keys1);
    const int nst0 = (keys0 + kKeys - 1) / kKeys, nst1 = (keys1 + kKeys - 1) / kKeys;
    const int nst = max(nst0, nst1);
    const int nblk = (nkeys + kBlockSize - 1) / kBlockSize;
    const int32_t* bt = a.block_tables + (size_t)b * a.max_blocks;

    // The first loads: a softmax warp's 32 rows of q, kLanes lanes a row, into the swizzled layout (zeros
    // past the chunk), and its first table entries; a converter's first pairs.
    constexpr int kLanes = D / 8, kPerLoad = 32 / kLanes;  // lanes of a row of q, rows of one load
    const int t_tile = (warp >> 2) & 1, w_row = (warp & 3) * 32;
    int first_id = -1;
    Converter<D> cvt{smem, bars, a, bt, kvh, L, nst, nblk, warp - kCvtWarp, lane,
                     L - C + a.by_group.div(row0)};
    if (warp < kSoftmaxWarps) {
        if (lane < nblk) first_id = __ldg(bt + lane);
        const int c = lane % kLanes, r0 = w_row + lane / kLanes, n = live_of(t_tile);
        const int cr = row0 + t_tile * kRows + r0;
        const int step_q = a.by_group.div(kPerLoad), step_h = kPerLoad - step_q * g;
        int qi = a.by_group.div(cr), qh = cr - qi * g;
        const uint32_t dst = smem_u32(smem + t_tile * P::kQTile + (c >> 3) * P::kQHalf);
        const __nv_bfloat16* src = a.q + (size_t)kvh * g * D + c * 8;
#pragma unroll 4
        for (int i = 0; i < kLanes; ++i) {
            const int r = r0 + i * kPerLoad;
            const bool in = r < n;
            cp_async16(dst + swz128(r, c & 7), in ? src + ((size_t)(q0 + qi) * a.num_heads + qh) * D : src, in);
            qi += step_q;
            qh += step_h;
            if (qh >= g) qh -= g, ++qi;
        }
        cp_async_commit();
    } else if (warp >= kCvtWarp) {
        cvt.start();
    }

    if (warp >= kCvtWarp) {
        cvt.run();
    } else if (warp >= kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idesc_s = idesc_f16(kKeys, false), idesc_o = idesc_f16(D, true);
        const int t = warp - kMmaWarp, myst = t ? nst1 : nst0;  // tile, and its stages
        const uint64_t qd = smem_desc_sw128(smem_u32(smem + t * P::kQTile), 0, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + P::kOffK), 0, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + P::kOffV), P::kKVHalf, 1024);
        const uint32_t tt = tmem + t * kTmemTile;
        const auto issue_s = [&](int j) {  // S(j) into its buffer j % 2
            const uint64_t kd = kd0 + (uint64_t)(((j % kKStages) * P::kStage) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_ew(tt + kTmemS + 64 * (j & 1), qd + (uint64_t)(((kk >> 2) * P::kQHalf + (kk & 3) * 32) >> 4),
                          kd + (uint64_t)(((kk >> 2) * P::kKVHalf + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
            tc_commit_ew(&bars->s_full[t][j & 1]);
        };
        const auto issue_o = [&](int j) {  // O += u(j) V(j)
            const uint64_t vd = vd0 + (uint64_t)(((j % kVStages) * P::kStage) >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                tc_mma_ts_ew(tt + kTmemO, tt + kTmemS + 64 * (j & 1) + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4),
                             idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
            tc_commit_ew(&bars->o_done[t]);
            if (j + 1 == myst) tc_commit_ew(&bars->o_final[t]);
        };
        // a tile without this stage only passes the slots on
        bool ok = mbar_wait_warp(&bars->q_full, 0);
        // tile 1 starts half a stage behind, and stays there: one tile's instructions run while the
        // other's warp waits and hands over
        // (tile 0 cannot get to S(3), the barrier's next phase: K(3) takes the slot of a K(0) not yet released)
        static_assert(kKStages == 3, "the phase waited for");
        if (t == 1 && nst0 > 1) ok = ok && mbar_wait_warp(&bars->s_full[0][1], 0);
        for (int j = 0; j < 2 && j < nst && ok; ++j) {
            ok = mbar_wait_warp(&bars->k_full[j], 0);
            if (!ok) break;
            tc_fence_after();
            if (j < myst) issue_s(j);
            tc_commit_ew(&bars->k_empty[j]);
        }
        for (int j = 0; j < nst && ok; ++j) {
            // u V(j), then S(j + 2) into the buffer that u(j) sits in
            ok = mbar_wait_warp(&bars->v_full[j % kVStages], (j / kVStages) & 1);
            if (ok && j < myst) ok = mbar_wait_warp(&bars->p_full[t][j & 1], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (j < myst) issue_o(j);
            tc_commit_ew(&bars->v_empty[j % kVStages]);
            if (j + 2 < nst) {
                ok = mbar_wait_warp(&bars->k_full[(j + 2) % kKStages], ((j + 2) / kKStages) & 1);
                if (!ok) break;
                tc_fence_after();
                if (j + 2 < myst) issue_s(j + 2);
                tc_commit_ew(&bars->k_empty[(j + 2) % kKStages]);
            }
        }
        // every MMA issued here has finished before the tensor memory is released
        tc_commit_ew(&bars->drain);
        if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
        if (!ok && lane == 0) atomicOr(a.status, kDevTimeout);
    } else {
        // ---------------------------------------------------------------- softmax: one row a thread
        const int t = t_tile, r = w_row + lane;  // tile, and its row: tensor memory lane
        const int myst = t ? nst1 : nst0;
        const int pos =  // last key the row sees
            r < live_of(t) ? L - C + a.by_group.div(row0 + t * kRows + r) : -1;
        const uint32_t tm = tmem + t * kTmemTile + ((uint32_t)((warp & 3) * 32) << 16);
        // exponents of blocks c0 + lane: a word a lane, the next 32 read ahead
        const auto entry = [&](int blk) { return blk < nblk ? __ldg(bt + blk) : -1; };
        const auto exps_of = [&](int blk, int id) -> int {
            if (blk >= nblk) return kExpBias * 257;
            return valid_exps(__ldg(a.exps + (size_t)(id < 0 || id >= a.num_blocks ? 0 : id) * a.num_kv_heads + kvh));
        };
        int ex = exps_of(lane, first_id), next_id = entry(32 + lane), next_ex = 0;
        // the row of q, normalised by a power of two, in place; a negative scale enters as -q, so that
        // maxima are of the scores as they are
        cp_async_wait<0>();
        __syncwarp();
        const auto piece = [&](int c) {
            return reinterpret_cast<uint4*>(smem + t * P::kQTile + (c >> 3) * P::kQHalf + swz128(r, c & 7));
        };
        uint32_t mag = 0u;  // the row's largest magnitude, as bf16
#pragma unroll
        for (int c = 0; c < kLanes; ++c) {
            const uint4 v = *piece(c);
            mag = max_mag2(max_mag2(max_mag2(max_mag2(mag, v.x), v.y), v.z), v.w);
        }
        if (max(mag & 0xffffu, mag >> 16) >= 0x7f80u) {  // infinities and NaN do not count
            mag = 0u;
#pragma unroll 1
            for (int c = 0; c < kLanes; ++c) {
                const uint4 v = *piece(c);
                mag = max_mag2(max_mag2(max_mag2(max_mag2(mag, finite2(v.x)), finite2(v.y)), finite2(v.z)),
                               finite2(v.w));
            }
        }
        const int eq = max(static_cast<int>(max(mag & 0xffffu, mag >> 16) >> 7) - 127 - 14, -110);
        const float qf = fabsf(a.scale_log2) * exp2_int(eq);
        const __nv_bfloat162 s2 = __float2bfloat162_rn(a.scale_log2 < 0.f ? -exp2_int(-eq) : exp2_int(-eq));
#pragma unroll
        for (int c = 0; c < kLanes; ++c) {
            const auto w = [&](uint32_t x) {  // exact but for f16's own end
                const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), s2);
                const uint32_t y = *reinterpret_cast<const uint32_t*>(&p);
                return pack_f16x2(bf16_lo(y), bf16_hi(y));
            };
            const uint4 v = *piece(c);
            *piece(c) = make_uint4(w(v.x), w(v.y), w(v.z), w(v.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
        float base = -INFINITY, l = 0.f;
        // of a stage's sum, past which it takes the maximum path; negative (every stage takes it) from a block with
        // a far_scale on
        float limit = kSumLimit;
        bool ok = true;
        // tcgen05.ld / st are warp-collective: what leads to one is decided by the whole warp
        for (int j = 0; j < myst; ++j) {
            const int at = (j * kParts) & 31;
            if (at == 0 && j > 0) {
                ex = next_ex;
                next_id = entry(j * kParts + 32 + lane);
            }
            if (at == 0) limit = __any_sync(0xffffffffu, far_scale(ex >> 8)) ? -1.f : limit;
            int ew[kParts];
#pragma unroll
            for (int i = 0; i < kParts; ++i) ew[i] = __shfl_sync(0xffffffffu, ex, at + i);
            if (at == 16) next_ex = exps_of(j * kParts + 16 + lane, next_id);
            const uint32_t buf = tm + kTmemS + 64 * (j & 1);
            ok = mbar_wait_warp(&bars->s_full[t][j & 1], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const int lim = pos - j * kKeys;
            const bool unmasked = __all_sync(0xffffffffu, lim >= kKeys - 1);
            uint32_t s[2][32];
            tmem_ld32_async(buf, s[0]);
            tmem_ld32_async(buf + 32, s[1]);
            tmem_wait_ld(s[0]);
            tmem_wait_ld(s[1]);
            // First against the row's base as it is.  The maximum, and with it a possible move of the
            // base, is taken only for a row's first visible stage, or when the sum of u passes
            // the limit; either is the warp's decision.
            float lsum = 0.f;
            const auto weigh = [&] {
                const float nbase = base == -INFINITY ? 0.f : -base;
                return unmasked ? stage_u<true>(s, lim, ew, qf, nbase, buf, lsum)
                                : stage_u<false>(s, lim, ew, qf, nbase, buf, lsum);
            };
            bool full = __any_sync(0xffffffffu, base == -INFINITY && lim >= 0);
            if (!full) full = __any_sync(0xffffffffu, !(weigh() <= limit));
            if (full) {
                tmem_wait_st();  // a first attempt's u: the second goes over it
                float second;
                const float top = unmasked ? stage_max<true>(s, lim, ew, qf, second)
                                           : stage_max<false>(s, lim, ew, qf, second);
                const float target = top - (top - second > kAlone ? (float)kHeadroom : kFlatHeadroom);
                const bool move = top > base + kRebase;  // always at a row's first visible key
                const bool rescale = move && base != -INFINITY;
                if (__any_sync(0xffffffffu, rescale)) {
                    // O changes once u V(j - 1) has finished: phase j - 1 of o_done (phases up to
                    // j - 2 are over, as S(j) followed u V(j - 2), and u V(j) waits for this u)
                    if (j > 0) ok = mbar_wait_warp(&bars->o_done[t], (j - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    scale_o<D>(tm + kTmemO, rescale ? fast_exp2(base - target) : 1.f);
                    // in two steps: l, whose terms carry 2^-kV, may count where the factor is zero
                    const float half = rescale ? fast_exp2(0.5f * (base - target)) : 1.f;
                    l = l * half * half;
                }
                if (move) base = target;
                weigh();
                if (limit < 0.f) lsum = stage_terms(s, lim, ew, qf, base == -INFINITY ? 0.f : -base - kHeadroom);
            }
            l += lsum;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[t][j & 1]);
        }
        if (ok && myst > 0) ok = mbar_wait_warp(&bars->o_final[t], 0);
        row_inv[t * kRows + r] = l > 0.f ? 1.f / (1 << kHeadroom) / l : 0.f;
        if (!ok && lane == 0) {
            *all_ok = 0;
            atomicOr(a.status, kDevTimeout);
        }
    }
    __syncthreads();
    tc_fence_after();
    // ---------------------------------------------------------------- epilogue
    // Warp: a quarter of a tile's rows and half of the columns, normalised, as 16-byte chunks into
    // the Q buffer ([row][chunk ^ row % 8]: no bank conflicts either way), then coalesced.
    constexpr int kChunks = D / 8;
    if (*all_ok) {
        const int t = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, c0 = (warp >> 3) * (D / 2);
        if (live_of(t)) {
            const float inv = row_inv[t * kRows + r];
            const uint32_t tm = tmem + t * kTmemTile + ((uint32_t)((warp & 3) * 32) << 16) + kTmemO;
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) {
                uint32_t o[32];
                tmem_ld32(tm + c0 + c, o);
                if (*some_nan) {
                    const int pos = L - C + a.by_group.div(row0 + t * kRows + r);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (first_nan[c0 + c + e] <= pos) o[e] = 0x7fffffffu;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const auto w = [&](int i) {
                        return pack_bf16x2(__uint_as_float(o[e + i]) * inv, __uint_as_float(o[e + i + 1]) * inv);
                    };
                    const int ch = (c0 + c + e) >> 3;
                    *reinterpret_cast<uint4*>(smem + t * P::kQTile + (r * kChunks + (ch ^ (r & 7))) * 16) =
                        make_uint4(w(0), w(2), w(4), w(6));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (*all_ok) {
        constexpr int kStep = kThreads / kChunks;  // rows between a thread's pieces
        const int ch = threadIdx.x % kChunks;
        int cr = threadIdx.x / kChunks;
        const int step_q = a.by_group.div(kStep), step_h = kStep - step_q * g;
        int qi = a.by_group.div(row0 + cr), h = row0 + cr - qi * g;
#pragma unroll 4
        for (int i = 0; i < 2 * kRows / kStep; ++i, cr += kStep) {
            const int r = cr & (kRows - 1);
            const uint4 v = *reinterpret_cast<const uint4*>(smem + (cr / kRows) * P::kQTile +
                                                            (r * kChunks + (ch ^ (r & 7))) * 16);
            if (cr < live)
                *reinterpret_cast<uint4*>(a.out + ((size_t)(q0 + qi) * a.num_heads + (size_t)kvh * g + h) * D + ch * 8) = v;
            qi += step_q;
            h += step_h;
            if (h >= g) h -= g, ++qi;
        }
    }
}

template <int D>
cudaError_t launch(const Pre8Args& p, unsigned ctas, cudaStream_t stream) {
    auto kern = prefill8_kernel<D>;
    static OncePerDevice configured;
    const cudaError_t e = configured.run([&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pre8<D>::kSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
        return r;
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Pre8<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_prefill8(const Pool8View& pool, const AttnArgs& a, cudaStream_t stream) {
    const int g = a.num_heads / pool.num_kv_heads;
    // a chunk of a few queries is a decode with a causal mask
    if (decode_mq_supported(g, a.max_chunk)) return launch_decode8_mq(pool, a, stream);
    Pre8Args p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = pool.k;
    p.v = pool.v;
    p.exps = reinterpret_cast<const uint16_t*>(pool.exps);
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.cu_q_lens = a.cu_q_lens;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.status = a.status;
    p.max_blocks = a.max_blocks;
    p.num_heads = a.num_heads;
    p.num_kv_heads = pool.num_kv_heads;
    p.num_blocks = pool.num_blocks;
    p.group = g;
    p.batch = a.batch;
    p.by_group = Divisor(g);
    p.by_batch = Divisor(a.batch);
    p.by_heads = Divisor(pool.num_kv_heads);
    p.scale_log2 = a.scale * kLog2e;
    // two tiles to a CTA, unless the tiles, one to an SM, all run at once
    const long long pairs = (long long)a.batch * pool.num_kv_heads;
    const long long tiles = ((long long)a.max_chunk * g + kRows - 1) / kRows;
    p.tiles_per_cta = tiles * pairs <= device_info().num_sms ? 1 : 2;
    p.ctas_per_pair = (int)((tiles + p.tiles_per_cta - 1) / p.tiles_per_cta);
    const long long ctas = p.ctas_per_pair * pairs;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;  // more CTAs than a grid holds
    return pool.head_dim == 128 ? launch<128>(p, (unsigned)ctas, stream) : launch<64>(p, (unsigned)ctas, stream);
}

}  // namespace pa
