// pa_prefill8.cu -- chunked prefill over an 8-bit pool (pa_kv8.cuh) on the 5th-generation tensor
// cores.
//
// Query i of sequence s's chunk of C_s tokens sits at position L_s - C_s + i and attends causally
// to keys 0 .. that position.  The (query, head of the group) pairs of a (sequence, kv head)
// are the rows r = i g + h of its query tiles, 128 to a tile, whatever g is.  One CTA holds
// one tile, two CTAs share an SM (256 columns of tensor memory each), and the longest
// tiles launch first.
//
// Arithmetic: f16 operands and fp32 sums, as in pa_decode_lanes.cu.  A code is an f16 number, so K and V
// widen with one conversion per two codes and no multiplication; q is brought to a maximum in
// [2^14, 2^15) per row by a power of two.  The scales live in the softmax: with kK, kV the
// exponents of a key's block, s the raw product and f = log2(e) scale 2^(eq + kK),
//     u = 2^(s f + kV - base),   O += u codeV,   l += u 2^-kV,
// base following the row's maximum of s f + kV.  u is rounded to f16 (11 bits), which needs no
// second part even where a few weights dominate a row.
//
// Per stage of 64 keys (four pool blocks):
//   warps 5-7  read codes, 16 bytes a lane, widen them and store them in the 128-byte swizzled
//              layout of the MMA operands (rows past the sequence's end as zeros); a unit is one
//              block's K or V, units go to the three warps in turn, K one stage ahead of V, and a
//              warp's next unit is loaded before it waits for the slot of the one in hand
//   warp 4     S[128 x 64] = Q K^T into one of two 64-column buffers, O[128 x D] += u V with u
//              from tensor memory; per stage u V(j), then S(j + 2), which reuses u(j)'s buffer
//   warps 0-3  softmax, one row a thread: reads S, writes u over it.  The base is set by a row's
//              first visible stage and moves only when a stage's sum passes 2^15 (f16 ends at
//              2^16), then to the maximum, if that is more than 2^8 above; O is rescaled in
//              tensor memory by all rows of a warp together.
// At the end all eight warps normalise and store, a quarter of the rows and half the columns each.
#include <algorithm>
#include <cmath>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                 // MMA M: rows of a query tile
constexpr int kKeys = 64;                  // keys of a stage
constexpr int kParts = kKeys / kBlockSize;  // pool blocks of a stage
constexpr int kKStages = 3, kVStages = 2;
constexpr int kMmaWarp = 4, kCvtWarp = 5, kCvtWarps = 3;
constexpr int kThreads = 256;
constexpr int kCtasPerSm = 2;
constexpr int kTmemCols = 256;
constexpr uint32_t kTmemS = 0, kTmemO = 128;
constexpr float kSumLimit = 32768.f;      // a stage sum of u past this takes the maximum path
constexpr float kRebase = 8.f;            // log2 units a maximum must exceed the base by to move it
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct Pre8 {
    static constexpr int kHalves = D / 64;            // 64-column (128-byte) pieces of a row
    static constexpr int kQHalf = kRows * 128;
    static constexpr int kKVHalf = kKeys * 128;
    static constexpr int kStage = kHalves * kKVHalf;  // K or V of a stage
    static constexpr int kOffK = kHalves * kQHalf;
    static constexpr int kOffV = kOffK + kKStages * kStage;
    static constexpr int kOffBars = kOffV + kVStages * kStage;
    static constexpr int kOffInv = kOffBars + 256;     // [128] 1 / l, then whether every wait ended
    static constexpr int kSmem = kOffInv + kRows * 4 + 16;
    static constexpr int kLoads = kBlockSize * D / 512;  // 16-byte pieces of a block a lane takes
};
static_assert(kCtasPerSm * (Pre8<128>::kSmem + 1024) <= 228 * 1024, "shared memory of two resident CTAs");
static_assert(kCtasPerSm * kTmemCols <= 512, "tensor memory of two resident CTAs");

struct Bars8 {
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t q_full, s_full[2], p_full[2], o_done, o_final, drain;
    uint32_t tmem_base;
};
static_assert(sizeof(Bars8) <= 256, "barrier block");

struct Pre8Args {
    const __nv_bfloat16* q;
    const uint8_t *k, *v;
    const uint16_t* exps;  // K in the low byte
    const int32_t *block_tables, *seq_lens, *cu_q_lens;
    __nv_bfloat16* out;
    unsigned* status;
    int max_blocks, num_heads, num_kv_heads, num_blocks, group, batch, tiles;
    float scale_log2;
};

constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    return tc_idesc_bf16(kRows, n, b_mn_major) & ~((1u << 7) | (1u << 10));  // f16 A and B
}

// Unit u of the stream K(0), then K(j + 1), V(j) for j = 0, 1, ..., each kParts units (the last
// stage has no K(j + 1)).
struct Unit {
    int stage, part;
    bool is_v;
};
__device__ __forceinline__ Unit unit_of(int u, int nst) {
    const int grp = u / kParts;
    Unit r;
    r.part = u % kParts;
    const bool last = grp == 2 * nst - 1;
    r.is_v = last || (grp > 0 && grp % 2 == 0);
    r.stage = last ? nst - 1 : r.is_v ? grp / 2 - 1 : (grp + 1) / 2;
    return r;
}

template <int D>
__device__ __forceinline__ void widen_units(uint8_t* smem, Bars8* bars, const Pre8Args& a, const int32_t* bt, int kvh,
                                            int L, int nst, int nblk, int w) {
    using P = Pre8<D>;
    const int lane = threadIdx.x & 31;
    const int total = 2 * nst * kParts;
    // entries of blocks c0 + lane and the 32 after them; units walk the blocks of K one stage ahead
    // of V's, and the loads run up to kAhead units ahead of that
    constexpr int kAhead = 3;
    uint4 codes[kAhead][P::kLoads];
    int c0 = 0;
    const auto entry = [&](int blk) -> int {
        if (blk >= nblk) return -1;
        const int id = __ldg(bt + blk);
        if (id >= 0 && id < a.num_blocks) return id;
        atomicOr(a.status, kDevOutOfRange);
        return 0;  // read inside the pool; the status word reports the bad id
    };
    int cur = entry(lane), nxt = entry(32 + lane);
    const auto load = [&](uint4 (&to)[P::kLoads], int u) {
        const Unit n = unit_of(u, nst);
        const int lb = n.stage * kParts + n.part;
#pragma unroll
        for (int i = 0; i < P::kLoads; ++i) to[i] = make_uint4(0u, 0u, 0u, 0u);
        // V units trail, so the window moves on once V has left it
        if (n.is_v && lb >= c0 + 32) {
            c0 += 32;
            cur = nxt;
            nxt = entry(c0 + 32 + lane);
        }
        const int id = __shfl_sync(0xffffffffu, lb < c0 + 32 ? cur : nxt, lb & 31);
        if (id < 0) return;  // past the keys the tile needs: zeros
        const size_t tile = ((size_t)id * a.num_kv_heads + kvh) * (kBlockSize * D);
        const uint4* src = reinterpret_cast<const uint4*>((n.is_v ? a.v : a.k) + tile) + lane;
#pragma unroll
        for (int i = 0; i < P::kLoads; ++i) {
            // V rows past the sequence's end count as zeros (u is 0 there, but 0 times NaN is NaN)
            const int row = (i * 32 + lane) / (D / 16);
            if (!n.is_v || lb * kBlockSize + row < L) to[i] = __ldg(src + i * 32);
        }
    };
    bool ok = true;
    const auto store = [&](const uint4 (&from)[P::kLoads], int u) {
        const Unit n = unit_of(u, nst);
        const int nslots = n.is_v ? kVStages : kKStages, slot = n.stage % nslots;
        uint64_t* empty = n.is_v ? bars->v_empty : bars->k_empty;
        if (n.stage >= nslots) ok = mbar_wait_warp(&empty[slot], ((n.stage / nslots) & 1) ^ 1);
        if (!ok) return;
        uint8_t* dst = smem + (n.is_v ? P::kOffV : P::kOffK) + slot * P::kStage + n.part * (kBlockSize * 128);
#pragma unroll
        for (int i = 0; i < P::kLoads; ++i) {
            // 16 codes: the 16-byte chunks ch, ch + 1 of column half h; lanes of the second half
            // store them in the other order, so that the lanes of one row hit different banks
            const int piece = i * 32 + lane, row = piece / (D / 16), c = piece % (D / 16);
            const int h = c >> 2, ch = (c & 3) * 2;
            const uint4 now = from[i];
            uint4 lo, hi;
            e4m3x4_to_f16x4(now.x, lo.x, lo.y);
            e4m3x4_to_f16x4(now.y, lo.z, lo.w);
            e4m3x4_to_f16x4(now.z, hi.x, hi.y);
            e4m3x4_to_f16x4(now.w, hi.z, hi.w);
            uint8_t* at = dst + h * P::kKVHalf;
            *reinterpret_cast<uint4*>(at + swz128(row, ch + h)) = h ? hi : lo;
            *reinterpret_cast<uint4*>(at + swz128(row, ch + 1 - h)) = h ? lo : hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(n.is_v ? &bars->v_full[slot] : &bars->k_full[slot]);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (w + i * kCvtWarps < total) load(codes[i], w + i * kCvtWarps);
    for (int u0 = w; u0 < total && ok; u0 += kAhead * kCvtWarps)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int u = u0 + i * kCvtWarps;
            if (u >= total || !ok) break;
            store(codes[i], u);
            if (u + kAhead * kCvtWarps < total) load(codes[i], u + kAhead * kCvtWarps);
        }
    if (!ok && lane == 0) atomicOr(a.status, kDevTimeout);
}

// The scales of a stage's four blocks as one row's softmax takes them.
struct StageScales {
    float f[kParts], kv[kParts];  // factor on s; exponent of V
};

// Largest s f + kV of the stage's visible keys c <= lim (all of them with kAll).
template <bool kAll>
__device__ __forceinline__ float stage_max(const uint32_t (&s)[2][32], int lim, const StageScales& sc) {
    float best = -INFINITY;
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
        const float m = fmaxf(m0, m1);
        best = fmaxf(best, m == -INFINITY ? m : fmaf(m, sc.f[i], sc.kv[i]));
    }
    return best;
}

// u of the stage against `nbase` (= -base), as f16 pairs into the 32 columns at `dst`; returns their
// plain sum, and adds the sum of u 2^-kV to lsum.
template <bool kAll>
__device__ __forceinline__ float stage_u(const uint32_t (&s)[2][32], int lim, const StageScales& sc, float nbase,
                                         uint32_t dst, float& lsum) {
    float all = 0.f;
    lsum = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const float off = sc.kv[i] + nbase;
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        uint32_t pw[8];
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
            const int c = i * 16 + t;
            float x0, x1;
            fma_x2(x0, x1, __uint_as_float(s[c >> 5][c & 31]), __uint_as_float(s[c >> 5][(c & 31) + 1]), sc.f[i],
                   sc.f[i], off, off);
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
        lsum = fmaf(sum, exp2_int(-(int)sc.kv[i]), lsum);
        tmem_st8_nowait(dst + 8 * i, pw[0], pw[1], pw[2], pw[3], pw[4], pw[5], pw[6], pw[7]);
    }
    return all;
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm) prefill8_kernel(const __grid_constant__ Pre8Args a) {
    using P = Pre8<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars8* bars = reinterpret_cast<Bars8*>(smem + P::kOffBars);
    float* row_inv = reinterpret_cast<float*>(smem + P::kOffInv);
    int* all_ok = reinterpret_cast<int*>(row_inv + kRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blockIdx.x = (rank * batch + b) * num_kv_heads + kvh: rank 0 is every chunk's last tile
    const int kvh = (int)(blockIdx.x % (unsigned)a.num_kv_heads);
    const int rb = (int)(blockIdx.x / (unsigned)a.num_kv_heads);
    const int b = rb % a.batch, rank = rb / a.batch;
    pdl_wait();
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(a.status, kDevOutOfRange);
        return;
    }
    const int g = a.group;
    const int q0 = a.cu_q_lens[b];
    const int C = a.cu_q_lens[b + 1] - q0;
    const int L = a.seq_lens[b];
    if (C < 0 || L < C || L > a.max_blocks * kBlockSize) {
        if (threadIdx.x == 0 && rank == 0 && kvh == 0) atomicOr(a.status, kDevOutOfRange);
        return;
    }
    const long long rows = (long long)C * g;
    const long long need = (rows + kRows - 1) / kRows;
    // a chunk longer than max_chunk: the grid covers its first tiles, the rest is reported
    if (rank == 0 && kvh == 0 && threadIdx.x == 0 && need > a.tiles) atomicOr(a.status, kDevOutOfRange);
    const int covered = (int)min(need, (long long)a.tiles);
    if (rank >= covered) return;
    const int row0 = (covered - 1 - rank) * kRows;
    const int live = (int)min((long long)kRows, rows - row0);
    const int nkeys = L - C + (row0 + live - 1) / g + 1;  // keys the tile's last query sees
    const int nst = (nkeys + kKeys - 1) / kKeys;
    const int nblk = (nkeys + kBlockSize - 1) / kBlockSize;
    const int32_t* bt = a.block_tables + (size_t)b * a.max_blocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bars->k_full[s], kParts);
            mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&bars->v_full[s], kParts);
            mbar_init(&bars->v_empty[s], 1);
        }
        mbar_init(&bars->q_full, kRows);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], kRows);
        }
        mbar_init(&bars->o_done, 1);
        mbar_init(&bars->o_final, 1);
        mbar_init(&bars->drain, 1);
        *all_ok = 1;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp >= kCvtWarp) {
        widen_units<D>(smem, bars, a, bt, kvh, L, nst, nblk, warp - kCvtWarp);
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idesc_s = idesc_f16(kKeys, false), idesc_o = idesc_f16(D, true);
        const uint64_t qd = smem_desc_sw128(smem_u32(smem), 0, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + P::kOffK), 0, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + P::kOffV), P::kKVHalf, 1024);
        const auto issue_s = [&](int j) {  // S(j) into buffer j % 2
            const uint64_t kd = kd0 + (uint64_t)(((j % kKStages) * P::kStage) >> 4);
            const uint32_t d = tmem + kTmemS + 64 * (j & 1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_ew(d, qd + (uint64_t)(((kk >> 2) * P::kQHalf + (kk & 3) * 32) >> 4),
                          kd + (uint64_t)(((kk >> 2) * P::kKVHalf + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
            tc_commit_ew(&bars->s_full[j & 1]);
            tc_commit_ew(&bars->k_empty[j % kKStages]);
        };
        const auto issue_o = [&](int j) {  // O += u(j) V(j), u(j) in buffer j % 2
            const uint64_t vd = vd0 + (uint64_t)(((j % kVStages) * P::kStage) >> 4);
            const uint32_t p = tmem + kTmemS + 64 * (j & 1);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                tc_mma_ts_ew(tmem + kTmemO, p + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o,
                             (j > 0 || kk > 0) ? 1u : 0u);
            tc_commit_ew(&bars->o_done);
            tc_commit_ew(&bars->v_empty[j % kVStages]);
            if (j + 1 == nst) tc_commit_ew(&bars->o_final);
        };
        bool ok = mbar_wait_warp(&bars->q_full, 0);
        for (int j = 0; j < 2 && j < nst && ok; ++j) {
            ok = mbar_wait_warp(&bars->k_full[j], 0);
            if (!ok) break;
            tc_fence_after();
            issue_s(j);
        }
        for (int j = 0; j < nst && ok; ++j) {
            ok = mbar_wait_warp(&bars->v_full[j % kVStages], (j / kVStages) & 1);
            if (ok && j + 2 < nst) ok = mbar_wait_warp(&bars->k_full[(j + 2) % kKStages], ((j + 2) / kKStages) & 1);
            if (ok) ok = mbar_wait_warp(&bars->p_full[j & 1], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_o(j);
            if (j + 2 < nst) issue_s(j + 2);  // after u V(j), whose u sits in its buffer
        }
        // every MMA issued here has finished before the tensor memory is released
        tc_commit_ew(&bars->drain);
        if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
        if (!ok && lane == 0) atomicOr(a.status, kDevTimeout);
    } else {
        // ---------------------------------------------------------------- softmax: one row a thread
        const int r = threadIdx.x;
        const bool valid = r < live;
        const int qi = (row0 + r) / g, h = (row0 + r) % g;
        const int pos = valid ? L - C + qi : -1;  // last key the row sees
        const uint32_t tm = tmem + ((uint32_t)(warp * 32) << 16);
        // exponents of blocks c0 + lane: a word a lane, the next 32 read ahead
        const auto entry = [&](int blk) { return blk < nblk ? __ldg(bt + blk) : -1; };
        const auto exps_of = [&](int blk, int id) -> int {
            if (blk >= nblk) return kExpBias * 257;
            return __ldg(a.exps + (size_t)(id < 0 || id >= a.num_blocks ? 0 : id) * a.num_kv_heads + kvh);
        };
        int ex = exps_of(lane, entry(lane)), next_id = entry(32 + lane), next_ex = 0;
        int eq;
        {
            // the row of q, normalised, into the swizzled layout (zeros past the chunk); a
            // negative scale enters as -q, so that maxima are of the scores as they are
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + ((size_t)(q0 + (valid ? qi : 0)) * a.num_heads + (size_t)kvh * g + h) * D);
            uint4 v[D / 8];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) v[c] = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = fabsf(bf16_lo(w[i])), y = fabsf(bf16_hi(w[i]));
                    amax = fmaxf(amax, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
                }
            }
            eq = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -110);
            const float s = a.scale_log2 < 0.f ? -exp2_int(-eq) : exp2_int(-eq);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const auto w = [&](uint32_t x) { return pack_f16x2(bf16_lo(x) * s, bf16_hi(x) * s); };
                *reinterpret_cast<uint4*>(smem + (c >> 3) * P::kQHalf + swz128(r, c & 7)) =
                    make_uint4(w(v[c].x), w(v[c].y), w(v[c].z), w(v[c].w));
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars->q_full);
        }
        const float sl = fabsf(a.scale_log2);
        float base = -INFINITY, l = 0.f;
        bool ok = true;
        // tcgen05.ld / st are warp-collective: what leads to one is decided by the whole warp
        for (int j = 0; j < nst; ++j) {
            const int at = (j * kParts) & 31;
            if (at == 0 && j > 0) {
                ex = next_ex;
                next_id = entry(j * kParts + 32 + lane);
            }
            StageScales sc;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const int e = __shfl_sync(0xffffffffu, ex, at + i);
                sc.f[i] = sl * exp2_int(eq + (e & 255) - kExpBias);
                sc.kv[i] = static_cast<float>((e >> 8) - kExpBias);
            }
            if (at == 16) next_ex = exps_of(j * kParts + 16 + lane, next_id);
            const uint32_t buf = tm + kTmemS + 64 * (j & 1);
            ok = mbar_wait_warp(&bars->s_full[j & 1], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const int lim = pos - j * kKeys;
            const bool unmasked = __all_sync(0xffffffffu, lim >= kKeys - 1);
            uint32_t s[2][32];
            tmem_ld32_async(buf, s[0]);
            tmem_ld32_async(buf + 32, s[1]);
            tmem_wait_ld(s[0]);
            tmem_wait_ld(s[1]);
            const auto weigh = [&](float& lsum) {
                const float nbase = base == -INFINITY ? 0.f : -base;
                return unmasked ? stage_u<true>(s, lim, sc, nbase, buf, lsum)
                                : stage_u<false>(s, lim, sc, nbase, buf, lsum);
            };
            float lsum = 0.f;
            bool full = __any_sync(0xffffffffu, base == -INFINITY && lim >= 0);
            if (!full) full = __any_sync(0xffffffffu, !(weigh(lsum) <= kSumLimit));
            if (full) {
                tmem_wait_st();  // a first attempt's u: the second goes over it
                const float mx = unmasked ? stage_max<true>(s, lim, sc) : stage_max<false>(s, lim, sc);
                const float top = fmaxf(base, mx);
                const bool move = top > base + kRebase;  // always at a row's first visible key
                const bool rescale = move && base != -INFINITY;
                const float f = rescale ? fast_exp2(base - top) : 1.f;
                if (__any_sync(0xffffffffu, rescale)) {
                    // O changes once u V(j - 1) has finished: phase j - 1 of o_done (phases up to
                    // j - 2 are over, as S(j) followed u V(j - 2), and u V(j) waits for this u)
                    if (j > 0) ok = mbar_wait_warp(&bars->o_done, (j - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    scale_o<D>(tm + kTmemO, f);
                }
                if (move) {
                    // in two steps: l, whose terms carry 2^-kV, may count where f alone is zero
                    if (rescale) {
                        const float h = fast_exp2(0.5f * (base - top));
                        l = l * h * h;
                    }
                    base = top;
                }
                weigh(lsum);
            }
            l += lsum;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_full[j & 1]);
        }
        if (ok) ok = mbar_wait_warp(&bars->o_final, 0);
        row_inv[r] = l > 0.f ? 1.f / l : 0.f;
        if (!ok && lane == 0) {
            *all_ok = 0;
            atomicOr(a.status, kDevTimeout);
        }
    }
    __syncthreads();
    tc_fence_after();
    // ---------------------------------------------------------------- epilogue
    if (*all_ok) {
        const int r = (warp & 3) * 32 + lane;
        const bool valid = r < live;
        const int qi = (row0 + r) / g, h = (row0 + r) % g;
        __nv_bfloat16* dst =
            a.out + ((size_t)(q0 + (valid ? qi : 0)) * a.num_heads + (size_t)kvh * g + h) * D;
        const float inv = row_inv[r];
        const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kTmemO;
        const int c0 = (warp >> 2) * (D / 2);
#pragma unroll
        for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            tmem_ld32(tm + c0 + c, o);
            if (valid) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const auto w = [&](int i) {
                        return pack_bf16x2(__uint_as_float(o[e + i]) * inv, __uint_as_float(o[e + i + 1]) * inv);
                    };
                    *reinterpret_cast<uint4*>(dst + c0 + c + e) = make_uint4(w(0), w(2), w(4), w(6));
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
    p.tiles = (int)(((long long)a.max_chunk * g + kRows - 1) / kRows);
    p.scale_log2 = a.scale * kLog2e;
    const long long ctas = (long long)p.tiles * a.batch * pool.num_kv_heads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;  // more CTAs than a grid holds
    return pool.head_dim == 128 ? launch<128>(p, (unsigned)ctas, stream) : launch<64>(p, (unsigned)ctas, stream);
}

}  // namespace pa
