// pa_decode_lanes.cu -- paged GQA decode with lane-private loads: over an 8-bit pool (pa_kv8.cuh:
// e4m3 codes, one power-of-two scale per block, kv head and tensor), and, over either pool,
// with the attention weight every block got added up.
//
//   o = sum_t softmax_t(scale <q, K_t>) V_t,   8-bit: K_t = codeK_t 2^kK(block), V_t = codeV_t 2^kV(block)
//
// One CTA serves one (sequence, kv head, split); its warps, and the splits of a sequence
// (one thread-block cluster, merged through distributed shared memory), take the blocks
// round-robin, so a warp's block indices do not depend on the sequence's length.
//
// Products, 8 bits.  The codes enter the tensor core as f16, which holds every e4m3 value
// exactly, at one conversion per two codes.  (Codes as they are against q in two e4m3 parts, without a
// conversion: 64 x ~1088 tokens 27.4 us against 25.9, 4 queries of each 42.8 against 32.4.)  K's
// scale joins the softmax scale (one factor per block and head).  q enters as f16 too, after its
// row is brought to a maximum in [2^14, 2^15) by a power of two that joins the same factor: an
// element loses bits only below 2^-29 of the row's maximum.  V's scale joins the exponent: with
// x = log2(e) scale <q, K> the weight the V product takes is u = 2^(x + kV - m + 7), m following
// the maximum of x + kV, so u fits f16 whatever the blocks' scales, and the largest contributions,
// not the largest probabilities, set its range.  u is rounded to f16's 11 bits (an eighth of the
// rounding of the bf16 result) where it is more than 2^-21 of the largest, to fewer below, and is zero below
// 2^-32 (kHeadroom); the normaliser adds u 2^(-kV - 7) in fp32, unrounded.  Where scales lie far apart
// (far_scale) it adds 2^(x - m), each by an exponential of its own: u may be zero where that is not.
// 16 bits: the same with kK = kV = 0 on bf16 MMAs, u carried as two bf16 parts.
//
// Loads.  Which d values make one MMA step, and which token is which MMA row, is free as long as q,
// u and the output agree, so every lane takes 16-byte pieces of a few rows as its fragments, with
// no ldmatrix and no exchange between lanes.  Each warp fetches its own blocks by TMA, K and V of a
// block in one box (their pools are two planes of one tensor map), into a private ring of
// swizzled slots, in which the pieces are chosen so that an access has no bank conflict: no
// barrier between warps, and one copy instruction a block.
//
// Weights.  A block's sum of 2^x per head goes to a workspace as it is computed; once the
// sequence's maximum and normaliser are known (after the merge) the CTA that read the block turns
// the sums into weights, adds the group's heads in order and updates its own entry: no
// atomics, no second launch.
//
// Measured on GB300, 32 q / 8 kv heads of d 128, 8-bit: 64 x ~1088 tokens 25.6 us (84% of the copy bandwidth;
// 23.1 with the copies alone), 64 x ~8192 with 64 q heads 164 us (98%), 4 queries of each of 64 x ~1088
// 31.5 us, 1 x 1152 6.1 us; with weights 64 x ~1088 28.1 us, bf16 45 us (95%).  Long batches are bound by
// memory, short ones by the chain table, block, merge and by the ends of their one wave.  Splits follow the
// tables' width, not the lengths: 64 x ~1088 in tables of 576 blocks and more runs in two splits, 30.4 us.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <int BITS, int D>
struct Lanes {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kBlockBytes = 2 * kBlockSize * kRowBytes;  // K and V of one (block, kv head)
    static constexpr int kPlane = kBlockSize * kRowBytes;  // K or V of one (block, kv head)
    static constexpr int kKChunks = kRowBytes / 64;                 // of a K row
    static constexpr int kVChunks = kRowBytes > 128 ? 2 : 1;                 // of a V row (half of one at 64 bytes)
    // merge scratch: per warp, and for the CTA, m[16], l[16], O[16][kRow]
    static constexpr int kRow = D + 4;
    static constexpr int kPart = 32 + 16 * kRow;
    static constexpr int merge_bytes(int warps) { return (warps + 1) * kPart * 4; }
    // blocks in flight per warp: what an SM's shared memory holds for the warps that run on it
    __host__ __device__ static constexpr int stages(int warps, int ctas) {
        return 196608 / (ctas * warps * kBlockBytes);
    }
    __host__ __device__ static constexpr int ring_bytes(int warps, int ctas) {
        return stages(warps, ctas) * warps * kBlockBytes;
    }
    // behind the rings and their barriers: the q fragments, where the registers of four warps have no
    // room for them (the same for every warp; 8 x ~2000 tokens, 16 heads a group: 14.4 us, with
    // three warps and q in registers 15.8, with four and 112 bytes of spills 15.4)
    __host__ __device__ static constexpr bool q_shared(int nt) { return BITS == 8 && D == 128 && nt == 2; }
    __host__ __device__ static constexpr int q_at(int warps, int ctas) {
        return (ring_bytes(warps, ctas) + stages(warps, ctas) * warps * 8 + 15) / 16 * 16;
    }
    static constexpr int smem(int warps, int ctas, int nt) {
        const int ring = q_at(warps, ctas) + (q_shared(nt) ? D / 16 * 32 * 16 : 0);
        return ring > merge_bytes(warps) ? ring : merge_bytes(warps);
    }
    static constexpr int kQuads = D / 32;  // 4-float groups of O a lane holds per head
    // which group of a head's row (d / 4) the lane's MMA tiles 2 w, 2 w + 1 hold
    __device__ static constexpr int quad(int gid, int w) {
        return BITS == 16 && D == 128 ? (w >> 1) * 16 + gid * 2 + (w & 1) : gid * kQuads + w;
    }
};

struct LanesArgs {
    const __nv_bfloat16* q;
    const uint8_t* k;
    const uint8_t* v;
    const uint16_t* exps;  // 8 bits: K in the low byte
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;  // multi-query only
    __nv_bfloat16* out;
    float* weights;  // [B, Hkv, max_blocks], or null
    float* ws;       // [B, Hkv, max_blocks, 8 NT] log2 of a block's summed weight per column
    unsigned* status;
    int max_blocks, num_heads, num_kv_heads, num_blocks, group;
    float scale_log2, decay;
    // one box brings K and V of a block (their pools as two planes of one map), and whether
    // K is the second plane; else a box each
    int paired, k_second;
};

// Warps of a CTA: 4, or 3 where a thread needs more than 128 registers (16-bit rows of d 128), so
// that four CTAs fit an SM in either case: 512 CTAs (64 sequences of 8 kv heads) are then one wave.  WIDE 1, 2: twice and
// four times as many, two CTAs and one an SM, where even the most splits leave SMs empty.
__host__ __device__ constexpr bool fits128(int bits, int d, int nt) { return d == 64 || bits == 8; }
__host__ __device__ constexpr int warps_of(int bits, int d, int nt, int wide) {
    return (fits128(bits, d, nt) ? 4 : 3) << wide;
}
__host__ __device__ constexpr int ctas_of(int wide) { return 4 >> wide; }

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
// One box of a pool map: x = 0, row, then for 16-bit rows their 128-byte halves, then K and V.
template <bool HALVES>
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar, uint64_t policy) {
    if constexpr (HALVES)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %2, %2}], [%4], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %2}], [%4], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar), "l"(policy)
            : "memory");
}
// log2 on the special-function unit (0 gives -inf)
__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A normaliser l = sum of 2^(x - base) moved from one base to one 2^-d higher: l 2^d.  Its terms carry
// 2^-kV, so l may be as large as 2^100 where x + kV is the base, and l 2^d matters where 2^d alone
// is zero in fp32 (blocks of V at the two ends of the scales' range).
__device__ __forceinline__ float rescale_sum(float l, float d) {
    const float h = fast_exp2(0.5f * d);
    return l * h * h;
}

// 2^x down to fp32's last subnormal (fast_exp2 ends at 2^-126), for terms of the normaliser.
__device__ __forceinline__ float exp2_term(float x) {
    const float h = fast_exp2(0.5f * x);
    return h * h;
}

// Where group `grp` (4 floats) of a head's row sits in the merge scratch: the lanes that write one
// instruction's groups hit different banks.
__device__ __forceinline__ int quad_at(int grp) { return grp ^ ((grp >> 2) & 1); }

template <int BITS, int D, int NT, bool MQ, bool WEIGHTS, int WIDE>
__global__ void __launch_bounds__(warps_of(BITS, D, NT, WIDE) * 32, ctas_of(WIDE))
    decode_lanes_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ LanesArgs a) {
    static_assert(!MQ || BITS == 8, "codes of 8 bits");
    using Sh = Lanes<BITS, D>;
    constexpr int kWarps = warps_of(BITS, D, NT, WIDE), kThreads = kWarps * 32;
    constexpr int kCtas = ctas_of(WIDE);
    constexpr int kStages = Sh::stages(kWarps, kCtas);  // ring slots per warp
    constexpr int kSteps = D / 16;    // MMA steps over d (K), tiles of d (V)
    // u at a column's maximum is 2^kHead, and moves the base past kTop (f16 ends at 2^16)
    constexpr int kHead = BITS == 8 ? kHeadroom : 0;
    constexpr float kTop = BITS == 8 ? 32768.f : 1024.f;
    constexpr int kRowB = Sh::kRowBytes;
    extern __shared__ __align__(1024) uint8_t smem[];

    uint32_t ncl;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncl));
    const int sub = static_cast<int>(ncl), rank = blockIdx.x % sub;
    const int kvh = blockIdx.y, b = blockIdx.z;
    // (by a shuffle, so that the compiler knows it is the same for all lanes and keeps what follows from it
    // in uniform registers: 4 x 64 queries 30.7 us against 32.5, d 64 64 x ~4000 48.8 against 53.4)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3;
    // Which row of a block is which MMA row or key: neighbouring ones are kNext rows apart, which the
    // swizzle (of 128-byte rows by their index modulo 8, of 64-byte rows by half of it) and the row
    // length put into different banks.  trow: the row of MMA row gid (gid + 8: trow + 8).
    constexpr int kNext = kRowB == 64 ? 1 : 4;
    const int trow = kRowB == 64 ? gid : (gid >> 1) | ((gid & 1) << 2);
    const int g = a.group;
    const int first = rank * kWarps + warp, stride = sub * kWarps;  // this warp's blocks
    const int32_t* bt = a.block_tables + (size_t)b * a.max_blocks;
    pdl_wait();
    if (smem_u32(smem) & 1023u) {  // the swizzled slots need the declared alignment
        if (threadIdx.x == 0) atomicOr(a.status, kDevOutOfRange);
        return;
    }

    // lane l keeps the id and exponents of the warp's block number c0 + l; the table entry does
    // not wait for the length (an entry past the sequence's blocks is not used)
    const auto entry_at = [&](int k) { return first + (long long)k * stride; };
    int id = entry_at(lane) < a.max_blocks ? __ldg(bt + entry_at(lane)) : 0;
    int L = a.seq_lens[b];
    if (L < 0 || L > a.max_blocks * kBlockSize) {
        if (threadIdx.x == 0) atomicOr(a.status, kDevOutOfRange);
        L = L < 0 ? 0 : a.max_blocks * kBlockSize;
    }
    int C = 1, q0 = b;
    if (MQ) {
        q0 = a.cu_q_lens[b];
        C = a.cu_q_lens[b + 1] - q0;
        if (C < 0 || C > L || C * g > 8 * NT) {
            if (threadIdx.x == 0) atomicOr(a.status, kDevOutOfRange);
            C = 0;
        }
    }
    const int R = MQ ? C * g : g;  // columns in use: (query, head of the group)
    const int nb = R == 0 ? 0 : (L + kBlockSize - 1) / kBlockSize;
    const int n = nb > first ? (nb - first + stride - 1) / stride : 0;  // blocks of this warp

    const auto checked = [&](int k, int raw) {
        if (k < n && (raw < 0 || raw >= a.num_blocks)) {
            atomicOr(a.status, kDevOutOfRange);
            return 0;  // read inside the pool; the status word reports the bad id
        }
        return k < n ? raw : 0;
    };
    const auto exps_of = [&](int k, int blk) -> int {
        if (BITS == 16) return kExpBias * 257;
        return k < n ? valid_exps(__ldg(a.exps + (size_t)blk * a.num_kv_heads + kvh)) : kExpBias * 257;
    };
    id = checked(lane, id);
    int ex = exps_of(lane, id);

    // a ring slot holds K and V of one block, [16 rows][64 or 128 B] swizzled (256-byte rows: two such
    // halves); each warp issues and waits for its own
    const uint32_t ring = smem_u32(smem) + warp * kStages * Sh::kBlockBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sh::ring_bytes(kWarps, kCtas)) + warp * kStages;
    const uint64_t policy = l2_evict_first_policy();
    const auto issue = [&](int slot, int blk) {
        const int row = (blk * a.num_kv_heads + kvh) * kBlockSize;
        const uint32_t dst = ring + slot * Sh::kBlockBytes, bar = smem_u32(&full[slot]);
        mbar_arrive_expect_tx(&full[slot], Sh::kBlockBytes);
        tma_block<(kRowB > 128)>(dst, &tm_k, row, bar, policy);
        if (!a.paired) tma_block<(kRowB > 128)>(dst + Sh::kPlane, &tm_v, row, bar, policy);
    };
    if (lane < kStages) mbar_init(&full[lane], 1);
    if (lane == 0) {
        prefetch_tensormap(&tm_k);
        if (!a.paired) prefetch_tensormap(&tm_v);
    }
    fence_mbar_init();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
        const int blk = __shfl_sync(0xffffffffu, id, k);
        if (k < n && lane == 0) issue(k, blk);
    }

    // q as B fragments: column gid of each n-tile, the d values this lane's K pieces hold
    uint32_t qb[NT][kSteps][2];
    float qf[NT][2];    // of this thread's columns nt * 8 + 2 tig (+1): factor on the raw score
    int colpos[NT][2];  // and the last key they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = nt * 8 + gid;
        const __nv_bfloat16* row = nullptr;
        if (col < R) {
            const size_t tok = MQ ? (size_t)q0 + col / g : (size_t)b;
            row = a.q + (tok * a.num_heads + (size_t)kvh * g + (MQ ? col % g : col)) * D;
        }
        int e = 0;
        if constexpr (BITS == 8) {
            float f[kSteps][4];
            float amax = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint2 w = row ? __ldg(reinterpret_cast<const uint2*>(row + (s >> 2) * 64 + tig * 16 + (s & 3) * 4))
                                    : make_uint2(0u, 0u);
                f[s][0] = bf16_lo(w.x);
                f[s][1] = bf16_hi(w.x);
                f[s][2] = bf16_lo(w.y);
                f[s][3] = bf16_hi(w.y);
#pragma unroll
                for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(f[s][j]) < INFINITY ? fabsf(f[s][j]) : 0.f);
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -110);
            const float s2 = exp2_int(-e);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                qb[nt][s][0] = pack_f16x2(f[s][0] * s2, f[s][1] * s2);
                qb[nt][s][1] = pack_f16x2(f[s][2] * s2, f[s][3] * s2);
            }
        } else {
#pragma unroll
            for (int c = 0; c < Sh::kKChunks; ++c) {
                const uint4 w = row ? __ldg(reinterpret_cast<const uint4*>(row + c * 32 + tig * 8))
                                    : make_uint4(0u, 0u, 0u, 0u);
                qb[nt][2 * c][0] = w.x;
                qb[nt][2 * c][1] = w.y;
                qb[nt][2 * c + 1][0] = w.z;
                qb[nt][2 * c + 1][1] = w.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            qf[nt][j] = a.scale_log2 * exp2_int(__shfl_sync(0xffffffffu, e, (2 * tig + j) * 4));
            const int oc = nt * 8 + 2 * tig + j;
            colpos[nt][j] = MQ ? L - C + (oc < R ? oc / g : 0) : L - 1;  // unused columns: as the first
        }
    }

    constexpr bool kQShared = Sh::q_shared(NT);
    const uint32_t q_smem = smem_u32(smem) + Sh::q_at(kWarps, kCtas) + lane * 16;
    if constexpr (kQShared) {
        if (warp == 0) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                sts16(q_smem + s * 512, make_uint4(qb[0][s][0], qb[0][s][1], qb[NT - 1][s][0], qb[NT - 1][s][1]));
        }
        __syncthreads();
    }

    float ot[NT][kSteps][4];
    float m[NT][2], l[NT][2];  // base and normaliser of the columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) ot[nt][s][0] = ot[nt][s][1] = ot[nt][s][2] = ot[nt][s][3] = 0.f;
    }

    const int all_see = MQ ? L - C : L - 1;  // every column sees keys up to this one
    int nid = 0, nex = 0;
    // This lane's pieces of a slot.  K: rows trow, trow + 8, 16-byte chunks tig, tig + 4, ...  V: keys
    // 2 tig, 2 tig + 1 (+ 8) are rows kNext apart, chunk gid (64-byte rows: half of chunk gid / 2);
    // the lanes that would meet the others' banks take the two in the other order, and the byte
    // permutations below put the pair right.
    constexpr int kSlotRow = kRowB == 64 ? 64 : 128;
    const bool swapped = kRowB == 64 ? gid >> 1 & 1 : gid & 1;
    const int vrow = (kRowB == 64 ? 2 * tig : tig) + (swapped ? kNext : 0);
    uint32_t k_off, v_off, v_flip;  // v_flip: row ^ kNext, and the chunk with it
    if constexpr (kRowB == 64) {
        k_off = trow * 64 + ((tig ^ (trow >> 1 & 3)) << 4);
        v_off = vrow * 64 + (((gid >> 1) ^ tig) << 4) + (gid & 1) * 8;
        v_flip = v_off ^ 64;
    } else {
        k_off = trow * 128 + ((tig ^ trow) << 4);
        v_off = vrow * 128 + ((gid ^ vrow) << 4);
        v_flip = v_off ^ (4 * 128 | 4 << 4);
    }
    k_off += a.k_second ? Sh::kPlane : 0;
    v_off += a.k_second ? 0 : Sh::kPlane;
    v_flip += a.k_second ? 0 : Sh::kPlane;
    bool ok = true;
    bool far = false;  // some block so far has a far_scale
    int slot = 0, parity = 0, k = 0;
    for (; k < n; ++k) {
        const int at = k & 31;
        // the next 32 entries, then (once they have come) their exponents
        if (at == 0 && k + 32 + lane < n) nid = __ldg(bt + entry_at(k + 32 + lane));
        if (at == 16) {
            nid = checked(k + 16 + lane, nid);
            nex = exps_of(k + 16 + lane, nid);
        }
        const uint32_t st_at = ring + slot * Sh::kBlockBytes;
        ok = mbar_wait_warp(&full[slot], parity);
        if (!ok) break;
        float kscale = 1.f, unscale = 1.f, fev = 0.f;  // 2^kK, 2^(-kV - kHead), kV
        if constexpr (BITS == 8) {
            const int e = __shfl_sync(0xffffffffu, ex, at);
            kscale = __int_as_float((e & 255) << 23);
            unscale = __int_as_float((2 * kExpBias - kHead - (e >> 8)) << 23);
            fev = static_cast<float>((e >> 8) - kExpBias);
            far = far || far_scale(e >> 8);
        }
        const int kbase = static_cast<int>(entry_at(k)) * kBlockSize;

        // S^T = K q^T: rows are tokens gid, gid + 8, columns the heads; two chains of MMAs (one
        // per n-tile, or two of the one)
        float st[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) st[0][i] = st[1][i] = 0.f;
#pragma unroll
        for (int c = 0; c < Sh::kKChunks; ++c) {
            // chunk 4 (c % 2) + tig of 128-byte piece c / 2 of the rows
            const uint32_t at16 = st_at + (k_off ^ ((c & 1) << 6)) + (c >> 1) * (kBlockSize * 128);
            const uint4 p0 = lds16(at16), p8 = lds16(at16 + 8 * kSlotRow);
            const uint32_t w0[4] = {p0.x, p0.y, p0.z, p0.w}, w8[4] = {p8.x, p8.y, p8.z, p8.w};
            if constexpr (BITS == 8) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16x4(w0[s], a0, a2);
                    e4m3x4_to_f16x4(w8[s], a1, a3);
                    if constexpr (kQShared) {
                        const uint4 f = lds16(q_smem + (c * 4 + s) * 512);
                        mma_f16_16816(st[0], a0, a1, a2, a3, f.x, f.y);
                        mma_f16_16816(st[1], a0, a1, a2, a3, f.z, f.w);
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(st[NT == 1 ? s & 1 : nt], a0, a1, a2, a3, qb[nt][c * 4 + s][0],
                                          qb[nt][c * 4 + s][1]);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816(st[NT == 1 ? s & 1 : nt], w0[2 * s], w8[2 * s], w0[2 * s + 1], w8[2 * s + 1],
                                  qb[nt][c * 2 + s][0], qb[nt][c * 2 + s][1]);
            }
        }
        // u against the columns' bases as they are; the bases move only in a warp's first block, or
        // when some u passes kTop, then to the maximum
        float u[NT][2][2];  // [column][token gid, gid + 8]
        const bool whole = kbase + kBlockSize - 1 <= all_see;
        bool move = k == 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float f = qf[nt][j] * kscale, off = fev + kHead - (m[nt][j] == -INFINITY ? 0.f : m[nt][j]);
                st[nt][j] = (NT == 1 ? st[0][j] + st[1][j] : st[nt][j]) * f;
                st[nt][2 + j] = (NT == 1 ? st[0][2 + j] + st[1][2 + j] : st[nt][2 + j]) * f;
                u[nt][j][0] = fast_exp2(st[nt][j] + off);
                u[nt][j][1] = fast_exp2(st[nt][2 + j] + off);
            }
        if (!whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lim = colpos[nt][j] - kbase;  // keys up to this one of the block are visible
                    if (trow > lim) u[nt][j][0] = 0.f, st[nt][j] = -INFINITY;
                    if (trow + 8 > lim) u[nt][j][1] = 0.f, st[nt][2 + j] = -INFINITY;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) move |= !(u[nt][j][0] <= kTop) || !(u[nt][j][1] <= kTop);
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(st[nt][j], st[nt][2 + j]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[nt][j], mx + fev);
                    const float base = mn == -INFINITY ? 0.f : mn;  // nothing visible so far
                    const float alpha = fast_exp2(m[nt][j] - base);
                    l[nt][j] = rescale_sum(l[nt][j], m[nt][j] - base);
                    m[nt][j] = mn;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        ot[nt][s][j] *= alpha;
                        ot[nt][s][2 + j] *= alpha;
                    }
                    u[nt][j][0] = fast_exp2(st[nt][j] + (fev + kHead - base));
                    u[nt][j][1] = fast_exp2(st[nt][2 + j] + (fev + kHead - base));
                }
        }
        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float sum[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[j] = (u[nt][j][0] + u[nt][j][1]) * unscale;
                if (far) {
                    const float base = m[nt][j] == -INFINITY ? 0.f : m[nt][j];
                    sum[j] = exp2_term(st[nt][j] - base) + exp2_term(st[nt][2 + j] - base);
                }
                l[nt][j] += sum[j];
            }
            if (WEIGHTS) {
                // over the 8 lanes of a column: lanes of odd gid end with column 1, the others with 0
                const bool odd = gid & 1;
                float t = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, odd ? sum[0] : sum[1], 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                float from = odd ? m[nt][1] : m[nt][0];
                if (far) {
                    // terms under m may be subnormal though they count: under the block's own maximum instead
                    float own[2], top[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        top[j] = fmaxf(st[nt][j], st[nt][2 + j]);
                        for (int o = 4; o < 32; o <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
                        const float base = top[j] == -INFINITY ? 0.f : top[j];
                        own[j] = fast_exp2(st[nt][j] - base) + fast_exp2(st[nt][2 + j] - base);
                        for (int o = 4; o < 32; o <<= 1) own[j] += __shfl_xor_sync(0xffffffffu, own[j], o);
                    }
                    t = odd ? own[1] : own[0];
                    from = odd ? top[1] : top[0];
                }
                if (gid < 2)
                    a.ws[(((size_t)b * a.num_kv_heads + kvh) * a.max_blocks + entry_at(k)) * (8 * NT) + nt * 8 +
                         2 * tig + gid] = fast_log2(t) + from;
            }
            // rows (tokens) x columns (heads) -> transposed: the B operand of the V product
            if constexpr (BITS == 8) {
                pb[nt][0] = movmatrix_t(pack_f16x2(u[nt][0][0], u[nt][1][0]));
                pb[nt][1] = movmatrix_t(pack_f16x2(u[nt][0][1], u[nt][1][1]));
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = pack_bf16x2(u[nt][0][i], u[nt][1][i]);
                    pb[nt][i] = movmatrix_t(hi);
                    pl[nt][i] = movmatrix_t(pack_bf16x2(u[nt][0][i] - bf16_lo(hi), u[nt][1][i] - bf16_hi(hi)));
                }
            }
        }
        // O^T += V^T u^T: tile rows gid, gid + 8 are neighbouring d
        constexpr int kVWords = kRowB / 32;  // words of each of the lane's four V rows
        uint32_t vw[4][kVWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t from = st_at + (r & 1 ? v_flip : v_off) + (r >> 1) * (8 * kSlotRow);
            if constexpr (kRowB == 64) {
                const uint2 p = lds8(from);
                vw[r][0] = p.x;
                vw[r][1] = p.y;
            } else {
#pragma unroll
                for (int c = 0; c < Sh::kVChunks; ++c) {
                    const uint4 p = lds16(from + c * (kBlockSize * 128));
                    vw[r][4 * c] = p.x;
                    vw[r][4 * c + 1] = p.y;
                    vw[r][4 * c + 2] = p.z;
                    vw[r][4 * c + 3] = p.w;
                }
            }
        }
        if (MQ ? !whole : kbase + kBlockSize > L) {
            // rows past the sequence's end: whatever they hold (NaN times u = 0 is NaN)
            uint32_t some = 0u;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = kbase + (vrow ^ (r & 1 ? kNext : 0)) + (r >> 1) * 8;
                if (key >= L) {
#pragma unroll
                    for (int w = 0; w < kVWords; ++w) vw[r][w] = 0u;
                }
                if (MQ && key > all_see) {
#pragma unroll
                    for (int w = 0; w < kVWords; ++w) {
                        some |= nan_bits(vw[r][w]);
                        vw[r][w] &= ~nan_codes(vw[r][w]);
                    }
                }
            }
            if (MQ && __any_sync(0xffffffffu, (some & 0x80808080u) != 0u)) {
                // keys that only some columns see: a NaN stays out of the product too, where it would reach
                // every column, and goes straight into the sums of those that see it
                const uint32_t plane = st_at + (a.k_second ? 0 : Sh::kPlane);
#pragma unroll 1
                for (int row = max(0, all_see + 1 - kbase); row < min(kBlockSize, L - kbase); ++row) {
                    uint32_t x[4];
                    if constexpr (kRowB == 64) {
                        const uint2 p = lds8(plane + row * 64 + (((gid >> 1) ^ (row >> 1 & 3)) << 4) + (gid & 1) * 8);
                        x[0] = p.x, x[1] = p.y;
                    } else {
                        const uint4 p = lds16(plane + row * 128 + ((gid ^ (row & 7)) << 4));
                        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w;
                    }
#pragma unroll
                    for (int w = 0; w < kSteps / 2; ++w) {
                        const uint32_t nan = nan_codes(x[w]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (kbase + row <= colpos[nt][j] && nan >> (8 * i) & 1u)
                                        ot[nt][2 * w + (i >> 1)][j + 2 * (i & 1)] = __int_as_float(0x7fffffff);
                    }
                }
            }
        }
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
            if constexpr (BITS == 8) {
                // codes of d, d+1 (then d+2, d+3) paired over keys 2 tig, 2 tig + 1 and over the next 8
                const uint32_t sel_lo = swapped ? 0x1504u : 0x5140u, sel_hi = swapped ? 0x3726u : 0x7362u;
                const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], sel_lo);
                const uint32_t hi = __byte_perm(vw[0][w], vw[1][w], sel_hi);
                const uint32_t lo8 = __byte_perm(vw[2][w], vw[3][w], sel_lo);
                const uint32_t hi8 = __byte_perm(vw[2][w], vw[3][w], sel_hi);
                uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
                e4m3x4_to_f16x4(lo, a0, a1);
                e4m3x4_to_f16x4(lo8, a2, a3);
                e4m3x4_to_f16x4(hi, c0, c1);
                e4m3x4_to_f16x4(hi8, c2, c3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16_16816(ot[nt][2 * w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_f16_16816(ot[nt][2 * w + 1], c0, c1, c2, c3, pb[nt][0], pb[nt][1]);
                }
            } else {
                const uint32_t sel_lo = swapped ? 0x1054u : 0x5410u, sel_hi = swapped ? 0x3276u : 0x7632u;
                const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], sel_lo);
                const uint32_t a1 = __byte_perm(vw[0][w], vw[1][w], sel_hi);
                const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], sel_lo);
                const uint32_t a3 = __byte_perm(vw[2][w], vw[3][w], sel_hi);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(ot[nt][w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_16816(ot[nt][w], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                }
            }
        }
        if (at == 31) {  // on to the next 32 blocks
            id = nid;
            ex = nex;
        }
        // refill the slot: the block's id is among the current 32, or (entries not yet moved up) the next
        const int next = k + kStages;
        const int next_id = __shfl_sync(0xffffffffu, (next >> 5) != ((k + 1) >> 5) ? nid : id, next & 31);
        __syncwarp();  // every lane has its pieces
        if (next < n && lane == 0) issue(slot, next_id);
        if (++slot == kStages) slot = 0, parity ^= 1;
    }
    if (!ok) {
        // a wait ran out: the copies in flight must still land before their memory is used again
        for (int left = min(n - k, kStages); left > 0; --left) {
            mbar_wait_warp(&full[slot], parity);
            if (++slot == kStages) slot = 0, parity ^= 1;
        }
        if (lane == 0) atomicOr(a.status, kDevTimeout);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float t = l[nt][j];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            l[nt][j] = t;
        }
    __syncthreads();  // every warp is done with its ring
    pdl_trigger();

    // ---- the warps' partial (m, l, O) of each column -> the CTA's
    float* part = reinterpret_cast<float*>(smem);
    float* cta = part + kWarps * Sh::kPart;
    {
        float* pm = part + warp * Sh::kPart;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = nt * 8 + 2 * tig + j;
                if (gid == 0) {
                    // a column with no score but NaN (l = NaN) has found no maximum, but must not pass for one
                    // without keys, which the merge leaves out
                    pm[col] = m[nt][j] == -INFINITY && l[nt][j] != 0.f ? 0.f : m[nt][j];
                    pm[16 + col] = l[nt][j];
                }
#pragma unroll
                for (int w = 0; w < Sh::kQuads; ++w)
                    *reinterpret_cast<float4*>(pm + 32 + col * Sh::kRow + 4 * quad_at(Sh::quad(gid, w))) =
                        make_float4(ot[nt][2 * w][j], ot[nt][2 * w][2 + j], ot[nt][2 * w + 1][j],
                                    ot[nt][2 * w + 1][2 + j]);
            }
    }
    __syncthreads();
    const int quads = R * (D / 4);
    const auto out_at = [&](int qd) -> __nv_bfloat16* {  // 4 consecutive d of one column's row
        const int col = qd / (D / 4);
        const size_t tok = MQ ? (size_t)q0 + col / g : (size_t)b;
        return a.out + (tok * a.num_heads + (size_t)kvh * g + (MQ ? col % g : col)) * D + qd % (D / 4) * 4;
    };
    const auto inverse = [](float den) { return den > 0.f ? 1.f / static_cast<float>(1 << kHead) / den : 0.f; };
    const auto store = [&](int qd, const float4& v, float inv) {
        uint2 w = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(out_at(qd)) = w;
    };
    for (int qd = threadIdx.x; qd < quads; qd += kThreads) {
        const int col = qd / (D / 4), grp = qd % (D / 4);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part[w * Sh::kPart + col]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* pm = part + w * Sh::kPart;
            if (pm[col] == -INFINITY) continue;
            const float wt = fast_exp2(pm[col] - M);
            const float4 v = *reinterpret_cast<const float4*>(pm + 32 + col * Sh::kRow + 4 * quad_at(grp));
            acc.x += wt * v.x;
            acc.y += wt * v.y;
            acc.z += wt * v.z;
            acc.w += wt * v.w;
            den += rescale_sum(pm[16 + col], pm[col] - M);
        }
        if (sub == 1) store(qd, acc, inverse(den));
        *reinterpret_cast<float4*>(cta + 32 + col * Sh::kRow + 4 * grp) = acc;
        if (grp == 0) {
            cta[col] = M;
            cta[16 + col] = den;
        }
    }
    __syncthreads();
    float* col_m = cta;        // per column: maximum and normaliser over the whole sequence
    float* col_l = cta + 16;
    if (sub > 1) {
        // ---- the cluster's partials: first every (m, l), then this rank's slice of O from all
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        float* wgt = part;                // [16 ranks][16] weight of a rank's partial
        float* lsum = part + 256;         // [16][16]
        col_m = part + 512;
        col_l = part + 528;
        for (int t = threadIdx.x; t < sub * R; t += kThreads) {
            const int r = t / R, col = t % R;
            const float* rc = cluster.map_shared_rank(cta, r);
            wgt[r * 16 + col] = rc[col];
            lsum[r * 16 + col] = rc[16 + col];
        }
        __syncthreads();
        if (threadIdx.x < R) {
            const int col = threadIdx.x;
            float M = -INFINITY, den = 0.f;
            for (int r = 0; r < sub; ++r) M = fmaxf(M, wgt[r * 16 + col]);
            for (int r = 0; r < sub; ++r) {
                const float mr = wgt[r * 16 + col];
                wgt[r * 16 + col] = mr == -INFINITY ? 0.f : fast_exp2(mr - M);
                if (mr != -INFINITY) den += rescale_sum(lsum[r * 16 + col], mr - M);
            }
            col_m[col] = M;
            col_l[col] = den;
        }
        __syncthreads();
        const int per = (quads + sub - 1) / sub;
        for (int qd = rank * per + threadIdx.x; qd < min(quads, (rank + 1) * per); qd += kThreads) {
            const int col = qd / (D / 4), grp = qd % (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < sub; ++r) {
                const float w = wgt[r * 16 + col];
                const float4 v =
                    *reinterpret_cast<const float4*>(cluster.map_shared_rank(cta, r) + 32 + col * Sh::kRow + 4 * grp);
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
            store(qd, acc, inverse(col_l[col]));
        }
    }
    if (WEIGHTS) {
        // this CTA's blocks: the columns' shares of the whole sequence's weight, added up
        float* lse = part + 576;  // log2 of a column's whole sum of 2^x; a NaN column adds nothing
        if (threadIdx.x < R) {
            const float den = col_l[threadIdx.x];
            lse[threadIdx.x] = den > 0.f ? col_m[threadIdx.x] + log2f(den) : INFINITY;
        }
        __syncthreads();
        const int own = nb > rank * kWarps ? nb - rank * kWarps : 0;
        for (int t = threadIdx.x; t < (own + stride - 1) / stride * kWarps; t += kThreads) {
            const int blk = rank * kWarps + t % kWarps + t / kWarps * stride;
            if (blk >= nb) continue;
            const float* lb = a.ws + (((size_t)b * a.num_kv_heads + kvh) * a.max_blocks + blk) * (8 * NT);
            float sum = 0.f;
            for (int col = 0; col < R; ++col)
                if (lse[col] < INFINITY) sum += fast_exp2(lb[col] - lse[col]);
            float* w = a.weights + ((size_t)b * a.num_kv_heads + kvh) * a.max_blocks + blk;
            *w = *w * a.decay + sum;
        }
    }
    if (sub > 1) cg::this_cluster().sync();  // keep this CTA's partial until every reader is done
}

// Either pool as the kernel sees it.
struct LanesPool {
    const void *k, *v, *exps;
    int num_blocks, num_kv_heads, head_dim;
};

template <int BITS, int D, int NT, bool MQ, bool WEIGHTS, int WIDE>
cudaError_t launch_as(const LanesPool& pool, const AttnArgs& a, int splits, cudaStream_t stream) {
    using Sh = Lanes<BITS, D>;
    auto kern = decode_lanes_kernel<BITS, D, NT, MQ, WEIGHTS, WIDE>;
    constexpr int kWarps = warps_of(BITS, D, NT, WIDE);
    static OncePerDevice configured;  // per instantiation
    cudaError_t se = configured.run([&] {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::smem(kWarps, ctas_of(WIDE), NT));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e;
    });
    if (se != cudaSuccess) return se;
    LanesArgs d;
    d.q = static_cast<const __nv_bfloat16*>(a.q);
    d.k = static_cast<const uint8_t*>(pool.k);
    d.v = static_cast<const uint8_t*>(pool.v);
    d.exps = static_cast<const uint16_t*>(pool.exps);
    d.block_tables = a.block_tables;
    d.seq_lens = a.seq_lens;
    d.cu_q_lens = a.cu_q_lens;
    d.out = static_cast<__nv_bfloat16*>(a.out);
    d.weights = a.weights;
    d.ws = a.ws_weights;
    d.status = a.status;
    d.max_blocks = a.max_blocks;
    d.num_heads = a.num_heads;
    d.num_kv_heads = pool.num_kv_heads;
    d.num_blocks = pool.num_blocks;
    d.group = a.num_heads / pool.num_kv_heads;
    d.scale_log2 = a.scale * kLog2e;
    d.decay = a.decay;
    PlaneMaps maps = {};
    if (!plane_maps(&maps, pool.k, pool.v, (long long)pool.num_blocks * pool.num_kv_heads * kBlockSize,
                                Sh::kRowBytes))
        return cudaErrorInvalidValue;
    d.paired = maps.paired;
    d.k_second = maps.k_second;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, pool.num_kv_heads, a.batch);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = Sh::smem(kWarps, ctas_of(WIDE), NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (splits > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = splits;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, maps.k, maps.v, d);
}

// How many clusters of `splits` CTAs the device runs at once; asked once per device.
int cluster_capacity(int wide, int splits) {
    static std::atomic<int> cached[64][3][17];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (const int c = cached[dev][wide][splits].load(std::memory_order_relaxed)) return c - 1;
    const auto ask = [&](auto kern, int warps, int smem) {
        int n = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(splits * 64);
        cfg.blockDim = dim3(warps * 32);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = splits;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess ? n : 0;
    };
    using Sh = Lanes<8, 128>;
    const int n = wide == 2   ? ask(decode_lanes_kernel<8, 128, 1, false, false, 2>, 16, Sh::smem(16, 1, 1))
                  : wide == 1 ? ask(decode_lanes_kernel<8, 128, 1, false, false, 1>, 8, Sh::smem(8, 2, 1))
                              : ask(decode_lanes_kernel<8, 128, 1, false, false, 0>, 4, Sh::smem(4, 4, 1));
    cudaGetLastError();
    cached[dev][wide][splits].store(n + 1, std::memory_order_relaxed);
    return n;
}

struct Split {
    int splits, wide;
};

// Splits of every (sequence, kv head), as CTAs of a cluster.  Measured on GB300, us a call:
//   * as many as run at once: 16 x ~4000 tokens, 8 kv heads (128 items) 24 at 4 splits against 33 at
//     1; one cluster too many costs a second wave (32 items: wide at 8 splits 16, at 9 23);
//   * but at least ten blocks a warp once every SM has a CTA: 30 x 1000 (240 items) 13.9 at 1,
//     15.4 at 2; 24 x ~1500 21.9 at 1, 17.5 at 3;
//   * wide where even the most splits leave room, at four blocks a warp: 1 x 32768 (8 items) 17.6 with
//     16 warps at 12 splits (13 would not all run at once), 20.7 with 8 warps, 25.9 with 4; 4 x 8192
//     15.8 with 8 warps at 8 splits, 17.2 with 4 at 16;
//   * two in a grid of over three CTAs an SM with long sequences, whose CTAs end far apart: 64 x 8192
//     152 against 159, but 64 x 2048 47 against 44.
Split split_for(int batch, int num_kv_heads, int max_blocks, int warps) {
    const int items = batch * num_kv_heads, sms = device_info().num_sms;
    if (items >= 3 * sms) return {max_blocks >= 320 ? 2 : 1, 0};
    if (items <= cluster_capacity(0, 16)) {
        for (int wide = 2; wide; --wide) {
            int s = wide == 2 ? 16 : 12;
            while (s > 1 && items > cluster_capacity(wide, s)) --s;
            if (wide == 2 && s < 12) continue;
            if (s > 1 && max_blocks >= 4 * s * (warps << wide)) return {s, wide};
        }
    }
    const int least = items >= sms ? 10 * warps : 4;  // blocks of a CTA
    int s = std::min(16, std::max(1, max_blocks / least));
    while (s > 1 && items > cluster_capacity(0, s)) --s;
    return {s, 0};
}

template <int BITS, int D, int NT, bool MQ, bool WEIGHTS>
cudaError_t launch_one(const LanesPool& pool, const AttnArgs& a, cudaStream_t stream) {
    const Split s = split_for(a.batch, pool.num_kv_heads, a.max_blocks, warps_of(BITS, D, NT, 0));
    return s.wide == 2   ? launch_as<BITS, D, NT, MQ, WEIGHTS, 2>(pool, a, s.splits, stream)
           : s.wide == 1 ? launch_as<BITS, D, NT, MQ, WEIGHTS, 1>(pool, a, s.splits, stream)
                         : launch_as<BITS, D, NT, MQ, WEIGHTS, 0>(pool, a, s.splits, stream);
}

template <int BITS, bool MQ, bool WEIGHTS>
cudaError_t dispatch(const LanesPool& pool, const AttnArgs& a, int columns, cudaStream_t stream) {
    if (pool.head_dim == 128)
        return columns > 8 ? launch_one<BITS, 128, 2, MQ, WEIGHTS>(pool, a, stream)
                           : launch_one<BITS, 128, 1, MQ, WEIGHTS>(pool, a, stream);
    return columns > 8 ? launch_one<BITS, 64, 2, MQ, WEIGHTS>(pool, a, stream)
                       : launch_one<BITS, 64, 1, MQ, WEIGHTS>(pool, a, stream);
}

LanesPool lanes_pool(const Pool8View& p) {
    return {p.k, p.v, p.exps, p.num_blocks, p.num_kv_heads, p.head_dim};
}

}  // namespace

cudaError_t launch_decode8(const Pool8View& pool, const AttnArgs& a, cudaStream_t stream) {
    const int g = a.num_heads / pool.num_kv_heads;
    return a.weights ? dispatch<8, false, true>(lanes_pool(pool), a, g, stream)
                     : dispatch<8, false, false>(lanes_pool(pool), a, g, stream);
}

cudaError_t launch_decode8_mq(const Pool8View& pool, const AttnArgs& a, cudaStream_t stream) {
    return dispatch<8, true, false>(lanes_pool(pool), a, a.max_chunk * (a.num_heads / pool.num_kv_heads), stream);
}

cudaError_t launch_decode_weights(const PoolView& pool, const AttnArgs& a, cudaStream_t stream) {
    const LanesPool p = {pool.k, pool.v, nullptr, pool.num_blocks, pool.num_kv_heads, pool.head_dim};
    return dispatch<16, false, true>(p, a, a.num_heads / pool.num_kv_heads, stream);
}

}  // namespace pa
