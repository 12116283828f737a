// pa_decode_lanes.cu -- paged GQA decode with lane-private loads: over an 8-bit pool (pa_kv8.cuh:
// e4m3 codes, one power-of-two scale per block, kv head and tensor), and, over either pool,
// with the attention weight every block got added up.
//
//   o = sum_t softmax_t(scale <q, K_t>) V_t,   8-bit: K_t = codeK_t 2^kK(block), V_t = codeV_t 2^kV(block)
//
// One CTA serves one (sequence, kv head, split); its four warps, and the splits of a sequence
// (one thread-block cluster, merged through distributed shared memory), take the blocks
// round-robin, so a warp's block indices do not depend on the sequence's length.
//
// Products, 8 bits.  The codes enter the tensor core as f16, which holds every e4m3 value
// exactly, at one conversion per two codes.  K's scale joins the softmax scale (one factor
// per block and head).  q enters as f16 too, after its row is brought to a maximum in
// [2^14, 2^15) by a power of two that joins the same factor: an element loses bits only below
// 2^-29 of the row's maximum.  V's scale joins the exponent: with x = log2(e) scale <q, K> the
// weight the V product takes is u = 2^(x + kV - my), my the running maximum of x + kV, so
// u <= 1 fits f16 whatever the blocks' scales, and the largest contributions, not the largest
// probabilities, set its range.  u is rounded to f16's 11 bits (an eighth of the rounding of the
// bf16 result); the normaliser adds u 2^-kV in fp32, unrounded.
// 16 bits: the same with kK = kV = 0 on bf16 MMAs, u carried as two bf16 parts.
//
// Loads.  A thread's MMA fragments want, per 16-token block, 16-byte pieces of a few rows --
// since which d values make one MMA step is free as long as q (or the output) agrees.  So every
// lane copies (cp.async) just the pieces its own fragments take into its own 16-byte columns of
// a ring in shared memory: every byte is copied once and read once, with no bank conflict, no
// ldmatrix, and no barrier between warps or lanes, and kStages blocks a warp are in flight.
//
// Weights.  A block's sum of 2^x per head goes to a workspace as it is computed; once the
// sequence's maximum and normaliser are known (after the merge) the CTA that read the block turns
// the sums into weights, adds the group's heads in order and updates its own entry: no
// atomics, no second launch.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include <cooperative_groups.h>

#include "pa_internal.h"
#include "pa_kv8.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.44269504088896340736f;

template <int BITS, int D>
struct Lanes {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kBlockBytes = 2 * kBlockSize * kRowBytes;  // K and V of one (block, kv head)
    static constexpr int kStages = 3 * 4096 / (kBlockBytes < 4096 ? kBlockBytes : 4096);  // blocks in flight per warp
    static constexpr int kPieces = kBlockBytes / 512;               // 16-byte pieces of a block a lane takes
    static constexpr int kKChunks = kRowBytes / 64;                 // of a K row
    static constexpr int kVChunks = kRowBytes >= 128 ? kRowBytes / 128 : 1;  // of a V row (half of one at 64 bytes)
    static constexpr int kRing = kWarps * kStages * kBlockBytes;
    // merge scratch over the ring: per warp, and for the CTA, m[16], l[16], O[16][kRow]
    static constexpr int kRow = D + 4;
    static constexpr int kPart = 32 + 16 * kRow;
    static constexpr int kMerge = (kWarps + 1) * kPart * 4;
    static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
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
};

// CTAs an SM is to hold: as many as the rings leave room for, one fewer where two n-tiles need
// more than 128 registers
__host__ __device__ constexpr int resident_ctas(int bits, int d, int nt) {
    return bits == 16 ? 2 : d == 128 && nt == 2 ? 3 : 4;
}

// Where group `grp` (4 floats) of a head's row sits in the merge scratch: the lanes that write one
// instruction's groups hit different banks.
__device__ __forceinline__ int quad_at(int grp) { return grp ^ ((grp >> 2) & 1); }

template <int BITS, int D, int NT, bool MQ, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, resident_ctas(BITS, D, NT))
    decode_lanes_kernel(const __grid_constant__ LanesArgs a) {
    using Sh = Lanes<BITS, D>;
    constexpr int kSteps = D / 16;    // MMA steps over d (K), tiles of d (V)
    constexpr int kRowB = Sh::kRowBytes;
    extern __shared__ __align__(16) uint8_t smem[];

    uint32_t ncl;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncl));
    const int sub = static_cast<int>(ncl), rank = blockIdx.x % sub;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3;
    const int g = a.group;
    const int first = rank * kWarps + warp, stride = sub * kWarps;  // this warp's blocks
    const int32_t* bt = a.block_tables + (size_t)b * a.max_blocks;
    pdl_wait();

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
        return k < n ? __ldg(a.exps + (size_t)blk * a.num_kv_heads + kvh) : kExpBias * 257;
    };
    id = checked(lane, id);
    int ex = exps_of(lane, id);

    const uint32_t ring = smem_u32(smem) + warp * Sh::kStages * Sh::kBlockBytes;
    const uint32_t mine = ring + lane * 16;
    const auto issue = [&](int k, int blk) {
        const size_t tile = ((size_t)blk * a.num_kv_heads + kvh) * (kBlockSize * kRowB);
        uint32_t dst = mine + (k % Sh::kStages) * Sh::kBlockBytes;
        const uint8_t* kp = a.k + tile + gid * kRowB + tig * 16;
        const uint8_t* vp = a.v + tile + 2 * tig * kRowB + gid * (kRowB >= 128 ? 16 : 8);
#pragma unroll
        for (int r = 0; r < 2; ++r)  // rows gid, gid + 8
#pragma unroll
            for (int c = 0; c < Sh::kKChunks; ++c, dst += 512) cp_async16(dst, kp + r * 8 * kRowB + c * 64);
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
            const uint8_t* src = vp + ((r & 1) + (r >> 1) * 8) * kRowB;
            if constexpr (kRowB >= 128) {
#pragma unroll
                for (int c = 0; c < Sh::kVChunks; ++c, dst += 512) cp_async16(dst, src + c * 128);
            } else {
                cp_async8(dst + (r >> 1) * 512 + (r & 1) * 8, src);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < Sh::kStages; ++k) {
        if (k < n) issue(k, __shfl_sync(0xffffffffu, id, k));
        cp_async_commit();
    }

    // q as B fragments: column gid of each n-tile, the d values this lane's K pieces hold
    uint32_t qb[NT][kSteps][2];
    int eq[NT][2];  // exponents of this thread's output columns nt * 8 + 2 tig (+1)
    int colpos[NT][2];
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
            eq[nt][j] = __shfl_sync(0xffffffffu, e, (2 * tig + j) * 4);
            const int oc = nt * 8 + 2 * tig + j;
            colpos[nt][j] = MQ ? (oc < R ? L - C + oc / g : -1) : L - 1;
        }
    }

    float ot[NT][kSteps][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) ot[nt][s][0] = ot[nt][s][1] = ot[nt][s][2] = ot[nt][s][3] = 0.f;
    }

    int nid = 0, nex = 0;
    for (int k = 0; k < n; ++k) {
        const int at = k & 31;
        // the next 32 entries, then (once they have come) their exponents
        if (at == 0 && k + 32 + lane < n) nid = __ldg(bt + entry_at(k + 32 + lane));
        if (at == 16) {
            nid = checked(k + 16 + lane, nid);
            nex = exps_of(k + 16 + lane, nid);
        }
        cp_async_wait<Sh::kStages - 1>();
        const int e = __shfl_sync(0xffffffffu, ex, at);
        const int ek = (e & 255) - kExpBias, ev = (e >> 8) - kExpBias;
        const int kbase = static_cast<int>(entry_at(k)) * kBlockSize;
        const uint4* piece = reinterpret_cast<const uint4*>(
            smem + (warp * Sh::kStages + k % Sh::kStages) * Sh::kBlockBytes + lane * 16);

        // S^T = K q^T: rows are tokens gid, gid + 8, columns the heads
        float st[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[nt][0] = st[nt][1] = st[nt][2] = st[nt][3] = 0.f;
#pragma unroll
        for (int c = 0; c < Sh::kKChunks; ++c) {
            const uint4 p0 = piece[c * 32], p8 = piece[(Sh::kKChunks + c) * 32];
            const uint32_t w0[4] = {p0.x, p0.y, p0.z, p0.w}, w8[4] = {p8.x, p8.y, p8.z, p8.w};
            if constexpr (BITS == 8) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t a0 = e4m3x2_to_f16x2(w0[s] & 0xffffu), a2 = e4m3x2_to_f16x2(w0[s] >> 16);
                    const uint32_t a1 = e4m3x2_to_f16x2(w8[s] & 0xffffu), a3 = e4m3x2_to_f16x2(w8[s] >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(st[nt], a0, a1, a2, a3, qb[nt][c * 4 + s][0], qb[nt][c * 4 + s][1]);
                }
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816(st[nt], w0[2 * s], w8[2 * s], w0[2 * s + 1], w8[2 * s + 1], qb[nt][c * 2 + s][0],
                                  qb[nt][c * 2 + s][1]);
            }
        }
        uint32_t pb[NT][2], pl[NT][2];
        const float unscale = exp2_int(-ev), fev = static_cast<float>(ev);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float u[2][2];  // [column][token gid, gid + 8]
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float f = a.scale_log2 * exp2_int(eq[nt][j] + ek);
                const int lim = colpos[nt][j] - kbase;  // keys up to this one of the block are visible
                const bool v0 = gid <= lim, v8 = gid + 8 <= lim;
                const float x0 = st[nt][j] * f, x8 = st[nt][2 + j] * f;
                float mx = fmaxf(v0 ? x0 : -INFINITY, v8 ? x8 : -INFINITY);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nt][j], mx + fev);
                const float base = mn == -INFINITY ? 0.f : mn;  // nothing visible so far
                alpha[j] = fast_exp2(m[nt][j] - base);
                m[nt][j] = mn;
                const float off = fev - base;
                u[j][0] = v0 ? fast_exp2(fmaf(st[nt][j], f, off)) : 0.f;
                u[j][1] = v8 ? fast_exp2(fmaf(st[nt][2 + j], f, off)) : 0.f;
                float sum = (u[j][0] + u[j][1]) * unscale;
                l[nt][j] = l[nt][j] * alpha[j] + sum;
                if (WEIGHTS) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    if (gid == j)
                        a.ws[(((size_t)b * a.num_kv_heads + kvh) * a.max_blocks + entry_at(k)) * (8 * NT) + nt * 8 +
                             2 * tig + j] = sum > 0.f ? log2f(sum) + base : -INFINITY;
                }
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                ot[nt][s][0] *= alpha[0];
                ot[nt][s][2] *= alpha[0];
                ot[nt][s][1] *= alpha[1];
                ot[nt][s][3] *= alpha[1];
            }
            // rows (tokens) x columns (heads) -> transposed: the B operand of the V product
            if constexpr (BITS == 8) {
                pb[nt][0] = movmatrix_t(pack_f16x2(u[0][0], u[1][0]));
                pb[nt][1] = movmatrix_t(pack_f16x2(u[0][1], u[1][1]));
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = pack_bf16x2(u[0][i], u[1][i]);
                    pb[nt][i] = movmatrix_t(hi);
                    pl[nt][i] = movmatrix_t(pack_bf16x2(u[0][i] - bf16_lo(hi), u[1][i] - bf16_hi(hi)));
                }
            }
        }
        // O^T += V^T u^T: keys 2 tig, 2 tig + 1 (+8); tile rows gid, gid + 8 are neighbouring d
        constexpr int kVWords = kRowB / 32;  // of each of the lane's four V rows
        uint32_t vw[4][kVWords];
        if constexpr (kRowB >= 128) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < Sh::kVChunks; ++c) {
                    const uint4 p = piece[(2 * Sh::kKChunks + r * Sh::kVChunks + c) * 32];
                    vw[r][4 * c] = p.x;
                    vw[r][4 * c + 1] = p.y;
                    vw[r][4 * c + 2] = p.z;
                    vw[r][4 * c + 3] = p.w;
                }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 p = piece[(2 * Sh::kKChunks + r) * 32];
                vw[2 * r][0] = p.x;
                vw[2 * r][1] = p.y;
                vw[2 * r + 1][0] = p.z;
                vw[2 * r + 1][1] = p.w;
            }
        }
        if (kbase + kBlockSize > L) {
            // rows past the sequence's end: whatever they hold (NaN times u = 0 is NaN)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (kbase + 2 * tig + (r & 1) + (r >> 1) * 8 >= L) {
#pragma unroll
                    for (int w = 0; w < kVWords; ++w) vw[r][w] = 0u;
                }
        }
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
            if constexpr (BITS == 8) {
                // codes of d, d+1 (then d+2, d+3) paired over keys 2 tig, 2 tig + 1 and over the next 8
                const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], 0x5140);
                const uint32_t hi = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                const uint32_t lo8 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
                const uint32_t hi8 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xffffu), a1 = e4m3x2_to_f16x2(lo >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(lo8 & 0xffffu), a3 = e4m3x2_to_f16x2(lo8 >> 16);
                const uint32_t c0 = e4m3x2_to_f16x2(hi & 0xffffu), c1 = e4m3x2_to_f16x2(hi >> 16);
                const uint32_t c2 = e4m3x2_to_f16x2(hi8 & 0xffffu), c3 = e4m3x2_to_f16x2(hi8 >> 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16_16816(ot[nt][2 * w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_f16_16816(ot[nt][2 * w + 1], c0, c1, c2, c3, pb[nt][0], pb[nt][1]);
                }
            } else {
                const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410);
                const uint32_t a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410);
                const uint32_t a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(ot[nt][w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_16816(ot[nt][w], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                }
            }
        }
        // refill the slot just read
        if (at == 31) {  // on to the next 32 blocks
            id = nid;
            ex = nex;
        }
        const int next = k + Sh::kStages;
        if (next < n) {
            // its id is among the current 32, or (its entries not yet moved up) among the next
            const bool ahead = (next >> 5) != ((k + 1) >> 5);
            issue(next, __shfl_sync(0xffffffffu, ahead ? nid : id, next & 31));
        }
        cp_async_commit();
    }
    cp_async_wait<0>();
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
                    pm[col] = m[nt][j];
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
            const float wt = pm[col] == -INFINITY ? 0.f : fast_exp2(pm[col] - M);
            const float4 v = *reinterpret_cast<const float4*>(pm + 32 + col * Sh::kRow + 4 * quad_at(grp));
            acc.x += wt * v.x;
            acc.y += wt * v.y;
            acc.z += wt * v.z;
            acc.w += wt * v.w;
            den += wt * pm[16 + col];
        }
        if (sub == 1) store(qd, acc, den > 0.f ? 1.f / den : 0.f);
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
                const float w = mr == -INFINITY ? 0.f : fast_exp2(mr - M);
                wgt[r * 16 + col] = w;
                den += w * lsum[r * 16 + col];
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
            store(qd, acc, col_l[col] > 0.f ? 1.f / col_l[col] : 0.f);
        }
    }
    if (WEIGHTS) {
        // this CTA's blocks: the columns' shares of the whole sequence's weight, added up
        const int own = nb > rank * kWarps ? nb - rank * kWarps : 0;
        for (int t = threadIdx.x; t < (own + stride - 1) / stride * kWarps; t += kThreads) {
            const int blk = rank * kWarps + t % kWarps + t / kWarps * stride;
            if (blk >= nb) continue;
            const float* lb = a.ws + (((size_t)b * a.num_kv_heads + kvh) * a.max_blocks + blk) * (8 * NT);
            float sum = 0.f;
            for (int col = 0; col < R; ++col) {
                const float den = col_l[col];
                if (den > 0.f) sum += fast_exp2(lb[col] - col_m[col]) / den;
            }
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

template <int BITS, int D, int NT, bool MQ, bool WEIGHTS>
cudaError_t launch_one(const LanesPool& pool, const AttnArgs& a, int splits, cudaStream_t stream) {
    using Sh = Lanes<BITS, D>;
    auto kern = decode_lanes_kernel<BITS, D, NT, MQ, WEIGHTS>;
    static OncePerDevice configured;  // per instantiation
    cudaError_t se = configured.run([&] {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, pool.num_kv_heads, a.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
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
    return cudaLaunchKernelEx(&cfg, kern, d);
}

template <int BITS, bool MQ, bool WEIGHTS>
cudaError_t dispatch(const LanesPool& pool, const AttnArgs& a, int columns, cudaStream_t stream) {
    const int splits = decode_splits_for(a.batch, pool.num_kv_heads, a.max_blocks);
    if (pool.head_dim == 128)
        return columns > 8 ? launch_one<BITS, 128, 2, MQ, WEIGHTS>(pool, a, splits, stream)
                           : launch_one<BITS, 128, 1, MQ, WEIGHTS>(pool, a, splits, stream);
    return columns > 8 ? launch_one<BITS, 64, 2, MQ, WEIGHTS>(pool, a, splits, stream)
                       : launch_one<BITS, 64, 1, MQ, WEIGHTS>(pool, a, splits, stream);
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
