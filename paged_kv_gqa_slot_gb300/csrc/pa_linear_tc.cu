// pa_linear_tc.cu -- linear attention over chunks of tokens (pa_linear_prefill) on the 5th-generation
// tensor cores.
//
// The recurrence S_t = a S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t, taken 128 tokens at a time.  With S the
// state before a chunk of n tokens and i, j its rows,
//   o_i = scale ( sum_{j <= i} a^{i-j} <q_i, k_j> v_j  +  a^{i+1} q_i^T S )
//   S'  = a^n S + sum_j (a^{n-1-j} k_j) v_j^T
// that is four products on the tensor core: Q K^T, P V (P the weighted, masked scores), Q S and K~^T V
// (K~ the weighted keys).  The powers enter as 2^{(i-j) log2 a} <= 1, so nothing overflows however
// strong the decay.
//
// Rounding.  P and S enter their products as bf16, one rounding of every term, as the outputs are bf16.  What is
// added to S stays there, so K~ enters as three bf16 parts, all 24 bits of it; and since the tensor core cuts its
// sums off instead of rounding them, K~^T V is summed from zero in every chunk, the small parts first, and added to
// a^n S by the threads in fp32.  The state is then within 2.5e-7 of 64 bits (two parts 2.4e-6; three, added to S by the
// tensor core, 1.0e-6: 24 sequences of up to 1100 tokens, 16 heads).  Where nothing decays and all terms have one sign it
// is within 9.3e-7 after 2^20 tokens, 8192 sums of fp32 later, with a mean error of 1e-9.
//
// What bounds it.  A token moves (2 heads + 2 kv heads) d 2 bytes; per SM and 128 tokens of one head that is
// 128 KB, about 5900 cycles of HBM time at d = 128, against 2800 of tensor core and 5000 of shared-memory
// bandwidth (the operands of the products, the copies, K~ and S).  A chunk takes 6300: shared memory, and the
// chain K~^T V, S, Q K^T, K~, which leaves the copies little slack; and items run in the caller's order, so that the
// longest may begin last (24 ragged: by a replay of the listed lengths about a quarter).  152 states x 1024 tokens
// 38.0 us (4.7 TB/s); 24 sequences of up to 1100 tokens, 16 heads, 77.5; 1 x 20000 tokens, 32 heads, 213.  At d = 64 25,
// 41 and 143.
//
// S stays in tensor memory in fp32 (lane: row of k, column: column of v).  Each chunk it is read once with the
// sums of the chunk before, and written back there and to shared memory as bf16.  Q S is read back, weighted by
// a^{i+1}, and P V added to it, which leaves room for the sums of K~^T V.
//
// Masked rows of P are zero, and 0 times a NaN or an infinity in V is NaN: V is looked over when it
// arrives, what is not finite becomes 0, and the first token it was seen at is noted per column; from
// that row on the column is NaN, and so is the state's.
//
// Few sequences leave most SMs idle, so a long one is cut into segments: first every segment but the last
// gathers what its own tokens add to the state (K~^T V alone, weighted to the segment's end), then one pass
// over the states turns these into what each segment begins with, and then all segments run at once.  It
// costs a second read of K and V (1 x 20000 tokens, 32 heads, whole: 500 us).
//
// An item is one (segment, sequence, kv head).  A CTA, one an SM, takes item after item: near the end of
// one it asks for a block of the grid that has not started (clusterlaunchcontrol), so that the
// copies of the next item run under the end of this one.  Warps: 0-3 P and the outputs (one row a
// thread), 4-7 the state (one row a thread), 4-11 K~, 12 MMA issue and tensor memory, 13 TMA loads of K and
// V, 14 of Q (one thread issues a copy in about half a microsecond), 15 the look at V, 16 the items.
// (K~ by warps 8-11 alone: 1 x 20000 218 us.  Copies sent to L2 a chunk ahead: 24 sequences 83 us against 80.)
// The loops over column blocks are not unrolled and rare paths are short: the roles run at the same time, and
// their code has to fit the instruction cache together (152 states x 1024 tokens took 52 us unrolled, 36 rolled up).
#include <algorithm>
#include <climits>

#include "pa_internal.h"
#include "pa_step.cuh"

namespace pa {
namespace {

constexpr int kChunk = 128;
constexpr int kThreads = 544;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kQLoadWarp = 14, kCleanWarp = 15, kItemWarp = 16;
constexpr int kHalf = kChunk * 128;  // [128 rows][64 columns] bf16

// One item: what its roles need.  chunks < 0: there is none, the CTA is done; 0: padding, zero rows.
struct Item {
    const float* begin;  // the state it begins with (null: zero)
    float* end;          // where its last state goes (null: nowhere)
    int row, len, chunks, kvh;
    float ld, la;        // the log decay, natural and to base 2
    int any_bad;         // a value of V was not finite
};

template <int D, bool kGather>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalf;
    // K~ is written and multiplied in pieces, as shared memory has no room for all of its middle and low parts beside
    // the rest (it has where nothing else is needed).  With V in one tile instead 1 x 20000 tokens take 232 us against
    // 221, with the low parts over S 230.
    static constexpr int kPieces = kGather ? 1 : 2;
    static constexpr int kRows = kChunk / kPieces;
    static constexpr int kPart = kRows * 128;              // [rows of a piece][64 columns] of the middle or low parts
    static constexpr int kOffK = 0;                        // two tiles; each becomes the high parts of K~ in place
    static constexpr int kOffMid = kOffK + 2 * kTile;
    static constexpr int kOffLow = kOffMid + kHalves * kPart;
    static constexpr int kOffV = kOffLow + kHalves * kPart;  // two tiles
    static constexpr int kOffQ = kOffV + 2 * kTile;
    static constexpr int kOffS = kOffQ + (kGather ? 0 : kTile);  // the state, bf16, D rows
    static constexpr int kOffBars = kOffS + (kGather ? 0 : D * 128 * kHalves);
    static constexpr int kOffItem = kOffBars + 384;    // two items
    static constexpr int kOffTab = kOffItem + 128;     // [2][32] a^31 .. a^0
    static constexpr int kOffBad = kOffTab + 256;      // [2][D] first token of a column with a value that is not finite
    static constexpr int kSmem = kOffBad + 2 * D * 4;
    // tensor memory: scores and P; the outputs; K~^T V; the state
    static constexpr uint32_t kColP = 0, kColO = 128, kColU = kColO + D, kColS = kColU + D;
    // gather: K~^T V of the high parts, by turns; what they add up to; K~^T V of the other parts
    static constexpr uint32_t kColHigh[2] = {0, 128}, kColSum = 128 + D, kColSmall = kColSum + D;
    static constexpr int kTmemCols = 512;
};
static_assert(Layout<128, false>::kSmem <= 227 * 1024, "shared memory");
static_assert(sizeof(Item) <= 64, "item");

// A barrier is waited for by the parity of its phase, so a phase may be over only once all who wait for the one before
// have seen that.  Each has behind it, therefore, something that they do after their wait:
//   k_full, v_full        the tile is loaded again after k_empty, v_empty: commits of the products that take K~ and V, issued
//                         after kt_full (which all who wait for k_full or k_raw arrive on) and v_clean
//   q_full, q_empty       one another: a copy, then the commit of the product that reads it
//   s_full, qs_full, o_full  committed after p_full of the head before, or of this one, which those who wait arrive on
//   p_full, o_empty       arrived on after s_full and o_full of the same head, committed by the warp that waits
//   k_raw, piece          committed by the warp that has waited for kt_full, which those who wait for them arrive on
//   kt_full, st_full      arrived on after k_raw, piece and u_full, committed by the warp that waits for these two
//   u_full                committed after st_full of its chunk (gather: of its item)
//   item_full, item_empty, soon, next  one another: two items, and a block is asked for after soon of the item before
// So it is safe that the first piece of K~ is written while Q S runs and the second while P V runs.
struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_clean[2], q_full, q_empty;
    uint64_t s_full, qs_full, p_full, o_full, o_empty;  // scores, Q S, P with Q S weighted, outputs ready; outputs read
    uint64_t k_raw, piece;                     // K may become K~: Q K^T of the chunk is done (gather: K~^T V of the
                                               // chunk before); K~^T V of its first piece is done
    uint64_t kt_full, st_full, u_full;         // a piece of K~ ready; the state ready for the chunk; K~^T V done
    uint64_t item_full[2], item_empty[2], soon, next, drain;
    uint4 reply;                               // of clusterlaunchcontrol
    uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 384, "barrier block");

struct TcArgs {
    LinearArgs l;
    float* segments;   // [batch][segs][kv heads][D][D]: what the segment before adds, then what this one begins with
    int group, segs, seg_chunks;
    float scale;
};

// Sequence b's rows; len 0: nothing to do.
struct Rows {
    int row, len, slot;
    bool fresh, bad;
};
__device__ __forceinline__ Rows rows_of(const LinearArgs& l, int b) {
    const PackedArgs& p = l.rows;
    const int c0 = p.cu_lens[b], c1 = p.cu_lens[b + 1], total = l.seq_lens[b];
    Rows r;
    r.slot = l.state_slots[b];
    r.row = c0;
    r.bad = c0 < 0 || c1 < c0 || c1 > p.num_tokens || total < c1 - c0;
    r.len = r.bad ? 0 : min(c1 - c0, p.max_len);
    r.fresh = total == c1 - c0;
    r.bad |= r.len > 0 && (c1 - c0 > p.max_len || r.slot >= l.num_slots);
    return r;
}
// d = (a0 * b0, a1 * b1), each rounded to nearest even
__device__ __forceinline__ void mul_x2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The items as one warp sees them, in order; next() waits for one and done() gives it back.
struct Items {
    Bars* bars;
    uint8_t* slots;
    int n = 0;
    __device__ __forceinline__ Item* next(bool& ok) {
        ok = __all_sync(0xffffffffu, ok);
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->item_full[n & 1], (n >> 1) & 1));
        Item* it = reinterpret_cast<Item*>(slots + (n & 1) * 64);
        return ok && it->chunks >= 0 ? it : nullptr;
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->item_empty[n & 1]);
        ++n;
    }
};

// kGather: only what the tokens of a segment add to the state (K~^T V), into a.segments.
template <int D, bool kGather>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                             const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const __grid_constant__ TcArgs a) {
    using L = Layout<D, kGather>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kOffBars);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, r = threadIdx.x & 127;
    const PackedArgs& p = a.l.rows;
    const int g = a.group;
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need the declared alignment
        if (threadIdx.x == 0) atomicOr(p.status, kDevOutOfRange);
        return;
    }
    if (threadIdx.x == kItemWarp * 32) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 1);
            mbar_init(&bars->v_clean[s], 32);
            mbar_init(&bars->item_full[s], 32);
            mbar_init(&bars->item_empty[s], kItemWarp);  // every other warp
        }
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->qs_full, 1);
        mbar_init(&bars->p_full, 128);
        mbar_init(&bars->o_full, 1);
        mbar_init(&bars->o_empty, 128);
        mbar_init(&bars->k_raw, 1);
        mbar_init(&bars->piece, 1);
        mbar_init(&bars->kt_full, 256);
        mbar_init(&bars->st_full, 128);
        mbar_init(&bars->u_full, 1);
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
    Items items{bars, smem + L::kOffItem};

    if (warp == kItemWarp) {
        // ---------------------------------------------------------------- the items
        // id = (segment * batch + b) * kv heads + kv head
        unsigned id = blockIdx.x;
        uint32_t phase = 0;
        for (int n = 0; ok; ++n) {
            bool there = true;
            if (n > 0) {  // the last copies of the item before are on their way, and a slot is free
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->soon, (n - 1) & 1));
                if (ok && n > 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars->item_empty[n & 1], ((n >> 1) & 1) ^ 1));
                if (ok) there = take_block(&bars->reply, &bars->next, phase, id, ok);
            }
            Item it = {nullptr, nullptr, 0, 0, -1, 0, 0.f, 0.f, 0};
            while (ok && there) {
                const int kvh = (int)(id % (unsigned)p.num_kv_heads), sb = (int)(id / (unsigned)p.num_kv_heads);
                const int b = sb % p.batch, seg = sb / p.batch;
                const Rows w = rows_of(a.l, b);
                if (!kGather && w.bad && kvh == 0 && seg == 0 && lane == 0) atomicOr(p.status, kDevOutOfRange);
                const int all = (w.len + kChunk - 1) / kChunk, first = seg * a.seg_chunks;
                const bool pad = w.slot < 0 || w.slot >= a.l.num_slots;
                const int chunks = min(a.seg_chunks, all - first);
                const bool last = first + chunks >= all;
                if (chunks > 0 && !(kGather && (last || pad))) {
                    const size_t dd = (size_t)D * D;
                    it.row = w.row + first * kChunk;
                    it.len = min(w.len - first * kChunk, chunks * kChunk);
                    it.chunks = pad ? 0 : chunks;
                    it.kvh = kvh;
                    it.ld = in_range(a.l.log_decay[kvh]);
                    it.la = it.ld * kLog2e;
                    if (!pad) {
                        float* state = a.l.state + ((size_t)w.slot * p.num_kv_heads + kvh) * dd;
                        // (the first of several segments begins with a copy: the last may end before it starts)
                        float* own = a.segments + (((size_t)b * a.segs + seg) * p.num_kv_heads + kvh) * dd;
                        if (kGather) {
                            it.end = own + (size_t)p.num_kv_heads * dd;  // for the next one
                        } else {
                            it.begin = seg == 0 && w.fresh ? nullptr : seg == 0 && last ? state : own;
                            it.end = last ? state : nullptr;
                            if (it.begin)
                                for (int i = lane * 128; i < D * D * 4; i += 32 * 128)
                                    prefetch_l2(reinterpret_cast<const char*>(it.begin) + i);
                        }
                    }
                    break;
                }
                there = take_block(&bars->reply, &bars->next, phase, id, ok);
            }
            if (!ok) break;
            if (lane == 0) *reinterpret_cast<Item*>(smem + L::kOffItem + (n & 1) * 64) = it;
            if (!kGather && there) {
                reinterpret_cast<float*>(smem + L::kOffTab)[(n & 1) * 32 + lane] =
                    fast_exp2((float)(31 - lane) * it.la);
                for (int i = lane; i < D; i += 32) reinterpret_cast<int*>(smem + L::kOffBad)[(n & 1) * D + i] = INT_MAX;
            }
            __syncwarp();
            mbar_arrive(&bars->item_full[n & 1]);
            if (!there) break;
        }
    } else if (warp == kLoadWarp) {
        // ---------------------------------------------------------------- TMA loads of K and V
        int kc = 0, vc = 0;  // copies issued
        for (const Item* it; (it = items.next(ok)); items.done()) {
            if (lane == 0) {
                const int row = it->row, kvh = it->kvh, chunks = it->chunks;
                for (int c = 0; c < chunks && ok; ++c) {
                    if (kc >= 2) ok = mbar_wait(&bars->k_empty[kc & 1], ((kc >> 1) & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars->k_full[kc & 1], L::kTile);
                    tma_load_rows(smem + L::kOffK + (kc & 1) * L::kTile, &tm_k, kvh, row + c * kChunk, 0,
                                  &bars->k_full[kc & 1]);
                    ++kc;
                    if (vc >= 2) ok = mbar_wait(&bars->v_empty[vc & 1], ((vc >> 1) & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars->v_full[vc & 1], L::kTile);
                    tma_load_rows(smem + L::kOffV + (vc & 1) * L::kTile, &tm_v, kvh, row + c * kChunk, 0,
                                  &bars->v_full[vc & 1]);
                    ++vc;
                }
                mbar_arrive(&bars->soon);
            }
            __syncwarp();
        }
        if (lane == 0) {  // before the CTA may leave: every copy issued here has landed
            for (int i = max(0, kc - 2); i < kc; ++i)
                if (!mbar_wait(&bars->k_full[i & 1], (i >> 1) & 1)) ok = false;
            for (int i = max(0, vc - 2); i < vc; ++i)
                if (!mbar_wait(&bars->v_full[i & 1], (i >> 1) & 1)) ok = false;
        }
    } else if (warp == kQLoadWarp) {
        // ---------------------------------------------------------------- TMA loads of Q
        int qc = 0;
        for (const Item* it; (it = items.next(ok)); items.done()) {
            if (!kGather && lane == 0) {
                const int row = it->row, kvh = it->kvh, chunks = it->chunks;
                for (int c = 0; c < chunks && ok; ++c) {
                    for (int h = 0; h < g; ++h) {
                        if (qc > 0) ok = mbar_wait(&bars->q_empty, (qc & 1) ^ 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars->q_full, L::kTile);
                        tma_load_rows(smem + L::kOffQ, &tm_q, kvh * g + h, row + c * kChunk, 0, &bars->q_full);
                        ++qc;
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0 && qc && !mbar_wait(&bars->q_full, (qc - 1) & 1)) ok = false;
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
        const uint64_t md = smem_desc_sw128(smem_u32(smem + L::kOffMid), L::kPart, 1024);
        const uint64_t ld = smem_desc_sw128(smem_u32(smem + L::kOffLow), L::kPart, 1024);
        int cc = 0, ii = 0;  // chunks and chunks' heads so far
        // K~^T V over a piece of K~, V from where its chunk's tiles begin; `first`: from zero.  The small parts come
        // first, or into sums of their own: the tensor core cuts every sum off to 24 bits.  (So the high parts are summed
        // over one chunk at most, also where a segment is gathered; what is cut off the small ones is 2^-8 of that.)
        auto issue_u = [&](int piece, uint64_t hd, uint64_t vd, bool first) {
            const uint32_t small = tmem + (kGather ? L::kColSmall : L::kColU);
            const uint32_t high = tmem + (kGather ? (cc & 1) * L::kColHigh[1] : L::kColU);
#pragma unroll
            for (int part = 0; part < 3; ++part) {
#pragma unroll
                for (int kk = 0; kk < L::kRows / 16; ++kk) {
                    const uint64_t off = (uint64_t)((kk * 16 * 128) >> 4);
                    const uint64_t all = off + (uint64_t)((piece * L::kPart) >> 4);
                    const uint64_t from = part == 0 ? ld + off : part == 1 ? md + off : hd + all;
                    const bool zero = kk == 0 && ((first && part == 0) || (kGather && part == 2));
                    tc_mma_ew(part == 2 ? high : small, from, vd + all, idesc_u, zero ? 0u : 1u);
                }
            }
        };
        for (const Item* it; (it = items.next(ok)); items.done()) {
            // (uniform, and with it all that is counted here)
            const int chunks = __shfl_sync(0xffffffffu, it->chunks, 0);
            for (int c = 0; c < chunks && ok; ++c, ++cc) {
                const uint64_t slot = (uint64_t)(((cc & 1) * L::kTile) >> 4), vd = vd0 + slot;
                if (!kGather) {
                    ok = mbar_wait_warp(&bars->k_full[cc & 1], (cc >> 1) & 1);
                    for (int h = 0; h < g && ok; ++h, ++ii) {
                        ok = mbar_wait_warp(&bars->q_full, ii & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                            tc_mma_ew(tmem + L::kColP, qd + off, kd0 + slot + off, idesc_s, kk > 0 ? 1u : 0u);
                        }
                        tc_commit_ew(&bars->s_full);
                        if (h == g - 1) tc_commit_ew(&bars->k_raw);
                        // Q S, once the state is in shared memory (and K~^T V before has been read), and the
                        // outputs before have been read
                        if (h == 0) ok = mbar_wait_warp(&bars->st_full, cc & 1);
                        if (ok && ii > 0) ok = mbar_wait_warp(&bars->o_empty, (ii - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_ew(tmem + L::kColO, qd + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                                      sd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, kk > 0 ? 1u : 0u);
                        tc_commit_ew(&bars->qs_full);
                        tc_commit_ew(&bars->q_empty);
                        if (h == 0) ok = mbar_wait_warp(&bars->v_clean[cc & 1], (cc >> 1) & 1);
                        if (h == g - 1) {  // the first piece of K~, and the second is written under P V
                            if (ok) ok = mbar_wait_warp(&bars->kt_full, 0);
                            if (!ok) break;
                            tc_fence_after();
                            issue_u(0, hd0 + slot, vd, true);
                            tc_commit_ew(&bars->piece);
                        }
                        if (ok) ok = mbar_wait_warp(&bars->p_full, ii & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < kChunk / 16; ++kk)
                            tc_mma_ts_ew(tmem + L::kColO, tmem + L::kColP + kk * 8,
                                         vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, 1u);
                        tc_commit_ew(&bars->o_full);
                    }
                } else {
                    if (c == 0) ok = mbar_wait_warp(&bars->st_full, items.n & 1);  // the item before has been read
                    if (ok) ok = mbar_wait_warp(&bars->v_full[cc & 1], (cc >> 1) & 1);
                }
                if (ok) ok = mbar_wait_warp(&bars->kt_full, kGather ? cc & 1 : 1);
                if (!ok) break;
                tc_fence_after();
                issue_u(L::kPieces - 1, hd0 + slot, vd, kGather && c == 0);
                if (!kGather || c + 1 == chunks) tc_commit_ew(&bars->u_full);
                if (kGather) tc_commit_ew(&bars->k_raw);
                tc_commit_ew(&bars->k_empty[cc & 1]);
                tc_commit_ew(&bars->v_empty[cc & 1]);
            }
        }
        // every MMA this warp issued has finished before the tensor memory is released
        tc_commit_ew(&bars->drain);
        if (!mbar_wait_warp(&bars->drain, 0)) ok = false;
    } else if (warp == kCleanWarp) {
        // ---------------------------------------------------------------- V looked over
        // (a segment that is gathered has no row of others, and its NaN belong into what it adds)
        int cc = 0;
        for (Item* it; (it = items.next(ok)); items.done()) {
            const int chunks = kGather ? 0 : it->chunks, len = it->len;
            int* bad = reinterpret_cast<int*>(smem + L::kOffBad) + (items.n & 1) * D;
            for (int c = 0; c < chunks && ok; ++c, ++cc) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[cc & 1], (cc >> 1) & 1));
                if (!ok) break;
                uint8_t* tile = smem + L::kOffV + (cc & 1) * L::kTile;
                // a pass that only reads (its loads run ahead), and only where something was found the repair
                uint32_t seen = 0;
#pragma unroll 8
                for (int i = lane; i < L::kTile / 16; i += 32)
                    seen |= not_finite(*reinterpret_cast<const uint4*>(tile + 16 * i));
                if (seen) {
#pragma unroll 1
                    for (int i = lane; i < L::kTile / 16; i += 32) {
                        const int half = i / (kHalf / 16), row = i / 8 % kChunk;
                        const int col = half * 64 + ((i & 7) ^ (row & 7)) * 8, t = c * kChunk + row;
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            uint16_t* x = reinterpret_cast<uint16_t*>(tile + 16 * i) + e;
                            if ((*x & 0x7f80u) != 0x7f80u) continue;
                            if (t < len) {
                                atomicMin(&bad[col + e], t);
                                it->any_bad = 1;
                            }
                            *x = 0;
                        }
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive(&bars->v_clean[cc & 1]);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------- the state (warps 4-7, row r of S), K weighted
        const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool mine = r < D;
        uint8_t* ss = smem + L::kOffS + r * 128;
        const bool keeps = warp < 8;
        int cc = 0, uc = 0;  // chunks; completed K~^T V that the state has waited for
        // S (at s_at) and K~^T V (at u_at), columns x .. x + 31
        auto both = [&](uint32_t (&s)[32], uint32_t (&u)[32], int x, uint32_t s_at, uint32_t u_at) {
            tmem_ld32_async(tm + s_at + x, s);
            tmem_ld32_async(tm + u_at + x, u);
            tmem_wait_ld(s);
            tmem_wait_ld(u);
        };
        auto sum = [&](uint32_t (&s)[32], int x, uint32_t s_at, uint32_t u_at) {  // S <- S + K~^T V
            uint32_t u[32];
            both(s, u, x, s_at, u_at);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) + __uint_as_float(u[e]));
        };
        auto step = [&](uint32_t (&s)[32], int x, const Decay& f) {  // S <- f S + K~^T V
            uint32_t u[32];
            both(s, u, x, L::kColS, L::kColU);
            if (f.near) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float s0 = __uint_as_float(s[e]), s1 = __uint_as_float(s[e + 1]), y0, y1;
                    fma_x2(y0, y1, s0, s1, f.x, f.x, __uint_as_float(u[e]), __uint_as_float(u[e + 1]));
                    add_x2(s0, s1, y0, y1);
                    s[e] = __float_as_uint(s0);
                    s[e + 1] = __float_as_uint(s1);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    s[e] = __float_as_uint(fmaf(__uint_as_float(s[e]), f.x, __uint_as_float(u[e])));
            }
        };
        for (const Item* it; (it = items.next(ok)); items.done()) {
            const int chunks = it->chunks, len = it->len;
            const float la = it->la;
            Decay f(0.f, 0.f);  // over the chunk before
            if (kGather && keeps) {
                tc_fence_before();
                mbar_arrive(&bars->st_full);
            }
            for (int c = 0; c < chunks && ok; ++c, ++cc) {
                if (!kGather && keeps) {
                    const float* from = it->begin;
                    if (c > 0) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_full, uc & 1));
                        ++uc;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    auto take = [&](uint32_t (&s)[32], int x) {  // kept, and as bf16 for Q S
                        tmem_st32_nowait(tm + L::kColS + x, s);
                        if (!mine) return;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                w[q] = pack_bf16x2(__uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1]));
                            const int chunk = (x + e) >> 3;
                            *reinterpret_cast<uint4*>(ss + (chunk >> 3) * (D * 128) + (((chunk & 7) ^ (r & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    };
                    if (c > 0) {
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            uint32_t s[32];
                            step(s, x, f);
                            take(s, x);
                        }
                    } else {
                        const bool there = mine && from;
                        const float* row = from + (size_t)r * D;
                        const bool wide = (reinterpret_cast<uintptr_t>(from) & 31u) == 0;
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            uint32_t s[32];
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                if (there)
                                    load_32(row + x + e, s + e, wide);
                                else
#pragma unroll
                                    for (int i = 0; i < 8; ++i) s[e + i] = 0u;
                            }
                            take(s, x);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    fence_proxy_async_smem();
                    mbar_arrive(&bars->st_full);
                    if (c == 0 || len - c * kChunk < kChunk) f = Decay(it->ld, (float)min(kChunk, len - c * kChunk));
                }
                const int n = min(kChunk, len - c * kChunk);
                // weighted to the end of the chunk, or of the segment
                const int left = kGather ? len - c * kChunk : n;
                // a thread: of a row of the piece kParts of its 16-byte parts, kStep loads in flight together
                constexpr int kParts = D / 8 * L::kRows / 256, kStep = kParts < 4 ? kParts : 4;
                const int at_k = keeps ? 128 + r : r, pr = at_k & (L::kRows - 1), first = at_k / L::kRows * kParts;
#pragma unroll 1
                for (int piece = 0; piece < L::kPieces && ok; ++piece) {
                    if (kGather) {
                        // Not before the products of the chunk before are done.  kt_full is waited for by parity, and K
                        // has two tiles: without this wait both could be weighted, and two phases of kt_full be over,
                        // while the issuing warp still waited for a V that came late; it then waited for a phase that its
                        // own commits had to bring about.  (An earlier form, with room for the low parts of both tiles,
                        // did so for about one chunk in 10^5, until the waits ran out.  In turn is faster, too.)
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_full[cc & 1], (cc >> 1) & 1));
                        if (ok && cc > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_raw, (cc - 1) & 1));
                    } else {  // (the first: it also means that the products of the chunk before are done)
                        ok = __all_sync(0xffffffffu, mbar_wait(piece ? &bars->piece : &bars->k_raw, cc & 1));
                    }
                    if (!ok) break;
                    const int row = piece * L::kRows + pr;
                    const float w = row < n ? fast_exp2((float)(left - 1 - row) * la) : 0.f;
                    uint8_t* hi = smem + L::kOffK + (cc & 1) * L::kTile + row * 128;
                    uint8_t* mid = smem + L::kOffMid + pr * 128;
                    uint8_t* low = smem + L::kOffLow + pr * 128;
#pragma unroll 1
                    for (int i0 = first; i0 < first + kParts; i0 += kStep) {
                        uint4 in[kStep];
                        const int half = i0 >> 3;
#pragma unroll
                        for (int i = 0; i < kStep; ++i)
                            in[i] = row < n ? *reinterpret_cast<const uint4*>(
                                                  hi + half * kHalf + ((((i0 & 7) + i) ^ (row & 7)) << 4))
                                            : make_uint4(0u, 0u, 0u, 0u);  // not the sequence's own
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            const int at = (((i0 & 7) + i) ^ (row & 7)) << 4;
                            uint32_t x[4] = {in[i].x, in[i].y, in[i].z, in[i].w}, m[4], l[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {  // (the differences are exact)
                                float f0, f1;
                                mul_x2(f0, f1, bf16_lo(x[e]), bf16_hi(x[e]), w, w);
                                x[e] = pack_bf16x2(f0, f1);
                                f0 -= bf16_lo(x[e]);
                                f1 -= bf16_hi(x[e]);
                                m[e] = pack_bf16x2(f0, f1);
                                l[e] = pack_bf16x2(f0 - bf16_lo(m[e]), f1 - bf16_hi(m[e]));
                            }
                            *reinterpret_cast<uint4*>(hi + half * kHalf + at) = make_uint4(x[0], x[1], x[2], x[3]);
                            *reinterpret_cast<uint4*>(mid + half * L::kPart + at) = make_uint4(m[0], m[1], m[2], m[3]);
                            *reinterpret_cast<uint4*>(low + half * L::kPart + at) = make_uint4(l[0], l[1], l[2], l[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&bars->kt_full);
                }
                if (kGather && keeps && c > 0 && ok) {
                    // The high parts of the chunk before, whose products are done, to the others, in fp32, while those of
                    // this chunk run into the other columns.  (Summed in tensor memory over a segment of 128 chunks the state
                    // fell short by 6.4e-5, every sum being cut off.)  The next arrival on kt_full gives them back.
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t s[32];
                        if (c > 1)
                            sum(s, x, L::kColSum, ((cc - 1) & 1) * L::kColHigh[1]);
                        else
                            tmem_ld32(tm + ((cc - 1) & 1) * L::kColHigh[1] + x, s);
                        tmem_st32_nowait(tm + L::kColSum + x, s);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
            }
            if (chunks == 0 || !keeps) continue;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_full, uc & 1));
            ++uc;
            float* to = it->end;
            if (!ok || !to) continue;
            tc_fence_after();
            const bool wide = (reinterpret_cast<uintptr_t>(to) & 31u) == 0;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t s[32];
                if (!kGather) {
                    step(s, x, f);
                } else {
                    sum(s, x, L::kColSmall, ((cc - 1) & 1) * L::kColHigh[1]);
                    if (chunks > 1) {
                        uint32_t before[32];
                        tmem_ld32(tm + L::kColSum + x, before);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            s[e] = __float_as_uint(__uint_as_float(s[e]) + __uint_as_float(before[e]));
                    }
                }
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) store_32(to + (size_t)r * D + x + e, s + e, wide);
                }
            }
            if (!kGather && it->any_bad && mine) {
                const int* bad = reinterpret_cast<const int*>(smem + L::kOffBad) + (items.n & 1) * D;
#pragma unroll 1
                for (int x = 0; x < D; ++x)
                    if (bad[x] < len) to[(size_t)r * D + x] = __uint_as_float(0x7fffffffu);
            }
        }
        tc_fence_before();
    } else {
        // ---------------------------------------------------------------- P and the outputs: row r of the chunk
        const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float row = (float)r;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        int ii = 0;
        for (const Item* it; (it = items.next(ok)); items.done()) {
            if (kGather) continue;
            const int chunks = it->chunks, len = it->len;
            const float la = it->la;
            __nv_bfloat16* out = p.out + ((size_t)it->row * p.num_heads + (size_t)it->kvh * g) * D;
            if (chunks == 0) {  // padding: zero rows
                const int per = g * D / 8;
#pragma unroll 1
                for (long long i = r; i < (long long)len * per; i += 128)
                    *reinterpret_cast<uint4*>(out + (size_t)(i / per) * p.num_heads * D + i % per * 8) =
                        make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            const float lead = fast_exp2((row + 1.f) * la) * a.scale;
            const float* tab = reinterpret_cast<const float*>(smem + L::kOffTab) + (items.n & 1) * 32;
            const int* bad = reinterpret_cast<const int*>(smem + L::kOffBad) + (items.n & 1) * D;
            int c = 0, h = 0;
            for (; c < chunks; ++ii) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full, ii & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < kChunk; x += 32) {
                    // P goes over the first half of the scores: columns x / 2 .. x / 2 + 15 have been read
                    uint32_t w[16];
                    if (x < 32 * warp) {  // below the diagonal: a^{i-j} = a^{i-x-31} a^{31-(j-x)}
                        const float f = fast_exp2((row - (float)(x + 31)) * la) * a.scale;
                        uint32_t s[32];
                        tmem_ld32(tm + L::kColP + x, s);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(tab + e);
                            float y0, y1, y2, y3;
                            mul_x2(y0, y1, t.x, t.y, f, f);
                            mul_x2(y2, y3, t.z, t.w, f, f);
                            mul_x2(y0, y1, y0, y1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                            mul_x2(y2, y3, y2, y3, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                            w[e / 2] = pack_bf16x2(y0, y1);
                            w[e / 2 + 1] = pack_bf16x2(y2, y3);
                        }
                    } else if (x == 32 * warp) {  // on it: the powers one by one, as a^{-31} may overflow
                        const float base = row - (float)x;
                        uint32_t s[32];
                        tmem_ld32(tm + L::kColP + x, s);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float d0 = base - (float)e, d1 = base - (float)(e + 1);  // rows between j and i
                            float y0, y1;
                            mul_x2(y0, y1, d0, d1, la, la);
                            mul_x2(y0, y1, fast_exp2(y0), fast_exp2(y1), a.scale, a.scale);
                            mul_x2(y0, y1, y0, y1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                            w[e / 2] = pack_bf16x2(d0 >= 0.f ? y0 : 0.f, d1 >= 0.f ? y1 : 0.f);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = 0u;
                    }
                    tmem_st8_nowait(tm + L::kColP + x / 2, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
                    tmem_st8_nowait(tm + L::kColP + x / 2 + 8, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->qs_full, ii & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {  // Q S weighted, for P V to add to
                    uint32_t o[32];
                    tmem_ld32(tm + L::kColO + x, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * lead);
                    tmem_st32_nowait(tm + L::kColO + x, o);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_full);
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full, ii & 1));
                if (!ok) break;
                tc_fence_after();
                const int t = c * kChunk + r;
                __nv_bfloat16* dst = out + ((size_t)t * p.num_heads + h) * D;
                // two neighbouring lanes store 64 bytes of one row together, then of the other's; with this and the
                // state's 32-byte accesses 152 states x 1 chunk take 10.1 us against 11.3, x 8 34.1 against 36.0
                const bool odd = lane & 1;
                const bool even_row = (t & ~1) < len, odd_row = (t | 1) < len;
                __nv_bfloat16* first = out + ((size_t)(t & ~1) * p.num_heads + h) * D + (odd ? 16 : 0);
                const size_t step = (size_t)p.num_heads * D;
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32], v[16], w0[8], w1[8];
                    tmem_ld32(tm + L::kColO + x, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[8 + e], 1);
                        w0[e] = odd ? got : v[e];
                        w1[e] = odd ? v[8 + e] : got;
                    }
                    if (even_row) store_32(first + x, w0, wide);
                    if (odd_row) store_32(first + step + x, w1, wide);
                }
                __syncwarp();
                tc_fence_before();
                if (it->any_bad && t < len) {
#pragma unroll 1
                    for (int x = 0; x < D; ++x)
                        if (t >= bad[x]) dst[x] = __ushort_as_bfloat16(0x7fff);
                }
                mbar_arrive(&bars->o_empty);
                if (++h == g) {
                    h = 0;
                    ++c;
                }
            }
        }
        tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(p.status, kDevTimeout);
    __syncthreads();
    pdl_trigger();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// What each segment adds becomes what the next begins with: S <- a^(segment) S + what it adds, from the
// state the sequence has.  Four elements a thread; the segments of a sequence one after another.
template <int D>
__global__ void __launch_bounds__(256) linear_carry_kernel(const TcArgs a) {
    pdl_wait();
    pdl_trigger();
    const PackedArgs& p = a.l.rows;
    const int b = blockIdx.y, kvh = blockIdx.x / (D * D / 1024), at = blockIdx.x % (D * D / 1024) * 256 + threadIdx.x;
    const Rows w = rows_of(a.l, b);
    const int all = (w.len + kChunk - 1) / kChunk, n = (all + a.seg_chunks - 1) / a.seg_chunks - 1;
    if (n <= 0 || w.slot < 0 || w.slot >= a.l.num_slots) return;
    const Decay f(in_range(a.l.log_decay[kvh]), (float)(a.seg_chunks * kChunk));
    auto next = [&](float s, float x) { return fmaf(s, f.x, x) + (f.near ? s : 0.f); };
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!w.fresh) s = reinterpret_cast<const float4*>(a.l.state + ((size_t)w.slot * p.num_kv_heads + kvh) * D * D)[at];
    float4* seg = reinterpret_cast<float4*>(a.segments + ((size_t)b * a.segs * p.num_kv_heads + kvh) * D * D) + at;
    const size_t step = (size_t)p.num_kv_heads * D * D / 4;
    if (!w.fresh) seg[0] = s;
    seg += step;
    constexpr int kAhead = 4;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        float4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < n) x[i] = seg[(size_t)(i0 + i) * step];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i >= n) break;
            s.x = next(s.x, x[i].x);
            s.y = next(s.y, x[i].y);
            s.z = next(s.z, x[i].z);
            s.w = next(s.w, x[i].w);
            seg[(size_t)(i0 + i) * step] = s;
        }
    }
}

// Segments a sequence: as many as make the waves of items end soonest, counting an item's start, its state
// and what gathering costs as three chunks; one when the sequences and heads fill the GPU by themselves.
int segments_of(int batch, int num_kv_heads, int max_chunk) {
    const int sms = device_info().num_sms;
    const long long pairs = (long long)batch * num_kv_heads;
    const int chunks = (max_chunk - 1) / kChunk + 1;
    if (pairs >= sms || chunks < 8) return 1;
    int best = 1;
    long long least = LLONG_MAX;
    for (int n = 1; n <= 64 && n <= chunks / 2; ++n) {
        const long long waves = (pairs * n + sms - 1) / sms;
        const long long per = (chunks + n - 1) / n;
        const long long cost = waves * (n == 1 ? 2 * per : 3 * per + 6);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

template <int D>
cudaError_t launch(const LinearArgs& a, void* workspace, cudaStream_t stream) {
    static OncePerDevice configured;
    const cudaError_t e = configured.run([] {
        cudaError_t r = cudaFuncSetAttribute((const void*)linear_kernel<D, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D, false>::kSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute((const void*)linear_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Layout<D, true>::kSmem);
        return r;
    });
    if (e != cudaSuccess) return e;
    const PackedArgs& p = a.rows;
    TcArgs t;
    t.l = a;
    t.group = p.num_heads / p.num_kv_heads;
    t.scale = p.scale;
    t.segments = static_cast<float*>(workspace);
    // as many segments as the workspace was sized for, or fewer: no sequence is longer than the rows there are
    const int chunks = (std::min(a.max_chunk, p.num_tokens) - 1) / kChunk + 1;
    const int segs = segments_of(p.batch, p.num_kv_heads, a.max_chunk);
    t.seg_chunks = (chunks + segs - 1) / segs;
    t.segs = (chunks + t.seg_chunks - 1) / t.seg_chunks;
    CUtensorMap q, k, v;
    if (!strided_map(&q, p.q, p.num_tokens, p.num_heads, D, p.q_stride, 1, kChunk, D / 64) ||
        !strided_map(&k, p.k, p.num_tokens, p.num_kv_heads, D, p.k_stride, 1, kChunk, D / 64) ||
        !strided_map(&v, p.v, p.num_tokens, p.num_kv_heads, D, p.v_stride, 1, kChunk, D / 64))
        return cudaErrorInvalidValue;
    const long long pairs = (long long)p.batch * p.num_kv_heads;
    if (pairs * t.segs > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (t.segs > 1) {
        cfg.gridDim = dim3((unsigned)(pairs * (t.segs - 1)));
        cfg.dynamicSmemBytes = Layout<D, true>::kSmem;
        cudaError_t r = cudaLaunchKernelEx(&cfg, linear_kernel<D, true>, q, k, v, t);
        if (r != cudaSuccess) return r;
        cudaLaunchConfig_t carry = cfg;
        carry.gridDim = dim3(p.num_kv_heads * (D * D / 1024), p.batch);
        carry.blockDim = dim3(256);
        carry.dynamicSmemBytes = 0;
        r = cudaLaunchKernelEx(&carry, linear_carry_kernel<D>, t);
        if (r != cudaSuccess) return r;
    }
    cfg.gridDim = dim3((unsigned)(pairs * t.segs));
    cfg.dynamicSmemBytes = Layout<D, false>::kSmem;
    return cudaLaunchKernelEx(&cfg, linear_kernel<D, false>, q, k, v, t);
}

}  // namespace

int linear_segments(int batch, int num_kv_heads, int max_chunk) { return segments_of(batch, num_kv_heads, max_chunk); }

cudaError_t launch_linear_prefill_tc(const LinearArgs& a, void* workspace, cudaStream_t stream) {
    return a.rows.head_dim == 64 ? launch<64>(a, workspace, stream) : launch<128>(a, workspace, stream);
}

}  // namespace pa
