// pa_tables.cu -- block tables, lengths, slots and positions of a step built on the GPU from the
// requests' lengths (pa_kv_grow), and blocks given back to the free list (pa_kv_free).
//
// Both are prefix sums over the sequences followed by a write of every token's (every block's)
// entry: a chain of dependent reads and barriers, and at most a few MB, so latency bounds them.  One
// launch does it: a single thread-block cluster, every CTA of which sums the counts of a tile of
// sequences for itself (a tile is 512 sequences, one a thread) and then writes its share of the tile's
// rows.  What the call may update in place is written after a cluster barrier behind the last read of it.
// Inside a graph: 64 new rows 4.0 us, 16384 4.8, 65536 7.7; 4608 blocks back 5.4 us, 65536 8.4, 409600 29.
#include <algorithm>

#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;  // (8 CTAs: 65536 rows 11.3 us against 7.7, 65536 blocks back 11.8 against 8.4)
constexpr int kAhead = 8;        // rows (entries) of a thread whose loads are in flight together

// Inclusive sums over the CTA's threads; `total` gets the sum of all.  sums: kWarps words.
__device__ __forceinline__ long long block_scan(long long x, long long* sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0 && lane < kWarps) {
        long long s = sums[lane];
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const long long up = __shfl_up_sync((1u << kWarps) - 1, s, o);
            if (lane >= o) s += up;
        }
        sums[lane] = s;
    }
    __syncthreads();
    total = sums[kWarps - 1];
    incl += warp ? sums[warp - 1] : 0;
    __syncthreads();  // sums may be used again
    return incl;
}

// The last i in [0, kThreads) with first[i] <= x, where first is non-decreasing and first[0] <= x.
__device__ __forceinline__ int find_row(const int* first, int x) {
    int i = 0;
#pragma unroll
    for (int step = kThreads / 2; step > 0; step >>= 1)
        if (first[i + step] <= x) i += step;
    return i;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (int)(((unsigned)tokens + kBlockSize - 1) / kBlockSize); }

__global__ void __launch_bounds__(kThreads) grow_kernel(const GrowArgs a) {
    __shared__ long long sums[kWarps];
    __shared__ int s_first[kThreads];  // first row of each of the tile's sequences
    __shared__ int s_len[kThreads];    // its tokens before the step
    __shared__ int s_block[kThreads];  // blocks given to the sequences before it
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int asked_free = *a.num_free;
    const int have = min(max(asked_free, 0), a.capacity);
    if (tid == 0 && rank == 0 && have != asked_free) atomicOr(a.status, kDevOutOfRange);
    long long sum_need = 0, sum_new = 0;    // asked for by the sequences of the earlier tiles
    long long used = 0, rows = 0;           // given to them
    const long long most = (long long)a.max_blocks * kBlockSize;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        int len = 0, fresh = 0, need = 0, old_len = 0;
        if (b < a.batch) {
            old_len = len = a.seq_lens[b];
            fresh = a.new_lens[b];
            if (len < 0 || fresh < 0 || (long long)len + fresh > most) {
                if (rank == 0) atomicOr(a.status, kDevOutOfRange);
                len = fresh = 0;
            }
            need = blocks_of(len + fresh) - blocks_of(len);
        }
        long long t_need, t_new, t_used, t_rows;
        const long long cum_need = sum_need + block_scan(need, sums, t_need);
        const long long cum_new = sum_new + block_scan(fresh, sums, t_new);
        if ((need > 0 && cum_need > have) || cum_new > a.max_tokens) need = fresh = 0;
        const long long block = used + block_scan(need, sums, t_used) - need;
        const long long first = rows + block_scan(fresh, sums, t_rows) - fresh;
        s_first[tid] = (int)first;
        s_len[tid] = len;
        s_block[tid] = (int)block;
        cluster.sync();  // every CTA has read the tile's lengths; the tile's sums are in place
        if (rank == 0 && b < a.batch) {
            a.cu_lens[b] = (int)first;
            a.seq_lens_out[b] = old_len + fresh;
        }
        const long long step = ctas * kThreads, end = rows + t_rows;
        for (long long t0 = rows + rank * kThreads + tid; t0 < end; t0 += kAhead * step) {
            int seq[kAhead], pos[kAhead], id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long t = t0 + u * step;
                if (t >= end) break;
                const int i = seq[u] = find_row(s_first, (int)t);
                pos[u] = s_len[i] + (int)t - s_first[i];
                const int j = pos[u] / kBlockSize, mine = j - blocks_of(s_len[i]);  // mine >= 0: one of the new blocks
                id[u] = mine >= 0 ? a.free_blocks[have - 1 - (s_block[i] + mine)]
                                  : a.tables[(size_t)(b0 + i) * a.max_blocks + j];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long t = t0 + u * step;
                if (t >= end) break;
                const int i = seq[u], j = pos[u] / kBlockSize;
                if (j >= blocks_of(s_len[i]) && pos[u] % kBlockSize == 0)
                    a.tables[(size_t)(b0 + i) * a.max_blocks + j] = id[u];
                a.slots[t] = (int64_t)id[u] * kBlockSize + pos[u] % kBlockSize;
                a.positions[t] = pos[u];
                a.token_seqs[t] = b0 + i;
            }
        }
        sum_need += t_need;
        sum_new += t_new;
        used += t_used;
        rows += t_rows;
        __syncthreads();  // the tile's sums are free
    }
    for (long long t = rows + rank * kThreads + tid; t < a.max_tokens; t += ctas * kThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
        a.token_seqs[t] = -1;
    }
    cluster.sync();  // *num_free has been read by all
    if (rank == 0 && tid == 0) {
        a.cu_lens[a.batch] = (int)rows;
        *a.num_free_out = have - (int)used;
    }
}

__global__ void __launch_bounds__(kThreads) free_kernel(const FreeArgs a) {
    __shared__ long long sums[kWarps];
    __shared__ int s_first[kThreads + 1];  // first of each row's entries among the tile's, and their count
    __shared__ int s_warp[kWarps];      // blocks in the runs of the warps before this one
    __shared__ int s_all;               // blocks in the CTA's runs
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int asked_free = *a.num_free;
    const int begin = min(max(asked_free, 0), a.capacity);
    if (tid == 0 && rank == 0 && begin != asked_free) atomicOr(a.status, kDevOutOfRange);
    long long at = begin;
    for (long long r0 = 0; r0 < a.rows; r0 += kThreads) {
        const long long r = r0 + tid;
        int count = 0;
        if (r < a.rows) {
            const int asked = a.counts[r];
            count = min(max(asked, 0), a.width);
            if (count != asked && rank == 0) atomicOr(a.status, kDevOutOfRange);
        }
        long long total;  // below 2^31: kThreads rows of at most kFreeMaxWidth entries
        s_first[tid] = (int)(block_scan(count, sums, total) - count);
        if (tid == 0) s_first[kThreads] = (int)total;
        __syncthreads();
        // the tile's entries in runs, one a warp, each a multiple of 32 long
        const int n = (int)total, warps = ctas * kWarps;
        const int run = (int)((total + 32LL * warps - 1) / (32LL * warps)) * 32;
        const long long e0 = (long long)(rank * kWarps + warp) * run;
        const long long e1 = min(e0 + run, (long long)n);
        // -1 where there is no block; a lane's next entry is mostly in the row of its last (512 rows of 800: 53 us
        // against 79 when each is searched for)
        auto entry = [&](long long e, int& i) {
            if (e >= e1) return -1;
            if (s_first[i + 1] <= (int)e) i = find_row(s_first, (int)e);
            return a.ids[(size_t)(r0 + i) * a.width + ((int)e - s_first[i])];
        };
        int mine = 0, at_row = 0;
        for (long long e = e0; e < e1; e += 32 * kAhead) {
            int id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) id[u] = entry(e + 32 * u + lane, at_row);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) mine += __popc(__ballot_sync(0xffffffffu, id[u] >= 0));
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            int sum = 0;
            for (int w = 0; w < kWarps; ++w) {
                const int x = s_warp[w];
                s_warp[w] = sum;
                sum += x;
            }
            s_all = sum;
        }
        cluster.sync();
        long long before = at;
        for (int c = 0; c < ctas; ++c) {
            const int x = *cluster.map_shared_rank(&s_all, c);
            if (c < rank) before += x;
            at += x;
        }
        before += s_warp[warp];
        at_row = 0;
        for (long long e = e0; e < e1; e += 32 * kAhead) {
            int id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) id[u] = entry(e + 32 * u + lane, at_row);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const unsigned there = __ballot_sync(0xffffffffu, id[u] >= 0);
                const long long to = before + __popc(there & ((1u << lane) - 1));
                if (id[u] >= 0 && to < a.capacity) a.free_blocks[to] = id[u];
                before += __popc(there);
            }
        }
        cluster.sync();  // the CTAs' counts have been read
    }
    cluster.sync();  // *num_free has been read by all
    if (rank == 0 && tid == 0) {
        if (at > a.capacity) atomicOr(a.status, kDevOutOfRange);
        *a.num_free_out = (int)min(at, (long long)a.capacity);
    }
}

template <typename A>
cudaError_t launch_cluster(void (*kernel)(const A), const A& a, long long items, cudaStream_t stream) {
    static OncePerDevice configured;
    const cudaError_t e = configured.run([kernel] {
        return cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    // one item a thread before another CTA is taken in (four: 2048 rows 5.6 us against 4.2)
    const int ctas = (int)std::max(1LL, std::min<long long>(kMaxCluster, (items + kThreads - 1) / kThreads));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_grow(const GrowArgs& a, cudaStream_t stream) {
    return launch_cluster(grow_kernel, a, a.max_tokens, stream);
}

cudaError_t launch_free(const FreeArgs& a, cudaStream_t stream) {
    return launch_cluster(free_kernel, a, (long long)a.rows * a.width, stream);
}

}  // namespace pa
