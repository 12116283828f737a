/*
 * pagedattn.h -- C ABI of libpagedattn: grouped-query attention over a block-paged
 * KV cache, hand-written CUDA for GB300 (sm_103a).
 *
 * The operation.  The pages "Qwen3-4B / 8B / 32B" (section "Architecture Notes")
 * describe full attention with grouped-query attention -- Qwen3-4B: 32 query heads
 * over 8 KV heads, head dim 128; Qwen3-32B: 64 query heads, group 8 -- served from a
 * paged KV cache with prefix caching; section "Qwen3-32B Serving Load" gives a KV
 * budget of 21.4 GB = 5360 blocks for Qwen3-32B, which fixes 16-token blocks; section
 * "Warm Prefix-Cache TTFT" is the chunked prefill over a warm prefix.  For query head
 * h of a sequence, with g = num_heads / num_kv_heads and kv head h / g:
 *
 *     o = sum_{t in keys} softmax_t(scale * <q, K_t>) V_t
 *
 * K_t, V_t read at pool[block_tables[s][t / 16], h / g, t % 16, :].  Softmax in fp32
 * (online, base 2), bf16 inputs, bf16 output rounded to nearest even.  The probabilities
 * enter the P V product on the tensor cores as bf16 -- as two bf16 parts (about 16 bits)
 * wherever a few weights can dominate a row: always in pa_decode, pa_decode_splitkv and
 * pa_append_decode; in pa_prefill_chunked always at head_dim 64 or a group size that does
 * not divide 128, else in the query tiles holding a query that sees at most 128 keys, and
 * everywhere at |scale| sqrt(head_dim) > 2 -- with the softmax sum taken over exactly those
 * values; accumulation is fp32.
 *
 * Memory.  Every pointer argument is a DEVICE pointer of the current CUDA device
 * unless stated otherwise; the caller allocates and owns every buffer (the library
 * allocates no device memory).  Every call is asynchronous on `stream` (NULL = the
 * legacy default stream) and returns after the launch: the return code reports host
 * validation and launch errors only.  Problems the device finds (a block id or slot
 * outside the pool, a pipeline wait that timed out) set bits of a device status word
 * that pa_device_status() reads.  Calls are thread-safe.
 *
 * Layouts (all row-major, contiguous):
 *   pool K, V      [num_blocks, num_kv_heads, 16, head_dim]   bf16, 16-byte aligned
 *   slot           block_id * 16 + offset_in_block
 *   block_tables   [batch, max_blocks] int32; entries past ceil(seq_len / 16) never affect
 *                  a result (a decode may load up to 32 entries of a row, all within the row,
 *                  before it knows seq_len, and ignores those it does not need)
 *   seq_lens       [batch] int32, tokens in the sequence including any appended this step
 *   q, out         decode [batch, num_heads, head_dim]; prefill [sum of chunk lengths,
 *                  num_heads, head_dim]; bf16, 16-byte aligned
 *
 * Supported: block_size 16; head_dim 64 or 128; any group size for prefill, group
 * size <= 16 for decode; batch <= 65535.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle as cudaStream_t. */
typedef struct CUstream_st *pa_stream_t;

enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = -1,  /* host validation failed; nothing was launched */
    PA_ERR_UNSUPPORTED = -2,  /* block size, head dim or group size outside the compiled set */
    PA_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed */
    PA_ERR_OUT_OF_RANGE = -4, /* pa_device_status: a block id / slot / length outside the pool was skipped */
    PA_ERR_TIMEOUT = -5,      /* pa_device_status: a pipeline wait ran out (a bug, never expected) */
    PA_ERR_TOO_LARGE = -6,    /* pa_decode_splitkv_noalloc: the request does not fit its static scratch */
    PA_ERR_REJECTED = -7,     /* pa_bm_admit: the request's whole lifetime does not fit the pool */
    PA_ERR_NO_MEMORY = -8     /* pa_bm_*: no host memory; nothing has changed */
};

/* Device status bits reported by pa_device_status. */
#define PA_DEV_OUT_OF_RANGE 1u
#define PA_DEV_TIMEOUT 2u

/* The paged KV pool: two device tensors [num_blocks, num_kv_heads, block_size, head_dim] bf16. */
typedef struct {
    void *k_cache;
    void *v_cache;
    int32_t num_blocks;
    int32_t block_size;   /* must be 16 */
    int32_t num_kv_heads;
    int32_t head_dim;     /* 64 or 128 */
} pa_pool;

/*
 * An 8-bit pool: the same block-paged K and V as e4m3 codes, one byte each, and one power-of-two
 * scale for every (block, kv head) of K and of V:
 *   K[block, h, t, d] = e4m3(k_cache[block, h, t, d]) * 2^(exps[block, h, 0] - 127)
 *   V likewise with exps[block, h, 1].
 * exps holds values 27 .. 246 (2^-100 .. 2^119), in which every product is a normal bf16 number,
 * so reading the pool rounds nothing.  Half the bytes of a bf16 pool (and 2 per block and kv
 * head): half the time of a decode, and twice the blocks of a memory budget
 * (pa_kv_block_bytes with dtype_bytes = 1).  The caller owns the three tensors and zeroes
 * them, or at least writes a block's offset 0 before its other rows; exponents outside the range
 * (a zeroed pool's) are taken as its nearer end, by every call.
 */
typedef struct {
    void *k_cache;        /* [num_blocks, num_kv_heads, 16, head_dim] e4m3, 16-byte aligned */
    void *v_cache;
    void *exps;           /* [num_blocks, num_kv_heads, 2] uint8, 2-byte aligned */
    int32_t num_blocks;
    int32_t block_size;   /* must be 16 */
    int32_t num_kv_heads;
    int32_t head_dim;     /* 64 or 128 */
} pa_pool8;

/*
 * pa_kv_append -- write new K/V rows into their pool slots.
 * Defines: for t in [0, num_tokens) with slot_mapping[t] >= 0,
 *   k_cache[slot / 16, h, slot % 16, :] = k_new[t, h, :]  (and v likewise), every kv head h.
 * This is how a decode token or a prefill chunk enters the paged cache ("Qwen3-4B / 8B /
 * 32B", "Architecture Notes": paged KV cache; "Warm Prefix-Cache TTFT": only new tokens
 * are written on a prefix hit).  It must precede, on the same stream, the attention call
 * that reads those tokens.
 *   k_new, v_new   [num_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned
 *   slot_mapping   [num_tokens] int64; < 0 skips the row; >= num_blocks*16 is skipped and
 *                  sets PA_DEV_OUT_OF_RANGE.  Duplicate slots are a caller error.
 * Bit-exact copy.  num_tokens == 0 is a no-op; a call that would move 2^31 or more
 * 16-byte chunks (num_tokens * 2 * num_kv_heads * head_dim / 8) is PA_ERR_INVALID_ARG.
 */
int pa_kv_append(const pa_pool *pool, const void *k_new, const void *v_new, const int64_t *slot_mapping,
                 int32_t num_tokens, pa_stream_t stream);

/*
 * pa_kv_copy -- copy whole pool rows (every kv head, K and V): for t in [0, n),
 *   k_cache[dst / 16, h, dst % 16, :] = k_cache[src / 16, h, src % 16, :]  (and v likewise)
 * with src = src_slots[t], dst = dst_slots[t].  This is the copy on write of a prefix-cache
 * hit that ends inside a cached block ("Qwen3-4B / 8B / 32B", "Warm Prefix-Cache TTFT": a
 * warm request reuses the cached K/V of its prompt prefix): pa_bm_admit_cow returns the slot
 * pairs, and the copy must precede, on the same stream, the append of the request's own
 * tokens and any attention call that reads them.
 *   src_slots, dst_slots  [n] int64 device arrays; a pair with a negative slot is skipped, one
 *                         past the pool is skipped and sets PA_DEV_OUT_OF_RANGE.  A dst slot
 *                         that is also some pair's src slot is a caller error.
 * Bit-exact copy.
 */
int pa_kv_copy(const pa_pool *pool, const int64_t *src_slots, const int64_t *dst_slots, int32_t n,
               pa_stream_t stream);

/*
 * pa_kv_append8 -- pa_kv_append into an 8-bit pool: rows are rounded to e4m3 (to nearest even)
 * under their block's scale.  Per (block, kv head, K or V), with k(a) the smallest exponent
 * in [-100, 119] for which a <= 448 * 2^k(a), and a the new rows' largest finite magnitude:
 *   * when the call writes offset 0 of the block, the block begins anew: k = k(a), and the bytes
 *     of the rows it does not write stay as they are;
 *   * otherwise k = max(k_old, k(a)); if that is larger than k_old, the codes of the rows it does
 *     not write are multiplied by 2^(k_old - k) and rounded again, which loses bits only
 *     below 2^-6 * 2^k.
 * Infinities and values past 448 * 2^k saturate, a NaN stays one.  The rows a block receives
 * must be consecutive entries of slot_mapping (negative entries between them do not count), as
 * the tokens of a sequence are; a block that comes up again later in the same call is a caller
 * error, and so are calls that write the same block at the same time.  Of entries with the same
 * slot the last counts.  Arguments and errors otherwise as pa_kv_append.  Rows are not copied from
 * block to block of an 8-bit pool: admit requests with pa_bm_admit, whose hits are whole blocks.
 */
int pa_kv_append8(const pa_pool8 *pool, const void *k_new, const void *v_new, const int64_t *slot_mapping,
                  int32_t num_tokens, pa_stream_t stream);

/*
 * pa_decode -- one query token per sequence attends to keys [0, seq_lens[b]).
 * ("Qwen3-4B / 8B / 32B", "Architecture Notes": GQA over a paged KV cache; the query is
 * the newest token, already appended.)
 *   q, out         [batch, num_heads, head_dim] bf16
 *   scale          softmax scale, normally 1/sqrt(head_dim)
 * seq_lens[b] == 0 gives a zero row.  seq_lens[b] outside [0, max_blocks*16] is clamped
 * and sets PA_DEV_OUT_OF_RANGE.  When batch * num_kv_heads is small the library splits
 * each sequence over a thread-block cluster and merges in on-chip memory (no workspace).
 */
int pa_decode(const pa_pool *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
              const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale, void *out,
              pa_stream_t stream);

/*
 * pa_decode8 -- pa_decode over an 8-bit pool (same arguments, errors and splitting).  K and V are
 * taken exactly as stored; q enters the tensor core as f16 after each row is brought to a
 * maximum in [2^14, 2^15) by a power of two (exact for elements above 2^-29 of the row's
 * maximum), the softmax weights as f16, each with its block's V scale, under a running
 * maximum of their products; sums are fp32.  A NaN among the scores a head sees makes its result NaN.
 */
int pa_decode8(const pa_pool8 *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
               const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale, void *out,
               pa_stream_t stream);

/* Workspace of pa_decode_weights and pa_decode8_weights, in bytes (a float per block and query
 * head of a group, the group rounded up to 8 or 16).  Host-only, no CUDA call. */
size_t pa_weights_workspace_bytes(int32_t batch, int32_t num_heads, int32_t num_kv_heads, int32_t max_blocks);

/*
 * pa_decode_weights, pa_decode8_weights -- pa_decode / pa_decode8 that also add up the attention
 * weight every block got, for pa_kv_evict.  With p the softmax weights of the call,
 *   weights[b, h, j] = decay * weights[b, h, j] + sum of p over the query heads of kv head h and
 *                      the keys of logical block j          for j < ceil(seq_lens[b] / 16);
 * other entries stay as they are.  A sequence's row starts at zero.  Each entry is added up by
 * one thread in a fixed order, so a repeated call gives the same bits.  A query head whose
 * scores hold a NaN adds nothing.
 *   weights    [batch, num_kv_heads, max_blocks] fp32, updated in place
 *   decay      finite; 1 keeps the plain sum
 *   workspace  pa_weights_workspace_bytes(...) bytes, 4-byte aligned, not shared by calls that
 *              may run at the same time; nothing in it outlives the call
 */
int pa_decode_weights(const pa_pool *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
                      const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale, float decay,
                      float *weights, float *workspace, void *out, pa_stream_t stream);
int pa_decode8_weights(const pa_pool8 *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
                       const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale, float decay,
                       float *weights, float *workspace, void *out, pa_stream_t stream);

/*
 * pa_kv_evict -- evict the blocks with the lowest accumulated weight, so that no sequence keeps
 * more than keep_blocks.  Per sequence, nb = ceil(seq_len / 16) and e = max(0, nb - keep_blocks):
 * of the logical blocks [sink_blocks, nb - recent_blocks) the e with the lowest
 * W_j = sum_h weights[b, h, j] (fp64, rounded to fp32) leave, of equal ones the lower index first,
 * a NaN before all.  Then
 *   block_tables_out  the row without the e entries, in order, reserved entries past nb included;
 *                     the last e entries are -1
 *   weights_out       the rows likewise; the last e entries are 0
 *   seq_lens_out      seq_len - 16 e: later tokens are appended at the shortened positions (their
 *                     rotary positions, which K already carries, are the caller's)
 *   evicted           [batch, max_blocks] the ids that left, in order of their position, -1 behind
 *                     them (for pa_bm_evict); num_evicted [batch] = e
 * K and V do not move and no block is written, so blocks shared with other sequences are safe.
 * Any of the three outputs may be its input; otherwise the arrays must not overlap.  A seq_len
 * outside [0, max_blocks * 16] is clamped and sets PA_DEV_OUT_OF_RANGE.
 * sink_blocks >= 0, recent_blocks >= 1 (the block being filled stays), their sum at most
 * keep_blocks; max_blocks at most 49152, else PA_ERR_UNSUPPORTED.
 */
int pa_kv_evict(const int32_t *block_tables, const int32_t *seq_lens, const float *weights, int32_t batch,
                int32_t max_blocks, int32_t num_kv_heads, int32_t keep_blocks, int32_t sink_blocks,
                int32_t recent_blocks, int32_t *block_tables_out, int32_t *seq_lens_out, float *weights_out,
                int32_t *evicted, int32_t *num_evicted, pa_stream_t stream);

/*
 * pa_append_decode -- pa_kv_append of one new row per sequence followed by pa_decode, in
 * one launch (a decode step's append and attention fused; the pages' engines write a
 * token's K/V and then attend over it in every full-attention layer).  Equivalent to
 *   pa_kv_append(pool, k_new, v_new, slot_mapping, batch); pa_decode(pool, q, ...);
 * on the same stream, given that slot_mapping[b] is the slot of token seq_lens[b] - 1 of
 * sequence b (block_tables[b][(seq_lens[b]-1)/16] * 16 + (seq_lens[b]-1) % 16), as an
 * append for that token must be.
 *   k_new, v_new   [batch, num_kv_heads, head_dim] bf16, 16-byte aligned: the new rows
 *   slot_mapping   [batch] int64; < 0 skips the write (the decode then reads whatever the
 *                  slot holds).  Any other slot than the one above is not written and sets
 *                  PA_DEV_OUT_OF_RANGE.
 * Other arguments, errors and results as pa_decode.
 */
int pa_append_decode(const pa_pool *pool, const void *k_new, const void *v_new, const int64_t *slot_mapping,
                     const void *q, const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
                     int32_t batch, int32_t num_heads, float scale, void *out, pa_stream_t stream);

/*
 * Workspace of pa_decode_splitkv, in bytes: ws_o [batch, num_heads, P, head_dim] fp32
 * followed by ws_lse [batch, num_heads, P] fp32 (ws_lse may live anywhere 16-byte aligned;
 * this is their sum).  Host-only, no CUDA call.
 */
size_t pa_splitkv_workspace_bytes(int32_t batch, int32_t num_heads, int32_t head_dim, int32_t num_partitions);

/*
 * pa_decode_splitkv -- flash-decoding partitions of the decode above.  Partition p of P
 * covers logical blocks [p*ceil(nb/P), (p+1)*ceil(nb/P)) of the nb = ceil(seq_len/16)
 * blocks and writes its own normalised output O_p and natural-log log-sum-exp
 * lse_p = m_p + ln(l_p) of its scaled scores; an empty partition writes O_p = 0,
 * lse_p = -inf.  (Long-context decode: the pages' long prompts are 4097-16384 tokens,
 * "Warm Prefix-Cache TTFT" and the 4097/8192-token golden prompts.)
 *   num_partitions P in [1, 4096]
 *   ws_o           [batch, num_heads, P, head_dim] fp32, 16-byte aligned (scratch owned by caller)
 *   ws_lse         [batch, num_heads, P] fp32
 */
int pa_decode_splitkv(const pa_pool *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
                      const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale,
                      int32_t num_partitions, float *ws_o, float *ws_lse, pa_stream_t stream);

/*
 * pa_combine -- log-sum-exp merge of split-KV partitions:
 *   M = max_p lse_p;  w_p = exp(lse_p - M);  out = sum_p w_p O_p / sum_p w_p
 * (partitions with lse_p = -inf weigh 0; all empty gives a zero row).
 *   ws_o, ws_lse   as written by pa_decode_splitkv;  out [batch, num_heads, head_dim] bf16
 */
int pa_combine(const float *ws_o, const float *ws_lse, int32_t batch, int32_t num_heads, int32_t head_dim,
               int32_t num_partitions, void *out, pa_stream_t stream);

/*
 * pa_prefill_chunked -- a causal query chunk over a cached paged prefix plus itself.
 * Sequence b's chunk is q rows [cu_q_lens[b], cu_q_lens[b+1]) (C_b tokens); seq_lens[b]
 * counts the prefix AND the chunk (whose K/V pa_kv_append already wrote).  Chunk query i
 * sits at position seq_lens[b] - C_b + i and attends to keys 0 .. that position.
 * ("Qwen3-4B / 8B / 32B", "Warm Prefix-Cache TTFT": warm prefix hit, only the new chunk
 * is computed.)
 *   q, out         [cu_q_lens[batch], num_heads, head_dim] bf16
 *   cu_q_lens      [batch + 1] int32, non-decreasing, cu_q_lens[0] = 0
 *   max_chunk      an upper bound of max_b C_b (sizes the grid; rows beyond C_b are idle).  A
 *                  chunk longer than the grid covers is reported (PA_DEV_OUT_OF_RANGE in the
 *                  device status) and its rows past the grid are not written; the other
 *                  sequences' results are unaffected
 * A sequence with C_b > seq_lens[b] or seq_lens[b] > max_blocks*16 is skipped and sets
 * PA_DEV_OUT_OF_RANGE.
 */
int pa_prefill_chunked(const pa_pool *pool, const void *q, const int32_t *cu_q_lens, const int32_t *block_tables,
                       int32_t max_blocks, const int32_t *seq_lens, int32_t batch, int32_t num_heads,
                       int32_t max_chunk, float scale, void *out, pa_stream_t stream);

/*
 * pa_prefill_chunked8 -- pa_prefill_chunked over an 8-bit pool: same arguments and
 * errors, arithmetic as pa_decode8.  Chunks of at most 16 / group queries run on the decode kernel.
 * A NaN in V concerns the queries that see its key, and its column, alone.
 */
int pa_prefill_chunked8(const pa_pool8 *pool, const void *q, const int32_t *cu_q_lens, const int32_t *block_tables,
                        int32_t max_blocks, const int32_t *seq_lens, int32_t batch, int32_t num_heads,
                        int32_t max_chunk, float scale, void *out, pa_stream_t stream);

/*
 * pa_prefill_packed -- causal attention over whole prompts, packed one after another, before any
 * of their tokens is cached: row t of sequence b (rows cu_lens[b] .. cu_lens[b+1]) attends to the
 * rows cu_lens[b] .. t of its own sequence, query head h to kv head h / (num_heads / num_kv_heads).
 * K and V are read where the projection left them; pa_kv_append brings them into a pool, before
 * or after.  ("Qwen3-4B / 8B / 32B", "Warm Prefix-Cache TTFT": the cold prompts that table begins
 * with.)
 *   q              num_tokens rows of [num_heads, head_dim] bf16, 16-byte aligned, q_stride elements
 *                  apart; k, v: rows of [num_kv_heads, head_dim], k_stride and v_stride apart (views
 *                  of one fused projection, say).  A stride is a multiple of 8, at least its row and
 *                  below 2^39
 *   cu_lens        [batch + 1] int32, non-decreasing, within [0, num_tokens]
 *   max_len        an upper bound of the sequences' lengths (sizes the grid).  Rows past it are
 *                  reported (PA_DEV_OUT_OF_RANGE) and not written
 *   out            [num_tokens, num_heads, head_dim] bf16, contiguous, 16-byte aligned; rows outside
 *                  every sequence stay as they are.  It overlaps none of the inputs
 * A sequence whose rows are not within [0, num_tokens] is skipped and sets PA_DEV_OUT_OF_RANGE.  A
 * NaN or an infinity in K or V concerns the rows that see its key alone, in V its column alone; a
 * score of +inf makes its row NaN, one of -inf gives its key no weight, and a row of nothing else is NaN.
 * head_dim 64 or 128, any group size, batch <= 65535; arithmetic as pa_prefill_chunked (weights of up to
 * 2^8, summed with v in fp32: |v| from 2^-100 to 2^100 keeps within its range).
 */
int pa_prefill_packed(const void *q, const void *k, const void *v, const int32_t *cu_lens, int32_t batch,
                      int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t max_len, float scale, void *out,
                      pa_stream_t stream);

/*
 * pa_kv_grow -- a step's new tokens enter the sequences, without the host: blocks from a free list on
 * the GPU, and from the token counts everything that the step's other calls take.  Sequence b
 * holds seq_lens[b] tokens and asks for new_lens[b] more, which need
 *   need[b] = ceil((seq_lens[b] + new_lens[b]) / 16) - ceil(seq_lens[b] / 16)  blocks.
 * In the order of b, a sequence gets its tokens, all or none, when
 *   need[b] == 0 or need[0] + .. + need[b] <= *num_free,  and  new_lens[0] + .. + new_lens[b] <= max_tokens
 * (a request that does not fit holds its place: those behind it that need blocks wait too).  Then
 *   block_tables   [batch, max_blocks], in place: entries ceil(seq_lens[b] / 16) .. take the blocks, from
 *                  the end of the free list, free_blocks[*num_free - 1] first; all others stay
 *   seq_lens_out   [batch] the lengths, with the tokens given;  num_free_out [1] the blocks left
 *   cu_lens        [batch + 1] int32 first row of every sequence's new tokens; cu_lens[batch] the rows
 *   slot_mapping   [max_tokens] int64 cache slot of every row (pa_kv_append), -1 past the last
 *   positions      [max_tokens] int32 place of the row's token in its sequence, 0 past the last
 *   token_seqs     [max_tokens] int32 sequence of the row, -1 past the last
 * seq_lens_out may be seq_lens, num_free_out may be num_free; otherwise no two arrays overlap.  A
 * sequence with a negative length or count, or with more tokens than max_blocks * 16, gets none, asks
 * for none and sets PA_DEV_OUT_OF_RANGE; so does *num_free outside [0, capacity], which is clamped.
 *   free_blocks    [capacity] int32 block ids, the first *num_free of them free.  They are handed on
 *                  as they are: the calls that read the tables check them.  batch <= 65535
 */
int pa_kv_grow(int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens, const int32_t *new_lens,
               int32_t batch, const int32_t *free_blocks, int32_t capacity, const int32_t *num_free,
               int32_t max_tokens, int32_t *seq_lens_out, int32_t *num_free_out, int32_t *cu_lens,
               int64_t *slot_mapping, int32_t *positions, int32_t *token_seqs, pa_stream_t stream);

/*
 * pa_kv_free -- blocks go back to the free list of pa_kv_grow: the entries ids[r][0 .. counts[r]) that are
 * not negative, row after row in their order, to free_blocks[*num_free], [*num_free + 1], ...; then
 *   num_free_out   [1] the blocks free now (may be num_free)
 * ids is a block table (counts: the blocks of the sequences that have finished, 0 for the others) or
 * the `evicted` of pa_kv_evict (counts: its num_evicted).  A block that other sequences still use is the
 * caller's to keep out.
 *   ids            [rows, width] int32, width below 2^22 (else PA_ERR_UNSUPPORTED);  counts [rows]
 *                  int32, outside [0, width] clamped and reported
 * Blocks past the list's capacity are dropped; they, and *num_free outside [0, capacity] (clamped), set
 * PA_DEV_OUT_OF_RANGE.  No two arrays overlap but num_free_out and num_free.
 */
int pa_kv_free(const int32_t *ids, const int32_t *counts, int32_t rows, int32_t width, int32_t *free_blocks,
               int32_t capacity, const int32_t *num_free, int32_t *num_free_out, pa_stream_t stream);

/*
 * pa_linear_decode, pa_linear_prefill -- linear attention with a fixed decay for each head and a state for
 * each request (the family of retention and lightning attention).  It is not the recurrence of the pages'
 * hybrid stack ("Qwen3.5"), whose gated delta rule decays by a gate of every token and takes what the state
 * holds for a key out of it before adding.  With a = exp(log_decay[h]) of kv head h, over a sequence's tokens t,
 *   S_t = a S_{t-1} + k_t v_t^T  (head_dim x head_dim),   o_t = scale q_t^T S_t,
 * query head i reading the state of kv head i / (num_heads / num_kv_heads).  The state lives in
 *   state          [num_slots, num_kv_heads, head_dim (of k), head_dim (of v)] fp32, 16-byte aligned,
 * sequence b's in slot state_slots[b]; the call reads it and leaves the new one there.  A sequence
 * whose tokens are all this call's (seq_lens[b] equals its row count) begins with S = 0, whatever the
 * slot holds.
 *   log_decay      [num_kv_heads] fp32, taken into [-1e4, 0]
 *   state_slots    [batch] int32; a negative slot is padding: zero rows, no state.  One past num_slots
 *                  likewise, and sets PA_DEV_OUT_OF_RANGE.  The same slot twice is a caller error
 *   seq_lens       [batch] int32, tokens of the sequence including this call's
 *   q, k, v        rows of [heads, head_dim] bf16, q_stride, k_stride, v_stride elements apart, as
 *                  pa_prefill_packed's;  out contiguous bf16, overlapping nothing
 * pa_linear_decode: row b is sequence b's newest token; seq_lens[b] <= 0 is padding (zero row, no state).
 * pa_linear_prefill: rows cu_q_lens[b] .. cu_q_lens[b+1] are its newest tokens, any number; none leaves the
 * state as it is.  Rows outside every sequence stay as they are; rows past max_chunk, a sequence with
 * fewer tokens than rows and one whose rows are not within [0, num_tokens] as in pa_prefill_packed.
 * Both keep S in fp32 throughout.  A call with max_chunk up to 6 goes token by token and computes in fp32 alone,
 * as pa_linear_decode; a longer one takes 128 tokens at a time, in products of q, k and v as they are, the scores
 * and S (where q reads it) as bf16, and k's weighted rows (where S gathers them) in full, as three bf16
 * parts.  So a sequence's outputs may differ in their last bits with the max_chunk of its batch; its state is
 * right to 32 bits either way.  A NaN or an infinity in a row of v concerns its column from that row on, in one of k its
 * row of the state and the outputs from there on; either may turn NaN as a whole.
 *   workspace      pa_linear_workspace_bytes(...) bytes, 16-byte aligned (may be NULL where that is 0),
 *                  not shared by calls that may run at the same time; nothing in it outlives the call
 * head_dim 64 or 128, any group size, batch <= 65535.
 */
int pa_linear_decode(float *state, int32_t num_slots, const int32_t *state_slots, const void *q, const void *k,
                     const void *v, const float *log_decay, const int32_t *seq_lens, int32_t batch,
                     int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, float scale, void *out, pa_stream_t stream);
size_t pa_linear_workspace_bytes(int32_t batch, int32_t num_kv_heads, int32_t head_dim, int32_t max_chunk);
int pa_linear_prefill(float *state, int32_t num_slots, const int32_t *state_slots, const void *q, const void *k,
                      const void *v, const float *log_decay, const int32_t *cu_q_lens, const int32_t *seq_lens,
                      int32_t batch, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t max_chunk, float scale,
                      void *workspace, void *out, pa_stream_t stream);

/*
 * pa_device_status -- synchronise `stream`, then read the device status word of the
 * current device into *flags (PA_DEV_* bits, 0 = clean), clearing it when `clear` != 0.
 * Returns PA_OK, PA_ERR_OUT_OF_RANGE or PA_ERR_TIMEOUT according to the bits (timeout
 * first), PA_ERR_INVALID_ARG for a NULL flags pointer, PA_ERR_CUDA on a CUDA error.
 */
int pa_device_status(uint32_t *flags, int32_t clear, pa_stream_t stream);

/*
 * pa_selftest_wait_timeout -- a check of the error path the device status describes: one
 * thread waits, through the same bounded-wait helper the kernels use, on an mbarrier that
 * nothing ever arrives on, gives up after `limit_cycles` SM cycles (1 .. 2^40) and sets
 * PA_DEV_TIMEOUT, so that pa_device_status afterwards returns PA_ERR_TIMEOUT.  Nothing faults
 * and the context stays usable.  Asynchronous on `stream`.  Returns PA_OK,
 * PA_ERR_INVALID_ARG for a limit outside the range, or PA_ERR_CUDA.
 */
int pa_selftest_wait_timeout(uint64_t limit_cycles, pa_stream_t stream);

/*
 * pa_selftest_packed_pairs -- a check of how pa_prefill_packed finds its work.  Its blocks take over one another's
 * work in an order that is the hardware's, so each finds the sequence of a pair of tiles from the pair's number, whatever
 * it found before: the pairs of pair_tokens (2 .. 256) tokens of the sequences, counted one after another, those
 * of a sequence from its end.  For each of pairs[0 .. n), one after another as one block would,
 *   out            [n, 3] int32 first row and length of its sequence and the pair's first token, or -1, -1, -1 past the last
 * cu_lens, num_tokens and max_len as in pa_prefill_packed, and reported alike.  Asynchronous on `stream`.
 */
int pa_selftest_packed_pairs(const int32_t *cu_lens, int32_t batch, int32_t num_tokens, int32_t max_len,
                             int32_t pair_tokens, const int32_t *pairs, int32_t n, int32_t *out,
                             pa_stream_t stream);

/*
 * pa_decode_splitkv_noalloc -- split-KV decode and its log-sum-exp merge in one call that
 * allocates nothing and takes no workspace: out = pa_combine(pa_decode_splitkv(...)).
 * The pages have no counterpart of this call; it exists for callers that cannot allocate
 * device memory -- an engine whose memory is a fixed arena owned by someone else, a plugin
 * in a host framework that exposes no allocator, or a serving loop that must never call
 * cudaMalloc on its hot path (an allocation there can synchronise the whole device).
 *   Arguments as pa_decode_splitkv plus out [batch, num_heads, head_dim] bf16.
 *   The partition results live in one static device array of pa_noalloc_scratch_bytes()
 *   bytes (8 MiB) inside the library, held by every GPU that loads the library until the
 *   process exits.  A request whose workspace (pa_splitkv_workspace_bytes) exceeds it
 *   returns PA_ERR_TOO_LARGE before any launch.
 *   The first call on a device looks up the array's device address (one-time set-up on that
 *   device); make that first call before capturing any stream into a CUDA graph.  The address
 *   is kept for the life of the process: after cudaDeviceReset on a device, do not call this
 *   entry point on that device again (the library's module, and the array, may have moved).
 *   Every call uses the same array, so calls that may run at the same time on the GPU
 *   (different streams, or different host threads) race and must be serialised by the
 *   caller.  Nothing needs clearing between calls: each call overwrites every slot it reads.
 */
int pa_decode_splitkv_noalloc(const pa_pool *pool, const void *q, const int32_t *block_tables, int32_t max_blocks,
                              const int32_t *seq_lens, int32_t batch, int32_t num_heads, float scale,
                              int32_t num_partitions, void *out, pa_stream_t stream);

/* Size in bytes of the static scratch array of pa_decode_splitkv_noalloc. */
size_t pa_noalloc_scratch_bytes(void);

/* Number of cluster splits pa_decode uses for this shape on the current device. */
int pa_decode_num_splits(int32_t batch, int32_t num_kv_heads, int32_t max_blocks);

/*
 * Partition count suggested for pa_decode_splitkv on the current device (1..16): the
 * largest count, at most 16, whose CTAs (batch x num_kv_heads x count) fill no more than
 * four fifths of one wave of four per SM, keeping >= 8 blocks per partition (the library
 * runs each partition on a thread-block cluster of up to 4 CTAs when the partitions alone
 * leave the wave at least half empty).
 */
int pa_splitkv_num_partitions(int32_t batch, int32_t num_kv_heads, int32_t max_blocks);

/* ------------------------------------------------------------------------------------
 * Host-side KV block manager (no GPU involved).  "Qwen3-4B / 8B / 32B", "Architecture
 * Notes": the paged KV cache uses full-lifetime admission (a request that cannot fit is
 * rejected rather than left to hang under memory pressure) and a prefix cache, on by
 * default; "Qwen3-32B Serving Load": the KV budget is profiled at load (21.4 GB, 5360
 * blocks); "Warm Prefix-Cache TTFT": a warm request computes only what its cached prompt
 * prefix does not cover.
 *
 * Bytes of one block (K and V of every layer): num_layers * 2 * num_kv_heads * block_size
 * * head_dim * dtype_bytes, and for the 8-bit pool (dtype_bytes 1) 2 more per layer and kv head,
 * its exponents.  Qwen3-32B (64 layers, 8 kv heads, d 128, bf16, 16-token blocks)
 * gives 4 MiB, so 5360 blocks are 22.48 GB (20.94 GiB).  0 on a non-positive argument.
 */
int64_t pa_kv_block_bytes(int32_t num_layers, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          int32_t dtype_bytes);
/* Blocks a budget of budget_bytes holds (floor). */
int32_t pa_kv_budget_blocks(int64_t budget_bytes, int32_t num_layers, int32_t num_kv_heads, int32_t head_dim,
                            int32_t block_size, int32_t dtype_bytes);

/* Opaque manager of num_blocks pool blocks of block_size tokens; thread-safe.  NULL on a
 * bad argument or no memory.  Destroy with pa_bm_destroy. */
typedef struct pa_blockmgr pa_blockmgr;
pa_blockmgr *pa_bm_create(int32_t num_blocks, int32_t block_size, int32_t enable_prefix_cache);
void pa_bm_destroy(pa_blockmgr *bm);

/*
 * Admit request_id with its prompt tokens[0, n_tokens) and at most max_new_tokens tokens to
 * generate.  The blocks for its whole lifetime (n_tokens + max_new_tokens) are reserved now,
 * or nothing is and PA_ERR_REJECTED is returned.  With the prefix cache, the prompt's leading
 * full blocks whose token ids (and every token before them) match a cached block are shared
 * instead of reserved; at least the prompt's last token is always left to compute.
 *   block_table      out: the request's block ids, in token order (table_cap entries or more)
 *   n_blocks         out: ceil((n_tokens + max_new_tokens) / block_size)
 *   n_cached_tokens  out: prompt tokens whose K/V is already in the pool (a multiple of
 *                    block_size); compute tokens [n_cached_tokens, n_tokens) next.
 * PA_ERR_INVALID_ARG on a bad argument or a request id already admitted.
 */
int pa_bm_admit(pa_blockmgr *bm, int64_t request_id, const int32_t *tokens, int32_t n_tokens,
                int32_t max_new_tokens, int32_t *block_table, int32_t table_cap, int32_t *n_blocks,
                int32_t *n_cached_tokens);

/*
 * pa_bm_admit_cow -- pa_bm_admit that also reuses a prefix hit ending inside a block.  After
 * the prompt's matching full blocks, the cached block that follows the same prefix and whose
 * leading tokens match the prompt's next tokens longest (k of them, 1 <= k <= 15, leaving the
 * prompt's last token to compute) lends its first k rows: they are to be copied into the
 * request's own block at that position (its table entry n_cached_tokens / 16), a copy on
 * write, since a cached block is never written.
 *   copy_src, copy_dst  out: n_copy slot pairs (block_size - 1 entries of room) for pa_kv_copy,
 *                       which must run before the request's tokens [n_cached_tokens, ...) are
 *                       appended and attended; n_copy = 0 when there is no partial hit
 *   n_cached_tokens     out: tokens whose K/V is in the pool once that copy has run (any count)
 * The source block is held (one reference) until the request is released, so no other
 * request can take it before the copy.  Other arguments and results as pa_bm_admit.
 */
int pa_bm_admit_cow(pa_blockmgr *bm, int64_t request_id, const int32_t *tokens, int32_t n_tokens,
                    int32_t max_new_tokens, int32_t *block_table, int32_t table_cap, int32_t *n_blocks,
                    int32_t *n_cached_tokens, int64_t *copy_src, int64_t *copy_dst, int32_t *n_copy);

/*
 * Append n_new generated tokens to the request's token list (within its reserved lifetime)
 * and declare that the K/V of its first `computed` tokens is now in the pool.  Blocks that
 * are full within those tokens enter the prefix cache (one entry per distinct content).
 */
int pa_bm_commit(pa_blockmgr *bm, int64_t request_id, const int32_t *new_tokens, int32_t n_new, int32_t computed);

/*
 * pa_bm_evict -- blocks block_ids[0, n) leave the request (one row of pa_kv_evict's `evicted`): its
 * table closes up as the device's does, they lose a user, and the request's tokens, positions
 * and reserved lifetime shrink by n blocks.  Nothing the request computes afterwards enters the
 * prefix cache (its K/V saw only part of the prompt); blocks that are cached already stay.
 * The ids must be full blocks of the request in the order of its table, else PA_ERR_INVALID_ARG
 * and nothing changes.
 */
int pa_bm_evict(pa_blockmgr *bm, int64_t request_id, const int32_t *block_ids, int32_t n);

/* Release the request: its blocks lose a user; cached ones stay reusable until the allocator
 * needs them (the one released longest ago first), the rest are free at once. */
int pa_bm_release(pa_blockmgr *bm, int64_t request_id);

/* Pool slots of the request's tokens [start, start + n): the slot_mapping of pa_kv_append. */
int pa_bm_slots(pa_blockmgr *bm, int64_t request_id, int32_t start, int32_t n, int64_t *slots);

/* Free (never used or uncached), cached-but-idle, and in-use block counts (any may be NULL). */
int pa_bm_stats(pa_blockmgr *bm, int32_t *free_blocks, int32_t *cached_idle_blocks, int32_t *used_blocks);

/* Human-readable name of a status code (static string). */
const char *pa_status_str(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
