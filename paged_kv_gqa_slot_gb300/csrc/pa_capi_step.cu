// pa_capi_step.cu -- the C ABI of a hybrid stack's step: packed prompts, tables grown and freed on the
// GPU, linear attention.  Argument validation only; nothing is launched on a bad argument.
#include <cmath>

#include "pagedattn.h"
#include "pa_internal.h"

using namespace pa;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// a device array that must be there
bool array_ok(const void* p, unsigned n) { return p && aligned(p, n); }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Rows `stride` elements apart that hold `width` elements each.
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride < (1LL << 39); }

// What the packed calls check alike; PA_OK with batch 0 or no row is a call with nothing to do.
int check_rows(const void* q, const void* k, const void* v, int32_t batch, int32_t num_tokens, int32_t num_heads,
               int32_t num_kv_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride, int64_t v_stride,
               float scale, const void* out) {
    if (batch < 0 || batch > 65535 || num_tokens < 0) return PA_ERR_INVALID_ARG;
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0) return PA_OK;
    if (!array_ok(q, 16) || !array_ok(k, 16) || !array_ok(v, 16) || !array_ok(out, 16)) return PA_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, (int64_t)num_heads * head_dim) || !stride_ok(k_stride, (int64_t)num_kv_heads * head_dim) ||
        !stride_ok(v_stride, (int64_t)num_kv_heads * head_dim))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

PackedArgs rows_of(const void* q, const void* k, const void* v, int32_t batch, int32_t num_tokens, int32_t num_heads,
                   int32_t num_kv_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                   float scale, void* out) {
    PackedArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.batch = batch;
    a.num_tokens = num_tokens;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    return a;
}

int check_state(const float* state, int32_t num_slots, const int32_t* state_slots, const float* log_decay,
                const int32_t* seq_lens) {
    if (num_slots <= 0 || !array_ok(state, 16) || !array_ok(state_slots, 4) || !array_ok(log_decay, 4) ||
        !array_ok(seq_lens, 4))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace

extern "C" {

int pa_prefill_packed(const void* q, const void* k, const void* v, const int32_t* cu_lens, int32_t batch,
                      int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t max_len, float scale, void* out,
                      pa_stream_t stream) {
    const int rc = check_rows(q, k, v, batch, num_tokens, num_heads, num_kv_heads, head_dim, q_stride, k_stride,
                              v_stride, scale, out);
    if (rc) return rc;
    if (max_len < 0) return PA_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0 || max_len == 0) return PA_OK;
    if (!array_ok(cu_lens, 4)) return PA_ERR_INVALID_ARG;
    PackedArgs a = rows_of(q, k, v, batch, num_tokens, num_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride,
                           scale, out);
    a.cu_lens = cu_lens;
    a.max_len = max_len < num_tokens ? max_len : num_tokens;
    a.status = device_status_ptr();
    if (!a.status) return PA_ERR_CUDA;
    return from_cuda(launch_prefill_packed(a, (cudaStream_t)stream));
}

int pa_selftest_packed_pairs(const int32_t* cu_lens, int32_t batch, int32_t num_tokens, int32_t max_len,
                             int32_t pair_tokens, const int32_t* pairs, int32_t n, int32_t* out, pa_stream_t stream) {
    if (batch <= 0 || batch > 65535 || num_tokens < 0 || max_len < 0 || pair_tokens < 2 || pair_tokens > 256 || n < 0)
        return PA_ERR_INVALID_ARG;
    if (!array_ok(cu_lens, 4)) return PA_ERR_INVALID_ARG;
    if (n == 0) return PA_OK;
    if (!array_ok(pairs, 4) || !array_ok(out, 4)) return PA_ERR_INVALID_ARG;
    PackedArgs a = {};
    a.cu_lens = cu_lens;
    a.batch = batch;
    a.num_tokens = num_tokens;
    a.max_len = max_len;
    a.status = device_status_ptr();
    if (!a.status) return PA_ERR_CUDA;
    return from_cuda(launch_selftest_pairs(a, pair_tokens, pairs, n, out, (cudaStream_t)stream));
}

int pa_kv_grow(int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens, const int32_t* new_lens,
               int32_t batch, const int32_t* free_blocks, int32_t capacity, const int32_t* num_free,
               int32_t max_tokens, int32_t* seq_lens_out, int32_t* num_free_out, int32_t* cu_lens,
               int64_t* slot_mapping, int32_t* positions, int32_t* token_seqs, pa_stream_t stream) {
    if (batch < 0 || batch > 65535 || capacity < 0 || max_tokens < 0 || max_blocks <= 0 || max_blocks > 0x7fffffff / 16)
        return PA_ERR_INVALID_ARG;
    if (!array_ok(num_free, 4) || !array_ok(num_free_out, 4) || !array_ok(cu_lens, 4)) return PA_ERR_INVALID_ARG;
    if (capacity > 0 && !array_ok(free_blocks, 4)) return PA_ERR_INVALID_ARG;
    if (batch > 0 && (!array_ok(block_tables, 4) || !array_ok(seq_lens, 4) || !array_ok(new_lens, 4) ||
                      !array_ok(seq_lens_out, 4)))
        return PA_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!array_ok(slot_mapping, 8) || !array_ok(positions, 4) || !array_ok(token_seqs, 4)))
        return PA_ERR_INVALID_ARG;
    GrowArgs a = {block_tables, seq_lens, new_lens, free_blocks, num_free, seq_lens_out, num_free_out, cu_lens,
                  slot_mapping, positions, token_seqs, device_status_ptr(), max_blocks, batch, capacity, max_tokens};
    if (!a.status) return PA_ERR_CUDA;
    return from_cuda(launch_grow(a, (cudaStream_t)stream));
}

int pa_kv_free(const int32_t* ids, const int32_t* counts, int32_t rows, int32_t width, int32_t* free_blocks,
               int32_t capacity, const int32_t* num_free, int32_t* num_free_out, pa_stream_t stream) {
    if (rows < 0 || width < 0 || capacity < 0) return PA_ERR_INVALID_ARG;
    if (width > kFreeMaxWidth) return PA_ERR_UNSUPPORTED;
    if (!array_ok(num_free, 4) || !array_ok(num_free_out, 4)) return PA_ERR_INVALID_ARG;
    if (rows > 0 && (!array_ok(counts, 4) || (width > 0 && !array_ok(ids, 4)))) return PA_ERR_INVALID_ARG;
    if (capacity > 0 && !array_ok(free_blocks, 4)) return PA_ERR_INVALID_ARG;
    FreeArgs a = {ids, counts, free_blocks, num_free, num_free_out, device_status_ptr(), rows, width, capacity};
    if (!a.status) return PA_ERR_CUDA;
    return from_cuda(launch_free(a, (cudaStream_t)stream));
}

int pa_linear_decode(float* state, int32_t num_slots, const int32_t* state_slots, const void* q, const void* k,
                     const void* v, const float* log_decay, const int32_t* seq_lens, int32_t batch,
                     int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, float scale, void* out, pa_stream_t stream) {
    int rc = check_rows(q, k, v, batch, batch, num_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride, scale,
                        out);
    if (rc) return rc;
    if (batch == 0) return PA_OK;
    rc = check_state(state, num_slots, state_slots, log_decay, seq_lens);
    if (rc) return rc;
    LinearArgs a = {rows_of(q, k, v, batch, batch, num_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride,
                            scale, out),
                    state, state_slots, log_decay, seq_lens, num_slots, 1};
    a.rows.max_len = 1;
    a.rows.status = device_status_ptr();
    if (!a.rows.status) return PA_ERR_CUDA;
    return from_cuda(launch_linear_decode(a, (cudaStream_t)stream));
}

size_t pa_linear_workspace_bytes(int32_t batch, int32_t num_kv_heads, int32_t head_dim, int32_t max_chunk) {
    if (batch <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_chunk <= 0) return 0;
    return linear_workspace(batch, num_kv_heads, head_dim, max_chunk);
}

int pa_linear_prefill(float* state, int32_t num_slots, const int32_t* state_slots, const void* q, const void* k,
                      const void* v, const float* log_decay, const int32_t* cu_q_lens, const int32_t* seq_lens,
                      int32_t batch, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t max_chunk, float scale,
                      void* workspace, void* out, pa_stream_t stream) {
    int rc = check_rows(q, k, v, batch, num_tokens, num_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride,
                        scale, out);
    if (rc) return rc;
    if (max_chunk < 0) return PA_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0 || max_chunk == 0) return PA_OK;
    rc = check_state(state, num_slots, state_slots, log_decay, seq_lens);
    if (rc) return rc;
    if (!array_ok(cu_q_lens, 4)) return PA_ERR_INVALID_ARG;
    LinearArgs a = {rows_of(q, k, v, batch, num_tokens, num_heads, num_kv_heads, head_dim, q_stride, k_stride,
                            v_stride, scale, out),
                    state, state_slots, log_decay, seq_lens, num_slots, max_chunk};
    a.rows.cu_lens = cu_q_lens;
    a.rows.max_len = max_chunk < num_tokens ? max_chunk : num_tokens;
    if (linear_workspace(batch, num_kv_heads, head_dim, max_chunk) > 0 && !array_ok(workspace, 16))
        return PA_ERR_INVALID_ARG;
    a.rows.status = device_status_ptr();
    if (!a.rows.status) return PA_ERR_CUDA;
    return from_cuda(launch_linear_prefill(a, workspace, (cudaStream_t)stream));
}

}  // extern "C"
