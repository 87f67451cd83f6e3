// C ABI of the linear-attention and paged-cache calls: argument validation and dispatch.
#include <cmath>
#include <cstdint>

#include "kda_lin.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool head_size_ok(int d) { return d == 64 || d == 128; }
bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }

kda_status_t check_lin_dims(const kda_lin_dims_t *d) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (!dtype_ok(d->dtype) || !head_size_ok(d->dk) || !head_size_ok(d->dv)) return KDA_ERR_UNSUPPORTED;
    if (d->heads <= 0 || d->qk_heads <= 0 || d->heads % d->qk_heads != 0 || d->heads > (1 << 17) || d->num_seqs <= 0) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status_t check_paged_dims(const kda_paged_dims_t *d) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (!dtype_ok(d->dtype) || !head_size_ok(d->head_dim)) return KDA_ERR_UNSUPPORTED;
    if (d->rows < 0 || d->kv_heads <= 0 || d->pages <= 0 || d->page_size <= 0 || d->max_pages <= 0) return KDA_ERR_SHAPE;
    // a position within a row, and with the sign bit a token's place in the pool, are 32-bit
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL - 64 || (int64_t)d->pages * d->page_size > 0xffffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

}  // namespace

extern "C" size_t kda_lin_chunk_fwd_workspace_bytes(const kda_lin_dims_t *d, int packed) {
    if (check_lin_dims(d) != KDA_OK || d->batch <= 0 || d->seqlen <= 0 || d->dtype != KDA_BF16) return 0;
    return kda::lin_chunk_tc_workspace_bytes((int64_t)d->batch * d->seqlen, d->num_seqs, d->heads, d->dk, d->dv, packed != 0);
}

extern "C" kda_status_t kda_lin_chunk_fwd_bounded(const void *q, const void *k, const void *v, const float *g,
                                                  const float *head_g, const float *initial_state,
                                                  const int32_t *cu_seqlens, void *out, float *final_state,
                                                  void *workspace, size_t workspace_bytes, uint32_t wait_polls,
                                                  const kda_lin_dims_t *d, cudaStream_t stream) {
    kda_status_t st = check_lin_dims(d);
    if (st != KDA_OK) return st;
    if (d->batch <= 0 || d->seqlen < 0) return KDA_ERR_SHAPE;
    if (cu_seqlens == nullptr ? d->num_seqs != d->batch : d->batch != 1) return KDA_ERR_SHAPE;
    const int64_t tokens = (int64_t)d->batch * d->seqlen;
    if (tokens > 0x7fffffffLL - 64 || (int64_t)d->num_seqs * d->heads > 0x7fffffffLL / 4) return KDA_ERR_SHAPE;
    if (tokens > 0 && (!q || !k || !v || !out)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, out, initial_state, final_state};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(g, 4) || !aligned(head_g, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    if (initial_state && final_state && initial_state != final_state) {
        const char *x = reinterpret_cast<const char *>(initial_state), *y = reinterpret_cast<const char *>(final_state);
        const int64_t bytes = (int64_t)d->num_seqs * d->heads * d->dk * d->dv * 4;
        if (x < y + bytes && y < x + bytes) return KDA_ERR_SHAPE;   // partial overlap
    }
    const size_t need = kda_lin_chunk_fwd_workspace_bytes(d, cu_seqlens != nullptr);
    if (need > 0) {
        if (workspace == nullptr) return KDA_ERR_NULL;
        if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
    }
    if (kda::debug_check_lin_inputs(g, head_g, tokens, d->heads, cu_seqlens, d->num_seqs, d->seqlen, stream) != cudaSuccess) return KDA_ERR_CUDA;
    if (tokens == 0) {
        if (final_state == nullptr || final_state == initial_state) return KDA_OK;
        const size_t bytes = (size_t)d->num_seqs * d->heads * d->dk * d->dv * 4;
        const cudaError_t e = initial_state
            ? cudaMemcpyAsync(final_state, initial_state, bytes, cudaMemcpyDeviceToDevice, stream)
            : cudaMemsetAsync(final_state, 0, bytes, stream);
        return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    const kda::LinArgs a{q, k, v, g, head_g, initial_state, cu_seqlens, out, final_state,
                         (int64_t)d->seqlen, d->num_seqs, d->heads, d->qk_heads, d->dk, d->dv, wait_polls};
    // in place, a sequence's last part would write the state that its other parts start from
    const bool whole = initial_state && initial_state == final_state;
    const cudaError_t e = d->dtype == KDA_BF16 ? kda::launch_lin_chunk_tc(a, workspace, whole, stream)
                                               : kda::launch_lin_chunk_simt(a, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_lin_chunk_fwd(const void *q, const void *k, const void *v, const float *g,
                                          const float *head_g, const float *initial_state,
                                          const int32_t *cu_seqlens, void *out, float *final_state,
                                          void *workspace, size_t workspace_bytes, const kda_lin_dims_t *d,
                                          cudaStream_t stream) {
    return kda_lin_chunk_fwd_bounded(q, k, v, g, head_g, initial_state, cu_seqlens, out, final_state, workspace,
                                     workspace_bytes, 1u << 20, d, stream);
}

extern "C" kda_status_t kda_lin_recurrent_step(const void *q, const void *k, const void *v, const float *g,
                                               const float *head_g, float *state, const int32_t *state_indices,
                                               void *out, const kda_lin_dims_t *d, cudaStream_t stream) {
    kda_status_t st = check_lin_dims(d);
    if (st != KDA_OK) return st;
    if (d->seqlen != 1 || d->batch < 0) return KDA_ERR_SHAPE;
    if (state_indices == nullptr && d->num_seqs < d->batch) return KDA_ERR_SHAPE;
    if ((int64_t)d->batch * d->heads > 0x7fffffffLL / 4) return KDA_ERR_SHAPE;
    if (d->batch == 0) return KDA_OK;
    if (!q || !k || !v || !state || !out) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, out, state};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(g, 4) || !aligned(head_g, 4) || !aligned(state_indices, 4)) return KDA_ERR_ALIGN;
    const kda::LinStepArgs a{q, k, v, g, head_g, state, state_indices, out, d->batch, d->num_seqs, d->heads, d->qk_heads};
    cudaError_t e = kda::debug_check_lin_inputs(g, head_g, d->batch, d->heads, nullptr, 0, 0, stream);
    if (e == cudaSuccess) e = kda::launch_lin_step(a, d->dk, d->dv, d->dtype, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_paged_append(const void *k, const void *v, void *k_cache, void *v_cache,
                                         const int32_t *block_table, const int32_t *positions,
                                         const int32_t *cu_seqlens, int64_t tokens, const kda_paged_dims_t *d,
                                         cudaStream_t stream) {
    kda_status_t st = check_paged_dims(d);
    if (st != KDA_OK) return st;
    if (tokens < 0 || tokens > 0x7fffffffLL || (cu_seqlens == nullptr && tokens != d->rows)) return KDA_ERR_SHAPE;
    if (tokens == 0 || d->rows == 0) return KDA_OK;
    if (!k || !v || !k_cache || !v_cache || !block_table || !positions) return KDA_ERR_NULL;
    const void *ptrs[] = {k, v, k_cache, v_cache};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(block_table, 4) || !aligned(positions, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    const int64_t vecs = (int64_t)d->kv_heads * d->head_dim * (d->dtype == KDA_F32 ? 4 : 2) / 16;
    if (vecs > 0x7fffffffLL / 64) return KDA_ERR_SHAPE;
    const kda::AppendArgs a{k, v, k_cache, v_cache, block_table, positions, cu_seqlens, tokens,
                            d->rows, d->pages, d->page_size, d->max_pages, (int32_t)vecs};
    return kda::launch_paged_append(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" size_t kda_paged_attention_workspace_bytes(const kda_paged_dims_t *d) {
    if (check_paged_dims(d) != KDA_OK || d->heads <= 0 || d->heads % d->kv_heads != 0) return 0;
    return kda::paged_attention_workspace_bytes(d->rows, d->heads, d->kv_heads, (int64_t)d->max_pages * d->page_size,
                                                d->head_dim, d->dtype);
}

extern "C" kda_status_t kda_paged_attention(const void *q, const void *k_cache, const void *v_cache,
                                            const int32_t *block_table, const int32_t *seq_lens, float scale,
                                            void *out, float *lse, void *workspace, size_t workspace_bytes,
                                            const kda_paged_dims_t *d, cudaStream_t stream) {
    kda_status_t st = check_paged_dims(d);
    if (st != KDA_OK) return st;
    if (d->heads <= 0 || d->heads % d->kv_heads != 0 || !std::isfinite(scale)) return KDA_ERR_SHAPE;
    if ((int64_t)d->rows * d->heads > 0x7fffffffLL / 4) return KDA_ERR_SHAPE;
    if (d->rows == 0) return KDA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k_cache, v_cache, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
    const size_t need = kda_paged_attention_workspace_bytes(d);
    if (need > 0) {
        if (workspace == nullptr) return KDA_ERR_NULL;
        if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
    }
    const kda::PagedArgs a{q, k_cache, v_cache, block_table, seq_lens, out, lse, scale,
                           d->rows, d->heads, d->kv_heads, d->pages, d->page_size, d->max_pages};
    return kda::launch_paged_attention(a, d->head_dim, d->dtype, workspace, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
