// C ABI of the calls for branching decode: argument validation and dispatch.
#include <cmath>
#include <cstdint>

#include "kda_tree.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool head_size_ok(int d) { return d == 64 || d == 128; }
bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }
bool tokens_ok(int t) { return t >= 1 && t <= kda::kTreeMax; }
bool eps_ok(float e) { return e >= 0.f && e <= 1e30f; }   // also rejects NaN

// Whether any of the arrays of 32-bit numbers `out` overlaps another of them or one of `in` (NULL: none).
struct Ints {
    const void *p;
    int64_t n;
};
template <size_t O, size_t I> bool overlap(const Ints (&out)[O], const Ints (&in)[I]) {
    auto meet = [](const Ints &a, const Ints &b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && x < y + 4 * (uintptr_t)b.n && y < x + 4 * (uintptr_t)a.n;
    };
    for (size_t i = 0; i < O; ++i) {
        for (size_t j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return true;
        for (const Ints &x : in)
            if (meet(out[i], x)) return true;
    }
    return false;
}

kda_status_t check_state_dims(const kda_dims_t *d, const int32_t *state_indices) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (!dtype_ok(d->dtype) || !head_size_ok(d->dk) || !head_size_ok(d->dv)) return KDA_ERR_UNSUPPORTED;
    if (d->batch <= 0 || d->heads <= 0 || d->num_seqs <= 0 || !tokens_ok(d->seqlen)) return KDA_ERR_SHAPE;
    if (state_indices == nullptr && d->num_seqs < d->batch) return KDA_ERR_SHAPE;
    if ((int64_t)d->batch * d->heads > 0x7fffffffLL / 4) return KDA_ERR_SHAPE;   // (up to four CTAs each)
    return KDA_OK;
}

kda_status_t check_cache_dims(const kda_paged_dims_t *d) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (!dtype_ok(d->dtype) || !head_size_ok(d->head_dim)) return KDA_ERR_UNSUPPORTED;
    if (d->rows < 0 || d->kv_heads <= 0 || d->pages <= 0 || d->page_size <= 0 || d->max_pages <= 0) return KDA_ERR_SHAPE;
    // positions within a row, and a token's place in the pool, as in the paged-cache calls
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL - 64 || (int64_t)d->pages * d->page_size > 0xffffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status_t check_attention_dims(int32_t tokens, const kda_paged_dims_t *d) {
    const kda_status_t st = check_cache_dims(d);
    if (st != KDA_OK) return st;
    if (!tokens_ok(tokens) || d->heads <= 0 || d->heads % d->kv_heads != 0) return KDA_ERR_SHAPE;
    // positions with the drafted tokens', rows of (page, offset, head), outputs: all 32-bit
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL - 1024 || (int64_t)d->pages * d->page_size * d->kv_heads > 0x7fffffffLL) return KDA_ERR_SHAPE;
    if ((int64_t)d->rows * d->heads * tokens > 0x7fffffffLL / 4) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status_t check_pool_dims(const kda_paged_dims_t *d) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (d->rows < 0 || d->rows > 65536 || d->pages <= 0 || d->pages > (1 << 22) || d->page_size <= 0 || d->max_pages <= 0) return KDA_ERR_SHAPE;
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL - 64 || (int64_t)d->rows * d->max_pages > 0x7fffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda::PagedTreeArgs attention_args(int32_t tokens, const kda_paged_dims_t *d) {
    kda::PagedTreeArgs a{};
    a.p.rows = d->rows, a.p.heads = d->heads, a.p.kv_heads = d->kv_heads;
    a.p.pages = d->pages, a.p.page_size = d->page_size, a.p.max_pages = d->max_pages;
    a.tokens = tokens;
    return a;
}

kda_status_t tree_run(const void *q, const void *k, const void *v, const void *g, const void *beta, float qk_eps,
                      float *state, const int32_t *state_indices, const int32_t *parents, const int32_t *num_tokens,
                      const int32_t *accepted, void *out, bool commit, const kda_dims_t *d, cudaStream_t stream) {
    const kda_status_t st = check_state_dims(d, state_indices);
    if (st != KDA_OK) return st;
    if (!k || !v || !g || !beta || !state || (commit ? !accepted : !q || !out)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, state, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    const void *ints[] = {state_indices, parents, num_tokens, accepted};
    for (const void *p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    const kda::TreeArgs a{q, k, v, g, beta, state, state_indices, parents, num_tokens, accepted, out,
                          d->batch, d->num_seqs, d->heads, d->seqlen, qk_eps};
    if (kda::debug_check_tree_inputs(a, d->dk, d->dtype, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const cudaError_t e = commit ? kda::launch_recurrent_tree_commit(a, d->dk, d->dv, d->dtype, stream)
                                 : kda::launch_recurrent_tree(a, d->dk, d->dv, d->dtype, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" kda_status_t kda_recurrent_tree(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                           const float *state, const int32_t *state_indices, const int32_t *parents,
                                           const int32_t *num_tokens, void *out, const kda_dims_t *d, cudaStream_t stream) {
    return tree_run(q, k, v, g, beta, -1.f, const_cast<float *>(state), state_indices, parents, num_tokens, nullptr, out, false, d, stream);
}

extern "C" kda_status_t kda_recurrent_tree_qknorm(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                                  float qk_eps, const float *state, const int32_t *state_indices,
                                                  const int32_t *parents, const int32_t *num_tokens, void *out,
                                                  const kda_dims_t *d, cudaStream_t stream) {
    if (!eps_ok(qk_eps)) return KDA_ERR_SHAPE;
    return tree_run(q, k, v, g, beta, qk_eps, const_cast<float *>(state), state_indices, parents, num_tokens, nullptr, out, false, d, stream);
}

extern "C" kda_status_t kda_recurrent_tree_commit(const void *k, const void *v, const void *g, const void *beta, float *state,
                                                  const int32_t *state_indices, const int32_t *parents,
                                                  const int32_t *num_tokens, const int32_t *accepted, const kda_dims_t *d,
                                                  cudaStream_t stream) {
    return tree_run(nullptr, k, v, g, beta, -1.f, state, state_indices, parents, num_tokens, accepted, nullptr, true, d, stream);
}

extern "C" kda_status_t kda_recurrent_tree_commit_qknorm(const void *k, const void *v, const void *g, const void *beta,
                                                         float qk_eps, float *state, const int32_t *state_indices,
                                                         const int32_t *parents, const int32_t *num_tokens,
                                                         const int32_t *accepted, const kda_dims_t *d, cudaStream_t stream) {
    if (!eps_ok(qk_eps)) return KDA_ERR_SHAPE;
    return tree_run(nullptr, k, v, g, beta, qk_eps, state, state_indices, parents, num_tokens, accepted, nullptr, true, d, stream);
}

extern "C" size_t kda_paged_tree_attention_workspace_bytes(int32_t tokens, const kda_paged_dims_t *d) {
    if (check_attention_dims(tokens, d) != KDA_OK) return 0;
    return kda::paged_tree_workspace_bytes(attention_args(tokens, d), d->head_dim, d->dtype);
}

extern "C" kda_status_t kda_paged_tree_attention_bounded(const void *q, const void *k_cache, const void *v_cache,
                                                         const int32_t *block_table, const int32_t *seq_lens,
                                                         const int32_t *parents, const int32_t *num_tokens, int32_t tokens,
                                                         float scale, void *out, float *lse, void *workspace,
                                                         size_t workspace_bytes, uint32_t wait_polls,
                                                         const kda_paged_dims_t *d, cudaStream_t stream) {
    const kda_status_t st = check_attention_dims(tokens, d);
    if (st != KDA_OK) return st;
    if (!std::isfinite(scale)) return KDA_ERR_SHAPE;
    if (d->rows == 0) return KDA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k_cache, v_cache, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    const void *ints[] = {block_table, seq_lens, parents, num_tokens, lse};
    for (const void *p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    const size_t need = kda_paged_tree_attention_workspace_bytes(tokens, d);
    if (need > 0) {
        if (workspace == nullptr) return KDA_ERR_NULL;
        if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
    }
    kda::PagedTreeArgs a = attention_args(tokens, d);
    a.p.q = q, a.p.k_cache = k_cache, a.p.v_cache = v_cache, a.p.table = block_table, a.p.lens = seq_lens;
    a.p.out = out, a.p.lse = lse, a.p.scale = scale;
    a.parents = parents, a.num = num_tokens;
    return kda::launch_paged_tree(a, d->head_dim, d->dtype, workspace, wait_polls, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_paged_tree_attention(const void *q, const void *k_cache, const void *v_cache,
                                                 const int32_t *block_table, const int32_t *seq_lens,
                                                 const int32_t *parents, const int32_t *num_tokens, int32_t tokens,
                                                 float scale, void *out, float *lse, void *workspace,
                                                 size_t workspace_bytes, const kda_paged_dims_t *d, cudaStream_t stream) {
    return kda_paged_tree_attention_bounded(q, k_cache, v_cache, block_table, seq_lens, parents, num_tokens, tokens, scale, out, lse,
                                            workspace, workspace_bytes, 1u << 20, d, stream);
}

extern "C" kda_status_t kda_paged_tree_commit(void *k_cache, void *v_cache, const int32_t *block_table,
                                              const int32_t *seq_lens, const int32_t *parents, const int32_t *num_tokens,
                                              const int32_t *accepted, int32_t tokens, int32_t *new_lens,
                                              const kda_paged_dims_t *d, cudaStream_t stream) {
    const kda_status_t st = check_cache_dims(d);
    if (st != KDA_OK) return st;
    if (!tokens_ok(tokens) || (int64_t)d->max_pages * d->page_size > 0x7fffffffLL - 1024) return KDA_ERR_SHAPE;
    if (d->rows == 0) return KDA_OK;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !accepted) return KDA_ERR_NULL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return KDA_ERR_ALIGN;
    const void *ints[] = {block_table, seq_lens, parents, num_tokens, accepted, new_lens};
    for (const void *p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    const int64_t rows = d->rows;
    const Ints in[] = {{block_table, rows * d->max_pages}, {seq_lens == new_lens ? nullptr : seq_lens, rows}, {parents, rows * tokens},
                       {num_tokens, rows}, {accepted, rows}};
    const Ints out[] = {{new_lens, rows}};
    if (overlap(out, in)) return KDA_ERR_SHAPE;   // (a row's CTA would read what another has written)
    const int64_t vecs = (int64_t)d->kv_heads * d->head_dim * (d->dtype == KDA_F32 ? 4 : 2) / 16;
    if (vecs > 0x7fffffffLL / 64) return KDA_ERR_SHAPE;
    const kda::TreeCommitArgs a{k_cache, v_cache, block_table, seq_lens, parents, num_tokens, accepted, new_lens,
                                d->rows, tokens, d->pages, d->page_size, d->max_pages, (int32_t)vecs};
    return kda::launch_tree_commit(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_paged_fork(const int32_t *block_table, const int32_t *seq_lens, const int32_t *page_refs,
                                       const int32_t *sources, const int32_t *new_tokens, int32_t *new_table,
                                       int32_t *new_lens, int32_t *new_refs, int32_t *copies, int32_t *short_of,
                                       const kda_paged_dims_t *d, cudaStream_t stream) {
    const kda_status_t st = check_pool_dims(d);
    if (st != KDA_OK) return st;
    if (d->rows == 0 || d->max_pages > (1 << 30)) return KDA_ERR_SHAPE;   // (entries of a row, and a segment past them, are 32-bit)
    const int64_t rows = d->rows, entries = rows * d->max_pages;
    const Ints in[] = {{block_table, entries}, {seq_lens, rows}, {page_refs, d->pages}, {sources, rows}, {new_tokens, rows}};
    const Ints out[] = {{new_table, entries}, {new_lens, rows}, {new_refs, d->pages}, {copies, 2 * rows}, {short_of, 1}};
    for (const Ints &x : in)
        if (!x.p && &x != &in[4]) return KDA_ERR_NULL;   // (new_tokens may be)
    for (const Ints &x : out)
        if (!x.p) return KDA_ERR_NULL;
    for (const Ints &x : in)
        if (!aligned(x.p, 4)) return KDA_ERR_ALIGN;
    for (const Ints &x : out)
        if (!aligned(x.p, 4)) return KDA_ERR_ALIGN;
    if (overlap(out, in)) return KDA_ERR_SHAPE;
    const kda::ForkArgs a{block_table, seq_lens, page_refs, sources, new_tokens, new_table, new_lens, new_refs, copies, short_of,
                          d->rows, d->pages, d->page_size, d->max_pages};
    return kda::launch_fork(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_paged_compact(const int32_t *block_table, const int32_t *page_refs, int32_t *new_table,
                                          int32_t *new_refs, int32_t *copies, const kda_paged_dims_t *d, cudaStream_t stream) {
    const kda_status_t st = check_pool_dims(d);
    if (st != KDA_OK) return st;
    if (!page_refs || !new_refs || (d->rows > 0 && (!block_table || !new_table)) || (d->pages > 1 && !copies)) return KDA_ERR_NULL;
    const void *ints[] = {block_table, page_refs, new_table, new_refs, copies};
    for (const void *p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    const int64_t entries = (int64_t)d->rows * d->max_pages;
    const Ints in[] = {{block_table, entries}, {page_refs, d->pages}};
    const Ints out[] = {{new_table, entries}, {new_refs, d->pages}, {copies, d->pages / 2 * 2}};
    if (overlap(out, in)) return KDA_ERR_SHAPE;
    const kda::ForkArgs a{block_table, nullptr, page_refs, nullptr, nullptr, new_table, nullptr, new_refs, copies, nullptr,
                          d->rows, d->pages, d->page_size, d->max_pages};
    return kda::launch_compact(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_paged_copy(void *k_cache, void *v_cache, const int32_t *copies, int64_t count,
                                       const kda_paged_dims_t *d, cudaStream_t stream) {
    if (d == nullptr) return KDA_ERR_NULL;
    if (!dtype_ok(d->dtype) || !head_size_ok(d->head_dim)) return KDA_ERR_UNSUPPORTED;
    if (d->kv_heads <= 0 || d->pages <= 0 || d->page_size <= 0 || count < 0 || count > 0x7fffffffLL) return KDA_ERR_SHAPE;
    if ((int64_t)d->pages * d->page_size > 0xffffffffLL) return KDA_ERR_SHAPE;
    if (count == 0) return KDA_OK;
    if (!k_cache || !v_cache || !copies) return KDA_ERR_NULL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(copies, 4)) return KDA_ERR_ALIGN;
    const int64_t vecs = (int64_t)d->page_size * d->kv_heads * (d->head_dim * (d->dtype == KDA_F32 ? 4 : 2) / 16);
    return kda::launch_page_copy(k_cache, v_cache, copies, count, vecs, d->pages, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
