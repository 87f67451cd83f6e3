// Internal declarations of the calls for branching decode.
#pragma once

#include "kda_lin.h"

namespace kda {

constexpr int kTreeMax = KDA_TREE_TOKENS;

// The drafted token that token i of row n continues, -1 for none.
__device__ __forceinline__ int tree_parent(const int32_t *parents, int tokens, int n, int i) {
    if (parents == nullptr) return i - 1;
    const int p = __ldg(parents + (int64_t)n * tokens + i);
    return p < 0 || p >= i ? -1 : p;
}
// Drafted tokens of row n.
__device__ __forceinline__ int tree_count(const int32_t *num, int tokens, int n) {
    if (num == nullptr) return tokens;
    const int m = __ldg(num + n);
    return m < 0 ? 0 : (m < tokens ? m : tokens);
}

struct TreeArgs {
    const void *q, *k, *v, *g, *beta;
    float *state;
    const int32_t *idx, *parents, *num, *accepted;
    void *out;
    int32_t rows, slots, heads, tokens;
    float qk_eps;             // >= 0: q and k L2-normalised first
};

struct PagedTreeArgs {
    PagedArgs p;              // q, out and lse hold `tokens` drafted tokens per row
    const int32_t *parents, *num;
    int32_t tokens;
};

struct TreeCommitArgs {
    void *k_cache, *v_cache;
    const int32_t *table, *lens, *parents, *num, *accepted;
    int32_t *new_lens;
    int32_t rows, tokens, pages, page_size, max_pages;
    int32_t row_vecs;         // 16-byte vectors of one token's keys
};

struct ForkArgs {
    const int32_t *table, *lens, *refs, *sources, *new_tokens;
    int32_t *new_table, *new_lens, *new_refs, *copies, *short_of;
    int32_t rows, pages, page_size, max_pages;
};

cudaError_t launch_recurrent_tree(const TreeArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st);
cudaError_t launch_recurrent_tree_commit(const TreeArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st);
// Debug-build check of the log decays (see debug_check_inputs): at most 0, of the tokens that the call uses.
cudaError_t debug_check_tree_inputs(const TreeArgs &a, int dk, kda_dtype_t dt, cudaStream_t st);
size_t paged_tree_workspace_bytes(const PagedTreeArgs &a, int d, kda_dtype_t dt);
// polls: bound on each device wait of the tensor-core kernel (bf16)
cudaError_t launch_paged_tree(const PagedTreeArgs &a, int d, kda_dtype_t dt, void *workspace, uint32_t polls, cudaStream_t st);
// Waits for `st`, then reads and clears the count of expired bounded waits of that kernel.
cudaError_t take_tree_expiries(cudaStream_t st, unsigned int *count);
cudaError_t launch_tree_commit(const TreeCommitArgs &a, cudaStream_t st);
cudaError_t launch_fork(const ForkArgs &a, cudaStream_t st);
cudaError_t launch_compact(const ForkArgs &a, cudaStream_t st);
// page_vecs: 16-byte vectors of one page's keys
cudaError_t launch_page_copy(void *k_cache, void *v_cache, const int32_t *copies, int64_t count, int64_t page_vecs, int pages, cudaStream_t st);

}  // namespace kda
