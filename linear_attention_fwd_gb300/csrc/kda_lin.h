// Internal declarations of the linear-attention and paged-cache calls.
#pragma once

#include "kda_internal.h"

namespace kda {

// SMs of the GPU this library is written for: how far work is split is chosen against it, on the
// host, without asking the device (so that workspace sizes are plain arithmetic).
constexpr int kSms = 152;

struct LinArgs {
    const void *q, *k, *v;
    const float *g;           // [tokens, H] or nullptr
    const float *head_g;      // [H] or nullptr
    const float *s0;          // [N, H, dk, dv] or nullptr
    const int32_t *cu;        // [N + 1] or nullptr (dense)
    void *out;
    float *sT;                // [N, H, dk, dv] or nullptr
    int64_t seqlen;           // tokens per dense row, or total packed tokens
    int32_t num_seqs, heads, qk_heads, dk, dv;
    uint32_t wait_polls;      // bound on each device wait of the tensor-core kernel (polls)
};

struct LinStepArgs {
    const void *q, *k, *v;
    const float *g, *head_g;
    float *state;
    const int32_t *idx;
    void *out;
    int32_t rows, slots, heads, qk_heads;
};

// Token range of sequence n, clamped so that malformed offsets never index outside the tensors.
__device__ __forceinline__ void lin_range(const LinArgs &a, int n, int64_t &bos, int64_t &eos) {
    if (a.cu == nullptr) {
        bos = (int64_t)n * a.seqlen;
        eos = bos + a.seqlen;
    } else {
        int64_t b = __ldg(a.cu + n), e = __ldg(a.cu + n + 1);
        b = b < 0 ? 0 : (b > a.seqlen ? a.seqlen : b);
        e = e < b ? b : (e > a.seqlen ? a.seqlen : e);
        bos = b;
        eos = e;
    }
}

// Sums of log decays are kept as two floats (large part, rest), so that differences of them are exact to
// fp32 whatever their magnitude.
// (h, l) + (x, y): the sum of the large parts is split exactly, the small parts are added.
__device__ __forceinline__ void add2f(float &h, float &l, float x, float y) {
    const float s = h + x, b = s - h;
    l += y + ((h - (s - b)) + (x - b));
    h = s;
}
// A token's log decay g + hg in log2 units, 0 where `in` is false.  Below -1e5 it is that: the decay is zero
// in every format and the sums stay finite.  (NaN passes through.)
__device__ __forceinline__ void log2_decay(float g, float hg, bool in, float &hi, float &lo) {
    constexpr float kL = 1.44269502e+00f, kLl = 1.92596299e-08f;   // log2 e = kL + kLl
    const float s = g + hg, b = s - g, e = (g - (s - b)) + (hg - b);
    hi = s * kL;
    lo = fmaf(s, kL, -hi) + fmaf(s, kLl, e * kL);
    if (s < -6.9e4f) {
        hi = -1e5f;
        lo = 0.f;
    }
    if (!in) hi = lo = 0.f;
}

struct PagedArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *table, *lens;
    void *out;
    float *lse;
    float scale;
    int32_t rows, heads, kv_heads, pages, page_size, max_pages;
};

struct AppendArgs {
    const void *k, *v;
    void *k_cache, *v_cache;
    const int32_t *table, *positions, *cu;
    int64_t tokens;
    int32_t rows, pages, page_size, max_pages;
    int32_t row_vecs;         // 16-byte vectors of one token's keys (kv_heads * head_dim * size / 16)
};

// As debug_check_inputs, for linear attention: g [tokens, heads] + head_g [heads] at most 0 (either may be
// nullptr), packed offsets.
cudaError_t debug_check_lin_inputs(const float *g, const float *head_g, int64_t tokens, int heads, const int32_t *cu,
                                   int num_seqs, int64_t seqlen, cudaStream_t st);
cudaError_t launch_lin_chunk_simt(const LinArgs &a, cudaStream_t st);   // fp32
// bf16.  Sequences may be cut into parts that run side by side, which takes a workspace; `whole`: they
// are not.
cudaError_t launch_lin_chunk_tc(const LinArgs &a, void *workspace, bool whole, cudaStream_t st);
size_t lin_chunk_tc_workspace_bytes(int64_t tokens, int64_t num_seqs, int64_t heads, int dk, int dv, bool packed);
// Waits for `st`, then reads and clears the count of expired bounded waits of that kernel.
cudaError_t take_lin_expiries(cudaStream_t st, unsigned int *count);
cudaError_t launch_lin_step(const LinStepArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st);
cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st);
size_t paged_attention_workspace_bytes(int64_t rows, int heads, int kv_heads, int64_t max_tokens, int d, kda_dtype_t dt);
cudaError_t launch_paged_attention(const PagedArgs &a, int d, kda_dtype_t dt, void *workspace, cudaStream_t st);

}  // namespace kda
