// Paged key-value cache: append, and attention of one new token per row.
#include "kda_lin.h"

namespace kda {
namespace {

// ------------------------------------------------------------------ append
// A CTA moves kTokens consecutive tokens: one thread per token finds the token's place (row by
// bisection in the offsets, then page and offset), then all threads copy 16-byte vectors.  Bound
// by one read and one write of the new rows.
constexpr int kTokens = 8, kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) kda_paged_append_kernel(AppendArgs a) {
    __shared__ int64_t place[kTokens];   // the token's index in the cache, or -1
    const int64_t u0 = (int64_t)blockIdx.x * kTokens;
    if (threadIdx.x < kTokens) {
        const int64_t u = u0 + threadIdx.x;
        int64_t at = -1;
        if (u < a.tokens) {
            int row = (int)u;
            int64_t first = u;
            if (a.cu) {   // the last row that starts at or before u
                int lo = 0, hi = a.rows;   // cu[lo] <= u < cu[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (__ldg(a.cu + mid) <= u) lo = mid;
                    else hi = mid;
                }
                row = lo;
                first = __ldg(a.cu + lo);
                if (first > u || __ldg(a.cu + lo + 1) <= u) row = -1;
                if (first < 0) first = 0;
            }
            if (row >= 0) {
                const int64_t p = (int64_t)__ldg(a.positions + row) + (u - first);
                if (p >= 0 && p < (int64_t)a.max_pages * a.page_size) {
                    const int pg = (int)p / a.page_size;
                    const int page = __ldg(a.table + (int64_t)row * a.max_pages + pg);
                    if (page >= 0 && page < a.pages) at = (int64_t)page * a.page_size + ((int)p - pg * a.page_size);
                }
            }
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();
    const uint4 *k = static_cast<const uint4 *>(a.k), *v = static_cast<const uint4 *>(a.v);
    uint4 *kc = static_cast<uint4 *>(a.k_cache), *vc = static_cast<uint4 *>(a.v_cache);
    for (int x = threadIdx.x; x < kTokens * a.row_vecs; x += kAppendThreads) {
        const int tk = x / a.row_vecs, c = x - tk * a.row_vecs;
        const int64_t at = place[tk];
        if (at < 0) continue;
        const int64_t src = (u0 + tk) * a.row_vecs + c, dst = at * a.row_vecs + c;
        const uint4 kv = __ldcs(k + src), vv = __ldcs(v + src);
        kc[dst] = kv;
        vc[dst] = vv;
    }
}

// ------------------------------------------------------------------ attention
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One CTA per (row, query head); warps take tokens in turn, a lane holds D / 32 channels, and
// each warp keeps its own running maximum and sum; they are joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) kda_paged_attention_kernel(PagedArgs a) {
    constexpr int PER = D / 32;
    const int n = blockIdx.x / a.heads, h = blockIdx.x % a.heads, hk = h / (a.heads / a.kv_heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *q = static_cast<const T *>(a.q) + ((int64_t)n * a.heads + h) * D;
    const T *kc = static_cast<const T *>(a.k_cache), *vc = static_cast<const T *>(a.v_cache);
    int len = a.lens[n];
    len = len < 0 ? 0 : (len > a.max_pages * a.page_size ? a.max_pages * a.page_size : len);
    float qr[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        qr[e] = to_f(q[lane + 32 * e]);
        o[e] = 0.f;
    }
    const float sc = a.scale * kLog2e;
    for (int t = warp; t < len; t += kWarps) {
        const int pg = t / a.page_size;
        const int page = __ldg(a.table + (int64_t)n * a.max_pages + pg);
        if (page < 0 || page >= a.pages) continue;
        const int64_t at = (((int64_t)page * a.page_size + (t - pg * a.page_size)) * a.kv_heads + hk) * D + lane;
        float s = 0.f, vv[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            s = fmaf(qr[e], to_f(kc[at + 32 * e]), s);
            vv[e] = to_f(vc[at + 32 * e]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= sc;
        const float mn = fmaxf(m, s);
        const float at0 = mn == -INFINITY ? 0.f : mn;   // scores of -infinity weigh nothing
        const float f = exp2f(m - at0), p = exp2f(s - at0);
        m = mn;
        l = fmaf(l, f, p);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(o[e], f, p * vv[e]);
    }
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) sm_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w]);
    float f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        f[w] = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - mx);
        sum = fmaf(sm_l[w], f[w], sum);
    }
    T *out = static_cast<T *>(a.out) + ((int64_t)n * a.heads + h) * D;
    for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x = fmaf(sm_o[w][c], f[w], x);
        out[c] = from_f<T>(sum > 0.f ? x / sum : 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)n * a.heads + h] = sum > 0.f ? mx * kLn2 + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st) {
    const int64_t grid = (a.tokens + kTokens - 1) / kTokens;
    kda_paged_append_kernel<<<(unsigned)grid, kAppendThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_attention(const PagedArgs &a, int d, kda_dtype_t dt, void *workspace, cudaStream_t st) {
    (void)workspace;
    const unsigned grid = (unsigned)(a.rows * a.heads);
    if (dt == KDA_F32) {
        if (d == 128) kda_paged_attention_kernel<float, 128><<<grid, 32 * kWarps, 0, st>>>(a);
        else kda_paged_attention_kernel<float, 64><<<grid, 32 * kWarps, 0, st>>>(a);
    } else {
        if (d == 128) kda_paged_attention_kernel<__nv_bfloat16, 128><<<grid, 32 * kWarps, 0, st>>>(a);
        else kda_paged_attention_kernel<__nv_bfloat16, 64><<<grid, 32 * kWarps, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda
