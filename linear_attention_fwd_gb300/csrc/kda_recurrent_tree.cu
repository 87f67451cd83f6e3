// KDA for a tree of drafted tokens: every token's output from an unchanged state (verify), and the accepted
// path brought into the state (commit).
//
// Verify.  With E_ij = exp of the sum of g over the path from j (excluded) to i and E_i over the whole path
// ("はじめての自然言語処理 -- Kimi K3", section 3.1, the chunkwise form, with a tree in the place of a line),
//   u_i = beta_i (v_i - (E_i k_i)^T S) - sum_{j in A(i), j != i} beta_i (k_i . E_ij k_j) u_j,
//   o_i = (E_i q_i)^T S + sum_{j in A(i)} (q_i . E_ij k_j) u_j,
// so that the state is read once and no token's own state is formed.  A CTA takes a row's head:
//  1. the state is requested straight into B fragments (each warp the 16 value channels that it keeps to the
//     end), then the tokens' keys and decays are put into shared memory;
//  2. eight lanes walk a token's path to its root with the running product of the decays: every factor is
//     at most 1, no exponent of a sum is taken, and lines of 64 tokens need no bound on g.  They leave the two
//     coefficients of each pair, E_i k_i and E_i q_i;
//  3. (E k; E q) S on tensor cores (mma.sync, tf32; fp32 calls: three products of parts of 11 bits);
//  4. each warp solves for its channels' u in the order of the tokens' depth, and adds up the outputs as it goes,
//     without a barrier: four tokens of a depth at a time.
// Bound by reading the state: 64 KB per row and head at 128 x 128.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "kda_internal.h"
#include "kda_tree.h"

namespace kda {
namespace {

__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t y;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return y;
}
// D (16 x 8) += A (16 x 8) B (8 x 8), tf32 with fp32 sums
__device__ __forceinline__ void mma_1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T> __device__ __forceinline__ float4 load4(const T *p);
template <> __device__ __forceinline__ float4 load4<float>(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162 *>(&u.x), b = *reinterpret_cast<const __nv_bfloat162 *>(&u.y);
    const float2 x = __bfloat1622float2(a), y = __bfloat1622float2(b);
    return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }
__device__ __forceinline__ float4 mul4(float4 a, float b) { return make_float4(a.x * b, a.y * b, a.z * b, a.w * b); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) { return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c)))); }

// An operand as it is kept: rounded to tf32 once (fp32 calls split it where it is used).
template <bool kF32> __device__ __forceinline__ float4 operand(float4 x) {
    if constexpr (kF32) return x;
    return make_float4(__uint_as_float(tf32(x.x)), __uint_as_float(tf32(x.y)), __uint_as_float(tf32(x.z)), __uint_as_float(tf32(x.w)));
}

// Sum over the eight lanes of a group (every lane of the warp takes part).
__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

// A row of DK channels on eight lanes: lane l holds channels 32 m + 4 l .. + 3.
template <int DK> struct Row {
    float4 x[DK / 32];
    __device__ __forceinline__ float norm2() const {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < DK / 32; ++m) s = dot4(x[m], x[m], s);
        return sum8(s);
    }
    __device__ __forceinline__ void normalise(float eps) {   // x / sqrt(|x|^2 + eps); a zero row stays zero
        const float den = norm2() + eps, sc = den > 0.f ? rsqrtf(den) : 0.f;
#pragma unroll
        for (int m = 0; m < DK / 32; ++m) x[m] = mul4(x[m], sc);
    }
};

// One pair of a token with a token j of its path.
struct __align__(16) Pair {
    float a, b;   // beta_i (k_i . E_ij k_j), q_i . E_ij k_j
    int at;       // j
    int pad;
};

// Shared memory of a CTA, in bytes: [tokens] keys and decays, later the products with S (a: both, [2][T][max(DK, DV)]);
// E k and E q [2 T rounded up to 16][DK + 16] (so that a quarter-warp's 16-byte reads of two rows fall into
// different banks); pairs [T][T]; depth, parent, beta [T].
template <int DK, int DV> struct Shared {
    static constexpr int A = DK > DV ? DK : DV;   // a row of the first region
    static constexpr int B = DK + 16;
    static __host__ __device__ int rows(int T) { return (2 * T + 15) / 16 * 16; }
    static __host__ __device__ int region_b(int T) { return 2 * T * A * 4; }
    static __host__ __device__ int pairs(int T) { return region_b(T) + rows(T) * B * 4; }
    static __host__ __device__ int ints(int T) { return pairs(T) + T * T * (int)sizeof(Pair); }
    static __host__ __device__ int bytes(int T) { return ints(T) + 4 * T * 4; }
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(2 * DV, 256 / DV) kda_recurrent_tree_kernel(const TreeArgs a) {
    constexpr bool kF32 = sizeof(Tin) == 4;
    constexpr int kThreads = 2 * DV, kGroups = kThreads / 8, kSteps = DK / 16;
    using S = Shared<DK, DV>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int T = a.tokens;
    float *sk = reinterpret_cast<float *>(sm), *sa = sk + T * DK;             // keys, decays
    float *pk = sk, *pq = sk + T * S::A;                                      // later: products (u in place of the first)
    float *sb = reinterpret_cast<float *>(sm + S::region_b(T));               // E k, then E q
    Pair *pairs = reinterpret_cast<Pair *>(sm + S::pairs(T));
    int *depth = reinterpret_cast<int *>(sm + S::ints(T)), *parent = depth + T;
    float *beta = reinterpret_cast<float *>(parent + T);
    int *order = reinterpret_cast<int *>(beta + T);                           // tokens by depth; their depth above bit 8

    const int n = blockIdx.x / a.heads, h = blockIdx.x - n * a.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = a.idx ? __ldg(a.idx + n) : n;
    const int m = slot < 0 || slot >= a.slots ? 0 : tree_count(a.num, T, n);
    const int64_t first = ((int64_t)n * T * a.heads + h);                     // token i's row: first + i * heads
    for (int x = tid; x < (T - m) * DV; x += kThreads)                        // tokens past the count
        static_cast<Tin *>(a.out)[(first + (int64_t)(m + x / DV) * a.heads) * DV + x % DV] = from_f<Tin>(0.f);
    if (m == 0) return;

    // the state as B fragments: this lane's channels 16 s + 4 t4 + e of the keys, value channels c0 + 2 g and + 1
    const int g = lane >> 2, t4 = lane & 3, c0 = 16 * warp;
    float2 s[kSteps][4];
    {
        const float *src = a.state + ((int64_t)slot * a.heads + h) * (DK * DV) + (4 * t4) * DV + c0 + 2 * g;
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[st][e] = __ldcs(reinterpret_cast<const float2 *>(src + (16 * st + e) * DV));
    }
    const int grp = tid >> 3, l = tid & 7;
    for (int i0 = 0; i0 < m; i0 += kGroups) {
        const int i = i0 + grp < m ? i0 + grp : m - 1;   // (groups without a token repeat the last one's)
        const int64_t at = (first + (int64_t)i * a.heads) * DK + 4 * l;
        Row<DK> k;
        float4 d[DK / 32];
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
            k.x[x] = load4(static_cast<const Tin *>(a.k) + at + 32 * x);
            d[x] = load4(static_cast<const Tin *>(a.g) + at + 32 * x);
        }
        if (a.qk_eps >= 0.f) k.normalise(a.qk_eps);
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
            *reinterpret_cast<float4 *>(sk + i * DK + 32 * x + 4 * l) = k.x[x];
            *reinterpret_cast<float4 *>(sa + i * DK + 32 * x + 4 * l) = make_float4(expf(d[x].x), expf(d[x].y), expf(d[x].z), expf(d[x].w));
        }
        if (l == 0) {
            parent[i] = tree_parent(a.parents, T, n, i);
            beta[i] = to_f(static_cast<const Tin *>(a.beta)[first + (int64_t)i * a.heads]);
        }
    }
    __syncthreads();

    // the walks
    for (int i0 = 0; i0 < m; i0 += kGroups) {
        const bool mine = i0 + grp < m;
        const int i = mine ? i0 + grp : m - 1;
        const int64_t at = (first + (int64_t)i * a.heads) * DK + 4 * l;
        Row<DK> k, q;
        float4 d[DK / 32];
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
            q.x[x] = load4(static_cast<const Tin *>(a.q) + at + 32 * x);
            k.x[x] = *reinterpret_cast<const float4 *>(sk + i * DK + 32 * x + 4 * l);
            d[x] = make_float4(1.f, 1.f, 1.f, 1.f);
        }
        if (a.qk_eps >= 0.f) q.normalise(a.qk_eps);
        const float bt = beta[i];
        int j = mine ? i : -1, e = 0;
        while (__any_sync(0xffffffffu, j >= 0)) {
            const int jj = j >= 0 ? j : 0;
            float kk = 0.f, qq = 0.f;
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                const float4 y = mul4(*reinterpret_cast<const float4 *>(sk + jj * DK + 32 * x + 4 * l), d[x]);
                kk = dot4(k.x[x], y, kk);
                qq = dot4(q.x[x], y, qq);
            }
            kk = sum8(kk);
            qq = sum8(qq);
            if (j >= 0) {
                if (l == 0) pairs[i * T + e] = Pair{bt * kk, qq, j, 0};
#pragma unroll
                for (int x = 0; x < DK / 32; ++x) d[x] = mul4(d[x], *reinterpret_cast<const float4 *>(sa + jj * DK + 32 * x + 4 * l));
                j = parent[jj];
                ++e;
            }
        }
        if (mine) {
            if (l == 0) depth[i] = e;
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                *reinterpret_cast<float4 *>(sb + i * S::B + 32 * x + 4 * l) = operand<kF32>(mul4(k.x[x], d[x]));
                *reinterpret_cast<float4 *>(sb + (m + i) * S::B + 32 * x + 4 * l) = operand<kF32>(mul4(q.x[x], d[x]));
            }
        }
    }
    __syncthreads();   // keys and decays are read: their place takes the products
    if (tid < m) {     // (read behind the next barrier)
        const int mine = depth[tid];
        int rank = 0;
        for (int j = 0; j < m; ++j) rank += depth[j] < mine || (depth[j] == mine && j < tid);
        order[rank] = mine << 8 | tid;
    }

    if constexpr (!kF32) {   // the state as an operand
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[st][e] = make_float2(__uint_as_float(tf32(s[st][e].x)), __uint_as_float(tf32(s[st][e].y)));
    }
    for (int r0 = 0; r0 < 2 * m; r0 += 16) {   // rows r0 .. r0 + 15 of (E k; E q); those past 2 m hold anything
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        float4 v0, v1;
        const int ra = r0 + g, rb = ra + 8;
        if (ra < m) v0 = load4(static_cast<const Tin *>(a.v) + (first + (int64_t)ra * a.heads) * DV + c0 + 4 * t4);
        if (rb < m) v1 = load4(static_cast<const Tin *>(a.v) + (first + (int64_t)rb * a.heads) * DV + c0 + 4 * t4);
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            const float4 x = *reinterpret_cast<const float4 *>(sb + ra * S::B + 16 * st + 4 * t4);
            const float4 y = *reinterpret_cast<const float4 *>(sb + rb * S::B + 16 * st + 4 * t4);
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // two steps of 8 key channels
                const float f[4] = {p ? x.z : x.x, p ? y.z : y.x, p ? x.w : x.y, p ? y.w : y.y};
                const float2 b0 = s[st][2 * p], b1 = s[st][2 * p + 1];
                if constexpr (kF32) {
                    uint32_t fh[4], fl[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        fh[e] = tf32(f[e]);
                        fl[e] = tf32(f[e] - __uint_as_float(fh[e]));
                    }
                    const uint32_t h00 = tf32(b0.x), h10 = tf32(b1.x), h01 = tf32(b0.y), h11 = tf32(b1.y);
                    const uint32_t l00 = tf32(b0.x - __uint_as_float(h00)), l10 = tf32(b1.x - __uint_as_float(h10));
                    const uint32_t l01 = tf32(b0.y - __uint_as_float(h01)), l11 = tf32(b1.y - __uint_as_float(h11));
                    mma_1688(c[0], fl[0], fl[1], fl[2], fl[3], h00, h10);
                    mma_1688(c[1], fl[0], fl[1], fl[2], fl[3], h01, h11);
                    mma_1688(c[0], fh[0], fh[1], fh[2], fh[3], l00, l10);
                    mma_1688(c[1], fh[0], fh[1], fh[2], fh[3], l01, l11);
                    mma_1688(c[0], fh[0], fh[1], fh[2], fh[3], h00, h10);
                    mma_1688(c[1], fh[0], fh[1], fh[2], fh[3], h01, h11);
                } else {
                    const uint32_t a0 = __float_as_uint(f[0]), a1 = __float_as_uint(f[1]), a2 = __float_as_uint(f[2]), a3 = __float_as_uint(f[3]);
                    mma_1688(c[0], a0, a1, a2, a3, __float_as_uint(b0.x), __float_as_uint(b1.x));
                    mma_1688(c[1], a0, a1, a2, a3, __float_as_uint(b0.y), __float_as_uint(b1.y));
                }
            }
        }
        // c[t][0..1]: row ra, value channels c0 + 4 t4 + t and + 2 + t; c[t][2..3]: row rb
        auto put = [&](int r, float4 x, float4 v) {
            if (r < m) {
                const float b = beta[r];
                *reinterpret_cast<float4 *>(pk + r * S::A + c0 + 4 * t4) = make_float4(b * (v.x - x.x), b * (v.y - x.y), b * (v.z - x.z), b * (v.w - x.w));
            } else if (r < 2 * m) {
                *reinterpret_cast<float4 *>(pq + (r - m) * S::A + c0 + 4 * t4) = x;
            }
        };
        put(ra, make_float4(c[0][0], c[1][0], c[0][1], c[1][1]), v0);
        put(rb, make_float4(c[0][2], c[1][2], c[0][3], c[1][3]), v1);
    }
    __syncthreads();

    // u and the outputs of this warp's 16 value channels.  Tokens of the same depth do not depend on one another: each half of
    // the warp takes two of them at a time; of one alone, half of its pairs.
    const int ch = c0 + (lane & 15), half = lane >> 4;
    auto give = [&](int i, float w, float y, float x) {   // a token's sums: u, and its output
        const float u = pk[i * S::A + ch] - x;
        pk[i * S::A + ch] = u;
        static_cast<Tin *>(a.out)[(first + (int64_t)i * a.heads) * DV + ch] = from_f<Tin>(fmaf(w, u, pq[i * S::A + ch] + y));
    };
    for (int pos = 0; pos < m;) {
        const int o = order[pos + (lane & 3) < m ? pos + (lane & 3) : pos];
        const int depth0 = __shfl_sync(0xffffffffu, o, 0) >> 8;
        const int same = __popc(__ballot_sync(0xffffffffu, lane < 4 && pos + lane < m && (o >> 8) == depth0));   // (sorted: the first ones)
        const bool alone = same == 1, go0 = half < same, go1 = 2 + half < same;
        const int i0 = __shfl_sync(0xffffffffu, o, alone ? 0 : half) & 255, i1 = __shfl_sync(0xffffffffu, o, go1 ? 2 + half : 0) & 255;
        const Pair *r0 = pairs + i0 * T, *r1 = pairs + i1 * T;
        float x0 = 0.f, y0 = 0.f, x1 = 0.f, y1 = 0.f;
        if (alone) {
#pragma unroll 4
            for (int e = 1 + half; e < depth0; e += 2) {
                const Pair p = r0[e];
                const float u = pk[p.at * S::A + ch];
                x0 = fmaf(p.a, u, x0);
                y0 = fmaf(p.b, u, y0);
            }
            x0 += __shfl_xor_sync(0xffffffffu, x0, 16);
            y0 += __shfl_xor_sync(0xffffffffu, y0, 16);
        } else {
#pragma unroll 4
            for (int e = 1; e < depth0; ++e) {
                const Pair p0 = r0[e], p1 = r1[e];
                const float u0 = pk[p0.at * S::A + ch], u1 = pk[p1.at * S::A + ch];
                x0 = fmaf(p0.a, u0, x0);
                y0 = fmaf(p0.b, u0, y0);
                x1 = fmaf(p1.a, u1, x1);
                y1 = fmaf(p1.b, u1, y1);
            }
        }
        if (go0) give(i0, r0[0].b, y0, x0);
        if (go1) give(i1, r1[0].b, y1, x1);
        pos += same;
        __syncwarp();
    }
}

// Commit.  The path's tokens in order, each as in the decode step: vhat = (Diag(e^g) S)^T k, e = v - vhat,
// S <- Diag(e^g) S + beta k e^T.  A warp keeps all key channels of 16 value channels in registers (a lane every eighth
// key channel of four value channels), so that nothing between tokens is wider than a warp.  Bound by
// reading and writing the state once.
constexpr int kStaged = 8;   // tokens whose vectors are staged at once

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(2 * DV) kda_recurrent_tree_commit_kernel(const TreeArgs a) {
    constexpr int kThreads = 2 * DV, R = DK / 8, kGroups = kThreads / 8;
    __shared__ __align__(16) float2 ska[kStaged][DK];   // key, decay
    __shared__ __align__(16) float sv[kStaged][DV];
    __shared__ float sb[kStaged];
    __shared__ int up[kTreeMax], path[kTreeMax], s_len;
    const int n = blockIdx.x / a.heads, h = blockIdx.x - n * a.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = a.tokens;
    const int slot = a.idx ? __ldg(a.idx + n) : n;
    const int last = __ldg(a.accepted + n);
    if (slot < 0 || slot >= a.slots || last < 0 || last >= tree_count(a.num, T, n)) return;   // uniform across the block

    const int r = lane >> 2, c = 16 * warp + 4 * (lane & 3);
    float *S = a.state + ((int64_t)slot * a.heads + h) * (DK * DV) + r * DV + c;
    float4 s[R];
#pragma unroll
    for (int x = 0; x < R; ++x) s[x] = __ldcs(reinterpret_cast<const float4 *>(S + 8 * x * DV));
    for (int i = tid; i <= last; i += kThreads) up[i] = tree_parent(a.parents, T, n, i);
    __syncthreads();
    if (tid == 0) {
        int len = 0;
        for (int i = last; i >= 0; i = up[i]) ++len;
        s_len = len;
        for (int i = last; i >= 0; i = up[i]) path[--len] = i;
    }
    __syncthreads();
    const int len = s_len, grp = tid >> 3, l = tid & 7;
    for (int p0 = 0; p0 < len; p0 += kStaged) {
        const int nt = len - p0 < kStaged ? len - p0 : kStaged;
        if (p0 > 0) __syncthreads();   // the previous tokens' vectors are read
        for (int t0 = 0; t0 < nt; t0 += kGroups) {
            const int t = t0 + grp < nt ? t0 + grp : nt - 1;
            const int64_t row = ((int64_t)n * T + path[p0 + t]) * a.heads + h;
            Row<DK> k;
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) k.x[x] = load4(static_cast<const Tin *>(a.k) + row * DK + 32 * x + 4 * l);
            if (a.qk_eps >= 0.f) k.normalise(a.qk_eps);
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                const float4 d = load4(static_cast<const Tin *>(a.g) + row * DK + 32 * x + 4 * l);
                float4 *to = reinterpret_cast<float4 *>(&ska[t][32 * x + 4 * l]);
                to[0] = make_float4(k.x[x].x, expf(d.x), k.x[x].y, expf(d.y));
                to[1] = make_float4(k.x[x].z, expf(d.z), k.x[x].w, expf(d.w));
            }
            if (l == 0) sb[t] = to_f(static_cast<const Tin *>(a.beta)[row]);
        }
        for (int x = tid; x < nt * DV; x += kThreads) {
            const int64_t row = ((int64_t)n * T + path[p0 + x / DV]) * a.heads + h;
            sv[x / DV][x % DV] = to_f(static_cast<const Tin *>(a.v)[row * DV + x % DV]);
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            float4 vh = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < R; ++x) {
                const float2 ka = ska[t][r + 8 * x];
                s[x] = mul4(s[x], ka.y);
                vh = make_float4(fmaf(ka.x, s[x].x, vh.x), fmaf(ka.x, s[x].y, vh.y), fmaf(ka.x, s[x].z, vh.z), fmaf(ka.x, s[x].w, vh.w));
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                vh.x += __shfl_xor_sync(0xffffffffu, vh.x, o);
                vh.y += __shfl_xor_sync(0xffffffffu, vh.y, o);
                vh.z += __shfl_xor_sync(0xffffffffu, vh.z, o);
                vh.w += __shfl_xor_sync(0xffffffffu, vh.w, o);
            }
            const float4 v = *reinterpret_cast<const float4 *>(&sv[t][c]);
            const float b = sb[t];
            const float4 e = make_float4(b * (v.x - vh.x), b * (v.y - vh.y), b * (v.z - vh.z), b * (v.w - vh.w));
#pragma unroll
            for (int x = 0; x < R; ++x) {
                const float k = ska[t][r + 8 * x].x;
                s[x] = make_float4(fmaf(k, e.x, s[x].x), fmaf(k, e.y, s[x].y), fmaf(k, e.z, s[x].z), fmaf(k, e.w, s[x].w));
            }
        }
    }
#pragma unroll
    for (int x = 0; x < R; ++x) __stcs(reinterpret_cast<float4 *>(S + 8 * x * DV), s[x]);
}

template <typename Tin, int DK, int DV>
cudaError_t launch(const TreeArgs &a, bool commit, cudaStream_t st) {
    const unsigned grid = (unsigned)a.rows * (unsigned)a.heads;
    if (commit) {
        kda_recurrent_tree_commit_kernel<Tin, DK, DV><<<grid, 2 * DV, 0, st>>>(a);
        return cudaGetLastError();
    }
    const int bytes = Shared<DK, DV>::bytes(a.tokens);
    const cudaError_t e = cudaFuncSetAttribute(kda_recurrent_tree_kernel<Tin, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Shared<DK, DV>::bytes(kTreeMax));
    if (e != cudaSuccess) return e;
    kda_recurrent_tree_kernel<Tin, DK, DV><<<grid, 2 * DV, bytes, st>>>(a);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_d(const TreeArgs &a, int dk, int dv, bool commit, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? launch<Tin, 128, 128>(a, commit, st) : launch<Tin, 128, 64>(a, commit, st);
    return dv == 128 ? launch<Tin, 64, 128>(a, commit, st) : launch<Tin, 64, 64>(a, commit, st);
}

}  // namespace

cudaError_t launch_recurrent_tree(const TreeArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st) {
    return dt == KDA_F32 ? launch_d<float>(a, dk, dv, false, st) : launch_d<__nv_bfloat16>(a, dk, dv, false, st);
}
cudaError_t launch_recurrent_tree_commit(const TreeArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st) {
    return dt == KDA_F32 ? launch_d<float>(a, dk, dv, true, st) : launch_d<__nv_bfloat16>(a, dk, dv, true, st);
}

}  // namespace kda
