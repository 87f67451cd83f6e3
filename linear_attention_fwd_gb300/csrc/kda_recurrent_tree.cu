// KDA for a tree of drafted tokens: every token's output from an unchanged state (verify), and the accepted
// path brought into the state (commit).
//
// Verify.  With E_ij = exp of the sum of g over the path from j (excluded) to i and E_i over the whole path
// ("はじめての自然言語処理 -- Kimi K3", section 3.1, the chunkwise form, with a tree in the place of a line),
//   u_i = beta_i (v_i - (E_i k_i)^T S) - sum_{j in A(i), j != i} beta_i (k_i . E_ij k_j) u_j,
//   o_i = (E_i q_i)^T S + sum_{j in A(i)} (q_i . E_ij k_j) u_j,
// so that the state is read once and no token's own state is formed.  Nor is any u: with A the matrix of the pairs'
// beta_i (k_i . E_ij k_j) below its diagonal, B that of q_i . E_ij k_j and W_i = beta_i (v_i - (E_i k_i)^T S),
//   o = (E q) S + C W,   C (1 + A) = B,
// and a row of C comes from the rows of A on the token's path alone, without the state.  |c_ij| <= |q_i| |k_j| for
// normalised keys and beta <= 2 (a product of reflections at most lies between them).  A CTA takes a row's head:
//  1. the tokens' keys, decays and queries are requested; the state and the values are only sent for to the L2 cache,
//     which costs no registers, and are there when the walks are done;
//  2. eight lanes walk a token's path to its root with the running product of the decays: every factor is
//     at most 1, no exponent of a sum is taken, and lines of 64 tokens need no bound on g.  They leave A, B, E k and E q;
//  3. the same eight lanes walk the path again for the token's row of C;
//  4. (E k; E q) S and C W on tensor cores (mma.sync, tf32), the second added to the first in place, each warp the 16
//     value channels of which it reads the state straight into B fragments.  bf16 calls round E k, E q and S to 11 bits
//     (2^-11 relative, an eighth of the outputs' own rounding); C W, and everything in fp32 calls, is three products
//     of parts of 11 bits (in fp32 calls summed outside the tensor cores, see mma_parts: error 1.2e-7 of the outputs' root mean
//     square, 7e-7 to 9e-7 summed inside; the batch below in fp32 228 us, 215 so).  A W that is not finite is left out of
//     the product and added along the paths.
// 64 rows of 8 to 32 tokens, 64 heads of 128 x 128, bf16: 145 us, 361 MB, 2.5 TB/s.  Not DRAM but a CTA's chain of short phases bounds
// it: two CTAs an SM (three do not fit the registers, see below) issue in 45 % of the cycles, and the L1 data path, which the
// state's sectors and the walks' and tiles' shared-memory reads cross, is busy in 63 %.  Solving for u, channel by
// channel, and holding the state in registers from the start took 180 us.  tcgen05 would have to
// round the state on its way (its tf32 truncates) through 64 KB more of shared memory.
// These drafts' paths have 2.8 tokens (8 at most).  Deeper ones cost their walks' steps, one after another: 64 rows of 32 tokens, 64
// heads: 171 us in 5 levels, 182 in 8, 289 as a line (547 step by step); 16 rows of 64: 149, 155 and 320 (280 step by step).
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <type_traits>

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
__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}
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
    __device__ __forceinline__ float scale(float eps) const {   // 1 / sqrt(|x|^2 + eps); of a zero row, zero
        const float den = norm2() + eps;
        return den > 0.f ? rsqrtf(den) : 0.f;
    }
    __device__ __forceinline__ void normalise(float eps) {
        const float sc = scale(eps);
#pragma unroll
        for (int m = 0; m < DK / 32; ++m) x[m] = mul4(x[m], sc);
    }
};

// Shared memory of a CTA, in bytes:
//   keys and decays, [2][T][DK]; later W, [T rounded up to 8][DV + 8] (strides: so that what a warp reads at once falls
//   into different banks)
//   E k and E q, [rows][DK], chunk c of 16 bytes of row r at c ^ 4 (r & 1) for the same reason
//   two square matrices of the pairs, [T][stride]: beta_i (k_i . E_ij k_j) and q_i . E_ij k_j, later C; zero off the paths
//   parent, beta [T]
template <int DK, int DV> struct Shared {
    static constexpr int W = DV + 8;
    static __host__ __device__ int rows(int T) { return T <= 8 ? 16 : 2 * ((T + 15) / 16 * 16); }
    static __host__ __device__ int stride(int T) { return (T + 7) / 8 * 8 + 4; }
    static __host__ __device__ int region_b(int T) {
        const int x = 2 * T * DK * 4, y = (T + 7) / 8 * 8 * W * 4;
        return x > y ? x : y;
    }
    static __host__ __device__ int pairs(int T) { return region_b(T) + rows(T) * DK * 4; }
    static __host__ __device__ int ints(int T) { return pairs(T) + 2 * T * stride(T) * 4; }
    static __host__ __device__ int bytes(int T) { return ints(T) + 2 * T * 4; }
};

// Four channels of an input as they are.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 x;
    __device__ __forceinline__ void load(const float *p) { x = load4(p); }
    __device__ __forceinline__ float4 get() const { return x; }
};
template <> struct Raw<__nv_bfloat16> {
    uint2 x;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = __ldg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ float4 get() const {
        return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
    }
};

// Whether x may enter a product whose other operand can be zero (and neither of its parts overflows).
__device__ __forceinline__ bool tame(float x) { return fabsf(x) <= 1e38f; }

// c += A B in three products of parts of 11 bits, B of two tiles whose columns are interleaved.
struct Parts {
    uint32_t h, l;
    __device__ __forceinline__ explicit Parts(float x) {
        h = tf32(x);
        l = tf32(x - __uint_as_float(h));
    }
};
// kApart (fp32 calls): by themselves, the products of the leading parts last, and added to c by ordinary additions.  The tensor
// cores cut off what falls below their sums' last bit, always towards zero; over 16 steps in c that came to 2^-20 of it.
template <bool kApart> __device__ __forceinline__ void mma_parts(float (&to)[2][4], const float (&f)[4], float2 b0, float2 b1) {
    const Parts a0(f[0]), a1(f[1]), a2(f[2]), a3(f[3]), x0(b0.x), x1(b1.x), y0(b0.y), y1(b1.y);
    float apart[2][4] = {};
    auto &c = kApart ? apart : to;
    mma_1688(c[0], a0.l, a1.l, a2.l, a3.l, x0.h, x1.h);
    mma_1688(c[1], a0.l, a1.l, a2.l, a3.l, y0.h, y1.h);
    mma_1688(c[0], a0.h, a1.h, a2.h, a3.h, x0.l, x1.l);
    mma_1688(c[1], a0.h, a1.h, a2.h, a3.h, y0.l, y1.l);
    mma_1688(c[0], a0.h, a1.h, a2.h, a3.h, x0.h, x1.h);
    mma_1688(c[1], a0.h, a1.h, a2.h, a3.h, y0.h, y1.h);
    if constexpr (kApart)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[0][e] += apart[0][e], to[1][e] += apart[1][e];
}

// Four channels as two pairs for packed arithmetic: a walk's time is largely that of issuing its instructions.
struct Two {
    uint64_t lo, hi;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ explicit Two(const float *p) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p);
        lo = x.x, hi = x.y;
    }
    __device__ __forceinline__ explicit Two(float4 v) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(lo) : "f"(v.x), "f"(v.y));
        asm("mov.b64 %0, {%1, %2};" : "=l"(hi) : "f"(v.z), "f"(v.w));
    }
    __device__ __forceinline__ float4 get() const {
        float4 v;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(lo));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v.z), "=f"(v.w) : "l"(hi));
        return v;
    }
};
__device__ __forceinline__ Two mul2(const Two &a, const Two &b) {
    Two c;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.lo) : "l"(a.lo), "l"(b.lo));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.hi) : "l"(a.hi), "l"(b.hi));
    return c;
}
__device__ __forceinline__ void dot2(const Two &a, const Two &b, uint64_t &c) {   // (c's halves are summed at the end)
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a.lo), "l"(b.lo));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a.hi), "l"(b.hi));
}
__device__ __forceinline__ float halves(uint64_t c) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(c));
    return x + y;
}

// Up to 16 tokens have two tiles of products, whose accumulators leave the registers for three CTAs an SM (bf16): 4096
// heads of 8 tokens take 88 us, and 96 in the form for more, where three CTAs would spill (up to 32 tokens: 154 to 166 us, 145 with two).
template <typename Tin, int DK, int DV, bool kFew>
__global__ void __launch_bounds__(2 * DV, (kFew ? 384 : 256) / DV) kda_recurrent_tree_kernel(const TreeArgs a) {
    constexpr bool kF32 = sizeof(Tin) == 4;
    constexpr int kThreads = 2 * DV, kGroups = kThreads / 8, kSteps = DK / 16, kTiles = kFew ? 2 : 4, kAhead = kFew ? 2 : 4;
    using S = Shared<DK, DV>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int T = a.tokens, ST = S::stride(T);
    float *sk = reinterpret_cast<float *>(sm), *sa = sk + T * DK;             // keys, decays
    float *sw = sk;                                                           // later: W
    float *sb = reinterpret_cast<float *>(sm + S::region_b(T));               // E k, E q
    float *pa = reinterpret_cast<float *>(sm + S::pairs(T)), *pc = pa + T * ST;
    int *parent = reinterpret_cast<int *>(sm + S::ints(T));
    float *beta = reinterpret_cast<float *>(parent + T);

    const int n = blockIdx.x / a.heads, h = blockIdx.x - n * a.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = tid >> 3, l = tid & 7;
    const int slot = a.idx ? __ldg(a.idx + n) : n, count = tree_count(a.num, T, n);
    const int64_t first = ((int64_t)n * T * a.heads + h);                     // token i's row: first + i * heads
    Raw<Tin> k_raw[DK / 32], g_raw[DK / 32], q_raw[DK / 32];
    auto ask = [&](Raw<Tin> (&to)[DK / 32], const void *from, int i) {
        const Tin *p = static_cast<const Tin *>(from) + (first + (int64_t)i * a.heads) * DK;
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) to[x].load(p + 32 * x + 4 * l);
    };
    const int i_first = grp < T ? grp : T - 1;
    ask(k_raw, a.k, i_first);
    ask(g_raw, a.g, i_first);
    if constexpr (!kF32) ask(q_raw, a.q, i_first);
    const int t_own = tid < T ? tid : T - 1;
    const float beta_own = to_f(static_cast<const Tin *>(a.beta)[first + (int64_t)t_own * a.heads]);
    const int parent_own = tree_parent(a.parents, T, n, t_own);
    const int m = slot < 0 || slot >= a.slots ? 0 : count;

    // the state and the values are on their way to the L2 cache while the walks run
    const float *state = a.state + ((int64_t)(m > 0 ? slot : 0) * a.heads + h) * (DK * DV);
    if (m > 0) {
        constexpr int kPart = DK * DV * 4 / 4;
        if (tid < 4) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<const uint8_t *>(state) + tid * kPart), "n"(kPart) : "memory");
        constexpr int kLines = DV * (int)sizeof(Tin) / 128;
        for (int x = tid; x < m * kLines; x += kThreads)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const Tin *>(a.v) + (first + (int64_t)(x / kLines) * a.heads) * DV + x % kLines * (128 / (int)sizeof(Tin))));
    }
    constexpr int kVecs = DV * (int)sizeof(Tin) / 16;
    for (int x = tid; x < (T - m) * kVecs; x += kThreads)                     // outputs of tokens past the count
        reinterpret_cast<uint4 *>(static_cast<Tin *>(a.out) + (first + (int64_t)(m + x / kVecs) * a.heads) * DV)[x % kVecs] = make_uint4(0, 0, 0, 0);
    if (m == 0) return;
    for (int x = tid; x < 2 * m * ST / 4; x += kThreads) {                    // (rows of both; strides are multiples of four)
        const int half = x >= m * ST / 4;
        reinterpret_cast<float4 *>(half ? pc : pa)[x - half * (m * ST / 4)] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < m) parent[tid] = parent_own, beta[tid] = beta_own;
    for (int i0 = 0; i0 < m; i0 += kGroups) {
        const int i = i0 + grp < m ? i0 + grp : m - 1;   // (groups without a token repeat the last one's)
        if (i0 > 0 || i != i_first) {
            ask(k_raw, a.k, i);
            ask(g_raw, a.g, i);
        }
        Row<DK> k;
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) k.x[x] = k_raw[x].get();
        if (a.qk_eps >= 0.f) k.normalise(a.qk_eps);
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
            const float4 d = g_raw[x].get();
            *reinterpret_cast<float4 *>(sk + i * DK + 32 * x + 4 * l) = k.x[x];
            *reinterpret_cast<float4 *>(sa + i * DK + 32 * x + 4 * l) = make_float4(expf(d.x), expf(d.y), expf(d.z), expf(d.w));
        }
    }
    __syncthreads();

    // the walks
    const int q0 = m <= 8 ? 8 : (m + 15) / 16 * 16;      // E q's first row: up to 8 tokens share a tile of 16 rows
    for (int i0 = 0; i0 < m; i0 += kGroups) {
        const bool mine = i0 + grp < m;
        const int i = mine ? i0 + grp : m - 1;
        if (kF32 || i0 > 0 || i != i_first) ask(q_raw, a.q, i);
        Two k[DK / 32], q[DK / 32], d[DK / 32];
        {
            Row<DK> y;
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) y.x[x] = q_raw[x].get();
            if (a.qk_eps >= 0.f) y.normalise(a.qk_eps);
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                q[x] = Two(y.x[x]);
                k[x] = Two(sk + i * DK + 32 * x + 4 * l);
                d[x] = Two(make_float4(1.f, 1.f, 1.f, 1.f));
            }
        }
        const float weight = l & 1 ? 1.f : beta[i];
        float *to = (l & 1 ? pc : pa) + i * ST;              // odd lanes end up with q's sum, even ones with k's
        int j = mine ? i : -1;
        while (__any_sync(0xffffffffu, j >= 0)) {
            const int jj = j >= 0 ? j : 0;
            const float *kj = sk + jj * DK + 4 * l, *aj = kj + T * DK;
            uint64_t k2 = 0, q2 = 0;
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                const Two y = mul2(Two(kj + 32 * x), d[x]);
                dot2(k[x], y, k2);
                dot2(q[x], y, q2);
            }
            const float kk = halves(k2), qq = halves(q2);
            float sum = (l & 1 ? qq : kk) + __shfl_xor_sync(0xffffffffu, l & 1 ? kk : qq, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            if (j >= 0) {
                if (l == 1 || (l == 0 && j != i)) to[j] = weight * sum;
#pragma unroll
                for (int x = 0; x < DK / 32; ++x) d[x] = mul2(d[x], Two(aj + 32 * x));
                j = parent[jj];
            }
        }
        if (mine) {
            const int swap = 4 * (i & 1);
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                *reinterpret_cast<float4 *>(sb + i * DK + 4 * ((8 * x + l) ^ swap)) = operand<kF32>(mul2(k[x], d[x]).get());
                *reinterpret_cast<float4 *>(sb + (q0 + i) * DK + 4 * ((8 * x + l) ^ swap)) = operand<kF32>(mul2(q[x], d[x]).get());
            }
        }
    }
    __syncthreads();   // keys and decays are read: W takes their place

    // the state's B fragments: this lane's channels 16 st + 4 t4 + e of the keys, value channels c0 + 2 g and + 1
    const int g = lane >> 2, t4 = lane & 3, c0 = 16 * warp;
    float2 s[kAhead][4];
    auto load_state = [&](int st) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[st % kAhead][e] = __ldcs(reinterpret_cast<const float2 *>(state + (16 * st + 4 * t4 + e) * DV + c0 + 2 * g));
    };
#pragma unroll
    for (int st = 0; st < kAhead; ++st) load_state(st);

    // C's rows: along the path, each c_ij that is final is taken out of those above it.  Lane l has j = 8 x + l.
    auto rows_of_c = [&](auto n_regs) {
        constexpr int R = decltype(n_regs)::value;
        for (int i0 = 0; i0 < m; i0 += kGroups) {
            const bool mine = i0 + grp < m;
            const int i = mine ? i0 + grp : m - 1;
            float r[R];
#pragma unroll
            for (int x = 0; x < R; ++x) r[x] = 8 * x <= i ? pc[i * ST + 8 * x + l] : 0.f;
            int j = mine ? i : -1;
            while (__any_sync(0xffffffffu, j >= 0)) {
                const int jj = j >= 0 ? j : 0;
                const float *aj = pa + jj * ST + l;
                float c = r[0];
#pragma unroll
                for (int x = 1; x < R; ++x) c = jj >= 8 * x ? r[x] : c;
                c = __shfl_sync(0xffffffffu, c, (lane & 24) | (jj & 7));
                if (j >= 0) {
#pragma unroll
                    for (int x = 0; x < R; ++x)
                        if (8 * x < jj) r[x] = fmaf(-c, aj[8 * x], r[x]);
                    j = parent[jj];
                }
            }
            if (mine)
#pragma unroll
                for (int x = 0; x < R; ++x)
                    if (8 * x <= i) pc[i * ST + 8 * x + l] = r[x];
        }
    };
    if (m <= 32) rows_of_c(std::integral_constant<int, 4>());
    else rows_of_c(std::integral_constant<int, kTreeMax / 8>());

    const int m8 = (m + 7) / 8 * 8, tiles = (q0 + m + 15) / 16;
    bool met = false, bad = false;
    for (int t0 = 0; t0 < tiles; t0 += kTiles) {   // tiles of 16 rows of (E k; E q), four at a time; rows of no token hold anything
        float c[kTiles][2][4] = {};
        if (t0 > 0)
#pragma unroll
            for (int st = 0; st < kAhead; ++st) load_state(st);
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            float2 b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                b[e] = s[st % kAhead][e];
                if constexpr (!kF32) b[e] = make_float2(__uint_as_float(tf32(b[e].x)), __uint_as_float(tf32(b[e].y)));
            }
            if (st + kAhead < kSteps) load_state(st + kAhead);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if (t0 + t >= tiles) break;
                const float *row = sb + (16 * (t0 + t) + g) * DK + 4 * ((4 * st + t4) ^ (4 * (g & 1)));
                const float4 x = *reinterpret_cast<const float4 *>(row), y = *reinterpret_cast<const float4 *>(row + 8 * DK);
#pragma unroll
                for (int p = 0; p < 2; ++p) {   // two steps of 8 key channels
                    const float f[4] = {p ? x.z : x.x, p ? y.z : y.x, p ? x.w : x.y, p ? y.w : y.y};
                    const float2 b0 = b[2 * p], b1 = b[2 * p + 1];
                    if constexpr (kF32) {
                        mma_parts<true>(c[t], f, b0, b1);
                    } else {
                        const uint32_t a0 = __float_as_uint(f[0]), a1 = __float_as_uint(f[1]), a2 = __float_as_uint(f[2]), a3 = __float_as_uint(f[3]);
                        mma_1688(c[t][0], a0, a1, a2, a3, __float_as_uint(b0.x), __float_as_uint(b1.x));
                        mma_1688(c[t][1], a0, a1, a2, a3, __float_as_uint(b0.y), __float_as_uint(b1.y));
                    }
                }
            }
        }
        // c[t][e][0..1]: row ra, value channels c0 + 4 t4 + e and + 2 + e; c[t][e][2..3]: row rb
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int ra = 16 * (t0 + t) + g, rb = ra + 8;
            auto put = [&](int r, float4 x) {   // W, and zeros up to a multiple of eight
                if (r >= m8 || r >= q0) return;
                float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < m) {
                    const float4 v = load4(static_cast<const Tin *>(a.v) + (first + (int64_t)r * a.heads) * DV + c0 + 4 * t4);
                    const float b = beta[r];
                    w = make_float4(b * (v.x - x.x), b * (v.y - x.y), b * (v.z - x.z), b * (v.w - x.w));
                    bad |= !(tame(w.x) && tame(w.y) && tame(w.z) && tame(w.w));
                }
                *reinterpret_cast<float4 *>(sw + r * S::W + c0 + 4 * t4) = w;
            };
            put(ra, make_float4(c[t][0][0], c[t][1][0], c[t][0][1], c[t][1][1]));
            put(rb, make_float4(c[t][0][2], c[t][1][2], c[t][0][3], c[t][1][3]));
        }
        if (16 * (t0 + kTiles) <= q0) continue;
        if (!met) __syncthreads();   // C is there
        met = true;
        __syncwarp();                // and this warp's W
        const bool any_bad = __any_sync(0xffffffffu, bad);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int i0 = 16 * (t0 + t) - q0, ia = i0 + g, ib = ia + 8;
            if (t0 + t >= tiles || i0 + 8 < 0) continue;   // (16 rows of E k; up to 8 tokens share one tile)
            const bool in_a = ia >= 0 && ia < m, in_b = ib < m;
            for (int j = 0; j < m8 && j < i0 + 16; j += 8) {
                const float f[4] = {in_a ? pc[ia * ST + j + t4] : 0.f, in_b ? pc[ib * ST + j + t4] : 0.f,
                                    in_a ? pc[ia * ST + j + 4 + t4] : 0.f, in_b ? pc[ib * ST + j + 4 + t4] : 0.f};
                float2 x = *reinterpret_cast<const float2 *>(sw + (j + t4) * S::W + c0 + 2 * g);
                float2 y = *reinterpret_cast<const float2 *>(sw + (j + 4 + t4) * S::W + c0 + 2 * g);
                if (any_bad) {
                    x = make_float2(tame(x.x) ? x.x : 0.f, tame(x.y) ? x.y : 0.f);
                    y = make_float2(tame(y.x) ? y.x : 0.f, tame(y.y) ? y.y : 0.f);
                }
                mma_parts<kF32>(c[t], f, x, y);
            }
            if (any_bad) {   // what is not finite reaches the tokens that continue it, and no others
                auto add = [&](float x, float w, float &to) { to = tame(w) ? to : fmaf(x, w, to); };
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    for (int i = e ? ib : ia, j = (e ? in_b : in_a) ? i : -1; j >= 0; j = parent[j]) {
                        const float x = pc[i * ST + j];
                        const float4 w = *reinterpret_cast<const float4 *>(sw + j * S::W + c0 + 4 * t4);
                        add(x, w.x, c[t][0][2 * e]), add(x, w.y, c[t][1][2 * e]), add(x, w.z, c[t][0][2 * e + 1]), add(x, w.w, c[t][1][2 * e + 1]);
                    }
            }
            auto give = [&](int i, float4 o) { put4(static_cast<Tin *>(a.out) + (first + (int64_t)i * a.heads) * DV + c0 + 4 * t4, o); };
            if (in_a) give(ia, make_float4(c[t][0][0], c[t][1][0], c[t][0][1], c[t][1][1]));
            if (in_b) give(ib, make_float4(c[t][0][2], c[t][1][2], c[t][0][3], c[t][1][3]));
        }
    }
}

// Commit.  The path's tokens in order, each as in the decode step: vhat = (Diag(e^g) S)^T k, e = v - vhat,
// S <- Diag(e^g) S + beta k e^T.  A warp keeps all key channels of 16 value channels in registers (a lane every eighth
// key channel of four value channels), so that nothing between tokens is wider than a warp; a CTA has two
// warps, since value channels do not meet, and eight CTAs of an SM read, step and write at times of their own.  Bound by reading and
// writing the state once where paths are short: 256 rows of 1 to 16 drafted tokens, 0 to 5 of them accepted (1.8 on average), 64 heads,
// bf16: 332 us, 2.0 GB, 6.0 TB/s (64 channels a CTA: 337; all 128: 368; those with three CTAs an SM spill: 461).  Beyond
// that by the tokens' chains of product, sum over lanes and update, some 45 us a token: 305 us with 1 accepted in every
// row, 456 with 4, 623 with 8, 977 with 16.
constexpr int kStaged = 8;   // tokens whose vectors are staged at once
constexpr int kCols = 32;    // value channels of a CTA

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(2 * kCols, 8) kda_recurrent_tree_commit_kernel(const TreeArgs a) {
    constexpr int kSplit = DV / kCols, kThreads = 2 * kCols, R = DK / 8, kGroups = kThreads / 8;
    __shared__ __align__(16) float2 ska[kStaged][DK];   // key, decay
    __shared__ __align__(16) float sv[kStaged][kCols];
    __shared__ float sb[kStaged];
    __shared__ int up[kTreeMax], path[kTreeMax], s_len;
    const int unit = blockIdx.x / kSplit, col0 = (blockIdx.x - unit * kSplit) * kCols;
    const int n = unit / a.heads, h = unit - n * a.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = a.tokens;
    const int slot = a.idx ? __ldg(a.idx + n) : n;
    const int last = __ldg(a.accepted + n);
    if (slot < 0 || slot >= a.slots || last < 0 || last >= tree_count(a.num, T, n)) return;   // uniform across the block

    const int r = lane >> 2, c = 16 * warp + 4 * (lane & 3);
    float *S = a.state + ((int64_t)slot * a.heads + h) * (DK * DV) + r * DV + col0 + c;
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
        for (int x = tid; x < nt * kCols; x += kThreads) {
            const int64_t row = ((int64_t)n * T + path[p0 + x / kCols]) * a.heads + h;
            sv[x / kCols][x % kCols] = to_f(static_cast<const Tin *>(a.v)[row * DV + col0 + x % kCols]);
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
        kda_recurrent_tree_commit_kernel<Tin, DK, DV><<<grid * (DV / kCols), 2 * kCols, 0, st>>>(a);
        return cudaGetLastError();
    }
    const bool few = sizeof(Tin) == 2 && a.tokens <= 16;
    const auto kernel = few ? kda_recurrent_tree_kernel<Tin, DK, DV, sizeof(Tin) == 2> : kda_recurrent_tree_kernel<Tin, DK, DV, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shared<DK, DV>::bytes(few ? 16 : kTreeMax));
    if (e != cudaSuccess) return e;
    kernel<<<grid, 2 * DV, Shared<DK, DV>::bytes(a.tokens), st>>>(a);
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
