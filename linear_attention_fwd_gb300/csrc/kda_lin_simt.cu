// Linear attention with a decay for each head, chunkwise, for fp32 inputs (fp32 arithmetic).
//
// Chunks of C = 32 tokens, G_i = sum of the log decays of the chunk's tokens 0..i, S the state
// before the chunk:
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} (q_i . k_j) e^{G_i - G_j} v_j
//   S  <- e^{G_31} S + sum_j e^{G_31 - G_j} k_j v_j^T
// Every exponent is <= 0.  The sums G are kept as two floats, so that a difference is exact to fp32 whatever the magnitude of the sums (a token that forgets everything
// may stand next to tokens that forget nothing).
//
// The value channels of S are independent: a CTA runs a block of 32 of them for one (sequence,
// head), with its part of S in registers (and a copy in shared memory for the read-out).  Where
// that makes fewer CTAs than the SMs hold, a cluster of up to 8 CTAs shares a sequence's chunks:
// each CTA but the last first takes its chunks' state from zero, the states are exchanged through
// distributed shared memory (the true state before part r is the initial state and the parts before
// it, each decayed by what follows), and every CTA then runs its chunks.  (256 tokens x 2 heads of
// 64: 42 us with one CTA per sequence and block, 10 us with clusters of 8.)
//
// Bound by shared-memory reads: about 1.4 16-byte reads per 16 multiply-adds.
#include <cooperative_groups.h>

#include "kda_lin.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int C = 32, CB = 32, kThreads = 256, kMaxCluster = 8;

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float2 ld2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }

// Grid: (sequence, head, channel block) x X, clusters of X.
template <int DK>
__global__ void __launch_bounds__(kThreads) kda_lin_chunk_simt_kernel(const LinArgs a, const int X) {
    constexpr int LD = DK + 4;                 // row pitch of Q and K: 16-byte reads of 8 rows hit 8 bank groups
    constexpr int LA = C + 4;
    constexpr int PER = C * DK / 4 / kThreads; // 16-byte pieces of Q (and K) per thread
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * LD, *sV = sK + C * LD, *sS = sV + C * CB, *sA = sS + DK * CB;
    __shared__ float sGh[C], sGl[C], sW[C], sE[C], sDec;
    __shared__ float s_decay;                  // e^(the log decays of this CTA's chunks)
    const int t = threadIdx.x, blocks = a.dv / CB;
    const int rank = blockIdx.x % X, ub = blockIdx.x / X;
    const int unit = ub / blocks, c0 = (ub % blocks) * CB;
    const int n = unit / a.heads, h = unit - n * a.heads, hk = h / (a.heads / a.qk_heads);
    int64_t bos, eos;
    lin_range(a, n, bos, eos);
    const int64_t nc = (eos - bos + C - 1) / C;
    const int64_t first = bos + rank * nc / X * C, last = rank == X - 1 ? eos : bos + (rank + 1) * nc / X * C;
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k), *v = static_cast<const float *>(a.v);
    float *out = static_cast<float *>(a.out);

    // this thread's part of S: RT rows from r0, 4 columns from cc
    constexpr int RT = DK / 32;
    const int r0 = (t / 8) * RT, cc = (t % 8) * 4;
    const int64_t sbase = ((int64_t)n * a.heads + h) * DK * a.dv + c0 + cc;
    float4 s[RT];

    float4 pq[PER], pk[PER], pv;               // the next chunk's pieces
    float pg = 0.f, total_h = 0.f, total_l = 0.f;   // a token's log decay; (thread 31) the sum of the chunks'
    const float hg = a.head_g ? __ldg(a.head_g + h) : 0.f;
    auto fetch = [&](int64_t t0, bool with_q) {
        const int nr = last - t0 < C ? (int)(last - t0) : C;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int x = t + kThreads * e, r = x / (DK / 4), c = 4 * (x % (DK / 4));
            const int64_t at = ((t0 + r) * a.qk_heads + hk) * DK + c;
            pk[e] = r < nr ? ld4(k + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (with_q) pq[e] = r < nr ? ld4(q + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (t < 32) pg = a.g && t < nr ? __ldg(a.g + (t0 + t) * a.heads + h) : 0.f;
        const int r = t / 8, c = 4 * (t % 8);
        pv = r < nr ? ld4(v + ((t0 + r) * a.heads + h) * a.dv + c0 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    // The fetched chunk to shared memory, with its decays (tokens past the end: zeros without decay);
    // then the next one is fetched.
    auto stage = [&](int64_t t0, bool with_q) {
        __syncthreads();   // the previous chunk's tiles are consumed
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int x = t + kThreads * e, r = x / (DK / 4), c = 4 * (x % (DK / 4));
            st4(sK + r * LD + c, pk[e]);
            if (with_q) st4(sQ + r * LD + c, pq[e]);
        }
        st4(sV + (t / 8) * CB + 4 * (t % 8), pv);
        if (t < 32) {
            float Gh, Gl;
            log2_decay(pg, hg, t0 + t < last, Gh, Gl);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float yh = __shfl_up_sync(0xffffffffu, Gh, o), yl = __shfl_up_sync(0xffffffffu, Gl, o);
                if (t >= o) add2f(Gh, Gl, yh, yl);
            }
            const float eh = __shfl_sync(0xffffffffu, Gh, 31), el = __shfl_sync(0xffffffffu, Gl, 31);
            sGh[t] = Gh;
            sGl[t] = Gl;
            sE[t] = exp2f(Gh + Gl);
            sW[t] = exp2f((eh - Gh) + (el - Gl));
            if (t == 31) {
                sDec = exp2f(Gh + Gl);
                add2f(total_h, total_l, Gh, Gl);
            }
        }
        if (t0 + C < last) fetch(t0 + C, with_q);
        __syncthreads();
    };
    auto update = [&]() {   // S <- e^{G_31} S + sum_j w_j k_j v_j^T
        const float dec = sDec;
#pragma unroll
        for (int m = 0; m < RT; ++m) s[m] = make_float4(s[m].x * dec, s[m].y * dec, s[m].z * dec, s[m].w * dec);
#pragma unroll 4
        for (int j = 0; j < C; ++j) {
            const float w = sW[j];
            const float4 vv = ld4(sV + j * CB + cc);
            float kw[RT];
            if constexpr (RT == 4) {
                const float4 x = ld4(sK + j * LD + r0);
                kw[0] = x.x * w, kw[1] = x.y * w, kw[2] = x.z * w, kw[3] = x.w * w;
            } else {
                const float2 x = ld2(sK + j * LD + r0);
                kw[0] = x.x * w, kw[1] = x.y * w;
            }
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                s[m].x = fmaf(kw[m], vv.x, s[m].x);
                s[m].y = fmaf(kw[m], vv.y, s[m].y);
                s[m].z = fmaf(kw[m], vv.z, s[m].z);
                s[m].w = fmaf(kw[m], vv.w, s[m].w);
            }
        }
    };

    if (X > 1) {
        // the part's state from zero (not needed of the last part)
#pragma unroll
        for (int m = 0; m < RT; ++m) s[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rank < X - 1) {
            if (first < last) fetch(first, false);
            for (int64_t t0 = first; t0 < last; t0 += C) {
                stage(t0, false);
                update();
            }
#pragma unroll
            for (int m = 0; m < RT; ++m) st4(sS + (r0 + m) * CB + cc, s[m]);
            if (t == 31) s_decay = exp2f(total_h + total_l);
        }
        if (first < last) fetch(first, true);
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
#pragma unroll
        for (int m = 0; m < RT; ++m)
            s[m] = a.s0 ? ld4(a.s0 + sbase + (int64_t)(r0 + m) * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
        // (all remote reads of a row are in flight together: the parts' number is fixed, those not before this
        // one weigh nothing)
        float f[kMaxCluster - 1];
#pragma unroll
        for (int e = 0; e < kMaxCluster - 1; ++e) f[e] = e < rank ? *cluster.map_shared_rank(&s_decay, e) : 1.f;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            float4 x[kMaxCluster - 1];
#pragma unroll
            for (int e = 0; e < kMaxCluster - 1; ++e)
                x[e] = e < rank ? ld4(cluster.map_shared_rank(sS, e) + (r0 + m) * CB + cc) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kMaxCluster - 1; ++e)
                s[m] = make_float4(fmaf(f[e], s[m].x, x[e].x), fmaf(f[e], s[m].y, x[e].y), fmaf(f[e], s[m].z, x[e].z), fmaf(f[e], s[m].w, x[e].w));
        }
        cluster.sync();   // every state (the initial one too, which may be the final one's place) is read
    } else {
        if (first < last) fetch(first, true);
#pragma unroll
        for (int m = 0; m < RT; ++m)
            s[m] = a.s0 ? ld4(a.s0 + sbase + (int64_t)(r0 + m) * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int m = 0; m < RT; ++m) st4(sS + (r0 + m) * CB + cc, s[m]);

    const int ty = t / 16, tx = t % 16;
    for (int64_t t0 = first; t0 < last; t0 += C) {
        stage(t0, true);
        const int nr = last - t0 < C ? (int)(last - t0) : C;
        {   // A_ij = (q_i . k_j) e^{G_i - G_j}, j <= i: rows 2 ty, 2 ty + 1, columns tx, tx + 16
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 8
            for (int c = 0; c < DK; c += 4) {
                float4 qa[2], kb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qa[e] = ld4(sQ + (2 * ty + e) * LD + c);
                    kb[e] = ld4(sK + (tx + 16 * e) * LD + c);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        acc[e][f] = fmaf(qa[e].x, kb[f].x, fmaf(qa[e].y, kb[f].y, fmaf(qa[e].z, kb[f].z, fmaf(qa[e].w, kb[f].w, acc[e][f]))));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int i = 2 * ty + e, j = tx + 16 * f;
                    sA[i * LA + j] = j <= i ? acc[e][f] * exp2f((sGh[i] - sGh[j]) + (sGl[i] - sGl[j])) : 0.f;
                }
        }
        // o: rows 2 ty, 2 ty + 1, columns 2 tx, 2 tx + 1; the state's part first
        float o[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        auto rows4 = [&](const float *left, int ld, const float *right, int j) {   // four steps of o += left right
            float4 l[2];
            float2 r[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) l[e] = ld4(left + (2 * ty + e) * ld + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = ld2(right + (j + e) * CB + 2 * tx);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                o[e][0] = fmaf(l[e].x, r[0].x, fmaf(l[e].y, r[1].x, fmaf(l[e].z, r[2].x, fmaf(l[e].w, r[3].x, o[e][0]))));
                o[e][1] = fmaf(l[e].x, r[0].y, fmaf(l[e].y, r[1].y, fmaf(l[e].z, r[2].y, fmaf(l[e].w, r[3].y, o[e][1]))));
            }
        };
#pragma unroll 4
        for (int c = 0; c < DK; c += 4) rows4(sQ, LD, sS, c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            o[e][0] *= sE[2 * ty + e];
            o[e][1] *= sE[2 * ty + e];
        }
        __syncthreads();   // sA is there, sS is read
        update();
#pragma unroll 4
        for (int j = 0; j < C; j += 4) rows4(sA, LA, sV, j);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * ty + e < nr)
                *reinterpret_cast<float2 *>(out + ((t0 + 2 * ty + e) * a.heads + h) * a.dv + c0 + 2 * tx) = make_float2(o[e][0], o[e][1]);
#pragma unroll
        for (int m = 0; m < RT; ++m) st4(sS + (r0 + m) * CB + cc, s[m]);
    }
    if (a.sT && rank == X - 1)
#pragma unroll
        for (int m = 0; m < RT; ++m) st4(a.sT + sbase + (int64_t)(r0 + m) * a.dv, s[m]);
}

template <int DK>
cudaError_t launch_t(const LinArgs &a, cudaStream_t st) {
    constexpr int smem = (2 * C * (DK + 4) + (C + DK) * CB + C * (C + 4)) * 4;
    const cudaError_t e = cudaFuncSetAttribute(kda_lin_chunk_simt_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)a.num_seqs * a.heads * (a.dv / CB);
    const int64_t chunks = (a.cu ? a.seqlen / a.num_seqs : a.seqlen) / C;   // of a sequence, on average
    int X = kMaxCluster;   // as many CTAs as two per SM, a chunk each at least
    while (X > 1 && (ctas * X > 2 * kSms || chunks < X)) X /= 2;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)X;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * X));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = X > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_lin_chunk_simt_kernel<DK>, a, X);
}

}  // namespace

cudaError_t launch_lin_chunk_simt(const LinArgs &a, cudaStream_t st) {
    return a.dk == 128 ? launch_t<128>(a, st) : launch_t<64>(a, st);
}

}  // namespace kda
