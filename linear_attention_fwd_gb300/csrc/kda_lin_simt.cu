// Linear attention with a decay for each head, chunkwise, for fp32 inputs (fp32 arithmetic).
//
// Chunks of C = 32 tokens, G_i = sum of the log decays of the chunk's tokens 0..i, S the state
// before the chunk:
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} (q_i . k_j) e^{G_i - G_j} v_j
//   S  <- e^{G_31} S + sum_j e^{G_31 - G_j} k_j v_j^T
// Every exponent is <= 0.  The sums G are kept as two floats, so that a difference is exact to fp32
// whatever the magnitude of the sums (a token that forgets everything may stand next to tokens that
// forget nothing).
//
// The value channels of S are independent: a CTA runs a block of 32 of them for one (sequence,
// head), with its part of S in registers (and a copy in shared memory for the read-out).  Where
// that makes fewer CTAs than the SMs hold, a cluster of up to 8 CTAs shares a sequence's chunks:
// each CTA but the last first takes its chunks' state from zero, the states are exchanged through
// distributed shared memory (the true state before part r is the initial state and the parts before
// it, each decayed by what follows), and every CTA then runs its chunks.  (256 tokens x 2 heads of
// 64: 29 us with one CTA per sequence and block, 10.3 us with clusters of 8.)
//
// The products are 4 x 4 tiles of four lanes each, in packed fp32 pairs, so that eight 16-byte reads of
// shared memory feed 64 multiply-adds (with 2 x 2 tiles, 16 to 24: 8 x 1024 tokens x 32 heads of 128 took
// 1119 us, now 921).  Bound by the latency of a chunk's dependent steps, shared memory's above all, at two CTAs
// per SM (128 registers a thread): on that case 1.8 instructions a cycle, the fp32 pipe 47 % busy.  The CTAs of a
// head each compute its whole score tile, at d = 128 31 % of a CTA's multiply-adds.
#include <cooperative_groups.h>

#include "kda_lin.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int C = 32, CB = 32, kThreads = 256, kMaxCluster = 8;

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float2 ld2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ float2 lo2(float4 x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(float4 x) { return make_float2(x.z, x.w); }

// Sums over four neighbouring lanes of a 4 x 4 tile; lane e of the four gets row e.
__device__ __forceinline__ float4 sum_row(const float (&a)[4][4], int e) {
    float b[2][4], o[4];
    const bool up = e & 2, odd = e & 1;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int f = 0; f < 4; ++f) b[m][f] = (up ? a[2 + m][f] : a[m][f]) + __shfl_xor_sync(0xffffffffu, up ? a[m][f] : a[2 + m][f], 2);
#pragma unroll
    for (int f = 0; f < 4; ++f) o[f] = (odd ? b[1][f] : b[0][f]) + __shfl_xor_sync(0xffffffffu, odd ? b[0][f] : b[1][f], 1);
    return make_float4(o[0], o[1], o[2], o[3]);
}

// Grid: (sequence, head, channel block) x X, clusters of X.
template <int DK>
__global__ void __launch_bounds__(kThreads, 2) kda_lin_chunk_simt_kernel(const LinArgs a, const int X) {
    // Row pitches of 16 banks and a half: 64 bytes of two neighbouring rows fill the banks.  S and V have rows of
    // 32 floats, their 16-byte pieces at piece ^ 2 (row / 4 % 4) for the same reason.
    constexpr int LD = DK + 16, LA = C + 16;
    constexpr int PER = C * DK / 4 / kThreads; // 16-byte pieces of Q (and K) per thread
    extern __shared__ __align__(16) float smem[];
    float *sQ = smem, *sK = sQ + C * LD, *sV = sK + C * LD, *sS = sV + C * CB, *sA = sS + DK * CB;
    __shared__ __align__(16) float sGh[C], sGl[C], sW[C], sE[C];
    __shared__ float sDec;
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
        st4(sV + (t / 8) * CB + 4 * ((t % 8) ^ (2 * (t / 32 % 4))), pv);
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
    float *const my_s = sS + r0 * CB + 4 * ((t % 8) ^ (2 * (r0 / 4 % 4)));   // this thread's part in shared memory
    auto update = [&]() {   // S <- e^{G_31} S + sum_j w_j k_j v_j^T
        const float dec = sDec;
#pragma unroll
        for (int m = 0; m < RT; ++m) s[m] = make_float4(s[m].x * dec, s[m].y * dec, s[m].z * dec, s[m].w * dec);
#pragma unroll 2
        for (int j0 = 0; j0 < C; j0 += 4) {
            const float4 w4 = ld4(sW + j0);
            const float w[4] = {w4.x, w4.y, w4.z, w4.w};
            const int col = 4 * ((t % 8) ^ (2 * (j0 / 4 % 4)));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + e;
                const float4 vv = ld4(sV + j * CB + col);
                float kw[RT];
                if constexpr (RT == 4) {
                    const float4 x = ld4(sK + j * LD + r0);
                    kw[0] = x.x * w[e], kw[1] = x.y * w[e], kw[2] = x.z * w[e], kw[3] = x.w * w[e];
                } else {
                    const float2 x = ld2(sK + j * LD + r0);
                    kw[0] = x.x * w[e], kw[1] = x.y * w[e];
                }
#pragma unroll
                for (int m = 0; m < RT; ++m) {
                    const float2 k2 = make_float2(kw[m], kw[m]), x = __ffma2_rn(k2, lo2(vv), lo2(s[m])), y = __ffma2_rn(k2, hi2(vv), hi2(s[m]));
                    s[m] = make_float4(x.x, x.y, y.x, y.y);
                }
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
            for (int m = 0; m < RT; ++m) st4(my_s + m * CB, s[m]);
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
                x[e] = e < rank ? ld4(cluster.map_shared_rank(my_s, e) + m * CB) : make_float4(0.f, 0.f, 0.f, 0.f);
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
    for (int m = 0; m < RT; ++m) st4(my_s + m * CB, s[m]);

    // The products' 32 x 32 results as 4 x 4 tiles, each by four neighbouring lanes (`ks`) that take every
    // fourth 4 of the inner index; a warp has 8 rows x 16 columns.
    const int ks = t & 3, tc = t >> 2 & 3, wc = t >> 5 & 1, i0 = 8 * (t >> 6) + (t >> 4 & 1) * 4;
    const int grp = 4 * wc + tc;               // O: columns 4 grp .. + 3;  A: columns 16 wc + tc + 4 f
    for (int64_t t0 = first; t0 < last; t0 += C) {
        stage(t0, true);
        const int nr = last - t0 < C ? (int)(last - t0) : C;
        {   // A_ij = (q_i . k_j) e^{G_i - G_j}, j <= i
            float2 acc[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int f = 0; f < 4; ++f) acc[e][f] = make_float2(0.f, 0.f);
#pragma unroll 2
            for (int c = 4 * ks; c < DK; c += 16) {
                float4 qa[4], kb[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    qa[e] = ld4(sQ + (i0 + e) * LD + c);
                    kb[e] = ld4(sK + (16 * wc + tc + 4 * e) * LD + c);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int f = 0; f < 4; ++f) acc[e][f] = __ffma2_rn(hi2(qa[e]), hi2(kb[f]), __ffma2_rn(lo2(qa[e]), lo2(kb[f]), acc[e][f]));
            }
            float sum[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int f = 0; f < 4; ++f) sum[e][f] = acc[e][f].x + acc[e][f].y;
            const float4 row = sum_row(sum, ks);
            const float x[4] = {row.x, row.y, row.z, row.w};
            const int i = i0 + ks;
            const float gh = sGh[i], gl = sGl[i];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int j = 16 * wc + tc + 4 * f;
                sA[i * LA + j] = j <= i ? x[f] * exp2f((gh - sGh[j]) + (gl - sGl[j])) : 0.f;
            }
        }
        float2 o[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e][0] = o[e][1] = make_float2(0.f, 0.f);
        auto product = [&](const float *left, int ld, const float *right, int inner) {   // o += left right
#pragma unroll 2
            for (int c = 4 * ks; c < inner; c += 16) {
                float4 l[4], r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[e] = ld4(left + (i0 + e) * ld + c);
                    r[e] = ld4(right + (c + e) * CB + 4 * (grp ^ (2 * ks)));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float le[4] = {l[e].x, l[e].y, l[e].z, l[e].w};
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const float2 x = make_float2(le[f], le[f]);
                        o[e][0] = __ffma2_rn(x, lo2(r[f]), o[e][0]);
                        o[e][1] = __ffma2_rn(x, hi2(r[f]), o[e][1]);
                    }
                }
            }
        };
        product(sQ, LD, sS, DK);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 g2 = make_float2(sE[i0 + e], sE[i0 + e]);
            o[e][0] = __fmul2_rn(o[e][0], g2);
            o[e][1] = __fmul2_rn(o[e][1], g2);
        }
        __syncthreads();   // sA is there, sS is read
        update();
        product(sA, LA, sV, C);
        float tile[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tile[e][0] = o[e][0].x, tile[e][1] = o[e][0].y;
            tile[e][2] = o[e][1].x, tile[e][3] = o[e][1].y;
        }
        const float4 row = sum_row(tile, ks);
        if (i0 + ks < nr) st4(out + ((t0 + i0 + ks) * a.heads + h) * a.dv + c0 + 4 * grp, row);
#pragma unroll
        for (int m = 0; m < RT; ++m) st4(my_s + m * CB, s[m]);
    }
    if (a.sT && rank == X - 1)
#pragma unroll
        for (int m = 0; m < RT; ++m) st4(a.sT + sbase + (int64_t)(r0 + m) * a.dv, s[m]);
}

template <int DK>
cudaError_t launch_t(const LinArgs &a, cudaStream_t st) {
    constexpr int smem = (2 * C * (DK + 16) + (C + DK) * CB + C * (C + 16)) * 4;
    const auto kernel = kda_lin_chunk_simt_kernel<DK>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto shape = [&](int64_t clusters, int X) {
        at[0].val.clusterDim.x = (unsigned)X;
        cfg.gridDim = dim3((unsigned)(clusters * X));
    };
    struct Held {
        int of[kMaxCluster + 1] = {};   // clusters of X that the GPU holds at once
    };
    static const Held held = [&] {
        Held h;
        for (int X = 1; X <= kMaxCluster; ++X) {
            shape(1, X);
            if (cudaOccupancyMaxActiveClusters(&h.of[X], kernel, &cfg) != cudaSuccess) h.of[X] = 0;
        }
        if (h.of[1] < 1) h.of[1] = 2 * kSms;
        return h;
    }();
    // The cluster size that should end first: rounds of clusters, each a CTA's chunks (in the first walk a third of
    // the work) and two more for its start, half as much again per chunk where CTAs share an SM (5 x 1310
    // tokens x 10 heads: 201 us as one CTA, 190 to 227 as clusters; 1 x 1310: 82 us in clusters of 6, 197 as one).
    const int64_t ctas = (int64_t)a.num_seqs * a.heads * (a.dv / CB);
    // (packed: of the average one, whatever the lengths; the sequences run in the order given)
    const int64_t chunks = ((a.cu ? a.seqlen / a.num_seqs : a.seqlen) + C - 1) / C;   // of a sequence
    int X = 1;
    int64_t best = 0;
    for (int x = 1; x <= kMaxCluster && (x == 1 || x <= chunks); ++x) {
        if (held.of[x] < 1) continue;
        const int64_t per = (chunks + x - 1) / x, rounds = (ctas + held.of[x] - 1) / held.of[x];
        const int64_t cost = rounds * (3 * per + (x > 1 ? per : 0) + 6) * (ctas * x > kSms ? 3 : 2);
        if (x == 1 || cost < best) {
            best = cost;
            X = x;
        }
    }
    shape(ctas, X);
    cfg.numAttrs = X > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, X);
}

}  // namespace

cudaError_t launch_lin_chunk_simt(const LinArgs &a, cudaStream_t st) {
    return a.dk == 128 ? launch_t<128>(a, st) : launch_t<64>(a, st);
}

}  // namespace kda
