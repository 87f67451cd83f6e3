// Linear attention with a decay for each head, chunkwise, for fp32 inputs (fp32 arithmetic).
//
// Chunks of C = 32 tokens, G_i = sum of the log decays of the chunk's tokens 0..i, S the state
// before the chunk:
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} (q_i . k_j) e^{G_i - G_j} v_j
//   S  <- e^{G_31} S + sum_j e^{G_31 - G_j} k_j v_j^T
// Every exponent is <= 0.  The sums G are taken in fp64 and kept as two floats, so that a
// difference is exact to fp32 whatever the magnitude of the sums (a token that forgets everything
// may stand next to tokens that forget nothing).
//
// The value channels of S are independent: a CTA runs a block of 32 of them for one (sequence,
// head), with its part of S in registers (and a copy in shared memory for the read-out).
#include "kda_lin.h"

namespace kda {
namespace {

constexpr int C = 32, CB = 32, kThreads = 256;

template <int DK>
__global__ void __launch_bounds__(kThreads) kda_lin_chunk_simt_kernel(LinArgs a) {
    constexpr int LD = DK + 4;                 // row pitch of Q and K: 16-byte reads of 8 rows hit 8 bank groups
    extern __shared__ __align__(16) float smem[];
    float (*sQ)[LD] = reinterpret_cast<float (*)[LD]>(smem);
    float (*sK)[LD] = sQ + C;
    float (*sV)[CB] = reinterpret_cast<float (*)[CB]>(sK + C);
    float (*sS)[CB] = sV + C;
    __shared__ float sA[C][C + 1], sGh[C], sGl[C], sW[C], sE[C], sDec;
    const int t = threadIdx.x, blocks = a.dv / CB;
    const int unit = blockIdx.x / blocks, c0 = (int)(blockIdx.x % blocks) * CB;
    const int n = unit / a.heads, h = unit - n * a.heads, hk = h / (a.heads / a.qk_heads);
    int64_t bos, eos;
    lin_range(a, n, bos, eos);
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k), *v = static_cast<const float *>(a.v);
    float *out = static_cast<float *>(a.out);

    // this thread's part of S: RT rows from r0, 4 columns from cc
    constexpr int RT = DK / 32;
    const int r0 = (t / 8) * RT, cc = (t % 8) * 4;
    const int64_t sbase = ((int64_t)n * a.heads + h) * DK * a.dv + c0 + cc;
    float4 s[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        s[m] = a.s0 ? *reinterpret_cast<const float4 *>(a.s0 + sbase + (int64_t)(r0 + m) * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(&sS[r0 + m][cc]) = s[m];
    }
    for (int64_t t0 = bos; t0 < eos; t0 += C) {
        const int nr = eos - t0 < C ? (int)(eos - t0) : C;
        __syncthreads();   // the previous chunk's tiles are consumed
        for (int x = t; x < C * DK / 4; x += kThreads) {
            const int r = x / (DK / 4), c = 4 * (x % (DK / 4));
            float4 qv = make_float4(0.f, 0.f, 0.f, 0.f), kv = qv;
            if (r < nr) {
                const int64_t at = ((t0 + r) * a.qk_heads + hk) * DK + c;
                qv = *reinterpret_cast<const float4 *>(q + at);
                kv = *reinterpret_cast<const float4 *>(k + at);
            }
            *reinterpret_cast<float4 *>(&sQ[r][c]) = qv;
            *reinterpret_cast<float4 *>(&sK[r][c]) = kv;
        }
        {
            const int r = t / 8, c = 4 * (t % 8);
            *reinterpret_cast<float4 *>(&sV[r][c]) =
                r < nr ? *reinterpret_cast<const float4 *>(v + ((t0 + r) * a.heads + h) * a.dv + c0 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (t < 32) {
            double G = t < nr ? lin_log2_decay(a, t0 + t, h) : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, G, o);
                if (t >= o) G += y;
            }
            const double last = __shfl_sync(0xffffffffu, G, 31);
            sGh[t] = (float)G;
            sGl[t] = (float)(G - (double)(float)G);
            sE[t] = exp2f((float)G);
            sW[t] = exp2f((float)(last - G));
            if (t == 31) sDec = exp2f((float)G);
        }
        __syncthreads();
        {   // A_ij = (q_i . k_j) e^{G_i - G_j}, j <= i: rows 2 ty, 2 ty + 1, columns tx, tx + 16
            const int ty = t / 16, tx = t % 16;
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 8
            for (int c = 0; c < DK; c += 4) {
                float4 qa[2], kb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qa[e] = *reinterpret_cast<const float4 *>(&sQ[2 * ty + e][c]);
                    kb[e] = *reinterpret_cast<const float4 *>(&sK[tx + 16 * e][c]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        acc[e][f] += qa[e].x * kb[f].x + qa[e].y * kb[f].y + qa[e].z * kb[f].z + qa[e].w * kb[f].w;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int i = 2 * ty + e, j = tx + 16 * f;
                    sA[i][j] = j <= i ? acc[e][f] * exp2f((sGh[i] - sGh[j]) + (sGl[i] - sGl[j])) : 0.f;
                }
        }
        __syncthreads();
        {   // o: rows 2 ty, 2 ty + 1, columns 2 tx, 2 tx + 1
            const int ty = t / 16, tx = t % 16;
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 8
            for (int c = 0; c < DK; ++c) {
                const float2 sv = *reinterpret_cast<const float2 *>(&sS[c][2 * tx]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float qv = sQ[2 * ty + e][c];
                    acc[e][0] = fmaf(qv, sv.x, acc[e][0]);
                    acc[e][1] = fmaf(qv, sv.y, acc[e][1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                acc[e][0] *= sE[2 * ty + e];
                acc[e][1] *= sE[2 * ty + e];
            }
#pragma unroll 8
            for (int j = 0; j < C; ++j) {
                const float2 vv = *reinterpret_cast<const float2 *>(&sV[j][2 * tx]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p = sA[2 * ty + e][j];
                    acc[e][0] = fmaf(p, vv.x, acc[e][0]);
                    acc[e][1] = fmaf(p, vv.y, acc[e][1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * ty + e < nr) {
                    *reinterpret_cast<float2 *>(out + ((t0 + 2 * ty + e) * a.heads + h) * a.dv + c0 + 2 * tx) =
                        make_float2(acc[e][0], acc[e][1]);
                }
        }
        __syncthreads();   // sS is read
        const float dec = sDec;
#pragma unroll
        for (int m = 0; m < RT; ++m) s[m] = make_float4(s[m].x * dec, s[m].y * dec, s[m].z * dec, s[m].w * dec);
#pragma unroll 4
        for (int j = 0; j < C; ++j) {
            const float w = sW[j];
            const float4 vv = *reinterpret_cast<const float4 *>(&sV[j][cc]);
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const float kw = sK[j][r0 + m] * w;
                s[m].x = fmaf(kw, vv.x, s[m].x);
                s[m].y = fmaf(kw, vv.y, s[m].y);
                s[m].z = fmaf(kw, vv.z, s[m].z);
                s[m].w = fmaf(kw, vv.w, s[m].w);
            }
        }
#pragma unroll
        for (int m = 0; m < RT; ++m) *reinterpret_cast<float4 *>(&sS[r0 + m][cc]) = s[m];
    }
    if (a.sT)
#pragma unroll
        for (int m = 0; m < RT; ++m) *reinterpret_cast<float4 *>(a.sT + sbase + (int64_t)(r0 + m) * a.dv) = s[m];
}

template <int DK>
cudaError_t launch_t(const LinArgs &a, cudaStream_t st) {
    constexpr int smem = (2 * C * (DK + 4) + (C + DK) * CB) * 4;
    const cudaError_t e = cudaFuncSetAttribute(kda_lin_chunk_simt_kernel<DK>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)a.num_seqs * a.heads * (a.dv / CB);
    kda_lin_chunk_simt_kernel<DK><<<(unsigned)grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_chunk_simt(const LinArgs &a, cudaStream_t st) {
    return a.dk == 128 ? launch_t<128>(a, st) : launch_t<64>(a, st);
}

}  // namespace kda
