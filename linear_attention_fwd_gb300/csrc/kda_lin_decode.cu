// Linear attention with a decay for each head, single tokens on a pool of fp32 states:
//   S <- a S + k v^T,  o = S^T q,  a = exp(g + head_g).
// Columns of S are independent, so the state streams through registers once: each thread holds 4
// columns of a few rows, updates and stores them, and the read-out's partial sums over the rows
// meet in shared memory.  Bound by the state's one read and one write.
#include "kda_lin.h"

namespace kda {
namespace {

// One CTA per (row, head, block of CB value channels).
template <typename Tin, int DK, int DV, int CB, int kThreads>
__global__ void __launch_bounds__(kThreads) kda_lin_step_kernel(LinStepArgs a) {
    constexpr int CG = CB / 4;               // float4 column groups
    constexpr int RG = kThreads / CG;        // row groups
    constexpr int RPT = DK / RG;             // rows per thread
    static_assert(RPT >= 1 && RG * RPT == DK, "tile split");
    const int unit = blockIdx.x / (DV / CB), c0 = (int)(blockIdx.x % (DV / CB)) * CB;
    const int n = unit / a.heads, h = unit - n * a.heads;
    const int slot = a.idx ? __ldg(a.idx + n) : n;
    if (slot < 0 || slot >= a.slots) return;   // uniform across the block

    __shared__ __align__(16) float red[RG][CB];
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    float *S = a.state + ((int64_t)slot * a.heads + h) * (DK * DV) + c0;
    float4 s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        s[m] = __ldcs(reinterpret_cast<const float4 *>(S + (rg * RPT + m) * DV) + cg);

    const int hk = h / (a.heads / a.qk_heads);
    const Tin *q = static_cast<const Tin *>(a.q) + ((int64_t)n * a.qk_heads + hk) * DK + rg * RPT;
    const Tin *k = static_cast<const Tin *>(a.k) + ((int64_t)n * a.qk_heads + hk) * DK + rg * RPT;
    const Tin *v = static_cast<const Tin *>(a.v) + ((int64_t)n * a.heads + h) * DV + c0 + 4 * cg;
    float lg = 0.f;
    if (a.g) lg += __ldg(a.g + (int64_t)n * a.heads + h);
    if (a.head_g) lg += __ldg(a.head_g + h);
    const float al = expf(lg);
    float kr[RPT], qr[RPT], vc[4];
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        kr[m] = to_f(k[m]);
        qr[m] = to_f(q[m]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) vc[c] = to_f(v[c]);
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        s[m].x = fmaf(al, s[m].x, kr[m] * vc[0]);
        s[m].y = fmaf(al, s[m].y, kr[m] * vc[1]);
        s[m].z = fmaf(al, s[m].z, kr[m] * vc[2]);
        s[m].w = fmaf(al, s[m].w, kr[m] * vc[3]);
        __stcs(reinterpret_cast<float4 *>(S + (rg * RPT + m) * DV) + cg, s[m]);
        p[0] = fmaf(qr[m], s[m].x, p[0]);
        p[1] = fmaf(qr[m], s[m].y, p[1]);
        p[2] = fmaf(qr[m], s[m].z, p[2]);
        p[3] = fmaf(qr[m], s[m].w, p[3]);
    }
    *reinterpret_cast<float4 *>(&red[rg][4 * cg]) = make_float4(p[0], p[1], p[2], p[3]);
    __syncthreads();
    if (t < CB) {
        float o = 0.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) o += red[r][t];
        static_cast<Tin *>(a.out)[((int64_t)n * a.heads + h) * DV + c0 + t] = from_f<Tin>(o);
    }
}

// Fewer units than two per SM leave SMs idle or with half the work of others: a unit's columns then go to
// CTAs of 32 each, 128-byte rows (32 states of 128 x 128: 2.5 us against 3.2).  More units take whole states
// (470 of them: 12.8 us against 14.4 in blocks).
template <typename Tin, int DK, int DV>
cudaError_t launch_t(const LinStepArgs &a, cudaStream_t st) {
    const unsigned units = (unsigned)(a.rows * a.heads);
    if (units >= 2 * kSms) kda_lin_step_kernel<Tin, DK, DV, DV, 256><<<units, 256, 0, st>>>(a);
    else kda_lin_step_kernel<Tin, DK, DV, 32, 128><<<units * (DV / 32), 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_d(const LinStepArgs &a, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? launch_t<Tin, 128, 128>(a, st) : launch_t<Tin, 128, 64>(a, st);
    return dv == 128 ? launch_t<Tin, 64, 128>(a, st) : launch_t<Tin, 64, 64>(a, st);
}

}  // namespace

cudaError_t launch_lin_step(const LinStepArgs &a, int dk, int dv, kda_dtype_t dt, cudaStream_t st) {
    return dt == KDA_F32 ? launch_d<float>(a, dk, dv, st) : launch_d<__nv_bfloat16>(a, dk, dv, st);
}

}  // namespace kda
