// Attention of a draft's tokens over a paged cache, bf16, where the rows can only be short: one launch.
//
// A unit is a row's key/value head with a block of 16 of its query rows (drafted token x query head, token-major);
// a cluster of CTAs takes it, equal parts of its keys each, and joins them through distributed shared
// memory.  A row's drafted tokens are keys like the cached ones, at the positions behind them, masked by their paths.
// Within a CTA each of 4 warps takes every fourth group of 16 keys through a ring of its own (three stages of cp.async,
// page numbers fetched a group ahead), with the 16 query rows as the rows of mma.sync's tile; the weights enter the
// second product as a rounded bf16 and the rounded rest, as in kda_paged_attention.
// Bound by latency: a launch, the chain length - page - keys - scores - join.  One row of 777 tokens, 8 drafted, 8 heads of 4
// queries: 9.0 us, 15.6 in the other form.  Blocks of a head read the same keys anew, which counts against it where
// there are many (see tree_short_cluster).
#include <cooperative_groups.h>

#include "kda_paged_tree.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using namespace ptx;

constexpr int kWarps = 4, kThreads = 32 * kWarps, kStages = 3, kGroup = 16, kRows = 16, kMaxCluster = 8;

template <int D> struct Ring {
    static constexpr int RB = D * 2, CH = RB / 16;        // bytes of a key, 16-byte chunks of it
    static constexpr int STAGE = 2 * kGroup * RB;         // keys, then values
    static constexpr int BYTES = kStages * STAGE;         // one warp's
    // chunk c of row r lies at c ^ (r & 7): rows that a read touches together fall into different banks
};

template <int D>
__global__ void __launch_bounds__(kThreads) kda_paged_tree_short_kernel(const TreeAtt a, const int blocks, const int ctas) {
    using R = Ring<D>;
    extern __shared__ __align__(128) uint8_t ring_all[];
    __shared__ uint32_t sm_mask[kWarps][kStages];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows], sm_f[kWarps][kRows];
    __shared__ float2 got_ml[kRows];                       // maxima and sums of this CTA's rows, by each CTA
    __shared__ uint64_t anc[kTreeMax];
    __shared__ int up[kTreeMax], s_sick;
    __shared__ unsigned long long nf[D], weigh[kRows];    // drafted tokens whose value is not finite; that a row weighs
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedArgs &p = a.t.p;
    const int unit = blockIdx.x / ctas, rank = blockIdx.x % ctas;
    const int n = unit / (p.kv_heads * blocks), hk = unit / blocks % p.kv_heads, r0 = unit % blocks * kRows;
    const int m = tree_count(a.t.num, a.t.tokens, n), len = row_length(p, n), end = len + m;
    if (unit % (p.kv_heads * blocks) == 0) {               // tokens past the count
        const int64_t first = ((int64_t)n * a.t.tokens + m) * p.heads;
        const int rows = (a.t.tokens - m) * p.heads;
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + first * D);
        for (int i = rank * kThreads + tid; i < rows * (D / 8); i += ctas * kThreads) out[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = rank * kThreads + tid; i < rows; i += ctas * kThreads) p.lse[first + i] = -INFINITY;
    }
    const int rows = m * a.rep - r0 < kRows ? m * a.rep - r0 : kRows;
    if (rows <= 0) return;                                 // (the whole cluster)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA runs (see the join)
    const int2 parents = warp == 0 ? tree_parents(a, n, m) : make_int2(-1, -1);

    // this CTA's keys, in groups; positions past the table's width have no token
    const int groups_all = (end + kGroup - 1) / kGroup;
    const int ga = (int)((long long)rank * groups_all / ctas), gb = (int)((long long)(rank + 1) * groups_all / ctas);
    const int mine = gb - ga > warp ? (gb - ga - warp + kWarps - 1) / kWarps : 0;
    const int32_t *table = p.table + (int64_t)n * p.max_pages;
    const int64_t row_elems = (int64_t)p.kv_heads * D;
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.k_cache), *vc = static_cast<const __nv_bfloat16 *>(p.v_cache);
    uint8_t *ring = ring_all + warp * R::BYTES;
    const uint32_t ring_s = smem_u32(ring);

    auto token = [&](int i) { return (ga + warp + kWarps * i) * kGroup + lane % kGroup; };
    auto fetch = [&](int i) -> int {                       // page number of this lane's token of the warp's group i
        const int t = token(i);
        if (i >= mine || t >= end) return -1;
        const uint32_t pg = a.by_page((uint32_t)t);
        return pg < (uint32_t)p.max_pages ? __ldg(table + pg) : -1;
    };
    auto issue = [&](int i, int page) {                    // the warp's group i into stage i % kStages
        if (i < mine) {
            const int t = token(i), st = i % kStages;
            const uint32_t pg = a.by_page((uint32_t)t);
            const bool ok = page >= 0 && page < p.pages;
            const uint32_t slot = ok ? (uint32_t)page * (uint32_t)p.page_size + ((uint32_t)t - pg * (uint32_t)p.page_size) : 0u;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) sm_mask[warp][st] = mask;
            const uint32_t base = ring_s + st * R::STAGE;
#pragma unroll
            for (int c0 = 0; c0 < kGroup * R::CH; c0 += 32) {
                const int c = c0 + lane, r = c / R::CH, ch = c % R::CH;
                const uint32_t s = __shfl_sync(0xffffffffu, slot, r);
                const int64_t at = (int64_t)s * row_elems + hk * D + ch * 8;
                const uint32_t bytes = (mask >> r) & 1u ? 16u : 0u;   // 0: the chunk becomes zeros
                const uint32_t d = base + r * R::RB + ((ch ^ (r & 7)) << 4);
                cp16(d, kc + at, bytes);
                cp16(d + kGroup * R::RB, vc + at, bytes);
            }
        }
        cp_commit();
    };
    int pg[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) pg[i] = fetch(i);

    // the block's queries as A fragments (rows g and g + 8), their tokens' paths
    const int g = lane >> 2, t4 = lane & 3;
    auto q_row = [&](int r) {
        const int i = (int)a.by_rep((uint32_t)(r0 + r));
        return ((int64_t)n * a.t.tokens + i) * p.heads + hk * a.rep + (r0 + r - i * a.rep);
    };
    uint32_t qa[D / 16][4];
    {
        const uint32_t *q0 = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.q) + (g < rows ? q_row(g) : 0) * D) + t4;
        const uint32_t *q1 = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.q) + (g + 8 < rows ? q_row(g + 8) : 0) * D) + t4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qa[kk][0] = g < rows ? __ldg(q0 + 8 * kk) : 0u;
            qa[kk][1] = g + 8 < rows ? __ldg(q1 + 8 * kk) : 0u;
            qa[kk][2] = g < rows ? __ldg(q0 + 8 * kk + 4) : 0u;
            qa[kk][3] = g + 8 < rows ? __ldg(q1 + 8 * kk + 4) : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, pg[i]);
    int page = fetch(kStages - 1);
    if (warp == 0) tree_masks(parents, m, anc, up);
    for (int x = tid; x < D; x += kThreads) nf[x] = 0;
    if (tid < kRows) weigh[tid] = 0;
    if (tid == 0) s_sick = 0;
    __syncthreads();
    const uint64_t see0 = g < rows ? anc[a.by_rep((uint32_t)(r0 + g))] : 0, see1 = g + 8 < rows ? anc[a.by_rep((uint32_t)(r0 + g + 8))] : 0;

    const float sc = p.scale * kLog2e;
    float o[D / 8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const int kr = (lane & 7) + ((lane >> 4) << 3), kq = (lane >> 3) & 1;   // ldmatrix row, chunk (keys)
    const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vq = lane >> 4;   // and (values, transposed)
    for (int i = 0; i < mine; ++i) {
        cp_wait<kStages - 2>();
        __syncwarp();
        issue(i + kStages - 1, page);   // into the stage consumed by the previous iteration
        page = fetch(i + kStages);
        const int st = i % kStages;
        const uint32_t kb = ring_s + st * R::STAGE, vb = kb + kGroup * R::RB;
        const uint32_t mask = sm_mask[warp][st];
        const int t0 = (ga + warp + kWarps * i) * kGroup;
        const bool drafts = t0 + kGroup > len;
        if (drafts)   // what is not finite among the drafted tokens' values becomes zero, and NaN where it is weighed
            for (int c = lane; c < kGroup * R::CH; c += 32) {
                const int r = c / R::CH, ch = c % R::CH, j = t0 + r - len;
                if (j < 0 || j >= m) continue;
                uint4 *at = reinterpret_cast<uint4 *>(ring + st * R::STAGE + (kGroup + r) * R::RB + ((ch ^ (r & 7)) << 4));
                uint4 v = *at;
                auto ones = [](uint32_t z) { return (z & 0x7f807f80u) + 0x00800080u; };   // bits 15, 31: an exponent of all ones
                if (!((ones(v.x) | ones(v.y) | ones(v.z) | ones(v.w)) & 0x80008000u)) continue;
                uint32_t *w = &v.x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (((w[e] >> (16 * h)) & 0x7f80u) == 0x7f80u) {
                            w[e] &= h ? 0x0000ffffu : 0xffff0000u;
                            atomicOr(nf + 8 * ch + 2 * e + h, 1ull << j);
                        }
                *at = v;
                s_sick = 1;
            }
        __syncwarp();
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kb + kr * R::RB + (((2 * kk + kq) ^ (kr & 7)) << 4), b0, b1, b2, b3);
            mma_16816(s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
            mma_16816(s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b2, b3);
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * t4 + e, j = t0 + r - len;
                const bool here = (mask >> r) & 1u;
                const bool in0 = here && (j < 0 || ((see0 >> (j & 63)) & 1u)), in1 = here && (j < 0 || ((see1 >> (j & 63)) & 1u));
                s[nt][e] = in0 ? s[nt][e] * sc : -INFINITY;
                s[nt][2 + e] = in1 ? s[nt][2 + e] * sc : -INFINITY;
                mx0 = fmaxf(mx0, s[nt][e]);
                mx1 = fmaxf(mx1, s[nt][2 + e]);
            }
#pragma unroll
        for (int f = 1; f < 4; f <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, f));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, f));
        }
        if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {   // a larger maximum: bring the sums to it
            const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
            const float f0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= f0;
                o[j][1] *= f0;
                o[j][2] *= f1;
                o[j][3] *= f1;
            }
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        uint64_t w0 = 0, w1 = 0;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[nt][e] = ex2(s[nt][e] - z0);
                s[nt][2 + e] = ex2(s[nt][2 + e] - z1);
                l0 += s[nt][e];
                l1 += s[nt][2 + e];
                const int j = t0 + 8 * nt + 2 * t4 + e - len;
                if (drafts && j >= 0) {
                    w0 |= s[nt][e] != 0.f ? 1ull << (j & 63) : 0;
                    w1 |= s[nt][2 + e] != 0.f ? 1ull << (j & 63) : 0;
                }
            }
        if (w0) atomicOr(weigh + g, (unsigned long long)w0);
        if (w1) atomicOr(weigh + g + 8, (unsigned long long)w1);
        // the weights as A fragments: rounded, and the rounded rest
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = s[e >> 1][2 * (e & 1)], y0 = s[e >> 1][2 * (e & 1) + 1];
            ph[e] = pack_bf16(x0, y0);
            const float2 b = unpack_bf16(ph[e]);
            pl[e] = pack_bf16(x0 - b.x, y0 - b.y);
        }
#pragma unroll
        for (int jj = 0; jj < D / 16; ++jj) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vb + vr * R::RB + (((2 * jj + vq) ^ (vr & 7)) << 4), b0, b1, b2, b3);
            mma_16816(o[2 * jj], ph[0], ph[1], ph[2], ph[3], b0, b1);
            mma_16816(o[2 * jj + 1], ph[0], ph[1], ph[2], ph[3], b2, b3);
            mma_16816(o[2 * jj], pl[0], pl[1], pl[2], pl[3], b0, b1);
            mma_16816(o[2 * jj + 1], pl[0], pl[1], pl[2], pl[3], b2, b3);
        }
    }
    cp_wait<0>();
    __syncwarp();
#pragma unroll
    for (int f = 1; f < 4; f <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, f);
        l1 += __shfl_xor_sync(0xffffffffu, l1, f);
    }
    if (t4 == 0) {
        sm_m[warp][g] = m0;
        sm_m[warp][g + 8] = m1;
        sm_l[warp][g] = l0;
        sm_l[warp][g + 8] = l1;
    }
    float *os = reinterpret_cast<float *>(ring);   // the ring is drained: [rows][D]
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        *reinterpret_cast<float2 *>(os + g * D + 8 * j + 2 * t4) = make_float2(o[j][0], o[j][1]);
        *reinterpret_cast<float2 *>(os + (g + 8) * D + 8 * j + 2 * t4) = make_float2(o[j][2], o[j][3]);
    }
    __syncthreads();
    // Join the warps, and hand each row's outputs, maximum and sum to the CTA that has the row: what is written to another
    // SM is not waited for but at the barrier.  (With the others' parts read behind the barrier, and a second barrier before
    // leaving, one row of 777 tokens took 10.5 us, now 9.0.)
    const int share = kRows / ctas;                        // rows of a CTA
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // all CTAs run
    if (tid < rows) {
        float mx = sm_m[0][tid], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][tid]);
        const float z = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(sm_m[w][tid] - z);
            sm_f[w][tid] = f;
            sum = fmaf(sm_l[w][tid], f, sum);
        }
        cluster.map_shared_rank(got_ml, tid / share)[rank * share + tid % share] = make_float2(mx, sum);
    }
    __syncthreads();
    float *got = reinterpret_cast<float *>(ring_all + kWarps * R::BYTES);   // [CTA][share][D]
#pragma unroll 2
    for (int c = 4 * tid; c < rows * D; c += 4 * kThreads) {
        const int r = c / D, ch = c % D;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_f[w][r];
            const float4 x = *reinterpret_cast<const float4 *>(ring_all + w * R::BYTES + 4 * c);
            acc = make_float4(fmaf(x.x, f, acc.x), fmaf(x.y, f, acc.y), fmaf(x.z, f, acc.z), fmaf(x.w, f, acc.w));
        }
        if (s_sick) {
            const unsigned long long weighs = weigh[r];
            const float nan = __int_as_float(0x7fc00000);
            if (nf[ch] & weighs) acc.x = nan;
            if (nf[ch + 1] & weighs) acc.y = nan;
            if (nf[ch + 2] & weighs) acc.z = nan;
            if (nf[ch + 3] & weighs) acc.w = nan;
        }
        *reinterpret_cast<float4 *>(cluster.map_shared_rank(got, r / share) + (rank * share + r % share) * D + ch) = acc;
    }
    cluster.sync();
    for (int x = tid; x < share * (D / 2); x += kThreads) {
        const int mine_r = x / (D / 2), r = rank * share + mine_r, ch = 2 * (x % (D / 2));
        if (r >= rows) break;
        float2 ml[kMaxCluster], po[kMaxCluster];
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < kMaxCluster; ++e)
            if (e < ctas) {
                ml[e] = got_ml[e * share + mine_r];
                po[e] = *reinterpret_cast<const float2 *>(got + (e * share + mine_r) * D + ch);
                mx = fmaxf(mx, ml[e].x);
            }
        const float z = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kMaxCluster; ++e)
            if (e < ctas) {
                const float f = ex2(ml[e].x - z);
                sum = fmaf(ml[e].y, f, sum);
                acc = make_float2(fmaf(po[e].x, f, acc.x), fmaf(po[e].y, f, acc.y));
            }
        const int64_t to = q_row(r);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (sum == 0.f) acc = make_float2(0.f, 0.f);
        *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + to * D + ch) = pack_bf16(acc.x * inv, acc.y * inv);
        if (p.lse && ch == 0) p.lse[to] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
}

template <int D> cudaError_t launch_short(const TreeAtt &a, int blocks, int ctas, cudaStream_t st) {
    constexpr int smem = kWarps * Ring<D>::BYTES + kRows * D * 4;
    static_assert(kRows * D * 4 <= Ring<D>::BYTES, "a warp's outputs fit its ring");
    const cudaError_t e = cudaFuncSetAttribute(kda_paged_tree_short_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)((int64_t)a.t.p.rows * a.t.p.kv_heads * blocks * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, kda_paged_tree_short_kernel<D>, a, blocks, ctas);
}

int row_blocks(const PagedTreeArgs &t) { return (t.tokens * (t.p.heads / t.p.kv_heads) + kRows - 1) / kRows; }

}  // namespace

// CTAs of a cluster, as many as the SMs hold, up to 8.  0: the rows may be longer than a cluster takes in about the time that the
// two launches of the other form cost, or there are too many of them.
int tree_short_cluster(const PagedTreeArgs &t, int d) {
    // Of a CTA.  Over 17 shapes (1 to 32 rows, 1 to 64 drafted tokens, 1 to 8 key/value heads, 8 to 64 query heads) this form is faster in 17
    // at 400 tokens a CTA, in 15 at 512 (at most 6 % slower), in 11 at 640 (at most 16 %), in 6 at 800.  One row, 8 drafted, 8
    // key/value heads: 4088 tokens 17.3 us, 18.8 in the other form; 6392: 23.1 and 20.5; 64 drafted, 64 query heads: 448 tokens 20.8
    // and 25.7; 32 rows of 1016 tokens, one key/value head: 19.2 and 19.1.
    constexpr int kShortTokens = 512;
    const int64_t units = (int64_t)t.p.rows * t.p.kv_heads * row_blocks(t);
    const int most = d == 64 ? 4 * kSms : 2 * kSms;   // what the SMs hold at once
    int c = kMaxCluster;
    while (c > 1 && units * c > most) c /= 2;
    return units <= most && (int64_t)t.p.max_pages * t.p.page_size + t.tokens <= (int64_t)c * kShortTokens ? c : 0;
}

cudaError_t launch_tree_short(const TreeAtt &a, int d, int ctas, cudaStream_t st) {
    return d == 128 ? launch_short<128>(a, row_blocks(a.t), ctas, st) : launch_short<64>(a, row_blocks(a.t), ctas, st);
}

}  // namespace kda
