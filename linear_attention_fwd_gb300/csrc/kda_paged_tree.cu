// Attention of a draft's tokens over a paged cache: the fp32 kernel, and the join of partials.
#include "kda_paged_tree.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

// 256 threads take a block of 64 query rows and tiles of 32 keys in fp32 arithmetic: a thread has 4 rows x 2 keys of
// the scores and 4 rows x D / 16 channels of the outputs, both from shared memory in 16-byte reads; a row's maximum, sum
// and weights stay within the half warp that has the row.  The next tile is on its way in registers meanwhile.
// The accurate mode, bound by fp32 arithmetic and shared memory: 131,071 tokens x 8 heads, 512 query rows a head:
// 7.95 ms, 35 TFLOP/s; 32 rows of 200 to 16,384 tokens, 8 heads, up to 128 query rows each: 1.48 ms.
constexpr int kThreads = 256, kRb = 64, kKt = 32, kStart = 1;
constexpr int kSimtCtas = 2 * kSms;
static_assert(kRb == 1 << 6 && kKt == 1 << 5 && kSimtCtas <= 1 << 10, "their logarithms; see tree_cut");

template <int D> struct Simt {
    static constexpr int QS = D + 4, KS = D + 4, PS = kKt + 4;   // row strides in floats
    static constexpr int FLOATS = kRb * QS + kKt * KS + kKt * D + kRb * PS;
};

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(ptx::pack_bf16(v.x, v.y), ptx::pack_bf16(v.z, v.w));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) kda_paged_tree_attention_kernel(const TreeAtt a) {
    using S = Simt<D>;
    constexpr int CH = D / 4, RPT = kThreads / CH, LD = kKt / RPT;   // 16-byte chunks of a key, keys per step, steps of a tile
    constexpr int OC = D / 64;                                       // groups of four output channels per thread
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + kRb * S::QS, *sv = sk + kKt * S::KS, *sp = sv + kKt * D;
    __shared__ long long sm_sum[kThreads / 32];
    __shared__ uint64_t anc[kTreeMax];
    __shared__ int up[kTreeMax];
    __shared__ int64_t place[3][kKt];

    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const PagedArgs &p = a.t.p;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long W, G, x, x1, us;
    int n;
    if (!tree_share<kThreads>(a, sm_sum, W, G, x, x1, n, us)) return;
    TreeRow row = tree_row(a, n);
    int unit = tree_quotient(x - us, row.items);
    us += unit * row.items;

    const float sc = p.scale * kLog2e;
    const float *kc = static_cast<const float *>(p.k_cache), *vc = static_cast<const float *>(p.v_cache);
    for (bool first = true;; first = false) {
        const int hk = unit / row.blocks, r0 = (unit - hk * row.blocks) * kRb;
        const int rows = row.m * a.rep - r0 < kRb ? row.m * a.rep - r0 : kRb;
        const long long xe = us + row.items < x1 ? us + row.items : x1;
        const bool whole = x == us && xe == us + row.items;
        const int ia = (int)(x - us) - a.start, ib = (int)(xe - us) - a.start;
        const int ta = ia > 0 ? ia : 0, tb = ib;   // this share's tiles
        const int32_t *table = p.table + (int64_t)n * p.max_pages;
        // query row r: token i, head g of the group
        auto q_row = [&](int r, int &i) {
            i = (int)a.by_rep((uint32_t)(r0 + r));
            return ((int64_t)n * a.t.tokens + i) * p.heads + hk * a.rep + (r0 + r - i * a.rep);
        };
        __syncthreads();   // the last unit's tiles are read
        if (tid < 32) tree_masks(tree_parents(a, n, row.m), row.m, anc, up);
        for (int c = tid; c < kRb * CH; c += kThreads) {
            const int r = c / CH, ch = c % CH;
            int i;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) v = load4(static_cast<const float *>(p.q) + q_row(r, i) * D + 4 * ch);
            *reinterpret_cast<float4 *>(sq + r * S::QS + 4 * ch) = v;
        }
        auto locate = [&](int t) {   // places of tile t's keys (one warp)
            if (tid < kKt && t < tb) {
                const bool draft = t >= row.ctx;
                const int j = (draft ? t - row.ctx : t) * kKt + tid;
                place[t % 3][tid] = j < (draft ? row.m : row.len) ? tree_place(a, tree_page(a, table, draft ? row.len + j : j), draft ? row.len + j : j) : -1;
            }
        };
        float4 kr[LD], vr[LD];
        auto fetch = [&](int t) {
            if (t >= tb) return;
#pragma unroll
            for (int e = 0; e < LD; ++e) {
                const int64_t at = place[t % 3][tid / CH + e * RPT];
                kr[e] = vr[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at >= 0) {
                    const int64_t off = (at * p.kv_heads + hk) * D + 4 * (tid % CH);
                    kr[e] = load4(kc + off);
                    vr[e] = load4(vc + off);
                }
            }
        };
        locate(ta);
        __syncthreads();
        fetch(ta);
        locate(ta + 1);

        uint64_t see[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = (int)a.by_rep((uint32_t)(r0 + 4 * ty + r));
            see[r] = i < row.m ? anc[i] : 0;
        }
        float4 o[4][OC];
        float mx[4], l[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            mx[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < OC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int t = ta; t < tb; ++t) {
            if (t > ta) __syncthreads();   // the last tile is read
#pragma unroll
            for (int e = 0; e < LD; ++e) {
                const int key = tid / CH + e * RPT, ch = tid % CH;
                *reinterpret_cast<float4 *>(sk + key * S::KS + 4 * ch) = kr[e];
                *reinterpret_cast<float4 *>(sv + key * D + 4 * ch) = vr[e];
            }
            __syncthreads();
            fetch(t + 1);
            locate(t + 2);
            float s[4][2] = {};
#pragma unroll 4
            for (int c = 0; c < CH; ++c) {
                const float4 k0 = *reinterpret_cast<const float4 *>(sk + tx * S::KS + 4 * c);
                const float4 k1 = *reinterpret_cast<const float4 *>(sk + (tx + 16) * S::KS + 4 * c);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 q = *reinterpret_cast<const float4 *>(sq + (4 * ty + r) * S::QS + 4 * c);
                    s[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[r][0]))));
                    s[r][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[r][1]))));
                }
            }
            const bool draft = t >= row.ctx;
            const int j0 = draft ? (t - row.ctx) * kKt : 0;
            const bool in0 = place[t % 3][tx] >= 0, in1 = place[t % 3][tx + 16] >= 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[r][0] = in0 && (!draft || (see[r] >> (j0 + tx)) & 1) ? s[r][0] * sc : -INFINITY;
                s[r][1] = in1 && (!draft || (see[r] >> (j0 + tx + 16)) & 1) ? s[r][1] * sc : -INFINITY;
                float top = fmaxf(s[r][0], s[r][1]);
#pragma unroll
                for (int f = 1; f < 16; f <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, f));
                const float now = fmaxf(mx[r], top), z = now == -INFINITY ? 0.f : now, f = ex2(mx[r] - z);
                mx[r] = now;
                s[r][0] = ex2(s[r][0] - z);
                s[r][1] = ex2(s[r][1] - z);
                l[r] = fmaf(l[r], f, s[r][0] + s[r][1]);   // (of this lane's keys; joined at the end)
                sp[(4 * ty + r) * S::PS + tx] = s[r][0];
                sp[(4 * ty + r) * S::PS + tx + 16] = s[r][1];
#pragma unroll
                for (int c = 0; c < OC; ++c) o[r][c] = make_float4(o[r][c].x * f, o[r][c].y * f, o[r][c].z * f, o[r][c].w * f);
            }
            __syncwarp();
            for (int j = 0; j < kKt; j += 4) {
                float w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 y = *reinterpret_cast<const float4 *>(sp + (4 * ty + r) * S::PS + j);
                    w[r][0] = y.x, w[r][1] = y.y, w[r][2] = y.z, w[r][3] = y.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < OC; ++c) {
                        const float4 v = *reinterpret_cast<const float4 *>(sv + (j + e) * D + 64 * c + 4 * tx);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // a drafted token of another branch has no part in the sum, NaN and infinities included
                            if (draft && w[r][e] == 0.f) continue;
                            o[r][c] = make_float4(fmaf(w[r][e], v.x, o[r][c].x), fmaf(w[r][e], v.y, o[r][c].y), fmaf(w[r][e], v.z, o[r][c].z), fmaf(w[r][e], v.w, o[r][c].w));
                        }
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int f = 1; f < 16; f <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], f);
            const int at = 4 * ty + r;
            if (at >= rows) continue;
            if (whole) {
                int i;
                const int64_t to = q_row(at, i);
                const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    const float4 y = l[r] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv);
                    store4(static_cast<float *>(p.out) + to * D + 64 * c + 4 * tx, y);
                }
                if (p.lse && tx == 0) p.lse[to] = l[r] == 0.f ? -INFINITY : (mx[r] + log2f(l[r])) * kLn2;
            } else {
                const int64_t to = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * a.rb + at;   // slot 0: this CTA's first piece
#pragma unroll
                for (int c = 0; c < OC; ++c) *reinterpret_cast<float4 *>(a.part_o + to * D + 64 * c + 4 * tx) = o[r][c];
                if (tx == 0) *reinterpret_cast<float2 *>(a.part_ml + 2 * to) = make_float2(mx[r], l[r]);
            }
        }
        x = xe;
        if (x >= x1) break;
        us += row.items;
        if (++unit == row.blocks * p.kv_heads) {
            unit = 0;
            do row = tree_row(a, ++n); while (row.m == 0);
        }
    }
}

// Joins the parts of the units that fell into several shares, kJoinRows query rows a CTA.  Where there are few units, one
// CTA per unit and rows; else one per boundary between two shares (blockIdx.x + 1 is the share behind it),
// which takes the unit that the boundary cuts, unless an earlier one cuts it too.  Every CTA waits for the
// first kernel to end, so that nothing behind this kernel in the stream starts before that.  While they wait they write the outputs
// of the tokens past their row's count.
constexpr int kJoinThreads = 256, kJoinRows = 8;

template <typename T, int D, bool kByUnit>
__global__ void __launch_bounds__(kJoinThreads) kda_paged_tree_join_kernel(const TreeAtt a, const int ctas) {
    __shared__ long long sm_sum[kJoinThreads / 32];
    const PagedArgs &p = a.t.p;
    tree_clear<T, D, kJoinThreads>(a, blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
    int n = 0, b0 = blockIdx.x, b1 = b0, hk = 0, r0 = 0, rows = 0;
    long long us = 0, W, G;
    if (kByUnit) {
        const int blocks = (a.t.tokens * a.rep + a.rb - 1) / a.rb;   // of a row with all its tokens
        n = blockIdx.x / (p.kv_heads * blocks);
        const int u = blockIdx.x - n * p.kv_heads * blocks;
        long long mine = 0, ahead = 0;
        for (int i = threadIdx.x; i < p.rows; i += kJoinThreads) {
            const long long x = tree_items(a, i);
            mine += x;
            ahead += i < n ? x : 0;
        }
        W = block_sum<kJoinThreads>(mine, sm_sum);
        us = block_sum<kJoinThreads>(ahead, sm_sum);
        G = W < ctas ? W : ctas;
        const TreeRow row = tree_row(a, n);
        if (u < row.blocks * p.kv_heads) {
            us += u * row.items;
            hk = u / row.blocks;
            r0 = (u - hk * row.blocks) * a.rb;
            rows = row.m * a.rep - r0 < a.rb ? row.m * a.rep - r0 : a.rb;
            b0 = (int)(((us + 1) * G - 1) / W);   // (the shares that hold the unit's first item and its last)
            b1 = (int)(((us + row.items) * G - 1) / W);
        }
    } else {
        W = tree_total<kJoinThreads>(a, sm_sum);
        G = W < ctas ? W : ctas;
        if (b0 + 1 < G) {
            const long long x = (b0 + 1) * W / G;
            tree_find<kJoinThreads>(a, x, sm_sum, n, us);
            const TreeRow row = tree_row(a, n);
            const int unit = (int)((x - us) / row.items);
            us += unit * row.items;
            hk = unit / row.blocks;
            r0 = (unit - hk * row.blocks) * a.rb;
            rows = row.m * a.rep - r0 < a.rb ? row.m * a.rep - r0 : a.rb;
            if (x > us && b0 * W / G <= us) b1 = (int)(((us + row.items) * G - 1) / W);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (b1 == b0) return;
    const int64_t s0 = 2 * (int64_t)b0 + (us > b0 * W / G ? 1 : 0);   // its part in b0; then slot 0 of b0 + 1 .. b1
    constexpr int L = D / 4, PER = kJoinThreads / L;                  // lanes of a row, rows at once
    const int c4 = threadIdx.x % L;
    for (int r = blockIdx.y * kJoinRows + threadIdx.x / L; r < (int)(blockIdx.y + 1) * kJoinRows && r < rows; r += PER) {
        float mx = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAtOnce = 8;
        for (int b = b0; b <= b1; b += kAtOnce) {
            float2 v[kAtOnce];
            float4 o[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int64_t at = (b + e == b0 ? s0 : 2 * (int64_t)(b + e)) * a.rb + r;
                v[e] = b + e <= b1 ? __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + at) : make_float2(-INFINITY, 0.f);
                o[e] = b + e <= b1 ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = mx;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) top = fmaxf(top, v[e].x);
            const float z = top == -INFINITY ? 0.f : top, f0 = ex2(mx - z);
            mx = top;
            sum *= f0;
            acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const float f = ex2(v[e].x - z);
                sum = fmaf(v[e].y, f, sum);
                acc = make_float4(fmaf(o[e].x, f, acc.x), fmaf(o[e].y, f, acc.y), fmaf(o[e].z, f, acc.z), fmaf(o[e].w, f, acc.w));
            }
        }
        const int i = (int)a.by_rep((uint32_t)(r0 + r));
        const int64_t to = ((int64_t)n * a.t.tokens + i) * p.heads + hk * a.rep + (r0 + r - i * a.rep);
        if (sum == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f), sum = 1.f, mx = -INFINITY;
        const float inv = 1.f / sum;
        store4(static_cast<T *>(p.out) + to * D + 4 * c4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (p.lse && c4 == 0) p.lse[to] = (mx + log2f(sum)) * kLn2;
    }
}

template <int D> cudaError_t launch_simt(const TreeAtt &a, int ctas, cudaStream_t st) {
    constexpr int smem = Simt<D>::FLOATS * 4;
    cudaError_t e = cudaFuncSetAttribute(kda_paged_tree_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kda_paged_tree_attention_kernel<D><<<ctas, kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_tree_join(a, D, KDA_F32, ctas, st);
}

// CTAs of the kernel: never more than there can be tiles; two at least (a tile of cached tokens, one of drafted ones).
int simt_ctas(const PagedTreeArgs &t) {
    const int rep = t.p.heads / t.p.kv_heads;
    const int64_t units = (int64_t)t.p.rows * t.p.kv_heads * ((t.tokens * rep + kRb - 1) / kRb);
    const int64_t tiles = ((int64_t)t.p.max_pages * t.p.page_size + kKt - 1) / kKt + (t.tokens + kKt - 1) / kKt;
    return units >= kSimtCtas || units * tiles >= kSimtCtas ? kSimtCtas : (int)(units * tiles);
}

}  // namespace

cudaError_t launch_tree_join(const TreeAtt &a, int d, kda_dtype_t dt, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    const int rows = a.rep * a.t.tokens < a.rb ? a.rep * a.t.tokens : a.rb;
    const int64_t units = (int64_t)a.t.p.rows * a.t.p.kv_heads * (((int64_t)a.t.tokens * a.rep + a.rb - 1) / a.rb);
    const bool few = 2 * units <= ctas;
    cfg.gridDim = dim3((unsigned)(few ? units : ctas - 1), (unsigned)((rows + kJoinRows - 1) / kJoinRows));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = at;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // its CTAs may find their parts and wait before the
    at[0].val.programmaticStreamSerializationAllowed = 1;            // first kernel has ended
    cfg.numAttrs = 1;
    auto launch = [&](auto by_unit, auto by_boundary) { return few ? cudaLaunchKernelEx(&cfg, by_unit, a, ctas) : cudaLaunchKernelEx(&cfg, by_boundary, a, ctas); };
    using B = __nv_bfloat16;
    if (dt == KDA_F32)
        return d == 128 ? launch(kda_paged_tree_join_kernel<float, 128, true>, kda_paged_tree_join_kernel<float, 128, false>)
                        : launch(kda_paged_tree_join_kernel<float, 64, true>, kda_paged_tree_join_kernel<float, 64, false>);
    return d == 128 ? launch(kda_paged_tree_join_kernel<B, 128, true>, kda_paged_tree_join_kernel<B, 128, false>)
                    : launch(kda_paged_tree_join_kernel<B, 64, true>, kda_paged_tree_join_kernel<B, 64, false>);
}

size_t paged_tree_workspace_bytes(const PagedTreeArgs &t, int d, kda_dtype_t dt) {
    if (t.p.rows <= 0) return 0;
    if (dt == KDA_BF16) return tree_tc_workspace_bytes(t, d);
    return (size_t)simt_ctas(t) * 2 * kRb * (d + 2) * 4;
}

cudaError_t launch_paged_tree(const PagedTreeArgs &t, int d, kda_dtype_t dt, void *workspace, uint32_t polls, cudaStream_t st) {
    if (dt == KDA_BF16) return launch_tree_tc(t, d, workspace, polls, st);
    const int rep = t.p.heads / t.p.kv_heads, ctas = simt_ctas(t);
    float *ws = static_cast<float *>(workspace);
    const TreeAtt a{t, FastDiv((uint32_t)t.p.page_size), FastDiv((uint32_t)rep), rep, kRb, kKt, 6, 5, kStart, ws, ws + (size_t)ctas * 2 * kRb * d};
    return d == 128 ? launch_simt<128>(a, ctas, st) : launch_simt<64>(a, ctas, st);
}

}  // namespace kda
