// Paged key-value cache: append, and attention of one new token per row.
#include <cooperative_groups.h>

#include "kda_paged.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

// ------------------------------------------------------------------ append
// A CTA moves `per` consecutive tokens, a vector of 16 bytes of keys and one of values per thread and step.
// The first kAhead vectors of each are requested before the tokens' places are known: one thread per
// token finds its place (row by bisection in the offsets, then page and offset).  Bound by one read and
// one write of the new rows (49,700 tokens of 8 x 128 bf16: 30.6 us, 82 % of the measured copy rate;
// 32 us when the places come first).
constexpr int kAppendThreads = 256, kAhead = 4, kMaxTokens = 32;

__global__ void __launch_bounds__(kAppendThreads) kda_paged_append_kernel(const AppendArgs a, const int per) {
    __shared__ int64_t place[kMaxTokens];   // the token's index in the cache, or -1
    const int64_t u0 = (int64_t)blockIdx.x * per;
    const int tokens = a.tokens - u0 < per ? (int)(a.tokens - u0) : per, vecs = tokens * a.row_vecs;
    const uint4 *k = static_cast<const uint4 *>(a.k) + u0 * a.row_vecs, *v = static_cast<const uint4 *>(a.v) + u0 * a.row_vecs;
    uint4 kv[kAhead], vv[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
        const int x = threadIdx.x + kAppendThreads * e;
        if (x < vecs) {
            kv[e] = __ldcs(k + x);
            vv[e] = __ldcs(v + x);
        }
    }
    if (threadIdx.x < tokens) {
        const int64_t u = u0 + threadIdx.x;
        int64_t at = -1;
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
        place[threadIdx.x] = at;
    }
    __syncthreads();
    uint4 *kc = static_cast<uint4 *>(a.k_cache), *vc = static_cast<uint4 *>(a.v_cache);
    auto store = [&](int x, const uint4 &key, const uint4 &value) {
        const int tk = x / a.row_vecs;
        const int64_t at = place[tk];
        if (at < 0) return;
        const int64_t to = at * a.row_vecs + (x - tk * a.row_vecs);
        kc[to] = key;
        vc[to] = value;
    };
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
        const int x = threadIdx.x + kAppendThreads * e;
        if (x < vecs) store(x, kv[e], vv[e]);
    }
    for (int x = threadIdx.x + kAppendThreads * kAhead; x < vecs; x += kAppendThreads) store(x, __ldcs(k + x), __ldcs(v + x));
}

// ------------------------------------------------------------------ attention
// One new token per row over its cached tokens.  Bound by reading the cache once: a key/value head
// has 4 D FLOP per query head and token for 2 D elements read, far below the tensor cores' rate.
//
// Work.  A unit is a row's key/value head with a block of up to RP of its query heads; a unit's
// items are its tiles of 64 tokens (at least one) and, ahead of them, kStart that stand for the time a
// unit's start takes (30 rows of 1 to 16316 tokens, 8 key/value heads: 45 us, 89 us without them, 50 and
// 47 with two and five).  The items of all units, in order, are cut into
// equal shares, one per CTA (two CTAs per SM): each CTA finds its share from seq_lens on the
// device, since the host does not see the lengths.  A unit that ends up in several shares leaves
// one partial (running maximum, sum, unnormalised output) per share in the workspace, and a second
// kernel joins them in a fixed order, so results do not depend on timing.
// Where the rows can only be short (a row's share of the longest possible one at most kShortTokens),
// one cluster of CTAs takes a unit instead, equal parts each, and joins them through distributed shared
// memory: one launch and no workspace (one row of 777 tokens, 8 key/value heads: 5.7 us in a graph against 6.9).
// The host does not see the lengths, so what rows can be is read off the block table's width.
//
// Within a CTA each of 4 warps takes every fourth group of tokens through a ring of its own (three
// stages of cp.async, page numbers fetched one group ahead), so that the loop has no barrier wider
// than a warp.  The warps' running maxima and sums are joined when the unit ends.
//  - bf16: mma.sync m16n8k16, the block's 16 query heads as rows of the tile (rows past the heads
//    are zeros).  The weights enter the second product as a rounded bf16 and the rounded rest, so
//    that they are as good as 16 bits: one rounding alone would cost 2^-9 per weight, as much as
//    the output's own rounding.
//  - fp32: the same walk in fp32 arithmetic (four lanes share a token's channels).
constexpr int kWarps = 4, kTile = 64, kStages = 3, kAttThreads = 32 * kWarps;
constexpr int kStart = 3;   // a unit's start, in tiles
constexpr int kCtas = 2 * kSms;

struct AttArgs {
    PagedArgs p;
    FastDiv by_page;
    int32_t rep, blocks, rp;   // query heads per key/value head, head blocks, heads per block
    float *part_o, *part_ml;   // partials: [2 G][rp][D], [2 G][rp][2]
    int32_t cluster;           // CTAs of a unit (short rows)
};

__device__ __forceinline__ int row_tiles(const PagedArgs &a, int n) {
    const int t = (row_length(a, n) + kTile - 1) / kTile;
    return t > 0 ? t : 1;
}
__device__ __forceinline__ int row_items(const PagedArgs &a, int n) { return kStart + row_tiles(a, n); }   // of each of its units

// Block-wide: the row that holds item x (rows in order, `per` units of row_items each) and the number of
// items before that row.
template <int THREADS>
__device__ void find_row(const PagedArgs &a, int per, long long x, long long *sm, int &row, long long &before) {
    __shared__ int s_row;
    __shared__ long long s_before;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    long long run = 0;
    for (int base = 0; base < a.rows; base += THREADS) {
        const int n = base + t;
        const long long w = n < a.rows ? (long long)per * row_items(a, n) : 0;
        long long v = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) sm[warp] = v;
        __syncthreads();
        long long off = 0, tot = 0;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) {
            off += i < warp ? sm[i] : 0;
            tot += sm[i];
        }
        const long long first = run + off + v - w;
        if (n < a.rows && first <= x && x < first + w) {
            s_row = n;
            s_before = first;
        }
        run += tot;
        if (x < run) break;   // uniform
    }
    __syncthreads();
    row = s_row;
    before = s_before;
}

template <typename T, int D> struct Att {
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int GT = kF32 ? 8 : 16;                 // tokens of a group
    static constexpr int RB = D * (int)sizeof(T);            // bytes of a token's keys (or values)
    static constexpr int CH = RB / 16;                       // 16-byte chunks of them
    static constexpr int STAGE = 2 * GT * RB;                // keys, then values
    static constexpr int RING = kStages * STAGE;             // one warp's
    // chunk c of row r lies at c ^ swz(r): rows a read touches together fall into different banks
    static __device__ __forceinline__ int swz(int r) { return kF32 ? ((r & 1) << 2) | ((r >> 1) & 3) : (r & 7); }
};

template <typename T, int D, int RP, bool kShort>
__global__ void __launch_bounds__(kAttThreads, 2) kda_paged_attention_kernel(const AttArgs a) {
    using A = Att<T, D>;
    using namespace ptx;
    extern __shared__ __align__(128) uint8_t ring_all[];
    __shared__ long long sm_sum[kWarps];
    __shared__ uint32_t sm_mask[kWarps][kStages];
    __shared__ float sm_m[kWarps][RP], sm_l[kWarps][RP];
    __shared__ __align__(16) float sm_q[A::kF32 ? RP : 1][A::kF32 ? D : 4];
    __shared__ float sm_pm[kShort ? RP : 1], sm_pl[kShort ? RP : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedArgs &p = a.p;
    const int per = p.kv_heads * a.blocks;
    long long x, x1, us = 0;   // this CTA's share of the items; the current unit's first item
    int n, items, unit;        // row, its units' items, key/value head and head block within it
    if constexpr (kShort) {
        const int ru = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
        n = ru / per;
        unit = ru % per;
        items = row_tiles(p, n);
        x = (long long)rank * items / a.cluster;
        x1 = (long long)(rank + 1) * items / a.cluster;
    } else {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        long long mine = 0;
        for (int i = tid; i < p.rows; i += kAttThreads) mine += row_items(p, i);
        const long long W = per * block_sum<kAttThreads>(mine, sm_sum);
        const long long G = W < gridDim.x ? W : gridDim.x;   // shares: at least one item each
        if (blockIdx.x >= G) return;
        x1 = (blockIdx.x + 1) * W / G;
        x = blockIdx.x * W / G;
        find_row<kAttThreads>(p, per, x, sm_sum, n, us);
        items = row_items(p, n);
        unit = (int)((x - us) / items);
        us += (long long)unit * items;
    }

    uint8_t *ring = ring_all + warp * A::RING;
    const uint32_t ring_s = smem_u32(ring);
    const float sc = p.scale * kLog2e;
    const T *kc = static_cast<const T *>(p.k_cache), *vc = static_cast<const T *>(p.v_cache);
    const int64_t row_elems = (int64_t)p.kv_heads * D;

    for (bool first = true;; first = false) {
        const int hk = unit / a.blocks, h0 = (unit - hk * a.blocks) * RP;
        const int heads = a.rep - h0 < RP ? a.rep - h0 : RP;      // query heads of this block
        const int64_t hq = (int64_t)n * p.heads + (int64_t)hk * a.rep + h0;
        const long long xe = us + items < x1 ? us + items : x1;
        const bool whole = kShort ? a.cluster == 1 : x == us && xe == us + items;
        const int len = row_length(p, n);
        constexpr int S = kShort ? 0 : kStart;   // a unit's first items stand for its start
        const int ia = (int)(x - us) - S, ib = (int)(xe - us) - S;
        const int ta = ia > 0 ? ia * kTile : 0, tb = ib * kTile < len ? ib * kTile : len;
        const int groups = tb > ta ? (tb - ta + A::GT - 1) / A::GT : 0;
        const int mygroups = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;
        const int32_t *table = p.table + (int64_t)n * p.max_pages;

        // page number of this lane's token of the warp's group i (-1: none)
        const int r_own = lane % A::GT;
        auto token = [&](int i) { return ta + A::GT * (warp + kWarps * i) + r_own; };
        auto fetch = [&](int i) -> int {
            const int t = token(i);
            return i < mygroups && t < tb ? __ldg(table + a.by_page((uint32_t)t)) : -1;
        };
        auto issue = [&](int i, int page) {   // the warp's group i into stage i % kStages
            if (i < mygroups) {
                const int t = token(i), st = i % kStages;
                const uint32_t pg = a.by_page((uint32_t)t);
                const bool ok = page >= 0 && page < p.pages;
                const uint32_t slot = ok ? (uint32_t)page * (uint32_t)p.page_size + ((uint32_t)t - pg * (uint32_t)p.page_size) : 0u;
                const uint32_t mask = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) sm_mask[warp][st] = mask;
                const uint32_t base = ring_s + st * A::STAGE;
#pragma unroll
                for (int c0 = 0; c0 < A::GT * A::CH; c0 += 32) {
                    const int c = c0 + lane, r = c / A::CH, ch = c % A::CH;
                    const uint32_t s = __shfl_sync(0xffffffffu, slot, r);
                    const int64_t at = (int64_t)s * row_elems + hk * D + ch * (16 / (int)sizeof(T));
                    const uint32_t bytes = (mask >> r) & 1u ? 16u : 0u;   // 0: the chunk becomes zeros
                    const uint32_t d = base + r * A::RB + ((ch ^ A::swz(r)) << 4);
                    cp16(d, kc + at, bytes);
                    cp16(d + A::GT * A::RB, vc + at, bytes);
                }
            }
            cp_commit();
        };
        {
            int pg[kStages - 1];
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) pg[i] = fetch(i);
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) issue(i, pg[i]);
        }
        int page = fetch(kStages - 1);

        if constexpr (!A::kF32) {
            const int g = lane >> 2, t4 = lane & 3;
            // the block's queries as A fragments (rows g and g + 8)
            uint32_t qa[D / 16][4];
            const uint32_t *q0 = reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) + (hq + g) * D) + t4;
            const uint32_t *q1 = q0 + 8 * D / 2;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][0] = g < heads ? __ldg(q0 + 8 * kk) : 0u;
                qa[kk][1] = g + 8 < heads ? __ldg(q1 + 8 * kk) : 0u;
                qa[kk][2] = g < heads ? __ldg(q0 + 8 * kk + 4) : 0u;
                qa[kk][3] = g + 8 < heads ? __ldg(q1 + 8 * kk + 4) : 0u;
            }
            float o[D / 8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
            const int kr = (lane & 7) + ((lane >> 4) << 3), kq = (lane >> 3) & 1;   // ldmatrix row, chunk (keys)
            const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vq = lane >> 4;   // and (values, transposed)
            for (int i = 0; i < mygroups; ++i) {
                cp_wait<kStages - 2>();
                __syncwarp();
                issue(i + kStages - 1, page);   // into the stage consumed by the previous iteration
                page = fetch(i + kStages);
                const int st = i % kStages;
                const uint32_t kb = ring_s + st * A::STAGE, vb = kb + A::GT * A::RB;
                const uint32_t mask = sm_mask[warp][st];
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(kb + kr * A::RB + (((2 * kk + kq) ^ A::swz(kr)) << 4), b0, b1, b2, b3);
                    mma_16816(s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
                    mma_16816(s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b2, b3);
                }
                float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool in = (mask >> (8 * nt + 2 * t4 + e)) & 1u;
                        s[nt][e] = in ? s[nt][e] * sc : -INFINITY;
                        s[nt][2 + e] = in ? s[nt][2 + e] * sc : -INFINITY;
                        mx0 = fmaxf(mx0, s[nt][e]);
                        mx1 = fmaxf(mx1, s[nt][2 + e]);
                    }
#pragma unroll
                for (int sft = 1; sft < 4; sft <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sft));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sft));
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
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[nt][e] = ex2(s[nt][e] - z0);
                        s[nt][2 + e] = ex2(s[nt][2 + e] - z1);
                        l0 += s[nt][e];
                        l1 += s[nt][2 + e];
                    }
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
                    ldsm_x4_t(vb + vr * A::RB + (((2 * jj + vq) ^ A::swz(vr)) << 4), b0, b1, b2, b3);
                    mma_16816(o[2 * jj], ph[0], ph[1], ph[2], ph[3], b0, b1);
                    mma_16816(o[2 * jj + 1], ph[0], ph[1], ph[2], ph[3], b2, b3);
                    mma_16816(o[2 * jj], pl[0], pl[1], pl[2], pl[3], b0, b1);
                    mma_16816(o[2 * jj + 1], pl[0], pl[1], pl[2], pl[3], b2, b3);
                }
            }
            cp_wait<0>();
            __syncwarp();
#pragma unroll
            for (int sft = 1; sft < 4; sft <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, sft);
                l1 += __shfl_xor_sync(0xffffffffu, l1, sft);
            }
            if (t4 == 0) {
                sm_m[warp][g] = m0;
                sm_m[warp][g + 8] = m1;
                sm_l[warp][g] = l0;
                sm_l[warp][g + 8] = l1;
            }
            float *os = reinterpret_cast<float *>(ring);   // the ring is drained: [heads][D]
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                if (g < heads) *reinterpret_cast<float2 *>(os + g * D + 8 * j + 2 * t4) = make_float2(o[j][0], o[j][1]);
                if (g + 8 < heads) *reinterpret_cast<float2 *>(os + (g + 8) * D + 8 * j + 2 * t4) = make_float2(o[j][2], o[j][3]);
            }
        } else {
            constexpr int PC = A::CH / 4;         // chunks of a token's keys per lane (four lanes a token)
            constexpr int VC = D / 32;            // value channels per lane
            for (int c = tid; c < RP * D; c += kAttThreads)
                sm_q[c / D][c % D] = c / D < heads ? reinterpret_cast<const float *>(p.q)[hq * D + c] : 0.f;
            __syncthreads();
            float o[RP][VC], m[RP], l[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                m[r] = -INFINITY;
                l[r] = 0.f;
#pragma unroll
                for (int e = 0; e < VC; ++e) o[r][e] = 0.f;
            }
            const int tk = lane >> 2, part = lane & 3;
            for (int i = 0; i < mygroups; ++i) {
                cp_wait<kStages - 2>();
                __syncwarp();
                issue(i + kStages - 1, page);
                page = fetch(i + kStages);
                const int st = i % kStages;
                const uint8_t *kb = ring + st * A::STAGE, *vb = kb + A::GT * A::RB;
                const uint32_t mask = sm_mask[warp][st];
                float s[RP];
#pragma unroll
                for (int r = 0; r < RP; ++r) s[r] = 0.f;
#pragma unroll
                for (int j = 0; j < PC; ++j) {
                    const int ch = part + 4 * j;
                    const float4 kv = *reinterpret_cast<const float4 *>(kb + tk * A::RB + ((ch ^ A::swz(tk)) << 4));
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float4 qv = *reinterpret_cast<const float4 *>(&sm_q[r][4 * ch]);
                        s[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[r]))));
                    }
                }
                const bool in = (mask >> tk) & 1u;
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
                    s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
                    s[r] = in ? s[r] * sc : -INFINITY;
                    float mx = s[r];
#pragma unroll
                    for (int sft = 4; sft < 32; sft <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sft));
                    const float mn = fmaxf(m[r], mx), z = mn == -INFINITY ? 0.f : mn;
                    const float f = ex2(m[r] - z);
                    m[r] = mn;
                    s[r] = ex2(s[r] - z);
                    l[r] = fmaf(l[r], f, s[r]);
#pragma unroll
                    for (int e = 0; e < VC; ++e) o[r][e] *= f;
                }
#pragma unroll
                for (int t = 0; t < A::GT; ++t) {
                    float vv[VC];
                    const uint8_t *row = vb + t * A::RB;
                    if constexpr (VC == 4) {
                        const float4 x4 = *reinterpret_cast<const float4 *>(row + ((lane ^ A::swz(t)) << 4));
                        vv[0] = x4.x, vv[1] = x4.y, vv[2] = x4.z, vv[3] = x4.w;
                    } else {
                        const float2 x2 = *reinterpret_cast<const float2 *>(row + (((lane >> 1) ^ A::swz(t)) << 4) + 8 * (lane & 1));
                        vv[0] = x2.x, vv[1] = x2.y;
                    }
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float w = __shfl_sync(0xffffffffu, s[r], 4 * t);
#pragma unroll
                        for (int e = 0; e < VC; ++e) o[r][e] = fmaf(w, vv[e], o[r][e]);
                    }
                }
            }
            cp_wait<0>();
            __syncwarp();
            float *os = reinterpret_cast<float *>(ring);
#pragma unroll
            for (int r = 0; r < RP; ++r) {
#pragma unroll
                for (int sft = 4; sft < 32; sft <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], sft);
                if (lane == 0) {
                    sm_m[warp][r] = m[r];
                    sm_l[warp][r] = l[r];
                }
#pragma unroll
                for (int e = 0; e < VC; ++e) os[r * D + VC * lane + e] = o[r][e];
            }
        }
        __syncthreads();
        // join the warps; a whole unit's result is final, a part's goes to this CTA's slot 0 (its
        // first piece) or 1 (a later one)
        const int64_t slot = 2 * (int64_t)blockIdx.x + (first ? 0 : 1);
        for (int c = tid; c < heads * D; c += kAttThreads) {
            const int r = c / D;
            float mx = sm_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][r]);
            const float z = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sm_m[w][r] - z);
                sum = fmaf(sm_l[w][r], f, sum);
                acc = fmaf(reinterpret_cast<const float *>(ring_all + w * A::RING)[c], f, acc);
            }
            if (whole) {
                static_cast<T *>(p.out)[hq * D + c] = from_f<T>(sum == 0.f ? 0.f : acc / sum);
                if (p.lse && c % D == 0) p.lse[hq + r] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
            } else if constexpr (kShort) {
                reinterpret_cast<float *>(ring_all)[c] = acc;   // (read by this thread alone)
                if (c % D == 0) {
                    sm_pm[r] = mx;
                    sm_pl[r] = sum;
                }
            } else {
                a.part_o[slot * RP * D + c] = acc;
                if (c % D == 0) {
                    a.part_ml[(slot * RP + r) * 2] = mx;
                    a.part_ml[(slot * RP + r) * 2 + 1] = sum;
                }
            }
        }
        if constexpr (kShort) {
            if (whole) break;
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            for (int c = tid + kAttThreads * (int)cluster.block_rank(); c < heads * D; c += kAttThreads * a.cluster) {
                const int r = c / D;
                float mx = -INFINITY;
                for (int e = 0; e < a.cluster; ++e) mx = fmaxf(mx, cluster.map_shared_rank(sm_pm, e)[r]);
                const float z = mx == -INFINITY ? 0.f : mx;
                float sum = 0.f, acc = 0.f;
                for (int e = 0; e < a.cluster; ++e) {
                    const float f = ex2(cluster.map_shared_rank(sm_pm, e)[r] - z);
                    sum = fmaf(cluster.map_shared_rank(sm_pl, e)[r], f, sum);
                    acc = fmaf(reinterpret_cast<const float *>(cluster.map_shared_rank(ring_all, e))[c], f, acc);
                }
                static_cast<T *>(p.out)[hq * D + c] = from_f<T>(sum == 0.f ? 0.f : acc / sum);
                if (p.lse && c % D == 0) p.lse[hq + r] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
            }
            cluster.sync();   // the others have read this CTA's part
            break;
        }
        x = xe;
        if (x >= x1) break;
        us += items;          // the next unit
        if (++unit == per) {
            unit = 0;
            ++n;
            items = row_items(p, n);
        }
        __syncthreads();      // the rings and the warps' sums are read
    }
}

// Joins the parts of the units that fell into several shares, a head of the block per CTA.  Where there are
// few units (256 threads), one CTA per unit; else (128) one per boundary between two shares (blockIdx.x + 1
// is the share after it), which joins the unit that the boundary cuts, unless an earlier one cuts it too.
// Groups of D / 4 threads take every kGroups-th part, four of them at once, each group with a maximum
// and a sum of its own, which are joined in shared memory: a long row alone has some 300 parts, whose
// loads would otherwise wait for one another (a row of 100,000 tokens, one key/value head: 22 us for the
// whole call, 45 us with one group and a CTA per boundary).  Every CTA waits for the first kernel to
// end, so that nothing behind this kernel in the stream starts before that.
template <typename T, int D, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) kda_paged_join_kernel(const AttArgs a, const int ctas) {
    constexpr bool by_unit = kJoinThreads > 128;
    constexpr int kGroups = kJoinThreads / (D / 4), kAtOnce = 4;
    __shared__ long long sm_sum[kJoinThreads / 32];
    __shared__ float sm_m[kGroups], sm_l[kGroups];
    __shared__ __align__(16) float sm_o[kGroups][D];
    const PagedArgs &p = a.p;
    const int per = p.kv_heads * a.blocks, tid = threadIdx.x, r = blockIdx.y;
    long long mine = 0, ahead = 0;   // items of all rows (per unit), and of those before this CTA's
    int n = by_unit ? (int)blockIdx.x / per : 0;
    for (int i = tid; i < p.rows; i += kJoinThreads) {
        const int t = row_items(p, i);
        mine += t;
        ahead += i < n ? t : 0;
    }
    const long long W = per * block_sum<kJoinThreads>(mine, sm_sum);
    const long long G = W < ctas ? W : ctas;
    int unit = 0, h = a.rep, b0 = blockIdx.x, b1 = b0;   // the unit's first share and its last
    long long us = 0;
    if (by_unit) {
        unit = (int)blockIdx.x % per;
        const int items = row_items(p, n);
        us = per * block_sum<kJoinThreads>(ahead, sm_sum) + (long long)unit * items;
        b0 = (int)(((us + 1) * G - 1) / W);
        b1 = (int)(((us + items) * G - 1) / W);
        h = unit % a.blocks * a.rp + r;
    } else if (b0 + 1 < G) {
        const long long x = (b0 + 1) * W / G;
        find_row<kJoinThreads>(p, per, x, sm_sum, n, us);
        const int items = row_items(p, n);
        unit = (int)((x - us) / items);
        us += (long long)unit * items;
        h = unit % a.blocks * a.rp + r;
        if (x > us && b0 * W / G <= us) b1 = (int)(((us + items) * G - 1) / W);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (b1 == b0 || h >= a.rep) return;
    const int64_t s0 = 2 * (int64_t)b0 + (us > b0 * W / G ? 1 : 0);   // its part in b0; then slot 0 of b0 + 1 .. b1
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
    const int grp = tid / (D / 4), c4 = tid % (D / 4);
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = b0 + grp; b <= b1; b += kAtOnce * kGroups) {
        float2 v[kAtOnce];
        float4 o[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const int be = b + e * kGroups;
            const int64_t at = (be == b0 ? s0 : 2 * (int64_t)be) * a.rp + r;
            v[e] = be <= b1 ? __ldcg(ml + at) : make_float2(-INFINITY, 0.f);
            o[e] = be <= b1 ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
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
    *reinterpret_cast<float4 *>(&sm_o[grp][4 * c4]) = acc;
    if (c4 == 0) {
        sm_m[grp] = mx;
        sm_l[grp] = sum;
    }
    __syncthreads();
    if (tid >= D) return;
    mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < kGroups; ++e) mx = fmaxf(mx, sm_m[e]);
    const float z = mx == -INFINITY ? 0.f : mx;
    float out = 0.f;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < kGroups; ++e) {
        const float f = ex2(sm_m[e] - z);
        sum = fmaf(sm_l[e], f, sum);
        out = fmaf(sm_o[e][tid], f, out);
    }
    const int64_t hq = (int64_t)n * p.heads + (int64_t)(unit / a.blocks) * a.rep + h;
    static_cast<T *>(p.out)[hq * D + tid] = from_f<T>(sum == 0.f ? 0.f : out / sum);
    if (p.lse && tid == 0) p.lse[hq] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// Query heads of a block: 16 rows of the tensor-core tile, or in fp32 the least of 1, 4 and 8 that
// holds a key/value head's (more heads than that read the keys and values once per block).
int heads_per_block(kda_dtype_t dt, int rep) { return dt == KDA_BF16 ? 16 : (rep == 1 ? 1 : (rep <= 4 ? 4 : 8)); }

// Rows no longer than kShortTokens per CTA of a cluster take the one-launch form (a.cluster CTAs a unit):
// as many CTAs as the SMs hold, up to 8.  0: the rows may be longer.
constexpr int kShortTokens = 1024, kMaxCluster = 8;
int short_cluster(int64_t units, int64_t max_tokens, int d) {
    const int ctas = d == 64 ? 3 * kSms : kCtas;   // what the SMs hold at once
    int c = kMaxCluster;
    while (c > 1 && units * c > ctas) c /= 2;
    return max_tokens <= (int64_t)c * kShortTokens ? c : 0;
}

template <typename T, int D, int RP>
cudaError_t launch_att(const AttArgs &a, int grid, cudaStream_t st) {
    constexpr int smem = kWarps * Att<T, D>::RING;
    static_assert(RP * D * 4 <= Att<T, D>::RING, "a warp's outputs fit its ring");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.stream = st;
    cfg.attrs = at;
    if (a.cluster) {
        const cudaError_t e = cudaFuncSetAttribute(kda_paged_attention_kernel<T, D, RP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3((unsigned)((int64_t)a.p.rows * a.p.kv_heads * a.blocks * a.cluster));
        cfg.blockDim = dim3(kAttThreads);
        cfg.dynamicSmemBytes = smem;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)a.cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.numAttrs = a.cluster > 1 ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, kda_paged_attention_kernel<T, D, RP, true>, a);
    }
    cudaError_t e = cudaFuncSetAttribute(kda_paged_attention_kernel<T, D, RP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kda_paged_attention_kernel<T, D, RP, false><<<grid, kAttThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;   // (one CTA: nothing is split)
    const int64_t units = (int64_t)a.p.rows * a.p.kv_heads * a.blocks;
    const bool few = 2 * units <= grid;
    cfg.gridDim = dim3((unsigned)(few ? units : grid - 1), (unsigned)(a.rep < RP ? a.rep : RP));
    cfg.blockDim = dim3(few ? 256 : 128);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // the join's CTAs may start, find their parts
    at[0].val.programmaticStreamSerializationAllowed = 1;            // and wait before the first kernel has ended
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, kda_paged_join_kernel<T, D, 256>, a, grid) : cudaLaunchKernelEx(&cfg, kda_paged_join_kernel<T, D, 128>, a, grid);
}

// CTAs of the attention kernel: the items' share-out never needs more than there can be items.
int attention_ctas(int64_t rows, int64_t per, int64_t max_tokens) {
    const int64_t tiles = (max_tokens + kTile - 1) / kTile;
    if (rows * per >= kCtas || rows * per * tiles >= kCtas) return kCtas;
    return (int)(rows * per * tiles);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st) {
    // tokens of a CTA: what its threads request ahead, one at least
    int per = kAppendThreads * kAhead / a.row_vecs;
    per = per < 1 ? 1 : (per > kMaxTokens ? kMaxTokens : per);
    kda_paged_append_kernel<<<(unsigned)((a.tokens + per - 1) / per), kAppendThreads, 0, st>>>(a, per);
    return cudaGetLastError();
}

size_t paged_attention_workspace_bytes(int64_t rows, int heads, int kv_heads, int64_t max_tokens, int d, kda_dtype_t dt) {
    const int rep = heads / kv_heads, rp = heads_per_block(dt, rep), blocks = (rep + rp - 1) / rp;
    if (rows <= 0 || short_cluster(rows * kv_heads * blocks, max_tokens, d)) return 0;
    return (size_t)attention_ctas(rows, (int64_t)kv_heads * blocks, max_tokens) * 2 * rp * (d + 2) * 4;
}

cudaError_t launch_paged_attention(const PagedArgs &p, int d, kda_dtype_t dt, void *workspace, cudaStream_t st) {
    const int rep = p.heads / p.kv_heads, rp = heads_per_block(dt, rep), blocks = (rep + rp - 1) / rp;
    const int grid = attention_ctas(p.rows, (int64_t)p.kv_heads * blocks, (int64_t)p.max_pages * p.page_size);
    float *ws = static_cast<float *>(workspace);
    const AttArgs a{p, FastDiv((uint32_t)p.page_size), rep, blocks, rp, ws, ws ? ws + (size_t)grid * 2 * rp * d : nullptr,
                    short_cluster((int64_t)p.rows * p.kv_heads * blocks, (int64_t)p.max_pages * p.page_size, d)};
    if (dt == KDA_BF16)
        return d == 128 ? launch_att<__nv_bfloat16, 128, 16>(a, grid, st) : launch_att<__nv_bfloat16, 64, 16>(a, grid, st);
    if (d == 128)
        return rp == 1 ? launch_att<float, 128, 1>(a, grid, st) : rp == 4 ? launch_att<float, 128, 4>(a, grid, st) : launch_att<float, 128, 8>(a, grid, st);
    return rp == 1 ? launch_att<float, 64, 1>(a, grid, st) : rp == 4 ? launch_att<float, 64, 4>(a, grid, st) : launch_att<float, 64, 8>(a, grid, st);
}

}  // namespace kda
