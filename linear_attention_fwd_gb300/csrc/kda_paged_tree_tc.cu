// Attention of a draft's tokens over a paged cache on the sm_103a tensor cores (tcgen05 + TMEM + TMA), bf16.
//
// A unit has up to 256 query rows (drafted token x query head) of a row's key/value head; a CTA walks tiles of 128 keys
// with two chains of products, each with its scores and its outputs in tensor memory:
//   S = Q K^T (M = query rows, N = keys),   P = 2^(sc S - m) by the chain's warpgroup, a query row per thread,
//   O += P V, P from tensor memory as a rounded bf16 and the rounded rest (16 bits: one rounding alone would cost
//   2^-9 per weight, as much as the outputs' own rounding), V read across its rows.
// With more than 128 query rows the chains have 128 of them each and share the tiles; with fewer both have the same
// rows and take every second tile, and are joined at the end (a row's outputs of both chains lie in the same
// lane of tensor memory).  So one chain's softmax runs beside the other's products in either case.
// m follows the running maximum only where that has grown by more than 2^8, which is rare after the first
// tiles: then the chain's warpgroup scales O in tensor memory (its scores being there says that the
// product before has ended).
//
// Keys and values are gathered by TMA, four rows of the cache (page, offset, head) an instruction, so that pages
// of any size fit; places without a token (past the length, pages outside the pool) are rows past
// the tensor and arrive as zeros, and their scores are masked.  The drafted tokens have a tile of their own, masked
// by their paths.  A non-finite value among them is replaced by zero before the product (zero times NaN
// would reach other branches) and put back as NaN in the outputs of the tokens that weigh it.
//
// Roles: warps 0-3 and 4-7 the chains' softmax, warp 8 the loads, warp 9 the products (two more make up the warpgroup;
// 2 x 208 + 88 registers a thread out of the 3 x 168 of the launch).  They meet at mbarriers with bounded waits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_paged_tree.cuh"
#include "tc_ptx.cuh"

namespace kda {

// Count of bounded device waits that gave up since the host last read it.
__device__ unsigned int g_kda_tree_timeouts = 0;

namespace {

using namespace ptx;

constexpr int kThreads = 384, kRb = 256, kKt = 128;
constexpr int kRegsChain = 208, kRegsRest = 88;
constexpr float kSlack = 8.f;   // growth of the maximum, in powers of two, that m does not follow

template <int D> struct Tc {
    static constexpr uint32_t TILE = kKt * D * 2;                 // a tile of keys, of values, or of 128 query rows
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr uint32_t Q = 0, RING = 2 * TILE, MISC = RING + STAGES * TILE;
    static constexpr uint32_t BAR = MISC, MASK = BAR + 256, ANC = MASK + 8 * 16, UP = ANC + 512, ML = UP + 256;
    static constexpr uint32_t SEE = ML + 2 * 128 * 8, NF = SEE + 128 * 8, NFANY = NF + 2 * D * 8, TM = NFANY + 16;
    static constexpr uint32_t BYTES = TM + 16 + 1024;
    static_assert(BYTES <= 226 * 1024, "shared memory budget");
};
enum Bar { kFull = 0, kEmpty = 8, kQFull = 16, kQEmpty = 17, kS = 18 /* 2 */, kP = 20 /* 2 */, kO = 22 /* 2 */, kMeet = 24, kBars = 25 };

constexpr uint32_t TM_S = 0, TM_O = 256;   // + 128 for the second chain

__device__ __forceinline__ bool wait_small(uint32_t bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_wait(bar, parity & 1u, 1)) return true;
    return false;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(one));
    return one;
}
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Four rows of a two-dimensional tensor, 64 elements from x on: 4 x 128 bytes, one behind the other.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, const int (&r)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&w)[32]) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(w[i]);
    tmem_st32(taddr, v);
}

// A CTA's share of the items, piece by piece (every role walks it by itself).
struct Walk {
    long long x, x1, us;
    int n, unit;
    TreeRow row;
    // of the piece
    int hk, r0, rows, ta, c;    // key/value head, first query row, query rows, first tile, tiles
    bool whole, two;            // the whole unit; more than 128 rows
    long long xe;
    __device__ __forceinline__ void piece(const TreeAtt &a) {
        hk = unit / row.blocks;
        r0 = (unit - hk * row.blocks) * kRb;
        rows = row.m * a.rep - r0 < kRb ? row.m * a.rep - r0 : kRb;
        two = rows > 128;
        xe = us + row.items < x1 ? us + row.items : x1;
        whole = x == us && xe == us + row.items;
        const int ia = (int)(x - us) - kTreeStart, ib = (int)(xe - us) - kTreeStart;
        ta = ia > 0 ? ia : 0;
        c = ib - ta > 0 ? ib - ta : 0;
    }
    __device__ __forceinline__ bool next(const TreeAtt &a) {
        x = xe;
        if (x >= x1) return false;
        us += row.items;
        if (++unit == row.blocks * a.t.p.kv_heads) {
            unit = 0;
            do row = tree_row(a, ++n); while (row.m == 0);
        }
        piece(a);
        return true;
    }
    // Tiles of chain k, and the loads (counted within the piece) of tile i's keys and values: in the order of their use
    __device__ __forceinline__ int jobs(int k) const { return two ? c : (c + 1 - k) / 2; }
    __device__ __forceinline__ int tile(int k, int j) const { return two ? j : 2 * j + k; }
    __device__ __forceinline__ int k_load(int i) const { return two ? 2 * i : (i == 0 ? 0 : 2 * i - 1); }
    __device__ __forceinline__ int v_load(int i) const { return two ? 2 * i + 1 : (i < c - 1 ? 2 * i + 2 : 2 * c - 1); }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kda_paged_tree_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         const TreeAtt a, const uint32_t polls) {
    using L = Tc<D>;
    constexpr int S = L::STAGES, HALVES = D / 64;
    constexpr uint32_t HALF = L::TILE / HALVES;            // 64 channels of a tile's rows
    constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128), IDESC_PV = idesc_bf16_f32(128, D) | (1u << 16);   // B (V) MN-major
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long sm_sum[kThreads / 32];
    __shared__ int s_fail;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const PagedArgs &p = a.t.p;

    tree_clear<__nv_bfloat16, D, kThreads>(a, gridDim.x);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long W = tree_total<kThreads>(a, sm_sum);
    const long long G = W < gridDim.x ? W : gridDim.x;
    if (blockIdx.x >= G) return;
    Walk w;
    w.x = blockIdx.x * W / G;
    w.x1 = (blockIdx.x + 1) * W / G;
    tree_find<kThreads>(a, w.x, sm_sum, w.n, w.us);
    w.row = tree_row(a, w.n);
    w.unit = (int)((w.x - w.us) / w.row.items);
    w.us += w.unit * w.row.items;
    w.piece(a);
    const Walk start = w;

    auto bar = [&](int b) { return sb + L::BAR + 8 * b; };
    auto wait = [&](int b, uint32_t phase) { return wait_small(bar(b), phase, polls); };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    volatile int *nf_any = reinterpret_cast<volatile int *>(sm + L::NFANY);
    unsigned long long *nf = reinterpret_cast<unsigned long long *>(sm + L::NF);
    if (tid == 0) {
        s_fail = 0;
        nf_any[0] = nf_any[1] = 0;
        for (int s = 0; s < kQFull - kEmpty; ++s) {   // (also those past the stages: what gives up looks at all of them)
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1);
        }
        mbar_init(bar(kQFull), 1);
        mbar_init(bar(kQEmpty), 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(bar(kS + k), 2);     // the product, and the thread that issued it (which has seen the tile's masks)
            mbar_init(bar(kP + k), 4);     // the chain's warps
            mbar_init(bar(kO + k), 1);
        }
        mbar_init(bar(kMeet), 8);          // both chains' warps
        fence_mbar_init();
    }
    for (int x = tid; x < 2 * D; x += kThreads) nf[x] = 0;
    if (warp == 9) {
        tmem_alloc(sb + L::TM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sm + L::TM), 0);
    bool ok = true;

    if (warp < 8) {
        // ---- softmax
        regs_inc<kRegsChain>();
        const int k = warp >> 2, th = tid & 127;           // chain; query row of it
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16), ts = trow + TM_S + 128 * k;
        const float sc = p.scale * kLog2e;
        const uint32_t *masks = reinterpret_cast<const uint32_t *>(sm + L::MASK);
        uint64_t *anc = reinterpret_cast<uint64_t *>(sm + L::ANC);
        float2 *ml = reinterpret_cast<float2 *>(sm + L::ML);
        uint64_t *sees = reinterpret_cast<uint64_t *>(sm + L::SEE);
        uint32_t count = 0, ends = 0, tiles = 0, loads = 0, pieces = 0;   // phases so far
        uint32_t meets = 0;
        auto meet = [&] {   // all 256 threads of the chains
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kMeet));
            return all(wait(kMeet, meets++));
        };
        for (bool first = true;; first = false) {
            const bool has_draft = w.ta + w.c == w.row.tiles && w.c > 0;
            const int r = (w.two ? 128 * k : 0) + th;
            uint64_t see = 0;
            if (has_draft) {
                if (warp == 0) tree_masks(a, w.n, w.row.m, anc, reinterpret_cast<int *>(sm + L::UP));
                ok = meet();
                if (!ok) break;
                if (r < w.rows) see = anc[a.by_rep((uint32_t)(w.r0 + r))];
            }
            uint64_t weighs = 0;                            // drafted tokens with a weight
            float mr = -INFINITY, l = 0.f;
            const int jobs = w.jobs(k);
            for (int j = 0; j < jobs; ++j, ++count) {
                const int i = w.tile(k, j);
                const bool draft = w.ta + i == w.row.ctx;
                ok = all(wait(kS + k, count));
                if (!ok) break;
                tc_fence_after();
                const uint4 mk = *reinterpret_cast<const uint4 *>(masks + 4 * ((tiles + i) & 7));
                const bool open = !draft && (mk.x & mk.y & mk.z & mk.w) == 0xffffffffu;
                const uint32_t mw[4] = {mk.x, mk.y, mk.z, mk.w};   // column 4 x + e: bit x of word e
                auto in = [&](int col) {
                    const bool here = (mw[col & 3] >> (col >> 2)) & 1u;
                    return draft ? here && col < 64 && ((see >> (col & 63)) & 1u) : here;
                };
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[32];
                    tmem_ld32(ts + 32 * q, v);
                    if (open && sc >= 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) top = fmaxf(top, v[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (open || in(32 * q + e)) top = fmaxf(top, sc >= 0.f ? v[e] : -v[e]);
                    }
                }
                top = top == -INFINITY ? top : top * fabsf(sc);
                const bool grow = top > mr + kSlack || (mr == -INFINITY && top > mr);
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(mr - top) : 1.f;
                    if (grow) mr = top;
                    l *= f;
                    if (j > 0) {
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            float v[32];
                            tmem_ld32(trow + TM_O + 128 * k + 32 * q, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= f;
                            tmem_st32(trow + TM_O + 128 * k + 32 * q, v);
                        }
                    }
                }
                const float z = mr == -INFINITY ? 0.f : mr;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[32];
                    uint32_t u[32];   // 16 words of pairs, then of their rests: in the place of the scores that they come from
                    tmem_ld32(ts + 32 * q, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = ex2(fmaf(v[e], sc, -z));
                    if (!open) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = in(32 * q + e) ? v[e] : 0.f;
                        if (draft && q < 2) {
                            uint32_t bits = 0;
#pragma unroll
                            for (int e = 0; e < 32; ++e) bits |= v[e] != 0.f ? 1u << e : 0u;
                            weighs |= (uint64_t)bits << (32 * q);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[e & 3] += v[e];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        u[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                        const float2 b = unpack_bf16(u[e]);
                        u[16 + e] = pack_bf16(v[2 * e] - b.x, v[2 * e + 1] - b.y);
                    }
                    st32(ts + 32 * q, u);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (draft && (k == 0 || !w.two)) {
                    // the drafted tokens' values: what is not finite becomes zero
                    const int vl = (int)loads + w.v_load(i), st = vl % S;
                    ok = all(wait(kFull + st, vl / S));
                    if (!ok) break;
                    for (int x = th; x < w.row.m * (D / 8); x += 128) {
                        const int key = x / (D / 8), ch = x % (D / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(sm + L::RING + st * L::TILE + (ch >> 3) * HALF + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                        uint4 v = *at;
                        uint32_t *q = &v.x;
                        bool bad = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (((q[e] >> (16 * h)) & 0x7f80u) == 0x7f80u) {
                                    bad = true;
                                    q[e] &= h ? 0x0000ffffu : 0xffff0000u;
                                    atomicOr(nf + (pieces & 1) * D + 8 * ch + 2 * e + h, 1ull << key);
                                }
                        if (bad) {
                            *at = v;
                            nf_any[pieces & 1] = 1;
                            fence_async_smem();
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kP + k));
            }
            if (!ok) break;
            // outputs
            if (jobs > 0) ok = all(wait(kO + k, ends++));
            if (!ok) break;
            tc_fence_after();
            const bool stale = nf_any[(pieces + 1) & 1] != 0;
            if (!w.two) {
                ml[128 * k + th] = make_float2(mr, l);
                if (has_draft && ((w.c - 1) & 1) == k) sees[th] = weighs;   // (the chain that has the draft's tile)
            }
            ok = meet();
            if (!ok) break;
            tc_fence_after();
            const bool sick = has_draft && nf_any[pieces & 1] != 0;
            const unsigned long long *bad = nf + (pieces & 1) * D;
            if (has_draft && !w.two) weighs = sees[th];
            float f0 = 1.f, f1 = 0.f;
            const bool both = !w.two && w.c > 1;
            if (!w.two) {
                const float2 x0 = ml[th], x1 = ml[128 + th];
                mr = fmaxf(x0.x, x1.x);
                const float z = mr == -INFINITY ? 0.f : mr;
                f0 = ex2(x0.x - z);
                f1 = ex2(x1.x - z);
                l = fmaf(x0.y, f0, x1.y * f1);
            }
            if (w.two || w.c > 0) {
                // two: this chain's rows, all channels; else every row, this chain's half of the channels
                const int c0 = w.two ? 0 : k * (D / 2), c1 = w.two ? D : c0 + D / 2;
                const uint32_t to = trow + TM_O + (w.two ? 128 * k : 0);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int row = (int)a.by_rep((uint32_t)(w.r0 + r));
                const int64_t at = ((int64_t)w.n * a.t.tokens + row) * p.heads + w.hk * a.rep + (w.r0 + r - row * a.rep);
                const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * kRb + r;
                for (int ch = c0; ch < c1; ch += 32) {
                    float v[32];
                    tmem_ld32(to + ch, v);
                    if (!w.two) {
                        if (both) {
                            float y[32];
                            tmem_ld32(to + 128 + ch, y);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = fmaf(v[e], f0, y[e] * f1);
                        }
                    }
                    if (sick)
#pragma unroll 1
                        for (int e = 0; e < 32; ++e)
                            if (bad[ch + e] & weighs) {
#pragma unroll
                                for (int g = 0; g < 32; ++g) v[g] = g == e ? __int_as_float(0x7fc00000) : v[g];
                            }
                    if (r < w.rows) {
                        if (w.whole) {
                            uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at * D + ch);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t u[4];
#pragma unroll
                                for (int g = 0; g < 4; ++g) u[g] = pack_bf16(v[8 * e + 2 * g] * inv, v[8 * e + 2 * g + 1] * inv);
                                o[e] = l == 0.f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        } else {
                            float4 *o = reinterpret_cast<float4 *>(a.part_o + slot * D + ch);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                    }
                }
                if (r < w.rows && (w.two || k == 0)) {
                    if (w.whole) {
                        if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (mr + log2f(l)) * kLn2;
                    } else {
                        *reinterpret_cast<float2 *>(a.part_ml + 2 * slot) = make_float2(mr, l);
                    }
                }
            }
            if (w.c == 0) {   // a share that ends within a unit's start: nothing of it
                const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * kRb;
                for (int x = tid; x < w.rows * (D / 4); x += 256) reinterpret_cast<float4 *>(a.part_o + slot * D)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int x = tid; x < w.rows; x += 256) reinterpret_cast<float2 *>(a.part_ml + 2 * slot)[x] = make_float2(-INFINITY, 0.f);
            }
            if (stale) {   // the next piece starts with a clean slate
                for (int x = tid; x < D; x += 256) nf[((pieces + 1) & 1) * D + x] = 0;
                if (tid == 0) nf_any[(pieces + 1) & 1] = 0;
            }
            tc_fence_before();
            ok = meet();                                   // (the other chain has read its outputs, masks and sums)
            if (!ok) break;
            tiles += w.c;
            loads += 2 * w.c;
            ++pieces;
            if (!w.next(a)) break;
        }
    } else if (warp >= 10) {
        regs_dec<kRegsRest>();
    } else if (warp == 8) {
        // ---- loads
        regs_dec<kRegsRest>();
        const int none = p.pages * p.page_size * p.kv_heads, noq = p.rows * a.t.tokens * p.heads;   // rows past the tensors
        uint32_t load = 0, qs = 0, tiles = 0;
        for (;; ) {
            if (w.c > 0) {
                const int32_t *table = p.table + (int64_t)w.n * p.max_pages;
                auto places = [&](int i, int (&r)[4]) {
                    const int t = w.ta + i;
                    const bool draft = t == w.row.ctx;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * lane + e + (draft ? 0 : t * kKt);
                        const int64_t at = j < (draft ? w.row.m : w.row.len) ? tree_place(a, table, draft ? w.row.len + j : j) : -1;
                        r[e] = at < 0 ? none : (int)(at * p.kv_heads) + w.hk;
                    }
                };
                auto tile = [&](const CUtensorMap *map, const int (&r)[4]) {
                    const int s = load % S;
                    ok = all(load < S || wait(kEmpty + s, load / S - 1));
                    if (!ok) return false;
                    if (lane == 0) mbar_arrive_expect_tx(bar(kFull + s), L::TILE);
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) tma_gather4(sb + L::RING + s * L::TILE + h * HALF + lane * 512, map, bar(kFull + s), 64 * h, r);
                    ++load;
                    return true;
                };
                auto mask = [&](int i, const int (&r)[4]) {
                    uint32_t m[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = __ballot_sync(0xffffffffu, r[e] != none);
                    if (lane == 0) *reinterpret_cast<uint4 *>(sm + L::MASK + 16 * ((tiles + i) & 7)) = make_uint4(m[0], m[1], m[2], m[3]);
                    __syncwarp();
                };
                int r[4], next[4];
                places(0, r);
                // the queries
                ok = all(qs == 0 || wait(kQEmpty, qs - 1));
                if (!ok) break;
                ++qs;
                if (lane == 0) mbar_arrive_expect_tx(bar(kQFull), (w.two ? 2 : 1) * L::TILE);
                __syncwarp();
                for (int b = 0; b < (w.two ? 2 : 1); ++b) {
                    int qr[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int x = 128 * b + 4 * lane + e, i = (int)a.by_rep((uint32_t)(w.r0 + x));
                        qr[e] = x < w.rows ? (w.n * a.t.tokens + i) * p.heads + w.hk * a.rep + (w.r0 + x - i * a.rep) : noq;
                    }
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) tma_gather4(sb + L::Q + b * L::TILE + h * HALF + lane * 512, &tmq, bar(kQFull), 64 * h, qr);
                }
                mask(0, r);
                if (!tile(&tmk, r)) break;
                bool fine = true;
                for (int i = 0; i < w.c && fine; ++i) {
                    if (i + 1 < w.c) places(i + 1, next);
                    if (!w.two && i + 1 < w.c) {
                        mask(i + 1, next);
                        fine = tile(&tmk, next);
                    }
                    fine = fine && tile(&tmv, r);
                    if (w.two && i + 1 < w.c && fine) {
                        mask(i + 1, next);
                        fine = tile(&tmk, next);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = next[e];
                }
                if (!fine) break;
                tiles += w.c;
            }
            if (!w.next(a)) break;
        }
    } else {
        // ---- products; an elected lane issues
        regs_dec<kRegsRest>();
        const uint32_t one = elect_one();
        uint32_t loads = 0, qs = 0, jobs[2] = {0, 0};
        const uint64_t qd = sdesc_sw128(sb + L::Q), kd = sdesc_sw128(sb + L::RING), vd = sdesc_sw128_mn(sb + L::RING, HALF, 1024);
        for (;; ) {
            if (w.c > 0) {
                // scores of chain k, tile i; `loaded`: the tile has been waited for, `last`: its last use
                auto qk = [&](int k, int i, bool loaded, bool last) {
                    const int ld = (int)loads + w.k_load(i), s = ld % S;
                    ok = all(loaded || wait(kFull + s, ld / S));
                    if (!ok) return false;
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                            mma_f16_ss(tmem + TM_S + 128 * k, qd + (w.two ? k * (L::TILE >> 4) : 0) + off, kd + s * (L::TILE >> 4) + off, IDESC_QK, kk > 0);
                        }
                        mma_commit(bar(kS + k));
                        mbar_arrive(bar(kS + k));
                        if (last) mma_commit(bar(kEmpty + s));
                    }
                    __syncwarp();
                    return true;
                };
                // outputs of chain k, tile i, its j-th
                auto pv = [&](int k, int i, int j, bool loaded, bool last) {
                    const int ld = (int)loads + w.v_load(i), s = ld % S;
                    ok = all((loaded || wait(kFull + s, ld / S)) && wait(kP + k, jobs[k]));
                    if (!ok) return false;
                    ++jobs[k];
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int e = 1; e >= 0; --e)   // the rests first
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_f16_ts(tmem + TM_O + 128 * k, tmem + TM_S + 128 * k + 32 * (kk >> 1) + 8 * (kk & 1) + 16 * e,
                                           vd + s * (L::TILE >> 4) + ((2048 * kk) >> 4), IDESC_PV, j > 0 || e == 0 || kk > 0);
                        if (last) mma_commit(bar(kEmpty + s));
                        if (j + 1 == w.jobs(k)) mma_commit(bar(kO + k));
                    }
                    __syncwarp();
                    return true;
                };
                ok = all(wait(kQFull, qs++));
                if (!ok) break;
                bool fine = true;
                if (w.two) {
                    fine = qk(0, 0, false, false) && qk(1, 0, true, true);
                    for (int i = 0; i < w.c && fine; ++i) {
                        const bool more = i + 1 < w.c;
                        fine = pv(0, i, i, false, false) && (!more || qk(0, i + 1, false, false)) && pv(1, i, i, true, true) && (!more || qk(1, i + 1, true, true));
                        if (fine && i + 2 >= w.c && (more || w.c == 1) && one) mma_commit(bar(kQEmpty));
                    }
                } else {
                    fine = qk(0, 0, false, true) && (w.c < 2 || qk(1, 1, false, true));
                    if (fine && w.c <= 2 && one) mma_commit(bar(kQEmpty));
                    for (int i = 0; i < w.c && fine; ++i) {
                        fine = pv(i & 1, i, i >> 1, false, true) && (i + 2 >= w.c || qk(i & 1, i + 2, false, true));
                        if (fine && i + 3 == w.c && one) mma_commit(bar(kQEmpty));
                    }
                }
                __syncwarp();
                if (!fine) break;
                loads += 2 * w.c;
            }
            if (!w.next(a)) break;
        }
        // nothing arrives at a barrier after the CTA has ended
        for (uint32_t ld = loads > S ? loads - S : 0; ok && ld < loads; ++ld) ok = all(wait(kEmpty + ld % S, ld / S));
        if (ok && qs > 0) ok = all(wait(kQEmpty, qs - 1));
    }
    __syncwarp();
    if (!ok) s_fail = 1;
    tc_fence_before();
    __syncthreads();
    if (s_fail) {
        // A bounded wait gave up.  What is in flight lands first (each barrier that it completes is given a few
        // milliseconds for both parities), then all of the share's results are marked.
        if (tid == 0) {
            for (int b = 0; b < kBars; ++b) {
                wait_small(bar(b), 0, 1u << 12);
                wait_small(bar(b), 1, 1u << 12);
            }
            atomicAdd(&g_kda_tree_timeouts, 1u);
        }
        const float nan = __int_as_float(0x7fc00000);
        w = start;
        for (bool first = true;; first = false) {
            const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * kRb;
            for (int x = tid; x < w.rows * D; x += kThreads) {
                const int r = x / D, i = (int)a.by_rep((uint32_t)(w.r0 + r));
                const int64_t at = ((int64_t)w.n * a.t.tokens + i) * p.heads + w.hk * a.rep + (w.r0 + r - i * a.rep);
                if (w.whole) {
                    static_cast<__nv_bfloat16 *>(p.out)[at * D + x % D] = __float2bfloat16(nan);
                    if (p.lse && x % D == 0) p.lse[at] = nan;
                } else {
                    a.part_o[(slot + r) * D + x % D] = nan;
                    if (x % D == 0) a.part_ml[2 * (slot + r)] = a.part_ml[2 * (slot + r) + 1] = nan;
                }
            }
            if (!w.next(a)) break;
        }
        __syncthreads();
    }
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                   : nullptr;
    }();
    return fn;
}

// [rows][d] bf16 for gathers: boxes of 64 channels of one row, 128-byte swizzle; rows past the tensor are zeros.
bool make_map(CUtensorMap *m, const void *ptr, int64_t rows, int d) {
    auto enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    cuuint32_t box[2] = {64, 1};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs: one per SM, never more than there can be items.
int tc_ctas(const PagedTreeArgs &t) {
    const int rep = t.p.heads / t.p.kv_heads;
    const int64_t units = (int64_t)t.p.rows * t.p.kv_heads * (((int64_t)t.tokens * rep + kRb - 1) / kRb);
    const int64_t items = ((int64_t)t.p.max_pages * t.p.page_size + kKt - 1) / kKt + 1 + kTreeStart;
    return units >= kSms || units * items >= kSms ? kSms : (int)(units * items);
}

template <int D> cudaError_t launch_tc(const TreeAtt &a, int ctas, uint32_t polls, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    const PagedArgs &p = a.t.p;
    const int64_t cached = (int64_t)p.pages * p.page_size * p.kv_heads;
    if (!make_map(&mq, p.q, (int64_t)p.rows * a.t.tokens * p.heads, D) || !make_map(&mk, p.k_cache, cached, D) || !make_map(&mv, p.v_cache, cached, D))
        return cudaErrorInvalidValue;
    // what the roles' shares of registers add up to has to be there at the launch, else they would wait for ever
    static const bool enough = [] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kda_paged_tree_tc_kernel<D>) == cudaSuccess && f.numRegs * kThreads >= 256 * kRegsChain + 128 * kRegsRest;
    }();
    if (!enough) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kda_paged_tree_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tc<D>::BYTES);
    if (e != cudaSuccess) return e;
    kda_paged_tree_tc_kernel<D><<<ctas, kThreads, Tc<D>::BYTES, st>>>(mq, mk, mv, a, polls);
    e = cudaGetLastError();
    return e != cudaSuccess || ctas == 1 ? e : launch_tree_join(a, D, KDA_BF16, ctas, st);   // (one CTA: nothing is split)
}

}  // namespace

size_t tree_tc_workspace_bytes(const PagedTreeArgs &t, int d) { return (size_t)tc_ctas(t) * 2 * kRb * (d + 2) * 4; }

cudaError_t launch_tree_tc(const PagedTreeArgs &t, int d, void *workspace, uint32_t polls, cudaStream_t st) {
    const int rep = t.p.heads / t.p.kv_heads, ctas = tc_ctas(t);
    float *ws = static_cast<float *>(workspace);
    const TreeAtt a{t, FastDiv((uint32_t)t.p.page_size), FastDiv((uint32_t)rep), rep, kRb, kKt, ws, ws + (size_t)ctas * 2 * kRb * d};
    return d == 128 ? launch_tc<128>(a, ctas, polls, st) : launch_tc<64>(a, ctas, polls, st);
}

cudaError_t take_tree_expiries(cudaStream_t st, unsigned int *count) {
    static const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_kda_tree_timeouts, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_kda_tree_timeouts, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace kda
