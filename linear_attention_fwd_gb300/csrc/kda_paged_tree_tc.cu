// Attention of a draft's tokens over a paged cache on the sm_103a tensor cores (tcgen05 + TMEM + TMA), bf16.
//
// A unit has up to 256 query rows (drafted token x query head) of a row's key/value head; a CTA walks tiles of 64 keys
// with two chains of products, each with its outputs and two buffers of scores in tensor memory:
//   S = Q K^T (M = query rows, N = keys),   P = 2^(sc S - m) by the chain's warpgroup, a query row per thread,
//   O += P V, P from tensor memory as the upper half of its bits and the rounded rest (16 bits: bf16 alone would cost
//   2^-9 per weight, as much as the outputs' own rounding), V read across its rows.
// With more than 128 query rows the chains have 128 of them each and share the tiles; with fewer both have the same
// rows and take every second tile, and are joined at the end (a row's outputs of both chains lie in the same
// lane of tensor memory).  A chain's next scores are made while its softmax runs, so that the softmax waits for
// nothing but a tile's arrival.
// m follows the running maximum only where that has grown by more than 2^8, which is rare after the first
// tiles: then the chain's warpgroup waits for the last product into O and scales it in tensor memory.
//
// Tiles on pages of a multiple of 8 tokens come by TMA, a box of tokens an instruction, and so do the queries where a
// power of two of heads shares a key/value head; others, and most drafts, by cp.async.
// Scores of places without a token are masked, their values made zero behind the load.  (Gathers of four rows by TMA
// take 50 ns each, 6.5 us for 128 keys of 128 channels: 131,071 tokens x 8 heads, 512 query rows: 700 us, 430 by boxes at
// the time.)  The drafted tokens have a tile of their own, masked by their paths.  A non-finite value among them is replaced by zero before the product (zero
// times NaN would reach other branches) and put back as NaN in the outputs of the tokens that weigh it.
//
// Roles: warps 0-7 and 8-15 the chains' softmax, half of a tile's keys each four (a row's two threads agree on m; with
// one thread per row a chain's softmax took 2600 cycles a tile, mostly waits of its one warp per scheduler for its own
// results, twice the products' time); warps 16 and 17 the chains' products, 18 the keys' loads, 19 the values' and queries'.  They meet at mbarriers
// with bounded waits.
//
// With 256 query rows bound by the softmax and its hand-overs: 64 keys take 2260 cycles, 1900 of them the softmax warps' work,
// the products 1536 (the rests are a third); tensor pipe 61 % busy, instruction issue 60 %.  131,071 tokens x 8 heads, 512
// query rows a head: 292 to 311 us on different GPUs, 0.9 PFLOP/s without the rests, 1.36 with them.  With 128 rows or fewer a tile takes 1500 cycles,
// 5.9 TB/s of keys and values, and a unit's start and end 20 thousand beside them: 32 rows of 200 to 16,384 tokens, 8
// heads, 32 to 128 query rows each: 128 us, 4.0 TB/s.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_paged_tree.cuh"
#include "tc_ptx.cuh"

namespace kda {

// Count of bounded device waits that gave up since the host last read it.
__device__ unsigned int g_kda_tree_timeouts = 0;

namespace {

using namespace ptx;

// kStart: 5 is within 2.5 % of the best of 3, 5, 8 and 13 in each of twelve batches of short, mixed and long rows (3 up to 7 % slower:
// the batch above 137 us; 8 up to 7 %: 64 rows of 300 to 3000 tokens 95 us for 89; 13 up to 25 %: 102 rows of up to 1285 tokens 81 for 65),
// although a short row's unit takes as long as more tiles: units of a few tiles are then cut less often, and whole ones are unequal.
constexpr int kThreads = 640, kRb = 256, kKt = 64, kStart = 5;
static_assert(kRb == 1 << 8 && kKt == 1 << 6, "their logarithms");
constexpr float kSlack = 8.f;   // growth of the maximum, in powers of two, that m does not follow

template <int D> struct Tc {
    static constexpr uint32_t TILE = kKt * D * 2, QTILE = 128 * D * 2;   // keys or values; query rows of a chain
    static constexpr int STAGES = D == 128 ? 9 : 16;
    static constexpr uint32_t Q = 0, RING = 2 * QTILE, BAR = RING + STAGES * TILE;
    static constexpr uint32_t MASK = BAR + 512, ANC = MASK + 32 * 8, UP = ANC + 1024, ML = UP + 256;
    static constexpr uint32_t SEE = ML + 6 * 128 * 4, NF = SEE + 4 * 128 * 4, NFANY = NF + 2 * D * 8, TM = NFANY + 16;
    static constexpr uint32_t BYTES = TM + 16 + 1024;
    static_assert(BYTES <= 226 * 1024, "shared memory budget");
};
// kS, kP and kV are of a chain and a buffer (2 k + b): scores, weights, outputs.  A wait names a phase by its parity, so a
// barrier may be at most one phase behind what is waited for and none ahead.  That holds because the scores of a
// chain's tile j follow the outputs of its tile j - 2, and those of tile j the weights that their waiter makes.
enum Bar { kFull = 0, kEmpty = 16, kQFull = 32, kQEmpty = 33, kS = 34, kP = 38, kV = 42, kMeet = 46, kBars = 47 };

constexpr uint32_t TM_S = 0, TM_O = 256;   // + 128 for the second chain, + 64 for the second buffer

__device__ __forceinline__ bool wait_small(uint32_t bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_wait(bar, parity & 1u, 1)) return true;
    return false;
}
__device__ __forceinline__ bool test(uint32_t bar, uint32_t parity) {   // without waiting
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity & 1u)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
// Barrier `id` of 256 threads: whether x holds in any of them.
__device__ __forceinline__ bool any_of(int id, bool x) {
    uint32_t y;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y)
                 : "r"((uint32_t)x), "r"(id)
                 : "memory");
    return y != 0;
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(one));
    return one;
}

// Shared-memory operand descriptors here differ in their low words only: address, and for operands read across their rows
// the distance of their 64-channel halves.  The rest: 8-row groups 1024 bytes apart, version 1, 128-byte swizzle (see
// sdesc_sw128, sdesc_sw128_mn).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
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
        const int ia = (int)(x - us) - a.start, ib = (int)(xe - us) - a.start;
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
    // Chain k has jobs(k) tiles, the j-th is tile(k, j).  Scores are made `ahead` tiles ahead of the outputs; the loads of
    // tile i's keys and values, counted within the piece, are in that order.
    __device__ __forceinline__ int jobs(int k) const { return two ? c : (c + 1 - k) / 2; }
    __device__ __forceinline__ int tile(int k, int j) const { return two ? j : 2 * j + k; }
    __device__ __forceinline__ int ahead() const { return two ? 2 : 4; }
    // The drafted tokens' row in their tile where it comes by boxes (from the start of a box of the cache on), -1 where it does not
    __device__ __forceinline__ int shift(int box) const {
        const int o = box ? row.len & (box - 1) : 0;
        return box && o + row.m <= kKt ? o : -1;
    }
    __device__ __forceinline__ int k_load(int i) const { return i < ahead() ? i : 2 * i + 1 - ahead(); }
    __device__ __forceinline__ int v_load(int i) const { return i < c - ahead() ? 2 * i + ahead() : c + i; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kda_paged_tree_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         const TreeAtt a, const int qbox, const int box, const uint32_t polls) {
    using L = Tc<D>;
    constexpr int S = L::STAGES, HALVES = D / 64;
    constexpr uint32_t HALF = L::TILE / HALVES, QHALF = L::QTILE / HALVES;   // 64 channels of a tile's rows
    constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, kKt), IDESC_PV = idesc_bf16_f32(128, D) | (1u << 16);   // B (V) MN-major
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long sm_sum[kThreads / 32];
    __shared__ int s_fail;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const PagedArgs &p = a.t.p;

    if (tid == 0) {
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long W, G;
    Walk w;
    if (!tree_share<kThreads>(a, sm_sum, W, G, w.x, w.x1, w.n, w.us)) return;
    w.row = tree_row(a, w.n);
    w.unit = tree_quotient(w.x - w.us, w.row.items);
    w.us += w.unit * w.row.items;
    w.piece(a);

    auto bar = [&](int b) { return sb + L::BAR + 8 * b; };
    auto wait = [&](int b, uint32_t phase) { return wait_small(bar(b), phase, polls); };
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    volatile int *nf_any = reinterpret_cast<volatile int *>(sm + L::NFANY);
    unsigned long long *nf = reinterpret_cast<unsigned long long *>(sm + L::NF);
    if (tid == 0) {
        s_fail = 0;
        nf_any[0] = nf_any[1] = 0;
        for (int s = 0; s < 16; ++s) {             // (also those past the stages: what gives up looks at all of them)
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 2);         // both chains
        }
        mbar_init(bar(kQFull), 1);
        mbar_init(bar(kQEmpty), 2);                // both chains
        for (int x = 0; x < 4; ++x) {
            mbar_init(bar(kS + x), 2);             // the product, and the thread that issued it (which has seen the tile's masks)
            mbar_init(bar(kP + x), 8);             // the chain's warps
            mbar_init(bar(kV + x), 1);
        }
        mbar_init(bar(kMeet), 16);                 // both chains' warps
        fence_mbar_init();
    }
    for (int x = tid; x < 2 * D; x += kThreads) nf[x] = 0;
    if (warp == 16) {
        tmem_alloc(sb + L::TM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sm + L::TM), 0);
    bool ok = true;

    if (warp < 16) {
        // ---- softmax
        const int k = warp >> 3, half = (warp >> 2) & 1, th = tid & 127;   // chain; half of a tile's keys; query row
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = p.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc);
        const uint2 *masks = reinterpret_cast<const uint2 *>(sm + L::MASK);
        const uint64_t *anc = reinterpret_cast<const uint64_t *>(sm + L::ANC);         // [piece's parity][token]
        float *tops = reinterpret_cast<float *>(sm + L::ML), *sums = tops + 2 * 128;   // [chain][row]; [chain][half][row]
        uint32_t *sees = reinterpret_cast<uint32_t *>(sm + L::SEE);                    // [chain][half][row]
        uint32_t count = 0, meets = 0, tiles = 0, loads = 0, pieces = 0;   // jobs, barriers, tiles, loads and pieces so far
        auto outputs = [&] { return all(wait(kV + 2 * k + (int)((count - 1) & 1), (count - 1) >> 1)); };   // of the chain's last tile
        auto meet = [&] {   // all 512 threads of the chains
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kMeet));
            const uint32_t phase = meets++;
            return ok && all(wait(kMeet, phase));
        };
        // A warp that has given up (!ok) goes on without waiting until its chain leaves together, at one of the chain's barriers.
        bool gone = false;
        for (bool first = true;; first = false) {
            const bool has_draft = w.ta + w.c == w.row.tiles && w.c > 0;
            const int r = (w.two ? 128 * k : 0) + th;
            uint32_t weighs = 0;                            // drafted tokens with a weight
            float mr = -INFINITY, l = 0.f;
            const int jobs = w.jobs(k);
            for (int j = 0; j < jobs; ++j, ++count) {
                const int i = w.tile(k, j), b = 2 * k + (int)(count & 1);
                const bool draft = w.ta + i == w.row.ctx;
                ok = ok && all(wait(kS + b, count >> 1));
                tc_fence_after();
                const uint32_t ts = trow + TM_S + 64 * b + 32 * half;
                float v[32];
                tmem_ld32(ts, v);
                const uint2 here = masks[(tiles + i) & 31];   // places with a token
                uint32_t in = half ? here.y : here.x;
                const bool open = !draft && (here.x & here.y) == 0xffffffffu;   // (the same for the row's two threads)
                if (!open) {
                    if (draft) in &= r < w.rows ? (uint32_t)((anc[64 * (pieces & 1) + a.by_rep((uint32_t)(w.r0 + r))] << max(w.shift(box), 0)) >> (32 * half)) : 0u;
                    const float no = sc >= 0.f ? -INFINITY : INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = (in >> e) & 1u ? v[e] : no;
                }
                float top;
                {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = v[e];
                    if (sc >= 0.f) {
#pragma unroll
                        for (int e = 4; e < 32; e += 8)
#pragma unroll
                            for (int f = 0; f < 4; ++f) x[f] = e + 4 < 32 ? fmaxf(fmaxf(x[f], v[e + f]), v[(e + 4 + f) & 31]) : fmaxf(x[f], v[e + f]);
                        top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    } else {
#pragma unroll
                        for (int e = 4; e < 32; e += 4)
#pragma unroll
                            for (int f = 0; f < 4; ++f) x[f] = fminf(x[f], v[e + f]);
                        top = -fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
                    }
                }
                top = top == -INFINITY ? top : top * fabsf(sc);
                // the chain's threads go on together: where one has given up, or a row's maximum has grown
                if (any_of(1 + k, !ok || top > mr + kSlack || (mr == -INFINITY && top > mr))) {
                    if (any_of(1 + k, !ok)) {
                        gone = true;
                        break;
                    }
                    // (a row's two threads hand their maxima to one another in `sums`)
                    sums[(2 * k + half) * 128 + th] = top;
                    any_of(1 + k, false);
                    top = fmaxf(top, sums[(2 * k + (half ^ 1)) * 128 + th]);
                    any_of(1 + k, false);
                    const bool grow = top > mr + kSlack || (mr == -INFINITY && top > mr);
                    const float f = grow ? ex2(mr - top) : 1.f;
                    if (grow) mr = top;
                    l *= f;
                    if (j > 0) {
                        ok = outputs();
                        if (any_of(1 + k, !ok)) {
                            gone = true;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 64; ++q) {   // this half's channels
                            const uint32_t to = trow + TM_O + 128 * k + half * (D / 2) + 32 * q;
                            float o[32];
                            tmem_ld32(to, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tmem_st32(to, o);
                        }
                    }
                }
                const float z = mr == -INFINITY ? 0.f : -mr;
                const float2 z2 = make_float2(z, z);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y = __ffma2_rn(make_float2(v[e], v[e + 1]), sc2, z2);
                    v[e] = ex2(y.x);
                    v[e + 1] = ex2(y.y);
                }
                if (!open) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = (in >> e) & 1u ? v[e] : 0.f;
                        bits |= v[e] != 0.f ? 1u << e : 0u;
                    }
                    if (draft) weighs = bits;
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                float u[32];   // 16 pairs of upper halves, then of the rests: in the place of the scores that they come from
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 x = make_float2(v[e], v[e + 1]);
                    sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], x);
                    const uint32_t a0 = __float_as_uint(x.x), a1 = __float_as_uint(x.y);
                    u[e / 2] = __uint_as_float(__byte_perm(a0, a1, 0x7632));
                    const float2 rest = __ffma2_rn(make_float2(__uint_as_float(a0 & 0xffff0000u), __uint_as_float(a1 & 0xffff0000u)), make_float2(-1.f, -1.f), x);
                    u[16 + e / 2] = __uint_as_float(pack_bf16(rest.x, rest.y));
                }
                tmem_st32(ts, u);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (!open) {
                    // values of places without a token become zero, and what is not finite among the drafted tokens' (by each
                    // chain that reads them, so that neither waits for the other: the second finds or writes the same)
                    const int vl = (int)loads + w.v_load(i), st = vl % S;
                    ok = ok && all(wait(kFull + st, vl / S));
                    if (ok)
#pragma unroll 1
                        for (int x0 = 0; x0 < kKt * (D / 8); x0 += 256) {
                            const int x = x0 + 128 * half + th, key = x / (D / 8), ch = x % (D / 8);
                            uint4 *at = reinterpret_cast<uint4 *>(sm + L::RING + st * L::TILE + (ch >> 3) * HALF + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                            const bool token = ((key < 32 ? here.x : here.y) >> (key & 31)) & 1u;
                            uint4 y = token && draft ? *at : make_uint4(0u, 0u, 0u, 0u);
                            auto ones = [](uint32_t z) { return (z & 0x7f807f80u) + 0x00800080u; };   // bits 15, 31: an exponent of all ones
                            const uint32_t full = ones(y.x) | ones(y.y) | ones(y.z) | ones(y.w);
                            if (full & 0x80008000u) {
#pragma unroll 1
                                for (int e = 0; e < 8; ++e) {
                                    uint32_t z = e < 4 ? (e < 2 ? y.x : y.y) : (e < 6 ? y.z : y.w);
                                    if (((z >> (16 * (e & 1))) & 0x7f80u) != 0x7f80u) continue;
                                    z &= e & 1 ? 0x0000ffffu : 0xffff0000u;
                                    if (e < 2) y.x = z;
                                    else if (e < 4) y.y = z;
                                    else if (e < 6) y.z = z;
                                    else y.w = z;
                                    atomicOr(nf + (pieces & 1) * D + 8 * ch + e, 1ull << key);
                                    nf_any[pieces & 1] = 1;
                                }
                            }
                            if (!token || (full & 0x80008000u)) *at = y;
                        }
                    fence_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kP + b));
            }
            if (gone) break;
            // outputs
            if (jobs > 0) ok = ok && outputs();
            tc_fence_after();
            const bool stale = nf_any[(pieces + 1) & 1] != 0;
            if (half == 0) tops[128 * k + th] = mr;
            sums[(2 * k + half) * 128 + th] = l;
            if (has_draft && (w.two || ((w.c - 1) & 1) == k)) sees[((w.two ? 2 * k : 0) + half) * 128 + th] = weighs;   // (of the chain that has the draft)
            tc_fence_before();
            ok = meet();
            tc_fence_after();
            const bool sick = has_draft && nf_any[pieces & 1] != 0;
            const bool both = !w.two && w.c > 1;
            float f0 = 1.f, f1 = 0.f;
            if (w.two) {
                l = sums[2 * k * 128 + th] + sums[(2 * k + 1) * 128 + th];
            } else {
                const float x0 = tops[th], x1 = tops[128 + th];
                mr = fmaxf(x0, x1);
                const float z = mr == -INFINITY ? 0.f : mr;
                f0 = ex2(x0 - z);
                f1 = ex2(x1 - z);
                l = fmaf(sums[th] + sums[128 + th], f0, (sums[256 + th] + sums[384 + th]) * f1);
            }
            if (w.c > 0) {
                // two: this chain's rows, this half of the channels; else every row, 32 channels of each warpgroup
                const int c0 = w.two ? half * (D / 2) : 32 * (2 * k + half), c1 = w.two ? c0 + D / 2 : (c0 < D ? c0 + 32 : c0);
                const uint32_t to = trow + TM_O + (w.two ? 128 * k : 0);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int row = (int)a.by_rep((uint32_t)(w.r0 + r));
                const int64_t at = ((int64_t)w.n * a.t.tokens + row) * p.heads + w.hk * a.rep + (w.r0 + r - row * a.rep);
                const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * kRb + r;
#pragma unroll 1
                for (int ch = c0; ch < c1; ch += 32) {
                    float v[32];
                    tmem_ld32(to + ch, v);
                    if (both) {
                        float y[32];
                        tmem_ld32(to + 128 + ch, y);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = fmaf(v[e], f0, y[e] * f1);
                    }
                    if (sick) {
                        // drafted tokens' values that are not finite, where they are weighed
                        const uint32_t *mask = sees + (w.two ? 256 * k : 0) + th;
                        const uint64_t mine = (uint64_t)mask[128] << 32 | mask[0];
                        const unsigned long long *bad = nf + (pieces & 1) * D + ch;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (bad[e] & mine) v[e] = __int_as_float(0x7fc00000);
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
                if (r < w.rows && half == 0 && (w.two || k == 0)) {
                    if (w.whole) {
                        if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (mr + log2f(l)) * kLn2;
                    } else {
                        *reinterpret_cast<float2 *>(a.part_ml + 2 * slot) = make_float2(mr, l);
                    }
                }
            } else {   // a share that ends within a unit's start: nothing of it
                const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * kRb;
                for (int x = tid; x < w.rows * (D / 4); x += 512) reinterpret_cast<float4 *>(a.part_o + slot * D)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int x = tid; x < w.rows; x += 512) reinterpret_cast<float2 *>(a.part_ml + 2 * slot)[x] = make_float2(-INFINITY, 0.f);
            }
            if (stale) {   // the next piece starts with a clean slate
                for (int x = tid; x < D; x += 512) nf[((pieces + 1) & 1) * D + x] = 0;
                if (tid == 0) nf_any[(pieces + 1) & 1] = 0;
            }
            tc_fence_before();
            ok = meet();                                   // (the others have read this thread's outputs, masks and sums)
            tiles += w.c;
            loads += 2 * w.c;
            pieces += w.c > 0;
            if (!w.next(a)) break;
        }
    } else if (warp >= 18) {
        // ---- loads: one warp the keys, one the queries and the values (a load costs a warp 900 cycles, mostly waits for its own
        // results; where one warp had both, it was what bound the kernel)
        const bool keys = warp == 18;
        constexpr int CH = D / 8, RPI = 32 / CH;            // 16-byte chunks of a row, rows of a warp's instruction
        const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.k_cache), *vc = static_cast<const __nv_bfloat16 *>(p.v_cache);
        uint32_t loads = 0, pieces = 0, tiles = 0;
        // Loads by cp.async that have not been reported yet (barriers, eight bits each, the oldest lowest): they are once
        // they have landed, before this warp waits for anything, and when there are four of them.
        uint32_t queue = 0;
        int queued = 0;
        auto report = [&] {
            switch (queued) {
                case 1: cp_wait<0>(); break;
                case 2: cp_wait<1>(); break;
                case 3: cp_wait<2>(); break;
                default: cp_wait<3>(); break;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(queue & 255));
            queue >>= 8;
            --queued;
        };
        auto sent = [&](int b) {
            cp_commit();
            queue |= (uint32_t)b << (8 * queued);
            if (++queued == 4) report();
        };
        auto reach = [&](int b, uint32_t phase) {           // waits for a barrier
            if (!all(test(bar(b), phase))) {
                while (queued > 0) report();
                ok = all(wait(b, phase));
            }
            return ok;
        };
        struct Place {
            int at[2];        // by boxes: the place of this lane's box, -1 for none; else of tokens `lane` and 32 + lane
            uint2 mask;       // places with a token
        };
        for (;; ) {
            if (w.c > 0) {
                const int32_t *table = p.table + (int64_t)w.n * p.max_pages;
                const int boxes = box ? kKt / box : 0;                      // of a tile, 8 at most
                const int shift = w.shift(box);
                auto by_box = [&](int i) { return box && (w.ta + i != w.row.ctx || shift >= 0); };
                // Pages are fetched well before they are needed: by boxes, those of four tiles by one load (eight lanes a tile), four
                // tiles ahead; else a tile's, a tile ahead.
                auto group_token = [&](int g) { return (w.ta + 4 * g + (lane >> 3)) * kKt + (lane & 7) * box; };
                auto group_page = [&](int g) {
                    const int t = group_token(g);
                    if ((lane & 7) >= boxes || 4 * g + (lane >> 3) >= w.c || t >= w.row.len) return -1;
                    return __ldg(table + a.by_page((uint32_t)t));           // (t is below the table's width)
                };
                auto tokens = [&](int i) {
                    const int t = w.ta + i;
                    const bool draft = t == w.row.ctx;
                    const int base = draft ? w.row.len : t * kKt, left = i < w.c ? (draft ? w.row.m : w.row.len - base) : 0;
                    return make_int2(lane < left ? tree_page(a, table, base + lane) : -1, lane + 32 < left ? tree_page(a, table, base + lane + 32) : -1);
                };
                int group = -1, page = box ? group_page(0) : -1;            // places of the current four tiles; pages of the next
                const bool has_draft = w.ta + w.c > w.row.ctx;
                int2 pre = make_int2(-1, -1);                               // pages that are asked for ahead
                if (!box) {
                    pre = tokens(0);
                } else if (has_draft && shift < 0) {
                    pre = tokens(w.c - 1);
                } else if (has_draft) {
                    const int t = w.row.len - shift + lane * box;           // the boxes of the drafted tokens
                    if (lane < boxes && t < w.row.len + w.row.m) pre.x = tree_page(a, table, t);
                }
                const int2 parents = keys && has_draft ? tree_parents(a, w.n, w.row.m) : make_int2(-1, -1);
                auto place = [&](int i) {                                   // asked for in order
                    Place x;
                    if (by_box(i)) {
                        const bool draft = w.ta + i == w.row.ctx;
                        if ((i & 3) == 0) {
                            const int t = group_token(i >> 2), pg = (int)a.by_page((uint32_t)t);
                            group = page >= 0 && page < p.pages ? page * p.page_size + (t - pg * p.page_size) : -1;
                            page = group_page((i >> 2) + 1);
                        }
                        const int at = __shfl_sync(0xffffffffu, group, (i & 3) * 8 + (lane & 7));
                        x.at[0] = lane >= boxes ? -1 : draft ? (int)tree_place(a, pre.x, w.row.len - shift + lane * box) : at;
                        x.at[1] = -1;
                        const uint32_t have = __ballot_sync(0xffffffffu, x.at[0] >= 0);
                        const int from = draft ? shift : 0, left = draft ? shift + w.row.m : w.row.len - (w.ta + i) * kKt;
                        x.mask = make_uint2(0xffffffffu, 0xffffffffu);
                        if (have != (1u << boxes) - 1 || left < kKt || draft) {
                            const int per = __ffs(box) - 1;                 // (a power of two)
                            x.mask.x = __ballot_sync(0xffffffffu, lane >= from && lane < left && ((have >> (lane >> per)) & 1u));
                            x.mask.y = __ballot_sync(0xffffffffu, lane + 32 >= from && lane + 32 < left && ((have >> ((lane + 32) >> per)) & 1u));
                        }
                        return x;
                    }
                    const int base = (w.ta + i == w.row.ctx ? w.row.len : (w.ta + i) * kKt) + lane;
                    x.at[0] = (int)tree_place(a, pre.x, base), x.at[1] = (int)tree_place(a, pre.y, base + 32);
                    x.mask = make_uint2(__ballot_sync(0xffffffffu, x.at[0] >= 0), __ballot_sync(0xffffffffu, x.at[1] >= 0));
                    if (!box) pre = tokens(i + 1);
                    return x;
                };
                const CUtensorMap *map = keys ? &tmk : &tmv;
                const __nv_bfloat16 *cache = keys ? kc : vc;
                auto tile = [&](const Place &x, int i) {
                    const uint32_t load = loads + (keys ? w.k_load(i) : w.v_load(i)), s = load % S;
                    const int full = kFull + (int)s;
                    if (load >= S && !reach(kEmpty + s, load / S - 1)) return false;
                    const uint32_t to = sb + L::RING + s * L::TILE;
                    if (by_box(i)) {
                        // (of the places without a token, scores are masked and values made zero behind the load)
                        const uint32_t have = __ballot_sync(0xffffffffu, x.at[0] >= 0);
                        if (lane == 0) mbar_arrive_expect_tx(bar(full), __popc(have) * box * D * 2);
                        __syncwarp();
                        if (x.at[0] >= 0)
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) tma_load_3d(to + h * HALF + lane * box * 128, map, bar(full), 64 * h, w.hk, x.at[0]);
                    } else {
                        const int c = lane % CH;
                        for (int y = 0; y < kKt / RPI; ++y) {
                            const int r = y * RPI + lane / CH;
                            const int a0 = __shfl_sync(0xffffffffu, x.at[0], r & 31), a1 = __shfl_sync(0xffffffffu, x.at[1], r & 31), at = r < 32 ? a0 : a1;
                            cp16(to + (c >> 3) * HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4), cache + ((int64_t)(at < 0 ? 0 : at) * p.kv_heads + w.hk) * D + 8 * c,
                                 at < 0 ? 0u : 16u);
                        }
                        sent(full);
                    }
                    return true;
                };
                if (pieces > 0 && !reach(kQEmpty, pieces - 1)) break;   // (the queries, and the paths before the last, are read)
                if (keys) {
                } else if (qbox) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(kQFull), (w.two ? 2 : 1) * L::QTILE);
                        const int at = w.n * a.t.tokens + (int)a.by_rep((uint32_t)w.r0);
                        for (int e = 0; e < (w.two ? 2 : 1); ++e)
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) tma_load_3d(sb + L::Q + e * L::QTILE + h * QHALF, &tmq, bar(kQFull), 64 * h, w.hk * a.rep, at + e * qbox);
                    }
                    __syncwarp();
                } else {
                    for (int y = 0; y < (w.two ? 256 : 128) / RPI; ++y) {
                        const int r = y * RPI + lane / CH, c = lane % CH, i = (int)a.by_rep((uint32_t)(w.r0 + r));
                        const bool in = r < w.rows;
                        const int64_t at = in ? ((int64_t)w.n * a.t.tokens + i) * p.heads + w.hk * a.rep + (w.r0 + r - i * a.rep) : 0;
                        cp16(sb + L::Q + (r >> 7) * L::QTILE + (c >> 3) * QHALF + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
                             static_cast<const __nv_bfloat16 *>(p.q) + at * D + 8 * c, in ? 16u : 0u);
                    }
                    sent(kQFull);
                }
                bool fine = true;
                for (int i = 0; i < w.c && fine; ++i) {
                    const Place x = place(i);
                    if (keys) {
                        if (w.ta + i == w.row.ctx)   // the drafted tokens' paths
                            tree_masks(parents, w.row.m, reinterpret_cast<uint64_t *>(sm + L::ANC) + 64 * (pieces & 1), reinterpret_cast<int *>(sm + L::UP));
                        if (lane == 0) *reinterpret_cast<uint2 *>(sm + L::MASK + 8 * ((tiles + i) & 31)) = x.mask;
                        __syncwarp();
                    }
                    fine = tile(x, i);
                }
                if (!fine) break;
                loads += 2 * w.c;
                tiles += w.c;
                ++pieces;
            }
            if (!w.next(a)) break;
        }
        while (queued > 0) report();
    } else {
        // ---- products, a warp for each chain.  Both go through all loads in order: one that is the other chain's alone is
        // awaited and released as well, so that no stage is ever two loads ahead of what a warp waits for.
        // The whole warp runs the loop and an elected lane issues, so that the operand descriptors can stay in
        // uniform registers.
        const int k = warp - 16;
        const uint32_t one = elect_one();
        uint32_t loads = 0, qs = 0, made = 0, used = 0;   // loads, pieces, scores and weights so far
        const uint32_t qd = ((sb + L::Q) >> 4) | (1u << 16), kd = ((sb + L::RING) >> 4) | (1u << 16), vd = ((sb + L::RING) >> 4) | ((HALF >> 4) << 16);
        for (;; ) {
            if (w.c > 0) {
                const int ahead = w.ahead();
                const uint32_t q0 = qd + (w.two ? k * (L::QTILE >> 4) : 0u);
                auto mine = [&](int i) { return w.two || (i & 1) == k; };
                auto pass = [&](uint32_t ld) {   // the other chain's
                    const uint32_t s = ld % S;
                    ok = all(wait(kFull + s, ld / S));
                    if (ok && lane == 0) mbar_arrive(bar(kEmpty + s));
                    return ok;
                };
                // scores of tile i
                auto qk = [&](int i) {
                    const uint32_t ld = loads + w.k_load(i), s = ld % S, b = 2 * k + (made & 1);
                    if (!mine(i)) return pass(ld);
                    ok = all(wait(kFull + s, ld / S));
                    if (!ok) return false;
                    tc_fence_after();
                    const uint32_t to = tmem + TM_S + 64 * b, k0 = kd + s * (L::TILE >> 4);
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(to, q0 + (((kk >> 2) * QHALF + (kk & 3) * 32) >> 4), k0 + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), IDESC_QK, kk > 0);
                        mma_commit(bar(kS + b));
                        mbar_arrive(bar(kS + b));
                        mma_commit(bar(kEmpty + s));
                    }
                    __syncwarp();
                    ++made;
                    return true;
                };
                // outputs of tile i
                auto pv = [&](int i) {
                    const uint32_t ld = loads + w.v_load(i), s = ld % S, b = 2 * k + (used & 1);
                    if (!mine(i)) return pass(ld);
                    ok = all(wait(kFull + s, ld / S) && wait(kP + b, used >> 1));
                    if (!ok) return false;
                    tc_fence_after();
                    const uint32_t to = tmem + TM_O + 128 * k, from = tmem + TM_S + 64 * b, v0 = vd + s * (L::TILE >> 4);
                    const uint32_t more = w.two ? i > 0 : i > 1;   // not the chain's first tile
                    if (one) {
#pragma unroll
                        for (int e = 1; e >= 0; --e)   // the rests first
#pragma unroll
                            for (int kk = 0; kk < kKt / 16; ++kk)
                                mma_ts(to, from + 32 * (kk >> 1) + 8 * (kk & 1) + 16 * e, v0 + ((2048 * kk) >> 4), IDESC_PV, e == 0 || kk > 0 ? 1u : more);
                        mma_commit(bar(kEmpty + s));
                        mma_commit(bar(kV + b));
                    }
                    __syncwarp();
                    ++used;
                    return true;
                };
                ok = all(wait(kQFull, qs++));
                if (!ok) break;
                bool fine = true;
                auto queries = [&](int made_all) {                // the piece's queries are read
                    if (fine && made_all && one) mma_commit(bar(kQEmpty));
                    __syncwarp();
                };
                for (int i = 0; i < ahead && i < w.c && fine; ++i) {
                    fine = qk(i);
                    queries(i + 1 == w.c);
                }
                for (int i = 0; i < w.c && fine; ++i) {
                    fine = pv(i);
                    if (fine && i + ahead < w.c) {
                        fine = qk(i + ahead);
                        queries(i + ahead + 1 == w.c);
                    }
                }
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
    if (!ok) s_fail = 1;   // (where a chain has left together, one of its warps has given up)
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
        w.x = tree_cut(blockIdx.x, W, G);                  // from the start of the share
        tree_find<kThreads>(a, w.x, sm_sum, w.n, w.us);
        w.row = tree_row(a, w.n);
        w.unit = (int)((w.x - w.us) / w.row.items);
        w.us += w.unit * w.row.items;
        w.piece(a);
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
    if (warp == 16) {
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

// [tokens][heads][d] bf16 as (d, heads, tokens): boxes of 64 channels of `of` heads and `box` tokens, 128-byte swizzle; what lies
// past the tensor is zeros.
bool make_map(CUtensorMap *m, const void *ptr, int64_t tokens, int heads, int d, int of, int box) {
    auto enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t boxes[3] = {64, (cuuint32_t)of, (cuuint32_t)box};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs: one per SM, never more than there can be items (seven at least: a start, a tile of cached tokens and one of drafted ones).
int tc_ctas(const PagedTreeArgs &t) {
    const int rep = t.p.heads / t.p.kv_heads;
    const int64_t units = (int64_t)t.p.rows * t.p.kv_heads * (((int64_t)t.tokens * rep + kRb - 1) / kRb);
    const int64_t items = ((int64_t)t.p.max_pages * t.p.page_size + kKt - 1) / kKt + 1 + kStart;
    return units >= kSms || units * items >= kSms ? kSms : (int)(units * items);
}

template <int D> cudaError_t launch_tc(const TreeAtt &a, int ctas, uint32_t polls, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    const PagedArgs &p = a.t.p;
    // tokens of a box: the largest power of two that divides the pages, of eight rows (a swizzle's period) at least
    int box = kKt;
    while (p.page_size % box) box /= 2;
    if (box < 8) box = 0;
    // the queries of 128 rows are a box where whole tokens make up 128 rows (those of the next row's tokens are not written)
    const int qbox = 128 % a.rep == 0 ? 128 / a.rep : 0;
    const int64_t cached = (int64_t)p.pages * p.page_size;
    if (!make_map(&mq, p.q, (int64_t)p.rows * a.t.tokens, p.heads, D, qbox ? a.rep : 1, qbox ? qbox : 8) ||
        !make_map(&mk, p.k_cache, cached, p.kv_heads, D, 1, box ? box : 8) || !make_map(&mv, p.v_cache, cached, p.kv_heads, D, 1, box ? box : 8))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kda_paged_tree_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tc<D>::BYTES);
    if (e != cudaSuccess) return e;
    kda_paged_tree_tc_kernel<D><<<ctas, kThreads, Tc<D>::BYTES, st>>>(mq, mk, mv, a, qbox, box, polls);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_tree_join(a, D, KDA_BF16, ctas, st);
}

}  // namespace

size_t tree_tc_workspace_bytes(const PagedTreeArgs &t, int d) { return tree_short_cluster(t, d) ? 0 : (size_t)tc_ctas(t) * 2 * kRb * (d + 2) * 4; }

cudaError_t launch_tree_tc(const PagedTreeArgs &t, int d, void *workspace, uint32_t polls, cudaStream_t st) {
    const int rep = t.p.heads / t.p.kv_heads, ctas = tc_ctas(t);
    float *ws = static_cast<float *>(workspace);
    const TreeAtt a{t, FastDiv((uint32_t)t.p.page_size), FastDiv((uint32_t)rep), rep, kRb, kKt, 8, 6, kStart, ws, ws + (size_t)ctas * 2 * kRb * d};
    if (const int c = tree_short_cluster(t, d)) return launch_tree_short(a, d, c, st);
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
