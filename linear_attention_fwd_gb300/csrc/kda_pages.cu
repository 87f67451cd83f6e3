// Pages of a paged cache: the accepted path of a draft moved together, rows forked, ended and extended, the
// pool closed up, pages copied.
#include <cooperative_groups.h>

#include "kda_paged.cuh"
#include "kda_tree.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

// ------------------------------------------------------------------ the accepted path
// One CTA per row.  A path's tokens ascend (a token continues an earlier one), so its r-th token a_r >= r goes to
// place r, which is no later token's old place: a thread that moves its 16 bytes of all tokens in order, some at a
// time, reads each before it is written.  Bound by the chain of reads ahead of the data (path, pages): 3.5 us for 256 rows of up
// to 32 drafted tokens, 8 heads of 128, bf16; 2.9 for one row.
constexpr int kCommitThreads = 256, kCommitAhead = 4;

__global__ void __launch_bounds__(kCommitThreads) kda_paged_tree_commit_kernel(const TreeCommitArgs a, const FastDiv by_page) {
    __shared__ int up[kTreeMax], path[kTreeMax], s_len;
    __shared__ int64_t from[kTreeMax], to[kTreeMax];
    const int n = blockIdx.x, tid = threadIdx.x, most = a.max_pages * a.page_size;
    int old = *static_cast<const volatile int32_t *>(a.lens + n);   // (new_lens may be the same array: read before it is written)
    old = old < 0 ? 0 : (old > most ? most : old);
    int last = __ldg(a.accepted + n);
    if (last >= tree_count(a.num, a.tokens, n)) last = -1;
    if (tid <= last) up[tid] = tree_parent(a.parents, a.tokens, n, tid);
    __syncthreads();
    if (tid == 0) {
        int len = 0;
        for (int i = last; i >= 0; i = up[i]) ++len;
        s_len = len;
        if (a.new_lens) a.new_lens[n] = old + len < most ? old + len : most;
        for (int i = last; i >= 0; i = up[i]) path[--len] = i;
    }
    __syncthreads();
    const int len = s_len;
    if (len == 0) return;
    auto place = [&](int pos) -> int64_t {
        const uint32_t pg = by_page((uint32_t)pos);
        if (pg >= (uint32_t)a.max_pages) return -1;
        const int page = __ldg(a.table + (int64_t)n * a.max_pages + pg);
        return page < 0 || page >= a.pages ? -1 : (int64_t)page * a.page_size + (pos - (int)pg * a.page_size);
    };
    if (tid < 2 * kTreeMax) {
        const int r = tid % kTreeMax;
        if (r < len) (tid < kTreeMax ? from : to)[r] = place(old + (tid < kTreeMax ? path[r] : r));
    }
    __syncthreads();
    for (int x = tid; x < 2 * a.row_vecs; x += kCommitThreads) {
        uint4 *c = static_cast<uint4 *>(x < a.row_vecs ? a.k_cache : a.v_cache) + (x < a.row_vecs ? x : x - a.row_vecs);
        for (int r0 = 0; r0 < len; r0 += kCommitAhead) {
            uint4 v[kCommitAhead];
            bool go[kCommitAhead];
#pragma unroll
            for (int e = 0; e < kCommitAhead; ++e) {
                const int r = r0 + e;
                go[e] = r < len && from[r] >= 0 && to[r] >= 0 && from[r] != to[r];
                if (go[e]) v[e] = c[from[r] * a.row_vecs];
            }
#pragma unroll
            for (int e = 0; e < kCommitAhead; ++e)
                if (go[e]) c[to[r0 + e] * a.row_vecs] = v[e];
        }
    }
}

// ------------------------------------------------------------------ tables and counts
// One cluster of CTAs does a call: its CTAs split the pages and the rows between them, meet at cluster barriers, and exchange
// their bitmaps of free pages with prefix sums over blocks and words through distributed shared memory, so that a
// call is one launch without a workspace.  Bound by its chains of dependent reads (row, length, page, count) and by the
// barriers: what a row needs is gathered by a thread each before warps go over its entries.  Fork of 8 rows of 44 pages and
// the copies of their last pages: 9.2 us; of 256 rows of 100 to 8000 tokens on pages of 16: 21.0 us (16 and 45 where each warp
// fetched what its rows need by itself).
constexpr int kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32, kBlock = 1024;   // pages of a block: 32 words of the bitmap
constexpr int kMaxCtas = 16, kLocalPages = 1 << 18, kLocalRows = 8192, kBatch = 1024;

struct PoolPlan {
    int ctas, blocks, all;     // CTAs; blocks of pages per CTA; all blocks where every CTA keeps the whole bitmap, else 0
    int rows;                  // rows per CTA
    int chunk, per_row;        // entries of a segment of a row; segments of a row
    int lanes;                 // of a warp for a segment: fewer than 32 where a row has no more than four entries for each
    int first;                 // rows where their first continuing row is found in shared memory, else 0
    int vec;                   // four entries of a table lie on 16 bytes
    int smem;
};

// A bitmap of free pages: words, free pages before each word within its block, and before each block.
struct Bitmap {
    uint32_t *words;
    uint16_t *in_block;
    int *blk;
    __device__ __forceinline__ Bitmap(uint8_t *at, int blocks)
        : words(reinterpret_cast<uint32_t *>(at)), in_block(reinterpret_cast<uint16_t *>(at + 128 * blocks)), blk(reinterpret_cast<int *>(at + 192 * blocks)) {}
};
__host__ __device__ constexpr int bitmap_bytes(int blocks) { return 192 * blocks + 4 * (blocks + 1); }

struct Pool {
    cg::cluster_group cluster;
    Bitmap mine, whole;        // of this CTA's blocks; of all
    const int *before;         // (shared) free pages before each CTA's blocks, [kMaxCtas]: all
    int blocks, all;

    __device__ __forceinline__ int free_pages() const { return before[kMaxCtas]; }
    // The number of free pages before page p.
    __device__ int free_before(int p) const {
        const int b = p / kBlock, word = (p % kBlock) / 32;
        const uint32_t below = (1u << (p % 32)) - 1;
        if (all) return whole.blk[b] + whole.in_block[32 * b + word] + __popc(whole.words[32 * b + word] & below);
        const int c = b / blocks, at = 32 * (b - c * blocks) + word;
        return before[c] + cluster.map_shared_rank(mine.blk, c)[b - c * blocks] + cluster.map_shared_rank(mine.in_block, c)[at] +
               __popc(cluster.map_shared_rank(mine.words, c)[at] & below);
    }
    // The k-th free page (k < their number).  (Not inlined: a short kernel's time is largely that of fetching its code.)
    __device__ __noinline__ int nth_free(int k) const {
        int c = 0, n = all;
        const int *pre = whole.blk;
        const uint16_t *in_block = whole.in_block;
        const uint32_t *words = whole.words;
        if (!all) {
            while (k >= before[c + 1]) ++c;
            k -= before[c];
            n = blocks;
            pre = cluster.map_shared_rank(mine.blk, c);
            in_block = cluster.map_shared_rank(mine.in_block, c);
            words = cluster.map_shared_rank(mine.words, c);
        }
        int lo = 0;   // pre[lo] <= k < pre[hi]
        for (int hi = n; hi - lo > 1;) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= k) lo = mid;
            else hi = mid;
        }
        k -= pre[lo];
        int w = 0;
#pragma unroll
        for (int step = 16; step > 0; step /= 2)
            if (in_block[32 * lo + w + step] <= k) w += step;
        k -= in_block[32 * lo + w];
        uint32_t x = words[32 * lo + w];
        int at = 0;
#pragma unroll
        for (int step = 16; step > 0; step /= 2) {   // the k-th bit set
            const int n_low = __popc(x & ((1u << step) - 1));
            if (k >= n_low) {
                k -= n_low;
                x >>= step;
                at += step;
            }
        }
        return (c * blocks + lo) * kBlock + 32 * w + at;
    }
};

// The bitmap of this CTA's pages, eight words a warp; `each` sees every page's count.  Block-wide.
template <typename F> __device__ __forceinline__ void scan_pages(const ForkArgs &a, Pool &P, F each) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int u = warp; u < 4 * P.blocks; u += kPoolWarps) {
        const int64_t p0 = (int64_t)P.cluster.block_rank() * P.blocks * kBlock + 256 * (int64_t)u + lane;
        int r[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) r[w] = p0 + 32 * w < a.pages ? __ldg(a.refs + p0 + 32 * w) : 1;
        uint32_t own = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint32_t bits = __ballot_sync(0xffffffffu, r[w] == 0);
            if (lane == w) own = bits;
            if (p0 + 32 * w < a.pages) each((int)(p0 + 32 * w), r[w]);
        }
        if (lane < 8) P.mine.words[8 * u + lane] = own;
    }
    __syncthreads();
    for (int b = warp; b < P.blocks; b += kPoolWarps) {
        const int n = __popc(P.mine.words[32 * b + lane]);
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        P.mine.in_block[32 * b + lane] = (uint16_t)(sum - n);
        if (lane == 31) P.mine.blk[b] = sum;
    }
}

// One warp: exclusive prefix sums of x[0 .. n), in place; returns the sum.
__device__ __forceinline__ int scan_warp(int *x, int n) {
    const int lane = threadIdx.x & 31;
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int v = i0 + lane < n ? x[i0 + lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (i0 + lane < n) x[i0 + lane] = run + s - v;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    return run;
}

// A barrier of all CTAs.
__device__ __forceinline__ void pool_sync(Pool &P, const PoolPlan &plan) {
    if (plan.ctas > 1) P.cluster.sync();
    else __syncthreads();
}

__device__ __forceinline__ Pool make_pool(const PoolPlan &plan, uint8_t *&sm) {
    Bitmap mine(sm, plan.blocks);
    sm += bitmap_bytes(plan.blocks);
    Bitmap whole(sm, plan.all);
    if (plan.all) sm += bitmap_bytes(plan.all);
    Pool P{cg::this_cluster(), mine, plan.ctas == 1 ? mine : whole};
    P.blocks = plan.blocks;
    P.all = plan.all;
    return P;
}
// The CTAs' totals (free pages; pages asked for), and theirs before each CTA.
struct Totals {
    int mine[2], free_before[kMaxCtas + 1];
    long long asked, ahead;   // by all CTAs, by those before this one
};
// Behind the CTAs' own bitmaps and totals: takes over what the others have.  Block-wide, with a barrier of all CTAs.
__device__ __forceinline__ void meet(Pool &P, const PoolPlan &plan, Totals &t) {
    pool_sync(P, plan);
    const int lane = threadIdx.x & 31, rank = (int)P.cluster.block_rank();
    if (threadIdx.x < 32) {
        const int *other = lane < plan.ctas ? P.cluster.map_shared_rank(t.mine, lane) : nullptr;
        const int free = other ? other[0] : 0, asked = other ? other[1] : 0;
        int f = free;
        long long s = asked;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, f, o);
            const long long z = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) f += y, s += z;
        }
        if (lane < kMaxCtas) t.free_before[lane] = f - free;
        if (lane == 31) t.free_before[kMaxCtas] = f, t.asked = s;
        if (lane == rank) t.ahead = s - asked;
    }
    P.before = t.free_before;
    __syncthreads();
    if (!plan.all || plan.ctas == 1) return;
#pragma unroll 1
    for (int i = threadIdx.x; i < plan.all * 32; i += kPoolThreads) {
        const int c = i / (32 * plan.blocks), at = i - c * 32 * plan.blocks;
        P.whole.words[i] = P.cluster.map_shared_rank(P.mine.words, c)[at];
        P.whole.in_block[i] = P.cluster.map_shared_rank(P.mine.in_block, c)[at];
        if (at % 32 == 0) P.whole.blk[i / 32] = P.before[c] + P.cluster.map_shared_rank(P.mine.blk, c)[at / 32];
    }
    if (threadIdx.x == 0) P.whole.blk[plan.all] = P.free_pages();
    __syncthreads();
}

// A row of the new table.
struct NewRow {
    int src, len, full, need;   // the old row (-1: none), its length, pages that it fills, entries that have to name a page
};
constexpr int kHeir = 1, kContinued = 2, kCopy = 4;   // the first row that continues src; the old row of this number goes on; its last page is copied
__device__ __forceinline__ bool row_part(const ForkArgs &a, const NewRow &r) { return r.len > r.full * a.page_size; }
__device__ __forceinline__ NewRow new_row(const ForkArgs &a, const FastDiv &by_page, int n) {
    NewRow r;
    r.src = __ldg(a.sources + n);
    r.len = r.full = r.need = 0;
    if (r.src < 0 || r.src >= a.rows) {
        r.src = -1;
        return r;
    }
    const int most = a.max_pages * a.page_size;
    r.len = __ldg(a.lens + r.src);
    r.len = r.len < 0 ? 0 : (r.len > most ? most : r.len);
    r.full = (int)by_page((uint32_t)r.len);
    const int more = a.new_tokens ? __ldg(a.new_tokens + n) : 0;
    const int64_t end = (int64_t)r.len + (more > 0 ? more : 0);
    r.need = a.max_pages;
    if (end < most) {
        r.need = (int)by_page((uint32_t)end);
        r.need += end > (int64_t)r.need * a.page_size;
    }
    return r;
}
__device__ __forceinline__ int valid(const ForkArgs &a, int p) { return p < 0 || p >= a.pages ? -1 : p; }
// The page that entry e keeps of the old row's, p (-1 for none).  Entries past the length are room to write to: the
// first row that continues the old one keeps those pages that no other entry names.
__device__ __forceinline__ int kept(const ForkArgs &a, const NewRow &r, int flags, int e, int p) {
    p = valid(a, p);
    if (r.src < 0 || p < 0 || e < r.full + (row_part(a, r) ? 1 : 0)) return r.src < 0 ? -1 : p;
    return (flags & kHeir) && __ldg(a.refs + p) == 1 ? p : -1;
}
// Entries e .. e + 3 of a row of a table, -1 past its end.
__device__ __forceinline__ int4 load4(const int32_t *row, int e, int end, bool vec) {
    if (vec && e + 4 <= end) return __ldg(reinterpret_cast<const int4 *>(row + e));
    int4 x;
    x.x = e < end ? __ldg(row + e) : -1;
    x.y = e + 1 < end ? __ldg(row + e + 1) : -1;
    x.z = e + 2 < end ? __ldg(row + e + 2) : -1;
    x.w = e + 3 < end ? __ldg(row + e + 3) : -1;
    return x;
}
__device__ __forceinline__ void store4(int32_t *row, int e, int end, bool vec, int4 x) {
    if (vec && e + 4 <= end) {
        *reinterpret_cast<int4 *>(row + e) = x;
        return;
    }
    if (e < end) row[e] = x.x;
    if (e + 1 < end) row[e + 1] = x.y;
    if (e + 2 < end) row[e + 2] = x.z;
    if (e + 3 < end) row[e + 3] = x.w;
}
__device__ __forceinline__ bool wants(const NewRow &r, int flags, int e, int p) { return (e < r.need && p < 0) || ((flags & kCopy) && e == r.full); }

// kNarrow: more rows than warps, of up to 64 entries, several to a warp (141 rows of one page: 10 us, 20 with a row a warp; 256
// wide rows by the same code: 21.6 us, 20.5 by their own).
template <bool kNarrow>
__global__ void __launch_bounds__(kPoolThreads) kda_paged_fork_kernel(const ForkArgs a, const PoolPlan plan, const FastDiv by_page) {
    extern __shared__ __align__(16) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ Totals totals;
    uint8_t *at = sm;
    NewRow *info = reinterpret_cast<NewRow *>(at);                            // of a batch of rows
    at += kBatch * sizeof(NewRow);
    Pool P = make_pool(plan, at);
    int *count = reinterpret_cast<int *>(at);                                 // pages that each segment asks for, then before it
    int *first = count + plan.rows * plan.per_row;                            // the first row that continues each old one
    uint8_t *flags = reinterpret_cast<uint8_t *>(first + plan.first);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)P.cluster.block_rank();
    const int lo = rank * plan.rows, rows = a.rows - lo < plan.rows ? (a.rows - lo > 0 ? a.rows - lo : 0) : plan.rows;   // this CTA's rows
    constexpr int kNone = 0x7fffffff;

    // (more rows than fit are kept in `copies` until those are written)
    if (plan.first) {
        for (int n = tid; n < a.rows; n += kPoolThreads) first[n] = kNone;
        __syncthreads();
        for (int n = tid; n < a.rows; n += kPoolThreads) {
            const int s = __ldg(a.sources + n);
            if (s >= 0 && s < a.rows) atomicMin(first + s, n);
        }
        scan_pages(a, P, [&](int p, int r) { a.new_refs[p] = r; });
        __syncthreads();
    } else {
        for (int n = lo + tid; n < lo + rows; n += kPoolThreads) a.copies[2 * (int64_t)n] = kNone;
        P.cluster.sync();
        for (int n = lo + tid; n < lo + rows; n += kPoolThreads) {
            const int s = __ldg(a.sources + n);
            if (s >= 0 && s < a.rows) atomicMin(a.copies + 2 * (int64_t)s, n);
        }
        scan_pages(a, P, [&](int p, int r) { a.new_refs[p] = r; });
        P.cluster.sync();
    }
    const int lanes = kNarrow ? plan.lanes : 32, at_once = 32 / lanes, sub = lane % lanes, part = lane / lanes;   // a segment's lanes; segments of a warp
    auto first_of = [&](int s) { return plan.first ? first[s] : __ldcg(a.copies + 2 * (int64_t)s); };

    for (int r0 = 0; r0 < rows; r0 += kBatch) {
        const int nr = rows - r0 < kBatch ? rows - r0 : kBatch;
        if (tid < nr) {
            const int n = lo + r0 + tid;
            const NewRow r = new_row(a, by_page, n);
            int fl = (r.src >= 0 && first_of(r.src) == n ? kHeir : 0) | (first_of(n) != kNone ? kContinued : 0);
            if (r.src >= 0 && row_part(a, r)) {
                const int p = valid(a, __ldg(a.table + (int64_t)r.src * a.max_pages + r.full));
                if (p >= 0 && !((fl & kHeir) && __ldg(a.refs + p) == 1)) fl |= kCopy;
            }
            info[tid] = r;
            flags[r0 + tid] = (uint8_t)fl;
        }
        __syncthreads();
        for (int s0 = warp * at_once; s0 < nr * plan.per_row; s0 += kPoolWarps * at_once) {
            const bool here = !kNarrow || s0 + part < nr * plan.per_row;
            const int sg = here ? s0 + part : s0, i = sg / plan.per_row, e0 = (sg - i * plan.per_row) * plan.chunk;
            const NewRow r = info[i];
            const int fl = flags[r0 + i], e1 = e0 + plan.chunk < a.max_pages ? e0 + plan.chunk : a.max_pages;
            int sum = 0;
            if (here && r.src >= 0 && e0 < r.need)
                for (int e = e0 + 4 * sub; e < e1; e += 4 * lanes) {
                    const int4 x = load4(a.table + (int64_t)r.src * a.max_pages, e, e1, plan.vec);
                    const int p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) sum += e + y < e1 && wants(r, fl, e + y, kept(a, r, fl, e + y, p[y]));
                }
            if constexpr (kNarrow)
                for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            else sum = __reduce_add_sync(0xffffffffu, sum);
            if (here && sub == 0) count[r0 * plan.per_row + sg] = sum;
        }
        __syncthreads();
    }
    if (warp == 0) {
        const int x = scan_warp(P.mine.blk, plan.blocks);
        if (lane == 0) P.mine.blk[plan.blocks] = totals.mine[0] = x;
    } else if (warp == 1) {
        const int x = scan_warp(count, rows * plan.per_row);
        if (lane == 0) totals.mine[1] = x;
    }
    meet(P, plan, totals);
    const long long ahead = totals.ahead;
    const int missing = totals.asked > P.free_pages() ? (int)(totals.asked - P.free_pages()) : 0;
    if (rank == 0 && tid == 0) *a.short_of = missing;

    for (int r0 = 0; r0 < rows; r0 += kBatch) {
        const int nr = rows - r0 < kBatch ? rows - r0 : kBatch;
        if (r0 > 0) __syncthreads();
        if (tid < nr) {
            const int n = lo + r0 + tid;
            if (rows > kBatch) info[tid] = new_row(a, by_page, n);            // (else they are still there)
            a.new_lens[n] = missing > 0 ? __ldg(a.lens + n) : info[tid].len;
            if (missing > 0 || !(flags[r0 + tid] & kCopy)) a.copies[2 * (int64_t)n] = a.copies[2 * (int64_t)n + 1] = -1;
        }
        if (rows > kBatch) __syncthreads();
        for (int s0 = warp * at_once; s0 < nr * plan.per_row; s0 += kPoolWarps * at_once) {
            const bool here = !kNarrow || s0 + part < nr * plan.per_row;
            const int sg = here ? s0 + part : s0, i = sg / plan.per_row, e0 = (sg - i * plan.per_row) * plan.chunk, n = lo + r0 + i;
            const NewRow r = info[i];
            const int last = e0 + plan.chunk < a.max_pages ? e0 + plan.chunk : a.max_pages, e1 = here ? last : e0;   // (no entries: nothing)
            const int fl = flags[r0 + i];
            const int32_t *old = a.table + (int64_t)n * a.max_pages;
            int32_t *to = a.new_table + (int64_t)n * a.max_pages;
            int k = (int)ahead + count[r0 * plan.per_row + sg];
            for (int eb = e0; eb < last; eb += 4 * lanes) {   // (once where a warp has several segments)
                const int e = eb + 4 * sub;
                if (missing > 0) {
                    store4(to, e, e1, plan.vec, load4(old, e, e1, plan.vec));
                    continue;
                }
                int4 x = make_int4(-1, -1, -1, -1), y = x;
                if (r.src >= 0) x = load4(a.table + (int64_t)r.src * a.max_pages, e, e1, plan.vec);
                const bool ends = !(fl & kContinued);                             // the old row of this number
                if (ends) y = load4(old, e, e1, plan.vec);
                int p[4] = {x.x, x.y, x.z, x.w};
                const int q[4] = {y.x, y.y, y.z, y.w};
                int want = 0;                                                     // a bit for each entry
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) {
                    const int was = p[i2];
                    p[i2] = kept(a, r, fl, e + i2, was);
                    if ((fl & kHeir) && e + i2 < e1 && p[i2] < 0 && valid(a, was) >= 0) atomicSub(a.new_refs + was, 1);   // given up
                    if (e + i2 < e1 && wants(r, fl, e + i2, p[i2])) want |= 1 << i2;
                }
                const bool shared = !(fl & kHeir);
                if (shared || ends)
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) {
                        if (shared && e + i2 < e1 && p[i2] >= 0 && !((fl & kCopy) && e + i2 == r.full)) atomicAdd(a.new_refs + p[i2], 1);
                        if (ends && e + i2 < e1 && valid(a, q[i2]) >= 0) atomicSub(a.new_refs + q[i2], 1);
                    }
                if (__any_sync(0xffffffffu, want != 0)) {
                    int s = __popc(want);
                    const int mine = s;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int z = __shfl_up_sync(0xffffffffu, s, o);
                        if (sub >= o) s += z;
                    }
                    int at = k + s - mine;
                    k += __shfl_sync(0xffffffffu, s, lane | (lanes - 1));
#pragma unroll 1
                    for (; want; want &= want - 1) {
                        const int i2 = __ffs(want) - 1, was = i2 == 0 ? p[0] : i2 == 1 ? p[1] : i2 == 2 ? p[2] : p[3], now = P.nth_free(at++);
                        p[0] = i2 == 0 ? now : p[0], p[1] = i2 == 1 ? now : p[1], p[2] = i2 == 2 ? now : p[2], p[3] = i2 == 3 ? now : p[3];
                        a.new_refs[now] = 1;
                        if ((fl & kCopy) && e + i2 == r.full) {
                            a.copies[2 * (int64_t)n] = was;
                            a.copies[2 * (int64_t)n + 1] = now;
                            if (fl & kHeir) atomicSub(a.new_refs + was, 1);       // the old row's own reference
                        }
                    }
                }
                store4(to, e, e1, plan.vec, make_int4(p[0], p[1], p[2], p[3]));
            }
        }
    }
    if (plan.ctas > 1) P.cluster.sync();  // the others have read this CTA's bitmap and totals
}

__global__ void __launch_bounds__(kPoolThreads) kda_paged_compact_kernel(const ForkArgs a, const PoolPlan plan) {
    extern __shared__ __align__(16) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ Totals totals;
    uint8_t *at = sm;
    Pool P = make_pool(plan, at);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)P.cluster.block_rank();
    const int threads = plan.ctas * kPoolThreads, gt = rank * kPoolThreads + tid;
    scan_pages(a, P, [](int, int) {});
    __syncthreads();
    if (warp == 0) {
        const int x = scan_warp(P.mine.blk, plan.blocks);
        if (lane == 0) P.mine.blk[plan.blocks] = totals.mine[0] = x;
    }
    meet(P, plan, totals);
    const int used = a.pages - P.free_pages();
    const int moves = used < a.pages ? P.free_before(used) : 0;   // free pages below `used`, and used ones past it
    // pages, a word a warp: those that move leave their new place in new_refs until the table is rewritten
    for (int w = warp; w < 32 * plan.blocks; w += kPoolWarps) {
        const int64_t p64 = (int64_t)rank * plan.blocks * kBlock + 32 * w + lane;
        if (p64 >= a.pages) continue;
        const int p = (int)p64;
        const uint32_t bits = P.mine.words[w];
        const bool in_use = !((bits >> lane) & 1u);
        if (in_use && p < used) {
            a.new_refs[p] = __ldg(a.refs + p);
        } else if (in_use) {
            const int ahead = P.before[rank] + P.mine.blk[w / 32] + P.mine.in_block[w] + __popc(bits & ((1u << lane) - 1));   // free pages before it
            const int r = p - ahead - (used - moves), to = P.nth_free(r);
            a.new_refs[to] = __ldg(a.refs + p);
            a.new_refs[p] = to;
            a.copies[2 * r] = p;
            a.copies[2 * r + 1] = to;
        } else if (p >= used) {
            a.new_refs[p] = 0;
        }
    }
    for (int r = moves + gt; r < a.pages / 2; r += threads) a.copies[2 * r] = a.copies[2 * r + 1] = -1;
    P.cluster.sync();
    const int64_t entries = (int64_t)a.rows * a.max_pages;
    for (int64_t i0 = gt; i0 < entries; i0 += 8 * (int64_t)threads) {
        int p[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) p[x] = i0 + x * (int64_t)threads < entries ? __ldg(a.table + i0 + x * (int64_t)threads) : -1;
#pragma unroll
        for (int x = 0; x < 8; ++x) p[x] = p[x] >= used && p[x] < a.pages ? __ldcg(a.new_refs + p[x]) : (p[x] >= 0 && p[x] < a.pages ? p[x] : -1);
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x * (int64_t)threads < entries) a.new_table[i0 + x * (int64_t)threads] = p[x];
    }
    P.cluster.sync();
    for (int p = used + gt; p < a.pages; p += threads) a.new_refs[p] = 0;
}

// ------------------------------------------------------------------ copies
// Works of 16 KB of a page, a page's keys and then its values, over CTAs that stay: each thread moves four 16-byte
// vectors at a time.  Bound by DRAM: 6,570 pages of 32 KB of keys and as much of values: 140 us, 6.1 TB/s of reads and writes.
constexpr int kCopyThreads = 256, kCopyAhead = 4, kCopyVecs = kCopyThreads * kCopyAhead;

// (not by the read-only path: the kernel ahead may write the list while this one is there already.  From the L2 cache alone, 6,570
// pages take 2 us more: a page's works read the same pair)
__device__ __forceinline__ int load_fresh(const int32_t *p) {
    int x;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

__global__ void __launch_bounds__(kCopyThreads) kda_paged_copy_kernel(uint4 *kc, uint4 *vc, const int32_t *copies, const int64_t works,
                                                                      const int per_page, const int64_t page_vecs, const int pages) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (launched before the kernel ahead of it has ended)
    for (int64_t w = blockIdx.x; w < works; w += gridDim.x) {
        const int64_t i = w / per_page;
        const int from = load_fresh(copies + 2 * i), to = load_fresh(copies + 2 * i + 1);
        if (from < 0 || from >= pages || to < 0 || to >= pages) continue;
        const int64_t v0 = (w - i * per_page) * kCopyVecs + threadIdx.x;
        uint4 v[kCopyAhead];
        auto at = [&](int page, int64_t x) { return x < page_vecs ? kc + page * page_vecs + x : vc + page * page_vecs + (x - page_vecs); };
#pragma unroll
        for (int e = 0; e < kCopyAhead; ++e)
            if (v0 + e * kCopyThreads < 2 * page_vecs) v[e] = __ldcs(at(from, v0 + e * kCopyThreads));
#pragma unroll
        for (int e = 0; e < kCopyAhead; ++e)
            if (v0 + e * kCopyThreads < 2 * page_vecs) *at(to, v0 + e * kCopyThreads) = v[e];
    }
}

PoolPlan pool_plan(const ForkArgs &a, bool fork) {
    PoolPlan p{};
    const int64_t blocks = (a.pages + kBlock - 1) / kBlock, entries = (int64_t)a.rows * a.max_pages;
    p.ctas = 1;
    while (p.ctas < kMaxCtas && (blocks * kBlock + entries) > (int64_t)p.ctas * 4 * kPoolThreads) p.ctas *= 2;
    p.blocks = (int)((blocks + p.ctas - 1) / p.ctas);
    p.all = p.ctas == 1 ? p.blocks : a.pages <= kLocalPages ? p.blocks * p.ctas : 0;
    p.smem = bitmap_bytes(p.blocks) + (p.all ? bitmap_bytes(p.all) : 0);
    if (fork) {
        p.chunk = 128;
        p.rows = (a.rows + p.ctas - 1) / p.ctas;
        while (p.chunk < a.max_pages && (int64_t)p.rows * ((a.max_pages + p.chunk - 1) / p.chunk) > 16384) p.chunk *= 2;
        p.per_row = (a.max_pages + p.chunk - 1) / p.chunk;
        p.lanes = p.rows > kPoolWarps ? 1 : 32;   // (a warp has one row anyway)
        while (p.lanes < 32 && 4 * p.lanes < a.max_pages) p.lanes *= 2;
        p.first = a.rows <= kLocalRows ? a.rows : 0;
        p.smem += kBatch * (int)sizeof(NewRow) + 4 * p.rows * p.per_row + 4 * p.first + p.rows;
        p.vec = a.max_pages % 4 == 0 && (reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.new_table)) % 16 == 0;
    }
    return p;
}

template <typename... A> cudaError_t launch_pool(void (*kernel)(A...), const PoolPlan &plan, cudaStream_t st, std::common_type_t<A>... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)plan.ctas);
    cfg.blockDim = dim3(kPoolThreads);
    cfg.dynamicSmemBytes = (size_t)plan.smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)plan.ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitArgs &a, cudaStream_t st) {
    kda_paged_tree_commit_kernel<<<(unsigned)a.rows, kCommitThreads, 0, st>>>(a, FastDiv((uint32_t)a.page_size));
    return cudaGetLastError();
}

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t st) {
    const PoolPlan plan = pool_plan(a, true);
    return launch_pool(plan.lanes < 32 ? kda_paged_fork_kernel<true> : kda_paged_fork_kernel<false>, plan, st, a, plan, FastDiv((uint32_t)a.page_size));
}

cudaError_t launch_compact(const ForkArgs &a, cudaStream_t st) {
    return launch_pool(kda_paged_compact_kernel, pool_plan(a, false), st, a, pool_plan(a, false));
}

cudaError_t launch_page_copy(void *kc, void *vc, const int32_t *copies, int64_t count, int64_t page_vecs, int pages, cudaStream_t st) {
    const int64_t per_page = (2 * page_vecs + kCopyVecs - 1) / kCopyVecs, works = count * per_page;
    if (per_page > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int64_t most = 8 * kSms;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)(works < most ? works : most));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, kda_paged_copy_kernel, static_cast<uint4 *>(kc), static_cast<uint4 *>(vc), copies, works, (int)per_page, page_vecs, pages);
}

}  // namespace kda
