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
// time, reads each before it is written.  Bound by the chain of reads ahead of the data (path, pages).
constexpr int kCommitThreads = 256, kCommitAhead = 4;

__global__ void __launch_bounds__(kCommitThreads) kda_paged_tree_commit_kernel(const TreeCommitArgs a, const FastDiv by_page) {
    __shared__ int up[kTreeMax], path[kTreeMax], s_len;
    __shared__ int64_t from[kTreeMax], to[kTreeMax];
    const int n = blockIdx.x, tid = threadIdx.x, most = a.max_pages * a.page_size;
    int old = __ldg(a.lens + n);
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
// One cluster of CTAs does a call: its CTAs split the pages and the table between them, meet at cluster barriers, and read
// one another's bitmap of free pages and prefix sums through distributed shared memory, so that a call is
// one launch without a workspace.
constexpr int kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32, kBlock = 1024;   // pages of a block: 32 words of the bitmap
constexpr int kMaxCtas = 8;

struct PoolPlan {
    int ctas, blocks;          // CTAs; blocks of pages per CTA
    int chunk, per_row, segs;  // entries of a segment of a row; segments of a row; per CTA
    int smem;
};

struct Pool {
    cg::cluster_group cluster;
    uint32_t *words;           // of this CTA's blocks: bit set: free
    int *blk;                  // free pages before each block (within the CTA); [blocks]: all
    int *totals;               // free pages; requests
    int before[kMaxCtas + 1];  // free pages before each CTA's blocks
    int blocks;

    // The number of free pages before page p.
    __device__ int free_before(int p) const {
        const int b = p / kBlock, c = b / blocks, lb = b - c * blocks;
        const uint32_t *w = cluster.map_shared_rank(words, c) + lb * 32;
        int x = before[c] + cluster.map_shared_rank(blk, c)[lb];
        const int word = (p % kBlock) / 32;
        for (int i = 0; i < word; ++i) x += __popc(w[i]);
        return x + __popc(w[word] & ((1u << (p % 32)) - 1));
    }
    // The k-th free page (k < their number).
    __device__ int nth_free(int k) const {
        int c = 0;
        while (k >= before[c + 1]) ++c;
        k -= before[c];
        const int *pre = cluster.map_shared_rank(blk, c);
        int lo = 0, hi = blocks;   // pre[lo] <= k < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= k) lo = mid;
            else hi = mid;
        }
        k -= pre[lo];
        const uint32_t *w = cluster.map_shared_rank(words, c) + lo * 32;
        int i = 0;
        uint32_t x = w[0];
        for (int y = __popc(x); k >= y; y = __popc(x)) {
            k -= y;
            x = w[++i];
        }
        for (; k > 0; --k) x &= x - 1;
        return (c * blocks + lo) * kBlock + 32 * i + __ffs(x) - 1;
    }
};

// The bitmap of this CTA's pages (a warp per block); each page's count goes to `each`.
template <typename F> __device__ __forceinline__ void scan_pages(const ForkArgs &a, Pool &P, F each) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = warp; b < P.blocks; b += kPoolWarps) {
        const int64_t p0 = ((int64_t)P.cluster.block_rank() * P.blocks + b) * kBlock + lane;
        int sum = 0;
        for (int w0 = 0; w0 < 32; w0 += 8) {
            int r[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const int64_t p = p0 + 32 * (w0 + w);
                r[w] = p < a.pages ? __ldg(a.refs + p) : 1;
            }
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint32_t bits = __ballot_sync(0xffffffffu, r[w] == 0);
                if (lane == 0) P.words[32 * b + w0 + w] = bits;
                sum += __popc(bits);
                const int64_t p = p0 + 32 * (w0 + w);
                if (p < a.pages) each((int)p, r[w]);
            }
        }
        if (lane == 0) P.blk[b] = sum;
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

__device__ __forceinline__ Pool make_pool(const PoolPlan &plan, uint8_t *sm, int *totals) {
    Pool P{cg::this_cluster()};
    P.blocks = plan.blocks;
    P.words = reinterpret_cast<uint32_t *>(sm);
    P.blk = reinterpret_cast<int *>(P.words + 32 * plan.blocks);
    P.totals = totals;
    return P;
}
// After a cluster barrier behind the CTAs' totals.
__device__ __forceinline__ void meet(Pool &P, const PoolPlan &plan) {
    int x = 0;
#pragma unroll
    for (int c = 0; c < kMaxCtas; ++c) {
        P.before[c] = x;
        x += c < plan.ctas ? P.cluster.map_shared_rank(P.totals, c)[0] : 0;
    }
    P.before[kMaxCtas] = x;
}

// An entry of the new table, before free pages are given out.
struct NewRow {
    int src, len, full, need;   // the old row (-1: none), its length, pages that it fills, entries that have to name a page
    bool heir, copy;            // the first row that continues src; its last page is copied
    __device__ __forceinline__ NewRow(const ForkArgs &a, const FastDiv &by_page, int n) {
        src = __ldg(a.sources + n);
        if (src < 0 || src >= a.rows) src = -1;
        len = full = need = 0;
        heir = copy = false;
        if (src < 0) return;
        const int most = a.max_pages * a.page_size;
        len = __ldg(a.lens + src);
        len = len < 0 ? 0 : (len > most ? most : len);
        full = (int)by_page((uint32_t)len);
        const int more = a.new_tokens ? __ldg(a.new_tokens + n) : 0;
        const int64_t end = (int64_t)len + (more > 0 ? more : 0);
        need = a.max_pages;
        if (end < most) {
            need = (int)by_page((uint32_t)end);
            need += end > (int64_t)need * a.page_size;
        }
    }
    __device__ __forceinline__ bool part(const ForkArgs &a) const { return len > full * a.page_size; }
    // the old entry that entry e keeps, -1 for none
    __device__ __forceinline__ int kept(const ForkArgs &a, int e) const {
        if (src < 0 || !(heir || e < full + (part(a) ? 1 : 0))) return -1;
        const int p = __ldg(a.table + (int64_t)src * a.max_pages + e);
        return p < 0 || p >= a.pages ? -1 : p;
    }
    __device__ __forceinline__ bool wants(int e, int p) const { return (e < need && p < 0) || (copy && e == full); }
};
constexpr int kHeir = 1, kContinued = 2, kCopy = 4;

__global__ void __launch_bounds__(kPoolThreads) kda_paged_fork_kernel(const ForkArgs a, const PoolPlan plan, const FastDiv by_page) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int totals[2];
    Pool P = make_pool(plan, sm, totals);
    int *count = P.blk + plan.blocks + 1;                                     // pages that each segment asks for, then before it
    uint8_t *flags = reinterpret_cast<uint8_t *>(count + plan.segs);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)P.cluster.block_rank();
    const int threads = plan.ctas * kPoolThreads, gt = rank * kPoolThreads + tid;

    // the first row that continues each old row: kept in `copies` until they are written
    for (int n = gt; n < a.rows; n += threads) a.copies[2 * n] = 0x7fffffff;
    P.cluster.sync();
    for (int n = gt; n < a.rows; n += threads) {
        const int s = __ldg(a.sources + n);
        if (s >= 0 && s < a.rows) atomicMin(a.copies + 2 * (int64_t)s, n);
    }
    scan_pages(a, P, [&](int p, int r) { a.new_refs[p] = r; });
    P.cluster.sync();

    // segment sg of the CTA: entries [e0, e1) of row n
    auto segment = [&](int sg, int &n, int &e0, int &e1) {
        const int64_t g = (int64_t)rank * plan.segs + sg;
        n = (int)(g / plan.per_row);
        e0 = (int)(g - (int64_t)n * plan.per_row) * plan.chunk;
        e1 = a.max_pages - e0 < plan.chunk ? a.max_pages : e0 + plan.chunk;
        return n < a.rows;
    };
    for (int sg = warp; sg < plan.segs; sg += kPoolWarps) {
        int n, e0, e1, sum = 0, fl = 0;
        if (segment(sg, n, e0, e1)) {
            NewRow r(a, by_page, n);
            r.heir = r.src >= 0 && __ldcg(a.copies + 2 * (int64_t)r.src) == n;
            if (r.src >= 0 && r.part(a)) {
                const int p = r.kept(a, r.full);
                r.copy = p >= 0 && !(r.heir && __ldg(a.refs + p) == 1);
            }
            for (int e = e0 + lane; e < e1; e += 32) sum += r.wants(e, r.kept(a, e));
            fl = (r.heir ? kHeir : 0) | (__ldcg(a.copies + 2 * (int64_t)n) != 0x7fffffff ? kContinued : 0) | (r.copy ? kCopy : 0);
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) {
            count[sg] = sum;
            flags[sg] = (uint8_t)fl;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int x = scan_warp(P.blk, plan.blocks);
        if (lane == 0) P.blk[plan.blocks] = totals[0] = x;
    } else if (warp == 1) {
        const int x = scan_warp(count, plan.segs);
        if (lane == 0) totals[1] = x;
    }
    P.cluster.sync();
    meet(P, plan);
    int64_t asked = 0, ahead = 0;
    for (int c = 0; c < plan.ctas; ++c) {
        const int x = P.cluster.map_shared_rank(totals, c)[1];
        ahead += c < rank ? x : 0;
        asked += x;
    }
    const int missing = asked > P.before[kMaxCtas] ? (int)(asked - P.before[kMaxCtas]) : 0;
    if (gt == 0) *a.short_of = missing;

    for (int sg = warp; sg < plan.segs; sg += kPoolWarps) {
        int n, e0, e1;
        if (!segment(sg, n, e0, e1)) continue;
        const int32_t *old = a.table + (int64_t)n * a.max_pages;
        int32_t *to = a.new_table + (int64_t)n * a.max_pages;
        if (missing > 0) {
            for (int e = e0 + lane; e < e1; e += 32) to[e] = __ldg(old + e);
            if (e0 == 0 && lane == 0) {
                a.new_lens[n] = __ldg(a.lens + n);
                a.copies[2 * (int64_t)n] = a.copies[2 * (int64_t)n + 1] = -1;
            }
            continue;
        }
        NewRow r(a, by_page, n);
        r.heir = flags[sg] & kHeir;
        r.copy = flags[sg] & kCopy;
        int k = (int)ahead + count[sg];
        for (int eb = e0; eb < e1; eb += 32) {
            const int e = eb + lane;
            int p = e < e1 ? r.kept(a, e) : -1;
            const bool want = e < e1 && r.wants(e, p);
            const uint32_t all = __ballot_sync(0xffffffffu, want);
            const int was = p;
            if (want) {
                p = P.nth_free(k + __popc(all & ((1u << lane) - 1)));
                a.new_refs[p] = 1;
            }
            k += __popc(all);
            if (e < e1) {
                to[e] = p;
                if (r.copy && e == r.full) {
                    a.copies[2 * (int64_t)n] = was;
                    a.copies[2 * (int64_t)n + 1] = p;
                    if (r.heir) atomicSub(a.new_refs + was, 1);          // the old row's own reference
                } else if (!r.heir && was >= 0) {
                    atomicAdd(a.new_refs + was, 1);
                }
                if (!(flags[sg] & kContinued)) {                          // old row n ends
                    const int q = __ldg(old + e);
                    if (q >= 0 && q < a.pages) atomicSub(a.new_refs + q, 1);
                }
            }
        }
        if (e0 == 0 && lane == 0) {
            a.new_lens[n] = r.len;
            if (!r.copy) a.copies[2 * (int64_t)n] = a.copies[2 * (int64_t)n + 1] = -1;
        }
    }
    P.cluster.sync();   // the others have read this CTA's bitmap
}

__global__ void __launch_bounds__(kPoolThreads) kda_paged_compact_kernel(const ForkArgs a, const PoolPlan plan) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int totals[2];
    Pool P = make_pool(plan, sm, totals);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)P.cluster.block_rank();
    const int threads = plan.ctas * kPoolThreads, gt = rank * kPoolThreads + tid;
    scan_pages(a, P, [](int, int) {});
    __syncthreads();
    if (warp == 0) {
        const int x = scan_warp(P.blk, plan.blocks);
        if (lane == 0) P.blk[plan.blocks] = totals[0] = x;
    }
    P.cluster.sync();
    meet(P, plan);
    const int used = a.pages - P.before[kMaxCtas];
    const int moves = used < a.pages ? P.free_before(used) : 0;   // free pages below `used`, and used ones past it
    // pages: those that move leave their new place in new_refs until the table is rewritten
    for (int b = warp; b < plan.blocks; b += kPoolWarps) {
        const int p0 = (rank * plan.blocks + b) * kBlock;
        int ahead = P.before[rank] + P.blk[b];                    // free pages before the word
        for (int w = 0; w < 32; ++w) {
            const uint32_t bits = P.words[32 * b + w];
            const int p = p0 + 32 * w + lane;
            const bool in_use = p < a.pages && !((bits >> lane) & 1u);
            if (in_use && p < used) {
                a.new_refs[p] = __ldg(a.refs + p);
            } else if (in_use) {
                const int r = p - (ahead + __popc(bits & ((1u << lane) - 1))) - (used - moves);
                const int to = P.nth_free(r);
                a.new_refs[to] = __ldg(a.refs + p);
                a.new_refs[p] = to;
                a.copies[2 * r] = p;
                a.copies[2 * r + 1] = to;
            } else if (p < a.pages && p >= used) {
                a.new_refs[p] = 0;
            }
            ahead += __popc(bits);
        }
    }
    for (int r = moves + gt; r < a.pages / 2; r += threads) a.copies[2 * r] = a.copies[2 * r + 1] = -1;
    P.cluster.sync();
    const int64_t entries = (int64_t)a.rows * a.max_pages;
    for (int64_t i = gt; i < entries; i += threads) {
        const int p = __ldg(a.table + i);
        a.new_table[i] = p >= used && p < a.pages ? __ldcg(a.new_refs + p) : (p >= 0 && p < a.pages ? p : -1);
    }
    P.cluster.sync();
    for (int p = used + gt; p < a.pages; p += threads) a.new_refs[p] = 0;
}

// ------------------------------------------------------------------ copies
// Works of 16 KB of a page, a page's keys and then its values, over CTAs that stay: each thread moves four 16-byte
// vectors at a time.
constexpr int kCopyThreads = 256, kCopyAhead = 4, kCopyVecs = kCopyThreads * kCopyAhead;

__global__ void __launch_bounds__(kCopyThreads) kda_paged_copy_kernel(uint4 *kc, uint4 *vc, const int32_t *copies, const int64_t works,
                                                                      const int per_page, const int64_t page_vecs, const int pages) {
    for (int64_t w = blockIdx.x; w < works; w += gridDim.x) {
        const int64_t i = w / per_page;
        const int from = __ldg(copies + 2 * i), to = __ldg(copies + 2 * i + 1);
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
    if (fork) {
        p.chunk = 128;
        while (p.chunk < a.max_pages && (int64_t)a.rows * ((a.max_pages + p.chunk - 1) / p.chunk) > 65536) p.chunk *= 2;
        p.per_row = (a.max_pages + p.chunk - 1) / p.chunk;
        p.segs = (int)(((int64_t)a.rows * p.per_row + p.ctas - 1) / p.ctas);
    }
    p.smem = 128 * p.blocks + 4 * (p.blocks + 1) + 5 * p.segs;
    return p;
}

template <typename... A> cudaError_t launch_pool(void (*kernel)(A...), const PoolPlan &plan, cudaStream_t st, std::common_type_t<A>... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
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
    return launch_pool(kda_paged_fork_kernel, pool_plan(a, true), st, a, pool_plan(a, true), FastDiv((uint32_t)a.page_size));
}

cudaError_t launch_compact(const ForkArgs &a, cudaStream_t st) {
    return launch_pool(kda_paged_compact_kernel, pool_plan(a, false), st, a, pool_plan(a, false));
}

cudaError_t launch_page_copy(void *kc, void *vc, const int32_t *copies, int64_t count, int64_t page_vecs, int pages, cudaStream_t st) {
    const int64_t per_page = (2 * page_vecs + kCopyVecs - 1) / kCopyVecs, works = count * per_page;
    if (per_page > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int64_t most = 8 * kSms;
    kda_paged_copy_kernel<<<(unsigned)(works < most ? works : most), kCopyThreads, 0, st>>>(static_cast<uint4 *>(kc), static_cast<uint4 *>(vc), copies, works,
                                                                                           (int)per_page, page_vecs, pages);
    return cudaGetLastError();
}

}  // namespace kda
