// Attention of a draft's tokens over a paged cache: how its work is shared out (both kernels and the join).
//
// A unit is a row's key/value head with a block of up to RB of its query rows (drafted token x query head of the
// group, token-major).  Its items are its tiles of cached tokens, its tiles of drafted tokens and, ahead of them,
// `start` that stand for the time a unit's start takes.  The items of all units, in order, are cut into equal
// shares, one per CTA; each CTA finds its share from seq_lens and num_tokens on the device.  A unit in
// several shares leaves one partial (maximum, sum, unnormalised output) per share in the workspace,
// and a second kernel joins them in a fixed order, so that results do not depend on timing.
#pragma once

#include "kda_paged.cuh"
#include "kda_tree.h"

namespace kda {

struct TreeAtt {
    PagedTreeArgs t;
    FastDiv by_page, by_rep;
    int32_t rep, rb, kt;       // query heads per key/value head, query rows per block, keys per tile
    int32_t rb_log, kt_log;    // (both are powers of two)
    int32_t start;             // a unit's start, in tiles
    float *part_o, *part_ml;   // partials: [2 ctas][rb][D], [2 ctas][rb][2]
};

struct TreeRow {
    int m, len, ctx, tiles, blocks;   // drafted and cached tokens; tiles of cached ones; all; query blocks
    long long items;                  // of one unit
};
__device__ __forceinline__ TreeRow tree_row(const TreeAtt &a, int n) {
    TreeRow r;
    r.m = tree_count(a.t.num, a.t.tokens, n);
    r.len = row_length(a.t.p, n);
    r.ctx = (r.len + a.kt - 1) >> a.kt_log;
    r.tiles = r.ctx + ((r.m + a.kt - 1) >> a.kt_log);
    r.blocks = (r.m * a.rep + a.rb - 1) >> a.rb_log;
    r.items = a.start + r.tiles;
    return r;
}
__device__ __forceinline__ long long tree_items(const TreeAtt &a, int n) {   // of all its units
    const TreeRow r = tree_row(a, n);
    return r.items * r.blocks * a.t.p.kv_heads;
}

// Block-wide: the items of all rows.
template <int THREADS> __device__ __forceinline__ long long tree_total(const TreeAtt &a, long long *sm) {
    long long mine = 0;
    for (int i = threadIdx.x; i < a.t.p.rows; i += THREADS) mine += tree_items(a, i);
    return block_sum<THREADS>(mine, sm);
}

// Block-wide: the row that holds item x and the number of items before that row.
template <int THREADS>
__device__ void tree_find(const TreeAtt &a, long long x, long long *sm, int &row, long long &before) {
    __shared__ int s_row;
    __shared__ long long s_before;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    long long run = 0;
    for (int base = 0; base < a.t.p.rows; base += THREADS) {
        const int n = base + t;
        const long long w = n < a.t.p.rows ? tree_items(a, n) : 0;
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
        if (first <= x && x < first + w) {
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

// Start of share `i` of `G` equal ones.
__device__ __forceinline__ long long tree_cut(int i, long long W, long long G) {
    return W < (1 << 20) ? (long long)((uint32_t)i * (uint32_t)W / (uint32_t)G) : i * W / G;   // (i <= G <= 2^10; 64-bit divisions take long)
}
__device__ __forceinline__ int tree_quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (int)((uint32_t)x / (uint32_t)y) : (int)(x / y);
}

// Block-wide: the items W of all rows, the CTAs G that have a share, this CTA's [x, x1), the row n that it starts in and the items
// before that row.  False: this CTA has none.
template <int THREADS>
__device__ __forceinline__ bool tree_share(const TreeAtt &a, long long *sm, long long &W, long long &G, long long &x, long long &x1, int &n, long long &before) {
    __shared__ int s_row;
    __shared__ long long s_before;
    const bool one = a.t.p.rows <= THREADS;   // a thread per row: their items are read and summed once
    long long w = 0, first = 0;
    if (one) {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        auto scan = [&](long long v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            return v;
        };
        w = t < a.t.p.rows ? tree_items(a, t) : 0;
        const long long v = scan(w);
        if (lane == 31) sm[warp] = v;
        __syncthreads();
        const long long sums = scan(lane < THREADS / 32 ? sm[lane] : 0);
        W = __shfl_sync(0xffffffffu, sums, 31);
        const long long ahead = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
        first = v - w + (warp > 0 ? ahead : 0);
    } else {
        W = tree_total<THREADS>(a, sm);
    }
    G = W < gridDim.x ? W : gridDim.x;
    if (blockIdx.x >= G) return false;
    x = tree_cut(blockIdx.x, W, G);
    x1 = tree_cut(blockIdx.x + 1, W, G);
    if (one) {
        if (first <= x && x < first + w) {
            s_row = threadIdx.x;
            s_before = first;
        }
        __syncthreads();
        n = s_row;
        before = s_before;
    } else {
        tree_find<THREADS>(a, x, sm, n, before);
    }
    return true;
}

// This lane's drafted tokens `lane` and 32 + lane of row n: what they continue, as it is given (nothing waits for it here).
__device__ __forceinline__ int2 tree_parents(const TreeAtt &a, int n, int m) {
    const int i = threadIdx.x & 31;
    if (a.t.parents == nullptr) return make_int2(i - 1, i + 31);
    const int32_t *p = a.t.parents + (int64_t)n * a.t.tokens + i;
    return make_int2(i < m ? __ldg(p) : -1, i + 32 < m ? __ldg(p + 32) : -1);
}
// Path masks of a row's drafted tokens (bit j of anc[i]: token j lies on the path to i), by one warp, path lengths
// doubled each step.
__device__ __forceinline__ void tree_masks(int2 parents, int m, uint64_t *anc, int *up) {
    const int lane = threadIdx.x & 31;
    anc[lane] = lane < m ? 1ull << lane : 0;
    anc[lane + 32] = lane + 32 < m ? 1ull << (lane + 32) : 0;
    up[lane] = lane >= m || parents.x < 0 || parents.x >= lane ? -1 : parents.x;
    up[lane + 32] = lane + 32 >= m || parents.y < 0 || parents.y >= lane + 32 ? -1 : parents.y;
    __syncwarp();
#pragma unroll 1
    for (int step = 1; step < kTreeMax; step <<= 1) {
        uint64_t x[2];
        int p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            p[e] = up[lane + 32 * e];
            x[e] = p[e] >= 0 ? anc[p[e]] : 0;
            p[e] = p[e] >= 0 ? up[p[e]] : -1;
        }
        if (!__any_sync(0xffffffffu, (x[0] | x[1]) != 0)) break;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            anc[lane + 32 * e] |= x[e];
            up[lane + 32 * e] = p[e];
        }
        __syncwarp();
    }
    __syncwarp();
}

// Place of a row's position in the cache of single tokens, -1 for none; in two steps, so that what is asked for ahead is not
// waited for where it is asked.
__device__ __forceinline__ int tree_page(const TreeAtt &a, const int32_t *table, int pos) {
    const uint32_t pg = a.by_page((uint32_t)pos);
    return pg < (uint32_t)a.t.p.max_pages ? __ldg(table + pg) : -1;
}
__device__ __forceinline__ int64_t tree_place(const TreeAtt &a, int page, int pos) {
    if (page < 0 || page >= a.t.p.pages) return -1;
    return (int64_t)page * a.t.p.page_size + (pos - (int)a.by_page((uint32_t)pos) * a.t.p.page_size);
}

// Outputs of the tokens past their row's count: zero and -infinity, by part `part` of `parts`.
template <typename T, int D, int THREADS> __device__ __forceinline__ void tree_clear(const TreeAtt &a, int part, int parts) {
    if (a.t.num == nullptr) return;
    const PagedArgs &p = a.t.p;
    for (int x = part; x < p.rows; x += parts) {
        const int m = tree_count(a.t.num, a.t.tokens, x);
        const int64_t first = ((int64_t)x * a.t.tokens + m) * p.heads;
        const int rows = (a.t.tokens - m) * p.heads;
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + first * D);
        const int64_t vecs = (int64_t)rows * (D * (int)sizeof(T) / 16);   // (past 32 bits where a row has 2^21 heads)
        for (int64_t i = threadIdx.x; i < vecs; i += THREADS) out[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = threadIdx.x; i < rows; i += THREADS) p.lse[first + i] = -INFINITY;
    }
}

size_t tree_tc_workspace_bytes(const PagedTreeArgs &t, int d);
// bf16; polls: bound on each device wait
cudaError_t launch_tree_tc(const PagedTreeArgs &t, int d, void *workspace, uint32_t polls, cudaStream_t st);
// The one-launch form of bf16 calls whose rows can only be short: CTAs per unit (0: not taken), and its launch.
int tree_short_cluster(const PagedTreeArgs &t, int d);
cudaError_t launch_tree_short(const TreeAtt &a, int d, int ctas, cudaStream_t st);
// Joins the partials that a kernel of `ctas` shares left.
cudaError_t launch_tree_join(const TreeAtt &a, int d, kda_dtype_t dt, int ctas, cudaStream_t st);

}  // namespace kda
