// What the kernels over a paged cache share.
#pragma once

#include "kda_lin.h"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// t / d for 0 <= t < 2^31, by one multiplication (d >= 1): q = (hi(m t) + t) >> l with
// l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1 (the round-up method for invariant divisors).
struct FastDiv {
    uint32_t m, l;
    explicit FastDiv(uint32_t d) : l(0) {
        while ((1ull << l) < d) ++l;
        m = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t t) const { return (__umulhi(m, t) + t) >> l; }
};

__device__ __forceinline__ int row_length(const PagedArgs &a, int n) {
    const int len = __ldg(a.lens + n), most = a.max_pages * a.page_size;
    return len < 0 ? 0 : (len > most ? most : len);
}

// Block-wide sum of one value per thread, in every thread.
template <int THREADS>
__device__ __forceinline__ long long block_sum(long long x, long long *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    long long s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += sm[w];
    return s;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x on the special-function unit (2^-22 relative; results below 2^-126 become 0, which drops
// weights that small against the largest, 1).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace kda
