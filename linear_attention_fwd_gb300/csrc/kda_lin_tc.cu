// Linear attention with a decay for each head, chunkwise, on the sm_103a tensor cores
// (tcgen05 + TMEM + TMA).  bf16 inputs and outputs, fp32 state, d_k of 64 or 128, computed at d_v = 128 (a
// head of 64 value channels reads the missing ones as zeros).
//
// Chunks of C = 64 tokens; G_i = sum of the chunk's log decays up to token i, S the state before
// the chunk, all products transposed so that the state's value channels are TMEM lanes:
//   (1) dS^T  = V^T K',                 K'_j = e^{G_63 - G_j} k_j,     then S <- e^{G_63} S + dS
//   (2) O_I^T = S^T Q^T                 (scaled by e^{G_i} per token in fp32 when it is read)
//   (3) O_J^T = V^T P^T,                P_ij = (q_i . k_j) e^{G_i - G_j}, j <= i
// Every exponent is <= 0.  The sums G are kept as two floats, so that a difference is exact to fp32
// whatever the sums' magnitude.
//
// Precision.  The tensor cores multiply bf16 exactly and add in fp32.  q, k and v enter as they
// are; what is computed enters as a sum of bf16 terms, each the rounding of what the ones before it
// left: K' as three (within 2^-22 of each product, 2^-26 RMS: the state is an fp32 result), S and P as two
// (2^-16: they end in bf16 outputs, whose own rounding is 2^-8).  bf16 has fp32's range, so no scale is
// carried.  The state itself stays in registers and takes each chunk's dS by an fp32 fused
// multiply-add: the tensor cores truncate their sums, which over many chunks would pile up.
//
// Roles (20 warps; registers shared out by setmaxnreg, 104 / 104 / 96 / 96 / 80 per warpgroup out of the 5 x
// 96 of the launch: measured against eleven other splits, 1 to 50 % slower for B=4 H=32 T=8192).
// Everything meets at mbarriers; there is no CTA-wide barrier inside the loop.
//   warps 0-7    K', then the state (64 key channels of one value channel per thread) and its bf16
//                terms to TMEM
//   warps 8-15   the scores (mma.sync), the previous chunk's outputs from TMEM to global memory, P
//                (decays and bf16 terms on the scores' fragments)
//   warp 16      TMA of the tiles, three chunks ahead
//   warp 17      issues the tensor-core products
//   warps 18, 19 the decay sums, each of every other chunk
// Per chunk the tensor pipe runs (1) 12 x M128 N128 K16, (2) 16 x M128 N64 K16, (3) 8 x M128 N64
// K16, in this order: K' of the next chunk is made during (2) and (3), and the S warps have the
// whole of (1) to turn dS of the chunk before into the operand of (2).
//
// Measured (B=4 H=32 T=8192 d=128, 128 CTAs): 286 us, 3.8 TB/s, 56 % of the measured copy rate; 2.2 us a
// chunk.  What bounds it is the issue rate with the chunk's chain of hand-overs.  Counted at T=1024: an SM issues
// about 10,000 warp instructions a chunk at 2.1 a cycle, the tensor pipe is busy 38 % of the time.
// No single part carries it: left out one at a time, P and K' save 35 us each, the scores 29, the
// products 27, S's terms 20, the outputs 15, the decay sums 9.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_lin.h"
#include "tc_ptx.cuh"

namespace kda {

// Count of bounded device waits that gave up since the host last read it.
__device__ unsigned int g_kda_lin_timeouts = 0;

namespace {

using namespace ptx;

constexpr int C = 64, NT = 20 * 32;
constexpr int kStages = 3;

// shared memory, byte offsets from a 1024-aligned base
constexpr uint32_t STAGE = 3 * 16384;                       // Q, K, V tiles [64][128] bf16, 128-byte swizzle
constexpr uint32_t OFF_KP = kStages * STAGE;                // K': three terms [64][128] bf16, same layout
constexpr uint32_t OFF_P = OFF_KP + 3 * 16384;              // P: two terms [64 i][64 j] bf16
constexpr uint32_t OFF_G = OFF_P + 2 * 8192;                // decay vectors, a slot per stage
constexpr uint32_t G_SLOT = 5 * 64 * 4 + 16;                //   G hi, G lo, e^{G_63 - G} as bf16 terms (two words a
                                                            //   token: first and second, third twice), e^G; e^{G_63}
constexpr uint32_t OFF_BAR = OFF_G + kStages * G_SLOT;
// A wait names a phase by its parity, so no barrier may complete a phase before every waiter has
// passed the one before.  That holds because each phase needs, directly or through others, an
// arrival that its slowest waiter makes after that pass; the products (1) run ahead of the S warps
// and so have a barrier for each of dS's buffers.
enum Bar { kFull = 0, kEmpty = 3, kKp = 6, kP = 7 /* kKp + 1 */, kReady = 8, kOFull = 9, kDone = 10, kBars = 12 };
constexpr uint32_t OFF_TM = OFF_BAR + kBars * 8;
constexpr uint32_t SMEM_BYTES = OFF_TM + 16 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(OFF_BAR % 8 == 0 && G_SLOT % 16 == 0, "alignment");

// tensor memory columns (lane = value channel)
constexpr uint32_t TM_DS = 0;       // (1), two buffers                         2 x 128
constexpr uint32_t TM_S16 = 256;    // S^T as two bf16 terms                    64 + 64
constexpr uint32_t TM_OI = 384;     // (2)                                      64
constexpr uint32_t TM_OJ = 448;     // (3)                                      64
constexpr uint32_t TM_COLS = 512;

constexpr uint32_t IDESC_SQ = idesc_bf16_f32(128, 64);                              // A in TMEM, B (Q) K-major
constexpr uint32_t IDESC_VP = idesc_bf16_f32(128, 64) | (1u << 15);                 // A (V) MN-major, B (P) K-major

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// mbar_wait with its loop kept a loop: unrolled at every place that waits, it would push the loop
// bodies out of the instruction cache (measured: half of the kernel's time).
__device__ __forceinline__ bool mbar_wait_small(uint32_t bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_wait(bar, parity, 1)) return true;
    return false;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<__nv_bfloat162 *>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t *>(&x); }

// Shared-memory operand descriptors here differ in their low words only: address, and for operands read
// across their rows (MN-major) the distance of their 64-column halves.  The rest: 8-row groups 1024 bytes
// apart, version 1, 128-byte swizzle (see sdesc_sw128, sdesc_sw128_mn).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return (saddr >> 4) | ((8192u >> 4) << 16); }
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate),
        "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate),
        "n"(kDescHigh)
        : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(one));
    return one;
}

// ldmatrix at a constant offset from an address
template <int OFF> __device__ __forceinline__ void ldsm_x4_at(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF));
}

// Two loads of 16 lanes x 32 columns as four 8-column fragments each (row lane / 4, columns 2 (lane % 4)
// and the next: registers 4 c, 4 c + 1; row + 8: 4 c + 2, 4 c + 3), and one wait.
__device__ __forceinline__ void tmem_ld_16x256b_x4_pair(uint32_t ta, uint32_t tb, float (&v)[16], float (&w)[16]) {
    uint32_t r[16], q[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]),
          "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]),
          "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
        : "r"(ta), "r"(tb)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = __uint_as_float(r[i]);
        w[i] = __uint_as_float(q[i]);
    }
}
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Scores of 16 query rows (from qa) against three blocks of 8 keys (from ka) over 32 channels: the
// KK-th such step.  A row's 16-byte pieces are 128-byte swizzled, halves of 64 channels 8 KB apart.
template <int KK> __device__ __forceinline__ void scores_step(uint32_t qa, uint32_t ka, float (&acc)[3][4]) {
    constexpr int H = (KK >> 1) * 8192, X = 64 * (KK & 1);
    uint32_t q0[4], q1[4], k0[4], k1[4], k2[4];
    ldsm_x4_at<H>(qa ^ X, q0);
    ldsm_x4_at<H>(ka ^ X, k0);
    ldsm_x4_at<H + 1024>(ka ^ X, k1);
    ldsm_x4_at<H + 2048>(ka ^ X, k2);
    ldsm_x4_at<H>(qa ^ X ^ 32, q1);
    mma_16816(acc[0], q0[0], q0[1], q0[2], q0[3], k0[0], k0[1]);
    mma_16816(acc[1], q0[0], q0[1], q0[2], q0[3], k1[0], k1[1]);
    mma_16816(acc[2], q0[0], q0[1], q0[2], q0[3], k2[0], k2[1]);
    mma_16816(acc[0], q1[0], q1[1], q1[2], q1[3], k0[2], k0[3]);
    mma_16816(acc[1], q1[0], q1[1], q1[2], q1[3], k1[2], k1[3]);
    mma_16816(acc[2], q1[0], q1[1], q1[2], q1[3], k2[2], k2[3]);
}

// w as three bf16 terms: the first | the second << 16, the third twice
__device__ __forceinline__ uint2 three_bf16(float w) {
    const float a = __bfloat162float(__float2bfloat16_rn(w)), b = __bfloat162float(__float2bfloat16_rn(w - a));
    const float c = (w - a) - b;
    return make_uint2(pack_bf16(a, b), pack_bf16(c, c));
}

// K' = k w in packed bf16 arithmetic, by THREADS threads: the keys of the tiles at `st` into three terms at
// `kp`, `term` bytes apart.  The factor comes as three bf16 terms; k w_0 = h + e and k w_1 = y + y' exactly
// (8-bit times 8-bit significands), m = e + y rounded, and the third term is what that rounding left
// plus y' + k w_2: the sum of the three is within 2^-22 (2^-26 RMS) of k w.  16-byte pieces lie at the
// same offsets in K and K'.  (Loads come before stores here and below: the compiler keeps their order,
// and a load behind a store waits its whole way.)
template <int THREADS, int kDk>
__device__ __forceinline__ void scale_keys(uint8_t *sm, uint32_t st, uint32_t kp, uint32_t term, const float *gv, int nr, int tid) {
    constexpr int E = 8 * kDk >= 2 * THREADS ? 2 : 1;
#pragma unroll 1
    for (int x0 = tid; x0 < 8 * kDk; x0 += E * THREADS) {
        uint4 uk[E];
        uint2 wk[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int x = x0 + THREADS * e;
            uk[e] = *reinterpret_cast<const uint4 *>(sm + st + 16384 + 16 * x);
            wk[e] = reinterpret_cast<const uint2 *>(gv + 128)[(x >> 3) & 63];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int x = x0 + THREADS * e, r = (x >> 3) & 63;
            const __nv_bfloat162 w0 = as_bf162(__byte_perm(wk[e].x, 0, 0x1010)), w1 = as_bf162(__byte_perm(wk[e].x, 0, 0x3232)),
                                 w2 = as_bf162(wk[e].y);
            if (nr < C && r >= nr) {   // rows past the sequence belong to another one: they never enter a product
                uk[e] = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4 *>(sm + st + 32768 + 16 * x) = uk[e];
                if (kDk == 64) *reinterpret_cast<uint4 *>(sm + st + 40960 + 16 * x) = uk[e];   // V is 128 wide
            }
            const uint32_t uw[4] = {uk[e].x, uk[e].y, uk[e].z, uk[e].w};
            uint32_t o0[4], o1[4], o2[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const __nv_bfloat162 kv = as_bf162(uw[c]);
                const __nv_bfloat162 hh = __hmul2_rn(kv, w0), ee = __hfma2(kv, w0, __hneg2(hh));
                const __nv_bfloat162 yy = __hmul2_rn(kv, w1), ye = __hfma2(kv, w1, __hneg2(yy));
                const __nv_bfloat162 mm = __hadd2_rn(ee, yy);
                const __nv_bfloat162 ll = __hadd2_rn(__hsub2_rn(yy, __hsub2_rn(mm, ee)), __hfma2(kv, w2, ye));
                o0[c] = as_u32(hh);
                o1[c] = as_u32(mm);
                o2[c] = as_u32(ll);
            }
            uint4 *to = reinterpret_cast<uint4 *>(sm + kp + 16 * x);
            to[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
            to[term / 16] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            to[term / 8] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
        }
    }
}

// x as a bf16 pair and the rest it leaves.  Values past the largest bf16 take that one (rounded they would be
// infinite, their rest minus infinity and the two terms' products NaN); the rest of a finite x is then at most
// 2^-8 of it and exact, as for any other x.
__device__ __forceinline__ uint32_t take_bf16(float2 &x) {
    uint32_t h;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x.y), "f"(x.x));
    x = __ffma2_rn(make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), make_float2(-1.f, -1.f), x);
    return h;
}

// The work of a CTA: part p of P of sequence n's chunks, [p nc / P, (p + 1) nc / P), for head h.  A
// sequence that is cut (see cut_of) has ceil(nc / target) parts (at most kMaxParts); its parts other than
// the last have a slot each for states (`slot`: the sequence's first).  P = 0: nothing.
struct Piece {
    int n, h, p, P, slot, bos, eos, pad;
};
static_assert(sizeof(Piece) == 32, "two 16-byte words");
constexpr int kMaxParts = 32;

struct CutRule {
    int most, target;   // sequences of more than `most` chunks are cut, into parts of about `target`
    int slots;
    int whole, parts;   // dense: (sequence, head) units before `whole` are not cut, the others into `parts`
    bool fold;          // no scan (see kFold)
    int alone;          // packed: the target where one sequence has four fifths of all chunks (0: none)
};

__device__ __forceinline__ Piece load_piece(const Piece *from) {
    const int4 x = __ldcg(reinterpret_cast<const int4 *>(from)), y = __ldcg(reinterpret_cast<const int4 *>(from) + 1);
    return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// Dense batches: the piece of CTA b by arithmetic.  kFullPass: over all parts, else over all but each
// cut unit's last.
template <bool kFullPass>
__device__ __forceinline__ Piece dense_piece(const LinArgs &a, int b, const CutRule &cut) {
    const int x = kFullPass ? b - cut.whole : b, cuts = a.num_seqs * a.heads - cut.whole;
    const int p = x >= 0 ? x / cuts : 0, u = x >= 0 ? cut.whole + x % cuts : b, P = x >= 0 ? cut.parts : 1, n = u / a.heads;
    return {n, u % a.heads, p, P, (n - cut.whole / a.heads) * (P - 1), (int)(n * a.seqlen), (int)((n + 1) * a.seqlen), 0};
}

// Packed sequences: one CTA makes the lists of pieces, `pre` of all parts but each sequence's last, `full`
// of all, longest parts first (the hardware dispatches low blocks first; more than kPlanThreads of them
// keep their order); what is left of the lists is P = 0.  A sequence that would need more slots than there
// are is not cut (only offsets that are not as documented come to that).  The lists are made here and
// not by each CTA for itself because that search, merely by being in the main kernel, cost its loops 40 %.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) lin_plan_kernel(const LinArgs a, const CutRule cut, Piece *pre, int pre_n, Piece *full, int full_n) {
    __shared__ int s_len[kPlanThreads], s_parts[kPlanThreads], s_slot[kPlanThreads], s_first[kPlanThreads], s_pre[kPlanThreads];
    __shared__ int s_sum[3][kPlanThreads / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, N = a.num_seqs, H = a.heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int used = 0, seqs = 0, cuts = 0;   // of the tiles before: slots asked for, parts, parts but each sequence's last
    for (int base = 0; base < N; base += kPlanThreads) {
        const int here = N - base < kPlanThreads ? N - base : kPlanThreads;
        int64_t b = 0, e = 0;
        if (t < here) lin_range(a, base + t, b, e);
        const int len = (int)(e - b), nc = (len + C - 1) / C;
        int parts = t < here ? 1 : 0, target = cut.target;
        if (cut.alone > 0 && N <= kPlanThreads) {
            const int most = __reduce_max_sync(0xffffffffu, nc), sum = __reduce_add_sync(0xffffffffu, nc);
            if (lane == 0) {
                s_sum[0][warp] = most;
                s_sum[1][warp] = sum;
            }
            __syncthreads();
            int x = 0, y = 0;
            for (int i = 0; i < kPlanThreads / 32; ++i) {
                x = s_sum[0][i] > x ? s_sum[0][i] : x;
                y += s_sum[1][i];
            }
            if ((int64_t)x * 5 > (int64_t)y * 4) target = cut.alone;
        }
        if (t < here && nc > cut.most) {
            parts = (nc + target - 1) / target;
            if (parts > kMaxParts) parts = kMaxParts;
        }
        __syncthreads();
        // slots before this sequence; one that would leave them is not cut, nor are those after it
        auto scan = [&](int x, int row) {   // exclusive over the block; the total in s_sum[row] of the last warp's end
            int v = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            if (lane == 31) s_sum[row][warp] = v;
            __syncthreads();
            int off = 0;
            for (int i = 0; i < warp; ++i) off += s_sum[row][i];
            return off + v - x;
        };
        auto total = [&](int row) {
            int x = 0;
            for (int i = 0; i < kPlanThreads / 32; ++i) x += s_sum[row][i];
            return x;
        };
        int slot = used + scan(parts > 0 ? parts - 1 : 0, 0);
        if (parts > 1 && slot + parts - 1 > cut.slots) parts = 1;
        const int key = parts > 0 ? (len + parts - 1) / parts : -1;   // a part's tokens
        s_len[t] = key;
        s_parts[t] = parts;
        s_slot[t] = slot;
        __syncthreads();
        // parts before this sequence, longest first when one tile holds them all
        int first = 0, before = 0;
        if (N <= kPlanThreads) {
            if (t < here)
                for (int i = 0; i < here; ++i) {
                    const bool ahead = s_len[i] > key || (s_len[i] == key && i < t);
                    first += ahead ? s_parts[i] : 0;
                    before += ahead ? s_parts[i] - 1 : 0;
                }
        } else {
            first = seqs + scan(parts, 1);
            before = cuts + scan(parts > 0 ? parts - 1 : 0, 2);
        }
        s_first[t] = first;
        s_pre[t] = before;
        used += total(0);
        if (N > kPlanThreads) {
            seqs += total(1);
            cuts += total(2);
        }
        __syncthreads();
        for (int i = warp; i < here; i += kPlanThreads / 32) {   // a warp per sequence
            int64_t sb, se;
            lin_range(a, base + i, sb, se);
            const int P = s_parts[i];
            for (int x = lane; x < P * H; x += 32) {
                const Piece piece{base + i, x % H, x / H, P, s_slot[i], (int)sb, (int)se, 0};
                const int f = s_first[i] * H + x, q = s_pre[i] * H + x;
                if (f < full_n) full[f] = piece;
                if (x < (P - 1) * H && q < pre_n) pre[q] = piece;
            }
        }
        if (N <= kPlanThreads) {   // all parts of all sequences
            int x = 0, y = 0;
            for (int i = 0; i < here; ++i) {
                x += s_parts[i];
                y += s_parts[i] - 1;
            }
            seqs = x;
            cuts = y;
        }
    }
    for (int x = seqs * H + t; x < full_n; x += kPlanThreads) full[x].P = 0;
    for (int x = cuts * H + t; x < pre_n; x += kPlanThreads) pre[x].P = 0;
}

// kFullPass: the whole forward of a part; a part other than the first starts from the state in the slot
// of the part before it.  Otherwise only the state that a part reaches from zero, into its slot of
// `locals`, and its total log2 decay; lin_scan_kernel then turns each slot into the true state behind
// its part.  There warps 0-15 make K' together, a chunk ahead of the products, and warps 0-7 the state: 1.1 us
// a chunk, its chain of hand-overs (8 warps and one K' at a time: 1.75 us).
// kFold (full pass over several packed sequences, after a first pass): sequences that are not cut start beside
// the first pass, and each part chains the states before it itself, so that there is no scan between the
// passes (16384 + 8192 + 8192 + 4096 tokens of 32 heads: 378 us, with a scan 473).  The CTAs of a part wait for the
// first pass at their start, all others at their end, so that the call's memory is not reused too early.
// kDk: the key channels, 64 or 128 (value channels are always 128 lanes; those a head lacks read as zeros).
template <bool kFullPass, int kDk, bool kFold>
__global__ void __launch_bounds__(NT, 1)
kda_lin_chunk_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv, const LinArgs a, const CutRule cut, const Piece *plan,
                        float *locals, double *decays) {
    constexpr uint32_t IDESC_KV = idesc_bf16_f32(128, kDk) | (1u << 15) | (1u << 16);   // A (V) and B (K') MN-major
    constexpr int KC = kDk / 2;                // key channels of the state per thread
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_fail;
    __shared__ double s_decay[2];
    __shared__ volatile int s_piece[4];   // unit, the part's slot, whether it is the last (read again at the end:
                                          // registers are scarce in the loop)
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int H = a.heads;
    // (launched before the kernel ahead of it has ended, see launch_lin_chunk_tc)
    auto wait_ahead = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (!kFold) wait_ahead();
    // (behind the wait: what depends on this pass may read the lists, which an earlier kernel made)
    if (!kFullPass) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Piece piece = plan ? load_piece(plan + blockIdx.x) : dense_piece<kFullPass>(a, blockIdx.x, cut);
    const int n = piece.n, h = piece.h, p = piece.p, P = piece.P, slot = piece.slot;
    if (kFold && P != 1) wait_ahead();
    if (P == 0) return;
    const int hk = h / (H / a.qk_heads);
    const int bos = piece.bos, eos = piece.eos;        // tokens are counted in 31 bits
    const int nc = (eos - bos + C - 1) / C;
    const int c_lo = (int)((int64_t)p * nc / P), c_hi = (int)((int64_t)(p + 1) * nc / P);
    const int chunks = c_hi - c_lo;
    const int first = bos + c_lo * C;                  // the part's first token
    const bool last_part = p == P - 1;
    if (chunks == 0 && kFullPass && !(last_part && a.sT)) {
        if (kFold) wait_ahead();
        return;
    }

    auto bar = [&](int b) { return sb + OFF_BAR + 8 * b; };
    if (tid == 0) {
        s_fail = 0;
        s_piece[0] = n * H + h;
        s_piece[1] = (slot + p) * H + h;
        s_piece[2] = last_part;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kFull + s), 1 + 32);                // the tiles, and the warp that writes the decay vectors
            mbar_init(bar(kEmpty + s), kFullPass ? 9 : 1);   // the products, and the warps that staged outputs there
        }
        mbar_init(bar(kKp), kFullPass ? 256 : 512);
        mbar_init(bar(kP), kFullPass ? 256 : 512);   // first pass: K' of odd chunks
        mbar_init(bar(kReady), 512);
        mbar_init(bar(kDone), 1);
        mbar_init(bar(kDone + 1), 1);
        mbar_init(bar(kOFull), 1);
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(sb + OFF_TM, TM_COLS);
        tmem_relinquish();
    }
    if (kFullPass && warp >= 12 && warp < 16)   // P's blocks above the diagonal stay zero
        for (int x = tid - 384; x < 1024; x += 128) *reinterpret_cast<uint4 *>(sm + OFF_P + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sm + OFF_TM), 0);
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int jl = 32 * (warp & 3) + lane;             // value channel of this thread's TMEM lane
    auto gslot = [&](int k) { return reinterpret_cast<float *>(sm + OFF_G + (k % kStages) * G_SLOT); };
    auto wait = [&](int b, uint32_t parity) { return mbar_wait_small(bar(b), parity & 1u, a.wait_polls); };
    auto done = [&](int k) { return wait(kDone + (k & 1), k >> 1); };
    bool ok = true;
    // K' of chunk k in the first pass, by 512 threads: chunk k + 1's is made while the products of chunk k run,
    // odd chunks' in the places of the Q tiles, which that pass does not load (the last products to read
    // from there, chunk k - 2's, are done).
    auto keys_of_pass_one = [&](int k) {
        if (!((k < 2 || done(k - 2)) && wait(kFull + k % kStages, k / kStages))) return false;
        const int left = eos - (first + k * C);
        scale_keys<512, kDk>(sm, (k % kStages) * STAGE, k & 1 ? 0 : OFF_KP, k & 1 ? STAGE : 16384, gslot(k), left < C ? left : C, tid);
        fence_async_smem();
        return true;
    };

    if (warp < 8) {
        // ---- S
        regs_inc<104>();
        const int i0 = KC * (warp >> 2);
        const int64_t sstep = (int64_t)kDk * a.dv;
        const bool mine = jl < a.dv;
        const int64_t at = (int64_t)i0 * a.dv + jl;
        float v[KC];
#pragma unroll
        for (int c = 0; c < KC; ++c) v[c] = 0.f;
        if (kFullPass && mine) {
            const float *from = p > 0 && !kFold ? locals + ((int64_t)(slot + p - 1) * H + h) * sstep : (a.s0 ? a.s0 + ((int64_t)n * H + h) * sstep : nullptr);
            if (from)
#pragma unroll
                for (int c = 0; c < KC; ++c) v[c] = __ldcg(from + at + (int64_t)c * a.dv);
#pragma unroll 1
            for (int e = 0; kFold && e < p; ++e) {   // the parts before this one
                const int64_t of = (int64_t)(slot + e) * H + h;
                const float f = exp2f((float)__ldcg(decays + of));
#pragma unroll
                for (int c = 0; c < KC; ++c) v[c] = fmaf(f, v[c], __ldcg(locals + of * sstep + at + (int64_t)c * a.dv));
            }
        }
        auto take_ds = [&](int k, float f) {   // v <- f v + dS of chunk k
            tc_fence_after();
            const float2 d2 = make_float2(f, f);
#pragma unroll
            for (int b = 0; b < KC / 32; ++b) {
                float w[32];
                tmem_ld32(trow + TM_DS + 128 * (k & 1) + i0 + 32 * b, w);
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 x = __ffma2_rn(d2, make_float2(v[32 * b + c], v[32 * b + c + 1]), make_float2(w[c], w[c + 1]));
                    v[32 * b + c] = x.x;
                    v[32 * b + c + 1] = x.y;
                }
            }
        };
        float dec = 0.f;   // e^(sum of the chunk's log decays)
        for (int k = 0; !kFullPass && k <= chunks; ++k) {
            float next = 0.f;
            if (k < chunks) {
                ok = keys_of_pass_one(k);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                next = gslot(k)[320];
                mbar_arrive(bar(kKp + (k & 1)));
            }
            if (k > 0) {
                ok = done(k - 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                take_ds(k - 1, dec);
                tc_fence_before();
            }
            dec = next;
        }
        for (int k = 0; kFullPass && k <= chunks; ++k) {
            // dS and K' of the chunk before are done with; this chunk's tile and decays landed
            if (k > 0) ok = done(k - 1);
            if (ok && k < chunks) ok = wait(kFull + k % kStages, k / kStages);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            if (k < chunks) {
                const uint32_t st = (k % kStages) * STAGE;
                const float *gv = gslot(k);
                const int left = eos - (first + k * C), nr = left < C ? left : C;
                scale_keys<256, kDk>(sm, st, OFF_KP, 16384, gv, nr, tid);
                fence_async_smem();
                mbar_arrive(bar(kKp));
            }
            if (k > 0) take_ds(k - 1, dec);
            if (k == chunks) break;
            dec = gslot(k)[320];
            if (kFullPass) {
                ok = k == 0 || wait(kOFull, k - 1);   // the chunk before has read its operand
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int b = 0; b < KC / 16; ++b) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float2 x = make_float2(v[16 * b + 2 * c], v[16 * b + 2 * c + 1]);
                        hi[c] = take_bf16(x);
                        lo[c] = pack_bf16(x.x, x.y);
                    }
                    tmem_st8u(trow + TM_S16 + i0 / 2 + 8 * b, hi);
                    tmem_st8u(trow + TM_S16 + 64 + i0 / 2 + 8 * b, lo);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(bar(kReady));
        }
        float *to = kFullPass ? (s_piece[2] ? a.sT : nullptr) : locals;
        if (ok && to && mine) {
            to += (int64_t)s_piece[kFullPass ? 0 : 1] * sstep + at;
#pragma unroll
            for (int c = 0; c < KC; ++c) to[(int64_t)c * a.dv] = v[c];
        }
    } else if (warp < 16) {
        // ---- scores, P and O, each of the two halves of these warps half of it
        regs_dec<96>();
        const int half = (warp - 8) >> 2;
        const int w4 = warp & 3, g = lane >> 2, t4 = lane & 3;
        // O: 32 tokens x 32 channels a warp.  TMEM is read as 8 x 8 fragments (channel, token), which stmatrix
        // turns into rows of a token's channels, 64 bytes with their 16-byte pieces swizzled.
        const int64_t tok_bytes = (int64_t)H * a.dv * 2;
        const uint32_t o_row = ((lane >> 4) * 8 + (lane & 7)) * 64, o_sw = (lane & 7) >> 1;
        const uint32_t o_st[2] = {o_row + ((((lane >> 3) & 1) ^ o_sw) << 4), o_row + (((2 + ((lane >> 3) & 1)) ^ o_sw) << 4)};
        const uint32_t o_ld = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
        const int64_t o_off = (32 * half + (lane >> 2)) * tok_bytes + (32 * w4 + 8 * (lane & 3)) * 2;
        // P: 20 blocks of 16 x 8 on or below the diagonal: the first half's warps take three of row block
        // I from c0, the second's two, so that each has at most two on the diagonal's 16 tokens
        const int I = half ? (w4 == 0 ? 0 : (w4 == 2 ? 3 : 1)) : (w4 < 2 ? 3 : 2);
        const int c0 = half ? (w4 == 1 ? 2 : (w4 == 2 ? 6 : 0)) : (w4 & 1 ? 3 : 0);
        const int i = 16 * I + g;
        const uint32_t qrow = sb + (16 * I + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
        const uint32_t krow = sb + 16384 + (8 * c0 + (lane & 7)) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
        uint8_t *prow = sm + OFF_P + i * 128 + 4 * t4;
        for (int k = 0; !kFullPass && k < chunks; ++k) {
            ok = keys_of_pass_one(k);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            mbar_arrive(bar(kKp + (k & 1)));
        }
        for (int k = 0; kFullPass && k <= chunks; ++k) {
            const uint32_t st = (k % kStages) * STAGE;
            const float *gv = gslot(k);
            const int left = eos - (first + k * C), nr = left < C ? left : C;
            float acc[3][4];
            if (k < chunks) {
                ok = wait(kFull + k % kStages, k / kStages);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                // scores, 32 channels at a time (the second half's third block is not used)
#pragma unroll
                for (int b = 0; b < 3; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[b][e] = 0.f;
                scores_step<0>(qrow + st, krow + st, acc);
                scores_step<1>(qrow + st, krow + st, acc);
                if constexpr (kDk == 128) {
                    scores_step<2>(qrow + st, krow + st, acc);
                    scores_step<3>(qrow + st, krow + st, acc);
                }
            }
            const uint32_t stg = ((k + kStages - 1) % kStages) * STAGE + 2048 * (warp - 8);
            if (k > 0) {   // the previous chunk's outputs; its P is consumed
                ok = wait(kOFull, k - 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *eg = gslot(k - 1) + 256 + 32 * half + 2 * t4;
                // 32 tokens x 32 channels into this warp's 2 KB of the chunk's (consumed) Q tile
                float2 e2[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) e2[c] = *reinterpret_cast<const float2 *>(eg + 8 * c);
#pragma unroll
                for (int L = 0; L < 2; ++L) {   // 16 channels
                    float v[16], w[16];
                    const uint32_t tl = trow + (L << 20) + 32 * half;
                    tmem_ld_16x256b_x4_pair(tl + TM_OI, tl + TM_OJ, v, w);
                    uint32_t x[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float2 y = __ffma2_rn(e2[c / 2], make_float2(v[2 * c], v[2 * c + 1]), make_float2(w[2 * c], w[2 * c + 1]));
                        x[c] = pack_bf16(y.x, y.y);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        stsm_x4_t(sb + stg + o_st[L] + 1024 * e, x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                }
                tc_fence_before();
            }
            if (k < chunks) {   // P
                mbar_arrive(bar(kReady));
                const int m0 = i < nr ? i : nr - 1, m1 = i + 8 < nr ? i + 8 : nr - 1;   // the last key of each row
                const float gh0 = gv[i], gh1 = gv[i + 8], gl0 = gv[64 + i], gl1 = gv[72 + i];
                const float2 neg = make_float2(-1.f, -1.f);
                float2 hj[3], lj[3];
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    const int j = (8 * (c0 + b) + 2 * t4) & 63;
                    hj[b] = *reinterpret_cast<const float2 *>(gv + j);
                    lj[b] = *reinterpret_cast<const float2 *>(gv + 64 + j);
                }
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    if (b == 2 && half) continue;
                    const int j = 8 * (c0 + b) + 2 * t4;
                    uint8_t *to = prow + (((c0 + b) ^ g) << 4);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const float gh = hh ? gh1 : gh0, gl = hh ? gl1 : gl0;
                        const int m = hh ? m1 : m0;
                        float2 x;
                        const float2 d = __fadd2_rn(__ffma2_rn(hj[b], neg, make_float2(gh, gh)), __ffma2_rn(lj[b], neg, make_float2(gl, gl)));
                        x = __fmul2_rn(make_float2(acc[b][2 * hh], acc[b][2 * hh + 1]), make_float2(ex2(d.x), ex2(d.y)));
                        x = make_float2(j <= m ? x.x : 0.f, j < m ? x.y : 0.f);
                        *reinterpret_cast<uint32_t *>(to + 1024 * hh) = take_bf16(x);
                        *reinterpret_cast<uint32_t *>(to + 1024 * hh + 8192) = pack_bf16(x.x, x.y);
                    }
                }
            }
            // (one fence for P and the staged outputs, whose place TMA takes next; the outputs' stores come
            // after it, as a fence waits for what is in flight)
            fence_async_smem();
            if (k < chunks) mbar_arrive(bar(kP));
            if (k > 0) {
                __syncwarp();
                uint4 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const uint4 *>(sm + stg + o_ld + 512 * e);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kEmpty + (k - 1) % kStages));
                const int t0 = first + (k - 1) * C, past = eos - t0 - 32 * half;
                uint8_t *o = static_cast<uint8_t *>(a.out) + (((int64_t)t0 * H + h) * a.dv) * 2 + o_off;
                const int rows = 32 * w4 < a.dv ? (past < 32 ? past : 32) - (lane >> 2) : 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * e < rows) *reinterpret_cast<uint4 *>(o + 8 * e * tok_bytes) = y[e];
            }
        }
    } else {
        regs_dec<80>();
        if (warp == 16) {
            // ---- tiles by TMA
            for (int k = 0; k < chunks; ++k) {
                const int s = k % kStages;
                ok = k < kStages || wait(kEmpty + s, k / kStages - 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t st = sb + s * STAGE, b = bar(kFull + s);
                    const int tok = first + k * C;
                    mbar_arrive_expect_tx(b, 16384 + (kFullPass ? 2 : 1) * 128 * kDk);
                    tma_load_3d(st + 16384, &tmk, b, 0, hk, tok);
                    if (kDk == 128) tma_load_3d(st + 24576, &tmk, b, 64, hk, tok);
                    tma_load_3d(st + 32768, &tmv, b, 0, h, tok);
                    tma_load_3d(st + 40960, &tmv, b, 64, h, tok);
                    if (kFullPass) {
                        tma_load_3d(st, &tmq, b, 0, hk, tok);
                        if (kDk == 128) tma_load_3d(st + 8192, &tmq, b, 64, hk, tok);
                    }
                }
                __syncwarp();
            }
        } else if (warp == 17) {
            // ---- tensor-core products.  The whole warp runs the loop and an elected lane issues, so that the
            // operand descriptors can stay in uniform registers (half the instructions per product).
            const uint32_t pd = desc_k(sb + OFF_P), kpd = desc_mn(sb + OFF_KP);
            const uint32_t one = elect_one();
            int s = 0;
            for (int k = 0; k < chunks; ++k) {
                const uint32_t vd = desc_mn(sb + s * STAGE + 32768), qd = desc_k(sb + s * STAGE);
                // dS of two chunks ago was taken before the S warps got ready for the chunk before (full pass) or
                // made this chunk's K' (first pass)
                ok = kFullPass ? wait(kKp, k) : wait(kKp + (k & 1), k >> 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ds = tmem + TM_DS + 128 * (k & 1);
                if (one) {
                    const uint32_t kd = kFullPass || !(k & 1) ? kpd : desc_mn(sb), term = (kFullPass || !(k & 1) ? 16384 : STAGE) >> 4;
#pragma unroll 1
                    for (int e = 2; e >= 0; --e)   // the smallest terms first
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(ds, vd + ((2048 * kk) >> 4), kd + term * e + ((2048 * kk) >> 4), IDESC_KV, e < 2 || kk > 0);
                    mma_commit(bar(kDone + (k & 1)));
                }
                __syncwarp();
                if (kFullPass) {
                    ok = wait(kReady, k);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (one) {
#pragma unroll 1
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int kk = 0; kk < kDk / 16; ++kk)
                                mma_ts(tmem + TM_OI, tmem + TM_S16 + 64 * e + 8 * kk, qd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4),
                                           IDESC_SQ, e + kk > 0);
                    }
                    __syncwarp();
                    ok = wait(kP, k);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (one) {
#pragma unroll 1
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(tmem + TM_OJ, vd + ((2048 * kk) >> 4), pd + ((8192 * e + 32 * kk) >> 4), IDESC_VP, e + kk > 0);
                        mma_commit(bar(kOFull));
                    }
                }
                if (one) mma_commit(bar(kEmpty + s));
                __syncwarp();
                if (++s == kStages) s = 0;
            }
            // nothing arrives at a barrier after the CTA has ended
            for (int k = chunks > kStages ? chunks - kStages : 0; ok && k < chunks; ++k) ok = wait(kEmpty + k % kStages, k / kStages);
        } else {
            // ---- the decay sums, every other chunk's: lane l holds tokens 2l and 2l + 1
            float th = 0.f, tl = 0.f;   // the part's sum
            const float hg = a.head_g ? __ldg(a.head_g + h) : 0.f;
            const float *gp = a.g ? a.g + (int64_t)(first + 2 * lane) * H + h : nullptr;
            float gx = 0.f, gy = 0.f;
            auto load_g = [&](int k) {
                const int t = first + k * C + 2 * lane;
                gx = gp && t < eos ? __ldg(gp + (int64_t)k * C * H) : 0.f;
                gy = gp && t + 1 < eos ? __ldg(gp + (int64_t)k * C * H + H) : 0.f;
            };
            const int k0 = warp & 1;
            if (k0 < chunks) load_g(k0);
            for (int k = k0; k < chunks; k += 2) {
                const int s = k % kStages;
                ok = k < kStages || wait(kEmpty + s, k / kStages - 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const int t = first + k * C + 2 * lane;
                float xh, xl, yh, yl;
                log2_decay(gx, hg, t < eos, xh, xl);
                log2_decay(gy, hg, t + 1 < eos, yh, yl);
                if (k + 2 < chunks) load_g(k + 2);
                float bh = xh, bl = xl;            // sums up to the lane's second token
                add2f(bh, bl, yh, yl);
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const float ph = __shfl_up_sync(0xffffffffu, bh, o), pl = __shfl_up_sync(0xffffffffu, bl, o);
                    if (lane >= o) add2f(bh, bl, ph, pl);
                }
                float ah = __shfl_up_sync(0xffffffffu, bh, 1), al = __shfl_up_sync(0xffffffffu, bl, 1);
                if (lane == 0) ah = al = 0.f;
                add2f(ah, al, xh, xl);             // and up to its first
                const float eh = __shfl_sync(0xffffffffu, bh, 31), el = __shfl_sync(0xffffffffu, bl, 31);
                float *gv = gslot(k);
                reinterpret_cast<float2 *>(gv)[lane] = make_float2(ah, bh);
                reinterpret_cast<float2 *>(gv + 64)[lane] = make_float2(al, bl);
                const uint2 wa = three_bf16(exp2f((eh - ah) + (el - al))), wb = three_bf16(exp2f((eh - bh) + (el - bl)));
                reinterpret_cast<uint4 *>(gv + 128)[lane] = make_uint4(wa.x, wa.y, wb.x, wb.y);
                reinterpret_cast<float2 *>(gv + 256)[lane] = make_float2(exp2f(ah + al), exp2f(bh + bl));
                if (lane == 0) gv[320] = exp2f(eh + el);
                if (!kFullPass) add2f(th, tl, eh, el);
                mbar_arrive(bar(kFull + s));
            }
            if (!kFullPass && lane == 0) s_decay[k0] = (double)th + (double)tl;
        }
    }
    __syncwarp();
    if (!ok) s_fail = 1;
    tc_fence_before();
    __syncthreads();
    if (s_fail) {
        // A bounded wait expired.  What is in flight lands first (each barrier it completes is given
        // a few milliseconds for both parities), then the part's results are marked.
        if (tid == 0) {
            for (int b = 0; b < kBars; ++b) {
                mbar_wait_small(bar(b), 0, 1u << 12);
                mbar_wait_small(bar(b), 1, 1u << 12);
            }
            atomicAdd(&g_kda_lin_timeouts, 1u);
        }
        const float nan = __int_as_float(0x7fc00000);
        float *to = kFullPass ? (s_piece[2] ? a.sT : nullptr) : locals;
        if (to) {
            to += (int64_t)s_piece[kFullPass ? 0 : 1] * a.dk * a.dv;
            for (int x = tid; x < a.dk * a.dv; x += NT) to[x] = nan;
        }
        if (kFullPass) {
            const int t1 = bos + (int64_t)c_hi * C < eos ? bos + c_hi * C : eos;
            for (int64_t x = tid; x < (int64_t)(t1 - first) * a.dv; x += NT)
                static_cast<__nv_bfloat16 *>(a.out)[((first + x / a.dv) * H + h) * a.dv + x % a.dv] = __float2bfloat16(nan);
        } else if (tid == 0) {
            decays[s_piece[1]] = 0.0;
        }
        __syncthreads();
    } else if (!kFullPass && tid == 0) {
        decays[s_piece[1]] = s_decay[0] + s_decay[1];
    }
    if (warp == 17) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, TM_COLS);
    }
    if (kFold) wait_ahead();   // (what this call's kernels read must not be overwritten by the next call's before)
}

// For each sequence that is cut: the state behind part p is e^{its decay} times the one before it plus
// the part's own from zero.  One CTA per slot, head and 1024 values; those of a sequence's first slot
// walk its parts.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(const LinArgs a, const CutRule cut, const Piece *plan, float *locals, const double *decays) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Piece piece = plan ? load_piece(plan + blockIdx.x) : dense_piece<false>(a, blockIdx.x, cut);
    if (piece.P == 0 || piece.p != 0) return;
    const int H = a.heads;
    const int64_t size = (int64_t)a.dk * a.dv, at = ((int64_t)blockIdx.y * kScanThreads + threadIdx.x) * 4;
    float4 s = a.s0 ? *reinterpret_cast<const float4 *>(a.s0 + ((int64_t)piece.n * H + piece.h) * size + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    auto part = [&](int p) { return (int64_t)(piece.slot + p) * H + piece.h; };
    auto state = [&](int p) { return reinterpret_cast<float4 *>(locals + part(p) * size + at); };
    constexpr int kAtOnce = 8;   // parts whose loads are in flight together
    for (int p0 = 0; p0 < piece.P - 1; p0 += kAtOnce) {
        float4 x[kAtOnce];
        double d[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (p0 + e < piece.P - 1) {
                x[e] = __ldcg(state(p0 + e));
                d[e] = __ldcg(decays + part(p0 + e));
            }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (p0 + e < piece.P - 1) {
                const float f = exp2f((float)d[e]);
                s = make_float4(fmaf(f, s.x, x[e].x), fmaf(f, s.y, x[e].y), fmaf(f, s.z, x[e].z), fmaf(f, s.w, x[e].w));
                *state(p0 + e) = s;
            }
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                   : nullptr;
    }();
    return fn;
}

// [tokens][H][d] bf16 as (d, H, tokens), 64 x 1 x 64 boxes, 128-byte swizzle.  The second box of a
// 64-wide head lies past the first dimension and lands as zeros, as do tokens past the end.
bool make_map(CUtensorMap *m, const void *ptr, int64_t tokens, int H, int d) {
    auto enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
    cuuint32_t box[3] = {64, 1, 64};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t take_lin_expiries(cudaStream_t st, unsigned int *count) {
    static const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_kda_lin_timeouts, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_kda_lin_timeouts, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e;
}

// How a call is cut, the CTAs of the two passes.  Cutting costs a first pass over K and V (half the time
// of the whole) of the parts but the last, so:
//  - of a dense batch's (sequence, head) units those that the last round of SMs has no full set of are cut
//    into as many parts as should end first (best_parts; T=8192: 160 units 336 us, whole 573; 70 units 229,
//    in two parts 264; 56 units of 13805 tokens 316, in two parts 364; 8 units of 32767 114 in 19);
//  - packed sequences, whose lengths only the device knows, run longest first, and those of more than
//    1.2 times an SM's equal share of all chunks are cut into parts of two thirds of it (15 mixes of lengths:
//    halves take between 9 % less and 14 % more time, thirds up to 29 % more; cutting from the whole share on
//    up to 26 % more).  Where one has four fifths of all chunks, that would make part of a second round: it is cut into
//    as many as one round holds (20000 of 21200 tokens, 16 heads: 148 us, 203 by two thirds).  One sequence
//    alone is cut as in a dense batch.
struct Cut {
    CutRule rule;
    int64_t pre, full;
};
constexpr int64_t kMinPart = 8;

// Parts, of at least kMinPart chunks, for `units` units of nc chunks each.  A CTA's time in tenths of a
// microsecond is about 22 a chunk and 70 once, in the first pass 11 and 60; the scan and the launches take 100.
static int64_t best_parts(int64_t units, int64_t nc) {
    auto rounds = [](int64_t ctas) { return (ctas + kSms - 1) / kSms; };
    int64_t parts = 1, best = rounds(units) * (22 * nc + 70);
    for (int64_t p = 2; p <= kMaxParts && p * kMinPart <= nc; ++p) {
        const int64_t per = (nc + p - 1) / p;
        const int64_t cost = rounds(units * p) * (22 * per + 70) + rounds(units * (p - 1)) * (11 * per + 60) + 100;
        if (cost < best) {
            best = cost;
            parts = p;
        }
    }
    const int64_t per = (nc + parts - 1) / parts;
    return (nc + per - 1) / per;
}

static Cut cut_of(int64_t tokens, int64_t num_seqs, int64_t heads, bool packed, bool whole) {
    const int64_t units = num_seqs * heads, chunks = ((packed ? tokens : tokens / num_seqs) + C - 1) / C;
    Cut c{{0x7fffffff, 1, 0, (int)units, 1, false, 0}, 0, units};
    if (whole) return c;
    if (!packed) {
        const int64_t cuts = units % kSms, kept = units - cuts, parts = cuts ? best_parts(cuts, chunks) : 1;
        if (parts == 1) return c;
        c.rule = {0, 1, (int)((num_seqs - kept / heads) * (parts - 1)), (int)kept, (int)parts, false, 0};
        c.pre = cuts * (parts - 1);
    } else if (num_seqs == 1) {
        const int64_t parts = best_parts(heads, chunks), target = (chunks + parts - 1) / parts;
        c.rule = {(int)target, (int)target, (int)(parts - 1), 0, 1, false, 0};
        c.pre = heads * (parts - 1);
    } else {
        const int64_t all = chunks + num_seqs, share = (all * heads + kSms - 1) / kSms;   // (each sequence's last chunk may be short)
        int64_t most = share + share / 5, target = share * 2 / 3;
        if (target < kMinPart) target = kMinPart;
        if (most < 2 * kMinPart) most = 2 * kMinPart;
        // at most all / (most + 1) sequences are cut, into ceil(nc / target) parts
        const int64_t slots = all <= most ? 0 : all / target;
        // one sequence with nearly all chunks: as many parts as one round of SMs holds
        const int64_t round = kSms / heads, alone = round >= 2 && (all + round - 1) / round >= target ? (all + round - 1) / round : 0;
        c.rule = {(int)most, (int)target, (int)slots, 0, 1, slots > 0, (int)alone};
        c.pre = slots * heads;
    }
    c.full = units + c.pre;
    return c;
}

// The workspace: the parts' states, their decays, and for packed sequences the two lists of pieces.
size_t lin_chunk_tc_workspace_bytes(int64_t tokens, int64_t num_seqs, int64_t heads, int dk, int dv, bool packed) {
    const Cut c = cut_of(tokens, num_seqs, heads, packed, false);
    return (size_t)c.rule.slots * heads * ((size_t)dk * dv * 4 + 8) + (packed ? (size_t)(c.pre + c.full) * sizeof(Piece) + 16 : 0);
}

cudaError_t launch_lin_chunk_tc(const LinArgs &a, void *workspace, bool whole, cudaStream_t st) {
    const int64_t tokens = a.cu ? a.seqlen : (int64_t)a.num_seqs * a.seqlen;
    const Cut c = cut_of(tokens, a.num_seqs, a.heads, a.cu != nullptr, whole);
    if (c.full > 0x7fffffffLL) return cudaErrorInvalidValue;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, a.q, tokens, a.qk_heads, a.dk) || !make_map(&mk, a.k, tokens, a.qk_heads, a.dk) ||
        !make_map(&mv, a.v, tokens, a.heads, a.dv))
        return cudaErrorInvalidValue;
    float *locals = static_cast<float *>(workspace);
    double *decays = reinterpret_cast<double *>(locals + (int64_t)c.rule.slots * a.heads * a.dk * a.dv);
    // Up to four kernels, each needing all of the one before (but see kFold): every one but the first may be
    // launched before that has ended and waits for it at its start, so that the launches overlap.
    bool first = true;
    auto launch = [&](auto kernel, dim3 grid, int threads, size_t smem, auto... args) {
        cudaError_t e = smem ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = at;
        cfg.numAttrs = first ? 0 : 1;
        first = false;
        return cudaLaunchKernelEx(&cfg, kernel, args...);
    };
    const bool wide = a.dk == 128;
    Piece *pre = nullptr, *full = nullptr;
    cudaError_t e = cudaSuccess;
    if (a.cu) {
        pre = reinterpret_cast<Piece *>((reinterpret_cast<uintptr_t>(decays + (int64_t)c.rule.slots * a.heads) + 15) & ~uintptr_t(15));
        full = pre + c.pre;
        e = launch(lin_plan_kernel, dim3(1), kPlanThreads, 0, a, c.rule, pre, (int)c.pre, full, (int)c.full);
    }
    const Piece *cpre = pre, *cfull = full;
    const double *cdecays = decays;
    if (e == cudaSuccess && c.pre > 0) {
        e = launch(wide ? kda_lin_chunk_tc_kernel<false, 128, false> : kda_lin_chunk_tc_kernel<false, 64, false>, dim3((unsigned)c.pre), NT, SMEM_BYTES,
                   mq, mk, mv, a, c.rule, cpre, locals, decays);
        if (e == cudaSuccess && !c.rule.fold)
            e = launch(lin_scan_kernel, dim3((unsigned)c.pre, (unsigned)(a.dk * a.dv / (4 * kScanThreads))), kScanThreads, 0,
                       a, c.rule, cpre, locals, cdecays);
    }
    if (e != cudaSuccess) return e;
    const auto whole_pass = c.rule.fold ? (wide ? kda_lin_chunk_tc_kernel<true, 128, true> : kda_lin_chunk_tc_kernel<true, 64, true>)
                                        : (wide ? kda_lin_chunk_tc_kernel<true, 128, false> : kda_lin_chunk_tc_kernel<true, 64, false>);
    return launch(whole_pass, dim3((unsigned)c.full), NT, SMEM_BYTES, mq, mk, mv, a, c.rule, cfull, locals, decays);
}

}  // namespace kda
