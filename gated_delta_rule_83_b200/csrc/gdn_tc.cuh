// gdn_tc.cuh -- tensor-core (tcgen05 / TMEM) kernels of the scalar-gate delta rule, bf16, dk = dv = 128.
//
// Chunk form, 64 tokens a chunk, g_i = sum_{m <= i} log alpha_m inside the chunk (log2 units), C = 64:
//     A_ij = beta_i 2^(g_i - g_j) k_i.k_j  (j < i)      X = (I + A)^-1
//     P_ij =        2^(g_i - g_j) q_i.k_j  (j <= i)
//     R_i = beta_i (v_i - 2^g_i S^T k_i)    U = X R      o_i = 2^g_i S^T q_i + (P U)_i
//     S <- 2^g_C S + sum_j 2^(g_C - g_j) k_j u_j^T
// Because the gate is one scalar a token it never enters a bf16 operand: k, q and v go to the tensor core
// as they came and the decays are applied in fp32 to its results, where every factor is <= 1 for
// log alpha <= 0.  No rescaling by a reference point is needed.
//
// Precision.  X, P, R, U and S are fp32; as tensor-core operands each is the sum of two bf16 parts
// (hi + lo, 16 significant bits) and a product takes hi.hi + hi.lo + lo.hi, one pass less where the
// other operand is an input.  Measured against 64 bits the states are off by 4..7e-6 where single bf16
// operands give 3e-3.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "prefill_tc.cuh"
#include "profile.cuh"
#include "tc_common.cuh"

namespace kda {
namespace gdn {

using namespace tc;

// ---- small helpers ---------------------------------------------------------------------------------
// One lane of a converged warp.  Inside this branch, with warp-uniform operands, the compiler issues an
// MMA in as few instructions as the tensor pipe takes to run it: 32 cycles for M = 128, N = 64 measured,
// against 50 in a branch on the thread index.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}
template <typename T> __device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// D[tmem] (+)= A[tmem] * B[smem desc]: A row i in lane i, two consecutive K elements a 32-bit column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// (a, b) as two packed bf16 pairs, hi + lo
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// 32 values -> 16 + 16 columns of an A operand
__device__ __forceinline__ void tmem_put_split32(uint32_t taddr, const float* x)
{
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) split2(x[2 * m], x[2 * m + 1], hi[m], lo[m]);
    tmem_st16u(taddr, hi);
    tmem_st16u(taddr + 16, lo);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* x)
{
    tmem_ld16(taddr, x);
    tmem_ld16(taddr + 16, x + 16);
    tmem_wait_ld();
}
// a whole warp waits; the answer is the same in every lane
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort)
{
    return __all_sync(0xffffffffu, mbar_wait_ab(bar, parity, abort));
}
// this warp's TMEM accesses are done -> one arrival on an mbarrier
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---- workspace slot of one (chunk, head) ---------------------------------------------------------------
// X and P as hi and lo 64 x 64 SW128 images, then fp32 rows of 64: 2^g, 2^(g_C - g), beta.
constexpr uint32_t kXhi = 0, kXlo = 8192, kPhi = 16384, kPlo = 24576, kScal = 32768;
constexpr uint32_t kSlot = kScal + 768;
constexpr int kGam = 0, kW = 64, kBeta = 128;  // float offsets in the scalar rows

// ----------------------------------------------------------------------------------------------------
// Per-chunk kernel: X, P and the scalar rows of each (chunk, head).
//
// One CTA of 256 threads a unit.  [k; q] k^T is one M = 128, N = 64 batch; its epilogue masks and decays
// the 128 x 64 result.  X comes from recursive doubling over 16 x 16 blocks in fp32 on CUDA cores: the
// product form's powers of A would lose the small entries, and the split images need X to 16 bits.
// Bound by the latency of that dependent chain, so CTAs are kept small (60 KB) to run three an SM.
// ----------------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr uint32_t kPrepA = 32768;                      // A / X fp32 [64][68]
constexpr uint32_t kPrepY = kPrepA + 64 * kAS * 4;      // scratch [32][36]
constexpr uint32_t kPrepMisc = kPrepY + 32 * 36 * 4;    // g, beta, barriers
constexpr uint32_t kPrepSmem = kPrepMisc + 1024 + 1024;

// (I + A)^-1 in place over a strictly lower 64 x 64 A (row stride kAS, zero on and above the diagonal)
__device__ __forceinline__ void invert_unit_lower(float* __restrict__ sA, float* __restrict__ sY)
{
    const int tid = threadIdx.x;
    {   // the four diagonal blocks: thread -> (block, column), forward substitution
        const int b = 16 * (tid >> 4), jj = tid & 15;
        float x[16];
        if (tid < 64) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float s = 0.f;
#pragma unroll
                for (int i4 = 0; i4 < r; i4 += 4) {
                    const float4 a4 = *reinterpret_cast<const float4*>(sA + (b + r) * kAS + b + i4);
                    const float av[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i4 + j < r) s = fmaf(av[j], x[i4 + j], s);
                }
                x[r] = (r == jj) ? 1.f : ((r < jj) ? 0.f : -s);
            }
        }
        __syncthreads();
        if (tid < 64) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sA[(b + r) * kAS + b + jj] = x[r];
        }
        __syncthreads();
    }
    {   // X_10 = -X_11 A_10 X_00 in each 32 x 32 half: thread -> (half, row, 4 columns)
        const int p = tid >> 6, ra = (tid >> 2) & 15, cc = (tid & 3) * 4;
        const int bi = 32 * p + 16, bj = 32 * p;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (tid < 128) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float a = sA[(bi + ra) * kAS + bj + k];
                const float4 x4 = *reinterpret_cast<const float4*>(sA + (bj + k) * kAS + bj + cc);
                y[0] = fmaf(a, x4.x, y[0]); y[1] = fmaf(a, x4.y, y[1]); y[2] = fmaf(a, x4.z, y[2]); y[3] = fmaf(a, x4.w, y[3]);
            }
            *reinterpret_cast<float4*>(sY + (p * 16 + ra) * 36 + cc) = make_float4(y[0], y[1], y[2], y[3]);
        }
        __syncthreads();
        if (tid < 128) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float a = sA[(bi + ra) * kAS + bi + k];
                const float4 y4 = *reinterpret_cast<const float4*>(sY + (p * 16 + k) * 36 + cc);
                x[0] = fmaf(a, y4.x, x[0]); x[1] = fmaf(a, y4.y, x[1]); x[2] = fmaf(a, y4.z, x[2]); x[3] = fmaf(a, y4.w, x[3]);
            }
            *reinterpret_cast<float4*>(sA + (bi + ra) * kAS + bj + cc) = make_float4(-x[0], -x[1], -x[2], -x[3]);
        }
        __syncthreads();
    }
    {   // the 32 x 32 block below the diagonal: thread -> (row, 4 columns)
        const int ra = tid >> 3, cc = (tid & 7) * 4;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float a = sA[(32 + ra) * kAS + k];
            const float4 x4 = *reinterpret_cast<const float4*>(sA + k * kAS + cc);
            y[0] = fmaf(a, x4.x, y[0]); y[1] = fmaf(a, x4.y, y[1]); y[2] = fmaf(a, x4.z, y[2]); y[3] = fmaf(a, x4.w, y[3]);
        }
        *reinterpret_cast<float4*>(sY + ra * 36 + cc) = make_float4(y[0], y[1], y[2], y[3]);
        __syncthreads();
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float a = sA[(32 + ra) * kAS + 32 + k];
            const float4 y4 = *reinterpret_cast<const float4*>(sY + k * 36 + cc);
            x[0] = fmaf(a, y4.x, x[0]); x[1] = fmaf(a, y4.y, x[1]); x[2] = fmaf(a, y4.z, x[2]); x[3] = fmaf(a, y4.w, x[3]);
        }
        *reinterpret_cast<float4*>(sA + (32 + ra) * kAS + cc) = make_float4(-x[0], -x[1], -x[2], -x[3]);
        __syncthreads();
    }
}

// g (log2 units, cumulative) and beta of a chunk's 64 tokens into shared memory, by one warp; tokens past
// the chunk's end carry no gate and no weight
__device__ __forceinline__ void load_scalars(const float* __restrict__ la, const float* __restrict__ beta, long long t0,
                                             int L, int H, int h, float* s_g, float* s_b)
{
    const int l = threadIdx.x & 31;
    float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
    if (2 * l < L) {
        a0 = la[(size_t)(t0 + 2 * l) * H + h] * kLog2e;
        b0 = beta[(size_t)(t0 + 2 * l) * H + h];
    }
    if (2 * l + 1 < L) {
        a1 = la[(size_t)(t0 + 2 * l + 1) * H + h] * kLog2e;
        b1 = beta[(size_t)(t0 + 2 * l + 1) * H + h];
    }
    float s = a0 + a1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, s, d);
        if (l >= d) s += y;
    }
    float before = __shfl_up_sync(0xffffffffu, s, 1);
    if (l == 0) before = 0.f;
    *reinterpret_cast<float2*>(s_g + 2 * l) = make_float2(before + a0, s);
    *reinterpret_cast<float2*>(s_b + 2 * l) = make_float2(b0, b1);
}

__device__ __forceinline__ void store_split8(uint8_t* hi, uint8_t* lo, uint32_t off, const float* x)
{
    uint4 h, l;
    split2(x[0], x[1], h.x, l.x);
    split2(x[2], x[3], h.y, l.y);
    split2(x[4], x[5], h.z, l.z);
    split2(x[6], x[7], h.w, l.w);
    *reinterpret_cast<uint4*>(hi + off) = h;
    *reinterpret_cast<uint4*>(lo + off) = l;
}

__global__ void __launch_bounds__(kPrepThreads)
gdn_prep_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const float* __restrict__ la, const float* __restrict__ beta, const WsHeader* __restrict__ hdr,
                const int* __restrict__ off, const int32_t* __restrict__ cu, int Tseq, int N, int H, int G,
                uint8_t* __restrict__ slots)
{
    extern __shared__ uint8_t smem_raw[];
    if (hdr->bad) return;
    if ((long long)blockIdx.x >= (long long)hdr->total_chunks * H) return;
    int h, n, L;
    long long t0;
    tc_unit(blockIdx.x, H, off, cu, Tseq, N, h, n, t0, L);
    uint8_t* sm = align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    float* sA = reinterpret_cast<float*>(sm + kPrepA);
    float* sY = reinterpret_cast<float*>(sm + kPrepY);
    float* s_g = reinterpret_cast<float*>(sm + kPrepMisc);
    float* s_b = s_g + 64;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kPrepMisc + 512);
    const uint32_t bar_in = sb + kPrepMisc + 528, bar_mma = bar_in + 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(bar_in, 1);
        mbar_init(bar_mma, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(bar_in, 32768);
        for (int a = 0; a < 2; ++a) {  // stacked [k; q]: atom columns of 128 rows
            tma_load_3d(sb + a * 16384, &tm_k, 64 * a, h / G, (int)t0, bar_in);
            tma_load_3d(sb + a * 16384 + 8192, &tm_q, 64 * a, h / G, (int)t0, bar_in);
        }
    }
    if (warp == 1) load_scalars(la, beta, t0, L, H, h, s_g, s_b);
    if (warp == 2) {
        tmem_alloc(smem_u32(s_tmem), 64);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(*s_tmem);
    bool ok = true;
    if (warp == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_in, 0));
        if (ok && elect_one()) {
            const uint64_t da = desc_kmajor(sb, 128, 0);
            const uint32_t id = idesc_bf16(128, 64, false, false);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint64_t d = da + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                mma_bf16(tmem, d, d, id, kk > 0);
            }
            mma_commit(bar_mma);
        }
        __syncwarp();
    }
    ok = __syncthreads_and(ok);
    ok = ok && mbar_wait(bar_mma, 0);
    fence_after_sync();
    // lanes 0..63: k_i.k_j, lanes 64..127: q_i.k_j; warps 0-3 columns 0..31, warps 4-7 columns 32..63
    const int wq = warp & 3, col0 = (warp >> 2) * 32, i = 32 * (wq & 1) + lane;
    uint8_t* img = sm;  // the [k; q] tile is consumed: the images take its place
    {
        float x[32];
        tmem_ld32(tmem + ((uint32_t)(32 * wq) << 16) + col0, x);
        const float gi = s_g[i], bi = s_b[i];
        const bool row = i < L, isA = wq < 2;
#pragma unroll
        for (int m = 0; m < 32; ++m) {
            const int j = col0 + m;
            // the select comes last: what lies past the chunk's end may be anything
            const float y = x[m] * ex2_approx(gi - s_g[j]);
            x[m] = (row && (isA ? j < i : j <= i)) ? y : 0.f;
        }
        if (isA) {
#pragma unroll
            for (int m = 0; m < 32; m += 4)
                *reinterpret_cast<float4*>(sA + i * kAS + col0 + m) =
                    make_float4(bi * x[m], bi * x[m + 1], bi * x[m + 2], bi * x[m + 3]);
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                store_split8(img + kPhi, img + kPlo, sw128_chunk_off(i, (col0 >> 3) + m, 64), x + 8 * m);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, 64);
    invert_unit_lower(sA, sY);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int e = tid + kPrepThreads * m, r = e >> 3, ch = e & 7;
        float x[8];
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(sA + r * kAS + 8 * ch);
        *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(sA + r * kAS + 8 * ch + 4);
        store_split8(img + kXhi, img + kXlo, sw128_chunk_off(r, ch, 64), x);
    }
    uint8_t* slot = slots + (size_t)blockIdx.x * kSlot;
    if (tid < 64) {
        float* sc = reinterpret_cast<float*>(slot + kScal);
        sc[kGam + tid] = ex2_approx(s_g[tid]);
        sc[kW + tid] = ex2_approx(s_g[63] - s_g[tid]);
        sc[kBeta + tid] = s_b[tid];
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == 0 && ok) {
        bulk_s2g(slot, sb, kScal);
        bulk_commit();
        bulk_wait_all();
    }
}

// ----------------------------------------------------------------------------------------------------
// Forward chain: one CTA a (sequence, head), chunks in order.
//
// The state is kept transposed, row = value column: every operand the chain itself produces (S, R, U)
// then is an A operand in TMEM that a thread writes from its own registers, and every input (k, q, X, P)
// is a B operand in shared memory as it was loaded.  Thread (warpgroup w, lane d) owns value column d:
// state channels 64 w .. 64 w + 63 and tokens 32 w .. 32 w + 31.
// Per chunk, M = 128:
//     D1 = S^T k^T     (N = 64, 16 MMAs)           R = beta (v - 2^g D1)
//     U  = R X^T       (N = 64, 9 MMAs + 3 narrow) U' = 2^(g_C - g) U
//     D3 = U' k        (N = 128, 8 MMAs)           S <- 2^g_C S + D3
//     Dq = S^T q^T (16), Po = U P^T (12)           o = 2^g Dq + Po, one chunk behind, off the chain
// TMEM columns: 0 D1 -> R -> U', 64 Dq, 128 U (accumulator, then operand), 192 Po, 256 S operand -> D3.
// Bound by the tensor pipe (about 2100 cycles a chunk) and three MMA round trips.
// ----------------------------------------------------------------------------------------------------
constexpr int kFThreads = 320;  // 8 compute warps, an MMA warp, a copy warp
constexpr uint32_t kFK = 0, kFV = 16384, kFQ = 32768, kFSlot = 49152;
constexpr uint32_t kFStage = kFSlot + 33792;  // the slot, padded to 1 KB
constexpr uint32_t kFMisc = 2 * kFStage;
constexpr uint32_t kFSmem = kFMisc + 256 + 1024;

// token rows L .. 63 of a 64 x 128 SW128 tile set to zero (256 threads)
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int L)
{
    for (int e = threadIdx.x; e < (64 - L) * 16; e += 256) {
        const int r = L + (e >> 4), ch = e & 15;
        *reinterpret_cast<uint4*>(tile + sw128_chunk_off(r, ch, 64)) = make_uint4(0, 0, 0, 0);
    }
}

__global__ void __launch_bounds__(kFThreads, 1)
gdn_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const float* S0, float* S_final,
                 __nv_bfloat16* __restrict__ out, const WsHeader* __restrict__ hdr, const int* __restrict__ off,
                 const int32_t* __restrict__ cu, int Tseq, int N, int H, int G, const uint8_t* __restrict__ slots)
{
    extern __shared__ uint8_t smem_raw[];
    if (hdr->bad) return;
    const int rank = blockIdx.x / H, h = blockIdx.x - rank * H, n = off[N + 1 + rank];
    const int jb = off[n], nch = off[n + 1] - jb;
    long long s0, s1;
    seq_bounds(n, cu, Tseq, s0, s1);
    uint8_t* sm = align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + kFMisc;
    const uint32_t bar_full = bars, bar_empty = bars + 16, bar_k = bars + 32, bar_u = bars + 40, bar_d = bars + 48,
                   bar_o = bars + 56, bar_s = bars + 64, bar_r = bars + 72, bar_u2 = bars + 80;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kFMisc + 96);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + kFMisc + 100);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 8);
        }
        mbar_init(bar_k, 1); mbar_init(bar_u, 1); mbar_init(bar_d, 1); mbar_init(bar_o, 1);
        mbar_init(bar_s, 8); mbar_init(bar_r, 8); mbar_init(bar_u2, 8);
        mbar_fence_init();
        *s_abort = 0;
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(*s_tmem);
    bool ok = true;

    if (warp == 9) {  // loads, two stages
        for (int it = 0; it < nch && ok; ++it) {
            const int s = it & 1;
            if (it >= 2) ok = warp_wait(bar_empty + 8 * s, (uint32_t)((it >> 1) - 1) & 1u, s_abort);
            if (ok && elect_one()) {
                const uint32_t st = sb + s * kFStage, f = bar_full + 8 * s;
                const int t = (int)(s0 + 64LL * it);
                mbar_arrive_expect_tx(f, 49152 + kSlot);
                for (int a = 0; a < 2; ++a) {
                    tma_load_3d(st + kFK + 8192 * a, &tm_k, 64 * a, h / G, t, f);
                    tma_load_3d(st + kFQ + 8192 * a, &tm_q, 64 * a, h / G, t, f);
                    tma_load_3d(st + kFV + 8192 * a, &tm_v, 64 * a, h, t, f);
                }
                bulk_g2s(st + kFSlot, slots + ((size_t)(jb + it) * H + h) * kSlot, kSlot, f);
            }
            __syncwarp();
        }
        for (int it = nch > 2 ? nch - 2 : 0; it < nch; ++it)  // no copy outlives the CTA, whatever gave up
            if (!ok) (void)mbar_wait(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u);
    } else if (warp == 8) {  // MMA issue
        const uint32_t id64 = idesc_bf16(128, 64, false, false), id32 = idesc_bf16(128, 32, false, false),
                       idd = idesc_bf16(128, 128, false, true);
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            const uint32_t st = sb + s * kFStage, par = (uint32_t)it & 1u;
            const uint64_t dk = desc_kmajor(st + kFK, 64, 0), dq = desc_kmajor(st + kFQ, 64, 0),
                           dkm = desc_mnmajor(st + kFK, 64, 0), dX = desc_kmajor(st + kFSlot, 64, 0);
            ok = ok && warp_wait(bar_full + 8 * s, (uint32_t)(it >> 1) & 1u, s_abort);
            ok = ok && warp_wait(bar_s, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {  // D1 = (S_hi + S_lo) k^T
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t a = tmem + 256 + 64 * (kk >> 2) + 8 * (kk & 3);
                    const uint64_t b = dk + (uint64_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4);
                    mma_ts(tmem, a, b, id64, kk > 0);
                    mma_ts(tmem, a + 32, b, id64, 1);
                }
                mma_commit(bar_k);
            }
            __syncwarp();
            if (it > 0) ok = ok && warp_wait(bar_empty + 8 * (s ^ 1), (uint32_t)((it - 1) >> 1) & 1u, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {  // Dq; the last chunk's has been read
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t a = tmem + 256 + 64 * (kk >> 2) + 8 * (kk & 3);
                    const uint64_t b = dq + (uint64_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4);
                    mma_ts(tmem + 64, a, b, id64, kk > 0);
                    mma_ts(tmem + 64, a + 32, b, id64, 1);
                }
            }
            __syncwarp();
            ok = ok && warp_wait(bar_r, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {  // U = R X^T; X is lower triangular: tokens 32..63 reach outputs 32..63 alone
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t a = tmem + 32 * (kk >> 1) + 8 * (kk & 1), d = tmem + 128 + (kk >> 1) * 32;
                    const uint64_t b = dX + (uint64_t)((kk * 32 + (kk >> 1) * 32 * 128) >> 4);
                    const uint32_t id = kk < 2 ? id64 : id32;
                    mma_ts(d, a, b, id, kk > 0);
                    mma_ts(d, a + 16, b, id, 1);
                    mma_ts(d, a, b + (kXlo >> 4), id, 1);
                }
                mma_commit(bar_u);
            }
            __syncwarp();
            ok = ok && warp_wait(bar_u2, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {  // D3 = U' k, over the state operand
                    const uint32_t a = tmem + 32 * (kk >> 1) + 8 * (kk & 1);
                    const uint64_t b = dkm + (uint64_t)((kk * 2048) >> 4);
                    mma_ts(tmem + 256, a, b, idd, kk > 0);
                    mma_ts(tmem + 256, a + 16, b, idd, 1);
                }
                mma_commit(bar_d);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {  // Po = U P^T
                    const uint32_t a = tmem + 128 + 32 * (kk >> 1) + 8 * (kk & 1), d = tmem + 192 + (kk >> 1) * 32;
                    const uint64_t b = dX + (uint64_t)((kPhi + kk * 32 + (kk >> 1) * 32 * 128) >> 4);
                    const uint32_t id = kk < 2 ? id64 : id32;
                    mma_ts(d, a, b, id, kk > 0);
                    mma_ts(d, a + 16, b, id, 1);
                    mma_ts(d, a, b + ((kPlo - kPhi) >> 4), id, 1);
                }
                mma_commit(bar_o);
            }
            __syncwarp();
        }
        if (nch > 0) (void)(ok && warp_wait(bar_o, (uint32_t)(nch - 1) & 1u, s_abort));
    } else {
        const int wg = warp >> 2, d = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const size_t srow = ((size_t)n * H + h) * 16384 + (size_t)wg * 64 * 128 + d;
        float S[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) S[c] = S0 ? S0[srow + (size_t)c * 128] : 0.f;
        auto put_state = [&]() {  // channels 64 w ..: 32 columns of hi, then 32 of lo
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int m = 0; m < 32; ++m) split2(S[2 * m], S[2 * m + 1], hi[m], lo[m]);
            tmem_st16u(tl + 256 + 64 * wg, hi);
            tmem_st16u(tl + 256 + 64 * wg + 16, hi + 16);
            tmem_st16u(tl + 256 + 64 * wg + 32, lo);
            tmem_st16u(tl + 256 + 64 * wg + 48, lo + 16);
            tmem_wait_st();
        };
        put_state();
        // o of chunk `it`: tokens 32 w .. 32 w + 31 of value column d
        auto write_out = [&](int it) {
            const int s = it & 1;
            const float* sc = reinterpret_cast<const float*>(sm + s * kFStage + kFSlot + kScal);
            ok = ok && mbar_wait_ab(bar_o, (uint32_t)it & 1u, s_abort);
            fence_after_sync();
            float x[32], y[32];
            tmem_ld16(tl + 64 + 32 * wg, x);
            tmem_ld16(tl + 64 + 32 * wg + 16, x + 16);
            tmem_ld16(tl + 192 + 32 * wg, y);
            tmem_ld16(tl + 192 + 32 * wg + 16, y + 16);
            tmem_wait_ld();
#pragma unroll
            for (int m = 0; m < 32; m += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(sc + kGam + 32 * wg + m);
                x[m] = fmaf(g4.x, x[m], y[m]);
                x[m + 1] = fmaf(g4.y, x[m + 1], y[m + 1]);
                x[m + 2] = fmaf(g4.z, x[m + 2], y[m + 2]);
                x[m + 3] = fmaf(g4.w, x[m + 3], y[m + 3]);
            }
            warp_arrive(bar_empty + 8 * s);  // stage, Dq and Po are free
            // neighbours exchange halves: the even lane stores columns (d, d + 1) of the even token
            const long long t = s0 + 64LL * it + 32 * wg;
            const int Lw = (int)(s1 - t < 32 ? s1 - t : 32);
            __nv_bfloat16* o = out + ((size_t)t * H + h) * 128 + (d & ~1);
            const bool odd = lane & 1;
#pragma unroll
            for (int m = 0; m < 32; m += 2) {
                const float give = odd ? x[m] : x[m + 1], keep = odd ? x[m + 1] : x[m];
                const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                const int tok = m + (odd ? 1 : 0);
                if (ok && tok < Lw)
                    *reinterpret_cast<uint32_t*>(o + (size_t)tok * H * 128) = odd ? pack_bf16(got, keep) : pack_bf16(keep, got);
            }
        };
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            const uint32_t par = (uint32_t)it & 1u;
            uint8_t* st = sm + s * kFStage;
            const float* sc = reinterpret_cast<const float*>(st + kFSlot + kScal);
            const int L = (int)(s1 - (s0 + 64LL * it) < 64 ? s1 - (s0 + 64LL * it) : 64);
            ok = ok && mbar_wait_ab(bar_full + 8 * s, (uint32_t)(it >> 1) & 1u, s_abort);
            if (L < 64) {  // rows past the sequence's end: another sequence's tokens
                if (ok) {
                    zero_tail_rows(st + kFK, L);
                    zero_tail_rows(st + kFQ, L);
                }
                fence_proxy_async();
            }
            warp_arrive(bar_s);
            if (it > 0) write_out(it - 1);
            float v[32];
            {
                const uint8_t* tv = st + kFV + (d >> 6) * 8192 + (d & 7) * 2;
#pragma unroll
                for (int m = 0; m < 32; ++m) {
                    const int j = 32 * wg + m;
                    v[m] = lds_bf16(tv + j * 128 + ((((d & 63) >> 3) ^ (j & 7)) << 4));
                }
            }
            float x[32];
            ok = ok && mbar_wait_ab(bar_k, par, s_abort);
            fence_after_sync();
            tmem_ld32(tl + 32 * wg, x);
#pragma unroll
            for (int m = 0; m < 32; m += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(sc + kGam + 32 * wg + m);
                const float4 b4 = *reinterpret_cast<const float4*>(sc + kBeta + 32 * wg + m);
                x[m] = b4.x * fmaf(-g4.x, x[m], v[m]);
                x[m + 1] = b4.y * fmaf(-g4.y, x[m + 1], v[m + 1]);
                x[m + 2] = b4.z * fmaf(-g4.z, x[m + 2], v[m + 2]);
                x[m + 3] = b4.w * fmaf(-g4.w, x[m + 3], v[m + 3]);
            }
            if (L < 64) {
#pragma unroll
                for (int m = 0; m < 32; ++m) x[m] = 32 * wg + m < L ? x[m] : 0.f;
            }
            tmem_put_split32(tl + 32 * wg, x);
            tmem_wait_st();
            warp_arrive(bar_r);
            const float last = sc[kGam + 63];
            ok = ok && mbar_wait_ab(bar_u, par, s_abort);
            fence_after_sync();
            tmem_ld32(tl + 128 + 32 * wg, x);
            tmem_put_split32(tl + 128 + 32 * wg, x);
#pragma unroll
            for (int m = 0; m < 32; m += 4) {
                const float4 w4 = *reinterpret_cast<const float4*>(sc + kW + 32 * wg + m);
                x[m] *= w4.x; x[m + 1] *= w4.y; x[m + 2] *= w4.z; x[m + 3] *= w4.w;
            }
            tmem_put_split32(tl + 32 * wg, x);
            tmem_wait_st();
            warp_arrive(bar_u2);
            ok = ok && mbar_wait_ab(bar_d, par, s_abort);
            fence_after_sync();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                tmem_ld32(tl + 256 + 64 * wg + c, x);
#pragma unroll
                for (int m = 0; m < 32; ++m) S[c + m] = fmaf(last, S[c + m], x[m]);
            }
            put_state();
        }
        if (nch > 0) write_out(nch - 1);
        if (S_final && ok) {
#pragma unroll
            for (int c = 0; c < 64; ++c) S_final[srow + (size_t)c * 128] = S[c];
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

inline size_t slots_bytes(long long units) { return (size_t)units * kSlot; }

inline cudaError_t launch_prep(const CUtensorMap& tq, const CUtensorMap& tk, const float* la, const float* beta,
                               const WsHeader* hdr, const int* off, const int32_t* cu, int Tseq, int N, int H, int Hk,
                               long long units, uint8_t* slots, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(gdn_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepSmem);
    if (e != cudaSuccess) return e;
    LaunchScope ls("gdn_prep", stream);
    gdn_prep_kernel<<<(unsigned)units, kPrepThreads, kPrepSmem, stream>>>(tq, tk, la, beta, hdr, off, cu, Tseq, N, H,
                                                                         H / Hk, slots);
    return cudaGetLastError();
}

inline cudaError_t launch_fwd(const void* q, const void* k, const void* v, const float* la, const float* beta,
                              const float* S0, float* S_final, void* out, const WsHeader* hdr, const int* off,
                              const int32_t* cu, int Tseq, int N, int H, int Hk, int max_chunks, long long Ttot,
                              uint8_t* slots, cudaStream_t stream)
{
    alignas(64) CUtensorMap tq{}, tk{}, tv{};
    const long long units = (long long)max_chunks * H;
    if (units > 0x7fffffffLL || (long long)N * H > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (Ttot > 0) {
        if (!make_token_map(&tq, q, true, Hk, Ttot, 64) || !make_token_map(&tk, k, true, Hk, Ttot, 64) ||
            !make_token_map(&tv, v, true, H, Ttot, 64))
            return cudaErrorInvalidValue;
        e = launch_prep(tq, tk, la, beta, hdr, off, cu, Tseq, N, H, Hk, units, slots, stream);
        if (e != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(gdn_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFSmem);
    if (e != cudaSuccess) return e;
    LaunchScope ls("gdn_chain", stream);
    gdn_chain_kernel<<<(unsigned)(N * H), kFThreads, kFSmem, stream>>>(tq, tk, tv, S0, S_final, (__nv_bfloat16*)out, hdr,
                                                                      off, cu, Tseq, N, H, H / Hk, slots);
    return cudaGetLastError();
}

}  // namespace gdn
}  // namespace kda
