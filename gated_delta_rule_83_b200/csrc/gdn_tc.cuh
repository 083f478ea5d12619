// gdn_tc.cuh -- tensor-core (tcgen05 / TMEM) kernels of the scalar-gate delta rule, bf16, dk and dv 64 or 128.
// Tiles are 128 wide; a width of 64 is padded with zeros by the tile loads (which fill what lies outside the
// tensor) and by masks where states and results enter and leave.
//
// Chunk form, 64 tokens a chunk, g_i = sum_{m <= i} log alpha_m inside the chunk (log2 units), C = 64:
//     A_ij = beta_i 2^(g_i - g_j) k_i.k_j  (j < i)      X = (I + A)^-1 diag(beta)
//     P_ij =        2^(g_i - g_j) q_i.k_j  (j <= i)     Y = P X
//     R_i = v_i - 2^g_i S^T k_i     U = X R      o_i = 2^g_i S^T q_i + (Y R)_i
//     S <- 2^g_C S + sum_j 2^(g_C - g_j) k_j u_j^T
// Y makes the output a product of what enters U as well, so that U is no operand of it.
// Because the gate is one scalar a token it never enters a bf16 operand: k, q and v go to the tensor core
// as they came and the decays are applied in fp32 to its results, where every factor is <= 1 for
// log alpha <= 0.  No rescaling by a reference point is needed.
//
// Precision.  X, P, Y, R, U and S are fp32; as tensor-core operands each is the sum of two bf16 parts
// (hi + lo, 16 significant bits) and a product takes hi.hi + hi.lo + lo.hi, one pass less where the
// other operand is an input.  Measured against 64 bits the states are off by 4..7e-6 where single bf16
// operands give 3e-3.  A third part would make 24 bits of them, for one and a half to two times the MMAs of a chain
// bound by their issue, and 576 TMEM columns where there are 512.  What is carried from chunk to chunk, S in the
// threads' registers, and what a product sums are fp32.
#pragma once

#include <cuda.h>

#include <cmath>

#include "common.cuh"
#include "head_gate.cuh"
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
// the dynamic shared memory from its first 1024-byte boundary on, still known to be shared memory: through a
// pointer cast from an integer every access would be a generic one
__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* raw) { return raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u); }
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
// pairs of fp32 values in one 64-bit register, for the two-wide FMA
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, 0xbf800000bf800000ull, a); }
// four consecutive floats of shared memory as two pairs
__device__ __forceinline__ void lds_pairs(uint32_t addr, f32x2& a, f32x2& b)
{
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
// a pair as two packed bf16 pairs, hi + lo
__device__ __forceinline__ void split2(f32x2 p, uint32_t& hi, uint32_t& lo)
{
    float a, b;
    unpair(p, a, b);
    hi = pack_bf16(a, b);
    unpair(sub2(p, pair(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u))), a, b);
    lo = pack_bf16(a, b);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) { split2(pair(a, b), hi, lo); }
// 32 values -> 16 + 16 columns of an A operand
__device__ __forceinline__ void tmem_put_split32(uint32_t taddr, const f32x2* x)
{
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) split2(x[m], hi[m], lo[m]);
    tmem_st16u(taddr, hi);
    tmem_st16u(taddr + 16, lo);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* x)
{
    tmem_ld16(taddr, x);
    tmem_ld16(taddr + 16, x + 16);
    tmem_wait_ld();
}
template <int REGS> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }
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
// 64 x 64 SW128 images X hi, X lo, Y hi, Y lo; then fp32 rows of 64: 2^g, 2^(g_C - g), beta, -2^g.
constexpr uint32_t kLo = 8192, kYofX = 16384, kScal = 32768;
constexpr uint32_t kSlot = kScal + 1024;
constexpr int kGam = 0, kW = 64, kBeta = 128, kNgam = 192;  // float offsets in the scalar rows
// The backward also takes P, (I + A)^-1 and 2^g q (64 x 128): hi and lo of each.
constexpr uint32_t kBwdP = 0, kBwdX = 16384, kBwdQ = 32768, kBwdSlot = 65536;
// ... and what the chains hand to the gradient kernel, per (chunk, head), hi and lo: the state before the chunk
// and its cotangent after it (128 value columns x 128 channels), U and dR (128 value columns x 64 tokens).
// Row d of these unswizzled images is value column d, 16-byte blocks of 8 columns 2 KB apart: a thread that
// owns row d stores whole blocks and a warp's store is one run of 512 bytes.
constexpr uint32_t kImgS = 0, kImgDs = 65536, kImgU = 131072, kImgDr = 163840, kImages = 196608;

// ----------------------------------------------------------------------------------------------------
// Per-chunk kernel: X, P and the scalar rows of each (chunk, head).
//
// One CTA of 256 threads a unit.  [k; q] k^T is one M = 128, N = 64 batch; its epilogue masks and decays
// the 128 x 64 result.  The inverse comes from recursive doubling over 8 x 8 blocks in fp32 on CUDA
// cores: the product form's powers of A would lose the small entries, and the split images need X to 16
// bits.  Y is a split M = 64 product.  Bound by that dependent chain's latency and its shared-memory accesses, so
// CTAs are kept small (57 KB, 64 registers) to run four an SM: A lies where Y will, over the consumed [k; q]
// tile.  32K tokens x 32 heads: 310 us (shared-memory pipe 70 % busy, issue slots 52 %, DRAM 23 %); 4 x 4 tiles
// in the last merge 313; larger tiles and three CTAs an SM cost 401 against 347 when that was changed.
// ----------------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr uint32_t kPrepP = kSlot;                      // P hi, lo; the slot takes the [k; q] tile's place
constexpr uint32_t kPrepA = kYofX;                      // A / inverse fp32 [64][68], to the slot's end
constexpr uint32_t kPrepY = kPrepP + 16384;             // scratch [32][36]
constexpr uint32_t kPrepMisc = kPrepY + 32 * 36 * 4;    // g, beta, barriers
constexpr uint32_t kPrepSmem = kPrepMisc + 1024 + 1024;
static_assert(kPrepA + 64 * kAS * 4 <= kSlot, "A fits behind X");

// rows b + K .., columns b .. of the inverse from the K x K blocks beside them, -X_11 (A_10 X_00): `t` numbers
// the 2 x 2 tiles of the block.  Small tiles: a chain of few loads, spread over the CTA.
template <int K>
__device__ __forceinline__ void merge_blocks(float* __restrict__ sA, float* __restrict__ sY, int t)
{
    constexpr int kTiles = (K / 2) * (K / 2);
    const bool active = t < 64 / (2 * K) * kTiles;
    const int b = 2 * K * (t / kTiles), r = 2 * (t % kTiles / (K / 2)), c = 2 * (t % (K / 2));
    float* y = sY + (b >> 1) * 36;  // K rows a pair
    auto product = [&](const float* P, int ps, const float* Q, int qs, float (&d)[2][2]) {
        d[0][0] = d[0][1] = d[1][0] = d[1][1] = 0.f;
#pragma unroll
        for (int k = 0; k < K; k += 4) {
            const float4 p0 = *reinterpret_cast<const float4*>(P + k), p1 = *reinterpret_cast<const float4*>(P + ps + k);
            const float a0[4] = {p0.x, p0.y, p0.z, p0.w}, a1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 q = *reinterpret_cast<const float2*>(Q + (k + e) * qs);
                d[0][0] = fmaf(a0[e], q.x, d[0][0]); d[0][1] = fmaf(a0[e], q.y, d[0][1]);
                d[1][0] = fmaf(a1[e], q.x, d[1][0]); d[1][1] = fmaf(a1[e], q.y, d[1][1]);
            }
        }
    };
    float d[2][2];
    if (active) {
        product(sA + (b + K + r) * kAS + b, kAS, sA + b * kAS + b + c, kAS, d);
        *reinterpret_cast<float2*>(y + r * 36 + c) = make_float2(d[0][0], d[0][1]);
        *reinterpret_cast<float2*>(y + (r + 1) * 36 + c) = make_float2(d[1][0], d[1][1]);
    }
    __syncthreads();
    if (active) {
        product(sA + (b + K + r) * kAS + b + K, kAS, y + c, 36, d);
        *reinterpret_cast<float2*>(sA + (b + K + r) * kAS + b + c) = make_float2(-d[0][0], -d[0][1]);
        *reinterpret_cast<float2*>(sA + (b + K + r + 1) * kAS + b + c) = make_float2(-d[1][0], -d[1][1]);
    }
    __syncthreads();
}

// (I + A)^-1 in place over a strictly lower 64 x 64 A (row stride kAS, zero on and above the diagonal)
__device__ __forceinline__ void invert_unit_lower(float* __restrict__ sA, float* __restrict__ sY)
{
    const int tid = threadIdx.x;
    {   // the eight 8 x 8 diagonal blocks: thread -> (block, column), forward substitution
        const int b = 8 * (tid >> 3), jj = tid & 7;
        float x[8];
        if (tid < 64) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float4 p = *reinterpret_cast<const float4*>(sA + (b + r) * kAS + b);
                const float4 q = *reinterpret_cast<const float4*>(sA + (b + r) * kAS + b + 4);
                const float av[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < r; ++i) s = fmaf(av[i], x[i], s);
                x[r] = (r == jj) ? 1.f : ((r < jj) ? 0.f : -s);
            }
        }
        __syncthreads();
        if (tid < 64) {
#pragma unroll
            for (int r = 0; r < 8; ++r) sA[(b + r) * kAS + b + jj] = x[r];
        }
        __syncthreads();
    }
    merge_blocks<8>(sA, sY, tid);
    merge_blocks<16>(sA, sY, tid);
    merge_blocks<32>(sA, sY, tid);
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

template <bool BWD>
__global__ void __launch_bounds__(kPrepThreads, 4)
gdn_prep_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const float* __restrict__ la, const float* __restrict__ beta, const WsHeader* __restrict__ hdr,
                const int* __restrict__ off, const int32_t* __restrict__ cu, int Tseq, int N, int H, int G,
                uint8_t* __restrict__ slots, uint8_t* __restrict__ bslots)
{
    extern __shared__ uint8_t smem_raw[];
    if (cu && (hdr->bad || (long long)blockIdx.x >= (long long)hdr->total_chunks * H)) return;
    int h, n, L;
    long long t0;
    tc_unit(blockIdx.x, H, off, cu, Tseq, N, h, n, t0, L);
    uint8_t* sm = aligned_smem(smem_raw);
    const uint32_t sb = smem_u32(sm);
    float* sA = reinterpret_cast<float*>(sm + kPrepA);
    float* sY = reinterpret_cast<float*>(sm + kPrepY);
    float* s_g = reinterpret_cast<float*>(sm + kPrepMisc);
    float* s_b = s_g + 64;
    float* s_gl = s_g + 128;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kPrepMisc + 768);
    const uint32_t bar_in = sb + kPrepMisc + 784, bar_mma = bar_in + 8;
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
    if (warp == 1) load_scalars(la, beta, t0, L, H, h, s_g, s_gl, s_b);
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
    if (!ok && warp == 0) (void)mbar_wait(bar_in, 0);  // no copy outlives the CTA
    ok = ok && mbar_wait(bar_mma, 0);
    fence_after_sync();
    if (BWD) {  // 2^g q, before A takes the tile's place
        uint8_t* bq = bslots + (size_t)blockIdx.x * kBwdSlot + kBwdQ;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int e = tid + kPrepThreads * m, r = e >> 4, ch = e & 15;
            const float gam = ex2_approx(s_g[r]);
            float x[8];
            unpack8(*reinterpret_cast<const uint4*>(sm + sw128_chunk_off(64 + r, ch, 128)), x);
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = r < L ? gam * x[c] : 0.f;
            store_split8(bq, bq + 16384, sw128_chunk_off(r, ch, 64), x);
        }
        __syncthreads();
    }
    // lanes 0..63: k_i.k_j, lanes 64..127: q_i.k_j; warps 0-3 columns 0..31, warps 4-7 columns 32..63
    const int wq = warp & 3, col0 = (warp >> 2) * 32, i = 32 * (wq & 1) + lane;
    uint8_t* img = sm;  // the [k; q] tile is consumed: the images take its place
    {
        float x[32];
        tmem_ld32(tmem + ((uint32_t)(32 * wq) << 16) + col0, x);
        const float gi = s_g[i], gli = s_gl[i], bi = s_b[i];
        const bool row = i < L, isA = wq < 2, above = col0 > 32 * (wq & 1);  // above the diagonal: zero
#pragma unroll
        for (int m = 0; m < 32; m += 4) {
            if (above) {
                x[m] = x[m + 1] = x[m + 2] = x[m + 3] = 0.f;
                continue;
            }
            const float4 g4 = *reinterpret_cast<const float4*>(s_g + col0 + m);
            const float4 l4 = *reinterpret_cast<const float4*>(s_gl + col0 + m);
            const float gj[4] = {g4.x, g4.y, g4.z, g4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = col0 + m + e;
                // the select comes last: what lies past the chunk's end may be anything
                const float y = x[m + e] * ex2_approx((gi - gj[e]) + (gli - lj[e]));
                x[m + e] = (row && (isA ? j < i : j <= i)) ? y : 0.f;
            }
        }
        if (isA) {
#pragma unroll
            for (int m = 0; m < 32; m += 4)
                *reinterpret_cast<float4*>(sA + i * kAS + col0 + m) =
                    make_float4(bi * x[m], bi * x[m + 1], bi * x[m + 2], bi * x[m + 3]);
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                store_split8(sm + kPrepP, sm + kPrepP + 8192, sw128_chunk_off(i, (col0 >> 3) + m, 64), x + 8 * m);
        }
    }
    fence_before_sync();
    __syncthreads();
    invert_unit_lower(sA, sY);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int e = tid + kPrepThreads * m, r = e >> 3, ch = e & 7;
        float x[8];
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(sA + r * kAS + 8 * ch);
        *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(sA + r * kAS + 8 * ch + 4);
        if (BWD) {
            uint8_t* bx = bslots + (size_t)blockIdx.x * kBwdSlot + kBwdX;
            store_split8(bx, bx + 8192, sw128_chunk_off(r, ch, 64), x);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] *= s_b[8 * ch + c];
        store_split8(img, img + kLo, sw128_chunk_off(r, ch, 64), x);
    }
    fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    if (tid < 64) {  // over A's end
        float* sc = reinterpret_cast<float*>(img + kScal);
        const float gam = ex2_approx(s_g[tid]);
        sc[kGam + tid] = gam;
        sc[kW + tid] = ex2_approx((s_g[63] - s_g[tid]) + (s_gl[63] - s_gl[tid]));
        sc[kBeta + tid] = s_b[tid];
        sc[kNgam + tid] = -gam;
    }
    if (warp == 0) {
        fence_after_sync();
        if (elect_one()) {  // Y = P X
            const uint64_t dp = desc_kmajor(sb + kPrepP, 64, 0), dx = desc_mnmajor(sb, 64, 0);
            const uint32_t id = idesc_bf16(64, 64, false, true);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint64_t a = dp + (uint64_t)((kk * 32) >> 4), b = dx + (uint64_t)((kk * 2048) >> 4);
                mma_bf16(tmem, a, b, id, kk > 0);
                mma_bf16(tmem, a + (8192 >> 4), b, id, 1);
                mma_bf16(tmem, a, b + (kLo >> 4), id, 1);
            }
            mma_commit(bar_mma);
            if (BWD) bulk_s2g(bslots + (size_t)blockIdx.x * kBwdSlot + kBwdP, sb + kPrepP, 16384);
        }
        __syncwarp();
    }
    ok = ok && mbar_wait(bar_mma, 1);
    fence_after_sync();
    {   // M = 64: row 16 (warp % 4) + lane % 16; the upper half-warp is 32 columns further
        float x[16];
        tmem_ld16_pair<32>(tmem + ((uint32_t)(32 * wq) << 16) + 16 * (warp >> 2), x);
        tmem_wait_ld();
        const int r = 16 * wq + (lane & 15), ch = 4 * (lane >> 4) + 2 * (warp >> 2);
        store_split8(img + kYofX, img + kYofX + kLo, sw128_chunk_off(r, ch, 64), x);
        store_split8(img + kYofX, img + kYofX + kLo, sw128_chunk_off(r, ch + 1, 64), x + 8);
    }
    fence_proxy_async();
    fence_before_sync();
    ok = __syncthreads_and(ok);
    if (warp == 0 && elect_one()) {
        if (ok) bulk_s2g(slots + (size_t)blockIdx.x * kSlot, sb, kSlot);
        bulk_commit();
        bulk_wait_all();
    }
    if (warp == 2) tmem_dealloc(tmem, 64);
}

// ----------------------------------------------------------------------------------------------------
// Forward chain: one CTA a (sequence, head), chunks in order.
//
// The state is kept transposed, row = value column: every operand the chain itself produces (S, R, U)
// then is an A operand in TMEM that a thread writes from its own registers, and every input (k, q, X, P)
// is a B operand in shared memory as it was loaded.  Compute thread (warpgroup w, lane d) owns value
// column d: state channels 64 w .. 64 w + 63 and tokens 32 w .. 32 w + 31.
// Per chunk, M = 128:
//     D1 = S^T k^T          (N = 64, 16 MMAs)        R' = -2^g D1
//     U  = v^T X^T + R' X^T (8 with Y's, 18 narrow)  U' = 2^(g_C - g) U
//     D3 = U' k             (N = 128, 8 MMAs)        S <- 2^g_C S + D3
//     Dq = S^T q^T (16), Po = R' Y^T + v^T Y^T (20)  o = 2^g Dq + Po by four warps of their own
// X and Y are lower triangular, so tokens 32..63 are no operand of outputs 0..31.  The two warpgroups run
// staggered: each has its own barriers, and the MMAs a warpgroup waits for are committed apart from the
// other's, so that one's conversions run under the other's MMAs.  v enters as an operand, never through
// registers.  What no thread waits for fills the tensor pipe's gaps: Dq under the making of R', R' Y^T under
// that of U', v^T Y^T and the next chunk's v^T X^T under the state's update.
// Bound by the round trips of the chain: 2.5 us a chunk with one CTA an SM (171 chunks of 96 CTAs 427 us, 32
// heads of 32K tokens in three segments), in which some 80 MMAs take one warp about 42 cycles each to issue and each of the
// six hand-overs between MMA and conversions costs about 140 cycles.  Measured and not taken: a second issuing
// warp (401 us there, but 340..355 against 323 for 8192 tokens x 16 heads, and spills in the backward's), four
// conversion warpgroups, the next chunk's D1 from the Gram matrix of the keys (one hand-over less; 24 warps'
// code leaves the instruction cache, 2.5 us).  ptxas spills 28 bytes of a thread here and 84 without outputs.
// TMEM columns: 0 D1 -> R', 64 Dq, 128 U, 192 Po, 256 S operand -> D3, 384 U'.
// ----------------------------------------------------------------------------------------------------
constexpr int kChainOut = 0;     // the prefill: writes out and S_final
constexpr int kChainStates = 1;  // the backward's recompute: writes each chunk's start state and U
constexpr int kChainEnds = 2;    // a segment's end state and transition, see below

// Segments.  With few (sequence, head) pairs the chunks' chain would leave most SMs idle, so a sequence is cut
// into segments of `len` chunks.  Over a segment the state maps affinely, S_end = M S_start + F: one CTA
// runs the chain from a zero state (F; the first segment's from S0), another from the identity without v
// (M, whose 128 columns take the place of the value columns); a small kernel then chains the segments
// (F'_g = M_g F'_{g-1} + F_g is the start state of segment g + 1) and the real pass runs all segments at once.
// The reverse chain's transition is M's transpose.  Segments of all sequences are numbered in order; every
// sequence has at least one.
struct Segments {
    int len;          // chunks a segment; 0: one segment a sequence, longest sequences first
    float* F;         // [segment][H][128][128]: end states, then start states of the segment after
    float* M;         // [segment][H][128][128]
};

// a state in global memory: [dk][dv] of the caller, or 128 x 128 of the workspace
struct StateRef {
    float* p;
    int stride, rows, cols;
};
// channels 64 wg .. + 63 of value column d, as pairs
__device__ __forceinline__ void load_state(const StateRef& s, int wg, int d, f32x2 (&S)[32])
{
    const bool in = s.p && d < s.cols && 64 * wg < s.rows;
    const float* p = s.p + (size_t)(64 * wg) * s.stride + d;
#pragma unroll
    for (int c = 0; c < 32; ++c)
        S[c] = in ? pair(p[(size_t)(2 * c) * s.stride], p[(size_t)(2 * c + 1) * s.stride]) : 0ull;
}
__device__ __forceinline__ void store_state(const StateRef& s, int wg, int d, const f32x2 (&S)[32])
{
    if (!s.p || d >= s.cols || 64 * wg >= s.rows) return;
    float* p = s.p + (size_t)(64 * wg) * s.stride + d;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        float a, b;
        unpair(S[c], a, b);
        p[(size_t)(2 * c) * s.stride] = a;
        p[(size_t)(2 * c + 1) * s.stride] = b;
    }
}

// chunks of the sequences before n; only packed input has a table
__device__ __forceinline__ int chunks_before(const int* __restrict__ off, const int32_t* cu, int Tseq, int n)
{
    return cu ? off[n] : n * ((Tseq + kChunk - 1) / kChunk);
}

// segment idx -> its sequence, number and the sequence's count; false past the last one (whole warps)
__device__ __forceinline__ bool find_segment(int idx, const int* __restrict__ off, const int32_t* cu, int Tseq, int N,
                                             const Segments& sg, int& n, int& seg, int& nseg)
{
    if (sg.len == 0) {
        n = cu ? off[N + 1 + idx] : idx;
        seg = 0;
        nseg = 1;
        return true;
    }
    if (!cu) {
        nseg = max(1, (chunks_before(off, cu, Tseq, 1) + sg.len - 1) / sg.len);
        n = idx / nseg;
        seg = idx - n * nseg;
        return n < N;
    }
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int n0 = 0; n0 < N; n0 += 32) {
        const int m = n0 + lane;
        const int cnt = m < N ? max(1, (off[m + 1] - off[m] + sg.len - 1) / sg.len) : 0;
        int inc = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, idx < base + inc);
        if (hit) {
            const int f = __ffs(hit) - 1;
            n = n0 + f;
            nseg = __shfl_sync(0xffffffffu, cnt, f);
            seg = idx - base - __shfl_sync(0xffffffffu, inc - cnt, f);
            return true;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

constexpr uint32_t kTmD1 = 0, kTmDq = 64, kTmU = 128, kTmPo = 192, kTmS = 256, kTmUw = 384;

template <int MODE> struct Chain {
    // 8 compute warps, [4 output warps], MMA, copies [, 2 idle: registers are shared out by warpgroup]
    static constexpr int kThreads = MODE == kChainOut ? 512 : 320;
    static constexpr int kMmaWarp = MODE == kChainOut ? 12 : 8;
    static constexpr uint32_t K = 0, V = 16384, Slot = 32768;  // (without outputs: X hi, X lo, scalars)
    static constexpr uint32_t Scal = Slot + (MODE == kChainOut ? kScal : 16384u);
    static constexpr uint32_t Q = Scal + 1024;                 // kChainOut
    static constexpr uint32_t Stage = MODE == kChainOut ? Q + 16384 : Scal + 1024;
    static constexpr uint32_t Misc = 2 * Stage;
    static constexpr uint32_t Smem = Misc + 512 + 2048 + 1024;
};

// NB 16-byte blocks of row d, from block b0 on, of an unswizzled image and of its lo image behind it
template <int NB>
__device__ __forceinline__ void store_blocks(uint8_t* img, uint32_t lo_off, int b0, int d, const uint32_t* hi,
                                             const uint32_t* lo)
{
    uint8_t* p = img + (size_t)b0 * 2048 + d * 16;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        *reinterpret_cast<uint4*>(p + i * 2048) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        *reinterpret_cast<uint4*>(p + lo_off + i * 2048) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
    }
}

// token rows L .. 63 of one 64-channel atom column set to zero by a warpgroup
__device__ __forceinline__ void zero_tail_rows(uint8_t* atom, int L)
{
    for (int e = threadIdx.x & 127; e < (64 - L) * 8; e += 128)
        *reinterpret_cast<uint4*>(atom + (L + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
}

// what the chains of a call share
struct ChainArgs {
    const WsHeader* hdr;
    const int* off;
    const int32_t* cu;
    int Tseq, N, H, G, dk, dv;
    const uint8_t* slots;
};

// chain `block` (segment * H + head); trans: kChainEnds from the identity, without v
template <int MODE>
__device__ __forceinline__ void chain_body(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                           const float* S0, float* S_final, __nv_bfloat16* __restrict__ out,
                                           const ChainArgs& ca, uint8_t* __restrict__ images, const Segments& sg, int block,
                                           bool trans)
{
    const int* __restrict__ off = ca.off;
    const int32_t* __restrict__ cu = ca.cu;
    const int Tseq = ca.Tseq, N = ca.N, H = ca.H, G = ca.G, dkw = ca.dk, dvw = ca.dv;
    const uint8_t* __restrict__ slots = ca.slots;
    using C = Chain<MODE>;
    constexpr bool kOut = MODE == kChainOut;
    extern __shared__ uint8_t smem_raw[];
    if (cu && ca.hdr->bad) return;
    const int sidx = block / H, h = block - sidx * H;
    int n, seg, nseg;
    if (!find_segment(sidx, off, cu, Tseq, N, sg, n, seg, nseg)) return;
    const size_t mine = ((size_t)n * H + h) * dkw * dvw, part = ((size_t)sidx * H + h) * 16384;
    if (MODE == kChainEnds && (seg == nseg - 1 || (trans && seg == 0))) {
        // Nothing starts from the last segment's end, and the first one's start is known.  The last one's place
        // keeps S0 instead: S_final may be S0, and the CTA that writes it is not the one that starts from it.
        if (!trans && S0)
            for (int e = threadIdx.x; e < dkw * dvw; e += Chain<MODE>::kThreads) sg.F[part + e] = S0[mine + e];
        return;
    }
    const int jb = chunks_before(off, cu, Tseq, n) + seg * sg.len, left = chunks_before(off, cu, Tseq, n + 1) - jb, nch = seg == nseg - 1 ? left : sg.len;
    long long s0, s1;
    seq_bounds(n, cu, Tseq, s0, s1);
    s0 += 64LL * seg * sg.len;
    float* s0p = !S0 ? nullptr
                 : MODE == kChainEnds || nseg == 1 ? const_cast<float*>(S0) + mine
                                                   : sg.F + ((size_t)(sidx + nseg - 1) * H + h) * 16384;
    const StateRef start = seg == 0 ? StateRef{s0p, dvw, dkw, dvw}
                                    : StateRef{MODE == kChainEnds ? nullptr : sg.F + part - (size_t)H * 16384, 128, 128, 128};
    const StateRef end = MODE == kChainEnds ? StateRef{(trans ? sg.M : sg.F) + part, 128, 128, 128}
                                            : StateRef{S_final && seg == nseg - 1 ? S_final + mine : nullptr, dvw, dkw, dvw};
    uint8_t* sm = aligned_smem(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + C::Misc;
    const uint32_t bar_full = bars, bar_empty = bars + 16, bar_k = bars + 32, bar_u = bars + 48, bar_d = bars + 64,
                   bar_s = bars + 80, bar_r = bars + 96, bar_w = bars + 112, bar_o = bars + 128, bar_q = bars + 136,
                   bar_z = bars + 144;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + C::Misc + 160);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + C::Misc + 164);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, kOut ? 13 : 9);  // readers' warps and the last MMAs
            mbar_init(bar_k + 8 * s, 1);
            mbar_init(bar_u + 8 * s, 1);
            mbar_init(bar_d + 8 * s, 1);
            mbar_init(bar_s + 8 * s, 4);
            mbar_init(bar_r + 8 * s, 4);
            mbar_init(bar_w + 8 * s, 4);
        }
        mbar_init(bar_o, 1);
        mbar_init(bar_q, 4);
        mbar_init(bar_z, 8);
        mbar_fence_init();
        *s_abort = 0;
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(*s_tmem);
    bool ok = true;

    // 512 threads x 128 registers at launch = 2 x 128 x 176 + 128 x 96 + 128 x 64
    if (kOut && warp >= 12) regs_dec<64>();
    if (warp == C::kMmaWarp + 1) {  // loads, two stages
        int issued = 0;
        for (int it = 0; it < nch && ok; ++it) {
            const int s = it & 1;
            if (it >= 2) ok = warp_wait(bar_empty + 8 * s, (uint32_t)((it >> 1) - 1) & 1u, s_abort);
            if (ok && elect_one()) {
                const uint32_t st = sb + s * C::Stage, f = bar_full + 8 * s;
                const int t = (int)(s0 + 64LL * it);
                const uint8_t* slot = slots + ((size_t)(jb + it) * H + h) * kSlot;
                mbar_arrive_expect_tx(f, kOut ? 49152 + kSlot : 32768 + 16384 + 1024);
                for (int a = 0; a < 2; ++a) {
                    tma_load_3d(st + C::K + 8192 * a, tm_k, 64 * a, h / G, t, f);
                    if (kOut) tma_load_3d(st + C::Q + 8192 * a, tm_q, 64 * a, h / G, t, f);
                    tma_load_3d(st + C::V + 8192 * a, tm_v, 64 * a, h, t, f);
                }
                if (kOut) {
                    bulk_g2s(st + C::Slot, slot, kSlot, f);
                } else {
                    bulk_g2s(st + C::Slot, slot, 16384, f);
                    bulk_g2s(st + C::Scal, slot + kScal, 1024, f);
                }
            }
            __syncwarp();
            issued = ok ? it + 1 : issued;
        }
        for (int it = issued > 2 ? issued - 2 : 0; it < issued; ++it)  // no copy outlives the CTA, whatever gave up
            (void)mbar_wait(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u);
    } else if (warp == C::kMmaWarp) {
        const uint32_t id128m = idesc_bf16(128, 128, false, true), id64 = idesc_bf16(128, 64, false, false),
                       id32 = idesc_bf16(128, 32, false, false), id64m = idesc_bf16(128, 64, false, true),
                       idv = idesc_bf16(128, 64, true, false);
        auto v_times = [&](uint32_t d, uint64_t dv, uint64_t b, uint32_t first) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint64_t a = dv + (uint64_t)((kk * 2048) >> 4), bb = b + (uint64_t)((kk * 32) >> 4);
                mma_bf16(d, a, bb, idv, kk > 0 || !first);
                mma_bf16(d, a, bb + (kLo >> 4), idv, 1);
            }
        };
        // U = v^T X^T of chunk `it`, into the accumulator that the chunk before has been read from
        auto issue_v = [&](int it) {
            const uint32_t st = sb + (it & 1) * C::Stage;
            ok = ok && warp_wait(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u, s_abort);
            ok = ok && warp_wait(bar_z, (uint32_t)it & 1u, s_abort);
            fence_after_sync();
            if (!trans && ok && elect_one()) v_times(tmem + kTmU, desc_mnmajor(st + C::V, 64, 0), desc_kmajor(st + C::Slot, 64, 0), 1);
            __syncwarp();
        };
        if (nch > 0) issue_v(0);
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            const uint32_t st = sb + s * C::Stage, par = (uint32_t)it & 1u;
            const uint64_t dk = desc_kmajor(st + C::K, 64, 0), dq = desc_kmajor(st + C::Q, 64, 0),
                           dkm = desc_mnmajor(st + C::K, 64, 0), dX = desc_kmajor(st + C::Slot, 64, 0),
                           dY = dX + (uint64_t)(kYofX >> 4);
            // S operand: channels 64 a .. of warpgroup a, hi at column 64 a, lo 32 further
            auto state_times = [&](uint32_t d, uint64_t b, int a, uint32_t id, uint32_t first) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t x = tmem + kTmS + 64 * a + 8 * kk;
                    const uint64_t bb = b + (uint64_t)((a * 8192 + kk * 32) >> 4);
                    mma_ts(d, x, bb, id, kk > 0 || !first);
                    mma_ts(d, x + 32, bb, id, 1);
                }
            };
            // R' (two k steps of warpgroup a) times rows of a split image
            auto r_times = [&](uint32_t d, uint64_t b, int a, uint32_t id, uint32_t first) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const uint32_t x = tmem + kTmD1 + 32 * a + 8 * kk;
                    const uint64_t bb = b + (uint64_t)((a * 64 + kk * 32) >> 4);
                    mma_ts(d, x, bb, id, kk > 0 || !first);
                    mma_ts(d, x + 16, bb, id, 1);
                    mma_ts(d, x, bb + (kLo >> 4), id, 1);
                }
            };
            ok = ok && warp_wait(bar_s, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) state_times(tmem + kTmD1, dk, 0, id64, 1);
            __syncwarp();
            ok = ok && warp_wait(bar_s + 8, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
                state_times(tmem + kTmD1, dk, 1, id32, 0);
                mma_commit(bar_k);
                state_times(tmem + kTmD1 + 32, dk + (uint64_t)(4096 >> 4), 1, id32, 0);
                mma_commit(bar_k + 8);
            }
            __syncwarp();
            if (kOut) {
                if (it > 0) ok = ok && warp_wait(bar_q, par ^ 1u, s_abort);  // the last chunk's Dq and Po are read
                fence_after_sync();
                if (ok && elect_one()) {
                    state_times(tmem + kTmDq, dq, 0, id64, 1);
                    state_times(tmem + kTmDq, dq, 1, id64, 0);
                }
                __syncwarp();
            }
            ok = ok && warp_wait(bar_r, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
                r_times(tmem + kTmU, dX, 0, id32, trans);
                mma_commit(bar_u);
                r_times(tmem + kTmU + 32, dX + (uint64_t)(4096 >> 4), 0, id32, trans);
            }
            __syncwarp();
            ok = ok && warp_wait(bar_r + 8, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
                r_times(tmem + kTmU + 32, dX + (uint64_t)(4096 >> 4), 1, id32, 0);
                mma_commit(bar_u + 8);
                if (kOut) {
                    r_times(tmem + kTmPo, dY, 0, id64, 1);
                    r_times(tmem + kTmPo + 32, dY + (uint64_t)(4096 >> 4), 1, id32, 0);
                }
            }
            __syncwarp();
            ok = ok && warp_wait(bar_w, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {  // D3 over the state operand, which D1 and Dq have consumed
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const uint32_t x = tmem + kTmUw + 8 * kk;
                    const uint64_t b = dkm + (uint64_t)((kk * 2048) >> 4);
                    mma_ts(tmem + kTmS, x, b, id128m, kk > 0);
                    mma_ts(tmem + kTmS, x + 16, b, id128m, 1);
                }
            }
            __syncwarp();
            ok = ok && warp_wait(bar_w + 8, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const uint32_t x = tmem + kTmUw + 32 + 8 * kk;
                        const uint64_t b = dkm + (uint64_t)(((2 + kk) * 2048 + a * 8192) >> 4);
                        mma_ts(tmem + kTmS + 64 * a, x, b, id64m, 1);
                        mma_ts(tmem + kTmS + 64 * a, x + 16, b, id64m, 1);
                    }
                    mma_commit(bar_d + 8 * a);
                }
                if (kOut) {
                    v_times(tmem + kTmPo, desc_mnmajor(st + C::V, 64, 0), dY, 0);
                    mma_commit(bar_o);
                }
                mma_commit(bar_empty + 8 * s);
            }
            __syncwarp();
            if (it + 1 < nch) issue_v(it + 1);
        }
    } else if (warp >= C::kMmaWarp) {  // idle
    } else if (kOut && warp >= 8) {  // output warps: value column d, all 64 tokens
        const int wq = warp & 3, d = 32 * wq + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
        float* s_gam = reinterpret_cast<float*>(sm + C::Misc + 512) + wq * 64;
        const bool odd = lane & 1;
        regs_dec<96>();
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            ok = ok && mbar_wait_ab(bar_full + 8 * s, (uint32_t)(it >> 1) & 1u, s_abort);
            {   // 2^g, kept past the stage's end
                const float* sc = reinterpret_cast<const float*>(sm + s * C::Stage + C::Scal) + kGam;
                const float2 g2 = *reinterpret_cast<const float2*>(sc + 2 * lane);
                __syncwarp();
                *reinterpret_cast<float2*>(s_gam + 2 * lane) = g2;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_empty + 8 * s);
            }
            ok = ok && mbar_wait_ab(bar_o, (uint32_t)it & 1u, s_abort);
            fence_after_sync();
            const long long t = s0 + 64LL * it;
            const int L = (int)(s1 - t < 64 ? s1 - t : 64);
            uint32_t z[32];  // tokens 2 m, 2 m + 1 of column d
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                float x[16], y[16];
                tmem_ld16(tl + kTmDq + c, x);
                tmem_ld16(tl + kTmPo + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int m = 0; m < 16; m += 4) {
                    const float4 g4 = *reinterpret_cast<const float4*>(s_gam + c + m);
                    z[(c + m) / 2] = pack_bf16(fmaf(g4.x, x[m], y[m]), fmaf(g4.y, x[m + 1], y[m + 1]));
                    z[(c + m) / 2 + 1] = pack_bf16(fmaf(g4.z, x[m + 2], y[m + 2]), fmaf(g4.w, x[m + 3], y[m + 3]));
                }
            }
            warp_arrive(bar_q);
            // neighbours exchange: the even lane stores columns (d, d + 1) of the even token, the odd lane of the odd
            const size_t row = (size_t)H * dvw;
            const int Lo = d < dvw && ok ? L - (odd ? 1 : 0) : 0;
            __nv_bfloat16* o = out + ((size_t)t * H + h) * dvw + (d & ~1) + (odd ? row : 0);
#pragma unroll
            for (int m = 0; m < 32; ++m) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, z[m], 1);
                const uint32_t two = odd ? __byte_perm(got, z[m], 0x7632) : __byte_perm(z[m], got, 0x5410);
                if (2 * m < Lo) *reinterpret_cast<uint32_t*>(o) = two;
                o += 2 * row;
            }
        }
    } else {
        const int wg = warp >> 2, d = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        if (kOut) regs_inc<176>();
        f32x2 S[32];
        load_state(start, wg, d, S);
        if (trans) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                S[c] = pair(64 * wg + 2 * c == d ? 1.f : 0.f, 64 * wg + 2 * c + 1 == d ? 1.f : 0.f);
        }
        // the state operand of chunk `it`, and for the backward its image
        auto put_state = [&](int it) {
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int m = 16 * b; m < 16 * b + 16; ++m) split2(S[m], hi[m], lo[m]);
                tmem_st16u(tl + kTmS + 64 * wg + 16 * b, hi + 16 * b);
                tmem_st16u(tl + kTmS + 64 * wg + 32 + 16 * b, lo + 16 * b);
            }
            tmem_wait_st();
            if (it < nch) {
                warp_arrive(bar_s + 8 * wg);
                if (MODE == kChainStates) store_blocks<8>(images + ((size_t)(jb + it) * H + h) * kImages + kImgS, 32768, 8 * wg, d, hi, lo);
            }
        };
        // The last chunk's token rows past the sequence's end hold other tokens, whose values may be anything:
        // cleared before the tensor core reads them.
        auto clear_tail = [&](int it) {
            const long long left = s1 - (s0 + 64LL * it);
            if (left < 64) {
                uint8_t* st = sm + (it & 1) * C::Stage;
                ok = ok && mbar_wait_ab(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u, s_abort);
                if (ok) {
                    zero_tail_rows(st + C::K + 8192 * wg, (int)left);
                    zero_tail_rows(st + C::V + 8192 * wg, (int)left);
                    if (kOut) zero_tail_rows(st + C::Q + 8192 * wg, (int)left);
                }
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_z);
        };
        if (nch > 0) clear_tail(0);
        put_state(0);
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            const uint32_t par = (uint32_t)it & 1u;
            const uint32_t sc = sb + s * C::Stage + C::Scal;
            ok = ok && mbar_wait_ab(bar_full + 8 * s, (uint32_t)(it >> 1) & 1u, s_abort);
            // this warpgroup's token rows of two scalars, while D1 runs
            f32x2 ng[16], w[16];
#pragma unroll
            for (int m = 0; m < 16; m += 2) {
                lds_pairs(sc + 4 * (kNgam + 32 * wg + 2 * m), ng[m], ng[m + 1]);
                lds_pairs(sc + 4 * (kW + 32 * wg + 2 * m), w[m], w[m + 1]);
            }
            float x[32];
            f32x2 y[16];
            ok = ok && mbar_wait_ab(bar_k + 8 * wg, par, s_abort);
            fence_after_sync();
            tmem_ld32(tl + kTmD1 + 32 * wg, x);
#pragma unroll
            for (int m = 0; m < 16; ++m) y[m] = mul2(ng[m], pair(x[2 * m], x[2 * m + 1]));
            tmem_put_split32(tl + kTmD1 + 32 * wg, y);
            tmem_wait_st();
            warp_arrive(bar_r + 8 * wg);
            float last1;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(last1) : "r"(sc + 4 * (kGam + 63)));
            const f32x2 last = pair(last1, last1);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
            ok = ok && mbar_wait_ab(bar_u + 8 * wg, par, s_abort);
            fence_after_sync();
            tmem_ld32(tl + kTmU + 32 * wg, x);
#pragma unroll
            for (int m = 0; m < 16; ++m) y[m] = mul2(w[m], pair(x[2 * m], x[2 * m + 1]));
            tmem_put_split32(tl + kTmUw + 32 * wg, y);
            tmem_wait_st();
            warp_arrive(bar_w + 8 * wg);
            if (it + 1 < nch) clear_tail(it + 1);
            if (MODE == kChainStates) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int m = 0; m < 16; ++m) split2(x[2 * m], x[2 * m + 1], hi[m], lo[m]);
                store_blocks<4>(images + ((size_t)(jb + it) * H + h) * kImages + kImgU, 16384, 4 * wg, d, hi, lo);
            }
            ok = ok && mbar_wait_ab(bar_d + 8 * wg, par, s_abort);
            fence_after_sync();
            {
                float z[64];
#pragma unroll
                for (int c = 0; c < 64; c += 16) tmem_ld16(tl + kTmS + 64 * wg + c, z + c);
                tmem_wait_ld();
#pragma unroll
                for (int m = 0; m < 32; ++m) S[m] = fma2(last, S[m], pair(z[2 * m], z[2 * m + 1]));
            }
            put_state(it + 1);
        }
        if (ok) store_state(end, wg, d, S);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int MODE>
__global__ void __launch_bounds__(Chain<MODE>::kThreads, 1)
gdn_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const float* S0, float* S_final, __nv_bfloat16* out,
                 const __grid_constant__ ChainArgs ca, const __grid_constant__ Segments sg)
{
    chain_body<MODE>(&tm_q, &tm_k, &tm_v, S0, S_final, out, ca, nullptr, sg, blockIdx.x, blockIdx.y == 1);
}

// [tokens][heads][d] bf16 as a 3-D map of 64-token, 64-channel boxes that land 128B-swizzled
inline bool make_map(CUtensorMap* m, const void* base, int heads, int d, long long ntok)
{
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)ntok};
    const cuuint64_t strides[2] = {2 * (cuuint64_t)d, 2 * (cuuint64_t)d * heads};
    const cuuint32_t box[3] = {64, 1, 64}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BWD>
cudaError_t launch_prep(const CUtensorMap& tq, const CUtensorMap& tk, const float* la, const float* beta,
                        const WsHeader* hdr, const int* off, const int32_t* cu, int Tseq, int N, int H, int Hk,
                        long long units, uint8_t* slots, uint8_t* bslots, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(gdn_prep_kernel<BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepSmem);
    if (e != cudaSuccess) return e;
    LaunchScope ls(BWD ? "gdn_bwd_prep" : "gdn_prep", stream);
    gdn_prep_kernel<BWD><<<(unsigned)units, kPrepThreads, kPrepSmem, stream>>>(tq, tk, la, beta, hdr, off, cu, Tseq, N, H,
                                                                              H / Hk, slots, bslots);
    return cudaGetLastError();
}

// F'_g = M_g F'_{g-1} + F_g over the inner segments of a sequence (forward), or, with the transposes and
// from the last segment down, F'_g = M_g^T F'_{g+1} + F_g (reverse).  One CTA a (sequence, head, 16 value
// columns), M in shared memory; a lane holds half a column of the state in registers (column lane % 16, key
// channels 64 (lane / 16) ..) and a warp makes 16 rows, so that M is read as broadcasts.  fp32 on CUDA cores: 12 us
// for three segments of 32 heads, of which two thirds is the copy of M and the launch.
constexpr int kJoinCols = 16, kJoinThreads = 256;
constexpr uint32_t kJoinSmem = 65536 + 1024;
template <bool REVERSE>
__device__ __forceinline__ void join_body(const ChainArgs& ca, const Segments& sg, int slice)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_first;
    __shared__ __align__(8) uint64_t s_bar;
    const int* __restrict__ off = ca.off;
    const int32_t* __restrict__ cu = ca.cu;
    const int Tseq = ca.Tseq, H = ca.H;
    if (cu && ca.hdr->bad) return;
    const int n = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int v = slice * kJoinCols + (lane & 15), k0 = 64 * (lane >> 4);
    uint8_t* sm = aligned_smem(smem_raw);
    const float* sM = reinterpret_cast<const float*>(sm);
    const uint32_t bar = smem_u32(&s_bar);
    // the sequence's first segment: the segments of those before it
    int part = 0;
    auto segments = [&](int m) {
        return (chunks_before(off, cu, Tseq, m + 1) - chunks_before(off, cu, Tseq, m) + sg.len - 1) / sg.len;
    };
    for (int m = threadIdx.x; m < n; m += kJoinThreads) part += max(1, segments(m));
    if (threadIdx.x == 0) {
        s_first = 0;
        mbar_init(bar, 1);
        mbar_fence_init();
    }
    __syncthreads();
    if (part) atomicAdd(&s_first, part);
    __syncthreads();
    const int first = s_first, nseg = segments(n);
    auto at = [&](int g) { return ((size_t)(first + g) * H + h) * 16384; };
    for (int i = 0; i + 2 < nseg; ++i) {
        const int g = REVERSE ? nseg - 2 - i : 1 + i, from = REVERSE ? g + 1 : g - 1;
        if (threadIdx.x == 0) {
            mbar_arrive_expect_tx(bar, 65536);
            bulk_g2s(smem_u32(sm), sg.M + at(g), 65536, bar);
        }
        float S[64];
        const float* src = sg.F + at(from) + (size_t)k0 * 128 + v;
#pragma unroll
        for (int k = 0; k < 64; ++k) S[k] = src[(size_t)k * 128];
        float* dst = sg.F + at(g) + (size_t)(16 * warp) * 128 + v;
        const uint32_t par = (uint32_t)i & 1u;
        const bool ok = mbar_wait(bar, par);
#pragma unroll 1
        for (int r = 0; r < 16; r += 4) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            const int row = 16 * warp + r;
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // four consecutive terms of row row + e, or (reverse) term k + e of rows row .. row + 3
                    const float4 w = *reinterpret_cast<const float4*>(REVERSE ? sM + (k0 + k + e) * 128 + row
                                                                              : sM + (row + e) * 128 + k0 + k);
                    if (REVERSE) {
                        acc[0] = fmaf(w.x, S[k + e], acc[0]); acc[1] = fmaf(w.y, S[k + e], acc[1]);
                        acc[2] = fmaf(w.z, S[k + e], acc[2]); acc[3] = fmaf(w.w, S[k + e], acc[3]);
                    } else {
                        acc[e] = fmaf(w.x, S[k], acc[e]); acc[e] = fmaf(w.y, S[k + 1], acc[e]);
                        acc[e] = fmaf(w.z, S[k + 2], acc[e]); acc[e] = fmaf(w.w, S[k + 3], acc[e]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], 16);
                if (ok && lane < 16) dst[(size_t)(r + e) * 128] += acc[e];
            }
        }
        if (!__syncthreads_and(ok)) {  // M consumed, F' visible to the CTA
            (void)mbar_wait(bar, par);  // the copy does not outlive the CTA
            break;
        }
    }
}

// slices 0 .. 7 forward, 8 .. 15 (the backward only) reverse
__global__ void __launch_bounds__(kJoinThreads)
gdn_join_kernel(const __grid_constant__ ChainArgs ca, const __grid_constant__ Segments fwd,
                const __grid_constant__ Segments rev)
{
    constexpr int kSlices = 128 / kJoinCols;
    if (blockIdx.z < kSlices) join_body<false>(ca, fwd, blockIdx.z);
    else join_body<true>(ca, rev, blockIdx.z - kSlices);
}

// Chunks a segment, from the number of chains c and their length L (for packed sequences the mean; the lengths
// are on the device).  G segments put c G CTAs into the real pass and c (2 G - 3) into the ends' (backward, both
// chains side by side: 2 c G and c (3 G - 4)); CTAs run one an SM, so G stays where neither needs a second
// wave.  Within that, a segment costs about 7 us (join, start of two passes), which against 5.2 (6.3) us a chunk
// of the two passes is least at G = sqrt(0.75 L).  Without segments a chunk costs 3.0 (3.9) us.
// Measured at the rule's G and without segments, us: prefill, 512 chunks, 32 heads G = 3 1041, 1517; 16 heads 6 589,
// 1583; 2 heads 19 230, 1223; 80 chains of 256 chunks 1 998 (2: 1288); backward, 32 heads 2 3236, 3680; 8 heads 7
// 960, 2402; 32 chains of 16 chunks 1 142 (2: 154).  The best G of a sweep over 1 .. 24 was at most 9 % faster.
inline int segment_length(int max_chunks, int N, int H, bool bwd)
{
    constexpr double kSms = 148;
    constexpr int kMaxSeqs = 1024;
    if (N > kMaxSeqs || max_chunks == 0) return 0;
    const double c = (double)N * H;
    const int L = (max_chunks + N - 1) / N;
    const double fit = bwd ? fmin(kSms / (2 * c), (kSms / c + 4) / 3) : fmin(kSms / c, (kSms / c + 3) / 2);
    const int G = (int)fmin(fit, sqrt(0.75 * L));
    if (G < 2 || (bwd ? 6.3 : 5.2) * L / G + 7.0 * G + 10.0 > 0.95 * (bwd ? 3.9 : 3.0) * L) return 0;
    return (L + G - 1) / G;
}
inline long long max_segments(int max_chunks, int N, int len) { return len ? max_chunks / len + N : N; }
inline size_t segments_bytes(int max_chunks, int N, int H, bool bwd)
{
    const int len = segment_length(max_chunks, N, H, bwd);
    return len ? (size_t)max_segments(max_chunks, N, len) * H * 65536 : 0;
}

template <int MODE>
cudaError_t launch_chain(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const float* S0,
                         float* S_final, void* out, const ChainArgs& ca, int max_chunks, const Segments& sg,
                         cudaStream_t stream)
{
    using C = Chain<MODE>;
    const cudaError_t e = cudaFuncSetAttribute(gdn_chain_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
    if (e != cudaSuccess) return e;
    LaunchScope ls(MODE == kChainOut ? "gdn_chain" : "gdn_ends", stream);
    const dim3 grid((unsigned)(max_segments(max_chunks, ca.N, sg.len) * ca.H), MODE == kChainEnds ? 2 : 1);
    gdn_chain_kernel<MODE><<<grid, C::kThreads, C::Smem, stream>>>(tq, tk, tv, S0, S_final, (__nv_bfloat16*)out, ca, sg);
    return cudaGetLastError();
}
inline cudaError_t launch_join(const ChainArgs& ca, const Segments& fwd, const Segments* rev, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(gdn_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmem);
    if (e != cudaSuccess) return e;
    LaunchScope ls("gdn_join", stream);
    gdn_join_kernel<<<dim3(ca.N, ca.H, 128 / kJoinCols * (rev ? 2 : 1)), kJoinThreads, kJoinSmem, stream>>>(
        ca, fwd, rev ? *rev : fwd);
    return cudaGetLastError();
}

// bytes behind the header and the chunk table: slots, segment states (end, transition)
inline size_t fwd_bytes(int max_chunks, int N, int H)
{
    return (size_t)max_chunks * H * kSlot + 2 * segments_bytes(max_chunks, N, H, false);
}

inline cudaError_t launch_fwd(const void* q, const void* k, const void* v, const float* la, const float* beta,
                              const float* S0, float* S_final, void* out, const WsHeader* hdr, const int* off,
                              const int32_t* cu, int Tseq, int N, int H, int Hk, int dk, int dv, int max_chunks,
                              long long Ttot, uint8_t* ws, cudaStream_t stream)
{
    alignas(64) CUtensorMap tq{}, tk{}, tv{};
    const long long units = (long long)max_chunks * H;
    if (units > 0x7fffffffLL || ((long long)max_chunks + N) * H > 0x7fffffffLL) return cudaErrorInvalidValue;
    uint8_t* segs = ws + units * kSlot;
    const size_t sb = segments_bytes(max_chunks, N, H, false);
    const Segments sg{Ttot > 0 ? segment_length(max_chunks, N, H, false) : 0, (float*)segs, (float*)(segs + sb)};
    const ChainArgs ca{hdr, off, cu, Tseq, N, H, H / Hk, dk, dv, ws};
    cudaError_t e = cudaSuccess;
    if (Ttot > 0) {
        if (!make_map(&tq, q, Hk, dk, Ttot) || !make_map(&tk, k, Hk, dk, Ttot) || !make_map(&tv, v, H, dv, Ttot))
            return cudaErrorInvalidValue;
        e = launch_prep<false>(tq, tk, la, beta, hdr, off, cu, Tseq, N, H, Hk, units, ws, nullptr, stream);
    }
    if (e == cudaSuccess && sg.len) {
        e = launch_chain<kChainEnds>(tq, tk, tv, S0, nullptr, nullptr, ca, max_chunks, sg, stream);
        if (e == cudaSuccess) e = launch_join(ca, sg, nullptr, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_chain<kChainOut>(tq, tk, tv, S0, S_final, out, ca, max_chunks, sg, stream);
}

}  // namespace gdn
}  // namespace kda
