// gdn_bwd_tc.cuh -- tensor-core backward of the scalar-gate delta rule, bf16, dk and dv 64 or 128.
//
// With the chunk form of gdn_tc.cuh (T = (I + A)^-1, w_j = 2^(g_C - g_j), D_ij = 2^(g_i - g_j)) and the
// cotangents dO and dS' (of the state after the chunk):
//     dU = P^T dO + w (k dS')             dR = T^T dU           dv = beta dR
//     dS = 2^g_C dS' + (2^g q)^T dO - k^T (beta 2^g dR)
//     PD = lower(dO U^T) . D              E = -strict_lower(dR U^T) . D         G = diag(beta) E
//     dq = 2^g dO S^T + PD k
//     dk = [-beta 2^g dR S^T + G k] + [w U dS'^T + PD^T q + G^T k] = [ka] + [kb]
//     dbeta_i = dR_i.v_i - 2^g_i k_i.(dR S^T)_i + (E . k k^T) row sum
//     dg_i = q_i.dq_i + k_i.ka_i - k_i.kb_i,  dg_C += sum_j w_j k_j.(U dS'^T)_j + 2^g_C <S, dS'>
//     dlog_alpha_i = sum of dg_m over m >= i in the chunk
// of which PD's diagonal cancels in each dg_i and the terms of w and U with the sum at C; they are left out:
//     dlog_alpha_i = sum over m >= i of [q.dq + k.ka - k.kb without them]_m + sum over m < i of w_m k_m.(U dS'^T)_m
//                    + 2^g_C <S, dS'>
// Without a start state a sequence's first gate multiplies zeros.  Its gradient is written as zero, where the sums
// would leave their rounding (1e-5).
// Three passes: per-chunk matrices (gdn_prep); side by side the forward states again and the reverse chain
// for dS' and dR (in segments, with a pass for their ends before); one CTA a (chunk, head) for the gradients.
// dg is taken from row products of terms that belong to this chunk, never from a sum over the whole sequence,
// whose cancellation would cost the small gates their digits.  Splits and accuracy as in the forward: 3..5e-6
// for every fp32 gradient.
#pragma once

#include "gdn_tc.cuh"

namespace kda {
namespace gdn {

// unswizzled MN-major operand of 128 contraction rows (one of the images): k step kk is 256 kk bytes on
__device__ __forceinline__ uint64_t desc_image(uint32_t addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 16;    // between blocks of 8 contraction rows
    d |= (uint64_t)(2048u >> 4) << 32;   // between blocks of 8 columns
    d |= (uint64_t)1u << 46;             // descriptor version for sm_100, no swizzle
    return d;
}

// ----------------------------------------------------------------------------------------------------
// Reverse chain: one CTA a (sequence, head), chunks from the last to the first.  The layout is the forward
// chain's (row = value column), the state is dS:
//     D1 = dS'^T k^T (16 MMAs)     dU = P^T dO + w D1      (P^T dO: 8, under the update before)
//     dR = dU T      (12)          y = -beta 2^g dR
//     D3 = dO^T (2^g q) + y k (8 of N = 128, under the making of dU; 16)     dS <- 2^g_C dS' + D3
// TMEM columns: 0 D1 -> dU, 64 P^T dO, 128 dR -> y, 256 dS operand -> D3.
// Bound like the forward chain, with one hand-over less: 4.2 us a chunk beside the forward chain of the same launch
// (256 chunks of 64 + 64 CTAs 1.06 ms, 32 heads of 32K tokens in two segments), as both write their images.
// ----------------------------------------------------------------------------------------------------
constexpr int kRThreads = 320;
constexpr uint32_t kRK = 0, kRDo = 16384, kRGq = 32768, kRP = 65536, kRX = 81920, kRScal = 98304, kRStage = 99328;
constexpr uint32_t kRMisc = 2 * kRStage, kRSmem = kRMisc + 512 + 1024;

// ENDS: no outputs, only a segment's start cotangent from a zero (the last segment's: the given) end one
template <bool ENDS>
__device__ __forceinline__ void reverse_body(const CUtensorMap* tm_k, const CUtensorMap* tm_do,
                                             const float* __restrict__ dS_final, float* __restrict__ dS0,
                                             __nv_bfloat16* __restrict__ dv_out, const ChainArgs& ca,
                                             const uint8_t* __restrict__ bslots, uint8_t* __restrict__ images,
                                             const Segments& sg, int block)
{
    const int* __restrict__ off = ca.off;
    const int32_t* __restrict__ cu = ca.cu;
    const int Tseq = ca.Tseq, N = ca.N, H = ca.H, G = ca.G, dkw = ca.dk, dvw = ca.dv;
    const uint8_t* __restrict__ slots = ca.slots;
    extern __shared__ uint8_t smem_raw[];
    if (cu && ca.hdr->bad) return;
    const int sidx = block / H, h = block - sidx * H;
    int n, seg, nseg;
    if (!find_segment(sidx, off, cu, Tseq, N, sg, n, seg, nseg)) return;
    if (ENDS && seg == 0) return;  // nothing ends at the first segment's start
    const int jb = chunks_before(off, cu, Tseq, n) + seg * sg.len, left = chunks_before(off, cu, Tseq, n + 1) - jb, nch = seg == nseg - 1 ? left : sg.len;
    long long s0, s1;
    seq_bounds(n, cu, Tseq, s0, s1);
    s0 += 64LL * seg * sg.len;
    const size_t mine = ((size_t)n * H + h) * dkw * dvw, part = ((size_t)sidx * H + h) * 16384;
    const StateRef start = seg == nseg - 1
                               ? StateRef{dS_final ? const_cast<float*>(dS_final) + mine : nullptr, dvw, dkw, dvw}
                               : StateRef{ENDS ? nullptr : sg.F + part + (size_t)H * 16384, 128, 128, 128};
    const StateRef end = ENDS ? StateRef{sg.F + part, 128, 128, 128}
                              : StateRef{dS0 && seg == 0 ? dS0 + mine : nullptr, dvw, dkw, dvw};
    uint8_t* sm = aligned_smem(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + kRMisc;
    const uint32_t bar_full = bars, bar_empty = bars + 16, bar_k = bars + 32, bar_d = bars + 48, bar_s = bars + 64,
                   bar_u = bars + 80, bar_r = bars + 88, bar_w = bars + 96, bar_z = bars + 104;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kRMisc + 112);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + kRMisc + 116);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 9);
            mbar_init(bar_k + 8 * s, 1);
            mbar_init(bar_d + 8 * s, 1);
            mbar_init(bar_s + 8 * s, 4);
        }
        mbar_init(bar_u, 1);
        mbar_init(bar_r, 8);
        mbar_init(bar_w, 8);
        mbar_init(bar_z, 8);
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
        int issued = 0;
        for (int it = 0; it < nch && ok; ++it) {
            const int s = it & 1, c = nch - 1 - it;
            if (it >= 2) ok = warp_wait(bar_empty + 8 * s, (uint32_t)((it >> 1) - 1) & 1u, s_abort);
            if (ok && elect_one()) {
                const uint32_t st = sb + s * kRStage, f = bar_full + 8 * s;
                const int t = (int)(s0 + 64LL * c);
                const size_t u = (size_t)(jb + c) * H + h;
                mbar_arrive_expect_tx(f, kRStage);
                for (int a = 0; a < 2; ++a) {
                    tma_load_3d(st + kRK + 8192 * a, tm_k, 64 * a, h / G, t, f);
                    tma_load_3d(st + kRDo + 8192 * a, tm_do, 64 * a, h, t, f);
                }
                bulk_g2s(st + kRGq, bslots + u * kBwdSlot + kBwdQ, 32768, f);
                bulk_g2s(st + kRP, bslots + u * kBwdSlot + kBwdP, 32768, f);
                bulk_g2s(st + kRScal, slots + u * kSlot + kScal, 1024, f);
            }
            __syncwarp();
            issued = ok ? it + 1 : issued;
        }
        for (int it = issued > 2 ? issued - 2 : 0; it < issued; ++it)  // no copy outlives the CTA, whatever gave up
            (void)mbar_wait(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u);
    } else if (warp == 8) {
        const uint32_t id64 = idesc_bf16(128, 64, false, false), id32 = idesc_bf16(128, 32, false, false),
                       id64m = idesc_bf16(128, 64, false, true), idE = idesc_bf16(128, 64, true, true),
                       idF = idesc_bf16(128, 128, true, true);
        auto issue_e = [&](int it) {  // P^T dO, into the accumulator that the chunk before has been read from
            const uint32_t st = sb + (it & 1) * kRStage;
            ok = ok && warp_wait(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u, s_abort);
            ok = ok && warp_wait(bar_z, (uint32_t)it & 1u, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
                const uint64_t a = desc_mnmajor(st + kRDo, 64, 0), b = desc_mnmajor(st + kRP, 64, 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t o = (uint64_t)((kk * 2048) >> 4);
                    mma_bf16(tmem + 64, a + o, b + o, idE, kk > 0);
                    mma_bf16(tmem + 64, a + o, b + o + (8192 >> 4), idE, 1);
                }
            }
            __syncwarp();
        };
        if (nch > 0) issue_e(0);
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1;
            const uint32_t st = sb + s * kRStage, par = (uint32_t)it & 1u;
            const uint64_t dk = desc_kmajor(st + kRK, 64, 0), dkm = desc_mnmajor(st + kRK, 64, 0),
                           dX = desc_mnmajor(st + kRX, 64, 0), dDo = desc_mnmajor(st + kRDo, 64, 0),
                           dGq = desc_mnmajor(st + kRGq, 64, 0);
            auto state_times = [&](uint32_t d, uint64_t b, int a, uint32_t id, uint32_t first) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t x = tmem + 256 + 64 * a + 8 * kk;
                    const uint64_t bb = b + (uint64_t)((a * 8192 + kk * 32) >> 4);
                    mma_ts(d, x, bb, id, kk > 0 || !first);
                    mma_ts(d, x + 32, bb, id, 1);
                }
            };
            ok = ok && warp_wait(bar_s, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) state_times(tmem, dk, 0, id64, 1);
            __syncwarp();
            ok = ok && warp_wait(bar_s + 8, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
                state_times(tmem, dk, 1, id32, 0);
                mma_commit(bar_k);
                state_times(tmem + 32, dk + (uint64_t)(4096 >> 4), 1, id32, 0);
                mma_commit(bar_k + 8);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {  // over the state operand, which D1 has consumed
                    const uint64_t o = (uint64_t)((kk * 2048) >> 4);
                    mma_bf16(tmem + 256, dDo + o, dGq + o, idF, kk > 0);
                    mma_bf16(tmem + 256, dDo + o, dGq + o + (16384 >> 4), idF, 1);
                }
            }
            __syncwarp();
            ok = ok && warp_wait(bar_r, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {  // dR = dU T
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t x = tmem + 32 * (kk >> 1) + 8 * (kk & 1);
                    const uint64_t b = dX + (uint64_t)((kk * 2048) >> 4);
                    mma_ts(tmem + 128, x, b, id64m, kk > 0);
                    mma_ts(tmem + 128, x + 16, b, id64m, 1);
                    mma_ts(tmem + 128, x, b + (8192 >> 4), id64m, 1);
                }
                mma_commit(bar_u);
            }
            __syncwarp();
            ok = ok && warp_wait(bar_w, par, s_abort);
            fence_after_sync();
            if (ok && elect_one()) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t x = tmem + 128 + 32 * (kk >> 1) + 8 * (kk & 1);
                        const uint64_t b = dkm + (uint64_t)((kk * 2048 + a * 8192) >> 4);
                        mma_ts(tmem + 256 + 64 * a, x, b, id64m, 1);
                        mma_ts(tmem + 256 + 64 * a, x + 16, b, id64m, 1);
                    }
                    mma_commit(bar_d + 8 * a);
                }
                mma_commit(bar_empty + 8 * s);
            }
            __syncwarp();
            if (it + 1 < nch) issue_e(it + 1);
        }
    } else {
        const int wg = warp >> 2, d = 32 * (warp & 3) + lane;
        const bool odd = lane & 1;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        f32x2 S[32];
        load_state(start, wg, d, S);
        auto put_state = [&](int it) {  // the operand of step `it` and its image, the cotangent after that chunk
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int m = 16 * b; m < 16 * b + 16; ++m) split2(S[m], hi[m], lo[m]);
                tmem_st16u(tl + 256 + 64 * wg + 16 * b, hi + 16 * b);
                tmem_st16u(tl + 256 + 64 * wg + 32 + 16 * b, lo + 16 * b);
            }
            tmem_wait_st();
            if (it < nch) {
                warp_arrive(bar_s + 8 * wg);
                if (!ENDS) store_blocks<8>(images + ((size_t)(jb + nch - 1 - it) * H + h) * kImages + kImgDs, 32768, 8 * wg, d, hi, lo);
            }
        };
        auto clear_tail = [&](int it) {
            const long long left = s1 - (s0 + 64LL * (nch - 1 - it));
            if (left < 64) {
                uint8_t* st = sm + (it & 1) * kRStage;
                ok = ok && mbar_wait_ab(bar_full + 8 * (it & 1), (uint32_t)(it >> 1) & 1u, s_abort);
                if (ok) {
                    zero_tail_rows(st + kRK + 8192 * wg, (int)left);
                    zero_tail_rows(st + kRDo + 8192 * wg, (int)left);
                }
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_z);
        };
        if (nch > 0) clear_tail(0);
        put_state(0);
        for (int it = 0; it < nch; ++it) {
            const int s = it & 1, c = nch - 1 - it;
            const uint32_t par = (uint32_t)it & 1u, sc = sb + s * kRStage + kRScal;
            const size_t u = (size_t)(jb + c) * H + h;
            ok = ok && mbar_wait_ab(bar_full + 8 * s, (uint32_t)(it >> 1) & 1u, s_abort);
            f32x2 w[16];  // token rows of the scalars are fetched ahead of each use, while an MMA runs
#pragma unroll
            for (int m = 0; m < 16; m += 2) lds_pairs(sc + 4 * (kW + 32 * wg + 2 * m), w[m], w[m + 1]);
            float last1;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(last1) : "r"(sc + 4 * (kGam + 63)));
            const f32x2 last = pair(last1, last1);
            float x[32];
            f32x2 y[16];
            {
                float e[32];
                ok = ok && mbar_wait_ab(bar_k + 8 * wg, par, s_abort);
                fence_after_sync();
                tmem_ld16(tl + 64 + 32 * wg, e);
                tmem_ld16(tl + 64 + 32 * wg + 16, e + 16);
                tmem_ld32(tl + 32 * wg, x);
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    y[m] = fma2(w[m], pair(x[2 * m], x[2 * m + 1]), pair(e[2 * m], e[2 * m + 1]));
            }
            tmem_put_split32(tl + 32 * wg, y);
            tmem_wait_st();
            warp_arrive(bar_r);
            f32x2 be[16];
#pragma unroll
            for (int m = 0; m < 16; m += 2) {
                lds_pairs(sc + 4 * (kBeta + 32 * wg + 2 * m), be[m], be[m + 1]);
                lds_pairs(sc + 4 * (kNgam + 32 * wg + 2 * m), w[m], w[m + 1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
            ok = ok && mbar_wait_ab(bar_u, par, s_abort);
            fence_after_sync();
            tmem_ld32(tl + 128 + 32 * wg, x);
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                y[m] = mul2(be[m], pair(x[2 * m], x[2 * m + 1]));  // dv
                w[m] = mul2(w[m], y[m]);
            }
            tmem_put_split32(tl + 128 + 32 * wg, w);
            tmem_wait_st();
            warp_arrive(bar_w);
            if (it + 1 < nch) clear_tail(it + 1);
            if (!ENDS) {  // while D3 runs: dR's image and dv
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int m = 0; m < 16; ++m) split2(x[2 * m], x[2 * m + 1], hi[m], lo[m]);
                store_blocks<4>(images + u * kImages + kImgDr, 16384, 4 * wg, d, hi, lo);
                const long long t = s0 + 64LL * c + 32 * wg;
                const int Lw = !ok || d >= dvw ? 0 : (int)(s1 - t < 32 ? s1 - t : 32) - (odd ? 1 : 0);
                const size_t row = (size_t)H * dvw;
                __nv_bfloat16* o = dv_out + ((size_t)t * H + h) * dvw + (d & ~1) + (odd ? row : 0);
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    float a, b;
                    unpair(y[m], a, b);
                    const uint32_t z = pack_bf16(a, b), got = __shfl_xor_sync(0xffffffffu, z, 1);
                    const uint32_t two = odd ? __byte_perm(got, z, 0x7632) : __byte_perm(z, got, 0x5410);
                    if (2 * m < Lw) *reinterpret_cast<uint32_t*>(o) = two;
                    o += 2 * row;
                }
            }
            ok = ok && mbar_wait_ab(bar_d + 8 * wg, par, s_abort);
            fence_after_sync();
            {
                float z[64];
#pragma unroll
                for (int cc = 0; cc < 64; cc += 16) tmem_ld16(tl + 256 + 64 * wg + cc, z + cc);
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
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// Both chains of the backward in one launch, since neither needs the other and each alone leaves SMs idle: blocks
// 0 .. nr - 1 reverse, the next nr forward, and with ENDS the next nr the forward transitions.  The joint kernel
// spills: 184 bytes of a thread, with ENDS 104 (ptxas).
template <bool ENDS>
__global__ void __launch_bounds__(kRThreads, 1)
gdn_bwd_chains_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_do, const float* S0, const float* dS_final, float* dS0,
                      __nv_bfloat16* dv_out, const __grid_constant__ ChainArgs ca, const uint8_t* bslots, uint8_t* images,
                      const __grid_constant__ Segments fwd, const __grid_constant__ Segments rev, int nr)
{
    const int b = blockIdx.x;
    if (b < nr)
        reverse_body<ENDS>(&tm_k, &tm_do, dS_final, dS0, dv_out, ca, bslots, images, rev, b);
    else
        chain_body<ENDS ? kChainEnds : kChainStates>(&tm_k, &tm_k, &tm_v, S0, nullptr, nullptr, ca, images, fwd,
                                                     b < 2 * nr ? b - nr : b - 2 * nr, b >= 2 * nr);
}

// ----------------------------------------------------------------------------------------------------
// Gradients of one (chunk, head): all products M = 64 (row = token), 256 threads.
//   first:  dO S^T and dR S^T (N = 128); dO U^T, dR U^T, k k^T and v dR^T (N = 64; of the last the diagonal)
//   then, with dS' in S's place and the split PD and G in dO's and v's:  U dS'^T, PD k, G k, PD^T q + G^T k
// 192 KB of operands and all of TMEM, one CTA an SM, so loads, MMAs and the conversions of a unit alternate: 32K
// tokens x 32 heads 1.24 ms, 4.3 GB at 0.54 of the copy bandwidth, tensor pipe 44 % busy.  Fetching dS' and the next
// unit's images into L2 ahead saves 0.08; all of the next unit's operands cost 0.06..0.16 instead.
// TMEM columns: 0 dO S^T, 128 dR S^T, 256 dO U^T, 320 dR U^T, 384 k k^T, 448 v dR^T; then 0 U dS'^T, 128 PD k,
// 256 G k, 384 PD^T q + G^T k.
// A thread holds 32 channels of a token row: row 16 (warp % 4) + lane % 16, channels 64 (lane / 16) +
// 32 (warp / 4) .. .
// ----------------------------------------------------------------------------------------------------
constexpr int kGThreads = 256;
constexpr uint32_t kGS = 0, kGU = 65536, kGDr = 98304, kGK = 131072, kGQ = 147456, kGDo = 163840, kGV = 180224,
                   kGPd = kGDo, kGG = kGV, kGMisc = 196608, kGSmem = kGMisc + 8192 + 1024;

constexpr unsigned kGAhead = 148;  // one CTA an SM

__device__ __forceinline__ void bulk_prefetch(const void* p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void grad_ld32(uint32_t taddr, float* x)
{
    tmem_ld16_pair<64>(taddr, x);
    tmem_ld16_pair<64>(taddr + 16, x + 16);
    tmem_wait_ld();
}

__global__ void __launch_bounds__(kGThreads, 1)
gdn_bwd_grads_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const float* __restrict__ la, const float* __restrict__ beta, __nv_bfloat16* __restrict__ dq,
                     __nv_bfloat16* __restrict__ dk, float* __restrict__ dq_acc, float* __restrict__ dk_acc,
                     float* __restrict__ dla, float* __restrict__ dbeta, const WsHeader* __restrict__ hdr,
                     const int* __restrict__ off, const int32_t* __restrict__ cu, int Tseq, int N, int H, int G, int dkw,
                     bool start, const uint8_t* __restrict__ images)
{
    extern __shared__ uint8_t smem_raw[];
    if (cu && (hdr->bad || (long long)blockIdx.x >= (long long)hdr->total_chunks * H)) return;
    int h, n, L;
    long long t0;
    tc_unit(blockIdx.x, H, off, cu, Tseq, N, h, n, t0, L);
    uint8_t* sm = aligned_smem(smem_raw);
    const uint32_t sb = smem_u32(sm);
    float* s_g = reinterpret_cast<float*>(sm + kGMisc);   // [64]
    float* s_b = s_g + 64;                                // [64]
    float* s_gl = s_g + 128;                              // [64]
    float* s_red = s_g + 192;                             // [4 sums][4 parts][64 rows]
    float* s_sds = s_red + 1024;                          // [8]
    float* s_pd = s_sds + 8;                              // [64] diagonal of PD
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kGMisc + 6144);
    const uint32_t bar_in = sb + kGMisc + 6160, bar_s = bar_in + 8, bar_ds = bar_in + 16, bar_read = bar_in + 24,
                   bar_m = bar_in + 32;  // 4 MMA barriers
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const uint8_t* img = images + (size_t)blockIdx.x * kImages;

    if (tid == 0) {
        mbar_init(bar_in, 1);
        mbar_init(bar_s, 1);
        mbar_init(bar_ds, 1);
        mbar_init(bar_read, 8);
        for (int i = 0; i < 4; ++i) mbar_init(bar_m + 8 * i, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(bar_in, kGMisc - 65536);
        mbar_arrive_expect_tx(bar_s, 65536);
        for (int a = 0; a < 2; ++a) {
            tma_load_3d(sb + kGDo + 8192 * a, &tm_do, 64 * a, h, (int)t0, bar_in);
            tma_load_3d(sb + kGV + 8192 * a, &tm_v, 64 * a, h, (int)t0, bar_in);
            tma_load_3d(sb + kGK + 8192 * a, &tm_k, 64 * a, h / G, (int)t0, bar_in);
            tma_load_3d(sb + kGQ + 8192 * a, &tm_q, 64 * a, h / G, (int)t0, bar_in);
        }
        bulk_g2s(sb + kGU, img + kImgU, 65536, bar_in);  // U and dR
        bulk_g2s(sb + kGS, img + kImgS, 65536, bar_s);
        bulk_prefetch(img + kImgDs, 65536);  // into L2 already
    }
    if (warp == 1) load_scalars(la, beta, t0, L, H, h, s_g, s_gl, s_b);
    if (warp == 2) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = uniform(*s_tmem);
    bool ok = mbar_wait(bar_in, 0);
    if (L < 64) {  // rows past the sequence's end hold other tokens
        const int a = tid >> 7;
        if (ok) {
            zero_tail_rows(sm + kGDo + 8192 * a, L);
            zero_tail_rows(sm + kGV + 8192 * a, L);
            zero_tail_rows(sm + kGK + 8192 * a, L);
            zero_tail_rows(sm + kGQ + 8192 * a, L);
        }
        fence_proxy_async();
    }
    ok = __syncthreads_and(ok);

    const uint64_t iS = desc_image(sb + kGS), iU = desc_image(sb + kGU), iR = desc_image(sb + kGDr);
    if (warp == 0) {
        if (ok && elect_one()) {
            const uint64_t kDo = desc_kmajor(sb + kGDo, 64, 0), kK = desc_kmajor(sb + kGK, 64, 0),
                           kV = desc_kmajor(sb + kGV, 64, 0);
            const uint32_t kn64 = idesc_bf16(64, 64, false, true), mn64 = idesc_bf16(64, 64, true, true),
                           kk64 = idesc_bf16(64, 64, false, false);
            constexpr uint64_t loU = 16384 >> 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t km = (uint64_t)(((k >> 2) * 8192 + (k & 3) * 32) >> 4), im = (uint64_t)((k * 256) >> 4);
                mma_bf16(tmem + 256, kDo + km, iU + im, kn64, k > 0);
                mma_bf16(tmem + 256, kDo + km, iU + loU + im, kn64, 1);
                mma_bf16(tmem + 320, iR + im, iU + im, mn64, k > 0);
                mma_bf16(tmem + 320, iR + loU + im, iU + im, mn64, 1);
                mma_bf16(tmem + 320, iR + im, iU + loU + im, mn64, 1);
                mma_bf16(tmem + 384, kK + km, kK + km, kk64, k > 0);
                mma_bf16(tmem + 448, kV + km, iR + im, kn64, k > 0);
                mma_bf16(tmem + 448, kV + km, iR + loU + im, kn64, 1);
            }
            mma_commit(bar_m);
        }
        __syncwarp();
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_s, 0));
        if (ok && elect_one()) {
            const uint64_t kDo = desc_kmajor(sb + kGDo, 64, 0);
            const uint32_t kn128 = idesc_bf16(64, 128, false, true), mn128 = idesc_bf16(64, 128, true, true);
            constexpr uint64_t loU = 16384 >> 4, loS = 32768 >> 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t km = (uint64_t)(((k >> 2) * 8192 + (k & 3) * 32) >> 4), im = (uint64_t)((k * 256) >> 4);
                mma_bf16(tmem, kDo + km, iS + im, kn128, k > 0);
                mma_bf16(tmem, kDo + km, iS + loS + im, kn128, 1);
                mma_bf16(tmem + 128, iR + im, iS + im, mn128, k > 0);
                mma_bf16(tmem + 128, iR + loU + im, iS + im, mn128, 1);
                mma_bf16(tmem + 128, iR + im, iS + loS + im, mn128, 1);
            }
            mma_commit(bar_m + 8);
        }
        __syncwarp();
    }

    const int wq = warp & 3, hw = warp >> 2, r = 16 * wq + (lane & 15), part = 2 * hw + (lane >> 4);
    const uint32_t tl = tmem + ((uint32_t)(32 * wq) << 16);
    const int c0 = 64 * (lane >> 4) + 32 * hw;   // this thread's channels
    const int j0 = 32 * (lane >> 4) + 16 * hw;   // its columns of the 64 x 64 products
    const float gi = s_g[r], gli = s_gl[r], bi = s_b[r], gam = ex2_approx(gi),
                wi = ex2_approx((s_g[63] - gi) + (s_gl[63] - gli));
    uint4 sh[8], sl[8];  // this thread's share of S for <S, dS'>, before dS' takes its place
    ok = ok && mbar_wait(bar_s, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sh[i] = *reinterpret_cast<const uint4*>(sm + kGS + (tid + 256 * i) * 16);
        sl[i] = *reinterpret_cast<const uint4*>(sm + kGS + 32768 + (tid + 256 * i) * 16);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_read);
    uint32_t pdh[8], pdl[8], gh[8], gl[8];
    float db = 0.f;
    ok = ok && mbar_wait(bar_m, 0);
    fence_after_sync();
    {
        float x[16], y[16], z[16], v[16];
        tmem_ld16_pair<32>(tl + 256 + 16 * hw, x);
        tmem_ld16_pair<32>(tl + 320 + 16 * hw, y);
        tmem_ld16_pair<32>(tl + 384 + 16 * hw, z);
        tmem_ld16_pair<32>(tl + 448 + 16 * hw, v);
        tmem_wait_ld();
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            const int j = j0 + m;
            const float D = ex2_approx((gi - s_g[j]) + (gli - s_gl[j]));
            if (j == r) s_pd[r] = r < L ? x[m] : 0.f;
            x[m] = (j < r && r < L) ? x[m] * D : 0.f;
            const float e = (j < r && r < L) ? -y[m] * D : 0.f;
            db = fmaf(e, z[m], db);
            if (j == r) db += v[m];
            y[m] = bi * e;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            split2(x[2 * m], x[2 * m + 1], pdh[m], pdl[m]);
            split2(y[2 * m], y[2 * m + 1], gh[m], gl[m]);
        }
    }
    float rq[32], ra[32];
    float kt = 0.f;
    ok = ok && mbar_wait(bar_m + 8, 0);
    fence_after_sync();
    if (warp == 0) {  // S is consumed
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_read, 0));
        if (ok && elect_one()) {
            mbar_arrive_expect_tx(bar_ds, 65536);
            bulk_g2s(sb + kGS, img + kImgDs, 65536, bar_ds);
            if (blockIdx.x + kGAhead < gridDim.x) {  // L2 takes what the unit that runs here next starts on
                bulk_prefetch(img + (size_t)kGAhead * kImages + kImgS, 65536);
                bulk_prefetch(img + (size_t)kGAhead * kImages + kImgU, 65536);
            }
        }
        __syncwarp();
    }
    grad_ld32(tl + 32 * hw, rq);
    grad_ld32(tl + 128 + 32 * hw, ra);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float k8[8];
        unpack8(*reinterpret_cast<const uint4*>(sm + kGK + sw128_chunk_off(r, (c0 >> 3) + b, 64)), k8);
#pragma unroll
        for (int e = 0; e < 8; ++e) kt = fmaf(k8[e], ra[8 * b + e], kt);
    }
#pragma unroll
    for (int m = 0; m < 32; ++m) {
        rq[m] *= gam;
        ra[m] *= -gam * bi;
    }
    db -= gam * kt;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t o = sw128_chunk_off(r, (j0 >> 3) + b, 64);
        *reinterpret_cast<uint4*>(sm + kGPd + o) = make_uint4(pdh[4 * b], pdh[4 * b + 1], pdh[4 * b + 2], pdh[4 * b + 3]);
        *reinterpret_cast<uint4*>(sm + kGPd + 8192 + o) = make_uint4(pdl[4 * b], pdl[4 * b + 1], pdl[4 * b + 2], pdl[4 * b + 3]);
        *reinterpret_cast<uint4*>(sm + kGG + o) = make_uint4(gh[4 * b], gh[4 * b + 1], gh[4 * b + 2], gh[4 * b + 3]);
        *reinterpret_cast<uint4*>(sm + kGG + 8192 + o) = make_uint4(gl[4 * b], gl[4 * b + 1], gl[4 * b + 2], gl[4 * b + 3]);
    }
    fence_proxy_async();
    fence_before_sync();
    ok = __syncthreads_and(ok);
    if (warp == 0) {
        fence_after_sync();
        if (ok && elect_one()) {
            const uint64_t kP = desc_kmajor(sb + kGPd, 64, 0), kG = desc_kmajor(sb + kGG, 64, 0),
                           mP = desc_mnmajor(sb + kGPd, 64, 0), mG = desc_mnmajor(sb + kGG, 64, 0),
                           mK = desc_mnmajor(sb + kGK, 64, 0), mQ = desc_mnmajor(sb + kGQ, 64, 0);
            const uint32_t kn = idesc_bf16(64, 128, false, true), mn = idesc_bf16(64, 128, true, true);
            constexpr uint64_t lo = 8192 >> 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t km = (uint64_t)((k * 32) >> 4), mm = (uint64_t)((k * 2048) >> 4);
                mma_bf16(tmem + 128, kP + km, mK + mm, kn, k > 0);
                mma_bf16(tmem + 128, kP + lo + km, mK + mm, kn, 1);
                mma_bf16(tmem + 256, kG + km, mK + mm, kn, k > 0);
                mma_bf16(tmem + 256, kG + lo + km, mK + mm, kn, 1);
                mma_bf16(tmem + 384, mP + mm, mQ + mm, mn, k > 0);
                mma_bf16(tmem + 384, mP + lo + mm, mQ + mm, mn, 1);
                mma_bf16(tmem + 384, mG + mm, mK + mm, mn, 1);
                mma_bf16(tmem + 384, mG + lo + mm, mK + mm, mn, 1);
            }
            mma_commit(bar_m + 16);
        }
        __syncwarp();
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_ds, 0));
        if (ok && elect_one()) {
            const uint32_t mn = idesc_bf16(64, 128, true, true);
            constexpr uint64_t loU = 16384 >> 4, loS = 32768 >> 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t im = (uint64_t)((k * 256) >> 4);
                mma_bf16(tmem, iU + im, iS + im, mn, k > 0);
                mma_bf16(tmem, iU + loU + im, iS + im, mn, 1);
                mma_bf16(tmem, iU + im, iS + loS + im, mn, 1);
            }
            mma_commit(bar_m + 24);
        }
        __syncwarp();
    }
    ok = ok && mbar_wait(bar_ds, 0);
    float sds = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a[8], b[8], c[8], e[8];
        unpack8(sh[i], a);
        unpack8(sl[i], b);
        unpack8(*reinterpret_cast<const uint4*>(sm + kGS + (tid + 256 * i) * 16), c);
        unpack8(*reinterpret_cast<const uint4*>(sm + kGS + 32768 + (tid + 256 * i) * 16), e);
#pragma unroll
        for (int m = 0; m < 8; ++m) sds = fmaf(a[m] + b[m], c[m] + e[m], sds);
    }
    ok = ok && mbar_wait(bar_m + 16, 0);
    fence_after_sync();
    const bool row = r < L && c0 < dkw && ok;
    const size_t orow = ((size_t)(t0 + r) * H + h) * dkw + c0;
    const float pd = s_pd[r];
    float dot = 0.f;
    {
        float x[32];
        grad_ld32(tl + 128 + 32 * hw, x);
#pragma unroll
        for (int m = 0; m < 32; ++m) rq[m] += x[m];
        grad_ld32(tl + 256 + 32 * hw, x);
#pragma unroll
        for (int m = 0; m < 32; ++m) ra[m] += x[m];
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float q8[8], k8[8];
        unpack8(*reinterpret_cast<const uint4*>(sm + kGQ + sw128_chunk_off(r, (c0 >> 3) + b, 64)), q8);
        unpack8(*reinterpret_cast<const uint4*>(sm + kGK + sw128_chunk_off(r, (c0 >> 3) + b, 64)), k8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dot = fmaf(q8[e], rq[8 * b + e], dot);
            dot = fmaf(k8[e], ra[8 * b + e], dot);
            rq[8 * b + e] = fmaf(pd, k8[e], rq[8 * b + e]);
        }
        if (row) {
            if (dq_acc) {
                *reinterpret_cast<float4*>(dq_acc + orow + 8 * b) = make_float4(rq[8 * b], rq[8 * b + 1], rq[8 * b + 2], rq[8 * b + 3]);
                *reinterpret_cast<float4*>(dq_acc + orow + 8 * b + 4) = make_float4(rq[8 * b + 4], rq[8 * b + 5], rq[8 * b + 6], rq[8 * b + 7]);
            } else {
                *reinterpret_cast<uint4*>(dq + orow + 8 * b) = pack8(rq + 8 * b);
            }
        }
    }
    ok = ok && mbar_wait(bar_m + 24, 0);
    fence_after_sync();
    float kw = 0.f;
    {
        float x[32], y[32];
        grad_ld32(tl + 32 * hw, x);
        grad_ld32(tl + 384 + 32 * hw, y);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float q8[8], k8[8];
            unpack8(*reinterpret_cast<const uint4*>(sm + kGQ + sw128_chunk_off(r, (c0 >> 3) + b, 64)), q8);
            unpack8(*reinterpret_cast<const uint4*>(sm + kGK + sw128_chunk_off(r, (c0 >> 3) + b, 64)), k8);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int m = 8 * b + e;
                const float a = wi * x[m];
                kw = fmaf(k8[e], a, kw);
                dot = fmaf(-k8[e], y[m], dot);
                ra[m] += fmaf(pd, q8[e], a + y[m]);
            }
            if (row && ok) {
                if (dk_acc) {
                    *reinterpret_cast<float4*>(dk_acc + orow + 8 * b) = make_float4(ra[8 * b], ra[8 * b + 1], ra[8 * b + 2], ra[8 * b + 3]);
                    *reinterpret_cast<float4*>(dk_acc + orow + 8 * b + 4) = make_float4(ra[8 * b + 4], ra[8 * b + 5], ra[8 * b + 6], ra[8 * b + 7]);
                } else {
                    *reinterpret_cast<uint4*>(dk + orow + 8 * b) = pack8(ra + 8 * b);
                }
            }
        }
    }
    s_red[part * 64 + r] = dot;
    s_red[256 + part * 64 + r] = kw;
    s_red[512 + part * 64 + r] = db;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sds += __shfl_xor_sync(0xffffffffu, sds, o);
    if (lane == 0) s_sds[warp] = sds;
    fence_before_sync();
    ok = __syncthreads_and(ok);
    if (!ok && warp == 0) {  // no copy outlives the CTA
        (void)mbar_wait(bar_in, 0);
        (void)mbar_wait(bar_s, 0);
        (void)mbar_wait(bar_ds, 0);
    }
    if (warp == 2) tmem_dealloc(tmem, 512);
    if (warp == 0 && ok) {
        auto sum4 = [&](int k, int i) {
            const float* p = s_red + 256 * k + i;
            return (p[0] + p[64]) + (p[128] + p[192]);
        };
        // dlog_alpha_i = sum of dot_m over m >= i  +  sum of kw_m over m < i  +  2^g_C <S, dS'>
        const float a0 = sum4(0, 2 * lane), a1 = sum4(0, 2 * lane + 1), k0 = sum4(1, 2 * lane), k1 = sum4(1, 2 * lane + 1);
        float s = a0 + a1, c = k0 + k1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, s, o), z = __shfl_up_sync(0xffffffffu, c, o);
            if (lane + o < 32) s += y;
            if (lane >= o) c += z;
        }
        float behind = __shfl_down_sync(0xffffffffu, s, 1), ahead = __shfl_up_sync(0xffffffffu, c, 1);
        if (lane == 31) behind = 0.f;
        if (lane == 0) ahead = 0.f;
        float end = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) end += s_sds[i];
        end *= ex2_approx(s_g[63]);
        const size_t o = (size_t)(t0 + 2 * lane) * H + h;
        const bool on_zero = !start && lane == 0 && t0 == (cu ? (long long)cu[n] : (long long)n * Tseq);
        if (2 * lane < L) {
            dla[o] = on_zero ? 0.f : (s + ahead) + end;
            dbeta[o] = sum4(2, 2 * lane);
        }
        if (2 * lane + 1 < L) {
            dla[o + H] = (behind + a1) + (ahead + k0) + end;
            dbeta[o + H] = sum4(2, 2 * lane + 1);
        }
    }
}

// dq and dk of a q/k head from its G value heads, in head order: rows of 4 * w channels, 16 bytes a thread.
// A stream of fp32 rows: 33 us for 8192 tokens x 16 value heads.
__global__ void __launch_bounds__(256)
gdn_bwd_heads_kernel(const float* __restrict__ dq_acc, const float* __restrict__ dk_acc, __nv_bfloat16* __restrict__ dq,
                     __nv_bfloat16* __restrict__ dk, long long quads, int G, int w, const WsHeader* __restrict__ hdr,
                     const int32_t* __restrict__ cu)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads || (cu && hdr->bad)) return;
    const long long row = i / w;
    const int c = (int)(i - row * w);
    const float4* acc = reinterpret_cast<const float4*>(blockIdx.y ? dk_acc : dq_acc) + row * G * w + c;
    float4 s = __ldcs(acc);
    for (int g = 1; g < G; ++g) {
        const float4 x = __ldcs(acc + (size_t)g * w);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    reinterpret_cast<uint2*>(blockIdx.y ? dk : dq)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// bytes behind the header and the chunk table: slots, backward slots, images, segment states (forward,
// transition, reverse), and with shared q/k heads fp32 dq, dk
struct BwdLayout {
    size_t slots, bslots, images, segs, seg_bytes, dq, dk, total;
};
inline BwdLayout bwd_layout(int max_chunks, int N, long long Ttot, int H, int dk, bool grouped)
{
    BwdLayout l;
    const long long units = (long long)max_chunks * H;
    l.slots = 0;
    l.bslots = l.slots + (size_t)units * kSlot;
    l.images = l.bslots + (size_t)units * kBwdSlot;
    l.segs = l.images + (size_t)units * kImages;
    l.seg_bytes = segments_bytes(max_chunks, N, H, true);
    l.dq = l.segs + 3 * l.seg_bytes;
    const size_t acc = grouped ? (size_t)Ttot * H * dk * sizeof(float) : 0;
    l.dk = l.dq + acc;
    l.total = l.dk + acc;
    return l;
}

inline cudaError_t launch_bwd(const void* q, const void* k, const void* v, const float* la, const float* beta,
                              const float* S0, const void* dout, const float* dS_final, void* dq, void* dk, void* dv,
                              float* dla, float* dbeta, float* dS0, const WsHeader* hdr, const int* off,
                              const int32_t* cu, int Tseq, int N, int H, int Hk, int dkw, int dvw, int max_chunks,
                              long long Ttot, uint8_t* ws, cudaStream_t stream)
{
    alignas(64) CUtensorMap tq{}, tk{}, tv{}, tdo{};
    const long long units = (long long)max_chunks * H;
    if (units > 0x7fffffffLL || 3 * ((long long)max_chunks + N) * H > 0x7fffffffLL) return cudaErrorInvalidValue;
    const bool grouped = Hk != H;
    const BwdLayout lay = bwd_layout(max_chunks, N, Ttot, H, dkw, grouped);
    uint8_t *slots = ws + lay.slots, *bslots = ws + lay.bslots, *images = ws + lay.images;
    const int len = Ttot > 0 ? segment_length(max_chunks, N, H, true) : 0;
    float* segs = (float*)(ws + lay.segs);
    const Segments fwd{len, segs, (float*)((uint8_t*)segs + lay.seg_bytes)};
    const Segments rev{len, (float*)((uint8_t*)segs + 2 * lay.seg_bytes), fwd.M};
    const ChainArgs ca{hdr, off, cu, Tseq, N, H, H / Hk, dkw, dvw, slots};
    float *dq_acc = grouped ? (float*)(ws + lay.dq) : nullptr, *dk_acc = grouped ? (float*)(ws + lay.dk) : nullptr;
    cudaError_t e = cudaSuccess;
    if (Ttot > 0) {
        if (!make_map(&tq, q, Hk, dkw, Ttot) || !make_map(&tk, k, Hk, dkw, Ttot) || !make_map(&tv, v, H, dvw, Ttot) ||
            !make_map(&tdo, dout, H, dvw, Ttot))
            return cudaErrorInvalidValue;
        e = launch_prep<true>(tq, tk, la, beta, hdr, off, cu, Tseq, N, H, Hk, units, slots, bslots, stream);
        if (e != cudaSuccess) return e;
    }
    constexpr uint32_t kSmem = kRSmem > Chain<kChainStates>::Smem ? kRSmem : Chain<kChainStates>::Smem;
    e = cudaFuncSetAttribute(gdn_bwd_chains_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(gdn_bwd_chains_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int nr = (int)(max_segments(max_chunks, N, len) * H);
    if (len) {
        {
            LaunchScope ls("gdn_bwd_ends", stream);
            gdn_bwd_chains_kernel<true><<<3 * nr, kRThreads, kSmem, stream>>>(tk, tv, tdo, S0, dS_final, nullptr, nullptr, ca,
                                                                            bslots, nullptr, fwd, rev, nr);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        if ((e = launch_join(ca, fwd, &rev, stream)) != cudaSuccess) return e;
    }
    {
        LaunchScope ls("gdn_bwd_chains", stream);
        gdn_bwd_chains_kernel<false><<<2 * nr, kRThreads, kSmem, stream>>>(tk, tv, tdo, S0, dS_final, dS0, (__nv_bfloat16*)dv,
                                                                         ca, bslots, images, fwd, rev, nr);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (Ttot == 0) return cudaSuccess;
    e = cudaFuncSetAttribute(gdn_bwd_grads_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
    if (e != cudaSuccess) return e;
    {
        LaunchScope ls("gdn_bwd_grads", stream);
        gdn_bwd_grads_kernel<<<(unsigned)units, kGThreads, kGSmem, stream>>>(
            tq, tk, tv, tdo, la, beta, (__nv_bfloat16*)dq, (__nv_bfloat16*)dk, dq_acc, dk_acc, dla, dbeta, hdr, off, cu,
            Tseq, N, H, H / Hk, dkw, S0 != nullptr, images);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (grouped) {
        LaunchScope ls("gdn_bwd_heads", stream);
        const long long quads = Ttot * Hk * (dkw / 4), blocks = (quads + 255) / 256;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        gdn_bwd_heads_kernel<<<dim3((unsigned)blocks, 2), 256, 0, stream>>>(
            dq_acc, dk_acc, (__nv_bfloat16*)dq, (__nv_bfloat16*)dk, quads, H / Hk, dkw / 4, hdr, cu);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace gdn
}  // namespace kda
