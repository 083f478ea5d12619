// state_cache.cuh -- fp32 recurrent states quantised into slots of an 8-bit cache, and read back.
//
// A row is the dv values of one (state, head, key channel).  Write: scale = max |row| / 127 and
// code = row / scale rounded to the nearest, ties to even, both quotients IEEE fp32 divisions; so the
// codes are a function of the values alone.  A row of zeros has scale 0 and codes 0; a row that holds
// an infinity or a NaN has scale NaN and codes 0 and reads back as NaN throughout.  int8 rather than an
// 8-bit float: under a row's own scale a uniform step is off by at most max/254, an e4m3 mantissa by up
// to 1/16 of each large value.  Read: value = code * scale.
//
// Both are one streaming pass: 4 + 1 bytes an element.  A thread moves 8 consecutive values of a row (one
// 32-byte access to the fp32 side, 8 bytes of codes) and holds kCacheRows rows in flight to cover the memory
// latency; the state's loads are issued before the slot is known.  Bound by HBM: 192 states of 32 heads,
// d = 128, read back in 67..70 us (0.92..0.96 of the copy bandwidth); 64 written in 37 us (0.70) and read in 28.  A
// writing CTA loads its rows once and leaves, so no load of its own runs under its conversions, and a vote of the
// whole CTA on repeated slots stands between the two; which costs how much is not measured.
#pragma once

#include "common.cuh"
#include "profile.cuh"

namespace kda {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 2;  // rows in flight per thread

// DV / 8 lanes own a row; a block covers so many rows of one state
template <int DV> __host__ __device__ constexpr int cache_block_rows() { return kCacheRows * kCacheThreads * 8 / DV; }

struct Float8 {
    float v[8];
};
__device__ __forceinline__ Float8 ld_stream8(const float* p)
{
    Float8 x;
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(x.v[0]), "=f"(x.v[1]), "=f"(x.v[2]), "=f"(x.v[3]), "=f"(x.v[4]), "=f"(x.v[5]), "=f"(x.v[6]),
                   "=f"(x.v[7])
                 : "l"(p));
    return x;
}
__device__ __forceinline__ void st_stream8(float* p, const Float8& x)
{
    asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x.v[0]), "f"(x.v[1]),
                 "f"(x.v[2]), "f"(x.v[3]), "f"(x.v[4]), "f"(x.v[5]), "f"(x.v[6]), "f"(x.v[7])
                 : "memory");
}

// Eight CTAs an SM (32 registers, 40 bytes spilled): 36.6 us for 64 states of 32 heads where five (43 registers,
// nothing spilled) take 40.3.
template <int DV>
__global__ void __launch_bounds__(kCacheThreads, 8)
state_cache_write_kernel(const float* __restrict__ S, int8_t* __restrict__ cache, float* __restrict__ scale,
                         const int32_t* __restrict__ slots, int N, int num_slots, int rows, int blocks)
{
    const int n = blockIdx.x / blocks, block = blockIdx.x % blocks;
    constexpr int LPR = DV / 8, RPB = kCacheThreads / LPR;  // lanes per row, rows per block pass
    const int lane = threadIdx.x % LPR;
    const int r0 = block * cache_block_rows<DV>() + threadIdx.x / LPR;
    // the slot, the entries behind it and the values are all under way before the first is looked at
    const int slot = slots[n], m0 = n + 1 + (int)threadIdx.x, behind = m0 < N ? slots[m0] : -1;
    Float8 x[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        if (r < rows) x[i] = ld_stream8(S + ((size_t)n * rows + r) * DV + 8 * lane);
    }
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (threadIdx.x == 0) set_error(KDA_ERR_INVALID_ARG);
        return;
    }
    // a later entry names the same slot: that one is kept
    bool later = behind == slot;
    for (int m = m0 + kCacheThreads; m < N; m += kCacheThreads) later |= slots[m] == slot;
    if (__syncthreads_or(later)) return;
    // the lanes of this thread's row
    const unsigned members = LPR == 16 ? 0xffffu << (threadIdx.x & 16) : 0xffu << (threadIdx.x & 24);
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        if (r >= rows) break;
        // |x| as an integer: ordered like the value, infinities above every number, NaN above those
        unsigned m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[i].v[e]) & 0x7fffffffu);
        m = __reduce_max_sync(members, m);
        const bool finite = m < 0x7f800000u;
        const float sc = finite ? __fdiv_rn(__uint_as_float(m), 127.f) : __uint_as_float(0x7fc00000u);
        uint32_t c[2] = {0u, 0u};
        if (finite && sc > 0.f) {
            // The product with the reciprocal is within 127 * 2 * 2^-24 = 1.6e-5 of the quotient, so both round to the
            // same integer unless it is that near a half; only there, and where the scale is a denormal (whose
            // reciprocal may overflow and whose quotients may pass 127), the divisions are made.  Rounding by adding
            // 1.5 * 2^23, whose last bits then hold the integer: conversions run at a quarter of the adds' rate.
            // (64 states of 32 heads: divisions and conversions 45 us.)
            constexpr float kMagic = 12582912.f;
            const float inv = __frcp_rn(sc);
            uint32_t k[8];
            bool divide = sc < 1.17549435e-38f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m2 = fmaf(x[i].v[e], inv, kMagic);
                divide |= !(fabsf(fmaf(x[i].v[e], inv, kMagic - m2)) < 0.4999f);
                k[e] = __float_as_uint(m2);
            }
            if (divide) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    k[e] = __float_as_uint(fminf(fmaxf(__fdiv_rn(x[i].v[e], sc), -127.f), 127.f) + kMagic);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                c[e >> 2] = __byte_perm(__byte_perm(k[e], k[e + 1], 0x0040), __byte_perm(k[e + 2], k[e + 3], 0x0040), 0x5410);
        }
        const size_t row = (size_t)slot * rows + r;
        reinterpret_cast<uint2*>(cache + row * DV)[lane] = make_uint2(c[0], c[1]);
        if (lane == 0) scale[row] = sc;
    }
}

template <int DV>
__global__ void __launch_bounds__(kCacheThreads)
state_cache_read_kernel(const int8_t* __restrict__ cache, const float* __restrict__ scale,
                        const int32_t* __restrict__ slots, float* __restrict__ S, int num_slots, int rows, int blocks)
{
    const int n = blockIdx.x / blocks, block = blockIdx.x % blocks;
    const int slot = slots[n];
    const bool there = slot >= 0 && slot < num_slots;  // no slot: the zero state of a new sequence
    if (slot >= num_slots && threadIdx.x == 0) set_error(KDA_ERR_INVALID_ARG);
    constexpr int LPR = DV / 8, RPB = kCacheThreads / LPR;
    const int lane = threadIdx.x % LPR;
    const int r0 = block * cache_block_rows<DV>() + threadIdx.x / LPR;
    uint2 c[kCacheRows];
    float sc[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        c[i] = make_uint2(0u, 0u);
        sc[i] = 0.f;
        if (there && r < rows) {
            const size_t row = (size_t)slot * rows + r;
            c[i] = reinterpret_cast<const uint2*>(cache + row * DV)[lane];
            sc[i] = scale[row];
        }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        if (r >= rows) break;
        Float8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x.v[e] = (float)(int8_t)((e < 4 ? c[i].x : c[i].y) >> (8 * (e & 3))) * sc[i];
        st_stream8(S + ((size_t)n * rows + r) * DV + 8 * lane, x);
    }
}

inline cudaError_t launch_state_cache_write(const float* S, int8_t* cache, float* scale, const int32_t* slots, int N,
                                            int num_slots, int rows, int dv, cudaStream_t stream)
{
    LaunchScope ls("state_cache_write", stream);
    const int per = dv == 128 ? cache_block_rows<128>() : cache_block_rows<64>();
    const int blocks = (rows + per - 1) / per;
    if ((long long)N * blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(N * blocks);
    if (dv == 128)
        state_cache_write_kernel<128><<<grid, kCacheThreads, 0, stream>>>(S, cache, scale, slots, N, num_slots, rows, blocks);
    else
        state_cache_write_kernel<64><<<grid, kCacheThreads, 0, stream>>>(S, cache, scale, slots, N, num_slots, rows, blocks);
    return cudaGetLastError();
}

inline cudaError_t launch_state_cache_read(const int8_t* cache, const float* scale, const int32_t* slots, float* S,
                                           int N, int num_slots, int rows, int dv, cudaStream_t stream)
{
    LaunchScope ls("state_cache_read", stream);
    const int per = dv == 128 ? cache_block_rows<128>() : cache_block_rows<64>();
    const int blocks = (rows + per - 1) / per;
    if ((long long)N * blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(N * blocks);
    if (dv == 128)
        state_cache_read_kernel<128><<<grid, kCacheThreads, 0, stream>>>(cache, scale, slots, S, num_slots, rows, blocks);
    else
        state_cache_read_kernel<64><<<grid, kCacheThreads, 0, stream>>>(cache, scale, slots, S, num_slots, rows, blocks);
    return cudaGetLastError();
}

}  // namespace kda
