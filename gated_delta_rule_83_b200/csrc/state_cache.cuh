// state_cache.cuh -- fp32 recurrent states quantised into slots of an 8-bit cache, and read back.
//
// A row is the dv values of one (state, head, key channel).  Write: scale = max |row| / 127 and
// code = row / scale rounded to the nearest, ties to even, both quotients IEEE fp32 divisions; so the
// codes are a function of the values alone.  A row of zeros has scale 0 and codes 0; a row that holds
// an infinity or a NaN has scale NaN and codes 0 and reads back as NaN throughout.  int8 rather than an
// 8-bit float: under a row's own scale a uniform step is off by at most max/254, an e4m3 mantissa by up
// to 1/16 of each large value.  Read: value = code * scale.
//
// Both are one streaming pass: 4 + 1 bytes an element.  A thread moves 4 consecutive values of a row
// (16 B fp32, 4 B codes), so every warp-wide access is a run of whole 128-byte lines, and holds 8 rows
// in flight at once to cover the memory latency.
#pragma once

#include "common.cuh"
#include "profile.cuh"

namespace kda {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 8;  // rows in flight per thread

// DV / 4 lanes own a row; a block covers kCacheRows * kCacheThreads * 4 / DV rows of one (state, head).
template <int DV> __host__ __device__ constexpr int cache_block_rows() { return kCacheRows * kCacheThreads * 4 / DV; }

// whether a later entry of `slots` names the same slot: the later one is kept
__device__ __forceinline__ bool slot_superseded(const int32_t* __restrict__ slots, int n, int N, int slot)
{
    bool later = false;
    for (int m = n + 1 + (int)threadIdx.x; m < N; m += kCacheThreads) later |= slots[m] == slot;
    return __syncthreads_or(later) != 0;
}

template <int DV>
__global__ void __launch_bounds__(kCacheThreads)
state_cache_write_kernel(const float* __restrict__ S, int8_t* __restrict__ cache, float* __restrict__ scale,
                         const int32_t* __restrict__ slots, int N, int num_slots, int rows)
{
    const int n = blockIdx.x;
    const int slot = slots[n];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (threadIdx.x == 0) set_error(KDA_ERR_INVALID_ARG);
        return;
    }
    if (slot_superseded(slots, n, N, slot)) return;
    constexpr int LPR = DV / 4, RPB = kCacheThreads / LPR;  // lanes per row, rows per block pass
    const int lane = threadIdx.x % LPR;
    const int r0 = blockIdx.y * cache_block_rows<DV>() + threadIdx.x / LPR;
    const unsigned members = LPR == 32 ? 0xffffffffu : (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    float4 x[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        x[i] = r < rows ? __ldcs(reinterpret_cast<const float4*>(S + ((size_t)n * rows + r) * DV) + lane)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        // |x| as an integer: ordered like the value, infinities above every number, NaN above those
        unsigned m = max(max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu),
                         max(__float_as_uint(x[i].z) & 0x7fffffffu, __float_as_uint(x[i].w) & 0x7fffffffu));
        m = __reduce_max_sync(members, m);
        const bool finite = m < 0x7f800000u;
        const float sc = finite ? __fdiv_rn(__uint_as_float(m), 127.f) : __uint_as_float(0x7fc00000u);
        char4 c = make_char4(0, 0, 0, 0);
        if (finite && sc > 0.f) {  // a denormal scale can leave a quotient above 127: clamped
            c.x = (signed char)fminf(fmaxf(rintf(__fdiv_rn(x[i].x, sc)), -127.f), 127.f);
            c.y = (signed char)fminf(fmaxf(rintf(__fdiv_rn(x[i].y, sc)), -127.f), 127.f);
            c.z = (signed char)fminf(fmaxf(rintf(__fdiv_rn(x[i].z, sc)), -127.f), 127.f);
            c.w = (signed char)fminf(fmaxf(rintf(__fdiv_rn(x[i].w, sc)), -127.f), 127.f);
        }
        if (r < rows) {
            const size_t row = (size_t)slot * rows + r;
            reinterpret_cast<char4*>(cache + row * DV)[lane] = c;
            if (lane == 0) scale[row] = sc;
        }
    }
}

template <int DV>
__global__ void __launch_bounds__(kCacheThreads)
state_cache_read_kernel(const int8_t* __restrict__ cache, const float* __restrict__ scale,
                        const int32_t* __restrict__ slots, float* __restrict__ S, int num_slots, int rows)
{
    const int n = blockIdx.x;
    const int slot = slots[n];
    const bool there = slot >= 0 && slot < num_slots;  // no slot: the zero state of a new sequence
    if (slot >= num_slots && threadIdx.x == 0) set_error(KDA_ERR_INVALID_ARG);
    constexpr int LPR = DV / 4, RPB = kCacheThreads / LPR;
    const int lane = threadIdx.x % LPR;
    const int r0 = blockIdx.y * cache_block_rows<DV>() + threadIdx.x / LPR;
    char4 c[kCacheRows];
    float sc[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        const bool in = there && r < rows;
        const size_t row = in ? (size_t)slot * rows + r : 0;
        c[i] = make_char4(0, 0, 0, 0);
        if (in) c[i] = reinterpret_cast<const char4*>(cache + row * DV)[lane];
        sc[i] = in ? scale[row] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const int r = r0 + i * RPB;
        if (r < rows)
            __stcs(reinterpret_cast<float4*>(S + ((size_t)n * rows + r) * DV) + lane,
                   make_float4((float)c[i].x * sc[i], (float)c[i].y * sc[i], (float)c[i].z * sc[i],
                               (float)c[i].w * sc[i]));
    }
}

inline cudaError_t launch_state_cache_write(const float* S, int8_t* cache, float* scale, const int32_t* slots, int N,
                                            int num_slots, int rows, int dv, cudaStream_t stream)
{
    LaunchScope ls("state_cache_write", stream);
    const int per = dv == 128 ? cache_block_rows<128>() : cache_block_rows<64>();
    const dim3 grid(N, (rows + per - 1) / per);
    if (dv == 128)
        state_cache_write_kernel<128><<<grid, kCacheThreads, 0, stream>>>(S, cache, scale, slots, N, num_slots, rows);
    else
        state_cache_write_kernel<64><<<grid, kCacheThreads, 0, stream>>>(S, cache, scale, slots, N, num_slots, rows);
    return cudaGetLastError();
}

inline cudaError_t launch_state_cache_read(const int8_t* cache, const float* scale, const int32_t* slots, float* S,
                                           int N, int num_slots, int rows, int dv, cudaStream_t stream)
{
    LaunchScope ls("state_cache_read", stream);
    const int per = dv == 128 ? cache_block_rows<128>() : cache_block_rows<64>();
    const dim3 grid(N, (rows + per - 1) / per);
    if (dv == 128)
        state_cache_read_kernel<128><<<grid, kCacheThreads, 0, stream>>>(cache, scale, slots, S, num_slots, rows);
    else
        state_cache_read_kernel<64><<<grid, kCacheThreads, 0, stream>>>(cache, scale, slots, S, num_slots, rows);
    return cudaGetLastError();
}

}  // namespace kda
