// head_gate.cuh -- the cumulative gate of a chunk with one forget gate a head, shared by the bf16 and the fp32
// chunk kernels.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace kda {

// g (log2 units, cumulative) and beta of a chunk's 64 tokens into shared memory, by one warp; tokens past
// the chunk's end carry no gate and no weight.  g is summed in 64 bits and kept as hi + lo: behind a token that
// forgets all (log alpha = -100, say) the decays between later tokens are differences of two large g, which
// in 32 bits alone would be off by 1e-5.  A gate below 2^-150 is 2^-150, which rounds every state to zero, so that
// log alpha = -inf needs no care elsewhere.
__device__ __forceinline__ void load_scalars(const float* __restrict__ la, const float* __restrict__ beta, long long t0,
                                             int L, int H, int h, float* s_g, float* s_gl, float* s_b)
{
    const int l = threadIdx.x & 31;
    float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
    if (2 * l < L) {
        a0 = la[(size_t)(t0 + 2 * l) * H + h] * tc::kLog2e;
        b0 = beta[(size_t)(t0 + 2 * l) * H + h];
    }
    if (2 * l + 1 < L) {
        a1 = la[(size_t)(t0 + 2 * l + 1) * H + h] * tc::kLog2e;
        b1 = beta[(size_t)(t0 + 2 * l + 1) * H + h];
    }
    a0 = a0 < -150.f ? -150.f : a0;  // (a NaN stays one)
    a1 = a1 < -150.f ? -150.f : a1;
    double s = (double)a0 + (double)a1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, d);
        if (l >= d) s += y;
    }
    double first = __shfl_up_sync(0xffffffffu, s, 1);
    first = (l == 0 ? 0.0 : first) + (double)a0;
    const float h0 = (float)first, h1 = (float)s;
    *reinterpret_cast<float2*>(s_g + 2 * l) = make_float2(h0, h1);
    *reinterpret_cast<float2*>(s_gl + 2 * l) = make_float2((float)(first - (double)h0), (float)(s - (double)h1));
    *reinterpret_cast<float2*>(s_b + 2 * l) = make_float2(b0, b1);
}

// 2^(g_r - g_i), the decay from token i to token r >= i
__device__ __forceinline__ float head_decay(const float* __restrict__ s_g, const float* __restrict__ s_gl, int r, int i)
{
    return tc::ex2_approx((s_g[r] - s_g[i]) + (s_gl[r] - s_gl[i]));
}

}  // namespace kda
