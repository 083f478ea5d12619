// gdn.cuh -- the gated delta rule with one forget gate a head, on the CUDA-core chunk kernels.
//
// fp32 inputs run there, in instances of the per-channel form's kernels that take the decays of a head in place of
// the channels' (head_gate.cuh).  The backward leaves the gate's gradient for each key channel; their sum is here.
// A call of a few hundred tokens is a chain of launches (61 us the prefill, 149 us the backward).
#pragma once

#include "common.cuh"
#include "profile.cuh"

namespace kda {

// One warp per (token, head): the sum over its dk channels, in a fixed order.  Without a start state the first
// gate of a sequence multiplies zeros: its gradient is zero, where the channels hold the rounding of terms that
// cancel.  Malformed offsets: nothing is written.
__global__ void __launch_bounds__(256)
gdn_sum_gate_kernel(const float* __restrict__ dla, float* __restrict__ out, long long rows, int dk, int H,
                    const WsHeader* __restrict__ hdr, const int32_t* __restrict__ cu, int Tseq, int N, bool start)
{
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows || (cu && hdr->bad)) return;
    if (!start) {
        const long long t = r / H;
        bool first;
        if (cu) {  // is t one of the offsets?
            int lo = 0, hi = N;  // the first i with cu[i] >= t; cu[N] is past every token
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] < t) lo = mid + 1; else hi = mid;
            }
            first = cu[lo] == t;
        } else {
            first = t % Tseq == 0;
        }
        if (first) {
            if (lane == 0) out[r] = 0.f;
            return;
        }
    }
    float s = 0.f;
    for (int c = lane; c < dk; c += 32) s += dla[r * dk + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) out[r] = s;
}

inline cudaError_t launch_gdn_sum_gate(const float* dla, float* out, long long rows, int dk, int H, const WsHeader* hdr,
                                       const int32_t* cu, int Tseq, int N, bool start, cudaStream_t stream)
{
    LaunchScope ls("gdn_sum_gate", stream);
    const long long blocks = (rows + 7) / 8;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    gdn_sum_gate_kernel<<<(unsigned)blocks, 256, 0, stream>>>(dla, out, rows, dk, H, hdr, cu, Tseq, N, start);
    return cudaGetLastError();
}

}  // namespace kda
