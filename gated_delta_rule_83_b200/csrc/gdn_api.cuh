// gdn_api.cuh -- C entry points of the scalar-gate delta rule and of the 8-bit state cache: argument
// validation, workspace carving and dispatch (the end of kda_lib.cu's translation unit).
#pragma once

namespace {

bool gdn_heads_ok(int H, int Hk) { return H > 0 && Hk > 0 && H % Hk == 0; }

// bf16 runs on the tensor cores.  fp32 inputs run on the CUDA-core chunk kernels: split into two bf16 parts they
// would lose eight of their bits.
bool gdn_use_tc(kda_dtype dt) { return dt == KDA_BF16; }

struct GdnFwdPlan {
    Plan f;
    bool tc;
    size_t total;
};

kda_status make_gdn_fwd_plan(int B, int T, int H, int dk, int dv, bool varlen, int num_seqs, kda_dtype dt,
                             GdnFwdPlan& p)
{
    const kda_status st = make_plan(B, T, H, dk, dv, varlen, num_seqs, dt, p.f);
    if (st != KDA_OK) return st;
    p.tc = gdn_use_tc(dt);
    p.total = sizeof(WsHeader) + p.f.off_bytes +
              (p.tc ? gdn::fwd_bytes(p.f.max_chunks, p.f.N, H)
                    : (size_t)p.f.max_chunks * H * round_up(sizeof(float) * simt_slot_floats(dk, dv), kAlign));
    return KDA_OK;
}

struct GdnBwdPlan {
    BwdPlan b;
    bool tc;
    size_t total;  // behind the backward's own (fp32): the gate's gradient for each key channel
};

kda_status make_gdn_bwd_plan(int B, int T, int H, int Hk, int dk, int dv, bool varlen, int num_seqs, kda_dtype dt,
                             GdnBwdPlan& p)
{
    const kda_status st = make_bwd_plan(B, T, H, Hk, 0u, dk, dv, varlen, num_seqs, dt, p.b);
    if (st != KDA_OK) return st;
    p.tc = gdn_use_tc(dt);
    if (p.tc) {
        p.total = sizeof(WsHeader) + p.b.f.off_bytes +
                  gdn::bwd_layout(p.b.f.max_chunks, p.b.f.N, p.b.f.Ttot, H, dk, Hk != H).total;
        return KDA_OK;
    }
    p.total = round_up(p.b.total_bytes, kAlign) + sizeof(float) * (size_t)p.b.f.Ttot * H * dk;
    return KDA_OK;
}

bool all_aligned16(std::initializer_list<const void*> ptrs)
{
    for (const void* x : ptrs)
        if (x && !aligned16(x)) return false;
    return true;
}

}  // namespace

extern "C" kda_status kda_gdn_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int varlen, int num_seqs,
                                                       kda_dtype dt, size_t* bytes)
{
    if (!bytes) return KDA_ERR_INVALID_ARG;
    GdnFwdPlan p;
    const kda_status st = make_gdn_fwd_plan(B, T, H, dk, dv, varlen != 0, num_seqs, dt, p);
    if (st != KDA_OK) return st;
    *bytes = p.total;
    return KDA_OK;
}

extern "C" kda_status kda_gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* log_alpha,
                                        const float* beta, const float* S0, const int32_t* cu_seqlens, int num_seqs,
                                        void* out, float* S_final, int B, int T, int H, int Hk, int dk, int dv,
                                        kda_dtype dt, void* workspace, size_t workspace_bytes, kda_stream_t stream_)
{
    cudaStream_t stream = (cudaStream_t)stream_;
    if (!gdn_heads_ok(H, Hk)) return KDA_ERR_INVALID_ARG;
    GdnFwdPlan p;
    const kda_status st = make_gdn_fwd_plan(B, T, H, dk, dv, cu_seqlens != nullptr, num_seqs, dt, p);
    if (st != KDA_OK) return st;
    if (p.f.Ttot > 0 && (!q || !k || !v || !log_alpha || !beta || !out)) return KDA_ERR_INVALID_ARG;
    if (!all_aligned16({q, k, v, S0, out, S_final}) || ((uintptr_t)log_alpha & 3u) || ((uintptr_t)beta & 3u) ||
        ((uintptr_t)cu_seqlens & 3u))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace % kAlign) || workspace_bytes < p.total) return KDA_ERR_WORKSPACE;
    char* ws = (char*)workspace;
    WsHeader* hdr = (WsHeader*)ws;
    int* off = (int*)(ws + sizeof(WsHeader));
    if (!p.tc || cu_seqlens) {  // the tensor-core kernels derive a regular batch's chunks themselves
        LaunchScope ls("chunk_table", stream);
        chunk_table_kernel<<<1, kTableThreads, 0, stream>>>(cu_seqlens, p.f.N, p.f.Tseq, p.f.Ttot, hdr, off,
                                                            off + p.f.N + 1);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    char* slots = ws + sizeof(WsHeader) + p.f.off_bytes;
    const cudaError_t e =
        p.tc ? gdn::launch_fwd(q, k, v, log_alpha, beta, S0, S_final, out, hdr, off, cu_seqlens, p.f.Tseq, p.f.N, H, Hk, dk,
                               dv, p.f.max_chunks, p.f.Ttot, (uint8_t*)slots, stream)
             : launch_simt_prefill<float, true>(q, k, v, log_alpha, beta, S0, S_final, out, hdr, off, cu_seqlens,
                                                p.f.Tseq, p.f.N, H, Hk, 0u, dk, dv, p.f.max_chunks, (float*)slots, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_gdn_chunk_bwd_workspace_size(int B, int T, int H, int Hk, int dk, int dv, int varlen,
                                                       int num_seqs, kda_dtype dt, size_t* bytes)
{
    if (!bytes || !gdn_heads_ok(H, Hk)) return KDA_ERR_INVALID_ARG;
    GdnBwdPlan p;
    const kda_status st = make_gdn_bwd_plan(B, T, H, Hk, dk, dv, varlen != 0, num_seqs, dt, p);
    if (st != KDA_OK) return st;
    *bytes = p.total;
    return KDA_OK;
}

extern "C" kda_status kda_gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* log_alpha,
                                        const float* beta, const float* S0, const int32_t* cu_seqlens, int num_seqs,
                                        const void* dout, const float* dS_final, void* dq, void* dk_out, void* dv_out,
                                        float* dlog_alpha, float* dbeta, float* dS0, int B, int T, int H, int Hk,
                                        int dk, int dv, kda_dtype dt, void* workspace, size_t workspace_bytes,
                                        kda_stream_t stream_)
{
    cudaStream_t stream = (cudaStream_t)stream_;
    if (!gdn_heads_ok(H, Hk)) return KDA_ERR_INVALID_ARG;
    GdnBwdPlan p;
    const kda_status st = make_gdn_bwd_plan(B, T, H, Hk, dk, dv, cu_seqlens != nullptr, num_seqs, dt, p);
    if (st != KDA_OK) return st;
    const long long Ttot = p.b.f.Ttot;
    if (Ttot > 0 && (!q || !k || !v || !log_alpha || !beta || !dout || !dq || !dk_out || !dv_out || !dlog_alpha ||
                     !dbeta))
        return KDA_ERR_INVALID_ARG;
    if (!all_aligned16({q, k, v, S0, dout, dS_final, dq, dk_out, dv_out, dS0}) || ((uintptr_t)log_alpha & 3u) ||
        ((uintptr_t)beta & 3u) || ((uintptr_t)dlog_alpha & 3u) || ((uintptr_t)dbeta & 3u) ||
        ((uintptr_t)cu_seqlens & 3u))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace % kAlign) || workspace_bytes < p.total) return KDA_ERR_WORKSPACE;
    if (p.tc) {
        const Plan& f = p.b.f;
        char* ws = (char*)workspace;
        WsHeader* hdr = (WsHeader*)ws;
        int* off = (int*)(ws + sizeof(WsHeader));
        if (cu_seqlens) {
            LaunchScope ls("chunk_table", stream);
            chunk_table_kernel<<<1, kTableThreads, 0, stream>>>(cu_seqlens, f.N, f.Tseq, f.Ttot, hdr, off, off + f.N + 1);
            if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
        }
        const cudaError_t e = gdn::launch_bwd(q, k, v, log_alpha, beta, S0, dout, dS_final, dq, dk_out, dv_out, dlog_alpha,
                                              dbeta, dS0, hdr, off, cu_seqlens, f.Tseq, f.N, H, Hk, dk, dv, f.max_chunks, Ttot,
                                              (uint8_t*)(ws + sizeof(WsHeader) + f.off_bytes), stream);
        return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    float* dgate = (float*)((char*)workspace + round_up(p.b.total_bytes, kAlign));
    cudaError_t e = run_backward<float, true>(q, k, v, log_alpha, beta, S0, cu_seqlens, dout, dS_final, dq, dk_out, dv_out,
                                              dgate, dbeta, dS0, H, Hk, 0u, dk, dv, p.b, (char*)workspace, stream);
    if (e == cudaSuccess && Ttot > 0)
        e = launch_gdn_sum_gate(dgate, dlog_alpha, Ttot * H, dk, H, (const WsHeader*)workspace, cu_seqlens, p.b.f.Tseq,
                                p.b.f.N, S0 != nullptr, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_gdn_decode_step(const void* q, const void* k, const void* v, const float* log_alpha,
                                          const float* beta, float* S_inout, void* out, int N, int H, int Hk, int dk,
                                          int dv, kda_dtype dt, kda_stream_t stream_)
{
    cudaStream_t stream = (cudaStream_t)stream_;
    if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (N < 0 || dk <= 0 || dv <= 0 || !gdn_heads_ok(H, Hk)) return KDA_ERR_INVALID_ARG;
    if (!dims_supported(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !log_alpha || !beta || !S_inout || !out) return KDA_ERR_INVALID_ARG;
    if (!all_aligned16({q, k, v, S_inout, out}) || ((uintptr_t)log_alpha & 3u) || ((uintptr_t)beta & 3u))
        return KDA_ERR_INVALID_ARG;
    const cudaError_t e = dt == KDA_BF16
        ? launch_gdn_decode<__nv_bfloat16>(q, k, v, log_alpha, beta, S_inout, out, N, H, Hk, dk, dv, stream)
        : launch_gdn_decode<float>(q, k, v, log_alpha, beta, S_inout, out, N, H, Hk, dk, dv, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

namespace {

kda_status check_cache_args(const void* S, const void* cache, const void* scale, const int32_t* slots, int N,
                            int num_slots, int H, int dk, int dv)
{
    if (N < 0 || num_slots < 0 || H <= 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (!dims_supported(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (H > 65535 || (long long)N * H * dk > (1LL << 32)) return KDA_ERR_UNSUPPORTED;  // rows of a launch
    if (N == 0) return KDA_OK;
    if (!S || !slots || (num_slots > 0 && (!cache || !scale))) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)S & 31u) || ((uintptr_t)cache & 15u) || ((uintptr_t)scale & 3u) || ((uintptr_t)slots & 3u))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_state_cache_write(const float* S, int8_t* cache, float* scale, const int32_t* slots, int N,
                                            int num_slots, int H, int dk, int dv, kda_stream_t stream_)
{
    const kda_status st = check_cache_args(S, cache, scale, slots, N, num_slots, H, dk, dv);
    if (st != KDA_OK || N == 0) return st;
    return launch_state_cache_write(S, cache, scale, slots, N, num_slots, H * dk, dv, (cudaStream_t)stream_) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

extern "C" kda_status kda_state_cache_read(const int8_t* cache, const float* scale, const int32_t* slots, float* S,
                                           int N, int num_slots, int H, int dk, int dv, kda_stream_t stream_)
{
    const kda_status st = check_cache_args(S, cache, scale, slots, N, num_slots, H, dk, dv);
    if (st != KDA_OK || N == 0) return st;
    return launch_state_cache_read(cache, scale, slots, S, N, num_slots, H * dk, dv, (cudaStream_t)stream_) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}
