// Host side of linear attention with one decay a head (kda_linear_* in include/kda.h):
// argument checks, workspace layout and dispatch.  Nothing here allocates device memory.
#include <algorithm>

#include "kda_host.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace {

struct LinLayout {
    size_t S, dS, gam, total;   // byte offsets in the workspace (SIMT path)
};

LinLayout simt_layout(const Plan& p, int H, int dk, int dv, bool bwd) {
    LinLayout L;
    const size_t ch = (size_t)p.n_chunks * H;
    size_t o = table_bytes(p);
    L.S = o; o = align_up(o + ch * dk * dv * sizeof(float));
    L.dS = o; if (bwd) o = align_up(o + ch * dk * dv * sizeof(float));
    L.gam = o; o = align_up(o + ch * sizeof(float));
    L.total = std::max(o, kAlign);
    return L;
}

kda_status check_decay(kda_decay decay) {
    return decay == KDA_DECAY_TOKEN || decay == KDA_DECAY_HEAD ? KDA_OK : KDA_ERR_SHAPE;
}

// The checks that the chunk calls share; fills the plan.  Grids put heads on y and
// sequence-heads on x.
kda_status plan_for(kda_decay decay, kda_dtype dtype, const int32_t* cu, int n_seqs, int B, int T, int H, int dk,
                    int dv, Plan& p) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    kda_status st = check_decay(decay);
    if (st != KDA_OK) return st;
    st = make_plan(B, T, H, dk, dv, kLinSimtChunk, cu, n_seqs, p);
    if (st != KDA_OK) return st;
    if (H > 65535 || (long long)p.n_seqs * H > 0x7fffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status make_maps(const Plan& p, int T, int C, char* ws, cudaStream_t s, ChunkMap& cmap, SeqMap& smap) {
    const int ncps = (int)(((long long)T + C - 1) / C);
    cmap = ChunkMap{nullptr, p.n_seqs, T, C, ncps};
    smap = SeqMap{nullptr, T, C, ncps};
    if (p.varlen) {
        cudaError_t err;
        upload_tables((SeqInfo*)ws, p.natural, p.by_len, p.n_chunks, C, s, &err);
        if (err != cudaSuccess) return KDA_ERR_CUDA;
        cmap.seqs = (const SeqInfo*)ws;
        cmap.chunks = chunk_table((SeqInfo*)ws, p.n_seqs);
        smap.order = (const SeqInfo*)ws + p.n_seqs;
    }
    return KDA_OK;
}

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return false;
    return true;
}

// A C entry point lets no C++ exception out (the sequence tables are std::vectors).
template <typename F>
kda_status guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return KDA_ERR_CUDA;
    }
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_linear_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype dtype,
                                           const int32_t* cu_seqlens_host, int n_seqs) {
    size_t n = 0;
    guarded([&] {
        Plan p;
        const kda_status st = plan_for(KDA_DECAY_TOKEN, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, p);
        if (st == KDA_OK) n = simt_layout(p, H, dk, dv, false).total;
        return st;
    });
    return n;
}

kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                kda_dtype dtype, const float* init_state, const int32_t* cu_seqlens_host, int n_seqs,
                                int B, int T, int H, int dk, int dv, void* o, float* final_state, void* workspace,
                                size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        Plan p;
        kda_status st = plan_for(decay, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, p);
        if (st != KDA_OK) return st;
        if (p.total_tokens > 0 && (!q || !k || !v || !log_alpha || !o)) return KDA_ERR_NULL;
        if (!workspace) return KDA_ERR_WORKSPACE;
        if (!all_aligned({q, k, v, log_alpha, (const void*)init_state, (const void*)o, (const void*)final_state}) ||
            ((uintptr_t)workspace & (kAlign - 1)) != 0)
            return KDA_ERR_ALIGN;
        const LinLayout L = simt_layout(p, H, dk, dv, false);
        if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
        if ((st = check_device()) != KDA_OK) return st;
        if (p.n_seqs == 0) return KDA_OK;
        cudaStream_t s = (cudaStream_t)stream;
        char* ws = (char*)workspace;
        ChunkMap cmap;
        SeqMap smap;
        if ((st = make_maps(p, T, kLinSimtChunk, ws, s, cmap, smap)) != KDA_OK) return st;
        const LinSimtWorkspace w{(float*)(ws + L.S), nullptr, (float*)(ws + L.gam)};
        const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
        return launch_lin_simt_fwd(dtype, q, k, v, dec, init_state, o, final_state, cmap, smap, p.n_chunks, p.n_seqs,
                                   H, dk, dv, w, s) == cudaSuccess
                   ? KDA_OK
                   : KDA_ERR_CUDA;
    });
}

size_t kda_linear_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype dtype,
                                           const int32_t* cu_seqlens_host, int n_seqs) {
    size_t n = 0;
    guarded([&] {
        Plan p;
        const kda_status st = plan_for(KDA_DECAY_TOKEN, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, p);
        if (st == KDA_OK) n = simt_layout(p, H, dk, dv, true).total;
        return st;
    });
    return n;
}

kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                kda_dtype dtype, const float* init_state, const int32_t* cu_seqlens_host, int n_seqs,
                                int B, int T, int H, int dk, int dv, const void* d_o, const float* d_final_state,
                                void* dq, void* dk_out, void* dv_out, void* dlog_alpha, float* d_init_state,
                                void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        Plan p;
        kda_status st = plan_for(decay, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, p);
        if (st != KDA_OK) return st;
        if (p.total_tokens > 0 && (!q || !k || !v || !log_alpha || !d_o || !dq || !dk_out || !dv_out ||
                                   (decay == KDA_DECAY_TOKEN && !dlog_alpha)))
            return KDA_ERR_NULL;
        if (!workspace) return KDA_ERR_WORKSPACE;
        if (!all_aligned({q, k, v, log_alpha, (const void*)init_state, d_o, (const void*)d_final_state,
                          (const void*)dq, (const void*)dk_out, (const void*)dv_out, (const void*)dlog_alpha,
                          (const void*)d_init_state}) ||
            ((uintptr_t)workspace & (kAlign - 1)) != 0)
            return KDA_ERR_ALIGN;
        const LinLayout L = simt_layout(p, H, dk, dv, true);
        if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
        if ((st = check_device()) != KDA_OK) return st;
        if (p.n_seqs == 0) return KDA_OK;
        cudaStream_t s = (cudaStream_t)stream;
        char* ws = (char*)workspace;
        ChunkMap cmap;
        SeqMap smap;
        if ((st = make_maps(p, T, kLinSimtChunk, ws, s, cmap, smap)) != KDA_OK) return st;
        const LinSimtWorkspace w{(float*)(ws + L.S), (float*)(ws + L.dS), (float*)(ws + L.gam)};
        const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
        return launch_lin_simt_bwd(dtype, q, k, v, dec, init_state, d_o, d_final_state, dq, dk_out, dv_out,
                                   dlog_alpha, d_init_state, cmap, smap, p.n_chunks, p.n_seqs, H, dk, dv, w, s) ==
                       cudaSuccess
                   ? KDA_OK
                   : KDA_ERR_CUDA;
    });
}

kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                  kda_dtype dtype, float* state, int N, int H, int dk, int dv, void* o, void* stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    kda_status st = check_decay(decay);
    if (st != KDA_OK) return st;
    if (N < 0 || H <= 0 || !((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return KDA_ERR_SHAPE;
    if ((long long)N * H > 0x7fffffffLL) return KDA_ERR_SHAPE;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !log_alpha || !state || !o) return KDA_ERR_NULL;
    if (!all_aligned({q, k, v, log_alpha, (const void*)state, (const void*)o})) return KDA_ERR_ALIGN;
    if ((st = check_device()) != KDA_OK) return st;
    const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
    return launch_lin_decode(dtype, q, k, v, dec, state, N, H, dk, dv, o, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
