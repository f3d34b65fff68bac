// Internal declarations of linear attention with one decay a head,
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_t = exp(log_alpha_t),
// shared by its CUDA sources (not part of the ABI).
#pragma once

#include "kda_internal.cuh"

namespace kda {

// The decay argument: one log decay per token and head in the inputs' dtype, or one
// per head in fp32.
struct LinDecay {
    const void* la;
    int per_head;
};

template <typename Tin>
__device__ __forceinline__ float lin_raw_decay(const LinDecay& d, size_t tok, int H, int h) {
    return d.per_head ? reinterpret_cast<const float*>(d.la)[h]
                      : to_f32(reinterpret_cast<const Tin*>(d.la)[tok * (size_t)H + h]);
}
// A NaN passes the floor (fmaxf would take it for a reset); the sums in fixed point, which have
// none, pass it on by themselves.
template <typename Tin>
__device__ __forceinline__ float lin_log_decay(const LinDecay& d, size_t tok, int H, int h) {
    const float x = lin_raw_decay<Tin>(d, tok, H, h);
    return x < kLogAlphaFloor ? kLogAlphaFloor : x;
}

// ---- CUDA-core path (fp32 inputs, or a width of 64): 64-token chunks -------------
constexpr int kLinSimtChunk = 64;

struct LinSimtWorkspace {
    float* S;       // [chunks, H, dk, dv] each chunk's update, then its start state
    float* dS;      // [chunks, H, dk, dv] (backward) the same for the reversed chain: gradient of the end state
    float* gam;     // [chunks, H] a chunk's whole decay
    float* parts;   // (backward) [chunks, H] x (3 x 64 + 1) what dlog_alpha is put together from
};

cudaError_t launch_lin_simt_fwd(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                                const float* init_state, void* o, float* final_state, const ChunkMap& cmap,
                                const SeqMap& smap, int n_chunks, int n_seqs, int H, int dk, int dv,
                                const LinSimtWorkspace& ws, cudaStream_t stream);

cudaError_t launch_lin_simt_bwd(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                                const float* init_state, const void* d_o, const float* d_final, void* dq, void* dk_out,
                                void* dv_out, void* dla, float* d_init, const ChunkMap& cmap, const SeqMap& smap,
                                int n_chunks, int n_seqs, int H, int dk, int dv, const LinSimtWorkspace& ws,
                                cudaStream_t stream);

cudaError_t launch_lin_decode(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                              float* state, int N, int H, int dk, int dv, void* o, cudaStream_t stream);

// ---- tensor-core path (bf16, 128 x 128): 128-token chunks, walked in segments ------
constexpr int kLinTcChunk = 128;

// Nanoseconds after which an extra wait in the first block of each kernel runs out; 0: none
// (kda_set_test_wait_limit).
struct TestStall {
    unsigned long long walk = 0, state = 0, grad = 0;
};

// `segs` / `smap` number segments of segs.C tokens as the CUDA-core path numbers chunks.
// With `split` the segments' own sums come first (seg_state [segments, H, dk, dv], seg_gam
// [segments, H]) and are chained into start states.  BV: value columns a block, 128 or 64.
cudaError_t launch_lin_tc_fwd(const void* q, const void* k, const void* v, LinDecay dec, const float* init_state,
                              void* o, float* final_state, const ChunkMap& segs, const SeqMap& smap, int n_segs,
                              int n_seqs, bool split, int BV, long long tokens, int H, float* seg_state,
                              float* seg_gam, int* err, TestStall stall, cudaStream_t stream);
// Backward, two parts.  States: the bf16 images of every chunk's start state and of its end
// state's gradient, [chunk image, H] x 32 KB, and d_init (seg_state and seg_gam hold both
// directions, one behind the other).  Gradients: everything else, from the images.
cudaError_t launch_lin_tc_states(const void* q, const void* k, const void* v, const void* d_o, LinDecay dec,
                                 const float* init_state, const float* d_final, float* d_init, const ChunkMap& segs,
                                 const SeqMap& smap, int n_segs, int n_seqs, bool split, long long tokens, int H,
                                 float* seg_state, float* seg_gam, uint8_t* images, uint8_t* d_images, int* err,
                                 TestStall stall, cudaStream_t stream);
cudaError_t launch_lin_tc_grad(const void* q, const void* k, const void* v, const void* d_o, LinDecay dec, void* dq,
                               void* dk, void* dv, void* dla, const ChunkMap& chunks, int n_chunks, long long tokens,
                               int H, const uint8_t* images, const uint8_t* d_images, int* err, TestStall stall,
                               cudaStream_t stream);

// end = start (or 0) for n sequences without tokens from rank `first` of smap on
cudaError_t launch_lin_empty_states(const float* start, float* end, const SeqMap& smap, int first, int n, int H,
                                    cudaStream_t stream);

}  // namespace kda
