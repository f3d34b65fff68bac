// Internal declarations of the query/key norm with rotation (not part of the ABI).
#pragma once

#include "kda_internal.cuh"

namespace kda {

// One of the two tensors of the call; strides in elements, the last dimension contiguous.
struct NormRopeSide {
    const void* in;      // [T, H, d]
    const void* dy;      // [T, H, d] (backward)
    void* out;           // [T, H, d]: y, or dx
    const void* w;       // [d] or null (ones)
    long long in_tok, in_head, dy_tok, dy_head, out_tok, out_head;
};

struct NormRopeArgs {
    NormRopeSide q, k;
    const int32_t* positions;   // [T]
    const float* inv_freq;      // [rot / 2]
    long long T;
    int Hq, Hk, rot;
    float eps;
    int groups, per;            // warps that share a token's heads, and heads each
};

int norm_rope_bwd_blocks();
cudaError_t launch_norm_rope(kda_dtype dtype, kda_dtype wdtype, NormRopeArgs A, int d, bool interleaved,
                             cudaStream_t stream);
// partial: fp32 [norm_rope_bwd_blocks()][2][d]
cudaError_t launch_norm_rope_bwd(kda_dtype dtype, kda_dtype wdtype, NormRopeArgs A, int d, bool interleaved,
                                 float* partial, void* dwq, void* dwk, cudaStream_t stream);

}  // namespace kda
