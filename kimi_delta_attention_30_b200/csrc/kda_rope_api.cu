// Host side of the query/key norm with rotation (kda_qk_norm_rope* in include/kda.h):
// argument checks and dispatch.
#include "kda_host.cuh"
#include "kda_rope.cuh"

namespace kda {
namespace {

// Rows that are only read: 16-byte aligned starts, no negative strides.
kda_status check_in(const kda_rows* x, size_t elem) {
    if (!x || !x->data) return KDA_ERR_NULL;
    if (x->token_stride < 0 || x->head_stride < 0) return KDA_ERR_SHAPE;
    if (!aligned16(x->data) || (size_t)x->token_stride * elem % 16 || (size_t)x->head_stride * elem % 16)
        return KDA_ERR_ALIGN;
    return KDA_OK;
}

// Rows that are written: besides, no two of them share an element (token-major or
// head-major order, gaps allowed).
kda_status check_out(const kda_rows* x, size_t elem, long long T, int H, int d) {
    const kda_status st = check_in(x, elem);
    if (st != KDA_OK) return st;
    const long long t = x->token_stride, h = x->head_stride;
    // `steps` strides of `inner` and a row fit into `outer` (without forming the product, which could overflow)
    auto fits = [&](long long outer, long long inner, long long steps) {
        return outer >= d && (steps == 0 || (inner >= d && (outer - d) / steps >= inner));
    };
    const bool token_major = T == 1 ? H == 1 || h >= d : fits(t, h, H - 1);
    const bool head_major = H == 1 ? T == 1 || t >= d : fits(h, t, T - 1);
    return token_major || head_major ? KDA_OK : KDA_ERR_SHAPE;
}

// A result in its input's own memory: the rows have to be the same ones.
kda_status check_in_place(const kda_rows* in, const kda_rows* out, long long T, int H) {
    if (in->data != out->data) return KDA_OK;
    return (T == 1 || in->token_stride == out->token_stride) && (H == 1 || in->head_stride == out->head_stride)
               ? KDA_OK
               : KDA_ERR_SHAPE;
}

kda_status check_sizes(kda_dtype dtype, kda_dtype wdtype, long long T, int Hq, int Hk, int d, int rot, float eps) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (wdtype != KDA_BF16 && wdtype != KDA_F32) return KDA_ERR_DTYPE;
    if (T < 0 || T > 0x7fffffffLL || Hq <= 0 || Hk <= 0 || Hq > 65535 || Hk > 65535) return KDA_ERR_SHAPE;
    if (d != 64 && d != 128) return KDA_ERR_SHAPE;
    if (rot < 0 || rot > d || rot % 16 != 0) return KDA_ERR_SHAPE;
    if (!(eps >= 0.f)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status first_error(const kda_status* st, int n) {
    for (int i = 0; i < n; ++i)
        if (st[i] != KDA_OK) return st[i];
    return KDA_OK;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_qk_norm_rope(const kda_rows* q, const kda_rows* k, const void* q_weight, const void* k_weight,
                            kda_dtype weight_dtype, const int32_t* positions, const float* inv_freq, kda_dtype dtype,
                            long long T, int Hq, int Hk, int d, int rot, float eps, int interleaved,
                            const kda_rows* q_out, const kda_rows* k_out, void* stream) {
    kda_status st = check_sizes(dtype, weight_dtype, T, Hq, Hk, d, rot, eps);
    if (st != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    const size_t e = dtype == KDA_F32 ? 4 : 2;
    const kda_status each[4] = {check_in(q, e), check_in(k, e), check_out(q_out, e, T, Hq, d),
                                check_out(k_out, e, T, Hk, d)};
    if ((st = first_error(each, 4)) != KDA_OK) return st;
    const kda_status place[2] = {check_in_place(q, q_out, T, Hq), check_in_place(k, k_out, T, Hk)};
    if ((st = first_error(place, 2)) != KDA_OK) return st;
    if (rot > 0 && (!positions || !inv_freq)) return KDA_ERR_NULL;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) || !aligned4(positions) ||
        !aligned4(inv_freq))
        return KDA_ERR_ALIGN;
    if ((st = check_device()) != KDA_OK) return st;
    NormRopeArgs A{};
    A.q = NormRopeSide{q->data, nullptr, q_out->data, q_weight, q->token_stride, q->head_stride, 0, 0,
                       q_out->token_stride, q_out->head_stride};
    A.k = NormRopeSide{k->data, nullptr, k_out->data, k_weight, k->token_stride, k->head_stride, 0, 0,
                       k_out->token_stride, k_out->head_stride};
    A.positions = positions;
    A.inv_freq = inv_freq;
    A.T = T;
    A.Hq = Hq;
    A.Hk = Hk;
    A.rot = rot;
    A.eps = eps;
    return launch_norm_rope(dtype, weight_dtype, A, d, interleaved != 0, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

size_t kda_qk_norm_rope_bwd_workspace_size(long long T, int Hq, int Hk, int d, int rot) {
    if (check_sizes(KDA_F32, KDA_F32, T, Hq, Hk, d, rot, 0.f) != KDA_OK) return 0;
    return align_up((size_t)norm_rope_bwd_blocks() * 2 * d * sizeof(float));
}

kda_status kda_qk_norm_rope_bwd(const kda_rows* q, const kda_rows* k, const void* q_weight, const void* k_weight,
                                kda_dtype weight_dtype, const int32_t* positions, const float* inv_freq,
                                kda_dtype dtype, long long T, int Hq, int Hk, int d, int rot, float eps,
                                int interleaved, const kda_rows* d_q_out, const kda_rows* d_k_out, const kda_rows* dq,
                                const kda_rows* dk, void* dq_weight, void* dk_weight, void* workspace,
                                size_t workspace_bytes, void* stream) {
    kda_status st = check_sizes(dtype, weight_dtype, T, Hq, Hk, d, rot, eps);
    if (st != KDA_OK) return st;
    if ((dq_weight && !aligned16(dq_weight)) || (dk_weight && !aligned16(dk_weight))) return KDA_ERR_ALIGN;
    if (T == 0) {   // sums over no rows
        if ((dq_weight || dk_weight) && (st = check_device()) != KDA_OK) return st;
        const size_t wb = (size_t)d * (weight_dtype == KDA_F32 ? 4 : 2);
        for (void* w : {dq_weight, dk_weight})
            if (w && cudaMemsetAsync(w, 0, wb, (cudaStream_t)stream) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const size_t e = dtype == KDA_F32 ? 4 : 2;
    const kda_status each[6] = {check_in(q, e),       check_in(k, e),           check_in(d_q_out, e),
                                check_in(d_k_out, e), check_out(dq, e, T, Hq, d), check_out(dk, e, T, Hk, d)};
    if ((st = first_error(each, 6)) != KDA_OK) return st;
    const kda_status place[4] = {check_in_place(q, dq, T, Hq), check_in_place(d_q_out, dq, T, Hq),
                                 check_in_place(k, dk, T, Hk), check_in_place(d_k_out, dk, T, Hk)};
    if ((st = first_error(place, 4)) != KDA_OK) return st;
    if (rot > 0 && (!positions || !inv_freq)) return KDA_ERR_NULL;
    if (!workspace) return KDA_ERR_WORKSPACE;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) || !aligned4(positions) ||
        !aligned4(inv_freq) || ((uintptr_t)workspace & (kAlign - 1)) != 0)
        return KDA_ERR_ALIGN;
    if (workspace_bytes < kda_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, d, rot)) return KDA_ERR_WORKSPACE;
    if ((st = check_device()) != KDA_OK) return st;
    NormRopeArgs A{};
    A.q = NormRopeSide{q->data, d_q_out->data, dq->data, q_weight, q->token_stride, q->head_stride,
                       d_q_out->token_stride, d_q_out->head_stride, dq->token_stride, dq->head_stride};
    A.k = NormRopeSide{k->data, d_k_out->data, dk->data, k_weight, k->token_stride, k->head_stride,
                       d_k_out->token_stride, d_k_out->head_stride, dk->token_stride, dk->head_stride};
    A.positions = positions;
    A.inv_freq = inv_freq;
    A.T = T;
    A.Hq = Hq;
    A.Hk = Hk;
    A.rot = rot;
    A.eps = eps;
    return launch_norm_rope_bwd(dtype, weight_dtype, A, d, interleaved != 0, (float*)workspace, dq_weight, dk_weight,
                                (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
