// One token of linear attention with one decay a head, the fp32 state updated in place:
//   S = a S + k v^T,   o = S^T q = a S_old^T q + (k . q) v.
//
// Bound by HBM: every state element is read once and written once (8 dk dv bytes against
// 5 dk dv operations): 256 sequences of 32 heads of 128 x 128 take 158 to 165 us, 6.5 to 6.8
// TB/s, the copy rate.  A block owns 32 value columns of one (sequence, head) state; the
// columns are independent of one another, so a single sequence's heads put four times as many
// blocks to work (the cost is the k . q product once per tile).  Blocks with all 128 columns
// took 161 us where this takes 158 (calls back to back) and 162 where this takes 165 (with
// other work between), 16.4 instead of 14.4 us for 16 sequences, 9.7 instead of 10.2 for 8.
// A thread keeps its slice of the state in registers between the read and the write; the
// column sums S^T q meet in shared memory.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int BV = 32;   // value columns a block

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2)
lin_decode_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v, LinDecay dec,
                  float* __restrict__ state, Tin* __restrict__ o, int H) {
    constexpr int V4 = BV / 4;          // float4 per row of the tile
    constexpr int RPP = kThreads / V4;  // rows covered by one pass of the block
    constexpr int NR = DK / RPP;        // rows held by each thread
    static_assert(NR >= 1 && DK % RPP == 0, "tile");
    __shared__ float sk[DK], sq[DK];
    __shared__ __align__(16) float sv[BV];
    __shared__ __align__(16) float red[RPP][BV];
    __shared__ float s_kq;

    const size_t nh = blockIdx.x / (DV / BV);
    const int j0 = (int)(blockIdx.x % (DV / BV)) * BV;
    const int tid = threadIdx.x, col4 = tid % V4, rg = tid / V4;
    float4* S4 = reinterpret_cast<float4*>(state + nh * DK * DV + j0);
    constexpr int LD4 = DV / 4;

    float4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = S4[(rg + i * RPP) * LD4 + col4];
    const float a = expf(lin_log_decay<Tin>(dec, nh / H, H, (int)(nh % H)));
    if (tid < DK) {
        sk[tid] = to_f32(k[nh * DK + tid]);
        sq[tid] = to_f32(q[nh * DK + tid]);
    }
    if (tid < BV) sv[tid] = to_f32(v[nh * DV + j0 + tid]);
    __syncthreads();
    if (tid < 32) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < DK; c += 32) x = fmaf(sk[c + tid], sq[c + tid], x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (tid == 0) s_kq = x;
    }
    const float4 v4 = reinterpret_cast<const float4*>(sv)[col4];
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int c = rg + i * RPP;
        const float qc = sq[c], kc = sk[c];
        s[i].x *= a; s[i].y *= a; s[i].z *= a; s[i].w *= a;
        p.x = fmaf(qc, s[i].x, p.x); p.y = fmaf(qc, s[i].y, p.y);
        p.z = fmaf(qc, s[i].z, p.z); p.w = fmaf(qc, s[i].w, p.w);
        s[i].x = fmaf(kc, v4.x, s[i].x); s[i].y = fmaf(kc, v4.y, s[i].y);
        s[i].z = fmaf(kc, v4.z, s[i].z); s[i].w = fmaf(kc, v4.w, s[i].w);
        S4[c * LD4 + col4] = s[i];
    }
    reinterpret_cast<float4*>(&red[rg][0])[col4] = p;
    __syncthreads();
    if (tid < BV) {
        float x = 0.f;
#pragma unroll
        for (int g = 0; g < RPP; ++g) x += red[g][tid];
        o[nh * DV + j0 + tid] = from_f32<Tin>(fmaf(s_kq, sv[tid], x));
    }
}

template <typename Tin, int DK, int DV>
void run(const void* q, const void* k, const void* v, LinDecay dec, float* state, int N, int H, void* o,
         cudaStream_t stream) {
    const long long nh = (long long)N * H;
    const Tin *Q = (const Tin*)q, *K = (const Tin*)k, *V = (const Tin*)v;
    lin_decode_kernel<Tin, DK, DV><<<(unsigned)(nh * (DV / BV)), kThreads, 0, stream>>>(Q, K, V, dec, state, (Tin*)o, H);
}

template <typename Tin>
cudaError_t pick(const void* q, const void* k, const void* v, LinDecay dec, float* state, int N, int H, int dk, int dv,
                 void* o, cudaStream_t stream) {
    if (dk == 128 && dv == 128) run<Tin, 128, 128>(q, k, v, dec, state, N, H, o, stream);
    else if (dk == 128) run<Tin, 128, 64>(q, k, v, dec, state, N, H, o, stream);
    else if (dv == 128) run<Tin, 64, 128>(q, k, v, dec, state, N, H, o, stream);
    else run<Tin, 64, 64>(q, k, v, dec, state, N, H, o, stream);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_decode(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                              float* state, int N, int H, int dk, int dv, void* o, cudaStream_t stream) {
    return dtype == KDA_F32 ? pick<float>(q, k, v, dec, state, N, H, dk, dv, o, stream)
                            : pick<__nv_bfloat16>(q, k, v, dec, state, N, H, dk, dv, o, stream);
}

}  // namespace kda
