// RMS norm of every query and key head, then the rotation of its first `rot` channels by
// position, in one pass, and the gradients of both.
//
//   r = 1 / sqrt(mean_c x_c^2 + eps),  y = x r w,  a channel pair (a, b) of y and the
//   angle t = position * inv_freq[pair]:  (a cos t - b sin t, b cos t + a sin t).
// Backward, with g the rotation of dy by -t and h = g w:
//   dw_c = sum over rows of g_c x_c r,   dx = r (h - x r^2 mean_c(h_c x_c)).
//
// Bound by HBM: a row is read once and written once, about ten operations an element.
// One warp takes one token and walks its heads, so the token's rotations are formed once
// (angles in turns in fp64, since a position near 10^6 times a frequency keeps only two
// digits of the angle in fp32; sincospif on the remainder) and stay in registers.  d / 16
// lanes share a row; a lane holds the two 8-channel vectors that rotate with each other
// (halves: vectors p and p + rot / 16; neighbours: vectors 2 p and 2 p + 1), so a rotation
// needs no exchange between lanes, and both loads of a lane are 16 bytes in bf16.
// When there are few tokens a token's heads are split over several warps, which form the
// rotations once each.
#include "kda_rope.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Where a lane's two vectors sit in a row, and whether they rotate.
struct Lane {
    int c0, c1;      // first channels of the two vectors
    bool turns;
    int pair;        // first rotation pair of the lane's eight
};
template <int D>
__device__ __forceinline__ Lane lane_of(int l, int rot, bool interleaved) {
    Lane L;
    const int half = rot / 16;   // pairs of vectors that rotate
    L.turns = l < half;
    L.pair = 8 * l;
    const int v0 = (interleaved || !L.turns) ? 2 * l : l;
    const int v1 = (interleaved || !L.turns) ? 2 * l + 1 : l + half;
    L.c0 = 8 * v0;
    L.c1 = 8 * v1;
    return L;
}

// cos and sin of the lane's eight pairs; (1, 0) where the lane does not rotate
__device__ __forceinline__ void rotations(const NormRopeArgs& A, long long tok, const Lane& L, int lane, int lanes,
                                          float2* cs, float (&co)[8], float (&si)[8]) {
    const int pairs = A.rot / 2;
    if (pairs > 0) {
        const double turns = (double)A.positions[tok] * 0.15915494309189533577;   // 1 / (2 pi)
        for (int i = lane; i < pairs; i += 32) {
            double t = turns * (double)A.inv_freq[i];
            t -= rint(t);
            float s, c;
            sincospif(2.f * (float)t, &s, &c);
            cs[i] = make_float2(c, s);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = L.turns ? cs[L.pair + i] : make_float2(1.f, 0.f);
        co[i] = x.x;
        si[i] = x.y;
    }
    __syncwarp();
}

// (a, b): the two vectors; halves rotate element i of one with element i of the other,
// neighbours rotate elements 2 i and 2 i + 1 of the same vector
template <bool INTER>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&co)[8], const float (&si)[8]) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * co[i] - y * si[i];
            a[2 * i + 1] = y * co[i] + x * si[i];
            b[2 * i] = z * co[4 + i] - w * si[4 + i];
            b[2 * i + 1] = w * co[4 + i] + z * si[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * co[i] - y * si[i];
            b[i] = y * co[i] + x * si[i];
        }
    }
}

// sum over the lanes that share a row
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ float rms_scale(float sum_sq, int d, float eps) {
    return inv_norm_from_sq(fmaf(sum_sq, 1.f / (float)d, eps));   // a zero row with eps = 0 stays zero
}

template <typename Tw>
__device__ __forceinline__ void weights8(const void* w, int c, float (&x)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 1.f;
    } else {
        load8(reinterpret_cast<const Tw*>(w) + c, x);
    }
}

template <typename Tin, typename Tw, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd(const __grid_constant__ NormRopeArgs A) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;   // lanes a row, rows a warp at a time
    __shared__ float2 cs[kWarps][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const long long task = (long long)blockIdx.x * kWarps + warp;
    const long long tok = task / A.groups;
    if (tok >= A.T) return;
    const int heads = A.Hq + A.Hk, per = (heads + A.groups - 1) / A.groups;
    const int h0 = (int)(task % A.groups) * per, h1 = min(heads, h0 + per);
    const Lane L = lane_of<D>(l, A.rot, INTER);
    float co[8], si[8];
    rotations(A, tok, L, lane, LANES, cs[warp], co, si);
#pragma unroll
    for (int side = 0; side < 2; ++side) {   // queries, then keys
        const int b = side ? max(h0, A.Hq) : h0, e = side ? h1 : min(h1, A.Hq);
        if (b >= e) continue;
        const NormRopeSide& X = side ? A.k : A.q;
        const int base = side ? A.Hq : 0;
        float w0[8], w1[8];
        weights8<Tw>(X.w, L.c0, w0);
        weights8<Tw>(X.w, L.c1, w1);
        const Tin* in = reinterpret_cast<const Tin*>(X.in) + tok * X.in_tok;
        Tin* out = reinterpret_cast<Tin*>(X.out) + tok * X.out_tok;
#pragma unroll 2
        for (int h = b - base; h < e - base; h += ROWS) {
            const bool live = h + sub < e - base;
            const Tin* p = in + (long long)(h + (live ? sub : 0)) * X.in_head;
            float a[8], c[8];
            load8(p + L.c0, a);
            load8(p + L.c1, c);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(c[i], c[i], ss));
            const float r = rms_scale(row_sum<LANES>(ss), D, A.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = a[i] * r * w0[i];
                c[i] = c[i] * r * w1[i];
            }
            rotate<INTER>(a, c, co, si);
            if (live) {
                Tin* d = out + (long long)(h + sub) * X.out_head;
                store8(d + L.c0, a);
                store8(d + L.c1, c);
            }
        }
    }
}

// Backward: a block walks tokens blockIdx.x * kWarps + warp, + gridDim.x * kWarps, ...; the
// weight gradients are summed in registers over a lane's rows, then over the block in a
// fixed order, and written as one partial row per block ([grid][2][D] fp32); the second
// kernel adds the partial rows in order, so the result does not depend on timing.
template <typename Tin, typename Tw, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd(const __grid_constant__ NormRopeArgs A,
                                                          float* __restrict__ partial) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    __shared__ float2 cs[kWarps][D / 2];
    __shared__ float acc[kWarps * ROWS][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const Lane L = lane_of<D>(l, A.rot, INTER);
    float g0[2][8], g1[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g0[0][i] = g0[1][i] = g1[0][i] = g1[1][i] = 0.f;
    for (long long tok = (long long)blockIdx.x * kWarps + warp; tok < A.T; tok += (long long)gridDim.x * kWarps) {
        float co[8], si[8];
        rotations(A, tok, L, lane, LANES, cs[warp], co, si);
#pragma unroll
        for (int i = 0; i < 8; ++i) si[i] = -si[i];   // the gradient turns back
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const NormRopeSide& X = side ? A.k : A.q;
            const int H = side ? A.Hk : A.Hq;
            float w0[8], w1[8];
            weights8<Tw>(X.w, L.c0, w0);
            weights8<Tw>(X.w, L.c1, w1);
            const Tin* in = reinterpret_cast<const Tin*>(X.in) + tok * X.in_tok;
            const Tin* dy = reinterpret_cast<const Tin*>(X.dy) + tok * X.dy_tok;
            Tin* out = reinterpret_cast<Tin*>(X.out) + tok * X.out_tok;
            for (int h = 0; h < H; h += ROWS) {
                const bool live = h + sub < H;
                const int hh = h + (live ? sub : 0);
                const Tin *p = in + (long long)hh * X.in_head, *dp = dy + (long long)hh * X.dy_head;
                float a[8], c[8], da[8], dc[8];
                load8(p + L.c0, a);
                load8(p + L.c1, c);
                load8(dp + L.c0, da);
                load8(dp + L.c1, dc);
                rotate<INTER>(da, dc, co, si);
                float ss = 0.f, hx = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(a[i], a[i], fmaf(c[i], c[i], ss));
                    hx = fmaf(da[i] * w0[i], a[i], fmaf(dc[i] * w1[i], c[i], hx));
                }
                const float r = rms_scale(row_sum<LANES>(ss), D, A.eps);
                const float m = row_sum<LANES>(hx) * r * r * r * (1.f / D);
                const float rl = live ? r : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    g0[side][i] = fmaf(da[i] * rl, a[i], g0[side][i]);
                    g1[side][i] = fmaf(dc[i] * rl, c[i], g1[side][i]);
                    a[i] = da[i] * w0[i] * r - a[i] * m;
                    c[i] = dc[i] * w1[i] * r - c[i] * m;
                }
                if (live) {
                    Tin* d = out + (long long)(h + sub) * X.out_head;
                    store8(d + L.c0, a);
                    store8(d + L.c1, c);
                }
            }
        }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
        store8(&acc[warp * ROWS + sub][L.c0], g0[side]);
        store8(&acc[warp * ROWS + sub][L.c1], g1[side]);
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float s = 0.f;
            for (int i = 0; i < kWarps * ROWS; ++i) s += acc[i][c];
            partial[((size_t)blockIdx.x * 2 + side) * D + c] = s;
        }
    }
}

// dw of one side a block row: 32 columns x 8 runs of partial rows
template <typename Tw, int D>
__global__ void __launch_bounds__(256) norm_rope_dw(const float* __restrict__ partial, int n, void* dwq, void* dwk) {
    __shared__ float red[8][33];
    const int side = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    void* out = side ? dwk : dwq;
    if (out == nullptr) return;
    float s = 0.f;
    const int per = (n + 7) / 8;
#pragma unroll 8
    for (int i = run * per; i < min(n, (run + 1) * per); ++i) s += partial[((size_t)i * 2 + side) * D + c];
    red[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x & 31];
        reinterpret_cast<Tw*>(out)[c] = from_f32<Tw>(s);
    }
}

template <typename Tin, typename Tw, int D>
cudaError_t run(const NormRopeArgs& A, bool inter, float* partial, int blocks, void* dwq, void* dwk, cudaStream_t s) {
    if (partial == nullptr) {
        if (inter) norm_rope_fwd<Tin, Tw, D, true><<<blocks, kThreads, 0, s>>>(A);
        else norm_rope_fwd<Tin, Tw, D, false><<<blocks, kThreads, 0, s>>>(A);
    } else {
        if (inter) norm_rope_bwd<Tin, Tw, D, true><<<blocks, kThreads, 0, s>>>(A, partial);
        else norm_rope_bwd<Tin, Tw, D, false><<<blocks, kThreads, 0, s>>>(A, partial);
        if (dwq != nullptr || dwk != nullptr)
            norm_rope_dw<Tw, D><<<dim3(D / 32, 2), 256, 0, s>>>(partial, blocks, dwq, dwk);
    }
    return cudaGetLastError();
}

cudaError_t pick(kda_dtype dtype, kda_dtype wdtype, const NormRopeArgs& A, int d, bool inter, float* partial,
                 int blocks, void* dwq, void* dwk, cudaStream_t s) {
    typedef __nv_bfloat16 bf;
    if (dtype == KDA_F32 && wdtype == KDA_F32)
        return d == 128 ? run<float, float, 128>(A, inter, partial, blocks, dwq, dwk, s)
                        : run<float, float, 64>(A, inter, partial, blocks, dwq, dwk, s);
    if (dtype == KDA_F32)
        return d == 128 ? run<float, bf, 128>(A, inter, partial, blocks, dwq, dwk, s)
                        : run<float, bf, 64>(A, inter, partial, blocks, dwq, dwk, s);
    if (wdtype == KDA_F32)
        return d == 128 ? run<bf, float, 128>(A, inter, partial, blocks, dwq, dwk, s)
                        : run<bf, float, 64>(A, inter, partial, blocks, dwq, dwk, s);
    return d == 128 ? run<bf, bf, 128>(A, inter, partial, blocks, dwq, dwk, s)
                    : run<bf, bf, 64>(A, inter, partial, blocks, dwq, dwk, s);
}

}  // namespace

int norm_rope_bwd_blocks(long long T) {
    const long long want = (T + kWarps - 1) / kWarps;
    return (int)(want < 148 * 4 ? want : 148 * 4);
}

cudaError_t launch_norm_rope(kda_dtype dtype, kda_dtype wdtype, NormRopeArgs A, int d, bool inter,
                             cudaStream_t stream) {
    // enough warps to fill the machine (32 a SM), but at least four rows' loads each
    const int heads = A.Hq + A.Hk, rows = 32 / (d / 16);
    long long groups = (148LL * 32 + A.T - 1) / A.T;
    const int most = (heads + rows - 1) / rows;
    A.groups = (int)(groups < 1 ? 1 : groups > most ? most : groups);
    const long long blocks = (A.T * A.groups + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return pick(dtype, wdtype, A, d, inter, nullptr, (int)blocks, nullptr, nullptr, stream);
}

cudaError_t launch_norm_rope_bwd(kda_dtype dtype, kda_dtype wdtype, const NormRopeArgs& A, int d, bool inter,
                                 float* partial, void* dwq, void* dwk, cudaStream_t stream) {
    return pick(dtype, wdtype, A, d, inter, partial, norm_rope_bwd_blocks(A.T), dwq, dwk, stream);
}

}  // namespace kda
