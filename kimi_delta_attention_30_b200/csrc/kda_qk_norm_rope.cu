// RMS norm of every query and key head, then the rotation of its first `rot` channels by
// position, in one pass, and the gradients of both.
//
//   r = 1 / sqrt(mean_c x_c^2 + eps),  y = x r w,  a channel pair (a, b) of y and the
//   angle t = position * inv_freq[pair]:  (a cos t - b sin t, b cos t + a sin t).
// Backward, with g the rotation of dy by -t and h = g w:
//   dw_c = sum over rows of g_c x_c r,   dx = r (h - x r^2 mean_c(h_c x_c)).
//
// Bound by HBM: a row is read once and written once, some five instructions an element (packed
// fp32 pairs), which is near the issue limit too: at 16 channels a lane a step of four rows
// takes about 80 instructions a warp forward.  16384 tokens of 32 heads of 128 bf16 channels:
// forward 47.5 us, 5.7 TB/s, 0.88 of the copy rate; backward 80 us, 5.0 TB/s (calls back to
// back; 51 and 89 us from a cold cache).  With few heads most lanes have no row of their own: 65536
// tokens of one query and one key head take 83 us forward, 134 backward, at 10 and 16 us for the
// bytes.  A warp walks tokens and, for each, its heads
// (or a part of them when there are few tokens), four or eight rows at a time: d / 16 lanes
// share a row, and a lane holds the two 8-channel vectors that rotate with each other
// (halves: vectors p and p + rot / 16; neighbours: vectors 2 p and 2 p + 1), so a rotation
// needs no exchange between lanes and loads are 16 bytes.  Loads run several steps ahead,
// across tokens and sides, through shared memory (asynchronous copies that the lane which
// made them reads).
//
// The rotations of a token are formed once, two pairs a lane, and exchanged through shared
// memory.  Angles are taken in turns in 64-bit fixed point: with f = inv_freq / (2 pi) as a
// fraction of 2^64 (from fp64, once a warp), position * f mod 2^64 is the angle's fraction of
// a turn, exact to position * 2^-53 of a turn (fp32 would keep two digits at position 10^6);
// sincospif of its top 32 bits.  Norm weight and rotation are multiplied once a token and
// side, so a row costs one rotation and one scaling.
#include "kda_launch.cuh"
#include "kda_rope.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Eight channels as they stand in memory: 16-byte pieces, copied asynchronously into shared
// memory by the lane that will read them (so a step needs no barrier), `pitch` bytes apart.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T> constexpr int pieces8() { return 8 * (int)sizeof(T) / 16; }
constexpr int kPiece = 32 * 16;   // one 16-byte piece of every lane

template <typename T>
__device__ __forceinline__ void copy8(uint32_t dst, const T* src) {
#pragma unroll
    for (int i = 0; i < pieces8<T>(); ++i) copy16(dst + i * kPiece, src + i * (16 / (int)sizeof(T)));
}
__device__ __forceinline__ void unpack8(uint4 v, float2 (&x)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void get8(const uint8_t* src, float2 (&x)[4]) {
    if constexpr (sizeof(T) == 2) {
        unpack8(*reinterpret_cast<const uint4*>(src), x);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + kPiece);
        x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
    }
}
__device__ __forceinline__ void store8(float* p, const float2 (&x)[4]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&x)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
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
__device__ __forceinline__ Lane lane_of(int l, int rot, bool interleaved) {
    Lane L;
    const int half = rot / 16;   // pairs of vectors that rotate
    L.turns = l < half;
    L.pair = 8 * l;
    L.c0 = 8 * ((interleaved || !L.turns) ? 2 * l : l);
    L.c1 = 8 * ((interleaved || !L.turns) ? 2 * l + 1 : l + half);
    return L;
}

// Turns a position advances, as fractions of 2^64, of the pairs lane and lane + 32.
template <int D>
struct Freq {
    static constexpr int N = (D / 2 + 31) / 32;
    unsigned long long f[N];
    __device__ __forceinline__ void load(const NormRopeArgs& A, int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f[i] = 0;
            if (lane + 32 * i < A.rot / 2) {
                double t = (double)A.inv_freq[lane + 32 * i] * 0.15915494309189533577;   // 1 / (2 pi)
                t -= floor(t);
                f[i] = (unsigned long long)(t * 18446744073709549568.0);   // below 2^64 even for t next to 1
            }
        }
    }
};

// cos and sin of the token's pairs, for the warp
template <int D>
__device__ __forceinline__ void rotations(const NormRopeArgs& A, int position, const Freq<D>& F, int lane, float2* cs) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Freq<D>::N; ++i) {
        if (lane + 32 * i < A.rot / 2) {
            const unsigned long long t = (unsigned long long)(long long)position * F.f[i];
            float s, c;
            sincospif((float)(int)(t >> 32) * (1.f / 2147483648.f), &s, &c);
            cs[lane + 32 * i] = make_float2(c, s);
        }
    }
    __syncwarp();
}

// those of the lane's eight pairs; (1, 0) where the lane does not rotate
__device__ __forceinline__ void lane_rotation(const float2* cs, const Lane& L, float2 (&co)[4], float2 (&si)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 x = L.turns ? *reinterpret_cast<const float4*>(&cs[L.pair + 2 * i]) : make_float4(1.f, 0.f, 1.f, 0.f);
        co[i] = make_float2(x.x, x.z);
        si[i] = make_float2(x.y, x.w);
    }
}

// sum over the lanes that share a row
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// 1 / sqrt(mean of squares + eps); 0 for a zero row with eps = 0, which stays zero, and NaN for a
// row that holds one, so that the whole row shows it
__device__ __forceinline__ float rms_scale(float sum_sq, int d, float eps) {
    const float m = fmaf(sum_sq, 1.f / (float)d, eps);
    return m == 0.f ? 0.f : rsqrtf(m);
}

template <typename Tw>
__device__ __forceinline__ void weights8(const void* w, int c, float2 (&x)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(1.f, 1.f);
    } else {
        const Tw* p = reinterpret_cast<const Tw*>(w) + c;
        if constexpr (sizeof(Tw) == 2) {
            unpack8(*reinterpret_cast<const uint4*>(p), x);
        } else {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
            x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
        }
    }
}

// Pairs of a lane's vectors.  Halves: element i of the first vector turns with element i of
// the second, so a packed pair of the first turns with a packed pair of the second.
// Neighbours: the elements are sorted into that form after loading (evens of both vectors,
// odds of both vectors) and back before storing.
template <bool INTER>
__device__ __forceinline__ void sort_pairs(float2 (&a)[4], float2 (&b)[4]) {
    if (INTER) {   // a: x0 x1 x2 x3 .., b: y0 y1 ..  ->  a: evens of a then of b, b: odds
        const float2 e[4] = {make_float2(a[0].x, a[1].x), make_float2(a[2].x, a[3].x), make_float2(b[0].x, b[1].x),
                             make_float2(b[2].x, b[3].x)};
        const float2 o[4] = {make_float2(a[0].y, a[1].y), make_float2(a[2].y, a[3].y), make_float2(b[0].y, b[1].y),
                             make_float2(b[2].y, b[3].y)};
#pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] = e[i]; b[i] = o[i]; }
    }
}
template <bool INTER>
__device__ __forceinline__ void unsort_pairs(float2 (&a)[4], float2 (&b)[4]) {
    if (INTER) {
        const float2 x[4] = {make_float2(a[0].x, b[0].x), make_float2(a[0].y, b[0].y), make_float2(a[1].x, b[1].x),
                             make_float2(a[1].y, b[1].y)};
        const float2 y[4] = {make_float2(a[2].x, b[2].x), make_float2(a[2].y, b[2].y), make_float2(a[3].x, b[3].x),
                             make_float2(a[3].y, b[3].y)};
#pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] = x[i]; b[i] = y[i]; }
    }
}

// A warp's steps in order: its (token, part of the heads) pairs, queries before keys, ROWS
// heads at a time.
struct Walk {
    long long tok, tok_step;
    int grp, grp_step, side, h, e;   // heads h .. h + ROWS - 1 of the side, below e
    bool new_tok, new_side;

    __device__ __forceinline__ bool enter(const NormRopeArgs& A) {   // the first step of the current pair
        if (tok >= A.T) return false;
        const int h0 = grp * A.per, h1 = min(A.Hq + A.Hk, h0 + A.per);
        side = h0 < A.Hq ? 0 : 1;
        h = side ? h0 - A.Hq : h0;
        e = side ? h1 - A.Hq : min(h1, A.Hq);
        new_tok = new_side = true;
        return true;
    }
    __device__ __forceinline__ bool start(const NormRopeArgs& A, long long first, long long step) {
        tok = first / A.groups;
        grp = (int)(first - tok * A.groups);
        tok_step = step / A.groups;
        grp_step = (int)(step - tok_step * A.groups);
        return enter(A);
    }
    template <int ROWS>
    __device__ __forceinline__ bool next(const NormRopeArgs& A) {
        new_tok = new_side = false;
        h += ROWS;
        if (h < e) return true;
        const int h1 = min(A.Hq + A.Hk, grp * A.per + A.per);
        if (side == 0 && h1 > A.Hq) {
            side = 1;
            h = 0;
            e = h1 - A.Hq;
            new_side = true;
            return true;
        }
        tok += tok_step;
        grp += grp_step;
        if (grp >= A.groups) {
            grp -= A.groups;
            ++tok;
        }
        return enter(A);
    }
};

// Steps in flight, the current one among them.
template <typename Tin> constexpr int kDepth() { return sizeof(Tin) == 2 ? 5 : 4; }
constexpr int kPos = 16;   // bytes behind a stage's pieces: the token's position

template <typename Tin, int VECS> constexpr int stage_bytes() { return VECS * pieces8<Tin>() * kPiece + kPos; }

// FULL (here and in the backward kernel): every channel turns, rot = D.  Where that is left open, the
// channels that do not turn are kept apart by a branch, which costs 1 to 3 % of the time (52.1 instead
// of 51.1 us forward, 82 instead of 80 backward, at the size above).
template <typename Tin, typename Tw, int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, sizeof(Tin) == 2 ? 5 : 4) norm_rope_fwd(const __grid_constant__ NormRopeArgs A) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;   // lanes a row, rows a warp at a time
    constexpr int DEPTH = kDepth<Tin>(), BYTES = stage_bytes<Tin, 2>(), VEC = pieces8<Tin>() * kPiece;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    uint8_t* stages = sm + warp * (DEPTH * BYTES + D / 2 * 8);
    float2* cs = reinterpret_cast<float2*>(stages + DEPTH * BYTES);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(stages) + lane * 16;
    const Lane L = lane_of(l, A.rot, INTER);
    Walk W, ahead;
    bool more = W.start(A, (long long)blockIdx.x * kWarps + warp, (long long)gridDim.x * kWarps);
    if (!more) return;
    ahead = W;
    bool any = true;
    auto load = [&](int s) {   // the steps ahead into stage s, one group a step (empty behind the last)
        if (any) {
            const NormRopeSide& X = ahead.side ? A.k : A.q;
            const Tin* p = reinterpret_cast<const Tin*>(X.in) + ahead.tok * X.in_tok +
                           (long long)min(ahead.h + sub, ahead.e - 1) * X.in_head;
            copy8(to + s * BYTES, p + L.c0);
            copy8(to + s * BYTES + VEC, p + L.c1);
            if (ahead.new_tok && A.rot > 0) copy4(to + s * BYTES + 2 * VEC - lane * 16, A.positions + ahead.tok);
            any = ahead.next<ROWS>(A);
        }
        copies_done();
    };
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) load(s);
    Freq<D> F;
    F.load(A, lane);
    float2 ca[4], cb[4], sa[4], sb[4];   // the rotation of the weighted row: a' = ca a + sb b, b' = cb b + sa a
    int stage = 0;
    while (more) {
        wait_copies<DEPTH - 2>();
        const uint8_t* from = stages + stage * BYTES;
        float2 x[4], y[4];
        get8<Tin>(from + lane * 16, x);
        get8<Tin>(from + VEC + lane * 16, y);
        const NormRopeSide& X = W.side ? A.k : A.q;
        if (W.new_tok) rotations<D>(A, *reinterpret_cast<const int*>(from + 2 * VEC), F, lane, cs);
        load(stage == 0 ? DEPTH - 1 : stage - 1);   // the stage before this one: read a step ago
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
        if (W.new_side) {
            float2 w0[4], w1[4], co[4], si[4];
            weights8<Tw>(X.w, L.c0, w0);
            weights8<Tw>(X.w, L.c1, w1);
            sort_pairs<INTER>(w0, w1);
            lane_rotation(cs, L, co, si);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ca[i] = mul2(co[i], w0[i]);
                cb[i] = mul2(co[i], w1[i]);
                sa[i] = mul2(si[i], w0[i]);
                sb[i] = neg2(mul2(si[i], w1[i]));
            }
        }
        sort_pairs<INTER>(x, y);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(x[i], x[i], fma2(y[i], y[i], ss));
        const float r1 = rms_scale(row_sum<LANES>(ss.x + ss.y), D, A.eps);
        const float2 r = make_float2(r1, r1);
        float2 u[4], v[4];
        // channels that do not turn stay apart: 0 times an infinity or NaN of another is none of theirs
        if (FULL || L.turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = mul2(fma2(ca[i], x[i], mul2(sb[i], y[i])), r);
                v[i] = mul2(fma2(cb[i], y[i], mul2(sa[i], x[i])), r);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = mul2(mul2(ca[i], x[i]), r);
                v[i] = mul2(mul2(cb[i], y[i]), r);
            }
        }
        unsort_pairs<INTER>(u, v);
        if (W.h + sub < W.e) {
            Tin* d = reinterpret_cast<Tin*>(X.out) + W.tok * X.out_tok + (long long)(W.h + sub) * X.out_head;
            store8(d + L.c0, u);
            store8(d + L.c1, v);
        }
        more = W.next<ROWS>(A);
    }
}

// Backward: the weight gradients are summed in registers over a lane's rows, then over the
// block in a fixed order, and written as one partial row per block ([grid][2][D] fp32); the
// second kernel adds the partial rows in order, so the result does not depend on timing.
// dw: sum over rows of (rotated gradient) x r; a lane sums one side at a time and adds it to
// the side's shared-memory row of its own at the end of the side's steps of a token.
template <typename Tin> constexpr int kBwdDepth() { return sizeof(Tin) == 2 ? 4 : 3; }

template <typename Tin, typename Tw, int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, sizeof(Tin) == 2 ? 4 : 3) norm_rope_bwd(const __grid_constant__ NormRopeArgs A,
                                                                                   float* __restrict__ partial) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    constexpr int DEPTH = kBwdDepth<Tin>(), BYTES = stage_bytes<Tin, 4>(), VEC = pieces8<Tin>() * kPiece;
    extern __shared__ __align__(16) uint8_t sm[];
    let_next_kernel_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    float* acc = reinterpret_cast<float*>(sm);   // [2][kWarps * ROWS][D]
    uint8_t* stages = sm + 2 * kWarps * ROWS * D * 4 + warp * (DEPTH * BYTES + D / 2 * 8);
    float2* cs = reinterpret_cast<float2*>(stages + DEPTH * BYTES);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(stages) + lane * 16;
    const Lane L = lane_of(l, A.rot, INTER);
    auto mine = [&](int side) { return acc + ((side * kWarps + warp) * ROWS + sub) * D; };
    float2 g0[4], g1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g0[i] = g1[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        store8(mine(side) + L.c0, g0);
        store8(mine(side) + L.c1, g1);
    }
    Walk W, ahead;
    bool more = W.start(A, (long long)blockIdx.x * kWarps + warp, (long long)gridDim.x * kWarps);
    ahead = W;
    bool any = more;
    auto load = [&](int s) {
        if (any) {
            const NormRopeSide& X = ahead.side ? A.k : A.q;
            const int hh = min(ahead.h + sub, ahead.e - 1);
            const Tin* p = reinterpret_cast<const Tin*>(X.in) + ahead.tok * X.in_tok + (long long)hh * X.in_head;
            const Tin* q = reinterpret_cast<const Tin*>(X.dy) + ahead.tok * X.dy_tok + (long long)hh * X.dy_head;
            copy8(to + s * BYTES, p + L.c0);
            copy8(to + s * BYTES + VEC, p + L.c1);
            copy8(to + s * BYTES + 2 * VEC, q + L.c0);
            copy8(to + s * BYTES + 3 * VEC, q + L.c1);
            if (ahead.new_tok && A.rot > 0) copy4(to + s * BYTES + 4 * VEC - lane * 16, A.positions + ahead.tok);
            any = ahead.next<ROWS>(A);
        }
        copies_done();
    };
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) load(s);
    Freq<D> F;
    F.load(A, lane);
    float2 co[4], si[4], w0[4], w1[4];
    int stage = 0;
    while (more) {
        wait_copies<DEPTH - 2>();
        const uint8_t* from = stages + stage * BYTES;
        float2 x[4], y[4], u[4], v[4];
        get8<Tin>(from + lane * 16, x);
        get8<Tin>(from + VEC + lane * 16, y);
        get8<Tin>(from + 2 * VEC + lane * 16, u);
        get8<Tin>(from + 3 * VEC + lane * 16, v);
        const int side = W.side;
        const NormRopeSide& X = side ? A.k : A.q;
        if (W.new_tok) rotations<D>(A, *reinterpret_cast<const int*>(from + 4 * VEC), F, lane, cs);
        load(stage == 0 ? DEPTH - 1 : stage - 1);
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
        if (W.new_side) {
            weights8<Tw>(X.w, L.c0, w0);
            weights8<Tw>(X.w, L.c1, w1);
            sort_pairs<INTER>(w0, w1);
            lane_rotation(cs, L, co, si);
        }
        const bool live = W.h + sub < W.e;
        sort_pairs<INTER>(x, y);
        sort_pairs<INTER>(u, v);
        if (FULL || L.turns) {   // the gradient turns back
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 g = fma2(co[i], u[i], mul2(si[i], v[i]));
                v[i] = fma2(co[i], v[i], neg2(mul2(si[i], u[i])));
                u[i] = g;
            }
        }
        float2 ss = make_float2(0.f, 0.f), hx = ss;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ss = fma2(x[i], x[i], fma2(y[i], y[i], ss));
            hx = fma2(mul2(u[i], w0[i]), x[i], fma2(mul2(v[i], w1[i]), y[i], hx));
        }
        const float r1 = rms_scale(row_sum<LANES>(ss.x + ss.y), D, A.eps);
        const float m1 = -row_sum<LANES>(hx.x + hx.y) * r1 * r1 * (1.f / D);
        const float2 r = make_float2(r1, r1), m = make_float2(m1, m1);
        const float2 rl = live ? r : make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 xr = mul2(x[i], rl), yr = mul2(y[i], rl);
            g0[i] = fma2(u[i], xr, g0[i]);
            g1[i] = fma2(v[i], yr, g1[i]);
            u[i] = fma2(mul2(u[i], w0[i]), r, mul2(xr, m));
            v[i] = fma2(mul2(v[i], w1[i]), r, mul2(yr, m));
        }
        unsort_pairs<INTER>(u, v);
        if (live) {
            Tin* d = reinterpret_cast<Tin*>(X.out) + W.tok * X.out_tok + (long long)(W.h + sub) * X.out_head;
            store8(d + L.c0, u);
            store8(d + L.c1, v);
        }
        more = W.next<ROWS>(A);
        if (!more || W.new_side) {   // the side's last step
            float4 *s0 = reinterpret_cast<float4*>(mine(side) + L.c0), *s1 = reinterpret_cast<float4*>(mine(side) + L.c1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 p = s0[i], q = s1[i];
                s0[i] = make_float4(p.x + g0[2 * i].x, p.y + g0[2 * i].y, p.z + g0[2 * i + 1].x, p.w + g0[2 * i + 1].y);
                s1[i] = make_float4(q.x + g1[2 * i].x, q.y + g1[2 * i].y, q.z + g1[2 * i + 1].x, q.w + g1[2 * i + 1].y);
                g0[2 * i] = g0[2 * i + 1] = g1[2 * i] = g1[2 * i + 1] = make_float2(0.f, 0.f);
            }
        }
    }
    if (partial == nullptr) return;
    // a neighbour rotation's sums stand sorted: channel 2 i of vector p at p's i-th half, 2 i + 1 at the other's
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
        const int side = c / D, ch = c % D;
        int at = ch;
        if (INTER) {
            const int p = ch / 16, k = ch % 16;                  // lane p holds channels 16 p .. 16 p + 15
            at = 16 * p + (k & 1) * 8 + k / 2;                   // evens of both vectors, then odds
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps * ROWS; ++i) s += acc[(side * kWarps * ROWS + i) * D + at];
        partial[((size_t)blockIdx.x * 2 + side) * D + ch] = s;
    }
}

// dw of one side a block row: 32 columns x 32 runs of partial rows
template <typename Tw, int D>
__global__ void __launch_bounds__(1024) norm_rope_dw(const float* partial, int n, void* dwq, void* dwk) {
    __shared__ float red[32][33];
    wait_for_kernels_before();
    const int side = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    void* out = side ? dwk : dwq;
    if (out == nullptr) return;
    float s = 0.f;
    const int per = (n + 31) / 32;
#pragma unroll 8
    for (int i = run * per; i < min(n, (run + 1) * per); ++i) s += __ldcg(partial + ((size_t)i * 2 + side) * D + c);
    red[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += red[i][threadIdx.x & 31];
        reinterpret_cast<Tw*>(out)[c] = from_f32<Tw>(s);
    }
}

template <typename Tin, typename Tw, int D>
cudaError_t run(const NormRopeArgs& A, bool inter, bool bwd, float* partial, int blocks, void* dwq, void* dwk,
                cudaStream_t s) {
    constexpr int ROWS = 512 / D, CS = D / 2 * 8;
    if (!bwd) {
        auto kern = A.rot == D ? inter ? norm_rope_fwd<Tin, Tw, D, true, true> : norm_rope_fwd<Tin, Tw, D, false, true>
                    : inter    ? norm_rope_fwd<Tin, Tw, D, true, false>
                               : norm_rope_fwd<Tin, Tw, D, false, false>;
        constexpr int smem = kWarps * (kDepth<Tin>() * stage_bytes<Tin, 2>() + CS);
        static_assert(smem <= 48 * 1024, "the default limit");
        kern<<<blocks, kThreads, smem, s>>>(A);
    } else {
        const bool dw = dwq != nullptr || dwk != nullptr;
        auto kern = A.rot == D ? inter ? norm_rope_bwd<Tin, Tw, D, true, true> : norm_rope_bwd<Tin, Tw, D, false, true>
                    : inter    ? norm_rope_bwd<Tin, Tw, D, true, false>
                               : norm_rope_bwd<Tin, Tw, D, false, false>;
        constexpr int smem = 2 * kWarps * ROWS * D * 4 + kWarps * (kBwdDepth<Tin>() * stage_bytes<Tin, 4>() + CS);
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<blocks, kThreads, smem, s>>>(A, dw ? partial : nullptr);
        const cudaError_t launched = cudaGetLastError();
        if (launched != cudaSuccess) return launched;
        if (dw) return launch_behind(norm_rope_dw<Tw, D>, dim3(D / 32, 2), 1024, 0, s, partial, blocks, dwq, dwk);
    }
    return cudaGetLastError();
}

cudaError_t pick(kda_dtype dtype, kda_dtype wdtype, const NormRopeArgs& A, int d, bool inter, bool bwd,
                 float* partial, int blocks, void* dwq, void* dwk, cudaStream_t s) {
    typedef __nv_bfloat16 bf;
    if (dtype == KDA_F32 && wdtype == KDA_F32)
        return d == 128 ? run<float, float, 128>(A, inter, bwd, partial, blocks, dwq, dwk, s)
                        : run<float, float, 64>(A, inter, bwd, partial, blocks, dwq, dwk, s);
    if (dtype == KDA_F32)
        return d == 128 ? run<float, bf, 128>(A, inter, bwd, partial, blocks, dwq, dwk, s)
                        : run<float, bf, 64>(A, inter, bwd, partial, blocks, dwq, dwk, s);
    if (wdtype == KDA_F32)
        return d == 128 ? run<bf, float, 128>(A, inter, bwd, partial, blocks, dwq, dwk, s)
                        : run<bf, float, 64>(A, inter, bwd, partial, blocks, dwq, dwk, s);
    return d == 128 ? run<bf, bf, 128>(A, inter, bwd, partial, blocks, dwq, dwk, s)
                    : run<bf, bf, 64>(A, inter, bwd, partial, blocks, dwq, dwk, s);
}

}  // namespace

namespace {

// Warps that share a token's heads: enough warps to fill the machine (`warps` an SM), but a
// whole step of rows each.
void split_heads(NormRopeArgs& A, int d, int warps) {
    const int heads = A.Hq + A.Hk, rows = 32 / (d / 16), steps = (heads + rows - 1) / rows;
    long long groups = (148LL * warps + A.T - 1) / A.T;
    groups = groups < 1 ? 1 : groups > steps ? steps : groups;
    A.per = (int)((steps + groups - 1) / groups) * rows;
    A.groups = (heads + A.per - 1) / A.per;
}

constexpr int kFwdBlocks = 148 * 5, kBwdBlocks = 148 * 4;   // what fits at once

}  // namespace

int norm_rope_bwd_blocks() { return kBwdBlocks; }

cudaError_t launch_norm_rope(kda_dtype dtype, kda_dtype wdtype, NormRopeArgs A, int d, bool inter,
                             cudaStream_t stream) {
    split_heads(A, d, kFwdBlocks / 148 * kWarps);
    const long long blocks = (A.T * A.groups + kWarps - 1) / kWarps;
    return pick(dtype, wdtype, A, d, inter, false, nullptr, (int)(blocks < kFwdBlocks ? blocks : kFwdBlocks), nullptr,
                nullptr, stream);
}

cudaError_t launch_norm_rope_bwd(kda_dtype dtype, kda_dtype wdtype, NormRopeArgs A, int d, bool inter,
                                 float* partial, void* dwq, void* dwk, cudaStream_t stream) {
    split_heads(A, d, kBwdBlocks / 148 * kWarps);
    const long long blocks = (A.T * A.groups + kWarps - 1) / kWarps;
    return pick(dtype, wdtype, A, d, inter, true, partial, (int)(blocks < kBwdBlocks ? blocks : kBwdBlocks), dwq, dwk,
                stream);
}

}  // namespace kda
