// Linear attention with one decay a head on the CUDA cores: the path for fp32 inputs
// and for widths of 64.
//
// With g_i the inclusive sum of log decays inside a chunk of C = 64 tokens and S the
// chunk's start state,
//   S'  = e^{g_C} S + sum_j e^{g_C - g_j} k_j v_j^T
//   o_i = e^{g_i} S^T q_i + sum_{j <= i} e^{g_i - g_j} (q_i . k_j) v_j
// so the only sequential part is S' from S, an elementwise multiply and add once every
// chunk's own sum is known.  Forward: (1) each chunk's sum, all chunks at once; (2) the
// chain over chunks, one thread per four state elements, which leaves every chunk's
// start state; (3) the outputs, all chunks at once.  Backward: the same two steps give
// the start states, and once more with (q, d_o), weights e^{g_i} and the order reversed
// the gradients dS' of the end states; then all chunks at once
//   P_ij = D_ij (q_i . k_j),  dA_ij = D_ij (d_o_i . v_j),  D_ij = e^{g_i - g_j} (j <= i)
//   dq_i = e^{g_i} S d_o_i + sum_j dA_ij k_j
//   dk_j = e^{g_C - g_j} dS' v_j + sum_i dA_ij q_i
//   dv_j = e^{g_C - g_j} dS'^T k_j + sum_i P_ij d_o_i
//   dlog_alpha_t = sum_{i >= t} e^{g_i} q_i . S d_o_i + sum_{j < t} e^{g_C - g_j} k_j . dS' v_j
//                + e^{g_C} <dS', S> + sum_{i >= t > j} dA_ij (q_i . k_j)
// where every term of the last lines is one that t's decay enters, so none is added and taken
// away again (the terms themselves have signs):
// the last sum runs over a rectangle of the pair products, taken as running sums along
// each row and then down the columns.  (Suffix sums of q_i . dq_i - k_i . dk_i give the
// same number, but the pairs with both ends behind t cancel there and leave their
// roundings: 4e-6 where the gradient is exactly zero.)
//
// Products are 64 x 64 register tiles (256 threads, 4 x 4 each) over operands in shared
// memory, every operand read as 16-byte vectors where its layout allows; fp32 throughout,
// as fp32 inputs ask for.  Shared-memory reads bound them (a 64^3 product takes 3.8 us a
// block), so small problems are spread wider: while the blocks find an SM each, sums and
// outputs use 16-row tiles (64 threads), and the backward always gives dq, dk and
// dv of a chunk to three blocks, which costs the pair products twice (16 units of 64^3
// instead of 13 at 64 x 128) and puts dlog_alpha's last sums into a kernel of its own.
// Decays are formed from g as a (hi, lo) pair.  Small problems are chains of short launches;
// each kernel behind the first starts early and loads and multiplies what needs only the
// call's inputs (outputs: the scores; gradients: the pair products) before it waits.  fp32,
// 256 tokens of 2 heads of 64: 12.3 us (20.5 without); backward of 5 sequences, 705 tokens of
// 3 heads of 64 x 128: 43 us, each from a cold cache.  Large sizes are far from their bytes: fp32,
// 2048 tokens of 16 heads of 64 (128): 56 (161) us forward, 134 (387) backward; bf16 heads of 64,
// which have no tensor-core path, 4 x 4096 tokens of 32 heads: 767 us forward, 2263 backward, at
// 42 and 73 us for the bytes.
#include "kda_launch.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kC = kLinSimtChunk;
constexpr int kThreads = 256;
constexpr int kLdM = kC + 1;   // pitch of the pair products, walked along rows and columns
constexpr int kLdP = kC + 4;   // row pitch of 64-wide tiles: rows start 4 banks apart

// acc += A B over K, A 64 x K and B K x 64.  Thread (ty, tx) owns rows 4 ty + r and
// columns 4 tx + c, or tx + 16 c with CI (which keeps reads of a B stored [column][k]
// free of bank conflicts).  AT: A stored [k][row].  BT: B stored [column][k].
template <int K, bool AT, bool BT, bool CI>
__device__ __forceinline__ void mm64(float (&acc)[4][4], const float* __restrict__ A, int lda,
                                     const float* __restrict__ B, int ldb, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float a[4][4], b[4][4];   // [k][row], [k][column]
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (AT) {
                const float4 x = *reinterpret_cast<const float4*>(A + (k + u) * lda + 4 * ty);
                a[u][0] = x.x; a[u][1] = x.y; a[u][2] = x.z; a[u][3] = x.w;
            } else {
                const float4 x = *reinterpret_cast<const float4*>(A + (4 * ty + u) * lda + k);
                a[0][u] = x.x; a[1][u] = x.y; a[2][u] = x.z; a[3][u] = x.w;
            }
            if (BT) {
                const float4 x = *reinterpret_cast<const float4*>(B + (CI ? tx + 16 * u : 4 * tx + u) * ldb + k);
                b[0][u] = x.x; b[1][u] = x.y; b[2][u] = x.z; b[3][u] = x.w;
            } else if (CI) {
#pragma unroll
                for (int c = 0; c < 4; ++c) b[u][c] = B[(k + u) * ldb + tx + 16 * c];
            } else {
                const float4 x = *reinterpret_cast<const float4*>(B + (k + u) * ldb + 4 * tx);
                b[u][0] = x.x; b[u][1] = x.y; b[u][2] = x.z; b[u][3] = x.w;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(a[u][r], b[u][c], acc[r][c]);
    }
}

__device__ __forceinline__ void clear(float (&acc)[4][4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
}

__device__ __forceinline__ void load_vec(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// ROWS token rows of COLS columns from column c0 of a [tokens, H, D] array; rows past `len`
// are zero (they belong to the next sequence).  Eight loads a thread stand before the first
// is stored: one at a time they are a round trip to memory each.
template <typename Tin, int ROWS, int COLS, int THREADS>
__device__ __forceinline__ void load_rows(float* dst, int ld, const Tin* __restrict__ src, long long tok0, int len, int H,
                                          int h, int D, int c0) {
    constexpr int V = COLS / 4, N = ROWS * V / THREADS, BATCH = N < 8 ? N : 8;
    static_assert(ROWS * V % THREADS == 0 && N % BATCH == 0, "tile");
#pragma unroll 1
    for (int n = 0; n < N; n += BATCH) {
        float x[BATCH][4];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int u = (n + i) * THREADS + threadIdx.x, r = u / V, c = (u % V) * 4;
            x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
            if (r < len) load_vec(src + ((size_t)(tok0 + r) * (size_t)H + h) * D + c0 + c, x[i]);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int u = (n + i) * THREADS + threadIdx.x;
            *reinterpret_cast<float4*>(dst + u / V * ld + (u % V) * 4) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        }
    }
}

// fp32 that a kernel before this one wrote
struct Written {
    float x;
};
__device__ __forceinline__ void load_vec(const Written* p, float (&x)[4]) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// ROWS x COLS of such a matrix with `pitch` columns
template <int ROWS, int COLS, int THREADS>
__device__ __forceinline__ void load_tile(float* dst, int ld, const float* src, int pitch) {
    load_rows<Written, ROWS, COLS, THREADS>(dst, ld, reinterpret_cast<const Written*>(src), 0, ROWS, 1, 0, pitch, 0);
}

// The chunk's inclusive cumulative log decay as (hi, lo), by the first warp; tokens past
// `len` add nothing, so g stays at the last token's value there.  Summed in 64-bit fixed
// point (32 fractional bits of log_alpha; exact sums).  A NaN among them is the whole chunk's.
template <typename Tin>
__device__ __forceinline__ void chunk_decay(float* gh, float* gl, const LinDecay& dec, size_t tok0, int len, int H,
                                            int h) {
    if (threadIdx.x < 32) {
        const int t = 2 * threadIdx.x;
        const float x = t < len ? lin_log_decay<Tin>(dec, tok0 + t, H, h) : 0.f;
        const float y = t + 1 < len ? lin_log_decay<Tin>(dec, tok0 + t + 1, H, h) : 0.f;
        const bool nan = __any_sync(0xffffffffu, x != x || y != y);
        const long long a = __float2ll_rn(x * 4294967296.f), b = __float2ll_rn(y * 4294967296.f);
        long long s = a + b;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long z = __shfl_up_sync(0xffffffffu, s, off);
            if ((int)threadIdx.x >= off) s += z;
        }
        const long long g[2] = {s - b, s};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float hi = __ll2float_rn(g[u]);
            gh[t + u] = nan ? __int_as_float(0x7fffffff) : hi * (1.f / 4294967296.f);
            gl[t + u] = __ll2float_rn(g[u] - __float2ll_rn(hi)) * (1.f / 4294967296.f);
        }
    }
}

// ---- (1) each chunk's own sum: ROWS x 64 of the state a block ------------------------
// Forward: sum_j e^{g_C - g_j} a_j b_j^T (a = k, b = v); reversed: sum_i e^{g_i} a_i b_i^T (q, d_o).
template <typename Tin>
struct UpdateSide {
    const Tin *a, *b;
    float* U;
};
template <typename Tin, int ROWS>
__global__ void __launch_bounds__(ROWS * 4) lin_update(UpdateSide<Tin> fwd, UpdateSide<Tin> rev, LinDecay dec,
                                                       ChunkMap cmap, int H, int DK, int DV, float* __restrict__ gam) {
    constexpr int LDA = ROWS + 4;
    __shared__ __align__(16) float sa[kC * LDA], sb[kC * kLdP];
    __shared__ float gh[kC], gl[kC], w[kC];
    let_next_kernel_start();
    int seq, tok0, len, idx;
    cmap.locate((int)blockIdx.x, seq, tok0, len, idx);
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int nv = DV / 64, tiles = nv * (DK / ROWS), z = (int)blockIdx.z % tiles;
    const bool REV = (int)blockIdx.z >= tiles;
    const UpdateSide<Tin>& A = REV ? rev : fwd;
    const int k0 = z / nv * ROWS, v0 = z % nv * 64;
    load_rows<Tin, kC, ROWS, ROWS * 4>(sa, LDA, A.a, tok0, len, H, h, DK, k0);
    load_rows<Tin, kC, 64, ROWS * 4>(sb, kLdP, A.b, tok0, len, H, h, DV, v0);
    chunk_decay<Tin>(gh, gl, dec, tok0, len, H, h);
    __syncthreads();
    if (tid < kC)
        w[tid] = REV ? exp_g(gh[tid], gl[tid]) : exp_gdiff(gh[kC - 1], gl[kC - 1], gh[tid], gl[tid]);
    __syncthreads();
    for (int u = tid; u < kC * ROWS / 4; u += blockDim.x) {
        float4* p = reinterpret_cast<float4*>(sa + u / (ROWS / 4) * LDA + u % (ROWS / 4) * 4);
        const float s = w[u / (ROWS / 4)];
        *p = make_float4(p->x * s, p->y * s, p->z * s, p->w * s);
    }
    __syncthreads();
    float acc[4][4];
    clear(acc);
    mm64<kC, true, false, false>(acc, sa, LDA, sb, kLdP, ty, tx);
    const size_t unit = (size_t)blockIdx.x * H + h;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(A.U + (unit * DK + k0 + 4 * ty + r) * DV + v0 + 4 * tx) =
            make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    if (blockIdx.z == 0 && tid == 0) gam[unit] = exp_g(gh[kC - 1], gl[kC - 1]);
}

// ---- (2) the chain over chunks, in place: X[n] = state before chunk n (REV: behind it)
struct ChainSide {
    float* X;
    const float* start;
    float* end;
};
__global__ void __launch_bounds__(kThreads) lin_chain(ChainSide fwd, ChainSide rev, const float* gam,
                                                      SeqMap smap, int H, int E4) {
    let_next_kernel_start();
    wait_for_kernels_before();
    const bool REV = blockIdx.z != 0;
    float* X = REV ? rev.X : fwd.X;
    const float* start = REV ? rev.start : fwd.start;
    float* end = REV ? rev.end : fwd.end;
    const SeqInfo sq = smap.get((int)blockIdx.x / H);
    const int h = (int)blockIdx.x % H;
    const int e = (int)blockIdx.y * kThreads + threadIdx.x;
    if (e >= E4) return;
    const int n = (sq.len + smap.C - 1) / smap.C;
    float4* x4 = reinterpret_cast<float4*>(X);
    const size_t sh = ((size_t)sq.seq * H + h) * E4 + e;
    float4 s = start ? reinterpret_cast<const float4*>(start)[sh] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;   // loads of that many chunks stand before the first is used
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        float4 u[kAhead];
        float g[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j < n) {
                const size_t unit = (size_t)(sq.chunk0 + (REV ? n - 1 - i0 - j : i0 + j)) * H + h;
                u[j] = __ldcg(x4 + unit * E4 + e);
                g[j] = __ldcg(gam + unit);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j < n) {
                const size_t unit = (size_t)(sq.chunk0 + (REV ? n - 1 - i0 - j : i0 + j)) * H + h;
                x4[unit * E4 + e] = s;
                s.x = fmaf(g[j], s.x, u[j].x);
                s.y = fmaf(g[j], s.y, u[j].y);
                s.z = fmaf(g[j], s.z, u[j].z);
                s.w = fmaf(g[j], s.w, u[j].w);
            }
        }
    }
    if (end) reinterpret_cast<float4*>(end)[sh] = s;
}

// ---- (3) outputs: ROWS tokens x 64 value columns a block -----------------------------
template <int DK, int ROWS> constexpr size_t out_smem() {
    return sizeof(float) * ((ROWS + kC) * (DK + 4) + (ROWS + kC) * kLdP + DK * kLdP);
}

template <typename Tin, int DK, int ROWS>
__global__ void __launch_bounds__(ROWS * 4) lin_out(const Tin* __restrict__ q, const Tin* __restrict__ k,
                                                    const Tin* __restrict__ v, LinDecay dec, ChunkMap cmap, int H, int DV,
                                                    const float* S, Tin* __restrict__ o) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float gh[kC], gl[kC];
    constexpr int LD = DK + 4;
    float *sq = sm, *sk = sq + ROWS * LD, *sv = sk + kC * LD, *sp = sv + kC * kLdP, *ss = sp + ROWS * kLdP;
    int seq, tok0, len, idx;
    cmap.locate((int)blockIdx.x, seq, tok0, len, idx);
    const int h = blockIdx.y, nv = DV / 64, v0 = (int)blockIdx.z % nv * 64, i0 = (int)blockIdx.z / nv * ROWS;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (i0 >= len) {
        wait_for_kernels_before();
        return;
    }
    load_rows<Tin, ROWS, DK, ROWS * 4>(sq, LD, q, (long long)tok0 + i0, len - i0, H, h, DK, 0);
    load_rows<Tin, kC, DK, ROWS * 4>(sk, LD, k, tok0, len, H, h, DK, 0);
    load_rows<Tin, kC, 64, ROWS * 4>(sv, kLdP, v, tok0, len, H, h, DV, v0);
    chunk_decay<Tin>(gh, gl, dec, tok0, len, H, h);
    __syncthreads();
    float acc[4][4];
    clear(acc);
    mm64<DK, false, true, true>(acc, sq, LD, sk, LD, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = i0 + 4 * ty + r, j = tx + 16 * c;
            sp[(4 * ty + r) * kLdP + j] = j <= i ? acc[r][c] * exp_gdiff(gh[i], gl[i], gh[j], gl[j]) : 0.f;
        }
    wait_for_kernels_before();
    load_tile<DK, 64, ROWS * 4>(ss, kLdP, S + ((size_t)blockIdx.x * H + h) * DK * DV + v0, DV);
    __syncthreads();
    clear(acc);
    mm64<DK, false, false, false>(acc, sq, LD, ss, kLdP, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float e = exp_g(gh[i0 + 4 * ty + r], gl[i0 + 4 * ty + r]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] *= e;
    }
    mm64<kC, false, false, false>(acc, sp, kLdP, sv, kLdP, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        if (i < len) {
            Tin* dst = o + ((size_t)(tok0 + i) * H + h) * DV + v0 + 4 * tx;
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = from_f32<Tin>(acc[r][c]);
        }
    }
}

// ---- backward: one (chunk, head) and one of dq, dk, dv a block ---------------------------
// k, d_o, the decayed pairs, q, v; the tiles of S and dS' go where a role is done with an
// operand, so that two blocks fit on an SM where the widths are 64 (backward of 1024 tokens of
// 16 heads 80 -> 69 us).
template <int DK, int DV> constexpr size_t grad_smem() {
    return sizeof(float) * (2 * kC * (DK + 4) + 2 * kC * (DV + 4) + kC * kLdP);
}

// sum over the 16 threads that share rows 4 ty + r, added to dst by the first of them
__device__ __forceinline__ void add_row_sums(float* dst, const float (&s)[4], int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float x = s[r];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (tx == 0) dst[4 * ty + r] += x;
    }
}

// What dlog_alpha is put together from, per unit = (chunk, head): a[i] = q_i . e^{g_i} (S d_o_i),
// b[j] = k_j . e^{g_C - g_j} (dS' v_j), r[t] = sum over i >= t > j, e = e^{g_C} <dS', S>.
struct DecayParts {
    float *a, *b, *r, *e;   // [units, 64] each, e [units]
};

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2)
lin_grad(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v, LinDecay dec,
         const Tin* __restrict__ d_o, ChunkMap cmap, int H, const float* S, const float* dS,
         Tin* __restrict__ dq, Tin* __restrict__ dk, Tin* __restrict__ dv, DecayParts parts) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float gh[kC], gl[kC], w[kC], ra[kC], red[kThreads / 32];
    constexpr int LK = DK + 4, LV = DV + 4;
    static_assert(DK * kLdP <= kC * LK + kC * LV, "dv's tile goes over q and v");
    float *sk = sm, *sd = sk + kC * LK, *sp = sd + kC * LV, *sq = sp + kC * kLdP, *sv = sq + kC * LK;
    let_next_kernel_start();
    int seq, tok0, len, idx;
    cmap.locate((int)blockIdx.x, seq, tok0, len, idx);
    const int h = blockIdx.y, role = blockIdx.z, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;   // dq, dk, dv
    float* tile = role == 0 ? sv : role == 1 ? sd : sq;   // once the pairs are formed
    const size_t unit = (size_t)blockIdx.x * H + h;
    const float *Sn = S + unit * DK * DV, *dSn = dS + unit * DK * DV;
    load_rows<Tin, kC, DK, kThreads>(sq, LK, q, tok0, len, H, h, DK, 0);
    load_rows<Tin, kC, DK, kThreads>(sk, LK, k, tok0, len, H, h, DK, 0);
    if (role < 2) load_rows<Tin, kC, DV, kThreads>(sv, LV, v, tok0, len, H, h, DV, 0);
    load_rows<Tin, kC, DV, kThreads>(sd, LV, d_o, tok0, len, H, h, DV, 0);
    chunk_decay<Tin>(gh, gl, dec, tok0, len, H, h);
    __syncthreads();
    if (tid < kC) {
        w[tid] = role == 0 ? exp_g(gh[tid], gl[tid]) : exp_gdiff(gh[kC - 1], gl[kC - 1], gh[tid], gl[tid]);
        ra[tid] = 0.f;
    }
    float p[4][4], a[4][4];
    clear(p);
    clear(a);
    if (role != 1) mm64<DK, false, true, true>(p, sq, LK, sk, LK, ty, tx);
    if (role != 2) mm64<DV, false, true, true>(a, sd, LV, sv, LV, ty, tx);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 4 * ty + r, j = tx + 16 * c;
            const float d = j <= i ? exp_gdiff(gh[i], gl[i], gh[j], gl[j]) : 0.f;
            sp[i * kLdP + j] = j <= i ? (role == 2 ? p[r][c] : a[r][c]) * d : 0.f;   // P, or dA
            if (role == 0) tile[i * kLdM + j] = j < i ? p[r][c] * a[r][c] * d : 0.f;
        }
    wait_for_kernels_before();
    if (role == 2) {
        float e = 0.f;   // <dS', S>
#pragma unroll 8
        for (int u = tid; u < DK * DV / 4; u += kThreads) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(Sn) + u), y = __ldcg(reinterpret_cast<const float4*>(dSn) + u);
            e += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
        if ((tid & 31) == 0) red[tid >> 5] = e;
    }
    __syncthreads();
    if (role == 2 && tid == 0) {
        float whole = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) whole += red[i];
        parts.e[unit] = whole * exp_g(gh[kC - 1], gl[kC - 1]);
    }
    if (role == 0) {   // r[t] = sum of the pair products over i >= t > j, four threads a row, then four a column
        const int i = tid >> 2, part = tid & 3;
        float* row = tile + i * kLdM + 16 * part;
        float run = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) run += row[j];
        float before = 0.f;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            const float y = __shfl_sync(0xffffffffu, run, u, 4);
            if (u < part) before += y;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            before += row[j];
            row[j] = before;
        }
        __syncthreads();
        const int t = tid >> 2;
        float sum = 0.f;
        for (int r = t + ((part - t) & 3); t > 0 && r < kC; r += 4) sum += tile[r * kLdM + t - 1];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (part == 0) parts.r[unit * kC + t] = sum;
    }
    if (role < 2) {   // dq from S and dA k, or dk from dS' and dA^T q
        const float* x = role ? sk : sq;
        Tin* out = role ? dk : dq;
        for (int k0 = 0; k0 < DK; k0 += 64) {
            __syncthreads();
            load_tile<64, DV, kThreads>(tile, LV, (role ? dSn : Sn) + (size_t)k0 * DV, DV);
            __syncthreads();
            clear(p);
            clear(a);
            if (role == 0) {
                mm64<DV, false, true, true>(p, sd, LV, tile, LV, ty, tx);
                mm64<kC, false, false, true>(a, sp, kLdP, sk + k0, LK, ty, tx);
            } else {
                mm64<DV, false, true, true>(p, sv, LV, tile, LV, ty, tx);
                mm64<kC, true, false, true>(a, sp, kLdP, sq + k0, LK, ty, tx);
            }
            float s1[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                const float wi = w[i];
                s1[r] = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = tx + 16 * c;
                    const float inter = wi * p[r][c];
                    s1[r] = fmaf(x[i * LK + k0 + j], inter, s1[r]);
                    if (i < len) out[((size_t)(tok0 + i) * H + h) * DK + k0 + j] = from_f32<Tin>(inter + a[r][c]);
                }
            }
            add_row_sums(ra, s1, ty, tx);
        }
        __syncthreads();
        if (tid < kC) (role ? parts.b : parts.a)[unit * kC + tid] = ra[tid];
    } else {
        for (int v0 = 0; v0 < DV; v0 += 64) {
            __syncthreads();
            load_tile<DK, 64, kThreads>(tile, kLdP, dSn + v0, DV);
            __syncthreads();
            clear(p);
            mm64<DK, false, false, false>(p, sk, LK, tile, kLdP, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) p[r][c] *= w[4 * ty + r];
            mm64<kC, true, false, false>(p, sp, kLdP, sd + v0, LV, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                if (i < len) {
                    Tin* dst = dv + ((size_t)(tok0 + i) * H + h) * DV + v0 + 4 * tx;
#pragma unroll
                    for (int c = 0; c < 4; ++c) dst[c] = from_f32<Tin>(p[r][c]);
                }
            }
        }
    }
}

// dlog_alpha of one unit a warp: suffix sums of a, exclusive prefix sums of b, two tokens a lane
template <typename Tin>
__global__ void __launch_bounds__(128) lin_decay_grad(DecayParts parts, LinDecay dec, ChunkMap cmap, int n_units, int H,
                                                      Tin* __restrict__ dla) {
    const int unit = (int)blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    wait_for_kernels_before();
    if (unit >= n_units) return;
    int seq, tok0, len, idx;
    cmap.locate(unit / H, seq, tok0, len, idx);
    const int h = unit % H, t = 2 * lane;
    const float2 a = __ldcg(reinterpret_cast<const float2*>(parts.a + (size_t)unit * kC) + lane);
    const float2 b = __ldcg(reinterpret_cast<const float2*>(parts.b + (size_t)unit * kC) + lane);
    const float2 r = __ldcg(reinterpret_cast<const float2*>(parts.r + (size_t)unit * kC) + lane);
    const float whole = __ldcg(parts.e + unit);
    float suf = a.x + a.y, pre = b.x + b.y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, suf, off), z = __shfl_up_sync(0xffffffffu, pre, off);
        if (lane + off < 32) suf += y;
        if (lane >= off) pre += z;
    }
    // the lane's own terms are left out by taking its neighbour's sums, not by subtraction
    float next = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
    if (lane == 31) next = 0.f;
    if (lane == 0) before = 0.f;
    const float x[2] = {suf + before + whole + r.x, next + a.y + before + b.x + whole + r.y};
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (t + u < len) {
            const size_t tok = (size_t)tok0 + t + u;
            const bool floored = lin_raw_decay<Tin>(dec, tok, H, h) < kLogAlphaFloor;
            dla[tok * H + h] = from_f32<Tin>(floored ? 0.f : x[u]);
        }
}

// Tiles of 16 rows as long as there is an SM for each of them: a quarter of the work a block,
// but the chunk's operands are read four times.  Forward with tiles of 16 and of 64 rows: 12.4
// and 14.4 us for 8 (chunk, head) pairs, 16.5 and 16.4 for 80, 26.3 and 18.5 for 128.
bool small_grid(long long blocks) { return 4 * blocks <= 148; }

template <typename Tin>
cudaError_t update_and_chain(UpdateSide<Tin> fwd, UpdateSide<Tin> rev, int sides, LinDecay dec, ChainSide cf, ChainSide cr,
                             const ChunkMap& cmap, const SeqMap& smap, int n_chunks, int n_seqs, int H, int dk, int dv,
                             float* gam, cudaStream_t s) {
    if (n_chunks > 0) {
        const int tiles = (dk / 64) * (dv / 64) * sides;
        const bool small = small_grid((long long)n_chunks * H * tiles);
        auto update = small ? lin_update<Tin, 16> : lin_update<Tin, 64>;
        if (sides == 2) {
            // The gradient kernel's 87 to 153 KB of shared memory can only come onto an SM beside
            // these two if the SM is divided for that already (50 -> 46 us for 14 chunks x 3 heads).
            cudaError_t e;
            const auto all = cudaFuncAttributePreferredSharedMemoryCarveout;
            if ((e = cudaFuncSetAttribute(update, all, cudaSharedmemCarveoutMaxShared)) != cudaSuccess ||
                (e = cudaFuncSetAttribute(lin_chain, all, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
                return e;
        }
        update<<<dim3(n_chunks, H, small ? 4 * tiles : tiles), small ? 64 : kThreads, 0, s>>>(fwd, rev, dec, cmap, H, dk, dv,
                                                                                             gam);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int e4 = dk * dv / 4;
    const dim3 grid((unsigned)n_seqs * H, e4 / kThreads, sides);
    if (n_chunks > 0) return launch_behind(lin_chain, grid, kThreads, 0, s, cf, cr, gam, smap, H, e4);
    lin_chain<<<grid, kThreads, 0, s>>>(cf, cr, gam, smap, H, e4);
    return cudaGetLastError();
}

template <typename Tin, int DK, int ROWS>
cudaError_t outputs(const void* q, const void* k, const void* v, LinDecay dec, void* o, const ChunkMap& cmap, int n_chunks,
                    int H, int dv, const LinSimtWorkspace& ws, cudaStream_t s) {
    auto kern = lin_out<Tin, DK, ROWS>;
    constexpr size_t smem = out_smem<DK, ROWS>();
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    return launch_behind(kern, dim3(n_chunks, H, dv / 64 * (kC / ROWS)), ROWS * 4, smem, s, (const Tin*)q, (const Tin*)k,
                         (const Tin*)v, dec, cmap, H, dv, ws.S, (Tin*)o);
}

template <typename Tin>
cudaError_t fwd(const void* q, const void* k, const void* v, LinDecay dec, const float* init, void* o, float* final,
                const ChunkMap& cmap, const SeqMap& smap, int n_chunks, int n_seqs, int H, int dk, int dv,
                const LinSimtWorkspace& ws, cudaStream_t s) {
    const UpdateSide<Tin> u{(const Tin*)k, (const Tin*)v, ws.S};
    const ChainSide c{ws.S, init, final};
    const cudaError_t err = update_and_chain<Tin>(u, u, 1, dec, c, c, cmap, smap, n_chunks, n_seqs, H, dk, dv, ws.gam, s);
    if (err != cudaSuccess || n_chunks == 0) return err;
    if (small_grid((long long)n_chunks * H * (dv / 64)))
        return dk == 128 ? outputs<Tin, 128, 16>(q, k, v, dec, o, cmap, n_chunks, H, dv, ws, s)
                         : outputs<Tin, 64, 16>(q, k, v, dec, o, cmap, n_chunks, H, dv, ws, s);
    return dk == 128 ? outputs<Tin, 128, 64>(q, k, v, dec, o, cmap, n_chunks, H, dv, ws, s)
                     : outputs<Tin, 64, 64>(q, k, v, dec, o, cmap, n_chunks, H, dv, ws, s);
}

template <typename Tin, int DK, int DV>
cudaError_t grad(const void* q, const void* k, const void* v, LinDecay dec, const void* d_o, void* dq, void* dk,
                 void* dv, void* dla, const ChunkMap& cmap, int n_chunks, int H, const LinSimtWorkspace& ws,
                 cudaStream_t s) {
    auto kern = lin_grad<Tin, DK, DV>;
    constexpr size_t smem = grad_smem<DK, DV>();
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    const int units = n_chunks * H;
    const size_t n = (size_t)units * kC;
    const DecayParts parts{ws.parts, ws.parts + n, ws.parts + 2 * n, ws.parts + 3 * n};
    const cudaError_t st = launch_behind(kern, dim3(n_chunks, H, 3), kThreads, smem, s, (const Tin*)q, (const Tin*)k,
                                         (const Tin*)v, dec, (const Tin*)d_o, cmap, H, ws.S, ws.dS, (Tin*)dq, (Tin*)dk,
                                         (Tin*)dv, parts);
    if (st != cudaSuccess || dec.per_head) return st;
    return launch_behind(lin_decay_grad<Tin>, (units + 3) / 4, 128, 0, s, parts, dec, cmap, units, H, (Tin*)dla);
}

template <typename Tin>
cudaError_t bwd(const void* q, const void* k, const void* v, LinDecay dec, const float* init, const void* d_o,
                const float* d_final, void* dq, void* dk_out, void* dv_out, void* dla, float* d_init,
                const ChunkMap& cmap, const SeqMap& smap, int n_chunks, int n_seqs, int H, int dk, int dv,
                const LinSimtWorkspace& ws, cudaStream_t s) {
    const UpdateSide<Tin> uf{(const Tin*)k, (const Tin*)v, ws.S}, ur{(const Tin*)q, (const Tin*)d_o, ws.dS};
    const ChainSide cf{ws.S, init, nullptr}, cr{ws.dS, d_final, d_init};
    const cudaError_t err = update_and_chain<Tin>(uf, ur, 2, dec, cf, cr, cmap, smap, n_chunks, n_seqs, H, dk, dv, ws.gam,
                                                  s);
    if (err != cudaSuccess || n_chunks == 0) return err;
    if (dk == 128 && dv == 128)
        return grad<Tin, 128, 128>(q, k, v, dec, d_o, dq, dk_out, dv_out, dla, cmap, n_chunks, H, ws, s);
    if (dk == 128) return grad<Tin, 128, 64>(q, k, v, dec, d_o, dq, dk_out, dv_out, dla, cmap, n_chunks, H, ws, s);
    if (dv == 128) return grad<Tin, 64, 128>(q, k, v, dec, d_o, dq, dk_out, dv_out, dla, cmap, n_chunks, H, ws, s);
    return grad<Tin, 64, 64>(q, k, v, dec, d_o, dq, dk_out, dv_out, dla, cmap, n_chunks, H, ws, s);
}

}  // namespace

cudaError_t launch_lin_simt_fwd(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                                const float* init_state, void* o, float* final_state, const ChunkMap& cmap,
                                const SeqMap& smap, int n_chunks, int n_seqs, int H, int dk, int dv,
                                const LinSimtWorkspace& ws, cudaStream_t stream) {
    auto f = dtype == KDA_F32 ? fwd<float> : fwd<__nv_bfloat16>;
    return f(q, k, v, dec, init_state, o, final_state, cmap, smap, n_chunks, n_seqs, H, dk, dv, ws, stream);
}

cudaError_t launch_lin_simt_bwd(kda_dtype dtype, const void* q, const void* k, const void* v, LinDecay dec,
                                const float* init_state, const void* d_o, const float* d_final, void* dq, void* dk_out,
                                void* dv_out, void* dla, float* d_init, const ChunkMap& cmap, const SeqMap& smap,
                                int n_chunks, int n_seqs, int H, int dk, int dv, const LinSimtWorkspace& ws,
                                cudaStream_t stream) {
    auto f = dtype == KDA_F32 ? bwd<float> : bwd<__nv_bfloat16>;
    return f(q, k, v, dec, init_state, d_o, d_final, dq, dk_out, dv_out, dla, d_init, cmap, smap, n_chunks, n_seqs, H,
             dk, dv, ws, stream);
}

}  // namespace kda
