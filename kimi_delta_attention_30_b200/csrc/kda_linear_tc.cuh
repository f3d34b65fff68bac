// Building blocks shared by the tensor-core kernels of linear attention with one decay a
// head: tensor maps over [tokens, H, 128] arrays, chunk gates, waits that can be given up.
#pragma once

#include <cuda.h>

#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lintc {

using namespace tc;

constexpr int kT = 128;               // tokens a chunk
constexpr int kD = 128;               // key and value width
constexpr uint32_t kTile = 32768;     // a 128 x 128 bf16 tile: two 64-column blocks of 128 rows x 128 bytes
constexpr uint32_t kBlock = 16384;

// ---- tensor maps --------------------------------------------------------------------
// A bf16 [tokens, H, 128] array as (channel, head, token).  Loads: boxes of 64 channels x 1
// head x 128 tokens in the 128-byte swizzle that the matrix descriptors name.  Stores: boxes
// of 64 or 32 channels (128- or 64-byte swizzle) x 1 head x 32 tokens, a warp's rows.  False
// if the driver does not offer the call or rejects the array.
bool make_map(CUtensorMap* map, const void* base, long long tokens, int H, int box_channels = 64, int box_tokens = 128);

// Number of a chunk's state image: chunks of different sequences never meet, since a sequence
// that ends inside a block of 128 tokens leaves a number out (seq_tok0: its first token).
__host__ __device__ __forceinline__ long long image_of(long long seq_tok0, long long seq) { return seq_tok0 / kT + seq; }

// Box (channels x0 .. x0 + 63, head h, tokens t0 .. t0 + 127) -> 16 KB of shared memory.
// Rows past the array's end read as zero.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x0, int h, int t0, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x0), "r"(h), "r"(t0), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}

// A warp's box back to global memory (channels from x0, tokens from t0; bulk groups track it).
__device__ __forceinline__ void tma_store_box(const CUtensorMap* map, const void* src, int x0, int h, int t0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(smem_u32(src)), "r"(x0), "r"(h), "r"(t0)
                 : "memory");
}

// Products are issued by a whole warp whose elected lane (`lead`) carries the instruction:
// control and descriptors then stay uniform for the warp.  A step of a rolled loop takes its
// 64 cycles that way; the same loop under a branch of one lane took 100.  Only the low words
// of the descriptors change from step to step.
__device__ __forceinline__ void mma_lead(uint32_t d_tmem, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                         uint32_t idesc, uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d_tmem),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate), "r"(lead));
}
// A in tensor memory: bf16 pairs, one row a lane.
__device__ __forceinline__ void mma_lead_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                            uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate), "r"(lead));
}

// Arrival on `bar` once the products issued so far are done; the same lane as theirs.
__device__ __forceinline__ void commit_lead(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

__host__ __device__ constexpr uint32_t idesc_amn_bmn(int M, int N) {
    return idesc_bf16_f32(M, N) | (1u << 15) | (1u << 16);
}

// One product over K = 128 as two loops of four steps of 16.  Not unrolled further: the roles
// of a block run different code at once, and what they run once a chunk has to stay small
// enough for the instruction caches (unrolled code cost five times its issue time in fetches).
// Descriptor steps, in 16-byte units: a K-major tile moves 32 bytes a step inside a
// 64-column block and 16 KB to the next block, an MN-major tile 16 rows of 128 bytes.
__device__ __forceinline__ uint32_t step_of(bool mn, int s) { return mn ? 128u : s == 3 ? 1024u - 6u : 2u; }

template <bool AMN, bool BMN>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
    uint32_t alo = (uint32_t)a, blo = (uint32_t)b, acc = add;
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            mma_lead(d, alo, (uint32_t)(a >> 32), blo, (uint32_t)(b >> 32), idesc, acc, lead);
            acc = 1u;
            alo += step_of(AMN, s);
            blo += step_of(BMN, s);
        }
}
// A in tensor memory, 128 bf16 a row: 32 words from a on and 32 from a + 64 on
__device__ __forceinline__ void product_ta(uint32_t d, uint32_t a, uint64_t b_mn, uint32_t idesc, uint32_t lead) {
    uint32_t blo = (uint32_t)b_mn, acc = 0u;
#pragma unroll 1
    for (int half = 0; half < 2; ++half, a += 64)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            mma_lead_ta(d, a + 8 * s, blo, (uint32_t)(b_mn >> 32), idesc, acc, lead);
            acc = 1u;
            blo += 128u;
        }
}

// 8 words (bf16 pairs) a lane into tensor memory
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t* w) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// ---- waits ----------------------------------------------------------------------------
// Every wait ends: after two seconds, or as soon as another role has given up, it returns
// false and the caller leaves its loop.  A warp decides by vote, so that its lanes stay
// together on the way out too.
struct Abort {
    uint32_t* flag;   // shared memory
    int* err;         // the workspace's error word
};
__device__ __forceinline__ bool given_up(uint64_t t0, const Abort& A) {
    if (*reinterpret_cast<volatile uint32_t*>(A.flag)) return true;
    if (globaltimer_ns() - t0 <= 2000000000ull) return false;
    atomicCAS(A.err, 0, (int)KDA_ERR_TIMEOUT);
    *reinterpret_cast<volatile uint32_t*>(A.flag) = 1u;
    return true;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const Abort& A) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63u) == 0u && __any_sync(0xffffffffu, given_up(t0, A))) return false;
    }
}
// The same for a single lane.
__device__ __forceinline__ bool wait_or_abort_lane(uint64_t* bar, uint32_t parity, const Abort& A) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0u && given_up(t0, A)) return false;
    }
}

// Test of the failure path (ns != 0: kda_set_test_wait_limit): one warp of the first block waits on
// a barrier that nothing completes before a role gives up, and then gives up as any wait that
// has run out.  True if it has.
__device__ __forceinline__ bool stall(uint64_t* never, unsigned long long ns, const Abort& A) {
    if (ns == 0ull || blockIdx.x != 0) return false;
    const bool out = !mbar_wait(never, 0u, ns);
    if (out) {
        atomicCAS(A.err, 0, (int)KDA_ERR_TIMEOUT);
        *reinterpret_cast<volatile uint32_t*>(A.flag) = 1u;
    }
    return __any_sync(0xffffffffu, out);
}
// The block's end (all roles are out of their loops): whether one of them gave up.  What the others
// had issued by then may still be on its way, so copies have to land and products to end first.
__device__ __forceinline__ bool gave_up(const Abort& A) { return *reinterpret_cast<volatile uint32_t*>(A.flag) != 0u; }
// (by the warp that issued the products)
__device__ __forceinline__ void drain_products(uint64_t* bar) {
    commit_lead(bar, elect_lane());
    mbar_wait(bar, 0u);
}

// ---- a chunk's decays -------------------------------------------------------------------
// The 128 tokens are four blocks of 32.  With g the inclusive sum of log decays from the
// chunk's start, every decay the kernels need is a product of numbers that are at most 1:
//   e^{g_i}       = start[R] erel[i]               R the block of i
//   e^{g_C - g_j} = end[B] col[j]                  B the block of j
//   e^{g_i - g_j} = erel[i] fac[R][B] col[j]       B < R
// with erel[i] = e^{g_i - (g before block R)}, col[j] = e^{(g at the end of block B) - g_j}.
// Inside a block e^{g_i - g_j} = 2^{rel2[i] - rel2[j]}.  Sums run in 64-bit fixed point
// (base-2 logarithms, 32 fractional bits): exact, so that resets (-100 a token) do not blur
// the decays behind them, and three times faster than in fp64 (1750 cycles a chunk, which
// held up the weighting warps).
struct Gates {
    float rel2[kT];      // log2 e (g_i - g before the block); erel is 2 to that
    float col[kT];
    float fac[4][4];
    float start[4];
    float end[4];
    float gam;           // e^{g_C}
    float pad[3];
};
static_assert(sizeof(Gates) == 1136, "gate buffer");

// Four log decays a lane (tokens 4 lane + u), zero past `len`.
template <typename Tin = __nv_bfloat16>
__device__ __forceinline__ void load_gates(float (&x)[4], const LinDecay& dec, long long tok0, int len, int H, int h,
                                           int lane) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int t = 4 * lane + u;
        x[u] = t < len ? lin_log_decay<Tin>(dec, (size_t)(tok0 + t), H, h) : 0.f;
    }
}

__device__ __forceinline__ long long fixed_log2(float log_alpha) {
    return __float2ll_rn(log_alpha * (1.4426950408889634f * 4294967296.f));
}
__device__ __forceinline__ float from_fixed(long long x) { return __ll2float_rn(x) * (1.f / 4294967296.f); }

// Inclusive sums over the warp's 128 tokens: p[u] inside the lane, the lane's total scanned.
// Fixed point has no NaN: where one is among the decays, the chunk's weights and its whole decay
// are set to it, so that results and states show it as they would any other NaN.
struct Sums {
    long long p[4], incl, before;   // incl: sum up to the lane's last token; before: ahead of its first
    bool nan;
};
__device__ __forceinline__ float or_nan(bool nan, float x) { return nan ? __int_as_float(0x7fffffff) : x; }
__device__ __forceinline__ Sums scan_gates(const float (&x)[4], int lane) {
    Sums S;
    S.nan = __any_sync(0xffffffffu, x[0] != x[0] || x[1] != x[1] || x[2] != x[2] || x[3] != x[3]);
    S.p[0] = fixed_log2(x[0]);
#pragma unroll
    for (int u = 1; u < 4; ++u) S.p[u] = S.p[u - 1] + fixed_log2(x[u]);
    S.incl = S.p[3];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, S.incl, off);
        if (lane >= off) S.incl += y;
    }
    S.before = S.incl - S.p[3];
    return S;
}

// One warp turns them into the chunk's gates.
__device__ __forceinline__ void make_gates(Gates* G, const float (&x)[4], int lane) {
    const Sums S = scan_gates(x, lane);
    const int blk = lane >> 3;
    long long s = __shfl_sync(0xffffffffu, S.incl, (8 * blk + 31) & 31);   // end of the block before
    if (blk == 0) s = 0;
    const long long e = __shfl_sync(0xffffffffu, S.incl, 8 * blk + 7);
    const long long all = __shfl_sync(0xffffffffu, S.incl, 31);
    float4 r2, co;
    float* r2p = &r2.x;
    float* cop = &co.x;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long g = S.before + S.p[u];
        r2p[u] = or_nan(S.nan, from_fixed(g - s));
        cop[u] = or_nan(S.nan, ex2_approx(from_fixed(e - g)));
    }
    reinterpret_cast<float4*>(G->rel2)[lane] = r2;
    reinterpret_cast<float4*>(G->col)[lane] = co;
    const int R = (lane >> 2) & 3, B = lane & 3;
    long long rs = __shfl_sync(0xffffffffu, S.incl, (8 * R + 31) & 31);
    const long long be = __shfl_sync(0xffffffffu, S.incl, 8 * B + 7);
    if (R == 0) rs = 0;
    if (lane < 16) G->fac[R][B] = B < R ? ex2_approx(from_fixed(rs - be)) : 0.f;
    if (lane < 16 && B == 0) G->start[R] = ex2_approx(from_fixed(rs));
    if (lane < 4) G->end[B] = ex2_approx(from_fixed(all - be));
    if (lane == 0) G->gam = or_nan(S.nan, ex2_approx(from_fixed(all)));
}

// The state chains need only the weights of a chunk's rows (e^{g_C - g}, reversed e^g) and
// its whole decay.
struct Weights {
    float w[kT];
    float gam;
    float pad[3];
};
__device__ __forceinline__ long long make_weights(Weights* W, const float (&x)[4], bool rev, int lane) {
    const Sums S = scan_gates(x, lane);
    const long long all = __shfl_sync(0xffffffffu, S.incl, 31);
    float4 w;
    float* wp = &w.x;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long g = S.before + S.p[u];
        wp[u] = or_nan(S.nan, ex2_approx(from_fixed(rev ? g : all - g)));
    }
    reinterpret_cast<float4*>(W->w)[lane] = w;
    if (lane == 0) W->gam = or_nan(S.nan, ex2_approx(from_fixed(all)));
    return all;
}

// Registers a thread of this warpgroup holds from here on (all four warps call it).
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One arrival for a warp, after everything its lanes wrote or read before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// 32 bytes a lane, its row's, in two stores: results are 16-byte aligned, no more is asked for
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// ---- the weighted rows as a bf16 pair ------------------------------------------------------
// One thread scales 8 N channels of a 64-column block's row, from 16-byte piece c0 on, by w:
// high parts to `hi` (which may be the row itself), low parts to `lo`, all in the same
// swizzled layout.  hi + lo carries 16 bits.
template <int N>
__device__ __forceinline__ void scale_split_row(const uint8_t* src_block, uint8_t* hi_block, uint8_t* lo_block, int row,
                                                int c0, float w, bool live) {
    const uint8_t* src = src_block + row * 128;
    uint8_t *hi = hi_block + row * 128, *lo = lo_block + row * 128;
    const float2 w2 = make_float2(w, w);
#pragma unroll 4
    for (int c = 0; c < N; ++c) {
        const uint32_t off = (uint32_t)(((c0 + c) ^ (row & 7)) << 4);
        uint4 x = *reinterpret_cast<const uint4*>(src + off), y = make_uint4(0u, 0u, 0u, 0u);
        if (live) {
            uint32_t* xp = &x.x;
            uint32_t* yp = &y.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = mul2(unpack_bf16x2(xp[i]), w2);
                split2(v.x, v.y, xp[i], yp[i]);
            }
        } else {
            x = y;   // rows past the chunk's end weigh nothing, whatever they hold
        }
        *reinterpret_cast<uint4*>(hi + off) = x;
        *reinterpret_cast<uint4*>(lo + off) = y;
    }
}

// Rows >= len of a tile of `blocks` 64-column blocks set to zero by `threads` threads.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int blocks, int len, int tid, int threads) {
    for (int u = tid; u < blocks * (kT - len) * 8; u += threads) {
        const int c = u & 7, r = len + (u >> 3) % (kT - len), b = (u >> 3) / (kT - len);
        *reinterpret_cast<uint4*>(tile + b * kBlock + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace lintc
}  // namespace kda
