// Gradients of linear attention with one decay a head on the tensor cores (bf16,
// d_k = d_v = 128), one 128-token chunk of one head at a time, once every chunk's start
// state S and the gradient Z of its end state are known (as bf16 images).  With
// D_ij = e^{g_i - g_j} (j <= i), w_j = e^{g_C - g_j}:
//   P = D . (Q K^T),  B = D . (dO V^T)                        rounded to bf16 as operands
//   dQ = e^g (dO S^T) + B K      dK = w (V Z^T) + B^T Q      dV = w (K Z) + P^T dO
//   dlog_alpha_t = sum_{i >= t} q_i . e^{g_i} (S dO_i) + sum_{j < t} k_j . w_j (Z v_j)
//                + e^{g_C} <Z, S> + sum_{i >= t > j} P_ij (dO V^T)_ij
// Every term of the last lines is one that t's decay enters, so none is added and taken away
// again; the last one, over a rectangle of M = P . (dO V^T) in fp32, is put together from sums over
// 32 x 32 blocks: columns and rows of the blocks wholly inside, and a running sum in the
// block on the diagonal.
//
// Eight products of 128^3 a chunk (4096 tensor cycles) against 288 KB of memory traffic
// (6.6 us an SM at the measured copy rate): bound by memory as long as loads overlap the
// work.  2048 (chunk, head) units take 138 to 146 us, 4.1 to 4.3 TB/s; of a unit's 17 K cycles
// the elementwise warps spend 14 K, and 3 K waiting for the next Q and K.  A block keeps one chunk
// in six 32 KB slots; a slot is loaded for the block's next chunk as soon as nothing needs it.
// P and B replace S and V.  The results leave through slots too (dV Z's, dQ K's, dK Q's: free by then, and needed last by the next chunk), one box
// a warp: stored from registers, a row a lane, they held the load/store pipe for 3000 cycles.
// 16 warps do the elementwise work: warp (R, B) owns rows 32 R + lane and columns
// 32 B + [0, 32).
#include <algorithm>

#include "kda_launch.cuh"
#include "kda_linear_tc.cuh"

namespace kda {
namespace lintc {
namespace {

constexpr int kGradThreads = 640;   // warps 0-15 elementwise, 16 products, 17 loads, 18 decays, 19 dlog_alpha
enum Slot { kQ = 0, kK, kV, kDO, kS, kZ, kSlotsN };
constexpr uint32_t kOffGates = kSlotsN * kTile;

struct GradSums {
    float a[4][kT];      // by column block: this block's part of q . e^g (S dO), a row each
    float b[4][kT];      // the same of k . w (Z v)
    float rows[4][kT];   // row sums of M in column block B (B before the row's block)
    float cols[4][kT];   // column sums of M in row block R (R behind the column's block)
    float diag[kT];      // the diagonal block's sums over i >= t > j
    float total[4][4];   // sums of whole blocks [R][B]
    float zs[16];        // <Z, S>, a warp each
};
constexpr uint32_t kOffSums = kOffGates + 2 * sizeof(Gates);
constexpr uint32_t kOffBars = kOffSums + sizeof(GradSums);
constexpr uint32_t kGradSmem = kOffBars + 256;
static_assert(kOffBars % 8 == 0 && kGradSmem <= 232448, "shared memory per block");

enum GradBar { kFull = 0, kFree = kSlotsN, kInter = 2 * kSlotsN, kKInter, kScores, kClean, kSRead, kPReady, kDvDone, kDqDone, kDkDone,
               kRead, kGFull = kRead + 3, kGEmpty = kGFull + 2, kSumsFull = kGEmpty + 2, kSumsEmpty, kDrain, kGradBars };

// lane l of the warp gets the sum over all lanes of v[l]
__device__ __forceinline__ float transpose_sum(float (&v)[32], int lane) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int k = 0; k < off; ++k) {
            const float send = up ? v[k] : v[k + off], keep = up ? v[k + off] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    return v[0];
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// dot of 16 values with 16 bf16 channels of a tile's row (channels c0 .. c0 + 15)
__device__ __forceinline__ float dot16(const float (&x)[16], const uint8_t* tile, int row, int c0) {
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 u = *reinterpret_cast<const uint4*>(tile + sw128_chunk(row, c0 + 8 * h, kT));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(x[8 * h + 2 * i], bf16_lo(w[i]), s);
            s = fmaf(x[8 * h + 2 * i + 1], bf16_hi(w[i]), s);
        }
    }
    return s;
}

__global__ void __launch_bounds__(kGradThreads, 1)
lin_grad_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
            const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, LinDecay dec,
            const __grid_constant__ CUtensorMap mdq, const __grid_constant__ CUtensorMap mdk,
            const __grid_constant__ CUtensorMap mdv, ChunkMap chunks, int n_units, int H,
            const uint8_t* __restrict__ s_images,
            const uint8_t* __restrict__ z_images, __nv_bfloat16* __restrict__ dq, __nv_bfloat16* __restrict__ dk,
            __nv_bfloat16* __restrict__ dv, __nv_bfloat16* __restrict__ dla, int* __restrict__ err, unsigned long long stall_ns) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBars);
    uint32_t* flags = reinterpret_cast<uint32_t*>(bars + kGradBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (smem_u32(sm) & 1023u) {
        if (tid == 0) atomicCAS(err, 0, (int)KDA_ERR_DEVICE);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kGradBars; ++i)   // one arrival a warp
            mbar_init(&bars[i], i == kClean || i == kSRead || i == kPReady || (i >= kRead && i < kRead + 3) || i == kSumsFull
                                    ? 16
                                : i == kGEmpty || i == kGEmpty + 1                    ? 17   // and the dlog_alpha warp
                                : i == kFree + kZ || i == kFree + kK || i == kFree + kQ ? 17   // results left, products done
                                                                                        : 1);
        mbar_init_fence();
        flags[1] = 0u;
    }
    if (warp == 16) {
        tmem_alloc(&flags[0], 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_kernels_before();   // the images
    const uint32_t tbase = flags[0];
    const uint32_t tA = tbase, tB = tbase + 128, tQ = tbase + 256, tK = tbase + 384;   // scores / dV parts, dQ, dK
    const Abort ab{&flags[1], err};
    Gates* gates = reinterpret_cast<Gates*>(sm + kOffGates);
    GradSums& sums = *reinterpret_cast<GradSums*>(sm + kOffSums);
    auto slot = [&](int i) { return sm + (uint32_t)i * kTile; };
    // unit -> chunk, head; `it` counts this block's units: the parity of every barrier but the gates'
    const int first = (int)blockIdx.x, step = (int)gridDim.x;
    constexpr int kOrder[kSlotsN] = {kS, kDO, kV, kZ, kK, kQ};   // loads, in the order the slots are free and needed
    int loads = 0;   // tiles asked for (the loads' lane): tile n stands in slot kOrder[n % 6]

    if (warp < 16) {   // ---- elementwise
        const int R = warp & 3, B = warp >> 2, row = 32 * R + lane;
        const uint32_t at = ((uint32_t)(32 * R) << 16) + 32 * B;   // this warp's lanes and columns
        int it = 0, tails = 0;   // units so far, and those with rows to clear
        const bool stalled = warp == 0 && stall(&bars[kDrain], stall_ns, ab);
        for (int u = first; !stalled && u < n_units; u += step, ++it) {
            const uint32_t par = (uint32_t)it & 1u;
            int seq, tok0, len, idx;
            chunks.locate(u / H, seq, tok0, len, idx);
            const int h = u % H;
            if (!wait_or_abort(&bars[kGFull + (it & 1)], (uint32_t)(it >> 1) & 1u, ab)) break;
            const Gates& G = gates[it & 1];
            if (len < kT) {   // rows of the next sequence: out of the sums over tokens
                if (!wait_or_abort(&bars[kFull + kQ], par, ab) || !wait_or_abort(&bars[kFull + kK], par, ab) ||
                    !wait_or_abort(&bars[kFull + kDO], par, ab))
                    break;
                zero_rows(slot(kQ), 2, len, tid, 512);
                zero_rows(slot(kK), 2, len, tid, 512);
                zero_rows(slot(kDO), 2, len, tid, 512);
                fence_async_smem();
                warp_arrive(&bars[kClean], lane);
                if (!wait_or_abort(&bars[kClean], (uint32_t)tails++ & 1u, ab)) break;
            }
            if (!wait_or_abort(&bars[kSumsEmpty], par ^ 1u, ab)) break;   // the last unit's sums are read
            const float r2 = G.rel2[row], er = ex2_approx(r2), wq = er * G.start[R], wk = G.col[row] * G.end[R];
            // the states' parts of dQ and dK: scaled where they stand, and their dots
            if (!wait_or_abort(&bars[kFull + kQ], par, ab) || !wait_or_abort(&bars[kFull + kK], par, ab)) break;
            bool ok = true;
#pragma unroll 1
            for (int side = 0; ok && side < 2; ++side) {
                if (!(ok = wait_or_abort(&bars[side ? kKInter : kInter], par, ab))) break;
                tc_fence_after();
                const uint32_t t = (side ? tK : tQ) + at;
                const float w = side ? wk : wq;
                float dot = 0.f;
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {
                    float x[16];
                    tmem_ld16(t + 16 * g, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] *= w;
                    tmem_st16(t + 16 * g, x);
                    dot += dot16(x, slot(side ? kK : kQ), row, 32 * B + 16 * g);
                }
                (side ? sums.b : sums.a)[B][row] = row < len ? dot : 0.f;
            }
            if (!ok) break;
            // <Z, S>, 1/16 of the tiles a warp
            if (!wait_or_abort(&bars[kFull + kS], par, ab) || !wait_or_abort(&bars[kFull + kZ], par, ab)) break;
            {
                float z = 0.f;
#pragma unroll 2
                for (int i = 0; i < 4; ++i) {
                    const uint32_t off = (uint32_t)(warp * 128 + i * 32 + lane) * 16;
                    const uint4 x = *reinterpret_cast<const uint4*>(slot(kS) + off), y = *reinterpret_cast<const uint4*>(slot(kZ) + off);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z = fmaf(bf16_lo(xs[e]), bf16_lo(ys[e]), z);
                        z = fmaf(bf16_hi(xs[e]), bf16_hi(ys[e]), z);
                    }
                }
                z = warp_sum(z);
                if (lane == 0) sums.zs[warp] = z;
            }
            warp_arrive(&bars[kSRead], lane);
            // P, B and the sums of M; P replaces S, once every warp has read its part
            if (!wait_or_abort(&bars[kScores], par, ab) || !wait_or_abort(&bars[kSRead], par, ab)) break;
            tc_fence_after();
            float m[32];
            if (B > R) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const uint32_t off = sw128_chunk(row, 32 * B + 8 * c, kT);
                    *reinterpret_cast<uint4*>(slot(kS) + off) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(slot(kV) + off) = make_uint4(0u, 0u, 0u, 0u);
                }
            } else {
                const float f = er * G.fac[R][B];
                const bool in = row < len;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float x[16], y[16];
                    tmem_ld16(tA + at + 16 * g, x);
                    tmem_ld16(tB + at + 16 * g, y);
                    tmem_ld_wait();
                    if (B < R) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float d = f * G.col[32 * B + 16 * g + e], p = in ? x[e] * d : 0.f;
                            m[16 * g + e] = in ? p * y[e] : 0.f;
                            x[e] = p;
                            y[e] = in ? y[e] * d : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int j = 16 * g + e;
                            const bool keep = in && j <= lane;
                            const float d = ex2_approx(r2 - G.rel2[32 * B + j]), p = keep ? x[e] * d : 0.f;
                            m[j] = keep && j < lane ? p * y[e] : 0.f;
                            x[e] = p;
                            y[e] = keep ? y[e] * d : 0.f;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t off = sw128_chunk(row, 32 * B + 16 * g + 8 * c, kT);
                        *reinterpret_cast<uint4*>(slot(kS) + off) =
                            make_uint4(pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                                       pack_bf16(x[8 * c + 4], x[8 * c + 5]), pack_bf16(x[8 * c + 6], x[8 * c + 7]));
                        *reinterpret_cast<uint4*>(slot(kV) + off) =
                            make_uint4(pack_bf16(y[8 * c], y[8 * c + 1]), pack_bf16(y[8 * c + 2], y[8 * c + 3]),
                                       pack_bf16(y[8 * c + 4], y[8 * c + 5]), pack_bf16(y[8 * c + 6], y[8 * c + 7]));
                    }
                }
            }
            tmem_st_wait();   // the scaled parts
            fence_async_smem();
            tc_fence_before();
            warp_arrive(&bars[kPReady], lane);
            if (B <= R) {
                if (B < R) {
                    float rs = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) rs += m[j];
                    sums.rows[B][row] = rs;
                    const float tot = warp_sum(rs);
                    if (lane == 0) sums.total[R][B] = tot;
                    sums.cols[R][32 * B + lane] = transpose_sum(m, lane);
                } else {   // running sums along the row (j < t), only of rows i >= t, then down the columns
                    float run = 0.f;
#pragma unroll
                    for (int t = 0; t < 32; ++t) {
                        const float here = m[t];
                        m[t] = t <= lane ? run : 0.f;
                        run += here;
                    }
                    sums.diag[32 * R + lane] = transpose_sum(m, lane);
                }
            }
            warp_arrive(&bars[kSumsFull], lane);
            warp_arrive(&bars[kGEmpty + (it & 1)], lane);
            // dV = w (K Z) + P^T dO, then dQ and dK
            const size_t base = ((size_t)(tok0 + row) * H + h) * kD + 32 * B;
            const bool whole = 32 * R + 32 <= len;
#pragma unroll 1
            for (int out = 0; out < 3; ++out) {
                if (!(ok = wait_or_abort(&bars[kDvDone + out], par, ab))) break;
                tc_fence_after();
                const int through = out == 0 ? kZ : out == 1 ? kK : kQ;
                uint8_t* stage = slot(through) + warp * 2048;
                __nv_bfloat16* dst = (out == 0 ? dv : out == 1 ? dq : dk) + base;
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {
                    float x[16];
                    tmem_ld16((out == 0 ? tB : out == 1 ? tQ : tK) + at + 16 * g, x);
                    if (out == 0) {
                        float y[16];
                        tmem_ld16(tA + at + 16 * g, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = fmaf(wk, y[e], x[e]);
                    } else {
                        tmem_ld_wait();
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                    if (whole) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            *reinterpret_cast<uint4*>(stage + lane * 64 + (((2 * g + c) ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    } else if (row < len) {
                        store32(dst + 16 * g, w);
                    }
                }
                tc_fence_before();
                warp_arrive(&bars[kRead + out], lane);   // the accumulator is free
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (whole) tma_store_box(out == 0 ? &mdv : out == 1 ? &mdq : &mdk, stage, 32 * B, h, tok0 + 32 * R);
                    bulk_commit();
                    if (out > 0) {   // the result before this one has left its slot
                        bulk_wait_read_but1();
                        mbar_arrive(&bars[kFree + (out == 1 ? kZ : kK)]);
                    }
                }
            }
            if (!ok) break;
            if (lane == 0) {
                bulk_wait_read_all();
                mbar_arrive(&bars[kFree + kQ]);
            }
        }
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        tmem_st_wait();   // (given up in between)
    } else if (warp == 16) {   // ---- products
        constexpr uint32_t iKK = idesc_bf16_f32(128, 128), iKM = idesc_bf16_f32_bmn(128, 128), iMM = idesc_amn_bmn(128, 128);
        const uint32_t lead = elect_lane(), base = smem_u32(sm);
        auto commit = [&](int bar) {
            if (lead) mma_commit(&bars[bar]);
        };
        auto ktile = [&](int i) { return sw128_desc(base + (uint32_t)i * kTile); };
        auto mtile = [&](int i) { return mn_desc_k(base + (uint32_t)i * kTile, kT, 0); };
        int it = 0, tails = 0;
        for (int u = first; u < n_units; u += step, ++it) {
            const uint32_t par = (uint32_t)it & 1u;
            int seq, tok0, len, idx;
            chunks.locate(u / H, seq, tok0, len, idx);
            // (each accumulator once the last unit's result has been read from it)
            if (it > 0 && !wait_or_abort(&bars[kRead + 1], par ^ 1u, ab)) break;
            if (!wait_or_abort(&bars[kFull + kDO], par, ab) || !wait_or_abort(&bars[kFull + kS], par, ab) ||
                (len < kT && !wait_or_abort(&bars[kClean], (uint32_t)tails++ & 1u, ab)))
                break;
            tc_fence_after();
            product<false, false>(tQ, ktile(kDO), ktile(kS), iKK, false, lead);
            commit(kInter);
            if (it > 0 && (!wait_or_abort(&bars[kRead + 2], par ^ 1u, ab) || !wait_or_abort(&bars[kRead], par ^ 1u, ab)))
                break;
            if (!wait_or_abort(&bars[kFull + kV], par, ab) || !wait_or_abort(&bars[kFull + kZ], par, ab)) break;
            tc_fence_after();
            product<false, false>(tK, ktile(kV), ktile(kZ), iKK, false, lead);
            commit(kKInter);
            if (!wait_or_abort(&bars[kFull + kQ], par, ab) || !wait_or_abort(&bars[kFull + kK], par, ab)) break;
            product<false, false>(tA, ktile(kQ), ktile(kK), iKK, false, lead);
            product<false, false>(tB, ktile(kDO), ktile(kV), iKK, false, lead);
            commit(kScores);
            // P is in S's slot, B in V's
            if (!wait_or_abort(&bars[kPReady], par, ab)) break;
            tc_fence_after();
            product<false, true>(tA, ktile(kK), mtile(kZ), iKM, false, lead);
            commit(kFree + kZ);
            product<true, true>(tB, mtile(kS), mtile(kDO), iMM, false, lead);
            commit(kDvDone);
            commit(kFree + kS);
            commit(kFree + kDO);
            product<false, true>(tQ, ktile(kV), mtile(kK), iKM, true, lead);
            commit(kDqDone);
            commit(kFree + kK);
            product<true, true>(tK, mtile(kV), mtile(kQ), iMM, true, lead);
            commit(kDkDone);
            commit(kFree + kV);
            commit(kFree + kQ);
        }
    } else if (warp == 17) {
        if (lane == 0) {   // ---- loads
            int it = 0;
            bool ok = true;
            for (int u = first; ok && u < n_units; u += step, ++it) {
                const uint32_t par = (uint32_t)it & 1u;
                int seq, tok0, len, idx;
                chunks.locate(u / H, seq, tok0, len, idx);
                const int h = u % H;
                const size_t image = (size_t)(image_of(tok0 - idx * kT, seq) + idx) * H + h;
                for (int i = 0; i < kSlotsN; ++i, ++loads) {
                    const int k = kOrder[i];
                    if (it > 0 && !(ok = wait_or_abort_lane(&bars[kFree + k], par ^ 1u, ab))) break;
                    uint64_t* bar = &bars[kFull + k];
                    mbar_arrive_expect_tx(bar, kTile);
                    if (k == kS || k == kZ) {
                        bulk_g2s(slot(k), (k == kS ? s_images : z_images) + image * kTile, kTile, bar);
                    } else {
                        const CUtensorMap* m = k == kQ ? &mq : k == kK ? &mk : k == kV ? &mv : &mdo;
                        tma_box(slot(k), m, 0, h, tok0, bar);
                        tma_box(slot(k) + kBlock, m, 64, h, tok0, bar);
                    }
                }
            }
        }
    } else if (warp == 18) {   // ---- decays
        float x[4], y[4];
        auto load = [&](int u, float(&to)[4]) {
            int seq, tok0, len, idx;
            chunks.locate(u / H, seq, tok0, len, idx);
            load_gates(to, dec, tok0, len, H, u % H, lane);
        };
        if (first < n_units) load(first, x);
        int it = 0;
        for (int u = first; u < n_units; u += step, ++it) {
            if (u + step < n_units) load(u + step, y);
            if (it >= 2 && !wait_or_abort(&bars[kGEmpty + (it & 1)], ((uint32_t)(it >> 1) & 1u) ^ 1u, ab)) break;
            make_gates(&gates[it & 1], x, lane);
            warp_arrive(&bars[kGFull + (it & 1)], lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = y[e];
        }
    } else {   // ---- dlog_alpha from the sums
        int it = 0;
        for (int u = first; u < n_units; u += step, ++it) {
            if (!wait_or_abort(&bars[kGFull + (it & 1)], (uint32_t)(it >> 1) & 1u, ab)) break;
            const float gam = gates[it & 1].gam;
            warp_arrive(&bars[kGEmpty + (it & 1)], lane);
            if (!wait_or_abort(&bars[kSumsFull], (uint32_t)it & 1u, ab)) break;
            // tokens 4 lane + e; the block of 32 is lane / 8
            const int blk = lane >> 3, t0 = 4 * lane;
            float a[4], b[4], rv[4], cv[4], dg[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t0 + e;
                a[e] = (sums.a[0][t] + sums.a[1][t]) + (sums.a[2][t] + sums.a[3][t]);
                b[e] = (sums.b[0][t] + sums.b[1][t]) + (sums.b[2][t] + sums.b[3][t]);
                rv[e] = cv[e] = 0.f;
                for (int o = 0; o < blk; ++o) rv[e] += sums.rows[o][t];          // pairs (t, j), j in blocks before
                for (int o = blk + 1; o < 4; ++o) cv[e] += sums.cols[o][t];      // pairs (i, t), i in blocks behind
                dg[e] = sums.diag[t];
            }
            float across = 0.f;   // pairs with i in a block behind and j in a block before
            for (int r = blk + 1; r < 4; ++r)
                for (int o = 0; o < blk; ++o) across += sums.total[r][o];
            float zs = 0.f;
            for (int w = 0; w < 16; ++w) zs += sums.zs[w];
            zs *= gam;
            warp_arrive(&bars[kSumsEmpty], lane);
            // suffix sums of a (chunk) and rv (block), exclusive prefix sums of b (chunk) and cv (block)
            const float as = (a[0] + a[1]) + (a[2] + a[3]), bs = (b[0] + b[1]) + (b[2] + b[3]);
            const float rs = (rv[0] + rv[1]) + (rv[2] + rv[3]), cs = (cv[0] + cv[1]) + (cv[2] + cv[3]);
            float sa = as, sr = rs, pb = bs, pc = cs;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float u1 = __shfl_down_sync(0xffffffffu, sa, off), u2 = __shfl_up_sync(0xffffffffu, pb, off);
                if (lane + off < 32) sa += u1;
                if (lane >= off) pb += u2;
                if (off < 8) {
                    const float u3 = __shfl_down_sync(0xffffffffu, sr, off, 8), u4 = __shfl_up_sync(0xffffffffu, pc, off, 8);
                    if ((lane & 7) + off < 8) sr += u3;
                    if ((lane & 7) >= off) pc += u4;
                }
            }
            float an = __shfl_down_sync(0xffffffffu, sa, 1), bp = __shfl_up_sync(0xffffffffu, pb, 1);
            float rn = __shfl_down_sync(0xffffffffu, sr, 1, 8), cp = __shfl_up_sync(0xffffffffu, pc, 1, 8);
            if (lane == 31) an = 0.f;
            if (lane == 0) bp = 0.f;
            if ((lane & 7) == 7) rn = 0.f;
            if ((lane & 7) == 0) cp = 0.f;
            if (dla != nullptr) {
                int seq, tok0, len, idx;
                chunks.locate(u / H, seq, tok0, len, idx);
                const int h = u % H;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float ta = an, tr = rn, tb = bp, tc = cp;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i >= e) { ta += a[i]; tr += rv[i]; }
                        else { tb += b[i]; tc += cv[i]; }
                    }
                    const int t = t0 + e;
                    if (t < len) {
                        const size_t tok = (size_t)tok0 + t;
                        const bool floored = lin_raw_decay<__nv_bfloat16>(dec, tok, H, h) < kLogAlphaFloor;
                        dla[tok * H + h] = __float2bfloat16_rn(floored ? 0.f : ta + tb + zs + (across + tr + tc + dg[e]));
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (gave_up(ab)) {
        if (warp == 16) drain_products(&bars[kDrain]);
#pragma unroll
        for (int j = 0; j < kSlotsN; ++j)   // the last tile of each slot
            if (loads > j) mbar_wait(&bars[kFull + kOrder[j]], (uint32_t)((loads - 1 - j) / kSlotsN) & 1u);
        __syncwarp();
    }
    if (warp == 16) tmem_dealloc(tbase, 512);
}

}  // namespace
}  // namespace lintc

using namespace lintc;

cudaError_t launch_lin_tc_grad(const void* q, const void* k, const void* v, const void* d_o, LinDecay dec, void* dq,
                               void* dk, void* dv, void* dla, const ChunkMap& chunks, int n_chunks, long long tokens,
                               int H, const uint8_t* images, const uint8_t* d_images, int* err, TestStall stall,
                               cudaStream_t s) {
    CUtensorMap mq, mk, mv, mdo;
    if (!make_map(&mq, q, tokens, H) || !make_map(&mk, k, tokens, H) || !make_map(&mv, v, tokens, H) ||
        !make_map(&mdo, d_o, tokens, H))
        return cudaErrorNotSupported;
    CUtensorMap mdq, mdk, mdv;
    if (!make_map(&mdq, dq, tokens, H, 32, 32) || !make_map(&mdk, dk, tokens, H, 32, 32) ||
        !make_map(&mdv, dv, tokens, H, 32, 32))
        return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(lin_grad_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem);
    if (e != cudaSuccess) return e;
    const int units = n_chunks * H;
    return launch_behind(lin_grad_tc, std::min(units, 148), kGradThreads, kGradSmem, s, mq, mk, mv, mdo, dec, mdq, mdk, mdv,
                         chunks, units, H, images, d_images, (__nv_bfloat16*)dq, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv,
                         dec.per_head ? nullptr : (__nv_bfloat16*)dla, err, stall.grad);
}

}  // namespace kda
