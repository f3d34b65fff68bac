// Linear attention with one decay a head on the tensor cores (bf16, d_k = d_v = 128).
//
// A block walks the 128-token chunks of one (segment, head, BV value columns) with the
// state in fp32 registers.  For a chunk with start state S (g: inclusive sum of its log
// decays, D_ij = e^{g_i - g_j} for j <= i):
//   A = Q K^T                      fp32 in tensor memory
//   P = A . D                      rounded to bf16, back into tensor memory as an A operand
//   O = P V + e^{g} (Q S)          S read as a bf16 copy
//   U = (e^{g_C - g} K)^T V        the weighted keys as a bf16 pair (two products); with half
//                                  the value columns the values are weighted instead, which
//                                  is half the work and leaves the keys as they are
//   S <- e^{g_C} S + U             fp32
// The only roundings to 8 bits are P and the copy of S that the queries read, both of the
// kind that o itself takes when it is stored; the state sees 16-bit operands, since its
// errors would be carried from chunk to chunk and it is returned in fp32.  That pair is what the
// fp32 states are off by: 2.2e-6 of their 2-norm against 64 bits, the sums alone 5.5e-7 (fp32
// products on the CUDA cores 2e-7).  A third part would take half of U's time again, on the path
// from chunk to chunk, and 32 KB (16 KB) of shared memory that neither layout has left.
//
// Roles, each with its own barriers, so that they work on different chunks at once: 8 warps
// form o and keep the state (warp w: rows 32 (w % 4) + lane, column half w / 4), 8 weight the
// keys (or values), 8 turn scores into P, one issues the products, one the loads, one forms
// the decays.  The state is off the products' path: U needs no state, so the chain from chunk
// to chunk is one multiply-add and the copy for the next queries.
//   All 128 value columns a block: five 32 KB slots hold Q, K, V in turn; products in the order
//   P V, Q S, U, then Q K^T of the next chunk (the keys are weighted in place, behind the
//   scores).  A chunk moves 576 KB through shared memory, 4500 cycles at 128 bytes a cycle, of
//   5500 seen; 148 blocks of 32 chunks take 112 to 119 us, 5.2 to 5.5 TB/s, 0.81 to 0.85 of
//   the copy rate (128 us from a cold cache; times below too are of calls back to back).
//   Half of them, where the pairs of sequence and head are fewer than the SMs: two chunks of
//   each operand and two sets of scores; products in the order Q S, U, then Q K^T of the next
//   chunk and P V, which give the state's warps time for S (86 us for 64 pairs of 32 chunks)
//   and, with 32-bit descriptor steps (78 us) and five waits a chunk instead of eight (73 us),
//   bring a chunk to 3700 cycles of 1920 that the products take alone: it is bound by
//   latencies around the one warp that issues them.  98 us with all columns a block.  Two
//   warps issuing (one Q S and U, the other Q K^T and P V) took 87 us instead of 78: the
//   second's products delay the state's.  A single call from a cold cache takes 77 to 82 us.
// Rows past a sequence's end are loaded with the box (they belong to the next sequence); K's
// are weighted with zero, V's are cleared, Q's only reach rows of o that are not stored.
#include <algorithm>

#include "kda_launch.cuh"
#include "kda_linear_tc.cuh"

namespace kda {
namespace lintc {

bool make_map(CUtensorMap* map, const void* base, long long tokens, int H, int box_channels, int box_tokens) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (Encode)fn;
    }();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)H * kD * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box_channels, 1, (cuuint32_t)box_tokens}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_channels == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kWalkThreads = 896;    // warps 0-7 o and the state, 8-15 weights, 16 products, 17 loads, 18 decays, 20-27 P
constexpr int kStateThreads = 640;   // the same without P

// an entry of a table that the kernel before wrote
__device__ __forceinline__ SeqInfo load_written(const SeqInfo* p) {
    static_assert(sizeof(SeqInfo) == sizeof(int4), "one load");
    const int4 x = __ldcg(reinterpret_cast<const int4*>(p));
    SeqInfo s;
    memcpy(&s, &x, sizeof s);
    return s;
}

// whether segment `idx` of sequence `seq` is its last
__device__ __forceinline__ bool last_segment(const ChunkMap& segs, int seq, int idx) {
    const int len = segs.seqs ? segs.seqs[seq].len : segs.T;
    return idx == (len + segs.C - 1) / segs.C - 1;
}

// ---- outputs ------------------------------------------------------------------------
constexpr int kSlots = 6;                              // barriers; five slots of 32 KB, or four and two halves
constexpr uint32_t kOffLo = 5 * kTile;                 // low parts of the weighted keys; both parts of the values
constexpr uint32_t kOffS = kOffLo + kTile;             // the state's copy (and o on its way out)
constexpr uint32_t kOffGates = kOffS + kTile;
constexpr uint32_t kOffBars = kOffGates + 2 * sizeof(Gates);
constexpr uint32_t kWalkSmem = kOffBars + 256;
static_assert(kWalkSmem <= 232448, "shared memory per block");

// Barriers in pairs are used by turns, one chunk the one and the next the other: what waits for
// one may come late by a chunk, but never by two.
enum WalkBar { kFull = 0, kScores = kSlots, kPReady = kScores + 2, kQsDone = kPReady + 2, kUDone = kQsDone + 2,
               kODone = kUDone + 2, kGFull = kODone + 2, kGEmpty = kGFull + 2, kKReady = kGEmpty + 2, kORead, kSReady,
               kDrain, kWalkBars };

template <int BV>
__global__ void __launch_bounds__(kWalkThreads, 1)
lin_walk(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
         const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, LinDecay dec, ChunkMap segs,
         const SeqInfo* order, int H, const float* __restrict__ init_state,
         const float* seg_start, __nv_bfloat16* __restrict__ o,
         float* __restrict__ final_state, int* __restrict__ err, unsigned long long stall_ns) {
    extern __shared__ __align__(1024) uint8_t sm[];
    constexpr int NV = kD / BV, HB = BV / 2;   // value tiles a head; state columns a thread
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBars);
    uint32_t* flags = reinterpret_cast<uint32_t*>(bars + kWalkBars);   // tensor-memory base, abort
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0 && blockIdx.x == 0 && seg_start == nullptr) *err = 0;   // first kernel of the call
    if (smem_u32(sm) & 1023u) {
        if (tid == 0) atomicCAS(err, 0, (int)KDA_ERR_DEVICE);
        return;
    }
    const int vt = (int)(blockIdx.x % NV), h = (int)(blockIdx.x / NV % H), seg = (int)(blockIdx.x / NV / H);
    const int j0 = vt * BV;
    int seq, tok0, len, idx;
    if (order != nullptr) {   // whole sequences, the longest first, so that the last blocks are short
        wait_for_kernels_before();   // the table
        const SeqInfo s = load_written(order + seg);
        seq = s.seq;
        tok0 = s.tok0;
        len = s.len;
        idx = 0;
        if (len == 0) {       // no tokens: the state stays
            const size_t at = ((size_t)seq * H + h) * kD * kD;
            for (int i = tid; final_state && vt == 0 && i < kD * kD; i += kWalkThreads)
                final_state[at + i] = init_state ? init_state[at + i] : 0.f;
            return;
        }
    } else {
        segs.locate(seg, seq, tok0, len, idx);
    }
    const int nch = (len + kT - 1) / kT;

    if (tid == 0) {
        for (int i = 0; i < kWalkBars; ++i)   // one arrival a warp
            mbar_init(&bars[i], i == kPReady || i == kPReady + 1 || i == kKReady || i == kSReady || i == kORead ? 8
                                : i == kGEmpty || i == kGEmpty + 1 ? 24
                                : BV == 64 && i < kFull + 2 ? 2 : 1);   // Q and K
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
    const uint32_t tbase = flags[0];
    // scores (and P), and Q S: two by turns where the accumulators leave room for them
    const uint32_t tU = tbase + 256, tPV = BV == 128 ? tbase + 384 : tbase + 320;
    auto tA = [&](int n) { return BV == 128 ? tbase : tbase + 128 * (n & 1); };
    auto tQS = [&](int n) { return BV == 128 ? tbase + 128 : tbase + 384 + 64 * (n & 1); };
    const Abort ab{&flags[1], err};
    // Where a chunk's tiles stand (kind 0 Q, 1 K, 2 V): five slots in turn (Q's is free first and
    // takes the next V); with half the value columns there is room for two of each kind, and a
    // chunk's Q and K share a barrier.
    enum { Q, K, V };
    auto offset = [&](int kind, int n) -> uint32_t {
        if (BV == 128) return (uint32_t)(3 * n + kind) % 5u * kTile;
        return kind == V ? 4 * kTile + (n & 1) * kBlock : (2 * kind + (n & 1)) * kTile;
    };
    auto full = [&](int kind, int n) {
        return &bars[kFull + (BV == 128 ? (int)((uint32_t)(3 * n + kind) % 5u) : 2 * (kind == V) + (n & 1))];
    };
    auto full_par = [&](int kind, int n) { return BV == 128 ? (uint32_t)(3 * n + kind) / 5u & 1u : (uint32_t)(n >> 1) & 1u; };
    auto wait_full = [&](int kind, int n) { return wait_or_abort(full(kind, n), full_par(kind, n), ab); };
    auto wait_pair = [&](int bar, int n) { return wait_or_abort(&bars[bar + (n & 1)], (uint32_t)(n >> 1) & 1u, ab); };
    Gates* gates = reinterpret_cast<Gates*>(sm + kOffGates);
    const int sp = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * sp) << 16;
    constexpr int kRing = BV == 128 ? 5 : 6;   // tiles in flight
    int loads = 0;                             // tiles asked for (the loads' lane)

    // 72 registers a thread at launch, 28 warps: 8 x 104 + 16 x 64 + 4 x 40 of 28 x 72
    if (warp >= 16 && warp < 20) fewer_registers<40>();
    else if (warp >= 8) fewer_registers<64>();
    if (warp < 8) {   // ---- o, and the state
        more_registers<104>();
        const int hb = warp >> 2, row = 32 * sp + lane;
        float s[HB];   // state row `row`, columns j0 + HB hb + [0, HB)
        {
            if (seg_start) wait_for_kernels_before();
            const float* src = seg_start ? seg_start + ((size_t)seg * H + h) * kD * kD
                               : init_state ? init_state + ((size_t)seq * H + h) * kD * kD
                                            : nullptr;
#pragma unroll
            for (int j = 0; j < HB; j += 4) {
                const float4 x = src ? *reinterpret_cast<const float4*>(src + (size_t)row * kD + j0 + HB * hb + j)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
            }
        }
        auto publish = [&]() {   // the state's bf16 copy, an MN-major B operand
            if (BV == 128) {     // o has left its buffer
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < HB; j += 8) {
                const uint4 w = make_uint4(pack_bf16(s[j], s[j + 1]), pack_bf16(s[j + 2], s[j + 3]),
                                           pack_bf16(s[j + 4], s[j + 5]), pack_bf16(s[j + 6], s[j + 7]));
                *reinterpret_cast<uint4*>(sm + kOffS + mn_chunk(row, HB * hb + j, kD)) = w;
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(&bars[kSReady], lane);
        };
        // o = P V + e^g (Q S)
        auto outputs = [&](int n, float eg) {
            if (!wait_pair(kODone, n) || (BV == 128 && !wait_pair(kQsDone, n)))   // BV = 64: P V comes last
                return false;
            tc_fence_after();
            // A lane's row in pieces of 32 bytes, straight to global memory, would cost the
            // load/store pipe 32 cycles a store; so the rows go by way of shared memory: into
            // the state's buffer, whose last reader is Q S (the copy takes one half of it when
            // BV is 64), and out in one box a warp.  Warps with rows past the end store theirs.
            const bool whole = 32 * sp + 32 <= len - n * kT;
            __nv_bfloat16* dst = o + ((size_t)(tok0 + n * kT + row) * H + h) * kD + j0 + HB * hb;
            uint8_t* stage = sm + kOffS + (BV == 128 ? hb * kBlock + 32 * sp * 128 : kBlock + (4 * hb + sp) * 2048);
            if (BV == 64) {      // the last o has left
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            }
#pragma unroll 1
            for (int g = 0; g < HB / 16; ++g) {
                float a[16], b[16];
                tmem_ld16(tPV + lanes + HB * hb + 16 * g, a);
                tmem_ld16(tQS(n) + lanes + HB * hb + 16 * g, b);
                tmem_ld_wait();
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 16; e += 2) w[e / 2] = pack_bf16(fmaf(eg, b[e], a[e]), fmaf(eg, b[e + 1], a[e + 1]));
                if (whole) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int x = BV == 128 ? (2 * g + c) ^ (lane & 7) : (2 * g + c) ^ ((lane >> 1) & 3);
                        *reinterpret_cast<uint4*>(stage + lane * (BV == 128 ? 128 : 64) + x * 16) =
                            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    }
                } else if (row < len - n * kT) {
                    store32(dst + 16 * g, w);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (whole && lane == 0) {
                tma_store_box(&mo, stage, j0 + HB * hb, h, tok0 + n * kT + 32 * sp);
                bulk_commit();
            }
            tc_fence_before();
            warp_arrive(&bars[kORead], lane);
            return true;
        };
        publish();
        bool ok = warp != 0 || !stall(&bars[kDrain], stall_ns, ab);
        for (int n = 0; ok && n < nch; ++n) {
            if (!(ok = wait_pair(kGFull, n))) break;
            const float gam = gates[n & 1].gam, eg = ex2_approx(gates[n & 1].rel2[row]) * gates[n & 1].start[sp];
            warp_arrive(&bars[kGEmpty + (n & 1)], lane);
            if (BV == 128 && !(ok = outputs(n, eg))) break;
            if (!(ok = wait_pair(kUDone, n))) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < HB / 16; ++g) {
                float a[16];
                tmem_ld16(tU + lanes + HB * hb + 16 * g, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) s[16 * g + e] = fmaf(gam, s[16 * g + e], a[e]);
            }
            if (n + 1 < nch) publish();   // Q S of this chunk was issued before its U, which is done
            if (BV == 64 && !(ok = outputs(n, eg))) break;
        }
        if (lane == 0) bulk_wait_read_all();   // before the block's shared memory goes
        if (final_state && ok && last_segment(segs, seq, idx)) {
            float* dst = final_state + (((size_t)seq * H + h) * kD + row) * kD + j0 + HB * hb;
#pragma unroll
            for (int j = 0; j < HB; j += 4)
                *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        }
    } else if (warp < 16) {   // ---- the weighted keys, or values
        const int blk = (warp >> 2) & 1, r = tid & 127;
        for (int n = 0; n < nch; ++n) {
            const int live = min(kT, len - n * kT);
            if (!wait_pair(kGFull, n)) break;
            const float w = gates[n & 1].col[r] * gates[n & 1].end[r >> 5];
            warp_arrive(&bars[kGEmpty + (n & 1)], lane);
            if (n > 0 && !wait_pair(kUDone, n - 1)) break;   // the last U has read the parts
            if (BV == 128) {   // in place: the scores have read the keys
                if (!wait_full(K, n) || !wait_pair(kScores, n)) break;
                uint8_t* tile = sm + offset(K, n) + blk * kBlock;
                scale_split_row<8>(tile, tile, sm + kOffLo + blk * kBlock, r, 0, w, r < live);
            } else {           // half the columns, into a buffer of their own (P V needs the values)
                if (!wait_full(V, n)) break;
                scale_split_row<4>(sm + offset(V, n), sm + kOffLo, sm + kOffLo + kBlock, r, 4 * blk, w, r < live);
                if (live < kT) {   // the keys' rows of the next sequence meet weights of zero
                    if (!wait_full(K, n)) break;
                    zero_rows(sm + offset(K, n), 2, live, tid - 256, 256);
                }
            }
            fence_async_smem();
            warp_arrive(&bars[kKReady], lane);
        }
    } else if (warp >= 20) {   // ---- P
        const int hb = (warp >> 2) & 1, row = 32 * sp + lane;
        for (int n = 0; n < nch; ++n) {
            const int live = min(kT, len - n * kT);
            if (!wait_pair(kGFull, n)) break;
            if (live < kT) {
                if (!wait_full(V, n)) break;
                zero_rows(sm + offset(V, n), BV / 64, live, tid - 640, 256);
                fence_async_smem();
            }
            const Gates& G = gates[n & 1];
            const float r2 = G.rel2[row], er = ex2_approx(r2);
            if (!wait_pair(kScores, n)) break;
            tc_fence_after();
            // this thread's row, 64 keys, 32 at a time; P's words go over scores already read
#pragma unroll 1
            for (int bb = 0; bb < 2; ++bb) {
                const int B = 2 * hb + bb;
                uint32_t w[16];
                if (B > sp) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0u;
                } else {
                    float x[2][16];
                    tmem_ld16(tA(n) + lanes + 32 * B, x[0]);
                    tmem_ld16(tA(n) + lanes + 32 * B + 16, x[1]);
                    tmem_ld_wait();
                    if (B < sp) {
                        const float f = er * G.fac[sp][B];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(&G.col[32 * B + e]);
                            const float* y = &x[e >> 4][e & 15];
                            w[e / 2] = pack_bf16(y[0] * (f * c.x), y[1] * (f * c.y));
                            w[e / 2 + 1] = pack_bf16(y[2] * (f * c.z), y[3] * (f * c.w));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(&G.rel2[32 * B + e]);
                            const float* y = &x[e >> 4][e & 15];
                            const float y0 = e <= lane ? y[0] * ex2_approx(r2 - c.x) : 0.f;
                            const float y1 = e + 1 <= lane ? y[1] * ex2_approx(r2 - c.y) : 0.f;
                            const float y2 = e + 2 <= lane ? y[2] * ex2_approx(r2 - c.z) : 0.f;
                            const float y3 = e + 3 <= lane ? y[3] * ex2_approx(r2 - c.w) : 0.f;
                            w[e / 2] = pack_bf16(y0, y1);
                            w[e / 2 + 1] = pack_bf16(y2, y3);
                        }
                    }
                }
                tmem_st8u(tA(n) + lanes + 64 * hb + 16 * bb, w);
                tmem_st8u(tA(n) + lanes + 64 * hb + 16 * bb + 8, w + 8);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&bars[kPReady + (n & 1)], lane);
            warp_arrive(&bars[kGEmpty + (n & 1)], lane);
        }
    } else if (warp == 16) {   // ---- products
        constexpr uint32_t iS = idesc_bf16_f32(128, 128), iB = idesc_bf16_f32_bmn(128, BV), iU = idesc_amn_bmn(128, BV);
        const uint32_t lead = elect_lane();
        const uint32_t base = smem_u32(sm), lo = base + kOffLo, st = base + kOffS;
        auto commit = [&](int bar) { commit_lead(&bars[bar], lead); };
        // The products' warp is the one that the chunks' time hangs on, and a wait costs it 100 to
        // 200 cycles even when there is nothing to wait for; so it looks at as few barriers as
        // will do (with half the value columns, five a chunk instead of eight).
        auto scores = [&](int n) {   // A = Q K^T
            if ((BV == 128 && !wait_full(Q, n)) || !wait_full(K, n)) return false;
            product<false, false>(tA(n), sw128_desc(base + offset(Q, n)), sw128_desc(base + offset(K, n)), iS, false, lead);
            commit(kScores + (n & 1));
            return true;
        };
        auto o_read = [&](int n) { return n < 0 || wait_or_abort(&bars[kORead], (uint32_t)n & 1u, ab); };
        auto values = [&](int n) {   // P V (BV = 64: the weighted values, which U has waited for, come from V)
            if ((BV == 128 && !wait_full(V, n)) || !wait_pair(kPReady, n) || (BV == 128 && !o_read(n - 1))) return false;
            tc_fence_after();
            product_ta(tPV, tA(n), mn_desc_k(base + offset(V, n), kT, 0), iB, lead);
            commit(kODone + (n & 1));
            return true;
        };
        bool ok = scores(0);
        for (int n = 0; ok && n < nch; ++n) {
            if (BV == 128 && !(ok = values(n))) break;
            // Q S
            if (!(ok = wait_or_abort(&bars[kSReady], (uint32_t)n & 1u, ab))) break;
            tc_fence_after();
            product<false, true>(tQS(n), sw128_desc(base + offset(Q, n)), mn_desc_k(st, kD, 0), iB, false, lead);
            if (BV == 128) commit(kQsDone + (n & 1));
            // K^T V with the weights, high then low parts
            if (!(ok = wait_or_abort(&bars[kKReady], (uint32_t)n & 1u, ab))) break;
            tc_fence_after();
            const uint64_t dk = mn_desc_k(base + offset(K, n), kT, 0), dv = mn_desc_k(base + offset(V, n), kT, 0);
            const uint64_t dl = mn_desc_k(lo, kT, 0);
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
                product<true, true>(tU, BV == 128 && part ? dl : dk,
                                    BV == 128 ? dv : dl + (uint64_t)(part ? kBlock >> 4 : 0), iU, part > 0, lead);
            commit(kUDone + (n & 1));
            if (BV == 128) {
                if (n + 1 < nch && !(ok = wait_pair(kODone, n) && scores(n + 1))) break;
            } else {
                // over the scores of the last chunk but one: o of that one has been read, so its
                // P V is done, and this one's may go over it
                if (!(ok = o_read(n - 1))) break;
                if (n + 1 < nch && !(ok = scores(n + 1))) break;
                if (!(ok = values(n))) break;
            }
        }
    } else if (warp == 17) {
        if (lane == 0) {   // ---- loads
            // A slot is free when the last product that reads its tile is done.
            for (; loads < 3 * nch; ++loads) {
                const int i = loads, n = i / 3, kind = i % 3;   // tile 3 n + kind
                if (i >= kRing) {
                    const int m = (i - kRing) / 3, was = (i - kRing) % 3;   // the tile before in this slot
                    const int bar = BV == 128 ? (was == Q ? kQsDone : kUDone) : was == V ? kODone : kUDone;
                    if (!wait_or_abort_lane(&bars[bar + (m & 1)], (uint32_t)(m >> 1) & 1u, ab)) break;
                }
                const CUtensorMap* map = kind == Q ? &mq : kind == K ? &mk : &mv;
                uint8_t* dst = sm + offset(kind, n);
                uint64_t* bar = full(kind, n);
                const int t = tok0 + n * kT;
                if (kind != V || BV == 128) {
                    mbar_arrive_expect_tx(bar, kTile);
                    tma_box(dst, map, 0, h, t, bar);
                    tma_box(dst + kBlock, map, 64, h, t, bar);
                } else {
                    mbar_arrive_expect_tx(bar, kBlock);
                    tma_box(dst, map, j0, h, t, bar);
                }
            }
        }
    } else if (warp == 18) {   // ---- decays
        float x[4], y[4];
        load_gates(x, dec, tok0, min(kT, len), H, h, lane);
        for (int n = 0; n < nch; ++n) {
            if (n + 1 < nch) load_gates(y, dec, (long long)tok0 + (n + 1) * kT, min(kT, len - (n + 1) * kT), H, h, lane);
            if (n >= 2 && !wait_or_abort(&bars[kGEmpty + (n & 1)], ((uint32_t)(n >> 1) & 1u) ^ 1u, ab)) break;
            make_gates(&gates[n & 1], x, lane);
            warp_arrive(&bars[kGFull + (n & 1)], lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = y[u];
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (gave_up(ab)) {
        if (warp == 16) drain_products(&bars[kDrain]);
        for (int j = max(0, loads - kRing); j < loads; ++j) mbar_wait(full(j % 3, j / 3), full_par(j % 3, j / 3));
        __syncwarp();
    }
    if (warp == 16) tmem_dealloc(tbase, 512);
}

// ---- states ---------------------------------------------------------------------------
// The state chain alone, S <- e^{g_C} S + (w A)^T B over the segment's chunks:
//   forward A = K, B = V, w = e^{g_C - g};  REV (chunks from last to first) A = Q, B = d_o,
//   w = e^{g}, S the gradient of the chunk's end state.
// With seg_end: from zero, the segment's own sum and whole decay (of every segment that
// another one follows in the chain).  With images (backward pass): from start, S ahead of
// each chunk as a bf16 operand image (image_of).  Warps 0-7 keep the state, 8-15 weight the
// rows; low parts and accumulators are double buffered, so both and the products overlap.
// One launch takes both directions (blocks from n_fwd on run in reverse).
struct StateSide {
    const float* start;       // [N, H, dk, dv] or null (zero)
    const float* seg_start;   // [segments, H, dk, dv] or null
    float* seg_end;           // [segments, H, dk, dv] (sums), or null
    float* seg_gam;           // [segments, H]
    uint8_t* images;          // [image, H] x 32 KB, or null
    float* end;               // [N, H, dk, dv] or null: the state behind the last chunk walked
};
constexpr int kStSlots = 4;
constexpr uint32_t kStLo = kStSlots * kTile;
constexpr uint32_t kStStage = kStLo + 2 * kTile;       // the state's image on its way out
constexpr int kStGateBufs = 4;
constexpr uint32_t kStGates = kStStage + kTile;
constexpr uint32_t kStBars = kStGates + kStGateBufs * sizeof(Weights);
constexpr uint32_t kStSmem = kStBars + 256;
static_assert(kStSmem <= 232448, "shared memory per block");
enum StBar { kSFull = 0, kSEmpty = kStSlots, kSWReady = 2 * kStSlots, kSUDone = kSWReady + 2, kSURead = kSUDone + 2,
             kSGFull = kSURead + 2, kSGEmpty = kSGFull + kStGateBufs, kSDrain = kSGEmpty + kStGateBufs, kStBarsN };

__global__ void __launch_bounds__(kStateThreads, 1)
lin_state(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
          const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo, LinDecay dec, ChunkMap segs,
          const SeqInfo* __restrict__ order, int H, int n_fwd, StateSide fwd, StateSide bwd, int clear_err, int* __restrict__ err,
          unsigned long long stall_ns) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kStBars);
    uint32_t* flags = reinterpret_cast<uint32_t*>(bars + kStBarsN);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    let_next_kernel_start();
    if (!clear_err) wait_for_kernels_before();
    else if (tid == 0 && blockIdx.x == 0) *err = 0;   // first kernel of the call
    if (smem_u32(sm) & 1023u) {
        if (tid == 0) atomicCAS(err, 0, (int)KDA_ERR_DEVICE);
        return;
    }
    const bool REV = (int)blockIdx.x >= n_fwd;
    const int unit = (int)blockIdx.x - (REV ? n_fwd : 0);
    const StateSide& A = REV ? bwd : fwd;
    const CUtensorMap *ma = REV ? &mq : &mk, *mb = REV ? &mdo : &mv;
    const int h = unit % H, seg = unit / H;
    int seq, tok0, len, idx;
    if (order != nullptr) {   // whole sequences, the longest first
        const SeqInfo s = order[seg];
        seq = s.seq;
        tok0 = s.tok0;
        len = s.len;
        idx = 0;
        if (len == 0) {       // no tokens: the state stays
            const size_t at = ((size_t)seq * H + h) * kD * kD;
            for (int i = tid; A.end && i < kD * kD; i += kStateThreads) A.end[at + i] = A.start ? A.start[at + i] : 0.f;
            return;
        }
    } else {
        segs.locate(seg, seq, tok0, len, idx);
    }
    const bool last = REV ? idx == 0 : last_segment(segs, seq, idx);
    if (A.seg_end && last) return;   // nothing follows it
    const int nch = (len + kT - 1) / kT;
    if (tid == 0) {
        for (int i = 0; i < kStBarsN; ++i)
            mbar_init(&bars[i], i >= kSWReady && i < kSWReady + 2 ? 8 : i >= kSURead && i < kSURead + 2 ? 8
                                : i >= kSGEmpty && i < kSGEmpty + kStGateBufs ? 16 : 1);
        mbar_init_fence();
        flags[1] = 0u;
    }
    if (warp == 16) {
        tmem_alloc(&flags[0], 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = flags[0];
    const Abort ab{&flags[1], err};
    auto chunk = [&](int n) { return REV ? nch - 1 - n : n; };
    auto slot = [&](int i) { return sm + (uint32_t)(i % kStSlots) * kTile; };   // tile i: A 2 n, B 2 n + 1
    auto full = [&](int i) { return &bars[kSFull + i % kStSlots]; };
    auto full_par = [&](int i) { return (uint32_t)(i / kStSlots) & 1u; };
    auto half_par = [&](int n) { return (uint32_t)(n >> 1) & 1u; };   // of barriers kept for chunks of either parity
    Weights* gates = reinterpret_cast<Weights*>(sm + kStGates);
    auto gates_full = [&](int n) {
        return wait_or_abort(&bars[kSGFull + n % kStGateBufs], (uint32_t)(n / kStGateBufs) & 1u, ab);
    };

    int loads = 0;   // tiles asked for (the loads' lane)
    if (warp >= 16) fewer_registers<40>();
    if (warp < 8) {   // ---- the state
        more_registers<120>();
        const int sp = warp & 3, hb = warp >> 2, row = 32 * sp + lane;
        const uint32_t lanes = (uint32_t)(32 * sp) << 16;
        float s[64];
        {
            const float* src = A.seg_end ? nullptr
                               : A.seg_start ? A.seg_start + ((size_t)seg * H + h) * kD * kD
                               : A.start ? A.start + ((size_t)seq * H + h) * kD * kD
                                         : nullptr;
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 x = src ? *reinterpret_cast<const float4*>(src + (size_t)row * kD + 64 * hb + j)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
            }
        }
        const long long image0 = image_of(tok0 - idx * segs.C, seq) + (long long)idx * (segs.C / kT);
        bool ok = warp != 0 || !stall(&bars[kSDrain], stall_ns, ab);
        for (int n = 0; ok && n < nch; ++n) {
            if (!(ok = gates_full(n))) break;
            const float gam = gates[n % kStGateBufs].gam;
            warp_arrive(&bars[kSGEmpty + n % kStGateBufs], lane);
            if (A.images) {   // this warp's 4 KB of the image: staged swizzled, copied out in one piece
                uint8_t* stage = sm + kStStage + hb * kBlock + 32 * sp * 128;
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (row & 7)) << 4)) =
                        make_uint4(pack_bf16(s[8 * c], s[8 * c + 1]), pack_bf16(s[8 * c + 2], s[8 * c + 3]),
                                   pack_bf16(s[8 * c + 4], s[8 * c + 5]), pack_bf16(s[8 * c + 6], s[8 * c + 7]));
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_s2g(A.images + ((image0 + chunk(n)) * H + h) * kTile + hb * kBlock + 32 * sp * 128, stage, 4096);
                    bulk_commit();
                }
            }
            if (!(ok = wait_or_abort(&bars[kSUDone + (n & 1)], half_par(n), ab))) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float a[16];
                tmem_ld16(tbase + 128 * (n & 1) + lanes + 64 * hb + 16 * g, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) s[16 * g + e] = fmaf(gam, s[16 * g + e], a[e]);
            }
            tc_fence_before();
            warp_arrive(&bars[kSURead + (n & 1)], lane);
        }
        if (lane == 0) bulk_wait_read_all();   // before the block's shared memory goes
        float* to = A.seg_end ? A.seg_end + ((size_t)seg * H + h) * kD * kD
                    : A.end && last ? A.end + ((size_t)seq * H + h) * kD * kD
                                    : nullptr;
        if (ok && to) {
            float* dst = to + (size_t)row * kD + 64 * hb;
#pragma unroll
            for (int j = 0; j < 64; j += 4)
                *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        }
    } else if (warp < 16) {   // ---- weighted rows
        const int r = tid & 127, blk = (tid - 256) >> 7;
        for (int n = 0; n < nch; ++n) {
            const int live = min(kT, len - chunk(n) * kT);
            if (!gates_full(n)) break;
            const float w = gates[n % kStGateBufs].w[r];
            warp_arrive(&bars[kSGEmpty + n % kStGateBufs], lane);
            if (!wait_or_abort(full(2 * n), full_par(2 * n), ab) ||
                (n >= 2 && !wait_or_abort(&bars[kSUDone + (n & 1)], half_par(n) ^ 1u, ab)))   // low parts are free
                break;
            if (live < kT) {
                if (!wait_or_abort(full(2 * n + 1), full_par(2 * n + 1), ab)) break;
                zero_rows(slot(2 * n + 1), 2, live, tid - 256, 256);
            }
            uint8_t *tile = slot(2 * n) + blk * kBlock, *low = sm + kStLo + (n & 1) * kTile + blk * kBlock;
            scale_split_row<8>(tile, tile, low, r, 0, w, r < live);
            fence_async_smem();
            warp_arrive(&bars[kSWReady + (n & 1)], lane);
        }
    } else if (warp == 16) {   // ---- products
        constexpr uint32_t iU = idesc_amn_bmn(128, 128);
        const uint32_t lead = elect_lane(), base = smem_u32(sm);
        auto commit = [&](int bar) {
            if (lead) mma_commit(&bars[bar]);
        };
        for (int n = 0; n < nch; ++n) {
            if (!wait_or_abort(full(2 * n + 1), full_par(2 * n + 1), ab) ||
                !wait_or_abort(&bars[kSWReady + (n & 1)], half_par(n), ab) ||
                (n >= 2 && !wait_or_abort(&bars[kSURead + (n & 1)], half_par(n) ^ 1u, ab)))
                break;
            tc_fence_after();
            const uint64_t b = mn_desc_k(base + (2 * n + 1) % kStSlots * kTile, kT, 0);
            const uint32_t d = tbase + 128 * (n & 1);
            product<true, true>(d, mn_desc_k(base + (2 * n) % kStSlots * kTile, kT, 0), b, iU, false, lead);
            product<true, true>(d, mn_desc_k(base + kStLo + (n & 1) * kTile, kT, 0), b, iU, true, lead);
            commit(kSUDone + (n & 1));
            commit(kSEmpty + (2 * n) % kStSlots);
            commit(kSEmpty + (2 * n + 1) % kStSlots);
        }
    } else if (warp == 17) {
        if (lane == 0) {   // ---- loads
            for (; loads < 2 * nch; ++loads) {
                const int i = loads;
                if (i >= kStSlots && !wait_or_abort_lane(&bars[kSEmpty + i % kStSlots], full_par(i) ^ 1u, ab)) break;
                const int t = tok0 + chunk(i / 2) * kT;
                mbar_arrive_expect_tx(full(i), kTile);
                tma_box(slot(i), i & 1 ? mb : ma, 0, h, t, full(i));
                tma_box(slot(i) + kBlock, i & 1 ? mb : ma, 64, h, t, full(i));
            }
        }
    } else if (warp == 18) {   // ---- decays
        float x[4], y[4];
        long long whole = 0;   // log decay of the segment
        load_gates(x, dec, (long long)tok0 + chunk(0) * kT, min(kT, len - chunk(0) * kT), H, h, lane);
        for (int n = 0; n < nch; ++n) {
            if (n + 1 < nch)
                load_gates(y, dec, (long long)tok0 + chunk(n + 1) * kT, min(kT, len - chunk(n + 1) * kT), H, h, lane);
            if (n >= kStGateBufs &&
                !wait_or_abort(&bars[kSGEmpty + n % kStGateBufs], ((uint32_t)(n / kStGateBufs) & 1u) ^ 1u, ab))
                break;
            whole += make_weights(&gates[n % kStGateBufs], x, REV, lane);
            warp_arrive(&bars[kSGFull + n % kStGateBufs], lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = y[u];
        }
        if (lane == 0 && A.seg_end) A.seg_gam[(size_t)seg * H + h] = ex2_approx(from_fixed(whole));
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (gave_up(ab)) {
        if (warp == 16) drain_products(&bars[kSDrain]);
        for (int j = max(0, loads - kStSlots); j < loads; ++j) mbar_wait(full(j), full_par(j));
        __syncwarp();
    }
    if (warp == 16) tmem_dealloc(tbase, 256);
}

// start state of every segment from the segments' own sums, in place (as the chunk chain
// of the CUDA-core path, with segments for chunks)
template <bool REV>
__global__ void __launch_bounds__(256) seg_chain(float* X, const float* gam,
                                                 const float* __restrict__ start, SeqMap smap, int H) {
    let_next_kernel_start();
    wait_for_kernels_before();
    const SeqInfo sq = smap.get((int)blockIdx.x / H);
    const int h = (int)blockIdx.x % H, e = (int)blockIdx.y * 256 + threadIdx.x;
    const int n = (sq.len + smap.C - 1) / smap.C;
    constexpr int E4 = kD * kD / 4;
    float4* x4 = reinterpret_cast<float4*>(X);
    float4 s = start ? reinterpret_cast<const float4*>(start)[((size_t)sq.seq * H + h) * E4 + e]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;   // loads of that many segments stand before the first is used
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        float4 u[kAhead];
        float g[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            u[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            g[j] = 0.f;
            if (i + 1 < n) {   // nothing follows the last segment: its own sum was not formed
                const size_t unit = (size_t)(sq.chunk0 + (REV ? n - 1 - i : i)) * H + h;
                u[j] = __ldcg(x4 + unit * E4 + e);
                g[j] = __ldcg(gam + unit);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            if (i < n) {
                x4[((size_t)(sq.chunk0 + (REV ? n - 1 - i : i)) * H + h) * E4 + e] = s;
                s.x = fmaf(g[j], s.x, u[j].x);
                s.y = fmaf(g[j], s.y, u[j].y);
                s.z = fmaf(g[j], s.z, u[j].z);
                s.w = fmaf(g[j], s.w, u[j].w);
            }
        }
    }
}

// states of sequences without tokens: the last `n_empty` of the longest-first order, or all
__global__ void __launch_bounds__(256) empty_states(const float* __restrict__ start, float* __restrict__ end,
                                                    SeqMap smap, int first, int H) {
    const SeqInfo sq = smap.get(first + (int)blockIdx.x / H);
    const size_t at = ((size_t)sq.seq * H + blockIdx.x % H) * (kD * kD / 4) + blockIdx.y * 256 + threadIdx.x;
    reinterpret_cast<float4*>(end)[at] = start ? reinterpret_cast<const float4*>(start)[at]
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename K>
cudaError_t allow_smem(K kern, uint32_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace
}  // namespace lintc

using namespace lintc;

cudaError_t launch_lin_empty_states(const float* start, float* end, const SeqMap& smap, int first, int n, int H,
                                    cudaStream_t s) {
    if (n <= 0 || end == nullptr || end == start) return cudaSuccess;
    empty_states<<<dim3((unsigned)n * H, kD * kD / 1024), 256, 0, s>>>(start, end, smap, first, H);
    return cudaGetLastError();
}

cudaError_t launch_lin_tc_fwd(const void* q, const void* k, const void* v, LinDecay dec, const float* init_state,
                              void* o, float* final_state, const ChunkMap& segs, const SeqMap& smap, int n_segs,
                              int n_seqs, bool split, int BV, long long tokens, int H, float* seg_state,
                              float* seg_gam, int* err, TestStall stall, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mo;
    if (!make_map(&mq, q, tokens, H) || !make_map(&mk, k, tokens, H) || !make_map(&mv, v, tokens, H) ||
        !make_map(&mo, o, tokens, H, BV / 2, 32))
        return cudaErrorNotSupported;
    cudaError_t e;
    if (split) {
        if ((e = allow_smem(lin_state, kStSmem)) != cudaSuccess) return e;
        const StateSide side{nullptr, nullptr, seg_state, seg_gam, nullptr, nullptr};
        lin_state<<<(unsigned)n_segs * H, kStateThreads, kStSmem, s>>>(mk, mv, mk, mv, dec, segs, nullptr, H, n_segs * H, side,
                                                                     side, 1, err, stall.state);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        e = launch_behind(seg_chain<false>, dim3((unsigned)n_seqs * H, kD * kD / 1024), 256, 0, s, seg_state, seg_gam,
                          init_state, smap, H);
        if (e != cudaSuccess) return e;
    }
    auto kern = BV == 128 ? lin_walk<128> : lin_walk<64>;
    if ((e = allow_smem(kern, kWalkSmem)) != cudaSuccess) return e;
    if (split)
        return launch_behind(kern, (unsigned)n_segs * H * (kD / BV), kWalkThreads, kWalkSmem, s, mq, mk, mv, mo, dec, segs,
                             nullptr, H, init_state, seg_state, (__nv_bfloat16*)o, final_state, err, stall.walk);
    if (smap.order)   // whole packed sequences go by the longest-first table, empty ones among them
        return launch_behind(kern, (unsigned)n_seqs * H * (kD / BV), kWalkThreads, kWalkSmem, s, mq, mk, mv, mo, dec, segs,
                             smap.order, H, init_state, nullptr, (__nv_bfloat16*)o, final_state, err, stall.walk);
    kern<<<(unsigned)n_segs * H * (kD / BV), kWalkThreads, kWalkSmem, s>>>(mq, mk, mv, mo, dec, segs, nullptr, H, init_state,
                                                                          nullptr, (__nv_bfloat16*)o, final_state, err,
                                                                          stall.walk);
    return cudaGetLastError();
}

// Backward, first part: the bf16 images of every chunk's start state and of the gradient of
// its end state, and the initial state's gradient.
cudaError_t launch_lin_tc_states(const void* q, const void* k, const void* v, const void* d_o, LinDecay dec,
                                 const float* init_state, const float* d_final, float* d_init, const ChunkMap& segs,
                                 const SeqMap& smap, int n_segs, int n_seqs, bool split, long long tokens, int H,
                                 float* seg_state, float* seg_gam, uint8_t* images, uint8_t* d_images, int* err,
                                 TestStall stall, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mdo;
    if (!make_map(&mq, q, tokens, H) || !make_map(&mk, k, tokens, H) || !make_map(&mv, v, tokens, H) ||
        !make_map(&mdo, d_o, tokens, H))
        return cudaErrorNotSupported;
    cudaError_t e;
    if ((e = allow_smem(lin_state, kStSmem)) != cudaSuccess) return e;
    const int units = n_segs * H;
    float *d_seg = seg_state + (size_t)units * kD * kD, *d_gam = seg_gam + units;
    if (split) {
        const StateSide f{nullptr, nullptr, seg_state, seg_gam, nullptr, nullptr};
        const StateSide r{nullptr, nullptr, d_seg, d_gam, nullptr, nullptr};
        lin_state<<<2u * units, kStateThreads, kStSmem, s>>>(mk, mv, mq, mdo, dec, segs, nullptr, H, units, f, r, 1, err,
                                                           stall.state);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const dim3 grid((unsigned)n_seqs * H, kD * kD / 1024);
        if ((e = launch_behind(seg_chain<false>, grid, 256, 0, s, seg_state, seg_gam, init_state, smap, H)) != cudaSuccess ||
            (e = launch_behind(seg_chain<true>, grid, 256, 0, s, d_seg, d_gam, d_final, smap, H)) != cudaSuccess)
            return e;
    }
    const StateSide f{init_state, split ? seg_state : nullptr, nullptr, nullptr, images, nullptr};
    const StateSide r{d_final, split ? d_seg : nullptr, nullptr, nullptr, d_images, d_init};
    if (split)
        return launch_behind(lin_state, 2u * units, kStateThreads, kStSmem, s, mk, mv, mq, mdo, dec, segs, nullptr, H, units,
                             f, r, 0, err, stall.state);
    const int n = smap.order ? n_seqs * H : units;
    lin_state<<<2u * n, kStateThreads, kStSmem, s>>>(mk, mv, mq, mdo, dec, segs, smap.order, H, n, f, r, 1, err,
                                                   stall.state);
    return cudaGetLastError();
}

}  // namespace kda
