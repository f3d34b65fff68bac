// Host side of linear attention with one decay a head (kda_linear_* in include/kda.h):
// argument checks, workspace layout and dispatch.  Nothing here allocates device memory.
#include <algorithm>
#include <initializer_list>

#include "kda_host.cuh"
#include "kda_launch.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace {

struct LinLayout {
    size_t S, dS, gam, parts, total;   // byte offsets in the workspace (SIMT path)
};

LinLayout simt_layout(const Plan& p, int H, int dk, int dv, bool bwd) {
    LinLayout L;
    const size_t ch = (size_t)p.n_chunks * H;
    size_t o = table_bytes(p);
    L.S = o; o = align_up(o + ch * dk * dv * sizeof(float));
    L.dS = o; if (bwd) o = align_up(o + ch * dk * dv * sizeof(float));
    L.gam = o; o = align_up(o + ch * sizeof(float));
    L.parts = o; if (bwd) o = align_up(o + ch * (3 * kLinSimtChunk + 1) * sizeof(float));
    L.total = std::max(o, kAlign);
    return L;
}

bool use_tc(kda_dtype dtype, int dk, int dv) { return dtype == KDA_BF16 && dk == 128 && dv == 128; }

// How the tensor-core walk is cut: segments of seg_chunks chunks, value columns a block.
struct Cut {
    int seg_chunks = 1;
    int BV = 128;
    bool split = false;
};

constexpr int kSms = 148;

// Microseconds a chunk of 128 tokens takes a block (one block an SM): all 128 value columns,
// half of them, and the state alone; a block's start and end; and what a split adds (the
// segments' chain, two more launches).  From 1 to 10 segments a sequence, 8 to 512 chunks
// and 16 to 704 blocks, times estimated with these are within 15 % of the measured ones
// (batches of unequal sequences take up to 30 % longer).  What the choice gains, in calls back to
// back: 64 pairs of 32 chunks in 73 us with half the columns a block, 98 with all, 107 in
// segments; 16 pairs of 128 chunks 103 us in segments, 255 and 367 without; 32 of 512: 607 to 619,
// 1003 and 1465.
constexpr double kWalk128 = 3.2, kWalk64 = 2.1, kStateOnly = 1.95, kRamp = 4.0, kSplitCost = 20.0;

long long longest_of(const Plan& chunks) {   // chunks of the longest sequence
    long long longest = 0;
    if (chunks.varlen)
        for (const SeqInfo& q : chunks.natural) longest = std::max<long long>(longest, (q.len + kLinTcChunk - 1) / kLinTcChunk);
    else
        longest = chunks.n_seqs ? chunks.n_chunks / chunks.n_seqs : 0;
    return longest;
}

long long segments_of(const Plan& chunks, long long longest, long long len) {   // of len chunks each
    if (!chunks.varlen) return (longest + len - 1) / len * chunks.n_seqs;
    long long segs = 0;
    for (const SeqInfo& q : chunks.natural) segs += ((q.len + kLinTcChunk - 1) / kLinTcChunk + len - 1) / len;
    return segs;
}

// Chunks a segment for `blocks` blocks of work (`per` of them a segment), so that as few as
// possible run behind the others: one segment more than fit would start another wave.
long long segment_len(const Plan& chunks, long long longest, long long per, long long blocks) {
    const long long even = (chunks.n_chunks * per + blocks - 1) / blocks;
    if (!chunks.varlen) {
        const long long segs = blocks / (per * chunks.n_seqs);   // a sequence
        return std::max<long long>(4, segs > 0 ? (longest + segs - 1) / segs : longest);
    }
    long long len = std::max<long long>(4, even);
    for (int i = 0; i < 16 && len < longest && segments_of(chunks, longest, len) * per > blocks; ++i)
        len += std::max<long long>(1, len / 16);
    return len;
}

// Time of `units` blocks, the longest of `len` chunks: whole waves where all are alike,
// otherwise (packed sequences, the longest first) what the machine's work adds up to.
double walk_time(const Plan& chunks, long long units, long long len, double work, bool alike, double t) {
    const double waves = (double)((units + kSms - 1) / kSms);
    return alike || !chunks.varlen ? waves * (len * t + kRamp)
                                   : std::max(len * t + kRamp, (work * t + units * kRamp) / kSms);
}

// The cut with the least estimated time.  A sequence's chunks follow one another, so with
// few (sequence, head) pairs most SMs would idle: two blocks of 64 value columns a pair
// repeat the scores and the weighted keys, and segments read k and v twice.
Cut choose_cut(const Plan& chunks, int H) {
    const long long longest = longest_of(chunks), total = chunks.n_chunks;
    Cut best;
    if (longest == 0) return best;
    best.seg_chunks = (int)longest;
    const long long pairs = (long long)chunks.n_seqs * H;
    double t = walk_time(chunks, pairs, longest, (double)total * H, false, kWalk128);
    const double t64 = walk_time(chunks, 2 * pairs, longest, 2.0 * total * H, false, kWalk64);
    if (t64 < t) {
        t = t64;
        best.BV = 64;
    }
    for (int m = 1; m <= 6; ++m) {
        const long long len = segment_len(chunks, longest, H, (long long)kSms * m);
        if (len >= longest) continue;
        const long long segs = segments_of(chunks, longest, len);
        const double ts = walk_time(chunks, segs * H, len, 0, true, kWalk128) +
                          walk_time(chunks, (segs - chunks.n_seqs) * H, len, 0, true, kStateOnly) + kSplitCost;
        if (ts < t) {
            t = ts;
            best = Cut{(int)len, 128, true};
        }
    }
    return best;
}

// The same for the backward pass's state chains (both directions side by side, all value
// columns): what a split saves in idle SMs against walking the chunks twice.
Cut choose_state_cut(const Plan& chunks, int H) {
    const long long longest = longest_of(chunks), total = chunks.n_chunks;
    Cut best;
    if (longest == 0) return best;
    best.seg_chunks = (int)longest;
    double t = walk_time(chunks, 2LL * chunks.n_seqs * H, longest, 2.0 * total * H, false, kStateOnly);
    for (int m = 1; m <= 6; ++m) {
        const long long len = segment_len(chunks, longest, 2LL * H, (long long)kSms * m);
        if (len >= longest) continue;
        const long long segs = segments_of(chunks, longest, len);
        const double ts = walk_time(chunks, 2 * segs * H, len, 0, true, kStateOnly) +
                          walk_time(chunks, 2 * (segs - chunks.n_seqs) * H, len, 0, true, kStateOnly) + kSplitCost;
        if (ts < t) {
            t = ts;
            best = Cut{(int)len, 128, true};
        }
    }
    return best;
}

struct TcLayout {
    Cut cut;
    Plan segs;          // segments as chunks
    size_t seg_tables, err, state, gam, images, d_images, total;
};

kda_status tc_layout(const Plan& chunks, const int32_t* cu, int n_seqs, int B, int T, int H, bool bwd, TcLayout& L) {
    L.cut = bwd ? choose_state_cut(chunks, H) : choose_cut(chunks, H);
    const kda_status st = plan_sequences(B, T, L.cut.seg_chunks * kLinTcChunk, cu, n_seqs, L.segs);
    if (st != KDA_OK) return st;
    if ((long long)L.segs.n_chunks * H * 2 > 0x7fffffffLL || (long long)chunks.n_chunks * H > 0x7fffffffLL)
        return KDA_ERR_SHAPE;
    const size_t n = L.cut.split ? (size_t)L.segs.n_chunks * H * (bwd ? 2 : 1) : 0;
    // a number a chunk image, one more a sequence (see image_of)
    const size_t images = bwd ? (size_t)(chunks.total_tokens / kLinTcChunk + chunks.n_seqs + 1) * H * 32768 : 0;
    size_t o = bwd ? table_bytes(chunks) : 0;
    L.seg_tables = o; o += table_bytes(L.segs);
    L.err = o; o += kAlign;
    L.state = o; o = align_up(o + n * 128 * 128 * sizeof(float));
    L.gam = o; o = align_up(o + n * sizeof(float));
    L.images = o; o += images;
    L.d_images = o; o += images;
    L.total = o;
    return KDA_OK;
}

// Sequences without tokens (the last of the longest-first order) that no walk visits: all of
// them, unless the walk goes by that order.
int empty_of(const Plan& p, bool split) {
    if (p.total_tokens == 0) return p.n_seqs;
    if (!split) return 0;
    int n = 0;
    for (const SeqInfo& q : p.natural) n += q.len == 0;
    return n;
}

kda_status check_decay(kda_decay decay) {
    return decay == KDA_DECAY_TOKEN || decay == KDA_DECAY_HEAD ? KDA_OK : KDA_ERR_SHAPE;
}

// The checks that the chunk calls share; fills the plan.  Grids put heads on y and
// sequence-heads on x, two blocks each (both directions of a backward pass, two column halves).
kda_status plan_for(kda_decay decay, kda_dtype dtype, const int32_t* cu, int n_seqs, int B, int T, int H, int dk,
                    int dv, int C, Plan& p) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    kda_status st = check_decay(decay);
    if (st != KDA_OK) return st;
    if (T > 0x7fffffff - C) return KDA_ERR_SHAPE;   // chunk ends are ints
    st = make_plan(B, T, H, dk, dv, C, cu, n_seqs, p);
    if (st != KDA_OK) return st;
    if (H > 65535 || 2LL * p.n_seqs * H > 0x7fffffffLL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

// The tables of a few sequences in one launch (2 KB of parameters): the sequence table and,
// from the parameters too, the chunk table, which otherwise waits for the first.
constexpr int kFewSeqs = 64;
struct FewSeqs {
    SeqInfo e[2 * kFewSeqs];   // natural order, then longest first
};
__global__ void __launch_bounds__(256) few_tables_write(SeqInfo* __restrict__ seqs, int n_seqs, int n_chunks, int C,
                                                        int4* __restrict__ chunks, const __grid_constant__ FewSeqs b) {
    let_next_kernel_start();
    const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    if (c < 2 * n_seqs) seqs[c] = b.e[c];
    if (c >= n_chunks) return;
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {   // last sequence whose first chunk is <= c
        const int mid = (lo + hi + 1) >> 1;
        if (b.e[mid].chunk0 <= c) lo = mid; else hi = mid - 1;
    }
    const SeqInfo sq = b.e[lo];
    const int idx = c - sq.chunk0;
    chunks[c] = make_int4(sq.tok0 + idx * C, min(C, sq.len - idx * C), sq.seq, idx);
}

cudaError_t write_tables(const Plan& p, int n_chunks, int C, SeqInfo* ws, cudaStream_t s) {
    cudaError_t err;
    if (p.n_seqs > kFewSeqs) {
        upload_tables(ws, p.natural, p.by_len, n_chunks, C, s, &err);
        return err;
    }
    FewSeqs b;
    std::copy(p.natural.begin(), p.natural.end(), b.e);
    std::copy(p.by_len.begin(), p.by_len.end(), b.e + p.n_seqs);
    few_tables_write<<<std::max(1, (n_chunks + 255) / 256), 256, 0, s>>>(ws, p.n_seqs, n_chunks, C,
                                                                        chunk_table(ws, p.n_seqs), b);
    return cudaGetLastError();
}

kda_status make_maps(const Plan& p, int T, int C, char* ws, cudaStream_t s, ChunkMap& cmap, SeqMap& smap,
                     bool chunk_entries = true) {
    const int ncps = (int)(((long long)T + C - 1) / C);
    cmap = ChunkMap{nullptr, p.n_seqs, T, C, ncps};
    smap = SeqMap{nullptr, T, C, ncps};
    if (p.varlen) {
        if (write_tables(p, chunk_entries ? p.n_chunks : 0, C, (SeqInfo*)ws, s) != cudaSuccess) return KDA_ERR_CUDA;
        cmap.seqs = (const SeqInfo*)ws;
        if (chunk_entries) cmap.chunks = chunk_table((SeqInfo*)ws, p.n_seqs);
        smap.order = (const SeqInfo*)ws + p.n_seqs;
    }
    return KDA_OK;
}

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return false;
    return true;
}

// log_alpha and its gradient are read and written one element at a time; slices of a table of
// decays seldom start on 16 bytes.
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Contiguous arrays of one call.  Results in an input's memory are refused, since blocks read
// inputs that others have written results over by then; but the last result, a state, may be the
// last input itself.
struct Span {
    const void* p;
    size_t bytes;
};
kda_status check_apart(std::initializer_list<Span> results, std::initializer_list<Span> inputs) {
    for (const Span& r : results)
        for (const Span& x : inputs) {
            if (!r.p || !x.p || !r.bytes || !x.bytes || (&r == results.end() - 1 && &x == inputs.end() - 1 && r.p == x.p)) continue;
            if ((uintptr_t)r.p < (uintptr_t)x.p + x.bytes && (uintptr_t)x.p < (uintptr_t)r.p + r.bytes)
                return KDA_ERR_SHAPE;
        }
    return KDA_OK;
}

// Bytes of the arrays of n token-heads and their sequences' states.
struct Sizes {
    size_t k, v, la, state;
    Sizes(kda_dtype dtype, kda_decay decay, size_t n, size_t seqs, int H, int dk, int dv) {
        const size_t e = dtype == KDA_F32 ? 4 : 2;
        k = n * dk * e;
        v = n * dv * e;
        la = decay == KDA_DECAY_HEAD ? (size_t)H * 4 : n * e;
        state = seqs * H * dk * dv * sizeof(float);
    }
};

TestStall take_stall() {
    TestStall t;
    t.walk = take_test_wait(KDA_TEST_WAIT_LINEAR_WALK);
    t.state = take_test_wait(KDA_TEST_WAIT_LINEAR_STATE);
    t.grad = take_test_wait(KDA_TEST_WAIT_LINEAR_GRAD);
    return t;
}

// A C entry point lets no C++ exception out (the sequence tables are std::vectors).
template <typename F>
kda_status guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return KDA_ERR_CUDA;
    }
}

kda_status chunk_status(bool bwd, const void* workspace, kda_dtype dtype, const int32_t* cu, int n_seqs, int B, int T,
                        int H, int dk, int dv, void* stream) {
    return guarded([&]() -> kda_status {
        Plan p;
        const bool tc = use_tc(dtype, dk, dv);
        kda_status st = plan_for(KDA_DECAY_TOKEN, dtype, cu, n_seqs, B, T, H, dk, dv, tc ? kLinTcChunk : kLinSimtChunk, p);
        if (st != KDA_OK) return st;
        if (!workspace) return KDA_ERR_NULL;
        if (!tc || p.total_tokens == 0) return KDA_OK;   // nothing waited
        TcLayout L;
        if ((st = tc_layout(p, cu, n_seqs, B, T, H, bwd, L)) != KDA_OK) return st;
        return read_error_word(workspace, L.err, stream);
    });
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_linear_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype dtype,
                                           const int32_t* cu_seqlens_host, int n_seqs) {
    size_t n = 0;
    guarded([&] {
        Plan p;
        const bool tc = use_tc(dtype, dk, dv);
        kda_status st = plan_for(KDA_DECAY_TOKEN, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv,
                                 tc ? kLinTcChunk : kLinSimtChunk, p);
        if (st != KDA_OK) return st;
        if (!tc) {
            n = simt_layout(p, H, dk, dv, false).total;
            return st;
        }
        TcLayout L;
        if ((st = tc_layout(p, cu_seqlens_host, n_seqs, B, T, H, false, L)) == KDA_OK) n = L.total;
        return st;
    });
    return n;
}

kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                kda_dtype dtype, const float* init_state, const int32_t* cu_seqlens_host, int n_seqs,
                                int B, int T, int H, int dk, int dv, void* o, float* final_state, void* workspace,
                                size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        Plan p;
        const bool tc = use_tc(dtype, dk, dv);
        kda_status st = plan_for(decay, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv,
                                 tc ? kLinTcChunk : kLinSimtChunk, p);
        if (st != KDA_OK) return st;
        if (p.total_tokens > 0 && (!q || !k || !v || !log_alpha || !o)) return KDA_ERR_NULL;
        if (!workspace) return KDA_ERR_WORKSPACE;
        if (!all_aligned({q, k, v, (const void*)init_state, (const void*)o, (const void*)final_state}) ||
            !aligned4(log_alpha) || ((uintptr_t)workspace & (kAlign - 1)) != 0)
            return KDA_ERR_ALIGN;
        const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
        const Sizes z(dtype, decay, (size_t)p.total_tokens * H, p.n_seqs, H, dk, dv);
        const auto apart = [&] {
            return check_apart({{o, z.v}, {final_state, z.state}},
                               {{q, z.k}, {k, z.k}, {v, z.v}, {log_alpha, z.la}, {init_state, z.state}});
        };
        if (tc) {
            TcLayout L;
            if ((st = tc_layout(p, cu_seqlens_host, n_seqs, B, T, H, false, L)) != KDA_OK) return st;
            if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
            if ((st = apart()) != KDA_OK) return st;
            if ((st = check_device()) != KDA_OK) return st;
            if (p.n_seqs == 0) return KDA_OK;
            cudaStream_t s = (cudaStream_t)stream;
            char* ws = (char*)workspace;
            ChunkMap segs;
            SeqMap smap;
            if ((st = make_maps(L.segs, T, L.cut.seg_chunks * kLinTcChunk, ws, s, segs, smap, L.cut.split)) != KDA_OK)
                return st;
            const int empty = empty_of(p, L.cut.split);
            const TestStall stall = take_stall();
            cudaError_t e = launch_lin_empty_states(init_state, final_state, smap, p.n_seqs - empty, empty, H, s);
            if (e == cudaSuccess && p.total_tokens > 0)
                e = launch_lin_tc_fwd(q, k, v, dec, init_state, o, final_state, segs, smap, L.segs.n_chunks, p.n_seqs,
                                      L.cut.split, L.cut.BV, p.total_tokens, H, (float*)(ws + L.state),
                                      (float*)(ws + L.gam), (int*)(ws + L.err), stall, s);
            return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
        }
        const LinLayout L = simt_layout(p, H, dk, dv, false);
        if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
        if ((st = apart()) != KDA_OK) return st;
        if ((st = check_device()) != KDA_OK) return st;
        if (p.n_seqs == 0) return KDA_OK;
        cudaStream_t s = (cudaStream_t)stream;
        char* ws = (char*)workspace;
        ChunkMap cmap;
        SeqMap smap;
        if ((st = make_maps(p, T, kLinSimtChunk, ws, s, cmap, smap)) != KDA_OK) return st;
        const LinSimtWorkspace w{(float*)(ws + L.S), nullptr, (float*)(ws + L.gam), nullptr};
        return launch_lin_simt_fwd(dtype, q, k, v, dec, init_state, o, final_state, cmap, smap, p.n_chunks, p.n_seqs,
                                   H, dk, dv, w, s) == cudaSuccess
                   ? KDA_OK
                   : KDA_ERR_CUDA;
    });
}

kda_status kda_linear_chunk_fwd_device_status(const void* workspace, kda_dtype dtype, const int32_t* cu_seqlens_host,
                                              int n_seqs, int B, int T, int H, int dk, int dv, void* stream) {
    return chunk_status(false, workspace, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, stream);
}

size_t kda_linear_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype dtype,
                                           const int32_t* cu_seqlens_host, int n_seqs) {
    size_t n = 0;
    guarded([&] {
        Plan p;
        const bool tc = use_tc(dtype, dk, dv);
        kda_status st = plan_for(KDA_DECAY_TOKEN, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv,
                                 tc ? kLinTcChunk : kLinSimtChunk, p);
        if (st != KDA_OK) return st;
        if (!tc) {
            n = simt_layout(p, H, dk, dv, true).total;
            return st;
        }
        TcLayout L;
        if ((st = tc_layout(p, cu_seqlens_host, n_seqs, B, T, H, true, L)) == KDA_OK) n = L.total;
        return st;
    });
    return n;
}

kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                kda_dtype dtype, const float* init_state, const int32_t* cu_seqlens_host, int n_seqs,
                                int B, int T, int H, int dk, int dv, const void* d_o, const float* d_final_state,
                                void* dq, void* dk_out, void* dv_out, void* dlog_alpha, float* d_init_state,
                                void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        Plan p;
        const bool tc = use_tc(dtype, dk, dv);
        kda_status st = plan_for(decay, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv,
                                 tc ? kLinTcChunk : kLinSimtChunk, p);
        if (st != KDA_OK) return st;
        if (p.total_tokens > 0 && (!q || !k || !v || !log_alpha || !d_o || !dq || !dk_out || !dv_out ||
                                   (decay == KDA_DECAY_TOKEN && !dlog_alpha)))
            return KDA_ERR_NULL;
        if (!workspace) return KDA_ERR_WORKSPACE;
        if (!all_aligned({q, k, v, (const void*)init_state, d_o, (const void*)d_final_state, (const void*)dq,
                          (const void*)dk_out, (const void*)dv_out, (const void*)d_init_state}) ||
            !aligned4(log_alpha) || !aligned4(dlog_alpha) || ((uintptr_t)workspace & (kAlign - 1)) != 0)
            return KDA_ERR_ALIGN;
        const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
        const Sizes z(dtype, decay, (size_t)p.total_tokens * H, p.n_seqs, H, dk, dv);
        const auto apart = [&] {
            return check_apart({{dq, z.k}, {dk_out, z.k}, {dv_out, z.v},
                                {decay == KDA_DECAY_HEAD ? nullptr : dlog_alpha, z.la}, {d_init_state, z.state}},
                               {{q, z.k}, {k, z.k}, {v, z.v}, {log_alpha, z.la}, {d_o, z.v}, {init_state, z.state},
                                {d_final_state, z.state}});
        };
        if (tc) {
            TcLayout L;
            if ((st = tc_layout(p, cu_seqlens_host, n_seqs, B, T, H, true, L)) != KDA_OK) return st;
            if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
            if ((st = apart()) != KDA_OK) return st;
            if ((st = check_device()) != KDA_OK) return st;
            if (p.n_seqs == 0) return KDA_OK;
            cudaStream_t s = (cudaStream_t)stream;
            char* ws = (char*)workspace;
            ChunkMap segs, chunks;
            SeqMap smap, cmap;
            if ((st = make_maps(L.segs, T, L.cut.seg_chunks * kLinTcChunk, ws + L.seg_tables, s, segs, smap,
                                L.cut.split)) != KDA_OK ||
                (st = make_maps(p, T, kLinTcChunk, ws, s, chunks, cmap)) != KDA_OK)
                return st;
            const int empty = empty_of(p, L.cut.split);
            const TestStall stall = take_stall();
            cudaError_t e = launch_lin_empty_states(d_final_state, d_init_state, smap, p.n_seqs - empty, empty, H, s);
            uint8_t *im = (uint8_t*)(ws + L.images), *dim = (uint8_t*)(ws + L.d_images);
            int* err = (int*)(ws + L.err);
            if (e == cudaSuccess && p.total_tokens > 0)
                e = launch_lin_tc_states(q, k, v, d_o, dec, init_state, d_final_state, d_init_state, segs, smap,
                                         L.segs.n_chunks, p.n_seqs, L.cut.split, p.total_tokens, H,
                                         (float*)(ws + L.state), (float*)(ws + L.gam), im, dim, err, stall, s);
            if (e == cudaSuccess && p.total_tokens > 0)
                e = launch_lin_tc_grad(q, k, v, d_o, dec, dq, dk_out, dv_out, dlog_alpha, chunks, p.n_chunks,
                                       p.total_tokens, H, im, dim, err, stall, s);
            return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
        }
        const LinLayout L = simt_layout(p, H, dk, dv, true);
        if (workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
        if ((st = apart()) != KDA_OK) return st;
        if ((st = check_device()) != KDA_OK) return st;
        if (p.n_seqs == 0) return KDA_OK;
        cudaStream_t s = (cudaStream_t)stream;
        char* ws = (char*)workspace;
        ChunkMap cmap;
        SeqMap smap;
        if ((st = make_maps(p, T, kLinSimtChunk, ws, s, cmap, smap)) != KDA_OK) return st;
        const LinSimtWorkspace w{(float*)(ws + L.S), (float*)(ws + L.dS), (float*)(ws + L.gam),
                                 (float*)(ws + L.parts)};
        return launch_lin_simt_bwd(dtype, q, k, v, dec, init_state, d_o, d_final_state, dq, dk_out, dv_out,
                                   dlog_alpha, d_init_state, cmap, smap, p.n_chunks, p.n_seqs, H, dk, dv, w, s) ==
                       cudaSuccess
                   ? KDA_OK
                   : KDA_ERR_CUDA;
    });
}

kda_status kda_linear_chunk_bwd_device_status(const void* workspace, kda_dtype dtype, const int32_t* cu_seqlens_host,
                                              int n_seqs, int B, int T, int H, int dk, int dv, void* stream) {
    return chunk_status(true, workspace, dtype, cu_seqlens_host, n_seqs, B, T, H, dk, dv, stream);
}

kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, const void* log_alpha, kda_decay decay,
                                  kda_dtype dtype, float* state, int N, int H, int dk, int dv, void* o, void* stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    kda_status st = check_decay(decay);
    if (st != KDA_OK) return st;
    if (N < 0 || H <= 0 || !((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return KDA_ERR_SHAPE;
    if ((long long)N * H * (dv / 32) > 0x7fffffffLL) return KDA_ERR_SHAPE;   // the grid
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !log_alpha || !state || !o) return KDA_ERR_NULL;
    if (!all_aligned({q, k, v, (const void*)state, (const void*)o}) || !aligned4(log_alpha)) return KDA_ERR_ALIGN;
    const Sizes z(dtype, decay, (size_t)N * H, N, H, dk, dv);
    if ((st = check_apart({{o, z.v}, {state, z.state}},
                          {{q, z.k}, {k, z.k}, {v, z.v}, {log_alpha, z.la}, {state, z.state}})) != KDA_OK)
        return st;
    if ((st = check_device()) != KDA_OK) return st;
    const LinDecay dec{log_alpha, decay == KDA_DECAY_HEAD};
    return launch_lin_decode(dtype, q, k, v, dec, state, N, H, dk, dv, o, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
