// Host-side helpers shared by the C entry points (defined in kda_api.cu): problem
// geometry, the sequence and chunk tables in the workspace, argument and device checks.
#pragma once

#include <stddef.h>
#include <vector>

#include "kda_internal.cuh"

namespace kda {

constexpr size_t kAlign = 256;   // workspace alignment and granularity

size_t align_up(size_t x);
bool aligned16(const void* p);

// Problem geometry shared by the workspace query and the launch.
struct Plan {
    int n_seqs = 0;
    int n_chunks = 0;
    long long total_tokens = 0;
    bool varlen = false;
    std::vector<SeqInfo> natural;   // chunk0 non-decreasing (varlen only)
    std::vector<SeqInfo> by_len;    // longest first (varlen only)
};

kda_status make_plan(int B, int T, int H, int dk, int dv, int C, const int32_t* cu, int n_seqs, Plan& p);

// The same for checked sizes and chunks of any length C.
kda_status plan_sequences(int B, int T, int C, const int32_t* cu, int n_seqs, Plan& p);

// Bytes of the sequence tables and the chunk table at the start of a workspace.
size_t table_bytes(const Plan& p);
// The per-chunk table follows the two sequence tables.
int4* chunk_table(SeqInfo* tables, size_t n_seqs);
// Natural order then longest first, 2 n_seqs entries at `dst`, then the per-chunk
// table of n_chunks entries of C tokens; returns the number of launches (with `mark`,
// timing-hook event i follows the i-th of them).
int upload_tables(SeqInfo* dst, const std::vector<SeqInfo>& natural, const std::vector<SeqInfo>& by_len,
                  int n_chunks, int C, cudaStream_t s, cudaError_t* err, bool mark = false);

// Device capability check, cached per device ordinal.
kda_status check_device();

// The limit that kda_set_test_wait_limit armed on this thread for the kernel of `bit` (0: none),
// disarmed by the asking.
unsigned long long take_test_wait(unsigned bit);

// Copy the error word at `offset` of the workspace to the host after `stream` finishes.
kda_status read_error_word(const void* workspace, size_t offset, void* stream);

}  // namespace kda
