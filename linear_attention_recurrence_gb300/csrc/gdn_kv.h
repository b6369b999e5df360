// Host-side interface between the C ABI of the paged 4-bit cache (gdn_kv_api.cu) and its
// kernel files, with the cache's layout.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

constexpr int kKvGroup = 16;  // elements of a row that share a scale

// The sequences of a call and their pages.
struct KvSeqs {
    const int32_t* cu;       // [n_seq + 1], or nullptr: n_seq sequences of per_seq rows each
    const int32_t* kv_lens;  // [n_seq]
    const int32_t* table;    // [n_seq][max_pages], rows table_stride apart
    int64_t table_stride;
    int64_t T;
    int64_t n_pages;
    int64_t per_seq;
    int n_seq, max_pages, page_log2;
};

// ---- appending (gdn_kv_append.cu) ----
struct KvAppendParams {
    const void *q, *k, *v;  // q may be nullptr
    void *q_out, *k_out, *v_out;  // each may be nullptr (q_out with q)
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride, v_out_stride;
    const float* inv_freq;  // [rotary / 2]
    const int32_t* positions;  // [T] or nullptr: a row's place in its cache
    const float *k_scale, *v_scale;  // [n_kv] or nullptr
    uint8_t* cache;
    KvSeqs s;
    int n_heads, n_kv, head_dim, rotary, interleaved, dtype;
    bool vector;  // every row of 16 bytes' pieces
};
cudaError_t launch_kv_append(const KvAppendParams& p, int sm_count, cudaStream_t s);

// ---- attention ----
struct KvAttentionParams {
    const void* q;
    void* out;
    float* lse;  // [T][n_heads] or nullptr
    int64_t q_stride, out_stride;
    const float *k_scale, *v_scale;
    const uint8_t* cache;
    KvSeqs s;
    float scale;  // of the scores, times log2 e
    int n_heads, n_kv, head_dim, causal, window, dtype;
    bool vector;  // q's and out's rows on 16-byte boundaries
    bool whole;   // (gdn_kv_few.cu's: its units are not cut)
    void* workspace;
    int* status;
};
// Sequences of at most so many rows (tokens x heads of a group) are gdn_kv_few.cu's, the others
// gdn_kv_prompt.cu's, whatever else a call has; each launch leaves the other's alone.
// Few / prompt, us: 16 sequences of up to 6000 tokens, 16 KV heads of 128, of 12 rows 53 / 162, of
// 24 115 / 188, of 48 214 / 159, one sequence of 32768, of 30 rows 63 / 86, of 60 120 / 87.
constexpr int kKvFewRows = 32;
// The launches of each count themselves (gdn_launch_count).
// On the warps' own MMAs, 8 or 16 rows at a time (gdn_kv_few.cu).
size_t kv_few_workspace(const KvSeqs& q, int n_kv, int head_dim, int sm_count);
cudaError_t launch_kv_few(const KvAttentionParams& p, int sm_count, cudaStream_t s);
// On tcgen05, 256 rows at a time (gdn_kv_prompt.cu).
int64_t kv_prompt_ctas(int64_t T, int n_seq, int n_heads, int n_kv);  // at most so many, where no unit is split
size_t kv_prompt_workspace(const KvSeqs& q, bool even, int n_heads, int n_kv, int head_dim, int sm_count);
cudaError_t launch_kv_prompt(const KvAttentionParams& p, int sm_count, cudaStream_t s);

}  // namespace gdn
