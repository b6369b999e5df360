// Host-side interface between the C ABI of the selective state space operators and
// the block norm (gdn_ssm_api.cu) and their kernel files.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

struct SsmSeqs;

// ---- causal convolution over packed sequences (gdn_ssm_conv.cu) ----
struct SsmConvParams {
    const void* x;
    void* y;
    int64_t x_stride, y_stride;  // elements between rows
    const float* w;              // [channels][width]
    const float* bias;           // [channels] or nullptr
    void* hist;                  // [n_slots][width - 1][channels] or nullptr
    const int32_t* cu;
    const int32_t* slots;
    const uint8_t* has_state;
    int n_seq, n_slots;
    int64_t T;
    int channels, width, activation, dtype;
    bool vector;                 // rows are whole pieces of 4 elements on boundaries of that size, w on 16 bytes
};
cudaError_t launch_ssm_conv(const SsmConvParams& p, int sm_count, cudaStream_t s);

// ---- selective scan over packed sequences ----
struct SsmScanParams {
    const void *x, *a, *B, *C, *z;  // z may be nullptr
    void* y;
    int64_t x_stride, a_stride, b_stride, c_stride, z_stride, y_stride;  // elements between rows
    const float *A_log, *dt_bias, *D;  // [n_heads]; D may be nullptr
    float* states;                     // [n_slots][n_heads][state_dim][head_dim] or nullptr
    const int32_t* cu;
    const int32_t* slots;
    const uint8_t* has_state;
    int n_seq, n_slots;
    int64_t T;
    int n_heads, n_groups, head_dim, state_dim, dtype;
};
// One token after the other, the state in registers (gdn_ssm_scan.cu).
cudaError_t launch_ssm_scan_tokens(const SsmScanParams& p, cudaStream_t s);

// Chunks of 128 tokens on the tensor cores (gdn_ssm_scan_tc.cu): 16-bit types, head_dim
// and state_dim 64 or 128, rows of x, B and C on 16-byte boundaries.
// Tokens per sequence from which it is taken, tensor / token form, BF16, us.  48 heads of
// 128 x 128: 1 sequence of 16 tokens 14 / 9, 32 15 / 15, 64 15 / 21, 128 15 / 33; 4 of 32
// 24 / 28; 32 of 16 114 / 100, of 32 120 / 161, of 128 136 / 547 (FP16 within 4 us of it).
// Heads of 64 meet between 32 and 64 tokens: 64 heads of 64 x 128, 1 sequence of 32 15 / 11, 64
// 14 / 15; 4 of 32 23 / 21; 32 of 32 134 / 105, of 64 138 / 197; 24 of 64 x 64, 32 of 32 58 / 34,
// of 64 60 / 56.
constexpr int kSsmTcMinTokens = 32;
bool ssm_scan_tc_sizes(int head_dim, int state_dim, int dtype, int64_t T, int n_seq);
size_t ssm_scan_tc_workspace(int64_t T, int n_seq, int n_heads, int head_dim, int state_dim, int sm_count);
cudaError_t launch_ssm_scan_tc(const SsmScanParams& p, void* workspace, int sm_count, cudaStream_t s);
// The status word of the bounded waits of the tensor form and the block norm: its address
// on the current device, and its value there, read and cleared (0 if none of them ran).
cudaError_t ssm_status_word(int** word);
cudaError_t ssm_take_status(int device, int* word);

// ---- one token of the convolution and the scan for each request (gdn_ssm_step.cu) ----
struct SsmStepParams {
    const void *xbc, *a, *z;  // z may be nullptr
    void* y;
    int64_t xbc_stride, a_stride, z_stride, y_stride;
    const float *conv_w, *conv_bias;  // [cw][width], [cw] or nullptr
    const float *A_log, *dt_bias, *D;
    void* hist;                       // [n_slots][width - 1][cw]
    float* states;
    const int32_t* slots;
    int batch, n_slots, n_heads, n_groups, head_dim, state_dim, width, activation, dtype;
};
cudaError_t launch_ssm_step(const SsmStepParams& p, int sm_count, cudaStream_t s);

// ---- norms around a block (gdn_block_norm.cu) ----
struct BlockNormParams {
    const void *b, *r, *gate;  // gate may be nullptr
    void *r_out, *y;
    int64_t b_stride, r_stride, gate_stride, r_out_stride, y_stride;
    const float *w_post, *w_pre;  // w_post may be nullptr
    float scale, eps;
    int64_t T;
    int dim, gate_sigmoid, dtype, stream_dtype;
    int vec;      // elements that every row's start is a multiple of (8, 4, 2 or 1)
    int* status;
};
cudaError_t launch_block_norm(const BlockNormParams& p, int sm_count, cudaStream_t s);

}  // namespace gdn
