// C ABI of the selective state space operators and the block norm (declared in
// include/gdn.h): argument checks and launches.
#include <cmath>
#include <cstdint>

#include "gdn.h"
#include "gdn_checks.h"
#include "gdn_ssm.h"

namespace {
using namespace gdn;

// Checks shared by the packed operators; GDN_OK also when nothing is left to do.
int check_seqs(int64_t T, int n_seq, int n_slots, const int32_t* cu, bool stateful) {
    if (T < 0) return bad("T < 0");
    if (T > kMaxRows) return unsupported("T too large for 32-bit sequence bounds");
    if (n_seq < 0) return bad("n_seq < 0");
    if (!cu && n_seq > 1) return bad("several sequences need cu_seqlens");
    if (stateful && n_slots <= 0) return bad("n_slots must be positive");
    return GDN_OK;
}

int check_heads(int n_heads, int n_groups, int head_dim, int state_dim) {
    if (n_heads <= 0 || n_groups <= 0 || head_dim <= 0 || state_dim <= 0)
        return bad("n_heads, n_groups, head_dim and state_dim must be positive");
    if (n_heads % n_groups != 0) return bad("n_heads must be a multiple of n_groups");
    if (head_dim % 32 != 0 || head_dim > 256) return unsupported("head_dim must be a multiple of 32, at most 256");
    if (state_dim != 16 && state_dim != 32 && state_dim != 64 && state_dim != 128)
        return unsupported("state_dim must be 16, 32, 64 or 128");
    if (n_heads > 65535) return unsupported("n_heads > 65535");
    return GDN_OK;
}

bool tensor_form(int head_dim, int state_dim, int dtype, int64_t T, int n_seq) {
    return gdn::internal_option(GDN_OPT_SSM_SCAN_FORM) == 0 &&
           gdn::ssm_scan_tc_sizes(head_dim, state_dim, dtype, T, n_seq);
}
}  // namespace

extern "C" {

int gdn_ssm_conv(const void* x, int64_t x_stride, const float* w, const float* bias, void* hist,
                 const int32_t* cu_seqlens, const int32_t* slots, const uint8_t* has_state, int n_seq, int n_slots,
                 void* y, int64_t y_stride, int64_t T, int channels, int width, int activation, int dtype,
                 void* cuda_stream) {
    using namespace gdn;
    if (int rc = check_seqs(T, n_seq, n_slots, cu_seqlens, hist != nullptr)) return rc;
    if (channels <= 0) return bad("channels must be positive");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (activation != 0 && activation != 1) return bad("activation must be 0 or 1");
    if (width < 2 || width > 4) return unsupported("width must be 2, 3 or 4");
    if (x_stride < 0 || y_stride < channels || x_stride > kMaxStride || y_stride > kMaxStride)
        return bad("row strides: x's must be >= 0, y's at least the number of channels");
    if (T == 0 || n_seq == 0) return GDN_OK;
    if (!x || !w || !y) return bad("null pointer");
    const int e = elem_bytes(dtype);
    if (!is_aligned(x, e) || !is_aligned(y, e) || !is_aligned(hist, e) || !is_aligned(w, 4) || !is_aligned(bias, 4) ||
        !is_aligned(cu_seqlens, 4) || !is_aligned(slots, 4))
        return bad("an argument is not aligned to its element");
    const Range ins[] = {rows_range(x, T, x_stride, channels, e), {w, static_cast<size_t>(channels) * width * 4},
                         {bias, bias ? static_cast<size_t>(channels) * 4 : 0},
                         {cu_seqlens, cu_seqlens ? (static_cast<size_t>(n_seq) + 1) * 4 : 0},
                         {slots, slots ? static_cast<size_t>(n_seq) * 4 : 0},
                         {has_state, has_state ? static_cast<size_t>(n_seq) : 0}};
    const Range outs[] = {rows_range(y, T, y_stride, channels, e),
                          {hist, hist ? static_cast<size_t>(n_slots) * (width - 1) * channels * e : 0}};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    const bool vector = is_aligned(x, 4 * e) && is_aligned(y, 4 * e) && is_aligned(hist, 4 * e) && is_aligned(w, 16) &&
                        channels % 4 == 0 && x_stride % 4 == 0 && y_stride % 4 == 0;
    if (channels > (vector ? 4 : 1) * 128 * 65535) return unsupported("too many channels");
    const SsmConvParams p{x, y, x_stride, y_stride, w, bias, hist, cu_seqlens, slots, has_state, n_seq, n_slots, T,
                          channels, width, activation, dtype, vector};
    cudaError_t err = launch_ssm_conv(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err != cudaSuccess) return cuda_bad(err, "convolution launch");
    internal_count_launch();
    return GDN_OK;
}

size_t gdn_ssm_scan_workspace_bytes(int64_t T, int n_seq, int n_heads, int head_dim, int state_dim, int dtype) {
    int sms = 0;
    if (T <= 0 || n_seq <= 0 || n_heads <= 0 || head_dim <= 0 || state_dim <= 0 ||
        !tensor_form(head_dim, state_dim, dtype, T, n_seq) || sm_count(&sms) != GDN_OK)
        return 0;
    return gdn::ssm_scan_tc_workspace(T, n_seq, n_heads, head_dim, state_dim, sms);
}

int gdn_ssm_scan(const void* x, int64_t x_stride, const void* a, int64_t a_stride, const void* B, int64_t b_stride,
                 const void* C, int64_t c_stride, const void* z, int64_t z_stride, const float* A_log,
                 const float* dt_bias, const float* D, float* states, const int32_t* cu_seqlens, const int32_t* slots,
                 const uint8_t* has_state, int n_seq, int n_slots, void* y, int64_t y_stride, int64_t T, int n_heads,
                 int n_groups, int head_dim, int state_dim, int dtype, void* workspace, size_t workspace_bytes,
                 void* cuda_stream) {
    using namespace gdn;
    if (int rc = check_seqs(T, n_seq, n_slots, cu_seqlens, states != nullptr)) return rc;
    if (int rc = check_heads(n_heads, n_groups, head_dim, state_dim)) return rc;
    if (!known_dtype(dtype)) return bad("unknown dtype");
    const int64_t xw = static_cast<int64_t>(n_heads) * head_dim, bw = static_cast<int64_t>(n_groups) * state_dim;
    const int64_t strides[] = {x_stride, a_stride, b_stride, c_stride, z ? z_stride : 0, y_stride};
    for (int64_t st : strides)
        if (st < 0 || st > kMaxStride) return bad("a row stride is out of range");
    if (y_stride < xw) return bad("y's row stride is below its row");
    if (T == 0 || n_seq == 0) return GDN_OK;
    if (!x || !a || !B || !C || !A_log || !dt_bias || !y) return bad("null pointer");
    const int e = elem_bytes(dtype);
    if (!is_aligned(x, e) || !is_aligned(a, e) || !is_aligned(B, e) || !is_aligned(C, e) || !is_aligned(z, e) ||
        !is_aligned(y, e) || !is_aligned(A_log, 4) || !is_aligned(dt_bias, 4) || !is_aligned(D, 4) ||
        !is_aligned(cu_seqlens, 4) || !is_aligned(slots, 4))
        return bad("an argument is not aligned to its element");
    if (!is_aligned(states, 16) || !is_aligned(workspace, 16)) return bad("states and workspace must be 16-byte aligned");
    const size_t need = gdn_ssm_scan_workspace_bytes(T, n_seq, n_heads, head_dim, state_dim, dtype);
    if (need && (!workspace || workspace_bytes < need)) return bad("the workspace is missing or too small");
    const size_t heads4 = static_cast<size_t>(n_heads) * 4;
    const Range ins[] = {rows_range(x, T, x_stride, xw, e), rows_range(a, T, a_stride, n_heads, e),
                         rows_range(B, T, b_stride, bw, e), rows_range(C, T, c_stride, bw, e),
                         rows_range(z, T, z_stride, xw, e), {A_log, heads4}, {dt_bias, heads4}, {D, D ? heads4 : 0},
                         {cu_seqlens, cu_seqlens ? (static_cast<size_t>(n_seq) + 1) * 4 : 0},
                         {slots, slots ? static_cast<size_t>(n_seq) * 4 : 0},
                         {has_state, has_state ? static_cast<size_t>(n_seq) : 0}};
    const Range outs[] = {rows_range(y, T, y_stride, xw, e),
                          {states, states ? static_cast<size_t>(n_slots) * xw * state_dim * 4 : 0},
                          {workspace, workspace ? need : 0}};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    if (static_cast<int64_t>(n_seq) * n_heads * (head_dim / 32) > INT32_MAX) return unsupported("n_seq * n_heads too large");
    const SsmScanParams p{x, a, B, C, z, y, x_stride, a_stride, b_stride, c_stride, z_stride, y_stride, A_log, dt_bias,
                          D, states, cu_seqlens, slots, has_state, n_seq, n_slots, T, n_heads, n_groups, head_dim,
                          state_dim, dtype};
    // TMA takes rows on 16-byte boundaries that lie one after the other
    auto tma_rows = [](const void* ptr, int64_t stride, int64_t width) {
        return is_aligned(ptr, 16) && stride % 8 == 0 && stride >= width;
    };
    cudaError_t err;
    if (tensor_form(head_dim, state_dim, dtype, T, n_seq) && (T / 512 + n_seq) * n_heads <= INT32_MAX &&
        tma_rows(x, x_stride, xw) &&
        tma_rows(B, b_stride, bw) && tma_rows(C, c_stride, bw) &&
        (!z || tma_rows(z, z_stride, xw)) && tma_rows(y, y_stride, xw)) {
        int sms = 0;
        if (int rc = sm_count(&sms)) return rc;
        err = launch_ssm_scan_tc(p, workspace, sms, static_cast<cudaStream_t>(cuda_stream));
    } else {
        err = launch_ssm_scan_tokens(p, static_cast<cudaStream_t>(cuda_stream));
    }
    if (err != cudaSuccess) return cuda_bad(err, "scan launch");
    internal_count_launch();
    return GDN_OK;
}

int gdn_ssm_step(const void* xbc, int64_t xbc_stride, const void* a, int64_t a_stride, const void* z, int64_t z_stride,
                 const float* conv_w, const float* conv_bias, const float* A_log, const float* dt_bias, const float* D,
                 void* hist, float* states, const int32_t* slots, int n_slots, void* y, int64_t y_stride, int batch,
                 int n_heads, int n_groups, int head_dim, int state_dim, int width, int activation, int dtype,
                 void* cuda_stream) {
    using namespace gdn;
    if (batch < 0) return bad("batch < 0");
    if (int rc = check_heads(n_heads, n_groups, head_dim, state_dim)) return rc;
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (activation != 0 && activation != 1) return bad("activation must be 0 or 1");
    if (n_slots <= 0) return bad("n_slots must be positive");
    if (!slots && n_slots < batch) return bad("fewer slots than requests");
    if (width < 2 || width > 4) return unsupported("width must be 2, 3 or 4");
    if (batch > 65535) return unsupported("batch > 65535");
    if (n_heads / n_groups * (head_dim / 32) > 2048) return unsupported("more than 65536 state columns per group");
    const int64_t xw = static_cast<int64_t>(n_heads) * head_dim;
    const int64_t cw = xw + 2 * static_cast<int64_t>(n_groups) * state_dim;
    const int64_t strides[] = {xbc_stride, a_stride, z ? z_stride : 0, y_stride};
    for (int64_t st : strides)
        if (st < 0 || st > kMaxStride) return bad("a row stride is out of range");
    if (y_stride < xw) return bad("y's row stride is below its row");
    if (batch == 0) return GDN_OK;
    if (!xbc || !a || !conv_w || !A_log || !dt_bias || !hist || !states || !y) return bad("null pointer");
    const int e = elem_bytes(dtype);
    if (!is_aligned(xbc, e) || !is_aligned(a, e) || !is_aligned(z, e) || !is_aligned(y, e) || !is_aligned(hist, e) ||
        !is_aligned(conv_w, 4) || !is_aligned(conv_bias, 4) || !is_aligned(A_log, 4) || !is_aligned(dt_bias, 4) ||
        !is_aligned(D, 4) || !is_aligned(slots, 4))
        return bad("an argument is not aligned to its element");
    if (!is_aligned(states, 16)) return bad("states must be 16-byte aligned");
    const size_t heads4 = static_cast<size_t>(n_heads) * 4;
    const Range ins[] = {rows_range(xbc, batch, xbc_stride, cw, e), rows_range(a, batch, a_stride, n_heads, e),
                         rows_range(z, batch, z_stride, xw, e), {conv_w, static_cast<size_t>(cw) * width * 4},
                         {conv_bias, conv_bias ? static_cast<size_t>(cw) * 4 : 0}, {A_log, heads4}, {dt_bias, heads4},
                         {D, D ? heads4 : 0}, {slots, slots ? static_cast<size_t>(batch) * 4 : 0}};
    const Range outs[] = {rows_range(y, batch, y_stride, xw, e),
                          {hist, static_cast<size_t>(n_slots) * (width - 1) * cw * e},
                          {states, static_cast<size_t>(n_slots) * xw * state_dim * 4}};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    const SsmStepParams p{xbc, a, z, y, xbc_stride, a_stride, z_stride, y_stride, conv_w, conv_bias, A_log, dt_bias, D,
                          hist, states, slots, batch, n_slots, n_heads, n_groups, head_dim, state_dim, width,
                          activation, dtype};
    cudaError_t err = launch_ssm_step(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err != cudaSuccess) return cuda_bad(err, "step launch");
    internal_count_launch();
    return GDN_OK;
}

int gdn_block_norm(const void* b, int64_t b_stride, const void* residual, int64_t residual_stride, const void* gate,
                   int64_t gate_stride, int gate_sigmoid, const float* w_post, const float* w_pre, float scale,
                   float eps, void* residual_out, int64_t residual_out_stride, void* y, int64_t y_stride, int64_t T,
                   int dim, int dtype, int residual_dtype, void* cuda_stream) {
    using namespace gdn;
    if (T < 0) return bad("T < 0");
    if (dim <= 0) return bad("dim must be positive");
    if (!known_dtype(dtype) || !known_dtype(residual_dtype)) return bad("unknown dtype");
    if (residual_dtype != dtype && residual_dtype != GDN_F32) return unsupported("the residual is FP32 or of the block's type");
    if (gate_sigmoid != 0 && gate_sigmoid != 1) return bad("gate_sigmoid must be 0 or 1");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return bad("eps must be finite and >= 0");
    if (!std::isfinite(scale)) return bad("scale must be finite");
    if (dim > 16384) return unsupported("dim > 16384");
    if (T > kMaxRows) return unsupported("T too large");
    const int64_t strides[] = {b_stride, residual_stride, gate ? gate_stride : 0, residual_out_stride, y_stride};
    for (int64_t st : strides)
        if (st < 0 || st > kMaxStride) return bad("a row stride is out of range");
    if (residual_out_stride < dim || y_stride < dim) return bad("an output's row stride is below dim");
    if (T == 0) return GDN_OK;
    if (!b || !residual || !w_pre || !residual_out || !y) return bad("null pointer");
    const int e = elem_bytes(dtype), er = elem_bytes(residual_dtype);
    if (!is_aligned(b, e) || !is_aligned(gate, e) || !is_aligned(y, e) || !is_aligned(residual, er) ||
        !is_aligned(residual_out, er) || !is_aligned(w_post, 4) || !is_aligned(w_pre, 4))
        return bad("an argument is not aligned to its element");
    const bool in_place = residual_out == residual;
    if (in_place && residual_out_stride != residual_stride && T > 1) return bad("in place, the residual strides must agree");
    const size_t w4 = static_cast<size_t>(dim) * 4;
    const Range ins[] = {rows_range(b, T, b_stride, dim, e),
                         in_place ? Range{nullptr, 0} : rows_range(residual, T, residual_stride, dim, er),
                         rows_range(gate, T, gate_stride, dim, e), {w_post, w_post ? w4 : 0}, {w_pre, w4}};
    const Range outs[] = {rows_range(residual_out, T, residual_out_stride, dim, er), rows_range(y, T, y_stride, dim, e)};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    // the widest access (8 elements and down) that every row's start and length allow
    int vec = 8;
    auto fits = [&](const void* p, int64_t stride, int elem) {
        const int64_t bytes = static_cast<int64_t>(vec) * elem < 16 ? vec * elem : 16;
        return is_aligned(p, bytes) && stride * elem % bytes == 0;
    };
    while (vec > 1 && !(dim % vec == 0 && fits(b, b_stride, e) && fits(residual, residual_stride, er) &&
                        fits(residual_out, residual_out_stride, er) && fits(y, y_stride, e) &&
                        (!gate || fits(gate, gate_stride, e))))
        vec /= 2;
    BlockNormParams p{b, residual, gate, residual_out, y, b_stride, residual_stride, gate_stride,
                            residual_out_stride, y_stride, w_post, w_pre, scale, eps, T, dim, gate_sigmoid, dtype,
                            residual_dtype, vec, nullptr};
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    if (cudaError_t err = ssm_status_word(&p.status); err != cudaSuccess) return cuda_bad(err, "block norm set-up");
    cudaError_t err = launch_block_norm(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err != cudaSuccess) return cuda_bad(err, "block norm launch");
    internal_count_launch();
    return GDN_OK;
}

}  // extern "C"
