// C ABI of the paged 4-bit cache (declared in include/gdn.h): argument checks and launches.
#include <cmath>
#include <cstdint>

#include "gdn.h"
#include "gdn_checks.h"
#include "gdn_kv.h"
#include "gdn_ssm.h"

namespace {
using namespace gdn;

// Checks shared by both operators, and the sequences; GDN_OK also when nothing is left to do.
int check_cache(KvSeqs* s, int64_t T, int n_seq, const int32_t* cu, int64_t n_pages, int page_size, int64_t table_stride,
                int max_pages, int n_heads, int n_kv, int head_dim) {
    if (T < 0) return bad("T < 0");
    if (T > kMaxRows) return unsupported("T too large for 32-bit sequence bounds");
    if (n_seq < 0) return bad("n_seq < 0");
    if (!cu && n_seq > 0 && T % n_seq != 0) return bad("sequences of different lengths need cu_seqlens");
    if (n_heads <= 0 || n_kv <= 0) return bad("n_heads and n_kv_heads must be positive");
    if (n_heads % n_kv != 0) return bad("n_heads must be a multiple of n_kv_heads");
    if (n_heads > 65535) return unsupported("n_heads > 65535");
    if (head_dim != 64 && head_dim != 128) return unsupported("head_dim must be 64 or 128");
    int log2 = 4;
    while (log2 < 8 && (1 << log2) < page_size) ++log2;
    if ((1 << log2) != page_size) return unsupported("page_size must be 16, 32, 64, 128 or 256");
    if (n_pages < 0 || n_pages > INT32_MAX) return bad("n_pages out of range");
    if (max_pages < 0) return bad("max_pages < 0");
    if (table_stride < max_pages || table_stride > kMaxStride) return bad("the table's row stride is out of range");
    s->T = T;
    s->n_seq = n_seq;
    s->per_seq = n_seq > 0 ? T / n_seq : 0;
    s->cu = cu;
    s->n_pages = n_pages;
    s->page_log2 = log2;
    s->table_stride = table_stride;
    s->max_pages = max_pages;
    return GDN_OK;
}
Range lens_range(const KvSeqs& s) { return {s.kv_lens, static_cast<size_t>(s.n_seq) * 4}; }
Range cu_range(const KvSeqs& s) { return {s.cu, s.cu ? (static_cast<size_t>(s.n_seq) + 1) * 4 : 0}; }
Range table_range(const KvSeqs& s) { return rows_range(s.table, s.n_seq, s.table_stride, s.max_pages, 4); }
size_t cache_bytes(const KvSeqs& s, int n_kv, int head_dim) {
    return static_cast<size_t>(s.n_pages) * n_kv * 2 * (static_cast<size_t>(head_dim / 2 + head_dim / kKvGroup) << s.page_log2);
}
// Whether some sequence may have few rows, or many: with cu_seqlens, of the T rows any number may be
// a sequence's.
bool may_have_few(int64_t rows_each, int group, bool even) {
    return even ? rows_each * group <= gdn::kKvFewRows : group <= gdn::kKvFewRows;
}
bool may_have_prompts(int64_t T, int64_t rows_each, int group, bool even) {
    return (even ? rows_each : T) * group > gdn::kKvFewRows;
}
// (Launches on one stream may use the same memory.)
size_t workspace_of(const KvSeqs& q, int n_heads, int n_kv, int head_dim, int sms) {
    const int group = n_heads / n_kv;
    const bool even = !q.cu;
    const size_t a = may_have_few(q.per_seq, group, even) ? kv_few_workspace(q, n_kv, head_dim, sms) : 0;
    const size_t b = may_have_prompts(q.T, q.per_seq, group, even) ? kv_prompt_workspace(q, even, n_heads, n_kv, head_dim, sms) : 0;
    return a > b ? a : b;
}
// Whether every row of `e`-byte elements starts on a 16-byte boundary.
bool rows16(const void* p, int64_t stride, int e) { return !p || (is_aligned(p, 16) && stride * e % 16 == 0); }
}  // namespace

extern "C" {

int gdn_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  const float* inv_freq, int rotary_dim, int interleaved, const int32_t* positions, const float* k_scale,
                  const float* v_scale, void* cache, int64_t n_pages, int page_size, const int32_t* block_table,
                  int64_t table_stride, int max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens, int n_seq,
                  void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* v_out,
                  int64_t v_out_stride, int64_t T, int n_heads, int n_kv_heads, int head_dim, int dtype,
                  void* cuda_stream) {
    KvAppendParams p{};
    if (int rc = check_cache(&p.s, T, n_seq, cu_seqlens, n_pages, page_size, table_stride, max_pages, n_heads, n_kv_heads,
                             head_dim))
        return rc;
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (rotary_dim < 0 || rotary_dim > head_dim) return bad("rotary_dim must be between 0 and head_dim");
    if (rotary_dim % 32 != 0) return unsupported("rotary_dim must be a multiple of 32");
    if (interleaved != 0 && interleaved != 1) return bad("interleaved must be 0 or 1");
    if (!q != !q_out) return bad("q and q_out come together");
    const int64_t qw = static_cast<int64_t>(n_heads) * head_dim, kw = static_cast<int64_t>(n_kv_heads) * head_dim;
    const int64_t strides[] = {q ? q_stride : 0, k_stride, v_stride, q_out ? q_out_stride : 0, k_out ? k_out_stride : 0,
                               v_out ? v_out_stride : 0};
    for (int64_t st : strides)
        if (st < 0 || st > kMaxStride) return bad("a row stride is out of range");
    if ((q_out && q_out_stride < qw) || (k_out && k_out_stride < kw) || (v_out && v_out_stride < kw))
        return bad("an output's row stride is below its row");
    if (T == 0 || n_seq == 0) return GDN_OK;
    if (!k || !v || !cache || !kv_lens || (!block_table && max_pages > 0) || (rotary_dim > 0 && !inv_freq))
        return bad("null pointer");
    const int e = elem_bytes(dtype);
    if (!is_aligned(q, e) || !is_aligned(k, e) || !is_aligned(v, e) || !is_aligned(q_out, e) || !is_aligned(k_out, e) ||
        !is_aligned(v_out, e) || !is_aligned(inv_freq, 4) || !is_aligned(positions, 4) || !is_aligned(k_scale, 4) ||
        !is_aligned(v_scale, 4) || !is_aligned(block_table, 4) || !is_aligned(kv_lens, 4) || !is_aligned(cu_seqlens, 4))
        return bad("an argument is not aligned to its element");
    if (!is_aligned(cache, 16)) return bad("the cache must be 16-byte aligned");
    const bool in_place = q && q == q_out;
    if (in_place && q_stride != q_out_stride && T > 1) return bad("in place, q's strides must agree");
    p.s.table = block_table;
    p.s.kv_lens = kv_lens;
    const size_t scale4 = static_cast<size_t>(n_kv_heads) * 4;
    const Range ins[] = {in_place ? Range{nullptr, 0} : columns_range(q, T, q_stride, qw, e), columns_range(k, T, k_stride, kw, e),
                         columns_range(v, T, v_stride, kw, e), {inv_freq, inv_freq ? static_cast<size_t>(rotary_dim) * 2 : 0},
                         {positions, positions ? static_cast<size_t>(T) * 4 : 0}, {k_scale, k_scale ? scale4 : 0},
                         {v_scale, v_scale ? scale4 : 0}, table_range(p.s), lens_range(p.s), cu_range(p.s)};
    const Range outs[] = {columns_range(q_out, T, q_out_stride, qw, e), columns_range(k_out, T, k_out_stride, kw, e),
                          columns_range(v_out, T, v_out_stride, kw, e), {cache, cache_bytes(p.s, n_kv_heads, head_dim)}};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    p.q = q, p.k = k, p.v = v, p.q_out = q_out, p.k_out = k_out, p.v_out = v_out;
    p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.q_out_stride = q_out_stride, p.k_out_stride = k_out_stride, p.v_out_stride = v_out_stride;
    p.inv_freq = inv_freq, p.positions = positions, p.k_scale = k_scale, p.v_scale = v_scale;
    p.cache = static_cast<uint8_t*>(cache);
    p.n_heads = n_heads, p.n_kv = n_kv_heads, p.head_dim = head_dim, p.rotary = rotary_dim, p.interleaved = interleaved;
    p.dtype = dtype;
    p.vector = rows16(q, q_stride, e) && rows16(k, k_stride, e) && rows16(v, v_stride, e) &&
               rows16(q_out, q_out_stride, e) && rows16(k_out, k_out_stride, e) && rows16(v_out, v_out_stride, e);
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    cudaError_t err = launch_kv_append(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err != cudaSuccess) return cuda_bad(err, "cache append launch");
    internal_count_launch();
    return GDN_OK;
}

size_t gdn_kv_attention_workspace_bytes(int64_t T, int n_seq, int even, int page_size, int max_pages, int n_heads,
                                        int n_kv_heads, int head_dim) {
    int sms = 0;
    KvSeqs q{};
    // (the bounds themselves are not looked at: any will do)
    const int32_t some = 0;
    if (T <= 0 || n_seq <= 0 ||
        check_cache(&q, T, n_seq, even ? nullptr : &some, 0, page_size, max_pages, max_pages, n_heads, n_kv_heads, head_dim) ||
        sm_count(&sms) != GDN_OK)
        return 0;
    return workspace_of(q, n_heads, n_kv_heads, head_dim, sms);
}

int gdn_kv_attention(const void* q, int64_t q_stride, const void* cache, int64_t n_pages, int page_size,
                     const int32_t* block_table, int64_t table_stride, int max_pages, const int32_t* kv_lens,
                     const int32_t* cu_seqlens, int n_seq, const float* k_scale, const float* v_scale, float scale,
                     int causal, int window, void* out, int64_t out_stride, float* lse, int64_t T, int n_heads,
                     int n_kv_heads, int head_dim, int dtype, void* workspace, size_t workspace_bytes,
                     void* cuda_stream) {
    KvAttentionParams p{};
    if (int rc = check_cache(&p.s, T, n_seq, cu_seqlens, n_pages, page_size, table_stride, max_pages, n_heads, n_kv_heads,
                             head_dim))
        return rc;
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (dtype == GDN_F32) return unsupported("attention over the cache takes 16-bit queries");
    if (causal != 0 && causal != 1) return bad("causal must be 0 or 1");
    if (window < 0) return bad("window < 0");
    if (window > 0 && !causal) return bad("a window goes with causal");
    const float scale2 = scale * 1.4426950408889634f;  // (exponentials are of base 2)
    if (!std::isfinite(scale2)) return bad("scale must be finite, times log2 e too");
    const int64_t qw = static_cast<int64_t>(n_heads) * head_dim;
    if (q_stride < 0 || q_stride > kMaxStride || out_stride > kMaxStride) return bad("a row stride is out of range");
    if (out_stride < qw) return bad("out's row stride is below its row");
    if (T == 0 || n_seq == 0) return GDN_OK;
    if (!q || !out || !kv_lens || (!cache && n_pages > 0) || (!block_table && max_pages > 0)) return bad("null pointer");
    const int e = elem_bytes(dtype);
    if (!is_aligned(q, e) || !is_aligned(out, e) || !is_aligned(lse, 4) || !is_aligned(k_scale, 4) ||
        !is_aligned(v_scale, 4) || !is_aligned(block_table, 4) || !is_aligned(kv_lens, 4) || !is_aligned(cu_seqlens, 4))
        return bad("an argument is not aligned to its element");
    if (!is_aligned(cache, 16) || !is_aligned(workspace, 16)) return bad("the cache and the workspace must be 16-byte aligned");
    p.s.table = block_table;
    p.s.kv_lens = kv_lens;
    int sms = 0;
    const int no_device = sm_count(&sms);  // (told behind what the arguments have wrong)
    const size_t need = no_device ? 0 : workspace_of(p.s, n_heads, n_kv_heads, head_dim, sms);
    if (need && (!workspace || workspace_bytes < need)) return bad("the workspace is missing or too small");
    const size_t scale4 = static_cast<size_t>(n_kv_heads) * 4;
    const Range ins[] = {columns_range(q, T, q_stride, qw, e), {cache, cache_bytes(p.s, n_kv_heads, head_dim)},
                         {k_scale, k_scale ? scale4 : 0}, {v_scale, v_scale ? scale4 : 0}, table_range(p.s),
                         lens_range(p.s), cu_range(p.s)};
    const Range outs[] = {columns_range(out, T, out_stride, qw, e),
                          {lse, lse ? static_cast<size_t>(T) * n_heads * 4 : 0}, {workspace, workspace ? need : 0}};
    if (any_overlap(ins, outs)) return bad("an output overlaps another argument");
    p.q = q, p.out = out, p.lse = lse, p.q_stride = q_stride, p.out_stride = out_stride;
    p.k_scale = k_scale, p.v_scale = v_scale, p.cache = static_cast<const uint8_t*>(cache);
    p.scale = scale2;
    p.n_heads = n_heads, p.n_kv = n_kv_heads, p.head_dim = head_dim, p.causal = causal, p.window = window, p.dtype = dtype;
    p.vector = rows16(q, q_stride, e) && rows16(out, out_stride, e);
    if (kv_prompt_ctas(T, n_seq, n_heads, n_kv_heads) > INT32_MAX / 2) return unsupported("too many rows and heads");
    p.workspace = workspace;
    if (no_device) return no_device;
    if (cudaError_t err = ssm_status_word(&p.status); err != cudaSuccess) return cuda_bad(err, "cache attention set-up");
    const int group = n_heads / n_kv_heads;
    const bool even = !cu_seqlens;
    cudaError_t err = cudaSuccess;
    if (may_have_few(p.s.per_seq, group, even)) err = launch_kv_few(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err == cudaSuccess && may_have_prompts(T, p.s.per_seq, group, even))
        err = launch_kv_prompt(p, sms, static_cast<cudaStream_t>(cuda_stream));
    if (err != cudaSuccess) return cuda_bad(err, "cache attention launch");
    return GDN_OK;
}

}  // extern "C"
