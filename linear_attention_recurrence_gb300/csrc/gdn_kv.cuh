// Shared by the kernels of the paged 4-bit cache: where a sequence's rows and pages lie, and
// the reading of codes and scales.
#pragma once

#include "gdn_kv.h"
#include "gdn_ssm.cuh"

namespace gdn {

// Rows [begin, end) of sequence s (none, where a bound is outside [0, T] or they decrease).
__device__ __forceinline__ void kv_rows(const KvSeqs& q, int s, int64_t& begin, int64_t& end) {
    if (q.cu) {
        begin = __ldg(q.cu + s);
        end = __ldg(q.cu + s + 1);
        if (begin < 0 || end > q.T || end < begin) end = begin = 0;
    } else {
        begin = s * q.per_seq;
        end = begin + q.per_seq;
    }
}
// Tokens that a sequence's row of the table has places for (below 2^31 by a few tiles, so that
// a place, and the last of its tile, is an int).
__device__ __forceinline__ int64_t kv_capacity(const KvSeqs& q) {
    const int64_t n = static_cast<int64_t>(q.max_pages) << q.page_log2;
    return n < INT32_MAX - 1023 ? n : INT32_MAX - 1023;
}
// The page of place `at` of sequence s, or -1 if there is none.
__device__ __forceinline__ int64_t kv_page(const KvSeqs& q, int s, int64_t at) {
    if (at < 0 || at >= kv_capacity(q)) return -1;
    const int32_t page = __ldg(q.table + s * q.table_stride + (at >> q.page_log2));
    return page >= 0 && page < q.n_pages ? page : -1;
}
// Bytes of one page of one KV head's keys (or values): codes, then scales.
__host__ __device__ __forceinline__ int64_t kv_plane(int page_log2, int head_dim) {
    return static_cast<int64_t>(head_dim / 2 + head_dim / kKvGroup) << page_log2;
}

// Two codes of a byte (the low half first), as FP16: exact.
__device__ __forceinline__ void e2m1_to_f16(uint32_t word, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(word));
}
// Two e4m3 scales (the low byte first), as FP16: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Whether one of four e4m3 bytes is a NaN (0x7f or 0xff).
__device__ __forceinline__ bool any_e4m3_nan(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

}  // namespace gdn
