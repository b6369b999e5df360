// Argument checks shared by the C entry points of the operators over packed rows.
#pragma once

#include <atomic>
#include <cstdint>
#include <string>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

inline int bad(const std::string& msg) { return internal_fail(GDN_ERR_INVALID_ARG, msg); }
inline int unsupported(const std::string& msg) { return internal_fail(GDN_ERR_UNSUPPORTED, msg); }

inline int cuda_bad(cudaError_t e, const char* what) {
    cudaGetLastError();  // the launch error is reported here, not by the caller's next call
    return internal_fail(GDN_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

inline int elem_bytes(int dtype) { return dtype == GDN_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == GDN_F32 || dtype == GDN_BF16 || dtype == GDN_F16; }
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A byte range of an argument; an empty one overlaps nothing.  Rows that lie apart (columns of a
// wider row, say) may have their distance and width too.
struct Range {
    const void* p;
    size_t n;
    size_t stride = 0, width = 0;  // in bytes; 0: not looked at
};
inline Range rows_range(const void* p, int64_t rows, int64_t stride, int64_t width, int elem) {
    if (!p || rows <= 0) return {nullptr, 0};
    return {p, static_cast<size_t>((rows - 1) * stride + width) * elem};
}
// The same, where other columns of the same wider rows are no overlap.
inline Range columns_range(const void* p, int64_t rows, int64_t stride, int64_t width, int elem) {
    Range r = rows_range(p, rows, stride, width, elem);
    if (r.n && rows > 1) r.stride = static_cast<size_t>(stride) * elem, r.width = static_cast<size_t>(width) * elem;
    return r;
}
inline bool overlaps(const Range& a, const Range& b) {
    if (!a.n || !b.n) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (a0 >= b0 + b.n || b0 >= a0 + a.n) return false;
    if (!a.stride || a.stride != b.stride || a.width > a.stride) return true;
    // rows the same distance apart: b's columns from a's first one on, around the row's end
    const size_t at = b0 >= a0 ? (b0 - a0) % a.stride : (a.stride - (a0 - b0) % a.stride) % a.stride;
    return at < a.width || at + b.width > a.stride;
}
template <int I, int O>
bool any_overlap(const Range (&ins)[I], const Range (&outs)[O]) {
    for (int i = 0; i < O; ++i) {
        for (int j = 0; j < I; ++j)
            if (overlaps(outs[i], ins[j])) return true;
        for (int j = i + 1; j < O; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

// Multiprocessors of the current device, asked once per device.
inline int sm_count(int* out) {
    static std::atomic<int> counts[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_bad(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return unsupported("device ordinal out of range");
    int n = counts[dev].load();
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_bad(e, "cudaDeviceGetAttribute");
        counts[dev].store(n);
    }
    *out = n;
    return GDN_OK;
}

inline constexpr int64_t kMaxRows = INT32_MAX - 4096;  // cu_seqlens and TMA coordinates are 32-bit
inline constexpr int64_t kMaxStride = int64_t{1} << 40;

}  // namespace gdn
