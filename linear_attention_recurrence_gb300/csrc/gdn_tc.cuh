// Shared by the kernels whose roles meet at mbarriers around 16-bit tcgen05 products: operand
// descriptors, MMAs, and bounded waits that a whole CTA gives up together.
#pragma once

#include "gdn_device.cuh"

namespace gdn {

constexpr uint32_t kBox = 16384;  // 128 rows x 64 elements, 128-byte swizzled

// ---- tcgen05, 16-bit operands ----
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// 128-byte swizzled operand whose rows are the K index (64 elements of M or N per row):
// blocks of 64 elements kBox apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t a) {
    return static_cast<uint64_t>((a & 0x3FFFF) >> 4) | (static_cast<uint64_t>(kBox >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// 128-byte swizzled operand whose rows are M or N (64 elements of K per row).
__device__ __forceinline__ uint64_t desc_k(uint32_t a) {
    return static_cast<uint64_t>((a & 0x3FFFF) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}
// 16 packed columns of this thread's lane.
__device__ __forceinline__ void tmem_st_u16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// CODE: what a wait that gave up reports.  CALL: polls behind the first are a call (a kernel that
// splits its registers unevenly can have none).
template <int CODE, bool CALL = true>
struct SyncOf {
    uint64_t* bar;
    volatile int* abort_flag;
    int* status;
};
// A poll suspends its thread for up to this long, so that waiting warps take few issue
// slots from the working ones; a wait gives up after kTcPolls of them (seconds).
constexpr uint32_t kSuspendNs = 20000, kTcPolls = 1u << 17;
__device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}
template <int CODE>
__device__ __forceinline__ bool wait_polls(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
    for (uint32_t i = 0; i < kTcPolls; ++i) {
        if (poll(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    *abort_flag = 1;
    report_error(status, CODE);
    return false;
}
// Waits for phase `n` (0, 1, ...) of a barrier.  False once some wait of the CTA gave up.
// (All but the first poll out of line: the code of all roles has to fit the caches.)
template <int CODE>
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
    return wait_polls<CODE>(bar, parity, abort_flag, status);
}
template <int CODE, bool CALL>
__device__ __forceinline__ bool wait_phase(const SyncOf<CODE, CALL>& s, int b, uint32_t n) {
    if constexpr (!CALL) return wait_polls<CODE>(&s.bar[b], n & 1, s.abort_flag, s.status);
    return poll(&s.bar[b], n & 1) || wait_more<CODE>(&s.bar[b], n & 1, s.abort_flag, s.status);
}
// The same for a whole warp: all lanes leave together, with one answer (the tensor-memory
// instructions behind a wait need a converged warp).
template <int CODE, bool CALL>
__device__ __forceinline__ bool wait_warp(const SyncOf<CODE, CALL>& s, int b, uint32_t n) {
    return __all_sync(0xffffffffu, wait_phase(s, b, n)) != 0;
}
// True in one lane of a converged warp.  (Not `lane == 0`: behind this predicate the compiler
// knows one lane runs and keeps the operands of MMAs and copies in uniform registers.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
// Waits (with a limit) until phase n of a copy's barrier has completed, whatever else happened.
__device__ __forceinline__ void land(uint64_t* bar, uint32_t n) {
    for (uint32_t i = 0; i < kTcPolls && !poll(bar, n & 1); ++i) {
    }
}
// Every MMA of the CTA ends before tensor memory is freed.
__device__ __forceinline__ void finish_mma(uint64_t* bar) {
    umma_commit(bar);
    for (uint32_t n = 0; n < kTcPolls && !poll(bar, 0); ++n) {
    }
}
// One arrival for the calling warp.
template <int CODE, bool CALL>
__device__ __forceinline__ void warp_arrive(const SyncOf<CODE, CALL>& s, int b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.bar[b]);
}

}  // namespace gdn
