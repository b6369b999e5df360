// Selective state space scan of 16-bit prompts on the tensor cores (sm_103a).
//
// The recurrence of gdn_ssm_scan.cu over chunks of 128 tokens.  Per head and chunk, with
// gamma_t the running sum of the log-decays inside the chunk, H the state before it and
// 16-bit x, B, C (the products' operands as they arrive):
//     G    = C B^T                                       128 x 128, K = state_dim
//     M    = G o e^(gamma_t - gamma_i) dt_i  (i <= t)    rounded to 16 bits
//     Y^T  = x^T M^T + (H^T C^T) diag(e^gamma_t)         128 x 128, K = 128 and state_dim
//     H^T <- e^gamma_last H^T + (w o x)^T B,  w_t = dt_t e^(gamma_last - gamma_t)
// in transposed form: head_dim is the MMA's M (tensor-memory lanes), so H^T stays in
// tensor memory as the FP32 accumulator of its update.  Every product is a tcgen05.mma
// of the rows' own type: H is rounded to it for the product with C (as M is: together
// one rounding of disjoint terms of y), but the update takes w o x in parts of that type
// (three of 8 bits for BF16, two of 11 for FP16), so the state keeps FP32's precision
// (in FP16 as far as its smallest step allows: 2^-24 of the chunk's largest w, whatever x is).
// An exponent of M is the sum of the log-decays behind token i up to t, from sums that start
// anew every 4 tokens (the difference of two sums from the chunk's start, up to 2^15, would be
// off by 2^-9); w comes from sums that start at the chunk's end.  So neither loses precision
// when the decay over the chunk is large.
// FP16's range is short: there dt and w enter M and the update divided by a power of two
// of each chunk (its largest dt, its largest w), which the output and the state's decay
// multiply back, so no step from 2^-60 to 2^24 leaves the range.  Nor do states and scores:
// H is rounded relative to a power of two of each 32 columns of x (their largest element), and
// where the scores of 32 tokens t pass the range, those are formed again relative to one of theirs.
//
// Work is one CTA per (head, segment of a sequence); it walks the segment's chunks.
// Where sequences x heads do not fill the device, sequences are cut into segments: a
// first launch forms, for every segment but the last, its own contribution to the state
// behind it (the update's product alone) and its decay; the second starts each segment
// from the sum of those before it.  The first walks a segment from its last chunk, with w
// down to the segment's end, so that its sum is never decayed.
//
// Warp roles (768 threads): warps 0-3 form M (lane = token); 4-7 the parts of w o x and the
// state's decay and rounding (lane = column of x); 8-19 the output; 20 issues the copies, 21
// the MMAs of the output's chain, 23 those of the state's (a tcgen05.mma waits in its thread
// while the tensor pipe is full, and the two chains wait for different roles), 22 forms the
// gates.  In the first launch warps 0-15 all form parts and 21 and 22 the gates.  A role's
// 16 x 16 tiles come and go as fragments (ldmatrix, stmatrix and the 16-lane forms of the
// tensor-memory accesses), so that x, z and y cross shared and global memory 16 bytes at a
// time although a lane's row is a column of x.
//
// What bounds it: the instructions of the roles around the products, and their latency, of
// the output's above all (5200 per scheduler and chunk, at a little under one in two cycles;
// the tensor pipe is busy a quarter of the time); memory next.  48 heads of 128 x 128, BF16,
// z: 32768 tokens of one sequence 496 us (the first launch 117 us, 1.4 us a chunk; the second
// 378 us, 4.4 us a chunk; 1.48 GB: 3.0 TB/s).  FP16 takes 535 us: the largest element of the
// state and the test of the scores, and what multiplies their powers back.  64 heads of
// 64 x 128, 8192 tokens: 208 us.  Steps on the way, BF16, 32768 tokens: z by 2-byte
// loads in the output 1052 us; fragments 883; eight output warps and z a half chunk ahead
// 792; the MMA chains apart and elected issuing lanes 691; code that fits the instruction
// caches (81 -> 55 KB: rolled loops, waits out of line) 670; x freed apart from B and C 652;
// twelve output warps 629; packed gates 619; the output in quarters of a chunk with two
// product buffers 550; descriptors stepped between MMAs 527; the first launch from the end
// 500; z and y addresses stepped 495; a quarter of Y1 ahead of G 491; exponents from groups of 4
// tokens 500; barriers by stage, one wait of the output for the state, x and the gates 496.
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "gdn_ssm.cuh"
#include "gdn_ssm.h"

namespace gdn {
namespace {

constexpr int L = 128;        // tokens per chunk
constexpr int kThreadsTc = 768;
constexpr int kOutGroups = 3;  // groups of 4 output warps
constexpr int kStages = 2, kMaxStages = 3;
constexpr int kCopyWarp = 20, kMmaWarp = 21, kGateWarp = 22, kStateMmaWarp = 23;

// tensor-memory columns
constexpr uint32_t TM_H = 0;     // H^T, FP32 [head_dim lanes][state_dim]
constexpr uint32_t TM_HB = 128;  // H^T in 16 bits, 2 per column
constexpr uint32_t TM_G = 192;   // G, 64 columns (tokens i) at a time [128 lanes t]
constexpr uint32_t TM_Y1 = 256;  // x^T M^T, two buffers of 32 columns (tokens t)
constexpr uint32_t TM_Y2 = 320;  // H^T C^T, 128 columns
constexpr uint32_t TM_XW = 448;  // parts of w o x: ring of blocks of 16 tokens, 8 columns a part
constexpr uint32_t TM_COLS = 512;

// shared memory, from a 1024-byte boundary
constexpr uint32_t kBox = 16384;  // 128 rows x 64 elements, 128-byte swizzled
constexpr uint32_t SM_C = 0, SM_B = 2 * kBox, SM_X = 4 * kBox, SM_STAGE = 6 * kBox;
constexpr uint32_t SM_M = kStages * SM_STAGE;           // columns i < 64: 128 rows; i >= 64: rows 64-127
constexpr uint32_t SM_GATE = SM_M + 24576;
constexpr uint32_t SM_GATE_STAGE = 2304;
constexpr uint32_t SM_IO = SM_GATE + kStages * SM_GATE_STAGE;  // an output warp's 512 bytes: 8 tokens x 32 columns
constexpr uint32_t SM_MISC = SM_IO + 4 * kOutGroups * 512;
constexpr uint32_t SM_TOTAL = SM_MISC + 464;
static_assert(SM_TOTAL <= 227 * 1024, "shared memory of the tensor form");
// A stage's gates, floats; log-decays are to the base 2.
constexpr uint32_t GT_COL = 0;      // M's column i: the sum of i's group of 4 tokens up to i, less log2 dt_i
constexpr uint32_t GT_ROW = 128;    // M's row t: the sum of t's group up to t
constexpr uint32_t GT_W = 256;      // w
constexpr uint32_t GT_E = 384;      // e^gamma_t
constexpr uint32_t GT_GROUP = 512;  // the sum of each of the 32 groups
constexpr uint32_t GT_FAR = 544;    // the sum from token 64 to each later group's start
constexpr uint32_t GT_WSCALE = 560, GT_DTSCALE = 561;  // 2^k of w and 2^j of dt (FP16)
constexpr uint32_t GT_SUM = 562;    // the sum of the chunk (PASS 1: and of those behind it)
// FP16, powers of two: what H^T was divided by, of each 32 columns of x, and M (dt's included),
// of each 32 tokens t
constexpr uint32_t GT_HSCALE = 564, GT_MSCALE = 568;
static_assert((GT_MSCALE + 4) * 4 <= SM_GATE_STAGE, "gates");

enum {
    B_FULL, B_XFULL = B_FULL + kMaxStages,  // B and C, and x, of a stage landed
    B_GATE = B_XFULL + kMaxStages,
    B_BCFREE = B_GATE + kMaxStages, B_EMPTY = B_BCFREE + kMaxStages,  // B and C, and x and the gates, are read
    B_H = B_EMPTY + kMaxStages,  // by stage: the state is rounded and decayed,
    B_M = B_H + kMaxStages,      // and each half of M formed (with the powers of two of both)
    B_G = B_M + 2 * kStages, B_GFREE, B_MFREE, B_HBFREE, B_S,
    B_Y1, B_Y1FREE = B_Y1 + 2,      // [2], by buffer
    B_Y2FREE = B_Y1FREE + 2,        // [2], by half
    B_XW = B_Y2FREE + 2,  // [8]
    B_XWFREE = B_XW + 8,
    B_TAIL = B_XWFREE + 8,
    B_INIT, B_FIN,
    NBAR
};
static_assert(kOutGroups >= 3, "the output warps bring the state's rows 32 .. 127");
static_assert(SM_MISC + NBAR * 8 + 16 <= SM_TOTAL, "barrier space");

__device__ int g_ssm_status;  // bits of kDevErr*

struct TcParams {
    CUtensorMap tm_x, tm_b, tm_c;  // [T][n_heads head_dim], [T][n_groups state_dim] twice; box 64 x 128
    CUtensorMap tm_z;              // as tm_x
    const void *a, *z;
    void* y;
    int64_t a_stride, z_stride, y_stride;
    const float *A_log, *dt_bias, *D;
    float* states;
    float* ws;        // [units][n_heads][state_dim][head_dim], or nullptr: no segments
    float* ws_decay;  // [units][n_heads]
    SsmSeqs q;
    int* status;
    int64_t units;    // the grid's: no fewer than the segments of disjoint sequences
    int seg;          // tokens per segment, a multiple of L
    int n_heads, n_groups;
};

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
__device__ __forceinline__ void tmem_st_u16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Fragments of a 16 x 16 tile, rows = columns of x (or lanes of tensor memory), columns =
// tokens: register k of the four holds tokens 8 (k >> 1) + 2 (lane & 3), + 1 of row
// (lane >> 2) + 8 (k & 1), 16 bits each (ldmatrix and stmatrix, transposed: in memory the
// rows are tokens); the FP32 loads give the same pairs in register pairs 2k, 2k + 1.
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 8 FP32 columns of 32 lanes of each of two accumulators, one wait: pair k of a result holds
// columns 2 (lane & 3), + 1 of row 8 k + (lane >> 2).
__device__ __forceinline__ void tmem_ld_frag(uint32_t a, uint32_t b, float2 (&va)[4], float2 (&vb)[4]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%16];\n"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%4,%5,%6,%7}, [%17];\n"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%8,%9,%10,%11}, [%18];\n"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%12,%13,%14,%15}, [%19];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
          "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15])
        : "r"(a), "r"(a + (16u << 16)), "r"(b), "r"(b + (16u << 16))
        : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        va[k] = make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
        vb[k] = make_float2(__uint_as_float(r[8 + 2 * k]), __uint_as_float(r[8 + 2 * k + 1]));
    }
}
// A 16-bit tile (16 lanes x 16 tokens) to 8 columns of tensor memory.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}
// Has box (x, y) fetched into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// ---- pairs of the 16-bit types ----
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The larger magnitudes of two pairs of FP16, with some sign (a NaN counts as none).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The power of two just above v, from 2^-60 (tensor memory holds the state times its inverse,
// in FP32: a state up to 2^67 stays finite there) to 2^24.
__device__ __forceinline__ float range_scale(float v) {
    int e = static_cast<int>((__float_as_uint(v) >> 23) & 255) - 126;
    e = e < -60 ? -60 : e > 24 ? 24 : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Arrivals that complete a phase of barrier b: one where a copy, a commit or the gate warp
// arrives, 4 where a role's warps do; a stage is free when the MMAs and every role that
// reads it are done.
__device__ constexpr int arrivals(int b, bool out) {
    if (b >= B_BCFREE && b < B_EMPTY) return out ? 2 : 1;
    if (b >= B_EMPTY && b < B_EMPTY + kMaxStages) return out ? 9 + 4 * kOutGroups : 16;
    if ((b >= B_H && b < B_M) || b == B_TAIL) return out ? 4 : 16;
    if (b == B_INIT) return 4 * kOutGroups;
    if ((b >= B_M && b < B_G) || b == B_GFREE) return 4;
    if (b >= B_Y1FREE && b < B_XW) return 4 * kOutGroups;
    if (b == B_FIN) return out ? 2 : 1;
    if (b >= B_XW && b < B_XWFREE) return out ? 4 : 16;
    return 1;
}

// (out of line: its 4 uses per lane would be most of the gate warp's code)
__device__ __noinline__ float softplus_call(float v) { return ssm_softplus(v); }

struct Sync {
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
// Waits for phase `n` (0, 1, ...) of a barrier.  False once some wait of the CTA gave up.
// (All but the first poll out of line: the code of all roles has to fit the caches.)
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
    for (uint32_t i = 0; i < kTcPolls; ++i) {
        if (poll(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    *abort_flag = 1;
    report_timeout(status);
    return false;
}
__device__ __forceinline__ bool wait_phase(const Sync& s, int b, uint32_t n) {
    return poll(&s.bar[b], n & 1) || wait_more(&s.bar[b], n & 1, s.abort_flag, s.status);
}
// The same for a whole warp: all lanes leave together, with one answer (the tensor-memory
// instructions behind a wait need a converged warp).
__device__ __forceinline__ bool wait_warp(const Sync& s, int b, uint32_t n) {
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
__device__ __forceinline__ void warp_arrive(const Sync& s, int b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.bar[b]);
}

// Where a lane's row of ldmatrix tile (lane >> 3) of the 16 columns from p0 and tokens 0-15
// lies in an x tile: token 8 (tile >> 1) + (lane & 7), columns p0 + 8 (tile & 1) .. + 7.
__device__ __forceinline__ uint32_t frag_offset(int p0, int lane) {
    const int p = p0 + 8 * ((lane >> 3) & 1), r = lane & 7;
    return (p >> 6) * kBox + (8 * (lane >> 4) + r) * 128 + ((((p & 63) >> 3) ^ r) << 4);
}

// The unit (sequence, segment) of a CTA, found by its sequences' segment counts.
struct Unit {
    int s, k, n_seg;      // sequence, segment of it, its segments
    int64_t begin;        // first row
    int len;              // rows
};
struct UnitScratch {  // shared memory of the search
    int64_t warp_sum[kThreadsTc / 32];
    int warp_seqs[kThreadsTc / 32];
    Unit found;
    int64_t found_u;
};
__device__ bool find_unit(const SsmSeqs& q, int seg, int64_t units, int64_t u, Unit* out, UnitScratch& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* warp_sum = sh.warp_seqs;
    Unit& found = sh.found;
    if (tid == 0) found.s = -1;
    int64_t base = 0;
    for (int s0 = 0; s0 < q.n_seq; s0 += kThreadsTc) {
        int64_t b = 0, e = 0;
        if (s0 + tid < q.n_seq) seq_rows(q, s0 + tid, b, e);
        const int n = static_cast<int>((e - b + seg - 1) / seg);
        int inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int64_t before = base;
        int total = 0;
        for (int w = 0; w < kThreadsTc / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            total += warp_sum[w];
        }
        const int64_t first = before + inc - n;
        // (a sequence whose segments pass the grid's end, as overlapping bounds may give, is left out)
        if (u >= first && u < first + n && first + n <= units) {
            const int k = static_cast<int>(u - first);
            found.s = s0 + tid;
            found.k = k;
            found.n_seg = n;
            found.begin = b + static_cast<int64_t>(k) * seg;
            found.len = static_cast<int>(e - found.begin < seg ? e - found.begin : seg);
        }
        base += total;
        __syncthreads();
        if (base > u) break;  // uniform
    }
    __syncthreads();
    *out = found;
    return found.s >= 0;
}

// The same for unit v of the segments that are not their sequence's last; *u: its number among all.
__device__ bool find_inner_unit(const SsmSeqs& q, int seg, int64_t units, int64_t v, int64_t* u, Unit* out,
                                UnitScratch& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreadsTc / 32;
    int64_t* warp_sum = sh.warp_sum;
    int* warp_seqs = sh.warp_seqs;
    Unit& found = sh.found;
    int64_t& found_u = sh.found_u;
    if (tid == 0) found.s = -1;
    int64_t base = 0, seqs = 0;  // segments, and sequences that have some
    for (int s0 = 0; s0 < q.n_seq; s0 += kThreadsTc) {
        int64_t b = 0, e = 0;
        if (s0 + tid < q.n_seq) seq_rows(q, s0 + tid, b, e);
        const int n = static_cast<int>((e - b + seg - 1) / seg);
        const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
        int64_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t w = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += w;
        }
        if (lane == 31) {
            warp_sum[warp] = inc;
            warp_seqs[warp] = __popc(some);
        }
        __syncthreads();
        int64_t first = base + inc - n, inner = -seqs - __popc(some & ((1u << lane) - 1));
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                first += warp_sum[w];
                inner -= warp_seqs[w];
            }
            base += warp_sum[w];
            seqs += warp_seqs[w];
        }
        inner += first;  // those before that are not last ones
        if (v >= inner && v < inner + n - 1 && first + n <= units) {
            const int k = static_cast<int>(v - inner);
            found.s = s0 + tid;
            found.k = k;
            found.n_seg = n;
            found.begin = b + static_cast<int64_t>(k) * seg;
            found.len = seg;
            found_u = first + k;
        }
        __syncthreads();
        if (base - seqs > v) break;  // uniform
    }
    __syncthreads();
    *out = found;
    *u = found_u;
    return found.s >= 0;
}

// PASS 0: outputs (and final states); PASS 1: the segments' contributions.
template <bool BF16, int P, int N, int PASS>
__global__ void __launch_bounds__(kThreadsTc, 1) ssm_scan_tc_kernel(const __grid_constant__ TcParams p) {
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int PARTS = BF16 ? 3 : 2;
    constexpr bool OUT = PASS == 0;
    // PASS 1 goes through a segment from its last chunk, w with the decay to the segment's end: the
    // sum needs no decay between chunks (for FP16 a change of its power of two).
    constexpr bool kStepped = OUT || !BF16;
    // PASS 1 has tensor memory for two chunks' parts, and 16 warps to form them
    constexpr int SLOTS = OUT ? 64 / (8 * PARTS) : 16;
    constexpr uint32_t TM_PARTS = OUT ? TM_XW : TM_HB;
    constexpr int X_FIRST = OUT ? 1 : 0, X_GROUPS = OUT ? 1 : 4;
    constexpr int GROUP = OUT ? 1 : 4;  // blocks whose parts share a barrier
    constexpr int NB = N / 64, PB = P / 64;
    // the stages: PASS 1 has no C, and room for three (its gates lie where M is else)
    constexpr int STAGES = OUT ? kStages : 3;
    constexpr uint32_t STAGE_BYTES = OUT ? SM_STAGE : 4 * kBox, B_AT = OUT ? SM_B : 0, X_AT = OUT ? SM_X : 2 * kBox;
    constexpr uint32_t GATE_AT = OUT ? SM_GATE : SM_M;
    static_assert(STAGES <= kMaxStages && 3 * 4 * kBox <= SM_M, "stages");
    // (all of the SM's shared memory is used, so there is none to round the address up in: the
    // kernel has no other, and its start is a multiple of 1024 as declared, or it gives up)
    extern __shared__ __align__(1024) unsigned char ssm_tc_smem[];
    unsigned char* sm = ssm_tc_smem;
    if (smem_addr(sm) % 1024 != 0) {
        if (threadIdx.x == 0) report_error(p.status, kDevErrLayout);
        return;
    }
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SM_MISC + NBAR * 8);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + SM_MISC + NBAR * 8 + 8);
    UnitScratch& scratch = *reinterpret_cast<UnitScratch*>(sm + GATE_AT);  // before the gates are written
    const Sync sy{bar, abort_flag, p.status};
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    const int h = blockIdx.x % p.n_heads;
    int64_t u = blockIdx.x / p.n_heads;
    Unit un;
    if constexpr (OUT) {
        if (!find_unit(p.q, p.seg, p.units, u, &un, scratch)) return;
    } else {  // (nothing reads a last segment's contribution)
        if (!find_inner_unit(p.q, p.seg, p.units, u, &u, &un, scratch)) return;
    }
    if constexpr (PASS == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int g = h % p.n_groups;
    const int nch = (un.len + L - 1) / L;

    if (tid == 0) {
#pragma unroll
        for (int b = 0; b < NBAR; ++b) mbar_init(&bar[b], arrivals(b, OUT));
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, TM_COLS);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // Rows n0 .. + 31 of the state before the segment, columns 32 wq + lane, to tensor memory.
    auto init_state = [&](int wq, int n0) {
        if constexpr (OUT) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the first launch's stores
        const int slot = p.states ? seq_slot(p.q, un.s) : -1, pcol = wq * 32 + lane;
        const bool from_ws = OUT && un.n_seg > 1;
        const bool old = !from_ws && un.k == 0 && slot >= 0 && seq_has_state(p.q, un.s);
        const int64_t unit_floats = static_cast<int64_t>(p.n_heads) * N * P;
        float* first = p.ws + ((u - un.k) * p.n_heads + h) * N * P + static_cast<int64_t>(n0) * P + pcol;  // segment 0's contribution
        float* kept = first + (un.n_seg - 1) * unit_floats;  // the state before the sequence, left by PASS 1
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
        if (old) {
            const float* src = p.states + ((static_cast<int64_t>(slot) * p.n_heads + h) * N + n0) * P + pcol;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = src[i * P];
        } else if (from_ws && un.k == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = kept[i * P];
        } else if (from_ws) {
            float keep = 1.f;
            for (int k = un.k - 1; k >= 0; --k) {
                const float* src = first + k * unit_floats;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(keep, src[i * P], v[i]);
                keep *= p.ws_decay[(u - un.k + k) * p.n_heads + h];
            }
        }
        if (PASS == 1 && un.k == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                kept[i * P] = v[i];
                v[i] = 0.f;
            }
        }
        if (kStepped) tmem_st32(tm + (static_cast<uint32_t>(wq * 32) << 16) + TM_H + n0, v);  // (else the first MMA sets it)
    };

    if (warp == kCopyWarp) {
        if (elect_one()) {
            // B and C are free earlier than x (whose last reader is the output); what is to come is
            // fetched into L2 two chunks ahead, as is z, which the output reads itself
            auto rows = [&](const CUtensorMap* map, int x0, int boxes, int row, unsigned char* dst, int b) {
                for (int i = 0; i < boxes; ++i) {
                    if (dst) tma_load_2d(dst + i * kBox, map, &bar[b], x0 + 64 * i, row);
                    else tma_prefetch_2d(map, x0 + 64 * i, row);
                }
            };
            const int row0 = static_cast<int>(un.begin);
            int bc = 0, xc = 0;
            for (int c = 0; c < nch; ++c) {
                const int s = c % STAGES, row = row0 + (OUT ? c : nch - 1 - c) * L, ahead = OUT ? row + STAGES * L : row - STAGES * L;
                unsigned char* st = sm + s * STAGE_BYTES;
                if (c + STAGES < nch) {
                    rows(&p.tm_b, g * N, NB, ahead, nullptr, 0);
                    if (OUT) rows(&p.tm_c, g * N, NB, ahead, nullptr, 0);
                    rows(&p.tm_x, h * P, PB, ahead, nullptr, 0);
                }
                if (OUT && p.z) rows(&p.tm_z, h * P, PB, row, nullptr, 0);
                auto bc_rows = [&]() {
                    if (c >= STAGES && !wait_phase(sy, B_BCFREE + s, c / STAGES - 1)) return false;
                    mbar_arrive_expect_tx(&bar[B_FULL + s], (OUT ? 2 : 1) * NB * kBox);
                    rows(&p.tm_b, g * N, NB, row, st + B_AT, B_FULL + s);
                    if (OUT) rows(&p.tm_c, g * N, NB, row, st + SM_C, B_FULL + s);
                    ++bc;
                    return true;
                };
                // (in the order in which they are freed)
                if (OUT && !bc_rows()) break;
                if (c >= STAGES && !wait_phase(sy, B_EMPTY + s, c / STAGES - 1)) break;
                mbar_arrive_expect_tx(&bar[B_XFULL + s], PB * kBox);
                rows(&p.tm_x, h * P, PB, row, st + X_AT, B_XFULL + s);
                ++xc;
                if (!OUT && !bc_rows()) break;
            }
            // the copies in flight land before the CTA ends, also after a wait that gave up
            for (int i = bc > STAGES ? bc - STAGES : 0; i < bc; ++i) land(&bar[B_FULL + i % STAGES], i / STAGES);
            for (int i = xc > STAGES ? xc - STAGES : 0; i < xc; ++i) land(&bar[B_XFULL + i % STAGES], i / STAGES);
        }
    } else if (OUT && warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t ID_G = idesc_f16(BF16, 128, 64, false, false);   // C, B: K-major
            constexpr uint32_t ID_Y1 = idesc_f16(BF16, 128, 32, true, false);   // x^T: M-major
            constexpr uint32_t ID_Y2 = idesc_f16(BF16, 128, 64, false, false);
            const uint32_t sm0 = smem_addr(sm);
            uint32_t gi = 0, yi = 0;
            auto issue_g = [&](int c, int half) {  // G's columns of tokens 64 half .. +63
                if (gi > 0 && !wait_phase(sy, B_GFREE, gi - 1)) return false;
                tc_fence_after_sync();
                const uint32_t st = sm0 + (c % STAGES) * STAGE_BYTES;
                uint64_t dc = desc_k(st + SM_C), db = desc_k(st + B_AT + half * 8192);
#pragma unroll 1
                for (int k = 0; k < N / 64; ++k, dc += kBox >> 4, db += kBox >> 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_ss(tm + TM_G, dc + 2 * j, db + 2 * j, ID_G, j > 0 || k > 0);
                umma_commit(&bar[B_G]);
                ++gi;
                return true;
            };
            auto issue_y1 = [&](int c, int q) {  // tokens t of quarter q, from tokens i up to its end
                if ((q & 1) == 0 && !wait_phase(sy, B_M + 2 * (c % STAGES) + (q >> 1), c / STAGES)) return false;
                if (yi > 1 && !wait_phase(sy, B_Y1FREE + (q & 1), (yi >> 1) - 1)) return false;
                tc_fence_after_sync();
                uint64_t dx = desc_mn(sm0 + (c % STAGES) * STAGE_BYTES + X_AT), dm = desc_k(sm0 + SM_M + q * 4096);
                const uint32_t d = tm + TM_Y1 + 32 * (q & 1);
#pragma unroll 1
                for (int k = 0; k <= q; ++k, dx += 256) {  // 32 tokens i; the second 64 in the other part of M
                    mma_ss(d, dx, dm, ID_Y1, k > 0);
                    mma_ss(d, dx + 128, dm + 2, ID_Y1, true);
                    dm += k == 1 ? ((kBox - 8192) >> 4) - 4 : 4;
                }
                umma_commit(&bar[B_Y1 + (q & 1)]);
                ++yi;
                return true;
            };
            auto issue_y2 = [&](int c, int half) {
                if (c > 0 && !wait_phase(sy, B_Y2FREE + half, c - 1)) return false;
                tc_fence_after_sync();
                uint64_t dc = desc_k(sm0 + (c % STAGES) * STAGE_BYTES + SM_C + half * 8192);
#pragma unroll 1
                for (int k = 0; k < N / 64; ++k, dc += kBox >> 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_ts(tm + TM_Y2 + 64 * half, tm + TM_HB + 32 * k + 8 * j, dc + 2 * j, ID_Y2, j > 0 || k > 0);
                return true;
            };
            // Order: H^T C^T, a quarter of Y1, the second half of G, a quarter of Y1, and again with the
            // next chunk's first half of G: what a quarter of the output needs while the one before
            // is read.  (A loop over the halves: the code of all roles
            // has to fit the instruction caches.)
            bool ok = wait_phase(sy, B_FULL, 0) && issue_g(0, 0);
#pragma unroll 1
            for (int n = 0; ok && n < 2 * nch; ++n) {
                const int c = n >> 1, half = n & 1, next = c + half;
                // (the state's rounding, B_H, comes after the zeroing of a last chunk's rows)
                if (half == 0) ok = wait_phase(sy, B_XFULL + c % STAGES, c / STAGES) && wait_phase(sy, B_H + c % STAGES, c / STAGES);
                ok = ok && issue_y2(c, half);
                if (!ok) break;
                if (half) {
                    umma_commit(&bar[B_HBFREE]);
                    umma_commit(&bar[B_BCFREE + c % STAGES]);
                }
                ok = issue_y1(c, 2 * half);
                if (ok && next < nch) {
                    if (half) ok = wait_phase(sy, B_FULL + next % STAGES, next / STAGES);
                    ok = ok && issue_g(next, half ^ 1);
                }
                ok = ok && issue_y1(c, 2 * half + 1);
                if (half && ok) {
                    umma_commit(&bar[B_MFREE]);
                    umma_commit(&bar[B_EMPTY + c % STAGES]);
                }
            }
            finish_mma(&bar[B_FIN]);
        }
    } else if (warp == kStateMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t ID_S = idesc_f16(BF16, 128, N, false, true);     // B: N-major
            const uint32_t sm0 = smem_addr(sm);
            bool ok = true;
            for (int c = 0; ok && c < nch; ++c) {
                const int s = c % STAGES;
                if (!wait_phase(sy, B_FULL + s, c / STAGES) || (kStepped && !wait_phase(sy, B_H + s, c / STAGES))) break;
#pragma unroll 1
                for (int j = 0; j < L / 16; j += GROUP) {  // GROUP blocks to a barrier
                    const uint32_t group = (c * (L / 16) + j) / GROUP, slot = group % (SLOTS / GROUP);
                    ok = wait_phase(sy, B_XW + slot, group / (SLOTS / GROUP));
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int i = 0; i < GROUP; ++i) {
                        const uint64_t b = desc_mn(sm0 + s * STAGE_BYTES + B_AT + (j + i) * 2048);
#pragma unroll
                        for (int q = 0; q < PARTS; ++q)
                            mma_ts(tm + TM_H, tm + TM_PARTS + ((slot * GROUP + i) * PARTS + q) * 8, b, ID_S,
                                   kStepped || group > 0 || i > 0 || q > 0);
                    }
                    umma_commit(&bar[B_XWFREE + slot]);
                }
                if (!ok) break;
                if (kStepped || c == nch - 1) umma_commit(&bar[B_S]);
                umma_commit(&bar[B_BCFREE + s]);
            }
            finish_mma(&bar[B_FIN]);
        }
    } else if (warp == kGateWarp || (!OUT && warp == kMmaWarp)) {
        const float A = ssm_rate(__ldg(p.A_log + h)), bias = __ldg(p.dt_bias + h);
        const T* a = static_cast<const T*>(p.a) + un.begin * p.a_stride + h;
        // PASS 1 has two gate warps, a chunk each in turn; they hand on the sum of the decays behind
        constexpr int GATES = OUT ? 1 : 2;
        for (int c = warp != kGateWarp ? 1 : 0; c < nch; c += GATES) {
            const int s = c % STAGES, chunk = OUT ? c : nch - 1 - c;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = chunk * L + 4 * lane + i;
                v[i] = t < un.len ? to_f<T>(a[t * p.a_stride]) : 0.f;
            }
            if (c >= STAGES && !wait_warp(sy, B_EMPTY + s, c / STAGES - 1)) break;
            float dt[4], g2[4], pre[4], suf[4];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool live = chunk * L + 4 * lane + i < un.len;
                dt[i] = live ? (OUT ? softplus_call(v[i] + bias) : ssm_softplus(v[i] + bias)) : 0.f;
                g2[i] = fmaxf(A * dt[i] * kLog2e, kMinLog2Decay);
                sum += g2[i];
                pre[i] = sum;
            }
            float up = sum, down = sum;  // inclusive sums over the lanes, from the half's start and the end
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float y = __shfl_down_sync(0xffffffffu, down, off);
                if (lane + off < 32) down += y;
                if (OUT && off < 16) {
                    const float x = __shfl_up_sync(0xffffffffu, up, off);
                    if ((lane & 15) >= off) up += x;
                }
            }
            const float first_half = __shfl_sync(0xffffffffu, up, 15);
            up = __shfl_up_sync(0xffffffffu, up, 1);
            down = __shfl_down_sync(0xffffffffu, down, 1);
            if ((lane & 15) == 0) up = 0.f;
            if (lane == 31) down = 0.f;
            float behind = 0.f;  // (PASS 1) the sum over the segment's chunks behind this one
            if (!OUT && c > 0) {
                if (!wait_warp(sy, B_GATE + (c - 1) % STAGES, (c - 1) / STAGES)) break;
                behind = reinterpret_cast<const float*>(sm + GATE_AT + (c - 1) % STAGES * SM_GATE_STAGE)[GT_SUM];
            }
            float after = down + behind;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                suf[i] = after;
                after += g2[i];
            }
            float* gt = reinterpret_cast<float*>(sm + GATE_AT + s * SM_GATE_STAGE);
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = dt[i] * ex2(suf[i]);
            if constexpr (!BF16) {
                float wm = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), dm = fmaxf(fmaxf(dt[0], dt[1]), fmaxf(dt[2], dt[3]));
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, off));
                    dm = fmaxf(dm, __shfl_xor_sync(0xffffffffu, dm, off));
                }
                const float ws = range_scale(wm), ds = range_scale(dm);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] *= 1.0f / ws;  // powers of two: exact
                    dt[i] *= 1.0f / ds;
                }
                if (lane == 0) {
                    gt[GT_WSCALE] = ws;
                    gt[GT_DTSCALE] = ds;
                }
            }
            if constexpr (OUT) {
                float col[4], e[4];
                const float before = lane < 16 ? up : first_half + up;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    col[i] = pre[i] - lg2(dt[i]);  // (no step: infinity, a factor of 0)
                    e[i] = ex2(before + pre[i]);
                }
                reinterpret_cast<float4*>(gt + GT_COL)[lane] = make_float4(col[0], col[1], col[2], col[3]);
                reinterpret_cast<float4*>(gt + GT_ROW)[lane] = make_float4(pre[0], pre[1], pre[2], pre[3]);
                reinterpret_cast<float4*>(gt + GT_E)[lane] = make_float4(e[0], e[1], e[2], e[3]);
                gt[GT_GROUP + lane] = sum;
                if (lane >= 16) gt[GT_FAR + lane - 16] = up;
            } else if (lane == 0) {
                gt[GT_SUM] = after;  // with this chunk's
            }
            reinterpret_cast<float4*>(gt + GT_W)[lane] = make_float4(w[0], w[1], w[2], w[3]);
            warp_arrive(sy, B_GATE + s);
        }
    } else if (OUT && warp < 4) {
        if constexpr (OUT) {
            // ---- M: lane = token t ----
            const int t = tid;
            const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
            unsigned char* m0 = sm + SM_M + t * 128;                   // columns 0-63 (no product reads past
            unsigned char* m1 = sm + SM_M + kBox + (t - 64) * 128;     // the diagonal block), 64-127 (t >= 64)
            uint32_t gi = 0;
            for (int c = 0; c < nch; ++c) {
                const int s = c % STAGES;
                if (!wait_warp(sy, B_GATE + s, c / STAGES)) break;
                float* gd = reinterpret_cast<float*>(sm + GATE_AT + s * SM_GATE_STAGE);
                const float row = gd[GT_ROW + t];
                int shift = 0;          // (FP16) the scores of the warp's rows are formed times 2^shift
                bool hopeless = false;  // (FP16) this row has an infinite score
                bool ok = true;
#pragma unroll 1
                for (int half = 0; half < 2; ++half, ++gi) {
                    ok = wait_warp(sy, B_G, gi) && (half || c == 0 || wait_warp(sy, B_MFREE, c - 1));
                    if (!ok) break;
                    tc_fence_after_sync();
                    unsigned char* m = half ? m1 : m0;
                    // 16 columns at a time, up to the block of 32 on the diagonal
                    const bool far = half == 0 && warp >= 2;
                    const int stop = far ? 64 : 32 * (warp + 1) - 64 * half;
                    const int first_shift = shift;
                    bool again = false;
                    do {
                        uint32_t largest = 0;  // (FP16) the row's largest magnitudes, a pair
                        // the sum from a group's start to t, group after group from t's own down
                        float base = far ? row + gd[GT_FAR + t / 4 - 16] : row;
                        if constexpr (!BF16) base += static_cast<float>(shift);
#pragma unroll 1
                        for (int j0 = stop - 16; j0 >= 0; j0 -= 16) {
                            float v[16];
                            tmem_ld16(tm + lanes + TM_G + j0, v);
                            const int above = t - 64 * half - j0;  // columns past it are above the diagonal
                            const float4* c4 = reinterpret_cast<const float4*>(gd + GT_COL + 64 * half + j0);
                            const float4 sums = *reinterpret_cast<const float4*>(gd + GT_GROUP + 16 * half + j0 / 4);
                            uint32_t o[8];
#pragma unroll
                            for (int k = 3; k >= 0; --k) {
                                const float4 c = c4[k];
                                if (k < above >> 2) base += k == 3 ? sums.w : k == 2 ? sums.z : k == 1 ? sums.y : sums.x;
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int j = 4 * k + 2 * i;
                                    const float2 d = ffma2(i ? make_float2(c.z, c.w) : make_float2(c.x, c.y),
                                                           make_float2(-1.f, -1.f), make_float2(base, base));
                                    const float2 a = fmul2(make_float2(ex2(d.x), ex2(d.y)), make_float2(v[j], v[j + 1]));
                                    // selected, not multiplied: what is above may be anything
                                    o[j / 2] = pack2<BF16>(j > above ? 0.f : a.x, j + 1 > above ? 0.f : a.y);
                                    if constexpr (!BF16) largest = max_abs2(largest, o[j / 2]);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                *reinterpret_cast<uint4*>(m + (((j0 / 8 + i) ^ (t & 7)) << 4)) =
                                    make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                        if constexpr (!BF16) {
                            // Scores above the range (C . B is) came out infinite: the warp's are formed again, a
                            // 16th as large, until none is (C . B < 2^40: 7 times at most); a row with an
                            // infinite C . B does not count in that.
                            const bool over = !hopeless && ((largest & 0x7fff) == 0x7c00 || (largest >> 16 & 0x7fff) == 0x7c00);
                            again = __any_sync(0xffffffffu, over) != 0;
                            if (again && shift > first_shift - 28) {
                                shift -= 4;
                            } else if (again) {
                                shift = first_shift;
                                hopeless |= over;
                            }
                        }
                    } while (again);
                    if constexpr (!BF16) {
                        if (half && shift != first_shift) {  // the first half's columns follow
                            const float f = pow2(shift - first_shift);
#pragma unroll 1
                            for (int i = 0; i < 32; ++i) {
                                uint32_t* at = reinterpret_cast<uint32_t*>(m0) + i;
                                const float2 v = unpack2<BF16>(*at);
                                *at = pack2<BF16>(v.x * f, v.y * f);
                            }
                        }
                        if (warp / 2 == half && lane == 0) gd[GT_MSCALE + warp] = gd[GT_DTSCALE] * pow2(-shift);
                    }
                    tc_fence_before_sync();
                    warp_arrive(sy, B_GFREE);
                    fence_async_smem();
                    warp_arrive(sy, B_M + 2 * s + half);
                }
                if (!ok) break;
                warp_arrive(sy, B_EMPTY + s);
            }
        }
    } else if (warp < 4 * (X_FIRST + X_GROUPS)) {
        // ---- the state, and the parts of w o x: X_GROUPS groups of 4 warps, lane = column pcol of x.
        // Group xg takes every X_GROUPS-th block of 16 tokens and the state rows n0, n0 + 32 X_GROUPS, .. ----
        const int wq = warp & 3, xg = (warp >> 2) - X_FIRST, pcol = wq * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const bool live = wq * 32 < P;  // uniform in a warp
        const int slot = p.states ? seq_slot(p.q, un.s) : -1;
        float* pool = p.states + (static_cast<int64_t>(slot) * p.n_heads + h) * N * P + pcol;
        if (live) {
#pragma unroll 1
            for (int n0 = 32 * xg; n0 < (OUT ? 32 : N); n0 += 32 * X_GROUPS) init_state(wq, n0);
            tmem_wait_st();
        }
        const uint32_t x_frag = frag_offset(wq * 32, lane), x_frag1 = frag_offset(wq * 32 + 16, lane);
        bool ok = true;
        float scale = 1.f;  // tensor memory holds H / scale
        for (int c = 0; ok && c < nch; ++c) {
            const int s = c % STAGES;
            unsigned char* st = sm + s * STAGE_BYTES;
            float* gt = reinterpret_cast<float*>(sm + GATE_AT + s * SM_GATE_STAGE);
            if (!wait_warp(sy, B_GATE + s, c / STAGES)) break;
            if (!wait_warp(sy, B_XFULL + s, c / STAGES)) break;
            // (PASS 1 has whole chunks alone: a sequence's last segment is not its)
            const int nv = OUT ? un.len - c * L : L;
            if (OUT && nv < L) {
                if (!wait_warp(sy, B_FULL + s, c / STAGES)) break;
                // rows behind the segment's end (another sequence's, which may hold anything) become
                // zeros in x and B, the operands whose rows are summed over
                for (int i = tid - 128 * X_FIRST; i < (L - nv) * 8; i += 128 * X_GROUPS) {
                    const uint32_t off = (nv + i / 8) * 128 + (i % 8) * 16;
#pragma unroll
                    for (int k = 0; k < PB; ++k) *reinterpret_cast<uint4*>(st + X_AT + k * kBox + off) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < NB; ++k) *reinterpret_cast<uint4*>(st + B_AT + k * kBox + off) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                warp_arrive(sy, B_TAIL);
                if (!wait_warp(sy, B_TAIL, 0)) break;
            }
            const float next_scale = BF16 ? 1.f : gt[GT_WSCALE];
            // the state's decay, and its rounding for the product with C
            auto state_step = [&]() {
                if (OUT && c == 0 && !wait_warp(sy, B_INIT, 0)) return false;
                if (c > 0 && (!wait_warp(sy, B_S, c - 1) || (OUT && !wait_warp(sy, B_HBFREE, c - 1)))) return false;
                tc_fence_after_sync();
                if (live) {
                    const float keep = (OUT ? gt[GT_E + L - 1] : 1.f) * (scale * (1.0f / next_scale));
                    float round_by = 1.f;  // (FP16) a power of two that brings the warp's largest below 2^15
                    if constexpr (OUT && !BF16) {
                        float most = 0.f;
#pragma unroll 1
                        for (int n0 = 0; n0 < N; n0 += 32) {
                            float v[32];
                            tmem_ld32(tm + lanes + TM_H + n0, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) most = fmaxf(most, fabsf(v[i]));
                        }
                        if (!(most < INFINITY)) most = 0.f;  // (of a column with an infinite element the rest does not count)
#pragma unroll
                        for (int off = 1; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                        // the power's exponent, and the scale's: both powers and their quotient in FP32's range
                        const int es = static_cast<int>(__float_as_uint(scale) >> 23) - 127;
                        int e = static_cast<int>(__float_as_uint(most) >> 23) - 126;
                        e = max(e, max(-110, -110 - es));
                        e = min(e, 142 - es);
                        round_by = pow2(15 - e);
                        if (lane == 0) gt[GT_HSCALE + wq] = pow2(es + e - 15);
                    }
#pragma unroll 1
                    for (int n0 = 32 * xg; n0 < N; n0 += 32 * X_GROUPS) {
                        float v[32];
                        tmem_ld32(tm + lanes + TM_H + n0, v);
                        if constexpr (OUT) {
                            uint32_t o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = BF16 ? pack2<BF16>(v[2 * i], v[2 * i + 1])
                                            : pack2<BF16>(v[2 * i] * round_by, v[2 * i + 1] * round_by);
                            tmem_st_u16(tm + lanes + TM_HB + n0 / 2, o);
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 d = fmul2(make_float2(v[i], v[i + 1]), make_float2(keep, keep));
                            v[i] = d.x;
                            v[i + 1] = d.y;
                        }
                        tmem_st32(tm + lanes + TM_H + n0, v);
                    }
                    tmem_wait_st();
                }
                scale = next_scale;
                tc_fence_before_sync();
                warp_arrive(sy, B_H + s);
                return true;
            };
            // with few slots the state goes first, with many the parts (they then wait for no update)
            if (OUT && !state_step()) break;
            // (PASS 1: a warp's two blocks of a chunk, unrolled: 32768 tokens 496 us, rolled 514)
#pragma unroll (OUT ? 1 : 2)
            for (int j = xg; j < L / 16; j += X_GROUPS) {
                // the parts are formed before the wait for their slot
                uint32_t part[2][PARTS][4];
                if (live) {
                    const uint32_t x = smem_addr(st) + X_AT + j * 2048;
                    const float2 w0 = *reinterpret_cast<const float2*>(gt + GT_W + 16 * j + 2 * (lane & 3));
                    const float2 w1 = *reinterpret_cast<const float2*>(gt + GT_W + 16 * j + 8 + 2 * (lane & 3));
#pragma unroll
                    for (int g2 = 0; g2 < 2; ++g2) {
                        uint32_t xr[4];
                        ldsm4t(x + (g2 ? x_frag1 : x_frag), xr);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float2 f = fmul2(unpack2<BF16>(xr[k]), k < 2 ? w0 : w1);
#pragma unroll
                            for (int q = 0; q < PARTS; ++q) {
                                part[g2][q][k] = pack2<BF16>(f.x, f.y);
                                const float2 back = unpack2<BF16>(part[g2][q][k]);
                                f = ffma2(back, make_float2(-1.f, -1.f), f);
                            }
                        }
                    }
                }
                const uint32_t blk = c * (L / 16) + j, xs = blk % SLOTS, xb = xs / GROUP;
                if (blk >= SLOTS && !wait_warp(sy, B_XWFREE + xb, blk / SLOTS - 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                if (live) {
#pragma unroll
                    for (int g2 = 0; g2 < 2; ++g2)
#pragma unroll
                        for (int q = 0; q < PARTS; ++q)
                            tmem_st_frag(tm + lanes + (g2 << 20) + TM_PARTS + (xs * PARTS + q) * 8, part[g2][q]);
                    tmem_wait_st();
                }
                tc_fence_before_sync();
                warp_arrive(sy, B_XW + xb);
            }
            if (!ok || (!OUT && kStepped && !state_step())) {
                ok = false;
                break;
            }
            warp_arrive(sy, B_EMPTY + s);
        }
        // the state behind the segment
        const bool keep_it = PASS == 1 || (slot >= 0 && un.k == un.n_seg - 1);
        if (ok && keep_it && wait_warp(sy, B_S, kStepped ? nch - 1 : 0)) {
            tc_fence_after_sync();
            float* dst = PASS == 1 ? p.ws + (u * p.n_heads + h) * N * P + pcol : pool;
            // (PASS 1) a first segment's includes the state before it, with the segment's decay
            const float* before = PASS == 1 && un.k == 0 ? dst + (un.n_seg - 1) * static_cast<int64_t>(p.n_heads) * N * P : nullptr;
            const float* last_gates = reinterpret_cast<const float*>(sm + GATE_AT + (nch - 1) % STAGES * SM_GATE_STAGE);
            const float decay = PASS == 1 ? exp2f(last_gates[GT_SUM]) : 0.f;
            if (PASS == 1 && tid == 0) p.ws_decay[u * p.n_heads + h] = decay;
            if (live) {
#pragma unroll 1
                for (int n0 = 32 * xg; n0 < N; n0 += 32 * X_GROUPS) {
                    float v[32];
                    tmem_ld32(tm + lanes + TM_H + n0, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] *= scale;
                        if (before) v[i] = fmaf(decay, before[static_cast<int64_t>(n0 + i) * P], v[i]);
                        dst[static_cast<int64_t>(n0 + i) * P] = v[i];
                    }
                }
            }
        }
        tc_fence_before_sync();
    } else if (warp < 8 + 4 * kOutGroups) {
        if constexpr (OUT) {
            // ---- the output: this warp's 32 columns of x, every kOutGroups-th block of 8 tokens ----
            const int wq = warp & 3, og = (warp - 8) >> 2;
            // the state's rows from 32 on, beside the state's own warps
            if (wq * 32 < P && 32 * (og + 1) < N) {
                init_state(wq, 32 * (og + 1));
                tmem_wait_st();
            }
            tc_fence_before_sync();
            warp_arrive(sy, B_INIT);
            const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
            const bool live = wq * 32 < P;
            const float D = p.D ? __ldg(p.D + h) : 0.f;
            const bool gated = p.z != nullptr;
            const int pf = wq * 32 + 8 * (lane >> 3), r8 = lane & 7;  // this lane's row of an 8 x 32 tile's ldmatrix
            const uint32_t x_frag = (pf >> 6) * kBox + r8 * 128 + ((((pf & 63) >> 3) ^ r8) << 4);
            // The warp's buffer holds 8 tokens x 32 columns, 64 bytes a token, 16-byte pieces swizzled;
            // global memory is read and written in pieces, this lane's piece lane & 3 of token lane >> 2.
            const uint32_t io = smem_addr(sm) + SM_IO + (warp - 8) * 512;
            auto piece = [](int t, int c) { return static_cast<uint32_t>(t * 64 + ((c ^ ((t >> 1) & 3)) << 4)); };
            const int pt = lane >> 2;
            const uint32_t io_piece = io + piece(pt, lane & 3), io_frag = io + piece(r8, lane >> 3);
            const int64_t col = static_cast<int64_t>(h) * P + wq * 32 + 8 * (lane & 3);
            const T* zp = gated ? static_cast<const T*>(p.z) + (un.begin + 8 * og + pt) * p.z_stride + col : nullptr;
            T* yp = static_cast<T*>(p.y) + (un.begin + 8 * og + pt) * p.y_stride + col;
            const int64_t z_step = 8 * kOutGroups * p.z_stride, y_step = 8 * kOutGroups * p.y_stride;
            int z_left = un.len - 8 * og - pt;  // rows from the next load's on
            // This warp's blocks of 8 tokens are og, og + kOutGroups, ..  A block's gates are formed in
            // the step before its own, and its z is loaded in the one before that (from L2, where
            // the copy warp has it fetched with the chunk's other operands).
            uint4 zq = {};
            auto load_z = [&]() {
                if (z_left > 0) zq = __ldcs(reinterpret_cast<const uint4*>(zp));
                z_left -= 8 * kOutGroups;
                zp += z_step;
            };
            uint32_t zr[4] = {};
            float2 gz[4];
            auto next_z = [&]() {  // the next block's z as a fragment
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(io_piece), "r"(zq.x), "r"(zq.y), "r"(zq.z), "r"(zq.w)
                             : "memory");
                __syncwarp();
                ldsm4t(io_frag, zr);
            };
            auto gates = [&]() {
#pragma unroll
                for (int k = 0; k < 4; ++k) gz[k] = silu2(unpack2<BF16>(zr[k]));
            };
            int b = og;  // the next block
            if (gated && live) {
                load_z();
                next_z();
                load_z();
                gates();
                __syncwarp();
            }
            bool ok = true;
            for (int c = 0; ok && c < nch; ++c) {
                const int s = c % STAGES;
                const uint32_t x = smem_addr(sm) + s * STAGE_BYTES + X_AT + x_frag;
                const float* gt = reinterpret_cast<const float*>(sm + GATE_AT + s * SM_GATE_STAGE);
                // (behind it are the state's warps' own waits for the gates and for x)
                if (!wait_warp(sy, B_H + s, c / STAGES)) break;
                const int nv = un.len - c * L;
                const float h_scale = BF16 ? 1.f : gt[GT_HSCALE + wq];
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    ok = wait_warp(sy, B_Y1 + (q & 1), 2 * c + (q >> 1)) &&
                         (BF16 || (q & 1) || wait_warp(sy, B_M + 2 * s + (q >> 1), c / STAGES));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const float m_scale = BF16 ? 1.f : gt[GT_MSCALE + q];
                    // (a rolled loop: the code of all roles has to fit the instruction caches; a step's
                    // loads come first, so that its arithmetic overlaps their latency; z and y take
                    // turns in the buffer)
#pragma unroll 1
                    for (; b < 16 * c + 4 * q + 4; b += kOutGroups) {
                        const int t0 = 8 * b - c * L;
                        if (live && t0 < nv) {
                            uint32_t xr[4], yr[4];
                            float2 y1[4], y2[4];
                            if (gated) {
                                next_z();
                                load_z();
                            }
                            ldsm4t(x + t0 * 128, xr);
                            float2 e2 = *reinterpret_cast<const float2*>(gt + GT_E + t0 + 2 * (lane & 3));
                            if constexpr (!BF16) e2 = fmul2(e2, make_float2(h_scale, h_scale));
                            tmem_ld_frag(tm + lanes + TM_Y1 + (t0 & 63), tm + lanes + TM_Y2 + t0, y1, y2);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float2 o = y1[k];
                                if constexpr (!BF16) o = fmul2(o, make_float2(m_scale, m_scale));
                                o = ffma2(e2, y2[k], o);
                                o = ffma2(make_float2(D, D), unpack2<BF16>(xr[k]), o);
                                if (gated) o = fmul2(o, gz[k]);
                                yr[k] = pack2<BF16>(o.x, o.y);
                            }
                            if (gated) gates();
                            __syncwarp();
                            stsm4t(io_frag, yr);
                            __syncwarp();
                            uint4 v;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                         : "r"(io_piece)
                                         : "memory");
                            if (t0 + pt < nv) __stcs(reinterpret_cast<uint4*>(yp), v);
                            yp += y_step;
                            __syncwarp();  // y is read: the buffer is free
                        }
                    }
                    tc_fence_before_sync();  // the products are read
                    warp_arrive(sy, B_Y1FREE + (q & 1));
                    if (q & 1) warp_arrive(sy, B_Y2FREE + (q >> 1));
                }
                if (!ok) break;
                warp_arrive(sy, B_EMPTY + s);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    __syncwarp();
    if (warp == kMmaWarp) tmem_dealloc(tm, TM_COLS);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

bool make_map16(CUtensorMap* m, bool bf16, const void* base, int64_t width, int64_t rows, int64_t stride) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, L}, one[2] = {1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base),
               dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int P, int N>
cudaError_t launch_pn(const TcParams& p, int64_t units, cudaStream_t s) {
    constexpr int bytes = SM_TOTAL;
    const unsigned grid = static_cast<unsigned>(units * p.n_heads);
    // (T / seg: no fewer than the segments of disjoint sequences that are not last ones)
    const unsigned inner = static_cast<unsigned>((units - p.q.n_seq) * p.n_heads);
    cudaError_t e;
    if (p.ws) {
        e = set_smem_once(reinterpret_cast<const void*>(ssm_scan_tc_kernel<BF16, P, N, 1>), bytes);
        if (e != cudaSuccess) return e;
        ssm_scan_tc_kernel<BF16, P, N, 1><<<inner, kThreadsTc, bytes, s>>>(p);
        internal_count_launch();
    }
    e = set_smem_once(reinterpret_cast<const void*>(ssm_scan_tc_kernel<BF16, P, N, 0>), bytes);
    if (e != cudaSuccess) return e;
    // Behind a first launch the second starts on the SMs as they fall free, and waits where it
    // first needs what that one leaves (2048 tokens, 48 heads: 60 us, 4 more without).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreadsTc);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ws ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, ssm_scan_tc_kernel<BF16, P, N, 0>, p);
}

template <bool BF16>
cudaError_t launch_b(const TcParams& p, int head_dim, int state_dim, int64_t units, cudaStream_t s) {
    if (head_dim == 128)
        return state_dim == 128 ? launch_pn<BF16, 128, 128>(p, units, s) : launch_pn<BF16, 128, 64>(p, units, s);
    return state_dim == 128 ? launch_pn<BF16, 64, 128>(p, units, s) : launch_pn<BF16, 64, 64>(p, units, s);
}

std::atomic<int*> g_status_word[64];  // its address on the devices it was asked for

}  // namespace

// Segments: with H heads, SMs / H segments of all tokens together fill the device; a
// segment is that share of the call's chunks, but at least a 16th of them (a segment sums
// the contributions of those before it).  One sequence, BF16, 128 x 128, us at segments of
// the share and at others: 48 heads, 1024 tokens (3 chunks) 42 (2 chunks 53, 4 46, uncut 48),
// 2048 (6) 60 (3 chunks 69, uncut 83); 16 heads, 1024 (1) 34 (2 chunks 36, 4 44, uncut 46);
// 8 heads, 4096 (2) 45 (4 chunks 48, uncut 147).  The first launch costs what 3 chunks do:
// sequences stay whole where segments save fewer (48 heads, 512 tokens: of 2 chunks 36,
// uncut 32; 16 heads, 384: of 1 chunk 30, uncut 26; 512: of 1 chunk 30, uncut 30).
// Several sequences are mostly whole segments, for which that launch is in vain, so theirs
// are 4 chunks at least (48 heads, 4 sequences of 512 tokens: segments of 4 chunks 70, uncut
// 60; 8 of 128: of 2 chunks 52, uncut 42).  Heads of 64 x 128: 64 heads, 2048 tokens (8) 71
// (4 chunks 78, uncut 85), 8192 (32) 208 (16 chunks 214, uncut 302); 80 heads, which are not
// cut (one segment fills more than half of the SMs), 2048 tokens 85 (8 chunks 108), 8192 303
// (16 chunks 295, 32 354); 128 heads, 8192 305 (32 chunks 368).
int64_t ssm_scan_segment(int64_t T, int n_seq, int n_heads, int sm_count) {
    const int64_t chunks = (T + L - 1) / L, least = n_seq > 1 ? 4 : 1;
    int64_t parts = sm_count / n_heads;
    if (parts > 16) parts = 16;
    if (parts < 1) parts = 1;
    int64_t share = (chunks + parts - 1) / parts;
    if (share < least) share = least;
    return (chunks - share < 3 ? chunks : share) * L;
}

bool ssm_scan_tc_sizes(int head_dim, int state_dim, int dtype, int64_t T, int n_seq) {
    return dtype != GDN_F32 && (head_dim == 64 || head_dim == 128) && (state_dim == 64 || state_dim == 128) &&
           T >= int64_t{kSsmTcMinTokens} * n_seq;
}

size_t ssm_scan_tc_workspace(int64_t T, int n_seq, int n_heads, int head_dim, int state_dim, int sm_count) {
    const int64_t seg = ssm_scan_segment(T, n_seq, n_heads, sm_count);
    if (seg >= T) return 0;
    const size_t units = static_cast<size_t>(T / seg) + n_seq;
    return units * n_heads * (static_cast<size_t>(head_dim) * state_dim + 4) * sizeof(float);
}

cudaError_t launch_ssm_scan_tc(const SsmScanParams& p, void* workspace, int sm_count, cudaStream_t s) {
    const bool bf16 = p.dtype == GDN_BF16;
    TcParams t{};
    if (!make_map16(&t.tm_x, bf16, p.x, static_cast<int64_t>(p.n_heads) * p.head_dim, p.T, p.x_stride) ||
        !make_map16(&t.tm_b, bf16, p.B, static_cast<int64_t>(p.n_groups) * p.state_dim, p.T, p.b_stride) ||
        !make_map16(&t.tm_c, bf16, p.C, static_cast<int64_t>(p.n_groups) * p.state_dim, p.T, p.c_stride) ||
        (p.z && !make_map16(&t.tm_z, bf16, p.z, static_cast<int64_t>(p.n_heads) * p.head_dim, p.T, p.z_stride)))
        return cudaErrorInvalidValue;
    const int64_t seg = ssm_scan_segment(p.T, p.n_seq, p.n_heads, sm_count);
    const int64_t units = p.T / seg + p.n_seq;
    t.a = p.a; t.z = p.z; t.y = p.y;
    t.a_stride = p.a_stride; t.z_stride = p.z_stride; t.y_stride = p.y_stride;
    t.A_log = p.A_log; t.dt_bias = p.dt_bias; t.D = p.D;
    t.states = p.states;
    if (seg < p.T) {
        t.ws = static_cast<float*>(workspace);
        t.ws_decay = t.ws + static_cast<size_t>(units) * p.n_heads * p.head_dim * p.state_dim;
    }
    t.q = SsmSeqs{p.cu, p.slots, p.has_state, p.n_seq, p.n_slots, p.T};
    t.units = units;
    t.seg = static_cast<int>(seg);
    t.n_heads = p.n_heads;
    t.n_groups = p.n_groups;
    cudaError_t e = ssm_status_word(&t.status);
    if (e != cudaSuccess) return e;
    return bf16 ? launch_b<true>(t, p.head_dim, p.state_dim, units, s) : launch_b<false>(t, p.head_dim, p.state_dim, units, s);
}

cudaError_t ssm_status_word(int** word) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    *word = g_status_word[dev].load();
    if (*word) return cudaSuccess;
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_ssm_status);
    if (e != cudaSuccess) return e;
    *word = static_cast<int*>(p);
    g_status_word[dev].store(*word);
    return cudaSuccess;
}

cudaError_t ssm_take_status(int device, int* word) {
    *word = 0;
    int* at = device >= 0 && device < 64 ? g_status_word[device].load() : nullptr;
    if (!at) return cudaSuccess;
    cudaError_t e = cudaMemcpy(word, at, sizeof(int), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && *word != 0) e = cudaMemset(at, 0, sizeof(int));
    return e;
}

}  // namespace gdn
