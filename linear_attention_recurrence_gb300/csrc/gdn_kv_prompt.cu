// Attention of prompts over a paged 4-bit cache on the tensor cores (sm_103a).
//
// A unit is 256 rows of one (sequence, KV head), a row being a (token, head of the KV head's
// group), in two tiles of 128; a CTA walks its cache in blocks of 128 tokens:
//     S = Q K^T           128 x 128 per tile, over head_dim
//     O += P V            128 x head_dim, P = 2^(S - m) rounded to FP16
// as FP16 tcgen05.mma with the scores and the output in tensor memory; P takes the place of the
// scores it came from and is the second product's operand there.  Why FP16, and why that is
// exact for K, V and Q, is said in gdn_kv_few.cu.
//
// Warp roles (640 threads): warps 0-3 the softmax of tile 0, 4-7 of tile 1 (a thread a row);
// 8-15 turn codes and scales into the operands' swizzled tiles, from registers that the next
// block's bytes already fill (K and V lie alike, a token a row: K is read with head_dim as the
// sum, V with the tokens); 16 and 17 issue the tiles' MMAs.  While one tile's softmax runs, the other tile's
// products do.  A row's maximum is renewed only when a score passes it by 2^7; the row's own
// thread then scales its part of O, which no product touches until its P is there.
//
// Where units x KV heads do not fill the device, a unit's blocks are split between CTAs, whose
// results a second launch joins.
//
// What bounds it: the products, and in them the reading of shared memory. A 128 x 64 x 16 product
// with both operands there takes 68 cycles (128 wide 96: 85 to 88 bytes a cycle), with the first in
// tensor memory 72 for 128 columns, so a block's take 3330 cycles of 4250 (887 of 1074 us at 10000
// tokens with nothing else done); bringing K and V takes 9%. Scores 128 wide would take a quarter less,
// but leave a tile one place for them, in which every hand-over (400 cycles from a product's issue to
// its waiter's next) stands in a row: 1255 us. 48 query and 16 KV heads of 128, BF16: 10000 tokens 1074 us
// (1.15 PFLOP/s), 2048 86 us, 509 behind 16384 219 us; 12 FP16 prompts of 8185 tokens behind up to
// 900, window 1024, 309 us. Steps, at 10000 tokens: 4 warps that bring K and V 1704 us, 8 1270; a tile's
// products a warp's each, scores by 64 1081.
#include <type_traits>

#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kRows = 256, kBlock = 128, kHalf = 64;  // of a unit; tokens of a block, and of a product
constexpr int kThreads = 640;
constexpr int kDequantWarp = 8, kMmaWarp = 16, kDequantWarps = kMmaWarp - kDequantWarp;
// Registers of the softmax warps, those that bring K and V, and the rest: together what the
// launch has (96 a thread).
static_assert(256 * 144 + 256 * 72 + 128 * 48 == kThreads * 96, "registers");
constexpr float kPShift = 8.f, kSlack = 7.f;  // as in gdn_kv_few.cu
constexpr int kMaxSplits = 16;

using Sync = SyncOf<kDevErrKv, false>;

// barriers: Q is there; K and V of a stage are; ... are read; by tile and half block: the scores are
// there, their P is, the output's product with it is done
enum { B_Q, B_K, B_V = B_K + 2, B_KFREE = B_V + 2, B_VFREE = B_KFREE + 2, B_S = B_VFREE + 2, B_P = B_S + 4, B_O = B_P + 4,
       B_FIN = B_O + 4, NBAR = B_FIN + 2 };
__device__ constexpr int arrivals(int b, int tiles) {
    if (b == B_Q) return kDequantWarp;
    if (b < B_KFREE) return kDequantWarps;  // the warps that bring K and V
    if (b < B_S) return tiles;              // commits of each tile's products
    if (b >= B_P && b < B_O) return 4;      // a tile's softmax warps
    return 1;
}

template <int D>
struct Smem {
    static constexpr uint32_t kTile = D / 64 * kBox;  // 128 rows
    static constexpr uint32_t Q = 0, K = 2 * kTile, V = K + 2 * kTile, BAR = V + 2 * kTile,
                              MISC = BAR + NBAR * 8, TOTAL = MISC + 64;
};
static_assert(Smem<128>::TOTAL <= 227 * 1024, "shared memory");

struct Unit {
    int64_t begin, rows, row0;  // of the sequence; the unit's first (token * group + head)
    int s;
};
struct Found {
    int64_t warp_sum[kThreads / 32];
    Unit unit;
};

__device__ __forceinline__ int64_t units_of(const KvAttentionParams& p, int s, int64_t& begin, int64_t& rows) {
    int64_t e;
    kv_rows(p.s, s, begin, e);
    rows = e - begin;
    const int64_t n = rows * (p.n_heads / p.n_kv);
    return n > kKvFewRows ? (n + kRows - 1) / kRows : 0;
}
// Unit u of all sequences' units, a sequence's last (which sees most) first.
__device__ bool find_unit(const KvAttentionParams& p, int64_t u, Unit* out, Found& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!p.s.cu) {  // sequences of the same rows
        const int64_t rows = p.s.per_seq, each = (rows * (p.n_heads / p.n_kv) + kRows - 1) / kRows, s = u / each;
        *out = Unit{s * rows, rows, (each - 1 - (u - s * each)) * kRows, static_cast<int>(s)};
        return s < p.s.n_seq;
    }
    if (tid == 0) sh.unit.s = -1;
    int64_t base = 0;
    for (int s0 = 0; s0 < p.s.n_seq; s0 += kThreads) {
        int64_t begin = 0, rows = 0;
        const int64_t n = s0 + tid < p.s.n_seq ? units_of(p, s0 + tid, begin, rows) : 0;
        int64_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 31) sh.warp_sum[warp] = inc;
        __syncthreads();
        int64_t before = base, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sh.warp_sum[w];
            total += sh.warp_sum[w];
        }
        const int64_t first = before + inc - n;
        if (u >= first && u < first + n) sh.unit = Unit{begin, rows, (first + n - 1 - u) * kRows, s0 + tid};
        base += total;
        __syncthreads();
        if (base > u) break;  // uniform
    }
    __syncthreads();
    *out = sh.unit;
    return out->s >= 0;
}

// What the joining launch needs to know of a unit (rows 0: there is none).
struct Part {
    int64_t begin, row0;
    int rows, head;
    int64_t pad;
};
template <int D>
constexpr int64_t kPartFloats = static_cast<int64_t>(kRows) * (D + 2);  // sums, then maxima and sums of probabilities

__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* v) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,"
        "%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <class T, int E>
__device__ __forceinline__ void load_row(const T* p, bool vector, float (&q)[E]) {
    if (vector) {
#pragma unroll
        for (int i = 0; i < E; i += 8) {
            float v[8];
            load_vec<T, 8>(p + i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) q[i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = to_f<T>(p[i]);
    }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const KvAttentionParams p, int splits, int64_t units) {
    using SM = Smem<D>;
    constexpr int NB = D / 64;
    constexpr uint32_t TM_S = 0, TM_O = 256;
    extern __shared__ __align__(1024) unsigned char kv_prompt_smem[];
    unsigned char* sm = kv_prompt_smem;
    if (smem_addr(sm) % 1024 != 0) {
        if (threadIdx.x == 0) {
            report_error(p.status, kDevErrKvLayout);
            // (the joining launch finds no unit, rather than what the workspace held)
            if (splits > 1 && blockIdx.x % splits == 0) static_cast<Part*>(p.workspace)[blockIdx.x / splits].rows = 0;
        }
        return;
    }
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SM::MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + SM::MISC + 8);
    const Sync sy{bar, abort_flag, p.status};
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int group = p.n_heads / p.n_kv;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int split = static_cast<int>(blockIdx.x % splits);
    const int64_t work = blockIdx.x / splits;  // (unit, head)
    const int head = static_cast<int>(work % p.n_kv);
    Part* part = reinterpret_cast<Part*>(p.workspace) + work;
    Unit un;
    const bool any = find_unit(p, work / p.n_kv, &un, *reinterpret_cast<Found*>(sm + SM::K));
    if (!any) {
        if (splits > 1 && split == 0 && tid == 0) part->rows = 0;
        return;
    }
    const int64_t left = un.rows * group - un.row0;
    const int rows = left < kRows ? static_cast<int>(left) : kRows;
    if (splits > 1 && split == 0 && tid == 0) *part = Part{un.begin, un.row0, rows, head, 0};
    const bool two = rows > kBlock;

    // the blocks that one of its rows may see, and this CTA's of them
    const int64_t len = __ldg(p.s.kv_lens + un.s), cap = kv_capacity(p.s);
    const int64_t held64 = len < cap ? (len < 0 ? 0 : len) : cap;
    const int held = static_cast<int>(held64);
    const int64_t place0 = len - un.rows + un.row0 / group, place1 = len - un.rows + (un.row0 + rows - 1) / group;
    int64_t lo = p.window > 0 ? place0 - p.window + 1 : 0, hi = p.causal && place1 + 1 < held64 ? place1 + 1 : held64;
    lo = lo < 0 ? 0 : lo;
    const int all0 = static_cast<int>(lo / kBlock), all1 = hi > lo ? static_cast<int>((hi + kBlock - 1) / kBlock) : all0;
    const int first = all0 + static_cast<int>(static_cast<int64_t>(all1 - all0) * split / splits);
    const int n = all0 + static_cast<int>(static_cast<int64_t>(all1 - all0) * (split + 1) / splits) - first;

    if (tid == 0) {
#pragma unroll
        for (int b = 0; b < NBAR; ++b) mbar_init(&bar[b], arrivals(b, two ? 2 : 1));
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp < kDequantWarp) {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        const int t = warp >> 2, r = t * kBlock + (warp & 3) * 32 + lane;  // tile, row
        if (t == 1 && !two) {
            warp_arrive(sy, B_Q);
        } else {
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t ts = tm + lanes + TM_S + t * kBlock, to = tm + lanes + TM_O + t * D;
            // ---- the row's queries
            const float ks = p.k_scale ? __ldg(p.k_scale + head) : 1.f;
            float up = (p.scale < 0) != (ks < 0) ? -1.f : 1.f, f = fabsf(p.scale);  // (the factor of the scores is never below 0)
            {
                constexpr int E = 64;
                const int64_t row = un.row0 + (r < rows ? r : 0), token = row / group;
                const int h = static_cast<int>(row - token * group) * p.n_kv + head;
                const T* src = static_cast<const T*>(p.q) + (un.begin + token) * p.q_stride + h * D;
                float most = 0;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
                    for (int b = 0; b < D; b += E) {
                        float q[E];
                        load_row<T, E>(src + b, p.vector, q);
#pragma unroll
                        for (int i = 0; i < E; ++i) most = fmaxf(most, fabsf(q[i]));
                    }
                    // a power of two that brings the largest to 2^13 .. 2^14
                    int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
                    e = e < -100 ? -100 : e > 127 ? 13 : e;  // (infinities and NaN as they are)
                    up *= __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                    f *= __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
                }
                if (r >= rows) up = 0.f;
                unsigned char* dst = sm + SM::Q + t * SM::kTile + (r % kBlock) * 128;
#pragma unroll
                for (int b = 0; b < D; b += E) {
                    float q[E];
                    load_row<T, E>(src + b, p.vector, q);
#pragma unroll
                    for (int i = 0; i < E; i += 8) {
                        uint4 v;
                        v.x = pack_f16(q[i] * up, q[i + 1] * up);
                        v.y = pack_f16(q[i + 2] * up, q[i + 3] * up);
                        v.z = pack_f16(q[i + 4] * up, q[i + 5] * up);
                        v.w = pack_f16(q[i + 6] * up, q[i + 7] * up);
                        *reinterpret_cast<uint4*>(dst + (b / 64) * kBox + (((i / 8) ^ (r & 7)) << 4)) = v;
                    }
                }
                if (p.k_scale) f *= fabsf(__ldg(p.k_scale + head));  // (last: queries sized against it keep the product in FP32's range)
                f = f < 1e-37f ? 1e-37f : f;  // (nor 0, which would make a NaN of a place that is not seen)
                fence_async_smem();
                warp_arrive(sy, B_Q);
            }
            // pages that are none, in this CTA's blocks (their tokens are not seen), from the one that the
            // first block lies in (a page may be longer than a block)
            const int64_t at0 = static_cast<int64_t>(first) * kBlock >> p.s.page_log2 << p.s.page_log2;
            const int64_t at1 = static_cast<int64_t>(first + n) * kBlock < held ? static_cast<int64_t>(first + n) * kBlock : held;
            bool holes = false;
            for (int64_t at = at0 + (static_cast<int64_t>(lane) << p.s.page_log2); at < at1; at += int64_t{32} << p.s.page_log2)
                holes |= kv_page(p.s, un.s, at) < 0;
            holes = __any_sync(0xffffffffu, holes);
            const int64_t place = len - un.rows + (un.row0 + r) / group;
            int from = 0, upto = held;
            if (p.causal && place + 1 < held) upto = place + 1 > 0 ? static_cast<int>(place + 1) : 0;
            if (p.window > 0 && place - p.window + 1 > 0) from = static_cast<int>(place - p.window + 1);
            if (r >= rows) from = 0, upto = INT32_MAX;  // (never looked at)
            float top = -INFINITY;
            float2 sums[4] = {};
            bool ok = true;
            for (int i = 0; i < 2 * n; ++i) {
                const int at = 2 * t + (i & 1);  // of the tile's two places
                const uint32_t ps = ts + (i & 1) * kHalf;
                if (!(ok = wait_warp(sy, B_S + at, i / 2))) break;
                tc_fence_after_sync();
                float s[kHalf];
                tmem_ld64(ps, s);
                const int token0 = first * kBlock + i * kHalf;
                if (__any_sync(0xffffffffu, token0 < from || token0 + kHalf > upto) || holes) {
#pragma unroll
                    for (int b = 0; b < kHalf / 16; ++b) {
                        const bool there = !holes || kv_page(p.s, un.s, token0 + 16 * b) >= 0;
#pragma unroll
                        for (int x = 16 * b; x < 16 * b + 16; ++x)
                            if (!there || token0 + x < from || token0 + x >= upto) s[x] = -INFINITY;
                    }
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};  // (four chains: few warps share a scheduler)
#pragma unroll
                for (int x = 4; x < kHalf; x += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x + 4 < kHalf ? fmaxf(s[x + k], s[x + 4 + k]) : s[x + k]);
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f;
                if (__any_sync(0xffffffffu, m > top + kSlack)) {
                    const float now = fmaxf(top, m), less = top == now ? 1.f : ex2(top - now);
                    top = now;
#pragma unroll
                    for (int x = 0; x < 4; ++x) sums[x] = fmul2(sums[x], make_float2(less, less));
                    if (i > 0) {
                        if (!(ok = wait_warp(sy, B_O + (at ^ 1), (i - 1) / 2))) break;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            tmem_ld16(to + c, o);
#pragma unroll
                            for (int x = 0; x < 16; x += 2) {
                                const float2 v = fmul2(make_float2(o[x], o[x + 1]), make_float2(less, less));
                                o[x] = v.x, o[x + 1] = v.y;
                            }
                            tmem_st16(to + c, o);
                        }
                    }
                }
                const float less = kPShift - (top == -INFINITY ? 0.f : top);
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 e = ffma2(make_float2(s[c + 2 * x], s[c + 2 * x + 1]), make_float2(f, f), make_float2(less, less));
                        e = make_float2(ex2(e.x), ex2(e.y));
                        sums[x & 3] = fadd2(sums[x & 3], e);
                        w[x] = pack_f16(e.x, e.y);
                    }
                    tmem_st_u16(ps + c / 2, w);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                warp_arrive(sy, B_P + at);
            }
            if (ok && n > 0) ok = wait_warp(sy, B_O + 2 * t + 1, n - 1);
            tc_fence_after_sync();
            const float l = ((sums[0].x + sums[1].x) + (sums[2].x + sums[3].x)) + ((sums[0].y + sums[1].y) + (sums[2].y + sums[3].y));
            if (ok && splits > 1) {
                float* o = reinterpret_cast<float*>(reinterpret_cast<Part*>(p.workspace) + units * p.n_kv) +
                           static_cast<int64_t>(blockIdx.x) * kPartFloats<D>;
#pragma unroll 1
                for (int c = 0; c < D && n > 0; c += 32) {
                    float v[32];
                    tmem_ld32(to + c, v);
                    if (r < rows) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(o + r * D + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
                o[kRows * D + r] = top;
                o[kRows * (D + 1) + r] = n > 0 ? l : 0.f;
            } else if (ok) {
                const int64_t row = un.row0 + r, token = row / group;
                const int h = static_cast<int>(row - token * group) * p.n_kv + head;
                // (two factors: one alone would leave FP32's range where the head's scale is small; in pairs, as
                // one at a time 10000 tokens take 1095 us, in pairs 1073)
                const float k = l == 0.f ? 0.f : 1.f / l, vs = p.v_scale ? __ldg(p.v_scale + head) : 1.f;
                T* dst = static_cast<T*>(p.out) + (un.begin + token) * p.out_stride + h * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    if (n > 0) {
                        tmem_ld32(to + c, v);
                    }
                    if (r < rows) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float w[8];
#pragma unroll
                            for (int x = 0; x < 8; x += 2) {
                                const float2 y = fmul2(fmul2(make_float2(v[i + x], v[i + x + 1]), make_float2(k, k)), make_float2(vs, vs));
                                w[x] = n == 0 || l == 0.f ? 0.f : y.x, w[x + 1] = n == 0 || l == 0.f ? 0.f : y.y;
                            }
                            if (p.vector) {
                                store_vec<T, 8>(dst + c + i, w);
                            } else {
#pragma unroll
                                for (int x = 0; x < 8; ++x) dst[c + i + x] = from_f<T>(w[x]);
                            }
                        }
                    }
                }
                if (p.lse && r < rows)
                    p.lse[(un.begin + token) * p.n_heads + h] =
                        n == 0 || l == 0.f ? -INFINITY : (top - kPShift + log2f(l)) * 0.6931471805599453f;
            }
        }
    } else if (warp < kMmaWarp) {
        // ---- K and V: an item is 32 codes of a token
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        constexpr int Q4 = D / 32, PER = 32 / Q4, ITEMS = kBlock / (kDequantWarps * PER);  // items of a token; tokens a warp covers; items a thread
        const int w = warp - kDequantWarp, quarter = lane % Q4, tok = w * PER + lane / Q4;  // + kDequantWarps PER i
        const int64_t plane = kv_plane(p.s.page_log2, D);
        struct Raw {
            uint4 code[ITEMS];
            uint32_t scale[ITEMS];  // of its two groups; K: those of V in the upper half
        };
        Raw raw[2];
        // pages of block j's tokens, looked up a block ahead
        int32_t page[ITEMS];
        auto look_up = [&](int j) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int at = (first + j) * kBlock + tok + kDequantWarps * PER * i;
                page[i] = at < held ? static_cast<int32_t>(kv_page(p.s, un.s, at)) : -1;
            }
        };
        auto fetch = [&](int j, int which, Raw& r) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int at = (first + j) * kBlock + tok + kDequantWarps * PER * i;
                r.code[i] = make_uint4(0, 0, 0, 0);
                r.scale[i] = 0;
                if (page[i] >= 0) {
                    const int in_page = at & ((1 << p.s.page_log2) - 1);
                    const uint8_t* k = p.cache + (static_cast<int64_t>(page[i]) * p.n_kv + head) * 2 * plane;
                    const uint8_t* mine = k + which * plane;
                    const int64_t scales = (int64_t{D / 2} << p.s.page_log2) + in_page * (D / kKvGroup) + 2 * quarter;
                    r.code[i] = __ldg(reinterpret_cast<const uint4*>(mine + in_page * (D / 2) + 16 * quarter));
                    r.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(mine + scales));
                    if (which == 0) r.scale[i] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(k + plane + scales))) << 16;
                }
            }
        };
        auto put = [&](int which, const Raw& r, unsigned char* dst) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int token = tok + kDequantWarps * PER * i;
                uint32_t two = r.scale[i] & 0xffff;
                if (which == 0) {
                    if (any_e4m3_nan(r.scale[i] >> 16)) two = 0x7f7f;  // a NaN scale of the token's V is one of its K
                } else {
                    if (any_e4m3_nan(two & 0xff)) two &= 0xff00;
                    if (any_e4m3_nan(two >> 8)) two &= 0xff;
                }
                const uint32_t f = e4m3_to_f16(two);
                const uint32_t s0 = __byte_perm(f, f, 0x1010), s1 = __byte_perm(f, f, 0x3232);
                // the lanes of a token's second half take their chunks in another order, so that
                // eight lanes' stores fall on different banks
                const bool swap = D == 128 && (quarter & 2);
                const uint32_t c[4] = {swap ? r.code[i].z : r.code[i].x, swap ? r.code[i].w : r.code[i].y,
                                       swap ? r.code[i].x : r.code[i].z, swap ? r.code[i].y : r.code[i].w};
                unsigned char* row = dst + (D == 128 ? (quarter >> 1) * kBox : 0) + token * 128;
                const int chunk0 = 4 * (quarter & 1);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t v[4];
                    e2m1_to_f16(c[x], v);
                    const uint32_t sc = (x < 2) != swap ? s0 : s1;
                    const int chunk = chunk0 + (swap ? x ^ 2 : x);
                    *reinterpret_cast<uint4*>(row + ((chunk ^ (token & 7)) << 4)) =
                        make_uint4(hmul2(v[0], sc), hmul2(v[1], sc), hmul2(v[2], sc), hmul2(v[3], sc));
                }
            }
        };
        if (n > 0) {
            look_up(0);
            fetch(0, 0, raw[0]);
        }
        for (int j = 0; j < n; ++j) {
            const int st = j & 1;
            fetch(j, 1, raw[1]);
            if (j + 1 < n) look_up(j + 1);
            if (j >= 2 && !wait_warp(sy, B_KFREE + st, j / 2 - 1)) break;
            put(0, raw[0], sm + SM::K + st * SM::kTile);
            fence_async_smem();
            warp_arrive(sy, B_K + st);
            if (j + 1 < n) fetch(j + 1, 0, raw[0]);
            if (j >= 2 && !wait_warp(sy, B_VFREE + st, j / 2 - 1)) break;
            put(1, raw[1], sm + SM::V + st * SM::kTile);
            fence_async_smem();
            warp_arrive(sy, B_V + st);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // a tile's products are a warp's each, so that one tile's wait for its last product (whose
        // operand P the next scores overwrite) leaves the tensor cores the other's
        const int t = warp - kMmaWarp;
        if (t < (two ? 2 : 1) && n > 0) {
            if (elect_one()) {
                constexpr uint32_t ID_S = idesc_f16(false, 128, kHalf, false, false);
                constexpr uint32_t ID_O = idesc_f16(false, 128, D, false, true);  // V: N-major
                const uint32_t sm0 = smem_addr(sm);
                auto scores = [&](int i) {  // of half block i
                    const uint32_t q = sm0 + SM::Q + t * SM::kTile, k = sm0 + SM::K + (i / 2 & 1) * SM::kTile + (i & 1) * (kHalf * 128);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint64_t dq = desc_k(q + b * kBox), dk = desc_k(k + b * kBox);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_ss(tm + TM_S + t * kBlock + (i & 1) * kHalf, dq + 2 * x, dk + 2 * x, ID_S, b > 0 || x > 0);
                    }
                    umma_commit(&bar[B_S + 2 * t + (i & 1)]);
                    if (i & 1) umma_commit(&bar[B_KFREE + (i / 2 & 1)]);
                };
                bool ok = wait_phase(sy, B_Q, 0) && wait_phase(sy, B_K, 0);
                tc_fence_after_sync();
                if (ok) {
                    scores(0);
                    scores(1);
                }
                for (int i = 0; ok && i < 2 * n; ++i) {
                    const int at = 2 * t + (i & 1);
                    if (!(ok = wait_phase(sy, B_V + (i / 2 & 1), i / 4) && wait_phase(sy, B_P + at, i / 2))) break;
                    tc_fence_after_sync();
                    const uint64_t dv = desc_mn(sm0 + SM::V + (i / 2 & 1) * SM::kTile + (i & 1) * (kHalf * 128));
#pragma unroll
                    for (int x = 0; x < kHalf / 16; ++x)
                        mma_ts(tm + TM_O + t * D, tm + TM_S + t * kBlock + (i & 1) * kHalf + 8 * x, dv + 128 * x, ID_O, i > 0 || x > 0);
                    umma_commit(&bar[B_O + at]);
                    if (i & 1) umma_commit(&bar[B_VFREE + (i / 2 & 1)]);
                    if (i + 2 >= 2 * n) continue;
                    // the scores after next take this half's place, once its product is done; the next are there
                    if (!(ok = wait_phase(sy, B_K + ((i / 2 + 1) & 1), (i / 2 + 1) / 2) && wait_phase(sy, B_O + at, i / 2))) break;
                    tc_fence_after_sync();
                    scores(i + 2);
                }
                finish_mma(&bar[B_FIN + t]);
            }
            __syncwarp();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

// Joins the splits of a unit's rows: a warp a row.
template <class T, int D>
__global__ void __launch_bounds__(256) kv_prompt_join_kernel(const KvAttentionParams p, int splits, int64_t units) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Part part = reinterpret_cast<const Part*>(p.workspace)[blockIdx.x];
    if (r >= part.rows) return;
    const float* base = reinterpret_cast<const float*>(reinterpret_cast<const Part*>(p.workspace) + units * p.n_kv) +
                        static_cast<int64_t>(blockIdx.x) * splits * kPartFloats<D>;
    float m = -INFINITY, l = 0, v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0;
    for (int k = 0; k < splits; ++k) m = fmaxf(m, base[k * kPartFloats<D> + kRows * D + r]);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
        const float* o = base + k * kPartFloats<D>;
        const float pl = o[kRows * (D + 1) + r];
        if (pl == 0.f) continue;  // (a split without blocks wrote no sums)
        const float f = ex2(o[kRows * D + r] - ref);
        l += f * pl;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 x = *reinterpret_cast<const float2*>(o + r * D + E * lane + i);
            v[i] += f * x.x;
            v[i + 1] += f * x.y;
        }
    }
    const int group = p.n_heads / p.n_kv;
    const int64_t row = part.row0 + r, token = row / group;
    const int h = static_cast<int>(row - token * group) * p.n_kv + part.head;
    const float f = l == 0.f ? 0.f : 1.f / l, vs = p.v_scale ? __ldg(p.v_scale + part.head) : 1.f;
    T* dst = static_cast<T*>(p.out) + (part.begin + token) * p.out_stride + h * D + E * lane;
#pragma unroll
    for (int i = 0; i < E; ++i) dst[i] = from_f<T>(l == 0.f ? 0.f : v[i] * f * vs);
    if (p.lse && lane == 0)
        p.lse[(part.begin + token) * p.n_heads + h] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * 0.6931471805599453f;
}

// Units of the grid: no fewer than the sequences have.
int64_t unit_bound(int64_t T, int n_seq, int group, bool even) {
    const int64_t seqs = n_seq < T ? n_seq : T;
    if (even) return seqs ? (T / n_seq * group + kRows - 1) / kRows * n_seq : 0;
    return T * group / kRows + seqs;
}

// CTAs that share a unit: 1 where units fill the device, else by the blocks that the busiest
// multiprocessor walks (a CTA's start and end take about two, the joining launch four; 509 tokens
// behind 16384, 96 CTAs: 3 splits 221 us, none 299).
int splits_of(const KvSeqs& q, int64_t ctas, int sm_count) {
    const int64_t blocks = ((static_cast<int64_t>(q.max_pages) << q.page_log2) + kBlock - 1) / kBlock;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int s = 1; s <= kMaxSplits && (s == 1 || (ctas * s <= 2 * sm_count && blocks / s >= 4)); ++s) {
        const int64_t cost = (ctas * s + sm_count - 1) / sm_count * ((blocks + s - 1) / s + 2) + (s > 1 ? 4 : 0);
        if (cost < least) least = cost, best = s;
    }
    return best;
}

template <class T, int D>
cudaError_t launch(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    const int64_t units = unit_bound(p.s.T, p.s.n_seq, p.n_heads / p.n_kv, p.s.cu == nullptr);
    const int64_t ctas = units * p.n_kv;
    const int splits = splits_of(p.s, ctas, sm_count);
    if (cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kv_prompt_kernel<T, D>), Smem<D>::TOTAL); e != cudaSuccess)
        return e;
    kv_prompt_kernel<T, D><<<static_cast<unsigned>(ctas * splits), kThreads, Smem<D>::TOTAL, s>>>(p, splits, units);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    internal_count_launch();
    if (splits == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), kRows / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prompt_join_kernel<T, D>, p, splits, units);
    if (e == cudaSuccess) internal_count_launch();
    return e;
}

}  // namespace

int64_t kv_prompt_ctas(int64_t T, int n_seq, int n_heads, int n_kv) {
    return unit_bound(T, n_seq, n_heads / n_kv, false) * n_kv;
}

size_t kv_prompt_workspace(const KvSeqs& q, bool even, int n_heads, int n_kv, int head_dim, int sm_count) {
    const int64_t ctas = unit_bound(q.T, q.n_seq, n_heads / n_kv, even) * n_kv;
    const int splits = splits_of(q, ctas, sm_count);
    return splits == 1 ? 0 : static_cast<size_t>(ctas) * (sizeof(Part) + sizeof(float) * splits * kRows * (head_dim + 2));
}

cudaError_t launch_kv_prompt(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    if (p.dtype == GDN_BF16)
        return p.head_dim == 128 ? launch<__nv_bfloat16, 128>(p, sm_count, s) : launch<__nv_bfloat16, 64>(p, sm_count, s);
    return p.head_dim == 128 ? launch<__half, 128>(p, sm_count, s) : launch<__half, 64>(p, sm_count, s);
}

}  // namespace gdn
