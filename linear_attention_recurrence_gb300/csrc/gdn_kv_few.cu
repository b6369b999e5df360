// Attention of few rows a sequence over a paged 4-bit cache (sm_103a): single tokens of many
// requests, drafted tokens.
//
// A unit is one (sequence, KV head, block of R = 8 or 16 rows), a row being a (token, head of
// the KV head's group); its work is the tiles of 32 tokens that one of its rows may see.  All
// units' tiles, in order, are cut into equal pieces, one for each CTA, so that ragged lengths
// fill the device evenly; a unit that several CTAs share leaves partial results in the
// workspace, which a second launch joins in order of the tokens.
//
// Every warp walks tiles of its own: it copies a tile's codes and scales into its own slots of
// shared memory (cp.async.bulk, two tiles ahead) and computes, transposed so that the few rows
// are the narrow side of m16n8k16 products:
//     S^T = K Q^T   (16 tokens x 8 rows, over head_dim), running maximum and sum of each row,
//     O^T += V^T P^T   (16 of head_dim x 8 rows, over 16 tokens)
// The order of head_dim in the first product's sum and of its lanes in the second is free, so
// each lane takes 32 neighbouring codes of a token of K, and 16 of V (one scale), whole words
// as they lie in memory; pairs of V's tokens are interleaved as codes, before they become FP16.
// S^T's fragments turn into P^T's by an 8 x 8 transposition in registers (movmatrix).
//
// Operands are FP16: a code times its scale is exact there (2 + 4 significant bits, 2^-10 to
// 2688), FP16 queries are, and BF16 queries after scaling a row by a power of two (what falls
// below 2^-24 then is 2^-38 of the row's largest).  Probabilities are rounded to FP16 once,
// times 2^8 so that one of 2^-32 still counts; sums are FP32.
//
// A token whose values hold a NaN scale gives its scores NaN instead, so that rows that do not
// see it keep clear of it.
//
// What bounds it: memory.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kTile = 32;    // tokens a warp takes at a time
constexpr int kSlots = 2;    // tiles in shared memory a warp
constexpr int kMinTiles = 16;  // a CTA's piece, at least
constexpr float kPShift = 8.f;

template <int NT>
constexpr int kWarps = NT == 1 ? 16 : 12;
template <int D>
constexpr int kTileBytes = 2 * kTile * (D / 2 + D / kKvGroup);

// A partial result: R rows of head_dim sums, then R maxima (base 2) and R sums.
template <int R, int D>
constexpr int kPartialFloats = R * (D + 2);

struct Unit {
    int s, head, block;
    int64_t begin;     // first row of the sequence
    int64_t rows;      // its rows (tokens)
    int64_t tiles;     // tiles of each of its units
    int64_t first;     // tile (of the sequence) that they begin with
    int64_t blocks;    // row blocks
};

struct Geometry {
    int64_t begin, rows, tiles, first, blocks, cost;
};
// What sequence s has to do: `tiles` for each of n_kv * blocks units.
__device__ __forceinline__ Geometry geometry(const KvAttentionParams& p, int s, int R) {
    Geometry g{};
    int64_t e;
    kv_rows(p.s, s, g.begin, e);
    g.rows = e - g.begin;
    if (g.rows == 0) return g;
    const int64_t len = __ldg(p.s.kv_lens + s);
    const int64_t cap = kv_capacity(p.s);
    const int64_t hi = len < cap ? (len < 0 ? 0 : len) : cap;
    int64_t lo = 0;
    if (p.window > 0) {
        lo = len - g.rows - p.window + 1;
        lo = lo < 0 ? 0 : lo;
    }
    g.first = lo / kTile;
    g.tiles = (hi + kTile - 1) / kTile - g.first;
    if (g.tiles < 1) g.tiles = 1;  // (its rows see nothing: the outputs are zeros)
    const int group = p.n_heads / p.n_kv;
    g.blocks = (g.rows * group + R - 1) / R;
    g.cost = g.tiles * g.blocks * p.n_kv;
    return g;
}

template <int W>
struct Scratch {
    int64_t warp_sum[W];
    int64_t found_base;
    int found;
};

// The sum of all sequences' tiles; and the sequence that holds tile `at` of them, with the
// tiles before it.  (at < 0: the sum alone.)
template <int W>
__device__ int64_t scan_tiles(const KvAttentionParams& p, int R, int64_t at, Scratch<W>& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t base = 0;
    for (int s0 = 0; s0 < p.s.n_seq; s0 += W * 32) {
        const int64_t n = s0 + tid < p.s.n_seq ? geometry(p, s0 + tid, R).cost : 0;
        int64_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 31) sh.warp_sum[warp] = inc;
        __syncthreads();
        int64_t before = base, total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int64_t v = sh.warp_sum[w];
            if (w < warp) before += v;
            total += v;
        }
        const int64_t first = before + inc - n;
        if (at >= first && at < first + n) {
            sh.found = s0 + tid;
            sh.found_base = first;
        }
        base += total;
        __syncthreads();
        if (at >= 0 && base > at) break;
    }
    return base;
}

// What the joining launch needs to know of a CTA whose first unit began in an earlier one and
// ends here.
struct Join {
    int64_t row;    // first row of the block (token * group + head), from the sequence's first
    int64_t begin;  // first row of the sequence
    int rows;       // rows of the block; 0: nothing to join
    int head;       // KV head
    int first_cta;  // the CTA that the unit began in
    int pad;
};

template <int R, int D>
__device__ __forceinline__ float* partial_of(void* ws, int ctas, int cta, int which) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + static_cast<size_t>(ctas) * sizeof(Join)) +
           (static_cast<int64_t>(cta) * 2 + which) * kPartialFloats<R, D>;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// An output row: its place in q and out, and the head.
__device__ __forceinline__ void row_of(int64_t row, int group, int n_kv, int kv_head, int64_t& token, int& head) {
    token = row / group;
    head = static_cast<int>(row - token * group) * n_kv + kv_head;
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(kWarps<NT> * 32, 1) kv_few_kernel(const KvAttentionParams p) {
    constexpr int W = kWarps<NT>, R = 8 * NT;
    constexpr int DL = D / 4;        // elements of a token's K that a lane takes (its words: DL / 8)
    constexpr int KS = D / 16;       // k-steps of S^T, M tiles of O^T
    constexpr int kPlane = kTile * (D / 2 + D / kKvGroup);  // K's, then V's, in a tile
    constexpr int kScales = kTile * D / 2;                  // their scales within it
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Scratch<W> scratch;
    __shared__ uint64_t bars[W * kSlots];
    __shared__ float warp_max[W][R], warp_sum[W][R];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int group = p.n_heads / p.n_kv;

    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars[warp * kSlots + i], 1);
    }
    mbar_init_fence();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int64_t total = scan_tiles<W>(p, R, -1, scratch);
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinTiles) per = kMinTiles;
    int64_t at = static_cast<int64_t>(blockIdx.x) * per;
    const int64_t end = at + per < total ? at + per : total;
    Join* join = static_cast<Join*>(p.workspace) + blockIdx.x;
    if (tid == 0) join->rows = 0;
    if (at >= end) return;
    scan_tiles<W>(p, R, at, scratch);
    int s = scratch.found;
    int64_t base = scratch.found_base;  // tiles before sequence s
    Geometry geo = geometry(p, s, R);

    unsigned char* slots = smem + warp * kSlots * kTileBytes<D>;
    uint64_t* bar = bars + warp * kSlots;
    uint32_t uses = 0;  // copies this warp has waited for

    while (at < end) {
        while (at >= base + geo.cost) {  // the next sequence with rows
            base += geo.cost;
            geo = geometry(p, ++s, R);
        }
        const int64_t unit = (at - base) / geo.tiles;  // head-major
        const int64_t unit_begin = base + unit * geo.tiles;
        const int head = static_cast<int>(unit / geo.blocks);
        const int64_t row0 = (unit - head * geo.blocks) * R;
        const int64_t left = geo.rows * group - row0;
        const int rows = left < R ? static_cast<int>(left) : R;
        const int64_t unit_end = unit_begin + geo.tiles;
        const int64_t stop = end < unit_end ? end : unit_end;
        const int n_tiles = static_cast<int>(stop - at);
        const int64_t tile0 = geo.first + (at - unit_begin);
        const int64_t len = __ldg(p.s.kv_lens + s);
        const int64_t cap = kv_capacity(p.s);
        const int held = static_cast<int>(len < cap ? len : cap);

        // what each lane copies of a tile: part (pages of 16 give two), and which of the four arrays
        const int part_log2 = p.s.page_log2 < 5 ? p.s.page_log2 : 5;
        const int parts = kTile >> part_log2;
        const int64_t plane = kv_plane(p.s.page_log2, D);
        const int part = lane >> 2, which = lane & 3;  // K codes, K scales, V codes, V scales
        const bool is_scale = which & 1;
        const int row_bytes = is_scale ? D / kKvGroup : D / 2;
        auto page_at = [&](int64_t tile) -> int64_t {
            const int64_t token = tile * kTile + (static_cast<int64_t>(part) << part_log2);
            return part < parts && token < held ? kv_page(p.s, s, token) : -1;
        };
        // issues the copies of a tile; returns which of its two halves there are
        auto fetch = [&](int64_t tile, int64_t page, int slot) -> uint32_t {
            const uint32_t there = __ballot_sync(0xffffffffu, page >= 0 && which == 0);
            const int n = __popc(there);
            if (lane == 0) {
                if (n)
                    mbar_arrive_expect_tx(&bar[slot], n * 2 * ((D / 2 + D / kKvGroup) << part_log2));
                else
                    mbar_arrive(&bar[slot]);
            }
            __syncwarp();
            if (page >= 0) {
                const int64_t token = tile * kTile + (static_cast<int64_t>(part) << part_log2);
                const int64_t in_page = token & ((int64_t{1} << p.s.page_log2) - 1);
                const uint8_t* src = p.cache + ((page * p.n_kv + head) * 2 + (which >> 1)) * plane +
                                     (is_scale ? (int64_t{D / 2} << p.s.page_log2) : 0) + in_page * row_bytes;
                unsigned char* dst = slots + slot * kTileBytes<D> + (which >> 1) * kPlane + (is_scale ? kScales : 0) +
                                     (part << part_log2) * row_bytes;
                bulk_load(dst, src, row_bytes << part_log2, &bar[slot]);
            }
            if (parts == 1) return there ? 3u : 0u;
            return (there & 1) | ((there >> 3) & 2);
        };
        uint32_t halves[kSlots];
        int64_t next_page = -1;
        const int mine = n_tiles > warp ? (n_tiles - warp + W - 1) / W : 0;  // this warp's tiles
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            halves[i] = i < mine ? fetch(tile0 + warp + i * W, page_at(tile0 + warp + i * W), i) : 0;
        if (mine > kSlots) next_page = page_at(tile0 + warp + kSlots * W);

        // the rows' queries (row 8 n + g, its elements DL c ..), scaled; and what each lane's
        // columns 8 n + 2 c, + 1 of S^T see: tokens [from, to)
        uint32_t qf[NT][DL / 2];
        float fac[2 * NT];
        int from[2 * NT], to[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            float q[DL];
#pragma unroll
            for (int i = 0; i < DL; ++i) q[i] = 0;
            if (r < rows) {
                int64_t token;
                int h;
                row_of(row0 + r, group, p.n_kv, head, token, h);
                const T* src = static_cast<const T*>(p.q) + (geo.begin + token) * p.q_stride + h * D + DL * c;
                if (p.vector) {
#pragma unroll
                    for (int i = 0; i < DL; i += 8) {
                        float v[8];
                        load_vec<T, 8>(src + i, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) q[i + k] = v[k];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < DL; ++i) q[i] = to_f<T>(src[i]);
                }
            }
            float unscale = 1.f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                float most = 0;
#pragma unroll
                for (int i = 0; i < DL; ++i) most = fmaxf(most, fabsf(q[i]));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // a power of two that brings the largest to 2^13 .. 2^14
                int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
                e = e < -100 ? -100 : e > 127 ? 13 : e;  // (infinities and NaN as they are)
                const float up = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                unscale = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
#pragma unroll
                for (int i = 0; i < DL; ++i) q[i] *= up;
            }
#pragma unroll
            for (int i = 0; i < DL / 2; ++i) qf[n][i] = pack_f16(q[2 * i], q[2 * i + 1]);
            const float f = unscale * p.scale * (p.k_scale ? __ldg(p.k_scale + head) : 1.f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                fac[2 * n + k] = __shfl_sync(0xffffffffu, f, 8 * c + 4 * k);
                const int col = 8 * n + 2 * c + k;
                const int64_t place = len - geo.rows + (row0 + col) / group;
                int64_t hi = p.causal ? place + 1 : held;
                hi = hi < held ? hi : held;
                const int64_t lo = p.window > 0 ? place - p.window + 1 : 0;
                // (a column behind the rows is never looked at, and holds no tile back)
                from[2 * n + k] = col < rows && lo > 0 ? static_cast<int>(lo) : 0;
                to[2 * n + k] = col >= rows ? INT32_MAX : hi > 0 ? static_cast<int>(hi) : 0;
            }
        }

        float o[NT][KS][4];
        float top[2 * NT], sum[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][t][k] = 0;
            top[2 * n] = top[2 * n + 1] = -INFINITY;
            sum[2 * n] = sum[2 * n + 1] = 0;
        }
        // tokens that all the lane's columns see
        int all_from = from[0], all_to = to[0];
#pragma unroll
        for (int k = 1; k < 2 * NT; ++k) {
            all_from = from[k] > all_from ? from[k] : all_from;
            all_to = to[k] < all_to ? to[k] : all_to;
        }
        const int pg = g ^ ((g >> 1) & 1);  // the token of row g: pairs (4 i + 2, 4 i + 3) swapped, which
                                            // spreads V's loads over the banks
        for (int i = 0; i < mine; ++i) {
            const int slot = i % kSlots;
            const int64_t tile = tile0 + warp + static_cast<int64_t>(i) * W;
            if (!mbar_wait(&bar[slot], (uses / kSlots) & 1)) {
                report_error(p.status, kDevErrKv);
                mbar_wait(&bar[slot], (uses / kSlots) & 1);  // the copy lands before the CTA can leave
            }
            __syncwarp();
            ++uses;
            const unsigned char* kc = slots + slot * kTileBytes<D>;
            const unsigned char* vc = kc + kPlane;
            const uint32_t there = halves[slot];
            const int token0 = static_cast<int>(tile) * kTile;
            const bool whole = there == 3 && token0 >= all_from && token0 + kTile <= all_to;
            float sc[2][NT][4];
            uint32_t vs[2];  // V's scales of the lane's 4 tokens of each half
            bool odd = false;
            // the lane's tokens of V: pairs (2 c, 2 c + 1), the odd lanes' swapped, and 8 behind
            const int t0 = 2 * c + (c & 1), t1 = 2 * c + 1 - (c & 1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const unsigned char* at_s = vc + kScales + 16 * b * (D / kKvGroup) + (g * KS >> 3);
                vs[b] = at_s[t0 * (D / kKvGroup)] | at_s[t1 * (D / kKvGroup)] << 8 |
                        at_s[(t0 + 8) * (D / kKvGroup)] << 16 | static_cast<uint32_t>(at_s[(t1 + 8) * (D / kKvGroup)]) << 24;
                odd |= any_e4m3_nan(vs[b]);
            }
            odd = __any_sync(0xffffffffu, odd || !whole);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // ---- S^T: tokens 16 b + pg, + 8
                uint32_t kw[2][DL / 8], ks[2][DL / 16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = 16 * b + 8 * h + pg;
                    const unsigned char* at_k = kc + tok * (D / 2) + c * (DL / 2);
                    uint32_t two;
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(at_k);
                        kw[h][0] = v.x, kw[h][1] = v.y, kw[h][2] = v.z, kw[h][3] = v.w;
                        two = *reinterpret_cast<const uint16_t*>(kc + kScales + tok * (D / kKvGroup) + 2 * c);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(at_k);
                        kw[h][0] = v.x, kw[h][1] = v.y;
                        two = kc[kScales + tok * (D / kKvGroup) + c];
                    }
                    if (odd) {  // a NaN scale of the token's V is one of its K
                        const unsigned char* at_v = vc + kScales + tok * (D / kKvGroup) + c * (DL / 16);
                        uint32_t v = at_v[0];
                        if (D == 128) v |= at_v[1] << 8;
                        if (any_e4m3_nan(v)) two = 0x7f7f;
                    }
                    const uint32_t f = e4m3_to_f16(two);
                    ks[h][0] = __byte_perm(f, f, 0x1010);
                    if constexpr (D == 128) ks[h][1] = __byte_perm(f, f, 0x3232);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[b][n][k] = 0;
#pragma unroll
                for (int w = 0; w < DL / 8; ++w) {  // 8 codes: two k-steps
                    uint32_t f0[4], f1[4];
                    e2m1_to_f16(kw[0][w], f0);
                    e2m1_to_f16(kw[1][w], f1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f0[k] = hmul2(f0[k], ks[0][w / 2]);
                        f1[k] = hmul2(f1[k], ks[1][w / 2]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a[4] = {f0[2 * k], f1[2 * k], f0[2 * k + 1], f1[2 * k + 1]};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(sc[b][n], a, qf[n][4 * w + 2 * k], qf[n][4 * w + 2 * k + 1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float v = sc[b][n][k] * fac[2 * n + (k & 1)];
                        if (odd) {
                            const int tok = token0 + 16 * b + 8 * (k >> 1) + pg;
                            if (!(there >> b & 1) || tok < from[2 * n + (k & 1)] || tok >= to[2 * n + (k & 1)]) v = -INFINITY;
                        }
                        sc[b][n][k] = v;
                    }
            }
            // ---- the rows' maxima; what was summed up under a smaller one shrinks
            float shift[2 * NT];
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float m = fmaxf(fmaxf(sc[0][n][k], sc[0][n][k + 2]), fmaxf(sc[1][n][k], sc[1][n][k + 2]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const int x = 2 * n + k;
                    const float now = fmaxf(top[x], m);
                    shift[x] = top[x] == now ? 1.f : ex2(top[x] - now);
                    grew |= top[x] != now;
                    top[x] = now;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sum[2 * n] *= shift[2 * n];
                    sum[2 * n + 1] *= shift[2 * n + 1];
#pragma unroll
                    for (int t = 0; t < KS; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[n][t][k] *= shift[2 * n + (k & 1)];
                }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t pf[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float m = top[2 * n + (k & 1)];
                        e[k] = ex2(sc[b][n][k] - (m == -INFINITY ? 0.f : m) + kPShift);
                        sum[2 * n + (k & 1)] += e[k];
                    }
                    pf[n][0] = transpose8x8(pack_f16(e[0], e[1]));
                    pf[n][1] = transpose8x8(pack_f16(e[2], e[3]));
                }
                uint32_t vw[4][KS / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = 16 * b + (k & 1 ? t1 : t0) + 8 * (k >> 1);
                    const unsigned char* at_v = vc + tok * (D / 2) + g * KS;
                    if constexpr (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2*>(at_v);
                        vw[k][0] = v.x, vw[k][1] = v.y;
                    } else {
                        vw[k][0] = *reinterpret_cast<const uint32_t*>(at_v);
                    }
                }
                uint32_t s0 = vs[b] & 0xffff, s1 = vs[b] >> 16;
                if (odd) {  // what no row sees, or holds a NaN, counts as 0
                    uint32_t keep = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = token0 + 16 * b + (k & 1 ? t1 : t0) + 8 * (k >> 1);
                        if ((there >> b & 1) && tok < held && !any_e4m3_nan(vs[b] >> (8 * k) & 0xff)) keep |= 0xffu << (8 * k);
                    }
                    s0 &= keep & 0xffff;
                    s1 &= keep >> 16;
                }
                s0 = e4m3_to_f16(s0);
                s1 = e4m3_to_f16(s1);
#pragma unroll
                for (int w = 0; w < KS / 4; ++w) {
                    // bytes of two tokens' codes of one element
                    const uint32_t lo0 = (vw[0][w] & 0x0f0f0f0fu) | ((vw[1][w] << 4) & 0xf0f0f0f0u);
                    const uint32_t hi0 = ((vw[0][w] >> 4) & 0x0f0f0f0fu) | (vw[1][w] & 0xf0f0f0f0u);
                    const uint32_t lo1 = (vw[2][w] & 0x0f0f0f0fu) | ((vw[3][w] << 4) & 0xf0f0f0f0u);
                    const uint32_t hi1 = ((vw[2][w] >> 4) & 0x0f0f0f0fu) | (vw[3][w] & 0xf0f0f0f0u);
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    e2m1_to_f16(lo0, a0);
                    e2m1_to_f16(hi0, a1);
                    e2m1_to_f16(lo1, a2);
                    e2m1_to_f16(hi1, a3);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t a[4] = {hmul2(a0[k], s0), hmul2(a1[k], s0), hmul2(a2[k], s1), hmul2(a3[k], s1)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(o[n][4 * w + k], a, pf[n][0], pf[n][1]);
                    }
                }
            }
            // ---- the slot is read: its next tile
            __syncwarp();
            if (i + kSlots < mine) {
                const int64_t next = tile + kSlots * W;
                const uint32_t h = fetch(next, next_page, slot);
#pragma unroll
                for (int k = 0; k < kSlots; ++k)
                    if (k == slot) halves[k] = h;
                if (i + kSlots + 1 < mine) next_page = page_at(next + W);
            }
        }
        // parities go by copies of each slot: an odd count of tiles leaves the slots apart
        if (uses % kSlots) {
            if (lane == 0) mbar_arrive(&bar[uses % kSlots]);
            ++uses;
        }

        // ---- the warps' results, joined through the slots' memory
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x) {
            float v = sum[x];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (g == 0) {
                const int r = 8 * (x / 2) + 2 * c + (x & 1);
                warp_max[warp][r] = top[x];
                warp_sum[warp][r] = v;
            }
        }
        __syncthreads();
        float* part_o = reinterpret_cast<float*>(smem);  // [W][R][D]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)  // row 8 n + 2 c + k, elements 2 KS g + ...: KS g' pairs
                    *reinterpret_cast<float2*>(part_o + (warp * R + 8 * n + 2 * c + k) * D + g * (D / 8) + 2 * t) =
                        make_float2(o[n][t][k], o[n][t][k + 2]);
        __syncthreads();
        const bool begins = at == unit_begin, ends = stop == unit_end;
        float* partial = partial_of<R, D>(p.workspace, gridDim.x, blockIdx.x, begins ? 1 : 0);
        for (int x = tid; x < rows * (D / 2); x += W * 32) {
            const int r = x / (D / 2), d = 2 * (x - r * (D / 2));
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) m = fmaxf(m, warp_max[w][r]);
            const float ref = m == -INFINITY ? 0.f : m;
            float l = 0, v0 = 0, v1 = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = ex2(warp_max[w][r] - ref);
                const float2 v = *reinterpret_cast<const float2*>(part_o + (w * R + r) * D + d);
                l += f * warp_sum[w][r];
                v0 += f * v.x;
                v1 += f * v.y;
            }
            if (begins && ends) {
                int64_t token;
                int h;
                row_of(row0 + r, group, p.n_kv, head, token, h);
                const float f = l == 0.f ? 0.f : (p.v_scale ? __ldg(p.v_scale + head) : 1.f) / l;
                T* dst = static_cast<T*>(p.out) + (geo.begin + token) * p.out_stride + h * D + d;
                dst[0] = from_f<T>(l == 0.f ? 0.f : v0 * f);
                dst[1] = from_f<T>(l == 0.f ? 0.f : v1 * f);
                if (p.lse && d == 0)
                    p.lse[(geo.begin + token) * p.n_heads + h] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float2*>(partial + r * D + d) = make_float2(v0, v1);
                if (d == 0) {
                    partial[R * D + r] = m;
                    partial[R * D + R + r] = l;
                }
            }
        }
        if (tid == 0 && !begins && ends)
            *join = Join{row0, geo.begin, rows, head, static_cast<int>(unit_begin / per), 0};
        fence_async_smem();  // (the slots' next copies come behind these reads and writes)
        __syncthreads();
        at = stop;
    }
}

// Joins the partial results of a unit that ends in CTA blockIdx.x: those of the CTA it began in
// (its second), then the first of each that follows.
template <class T, int D, int NT>
__global__ void __launch_bounds__(D) kv_join_kernel(const KvAttentionParams p, int ctas) {
    constexpr int R = 8 * NT;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Join j = static_cast<const Join*>(p.workspace)[blockIdx.x];
    const int r = blockIdx.y, d = threadIdx.x;
    if (r >= j.rows) return;
    const int n = static_cast<int>(blockIdx.x) - j.first_cta + 1;
    float m = -INFINITY, l = 0, v = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float* part = partial_of<R, D>(p.workspace, ctas, j.first_cta + i, i == 0 ? 1 : 0);
        const float pm = part[R * D + r], pl = part[R * D + R + r], pv = part[r * D + d];
        const float now = fmaxf(m, pm), ref = now == -INFINITY ? 0.f : now;
        const float f = ex2(m - ref), h = ex2(pm - ref);
        l = f * l + h * pl;
        v = f * v + h * pv;
        m = now;
    }
    int64_t token;
    int h;
    row_of(j.row + r, p.n_heads / p.n_kv, p.n_kv, j.head, token, h);
    const float f = (p.v_scale ? __ldg(p.v_scale + j.head) : 1.f) / l;
    static_cast<T*>(p.out)[(j.begin + token) * p.out_stride + h * D + d] = from_f<T>(l == 0.f ? 0.f : v * f);
    if (p.lse && d == 0)
        p.lse[(j.begin + token) * p.n_heads + h] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * 0.6931471805599453f;
}

template <class T, int D, int NT>
cudaError_t launch(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    constexpr int bytes = kWarps<NT> * kSlots * kTileBytes<D>, joined = kWarps<NT> * 8 * NT * D * 4;
    constexpr int smem = bytes > joined ? bytes : joined;
    if (cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kv_few_kernel<T, D, NT>), smem); e != cudaSuccess) return e;
    kv_few_kernel<T, D, NT><<<sm_count, kWarps<NT> * 32, smem, s>>>(p);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sm_count, 8 * NT);
    cfg.blockDim = dim3(D);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D, NT>, p, sm_count);
}

template <class T, int D>
cudaError_t by_rows(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    const int64_t group = p.n_heads / p.n_kv;
    const int64_t tokens = p.s.cu ? (p.s.T + p.s.n_seq - 1) / p.s.n_seq : p.s.per_seq;
    return tokens * group <= 8 ? launch<T, D, 1>(p, sm_count, s) : launch<T, D, 2>(p, sm_count, s);
}

}  // namespace

size_t kv_few_workspace(int head_dim, int sm_count) {
    return static_cast<size_t>(sm_count) * (sizeof(Join) + 2 * 16 * (head_dim + 2) * sizeof(float));
}

cudaError_t launch_kv_few(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    if (p.dtype == GDN_BF16)
        return p.head_dim == 128 ? by_rows<__nv_bfloat16, 128>(p, sm_count, s) : by_rows<__nv_bfloat16, 64>(p, sm_count, s);
    return p.head_dim == 128 ? by_rows<__half, 128>(p, sm_count, s) : by_rows<__half, 64>(p, sm_count, s);
}

}  // namespace gdn
