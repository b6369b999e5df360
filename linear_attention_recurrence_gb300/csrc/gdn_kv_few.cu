// Attention of few rows a sequence over a paged 4-bit cache (sm_103a): single tokens of many
// requests, drafted tokens.
//
// A unit is one (sequence, KV head, block of R = 8 or 16 rows), a row being a (token, head of
// the KV head's group); its work is the tiles of 64 tokens that one of its rows may see.  All
// units' tiles, in order, are cut into equal pieces, one for each warp, so that ragged lengths
// fill the device evenly; a unit that several warps share leaves partial results in the
// workspace, which a second launch joins in order of the tokens.
//
// A warp copies a tile's codes and scales into its own two slots of shared memory (cp.async: the
// bytes of small pages are too few for bulk copies) and computes, transposed so that the few rows
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
// What bounds it: the instructions, their latency and the half-rate pipes (19 a token and KV head,
// of which 4 convert codes, 4 scale them and 1 multiplies; issued in 57% of the cycles), then memory.
// 48 query and 16 KV heads of 128, BF16: 64 requests of up to 8192 tokens
// 139 us (0.64 GB at 4.6 TB/s; the join 9 of it), one of 32768 33 us, 16 of up to 6000 with 4 tokens
// each 51 us; 64 and 8 heads of 64, FP16: 250 requests of up to 1500 51 us. Steps, the first of
// these: warps of a CTA on one unit 310 us; CTAs of 4 warps 233; tiles of 64 tokens and maxima renewed
// seldom 180; a piece for each warp 157; plain asynchronous copies in place of bulk ones 150; code of
// their own for whole tiles 147; a unit's start counted in its pieces 140.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kSlots = 2;    // tiles in shared memory a warp
constexpr int kUnitTiles = 2;  // what a unit's start and end count for, in tiles (250 requests: 1 61 us, 2 55, 4 74)
// A row's maximum is renewed only once a score passes it by more than 2^kSlack: probabilities,
// times 2^kPShift, stay below 2^(kPShift + kSlack) (FP16 ends at 2^16).
constexpr float kPShift = 8.f, kSlack = 7.f;

// Warps are apart from one another: a unit's start (its lengths, pages and queries, one load after
// the other) and its end overlap with the other warps' work.  CTAs are only what they come in.
constexpr int kWarps = 4;
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 3 : 2;  // (16 rows in 168 registers spill: 16 x 4 tokens 88 us, in 255 78)
// Where there is enough to do, so many pieces for each resident warp: CTAs that end early make room.
// (64 requests: 2 158 us, 3 170, whose joins are more.)
constexpr int kWaves = 2;
template <int NT>
constexpr int kPiecesPerSm = kWarps * kCtasPerSm<NT> * kWaves;
// Tiles of a piece: a wave's share at most, down to kMinTiles, and no fewer than the waves leave.
// (Small pieces of 8, 16, 64 tiles: 16 x 4 tokens 74, 57, 57 us; 64 requests 147, 147, 152.)
constexpr int kMinTiles = 2, kSmallPiece = 16;

constexpr int kTile = 64;  // tokens a warp takes at a time
template <int D>
constexpr int kTileBytes = 2 * kTile * (D / 2 + D / kKvGroup);

// A partial result: R rows of head_dim sums, then R maxima (base 2) and R sums.
template <int R, int D>
constexpr int kPartialFloats = R * (D + 2);

struct Geometry {
    int64_t begin, rows, tiles, first, blocks, cost;
};
// Where no sequence has more tiles than this (by its row of the table), a unit is a warp's as a whole
// and nothing is joined: kWholeTiles, and kWholeTilesMany where there are units for all resident warps.
// Whole / joined, us, 16 KV heads of 128: 1 request of 256 tokens 14 / 16, of 512 20 / 16; 16 of 512 22 / 22,
// of 1024 35 / 27; 200 of 256 47 / 51, of 512 70 / 90, of 1024 113 / 123, of 2048 201 / 201; 8 of 64, 250 of up to
// 700 39 / 41, of up to 1500 63 / 55.
constexpr int kWholeTiles = 4, kWholeTilesMany = 16;
bool whole_units(const KvSeqs& q, int n_kv, int sm_count) {
    const bool many = static_cast<int64_t>(q.n_seq) * n_kv >= static_cast<int64_t>(sm_count) * kWarps * kCtasPerSm<1>;
    return (static_cast<int64_t>(q.max_pages) << q.page_log2) <= (many ? kWholeTilesMany : kWholeTiles) * kTile;
}
// A unit's part of the call's cost: its tiles, and its start and end.
__device__ __forceinline__ int64_t unit_cost(const KvAttentionParams& p, int64_t tiles) {
    return p.whole ? 1 : tiles + kUnitTiles;
}

// What sequence s has to do: `tiles` for each of n_kv * blocks units.
__device__ __forceinline__ Geometry geometry(const KvAttentionParams& p, int s, int R) {
    Geometry g{};
    int64_t e;
    kv_rows(p.s, s, g.begin, e);
    g.rows = e - g.begin;
    if (g.rows == 0) return g;
    const int group = p.n_heads / p.n_kv;
    if (g.rows * group > kKvFewRows) return g;  // (the other kernel's)
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
    g.blocks = (g.rows * group + R - 1) / R;
    g.cost = unit_cost(p, g.tiles) * g.blocks * p.n_kv;
    return g;
}

struct Scratch {
    int64_t warp_sum[kWarps];
    int64_t base[kWarps];  // of each warp's piece: the tiles before its sequence,
    int seq[kWarps];       // and the sequence
};

// Tiles of a piece, of `total` tiles, over the resident warps or kWaves times as many.  (Whole units: units.)
__device__ __forceinline__ int64_t piece_tiles(int64_t total, int64_t pieces, bool whole) {
    if (whole) return (total + pieces - 1) / pieces;
    const int64_t one = (total * kWaves + pieces - 1) / pieces, all = (total + pieces - 1) / pieces;
    const int64_t small = one < kSmallPiece ? one : kSmallPiece;
    const int64_t per = all > small ? all : small;
    return per > kMinTiles ? per : kMinTiles;
}

// Sums up all sequences' tiles and finds, for each of the CTA's warps, the sequence that its
// piece begins in.  Returns the tiles of a piece; 0: nothing is left for this CTA.
__device__ int64_t find_pieces(const KvAttentionParams& p, int R, int64_t* all, Scratch& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kThreads = kWarps * 32;
    const int64_t pieces = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t per = 0, total = 0, at = 0;
    // one round over the sequences for the sum, another for the places (the same one where a round has them all)
    for (int round = 0; round < 2; ++round) {
        int64_t base = 0;
        for (int s0 = 0; s0 < p.s.n_seq; s0 += kThreads) {
            const int64_t n = s0 + tid < p.s.n_seq ? geometry(p, s0 + tid, R).cost : 0;
            int64_t inc = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += v;
            }
            if (lane == 31) sh.warp_sum[warp] = inc;
            __syncthreads();
            int64_t before = base, sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int64_t v = sh.warp_sum[w];
                if (w < warp) before += v;
                sum += v;
            }
            const int64_t first = before + inc - n;
            base += sum;
            if (p.s.n_seq <= kThreads) {
                total = base;
                per = piece_tiles(total, pieces, p.whole);
                at = static_cast<int64_t>(blockIdx.x) * kWarps * per;
                round = 1;
            }
            if (round == 1) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const int64_t mine = at + w * per;
                    if (mine >= first && mine < first + n) {
                        sh.base[w] = first;
                        sh.seq[w] = s0 + tid;
                    }
                }
            }
            __syncthreads();
            if (round == 1 && base > at + (kWarps - 1) * per) break;  // uniform
        }
        if (round == 0) {
            total = base;
            per = piece_tiles(total, pieces, p.whole);
            at = static_cast<int64_t>(blockIdx.x) * kWarps * per;
            if (at >= total) break;
        }
    }
    *all = total;
    return per;
}

// What the joining launch needs to know of a piece whose first unit began in an earlier one and
// ends here.
struct Join {
    int64_t row;    // first row of the block (token * group + head), from the sequence's first
    int64_t begin;  // first row of the sequence
    int rows;       // rows of the block; 0: nothing to join
    int head;       // KV head
    int first_piece;  // the piece that the unit began in
    int pad;
};

template <int R, int D>
__device__ __forceinline__ float* partial_of(void* ws, int64_t pieces, int64_t piece, int which) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + pieces * sizeof(Join)) +
           (piece * 2 + which) * kPartialFloats<R, D>;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<NT>) kv_few_kernel(const KvAttentionParams p) {
    constexpr int R = 8 * NT;
    constexpr int B = 2;  // sixteens of tokens that are computed at a time
    constexpr int DL = D / 4;        // elements of a token's K that a lane takes (its words: DL / 8)
    constexpr int KS = D / 16;       // k-steps of S^T, M tiles of O^T
    constexpr int kPlane = kTile * (D / 2 + D / kKvGroup);  // K's, then V's, in a tile
    constexpr int kScales = kTile * D / 2;                  // their scales within it
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Scratch scratch;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int group = p.n_heads / p.n_kv;
    const int64_t pieces = static_cast<int64_t>(gridDim.x) * kWarps, piece = static_cast<int64_t>(blockIdx.x) * kWarps + warp;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int64_t total;
    const int64_t per = find_pieces(p, R, &total, scratch);
    int64_t at = piece * per;
    const int64_t end = at + per < total ? at + per : total;
    Join* join = static_cast<Join*>(p.workspace) + piece;
    if (lane == 0 && !p.whole) join->rows = 0;
    __syncwarp();
    if (at >= end) return;
    int s = scratch.seq[warp];
    int64_t base = scratch.base[warp];  // tiles before sequence s
    Geometry geo = geometry(p, s, R);

    unsigned char* slots = smem + warp * kSlots * kTileBytes<D>;

    while (at < end) {
        while (at >= base + geo.cost) {  // the next sequence with rows
            base += geo.cost;
            geo = geometry(p, ++s, R);
        }
        const int64_t cost = unit_cost(p, geo.tiles);
        const int64_t unit = (at - base) / cost;  // head-major
        const int64_t unit_begin = base + unit * cost;
        const int head = static_cast<int>(unit / geo.blocks);
        const int64_t row0 = (unit - head * geo.blocks) * R;
        const int64_t left = geo.rows * group - row0;
        const int rows = left < R ? static_cast<int>(left) : R;
        // its tiles from `begin_tile` to `end_tile` are this warp's (the first of a unit's cost is its start)
        const int64_t unit_end = unit_begin + cost;
        const int64_t stop = end < unit_end ? end : unit_end;
        const int64_t begin_tile = at - unit_begin > kUnitTiles ? at - unit_begin - kUnitTiles : 0;
        const int64_t end_tile = p.whole ? geo.tiles : stop - unit_begin > kUnitTiles ? stop - unit_begin - kUnitTiles : 0;
        const int n_tiles = static_cast<int>(end_tile - begin_tile);
        const int64_t tile0 = geo.first + begin_tile;
        if (n_tiles == 0) {
            at = stop;
            continue;
        }
        const int64_t len = __ldg(p.s.kv_lens + s);
        const int64_t cap = kv_capacity(p.s);
        const int held = static_cast<int>(len < cap ? len : cap);

        // A tile is one page's, or 2 or 4 small ones': lane i looks up part i of it.
        constexpr int kTileLog2 = 6, kParts = kTile / 16;
        const int part_log2 = p.s.page_log2 < kTileLog2 ? p.s.page_log2 : kTileLog2;
        const int64_t plane = kv_plane(p.s.page_log2, D);
        const int64_t scales_at = int64_t{D / 2} << p.s.page_log2;
        // the address of that part's first token of K's codes, or nullptr; its place in the page
        auto part_at = [&](int64_t tile) -> const uint8_t* {
            const int64_t token = tile * kTile + (static_cast<int64_t>(lane) << part_log2);
            const int64_t page = lane < kTile >> part_log2 && token < held ? kv_page(p.s, s, token) : -1;
            return page < 0 ? nullptr : p.cache + (page * p.n_kv + head) * 2 * plane;
        };
        // starts a tile's copies, 16 bytes a lane at a time; returns which of its sixteens of tokens there are
        auto fetch = [&](int64_t tile, const uint8_t* mine, int slot) -> uint32_t {
            const uint32_t parts = __ballot_sync(0xffffffffu, mine != nullptr);
            unsigned char* dst = slots + slot * kTileBytes<D> + 16 * lane;
            const int in_page = static_cast<int>(tile * kTile) & ((1 << p.s.page_log2) - 1);
            constexpr int TPI = 1024 / D, TPL = 256 / D;  // tokens of a warp's 512 bytes of codes; of a lane's 16 of scales
            if (part_log2 == kTileLog2) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), 0));
                if (src) {
                    const uint8_t* codes = src + in_page * (D / 2) + 16 * lane;
                    const uint8_t* scales = src + scales_at + in_page * (D / kKvGroup) + 16 * lane;
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
#pragma unroll
                        for (int i = 0; i < kTile / TPI; ++i) cp_async16(dst + which * kPlane + 512 * i, codes + which * plane + 512 * i);
                        if (lane < kTile / TPL) cp_async16(dst + which * kPlane + kScales, scales + which * plane);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kTile / TPI; ++i) {
                    const int part = (i * TPI) >> part_log2;
                    const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), part));
                    if (src) {
                        src += (i * TPI - (part << part_log2)) * (D / 2) + 16 * lane;
#pragma unroll
                        for (int which = 0; which < 2; ++which) cp_async16(dst + which * kPlane + 512 * i, src + which * plane);
                    }
                }
                const int token = (lane % (kTile / TPL)) * TPL, part = token >> part_log2;
                const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), part));
                if (src && lane < kTile / TPL) {
                    src += scales_at + (token - (part << part_log2)) * (D / kKvGroup);
#pragma unroll
                    for (int which = 0; which < 2; ++which) cp_async16(dst + which * kPlane + kScales, src + which * plane);
                }
            }
            uint32_t there = parts;
            if (part_log2 > 4) {
                there = 0;
#pragma unroll
                for (int b = 0; b < kParts; ++b) there |= (parts >> ((16 * b) >> part_log2) & 1) << b;
            }
            return there;
        };
        uint32_t halves[kSlots];
        const uint8_t* next_part = nullptr;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            halves[i] = i < n_tiles ? fetch(tile0 + i, part_at(tile0 + i), i) : 0;
            cp_async_commit();
        }
        if (n_tiles > kSlots) next_part = part_at(tile0 + kSlots);

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
            const float ks = p.k_scale ? __ldg(p.k_scale + head) : 1.f;
            if ((p.scale < 0) != (ks < 0)) {  // the factor of the scores is never below 0, so that it keeps their order
#pragma unroll
                for (int i = 0; i < DL; ++i) q[i] = -q[i];
            }
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
            // (the head's scale last: queries sized against it keep the product in FP32's range)
            const float f0 = fabsf(p.scale) * unscale * fabsf(ks);
            const float f = f0 < 1e-37f ? 1e-37f : f0;  // (nor 0, which would make a NaN of a place that is not seen)
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
        float top[2 * NT], less[2 * NT];
        float2 sum[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][t][k] = 0;
            top[2 * n] = top[2 * n + 1] = -INFINITY;
            less[2 * n] = less[2 * n + 1] = kPShift;
            sum[n] = make_float2(0, 0);
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
        for (int i = 0; i < n_tiles; ++i) {
            const int slot = i % kSlots;
            const int64_t tile = tile0 + i;
            cp_async_wait<kSlots - 1>();
            __syncwarp();
            const unsigned char* kc = slots + slot * kTileBytes<D>;
            const unsigned char* vc = kc + kPlane;
            const uint32_t there = halves[slot];
            const int token0 = static_cast<int>(tile) * kTile;
            const bool whole = there == (1u << kTile / 16) - 1 && token0 >= all_from && token0 + kTile <= all_to;
            // the lane's tokens of V: pairs (2 c, 2 c + 1), the odd lanes' swapped, and 8 behind
            const int t0 = 2 * c + (c & 1), t1 = 2 * c + 1 - (c & 1);
#pragma unroll 1
            for (int at16 = 0; at16 < kTile / 16; at16 += B) {  // B times 16 tokens
                const unsigned char* k16 = kc + 16 * at16 * (D / 2);
                const unsigned char* v16 = vc + 16 * at16 * (D / 2);
                const unsigned char* ks16 = kc + kScales + 16 * at16 * (D / kKvGroup);
                const unsigned char* vs16 = vc + kScales + 16 * at16 * (D / kKvGroup);
                const uint32_t there16 = there >> at16;
                uint32_t vs[B];  // V's scales of the lane's 4 tokens of each 16
                uint32_t nan = 0;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const unsigned char* at_s = vs16 + 16 * b * (D / kKvGroup) + (g * KS >> 3);
                    vs[b] = at_s[t0 * (D / kKvGroup)] | at_s[t1 * (D / kKvGroup)] << 8 |
                            at_s[(t0 + 8) * (D / kKvGroup)] << 16 | static_cast<uint32_t>(at_s[(t1 + 8) * (D / kKvGroup)]) << 24;
                    nan |= (vs[b] & 0x7f7f7f7fu) + 0x01010101u;
                }
                const bool odd = __any_sync(0xffffffffu, (nan & 0x80808080u) || !whole);  // not all seen by all, or a NaN
                const int token16 = token0 + 16 * at16;
                // (two copies of the code: branches within would keep instructions of different sixteens apart)
                auto step = [&](auto odd_tag) {
                constexpr bool odd = decltype(odd_tag)::value;
                float2 sc[B][NT][2];  // S^T: [token row g, + 8], columns 2 c, 2 c + 1
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    // ---- S^T: tokens 16 b + pg, + 8
                    uint32_t kw[2][DL / 8], ks[2][DL / 16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = 16 * b + 8 * h + pg;
                        const unsigned char* at_k = k16 + tok * (D / 2) + c * (DL / 2);
                        uint32_t two;
                        if constexpr (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(at_k);
                            kw[h][0] = v.x, kw[h][1] = v.y, kw[h][2] = v.z, kw[h][3] = v.w;
                            two = *reinterpret_cast<const uint16_t*>(ks16 + tok * (D / kKvGroup) + 2 * c);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(at_k);
                            kw[h][0] = v.x, kw[h][1] = v.y;
                            two = ks16[tok * (D / kKvGroup) + c];
                        }
                        if constexpr (odd) {  // a NaN scale of the token's V is one of its K
                            const unsigned char* at_v = vs16 + tok * (D / kKvGroup) + c * (DL / 16);
                            uint32_t v = at_v[0];
                            if (D == 128) v |= at_v[1] << 8;
                            if (any_e4m3_nan(v)) two = 0x7f7f;
                        }
                        const uint32_t f = e4m3_to_f16(two);
                        ks[h][0] = __byte_perm(f, f, 0x1010);
                        if constexpr (D == 128) ks[h][1] = __byte_perm(f, f, 0x3232);
                    }
                    float acc[NT][4], acc2[NT][4];  // two chains, so that products wait less for one another
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[n][k] = acc2[n][k] = 0;
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
                            for (int n = 0; n < NT; ++n)
                                mma16816(k ? acc2[n] : acc[n], a, qf[n][4 * w + 2 * k], qf[n][4 * w + 2 * k + 1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[n][k] += acc2[n][k];
                    if constexpr (odd) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int tok = token16 + 16 * b + 8 * (k >> 1) + pg;
                                if (!(there16 >> b & 1) || tok < from[2 * n + (k & 1)] || tok >= to[2 * n + (k & 1)])
                                    acc[n][k] = -INFINITY;
                            }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sc[b][n][0] = make_float2(acc[n][0], acc[n][1]);
                        sc[b][n][1] = make_float2(acc[n][2], acc[n][3]);
                    }
                }
                // ---- the rows' maxima, where a score passes one by far; what was summed up shrinks
                bool past = false;
                float most[2 * NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float m0 = sc[0][n][0].x, m1 = sc[0][n][0].y;
#pragma unroll
                    for (int x = 1; x < 2 * B; ++x) {
                        m0 = fmaxf(m0, sc[x / 2][n][x & 1].x);
                        m1 = fmaxf(m1, sc[x / 2][n][x & 1].y);
                    }
                    most[2 * n] = m0 * fac[2 * n];
                    most[2 * n + 1] = m1 * fac[2 * n + 1];
                    past |= most[2 * n] > top[2 * n] + kSlack || most[2 * n + 1] > top[2 * n + 1] + kSlack;
                }
                if (__any_sync(0xffffffffu, past)) {
#pragma unroll
                    for (int x = 0; x < 2 * NT; ++x) {
                        float m = most[x];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        const float now = fmaxf(top[x], m);
                        most[x] = top[x] == now ? 1.f : ex2(top[x] - now);
                        top[x] = now;
                        less[x] = kPShift - (now == -INFINITY ? 0.f : now);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sum[n].x *= most[2 * n];
                        sum[n].y *= most[2 * n + 1];
#pragma unroll
                        for (int t = 0; t < KS; ++t)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[n][t][k] *= most[2 * n + (k & 1)];
                    }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float2 e = ffma2(sc[b][n][h], make_float2(fac[2 * n], fac[2 * n + 1]), make_float2(less[2 * n], less[2 * n + 1]));
                            e = make_float2(ex2(e.x), ex2(e.y));
                            sum[n] = fadd2(sum[n], e);
                            pf[n][h] = transpose8x8(pack_f16(e.x, e.y));
                        }
                    uint32_t vw[4][KS / 4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = 16 * b + (k & 1 ? t1 : t0) + 8 * (k >> 1);
                        const unsigned char* at_v = v16 + tok * (D / 2) + g * KS;
                        if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(at_v);
                            vw[k][0] = v.x, vw[k][1] = v.y;
                        } else {
                            vw[k][0] = *reinterpret_cast<const uint32_t*>(at_v);
                        }
                    }
                    uint32_t s0 = vs[b] & 0xffff, s1 = vs[b] >> 16;
                    if constexpr (odd) {  // what no row sees, or holds a NaN, counts as 0
                        uint32_t keep = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tok = token16 + 16 * b + (k & 1 ? t1 : t0) + 8 * (k >> 1);
                            if ((there16 >> b & 1) && tok < held && !any_e4m3_nan(vs[b] >> (8 * k) & 0xff)) keep |= 0xffu << (8 * k);
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
                };
                if (odd)
                    step(std::true_type{});
                else
                    step(std::false_type{});
            }
            // ---- the slot is read: its next tile
            __syncwarp();
            if (i + kSlots < n_tiles) {
                const int64_t next = tile + kSlots;
                const uint32_t h = fetch(next, next_part, slot);
#pragma unroll
                for (int k = 0; k < kSlots; ++k)
                    if (k == slot) halves[k] = h;
                if (i + kSlots + 1 < n_tiles) next_part = part_at(next + 1);
            }
            cp_async_commit();
        }

        // ---- the rows' results, or this piece's part of them
        const bool begins = begin_tile == 0, ends = stop == unit_end;
        float* partial = partial_of<R, D>(p.workspace, pieces, piece, begins ? 1 : 0);
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x) {
            float l = x & 1 ? sum[x / 2].y : sum[x / 2].x;
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int n = x / 2, r = 8 * n + 2 * c + (x & 1);
            if (r >= rows) continue;
            float v[D / 8];  // elements g D / 8 .. of the row
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                v[2 * t] = o[n][t][x & 1];
                v[2 * t + 1] = o[n][t][2 + (x & 1)];
            }
            if (begins && ends) {
                int64_t token;
                int h;
                row_of(row0 + r, group, p.n_kv, head, token, h);
                const float f = l == 0.f ? 0.f : 1.f / l, vs = p.v_scale ? __ldg(p.v_scale + head) : 1.f;
#pragma unroll
                for (int t = 0; t < D / 8; ++t) v[t] = l == 0.f ? 0.f : v[t] * f * vs;
                T* dst = static_cast<T*>(p.out) + (geo.begin + token) * p.out_stride + h * D + g * (D / 8);
                if (p.vector) {
#pragma unroll
                    for (int t = 0; t < D / 8; t += 8) {
                        float w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = v[t + k];
                        store_vec<T, 8>(dst + t, w);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < D / 8; ++t) dst[t] = from_f<T>(v[t]);
                }
                if (p.lse && g == 0)
                    p.lse[(geo.begin + token) * p.n_heads + h] = l == 0.f ? -INFINITY : (top[x] - kPShift + log2f(l)) * 0.6931471805599453f;
            } else {
#pragma unroll
                for (int t = 0; t < D / 8; t += 2)
                    *reinterpret_cast<float2*>(partial + r * D + g * (D / 8) + t) = make_float2(v[t], v[t + 1]);
                if (g == 0) {
                    partial[R * D + r] = top[x];
                    partial[R * D + R + r] = l;
                }
            }
        }
        if (lane == 0 && !begins && ends)
            *join = Join{row0, geo.begin, rows, head, static_cast<int>((unit_begin + kUnitTiles) / per), 0};
        __syncwarp();
        at = stop;
    }
}

// A running softmax sum of 4 (or 2) elements of a row.
template <int E>
struct Running {
    float m, l, v[E];
};
template <int E>
__device__ __forceinline__ void join_into(Running<E>& a, const Running<E>& b) {
    const float now = fmaxf(a.m, b.m), ref = now == -INFINITY ? 0.f : now;
    const float f = ex2(a.m - ref), h = ex2(b.m - ref);
    a.l = f * a.l + h * b.l;
#pragma unroll
    for (int i = 0; i < E; ++i) a.v[i] = f * a.v[i] + h * b.v[i];
    a.m = now;
}

// Joins the partial results of the units that end in a piece they did not begin in: those of the
// piece it began in (its second), then the first of each that follows.  A CTA looks at pieces
// blockIdx.x, + gridDim.x, ... and joins row blockIdx.y of theirs: of few pieces a warp alone, of
// many all warps.
constexpr int kJoinWarps = 8, kJoinMost = 32, kJoinFew = 32;
template <class T, int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) kv_join_kernel(const KvAttentionParams p, int pieces) {
    constexpr int R = 8 * NT, E = D / 32;
    using Sum = Running<E>;
    __shared__ Join joins[kJoinMost];
    __shared__ Sum sums[kJoinWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // pieces [a, b) of a row: their maxima and sums a lane each, then their elements in order
    auto part_of_row = [&](const Join& j, int r, int a, int b) {
        Sum s{-INFINITY, 0.f, {}};
        for (int x0 = a; x0 < b; x0 += 32) {
            const int n = b - x0 < 32 ? b - x0 : 32;
            const float* first = partial_of<R, D>(p.workspace, pieces, j.first_piece + x0, 0);
            constexpr int64_t kNext = 2 * kPartialFloats<R, D>;
            const int second = x0 == 0 ? kPartialFloats<R, D> : 0;  // (of the piece that the unit began in)
            float pm = -INFINITY, pl = 0;
            if (lane < n) {
                const float* mine = first + lane * kNext + (lane == 0 ? second : 0) + R * D + r;
                pm = mine[0];
                pl = mine[R];
            }
            Sum o{pm, 0.f, {}};
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) o.m = fmaxf(o.m, __shfl_xor_sync(0xffffffffu, o.m, off));
            const float w = ex2(pm - (o.m == -INFINITY ? 0.f : o.m));
            o.l = w * pl;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) o.l += __shfl_xor_sync(0xffffffffu, o.l, off);
            for (int x = 0; x < n; x += 8) {
                float2 v[8][E / 2];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float* mine = first + (x + k) * kNext + (x + k == 0 ? second : 0) + r * D + E * lane;
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        v[k][i] = x + k < n ? *reinterpret_cast<const float2*>(mine + 2 * i) : make_float2(0, 0);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = __shfl_sync(0xffffffffu, w, (x + k) & 31);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        if (x + k < n) {
                            o.v[2 * i] = fmaf(f, v[k][i].x, o.v[2 * i]);
                            o.v[2 * i + 1] = fmaf(f, v[k][i].y, o.v[2 * i + 1]);
                        }
                    }
                }
            }
            if (x0 == a)
                s = o;
            else
                join_into(s, o);
        }
        return s;
    };
    auto write_row = [&](const Join& j, int r, const Sum& s) {
        int64_t token;
        int h;
        row_of(j.row + r, p.n_heads / p.n_kv, p.n_kv, j.head, token, h);
        const float f = s.l == 0.f ? 0.f : 1.f / s.l, vs = p.v_scale ? __ldg(p.v_scale + j.head) : 1.f;
        T* dst = static_cast<T*>(p.out) + (j.begin + token) * p.out_stride + h * D + E * lane;
#pragma unroll
        for (int i = 0; i < E; ++i) dst[i] = from_f<T>(s.l == 0.f ? 0.f : s.v[i] * f * vs);
        if (p.lse && lane == 0)
            p.lse[(j.begin + token) * p.n_heads + h] = s.l == 0.f ? -INFINITY : (s.m - kPShift + log2f(s.l)) * 0.6931471805599453f;
    };
    for (int first = blockIdx.x; first < pieces; first += kJoinMost * gridDim.x) {
        __syncthreads();
        bool many = false;
        if (tid < kJoinMost) {
            const int64_t piece = first + static_cast<int64_t>(tid) * gridDim.x;
            Join j{};
            if (piece < pieces) j = static_cast<const Join*>(p.workspace)[piece];
            j.pad = j.rows > r ? static_cast<int>(piece) - j.first_piece + 1 : 0;  // its pieces
            joins[tid] = j;
            many = j.pad > kJoinFew;
        }
        many = __syncthreads_or(many);
        for (int i = warp; i < kJoinMost; i += kJoinWarps) {
            const int n = joins[i].pad;
            if (n > 0 && n <= kJoinFew) write_row(joins[i], r, part_of_row(joins[i], r, 0, n));
        }
        if (!many) continue;
        for (int i = 0; i < kJoinMost; ++i) {
            const int n = joins[i].pad;
            if (n <= kJoinFew) continue;
            sums[warp][lane] = part_of_row(joins[i], r, n * warp / kJoinWarps, n * (warp + 1) / kJoinWarps);
            __syncthreads();
            if (warp == 0) {
                Sum s = sums[0][lane];
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) join_into(s, sums[w][lane]);
                write_row(joins[i], r, s);
            }
            __syncthreads();
        }
    }
}

template <class T, int D, int NT>
cudaError_t launch(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    constexpr int smem = kWarps * kSlots * kTileBytes<D>;
    const int ctas = sm_count * kCtasPerSm<NT> * kWaves;
    if (cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kv_few_kernel<T, D, NT>), smem); e != cudaSuccess) return e;
    kv_few_kernel<T, D, NT><<<ctas, kWarps * 32, smem, s>>>(p);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    internal_count_launch();
    if (p.whole) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    // (a row of the grid for each row that a unit may have)
    const int64_t rows = p.s.cu ? 8 * NT : p.s.per_seq * (p.n_heads / p.n_kv);
    cfg.gridDim = dim3(sm_count, static_cast<unsigned>(rows < 8 * NT ? rows : 8 * NT));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D, NT>, p, ctas * kWarps);
    if (e == cudaSuccess) internal_count_launch();
    return e;
}

template <class T, int D>
cudaError_t by_rows(const KvAttentionParams& p, int sm_count, cudaStream_t s) {
    const int64_t group = p.n_heads / p.n_kv;
    const int64_t tokens = p.s.cu ? (p.s.T + p.s.n_seq - 1) / p.s.n_seq : p.s.per_seq;
    return tokens * group <= 8 ? launch<T, D, 1>(p, sm_count, s) : launch<T, D, 2>(p, sm_count, s);
}

}  // namespace

size_t kv_few_workspace(const KvSeqs& q, int n_kv, int head_dim, int sm_count) {
    if (whole_units(q, n_kv, sm_count)) return 0;
    const size_t row = 2 * (head_dim + 2) * sizeof(float);
    const size_t a = kPiecesPerSm<1> * (sizeof(Join) + 8 * row), b = kPiecesPerSm<2> * (sizeof(Join) + 16 * row);
    return sm_count * (a > b ? a : b);
}

cudaError_t launch_kv_few(const KvAttentionParams& params, int sm_count, cudaStream_t s) {
    KvAttentionParams p = params;
    p.whole = whole_units(p.s, p.n_kv, sm_count);
    if (p.dtype == GDN_BF16)
        return p.head_dim == 128 ? by_rows<__nv_bfloat16, 128>(p, sm_count, s) : by_rows<__nv_bfloat16, 64>(p, sm_count, s);
    return p.head_dim == 128 ? by_rows<__half, 128>(p, sm_count, s) : by_rows<__half, 64>(p, sm_count, s);
}

}  // namespace gdn
