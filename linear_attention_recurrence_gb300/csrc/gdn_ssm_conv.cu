// Causal depthwise convolution over packed sequences, with bias and SiLU:
//     y[t][c] = act(bias[c] + sum_j w[c][j] X[t - (K - 1) + j][c]),   K = 2, 3 or 4,
// the K - 1 rows before a sequence's first token taken from its slot of the history
// (zeros for a new sequence); the slot then receives the sequence's last K - 1 rows.
//
// Bound by HBM: every row is read once and written once.  A thread holds 4 channels
// (their taps and bias in registers) and walks a tile of rows with the last K - 1 rows in
// registers and 8 rows' loads in flight, so a row is fetched once per tile.  The 8 rows are
// formed without a branch between them, in packed FP32 pairs: what a 16-bit row waits for is
// the latency of its arithmetic (BF16, 16384 x 10240: 172 us with a branch and single
// operations, 124 us so; 8 channels a thread 134 us, 4 rows in flight with 8 CTAs per SM 125,
// 16 rows 131).  16384 x 10240 in FP32 takes 205 us (6.5 TB/s), in BF16 124 us (5.4 TB/s).
//
// History without a race: the tile that holds a sequence's first row also owns the
// rows at positions 1 .. K - 2 (a tile boundary that would fall there moves behind
// them).  So the old history is read by exactly one thread per channel, which then
// writes the new one, in place.
#include "gdn_ssm.cuh"
#include "gdn_ssm.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows whose loads are in flight together

// Sequences whose begin is at or before rows r0 and r1 (all lanes get both counts; one
// pass of independent loads instead of two binary searches of dependent ones).
__device__ __forceinline__ void count_begins(const SsmSeqs& q, int64_t r0, int64_t r1, int& c0, int& c1) {
    c0 = c1 = 1;
    if (!q.cu) return;
    c0 = c1 = 0;
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < q.n_seq; i += 32) {
        const int v = i + lane < q.n_seq ? __ldg(q.cu + i + lane) : INT32_MAX;
        c0 += __popc(__ballot_sync(0xffffffffu, v <= r0));
        c1 += __popc(__ballot_sync(0xffffffffu, v <= r1));
    }
}

// Tile boundary r, moved behind the first K - 1 rows of the sequence that holds it.
template <int K>
__device__ __forceinline__ int64_t tile_edge(const SsmSeqs& q, int64_t r, int count) {
    if (count > 0) {
        int64_t b, e;
        seq_rows(q, count - 1, b, e);
        if (b < r && r < e && r - b < K - 1) r = b + (K - 1) < e ? b + (K - 1) : e;
    }
    return r;
}

// f = act(bias + the taps over the window and the row cur), and the window one row on.
// Pairs of channels in packed instructions, which round as single ones do.
template <int K, int VEC>
__device__ __forceinline__ void conv_row(const float (&w)[VEC][K], const float (&bias)[VEC], float (&win)[K - 1][VEC],
                                         const float (&cur)[VEC], int activation, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        float acc = bias[0];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) acc = fmaf(w[0][j], win[j][0], acc);
        acc = fmaf(w[0][K - 1], cur[0], acc);
        f[0] = activation ? ssm_silu(acc) : acc;
    } else {
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
            float2 acc = make_float2(bias[v], bias[v + 1]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                acc = ffma2(make_float2(w[v][j], w[v + 1][j]), make_float2(win[j][v], win[j][v + 1]), acc);
            acc = ffma2(make_float2(w[v][K - 1], w[v + 1][K - 1]), make_float2(cur[v], cur[v + 1]), acc);
            if (activation) acc = silu2(acc);
            f[v] = acc.x;
            f[v + 1] = acc.y;
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) win[j][v] = win[j + 1][v];
        win[K - 2][v] = cur[v];
    }
}

template <class T, int K, int VEC>
__global__ void __launch_bounds__(kThreads, 5) ssm_conv_kernel(const SsmConvParams p, const SsmSeqs q, int tile_rows) {
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * tile_rows;
    const int64_t r1 = r0 + tile_rows < q.T ? r0 + tile_rows : q.T;
    int c0, c1;
    count_begins(q, r0, r1, c0, c1);
    const int64_t lo = tile_edge<K>(q, r0, c0), hi = r1 < q.T ? tile_edge<K>(q, r1, c1) : q.T;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (c >= p.channels) return;

    float w[VEC][K], bias[VEC];
    if constexpr (VEC > 1) {  // the thread's VEC K taps lie together, on a 16-byte boundary
        float flat[VEC * K];
#pragma unroll
        for (int i = 0; i < VEC * K; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p.w + static_cast<int64_t>(c) * K + i));
            flat[i] = f.x;
            flat[i + 1] = f.y;
            flat[i + 2] = f.z;
            flat[i + 3] = f.w;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int j = 0; j < K; ++j) w[v][j] = flat[v * K + j];
    } else {
#pragma unroll
        for (int j = 0; j < K; ++j) w[0][j] = __ldg(p.w + static_cast<int64_t>(c) * K + j);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) bias[v] = p.bias ? __ldg(p.bias + c + v) : 0.f;
    const T* x = static_cast<const T*>(p.x) + c;
    T* y = static_cast<T*>(p.y) + c;
    T* hist = static_cast<T*>(p.hist);

    int64_t r = lo, b, e;
    int s = c0 > 0 ? c0 - 1 : 0;
    seq_rows(q, s, b, e);
    while (r < hi) {
        while (e <= r) {
            if (++s >= q.n_seq) return;
            seq_rows(q, s, b, e);
        }
        if (r < b) {  // rows of no sequence
            r = b < hi ? b : hi;
            continue;
        }
        float win[K - 1][VEC];
        if (r == b) {
            const int slot = hist ? seq_slot(q, s) : -1;
            T* h = hist + (static_cast<int64_t>(slot) * (K - 1)) * p.channels + c;
            const bool old = slot >= 0 && seq_has_state(q, s);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) win[j][v] = 0.f;
                if (old) load_vec<T, VEC>(h + static_cast<int64_t>(j) * p.channels, win[j]);
            }
            if (slot >= 0) {
                const int64_t len = e - b;
#pragma unroll
                for (int j = 0; j < K - 1; ++j) {
                    const int64_t at = len - (K - 1) + j;  // the row that becomes history row j
                    float f[VEC];
                    if (at >= 0) {
                        load_vec<T, VEC>(x + (b + at) * p.x_stride, f);
                    } else {  // a short sequence keeps rows of the old history, each behind the one written here
#pragma unroll
                        for (int v = 0; v < VEC; ++v) f[v] = 0.f;
                        if (old) load_vec<T, VEC>(h + (at + (K - 1)) * p.channels, f);
                    }
                    store_vec<T, VEC>(h + static_cast<int64_t>(j) * p.channels, f);
                }
            }
        } else {
            // (the tile's edge is K - 1 rows into the sequence at least, unless bounds step back
            // and r is where an overlapping sequence ended: rows before the sequence are not read)
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                const int64_t at = r - (K - 1) + j;
                load_vec<T, VEC>(x + (at > b ? at : b) * p.x_stride, win[j]);
            }
        }
        const int64_t stop = e < hi ? e : hi;
        const T* xr = x + r * p.x_stride;
        T* yr = y + r * p.y_stride;
        for (int left = static_cast<int>(stop - r); left > 0; left -= kAhead) {
            // (rows past the last are formed from it and left out: no branch between the rows)
            Vec<T, VEC> raw[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                raw[u] = *reinterpret_cast<const Vec<T, VEC>*>(xr);
                if (u + 1 < left) xr += p.x_stride;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float cur[VEC], f[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) cur[v] = to_f<T>(raw[u].v[v]);
                conv_row<K, VEC>(w, bias, win, cur, p.activation, f);
                if (u < left) store_vec<T, VEC>(yr, f);
                yr += p.y_stride;
            }
        }
        r = stop;
    }
}

template <class T, int K>
void launch_k(const SsmConvParams& p, const SsmSeqs& q, int sm_count, cudaStream_t s) {
    constexpr int V = 4;
    const int vec = p.vector ? V : 1;
    const int blocks_y = (p.channels + kThreads * vec - 1) / (kThreads * vec);
    // A tile fetches the K - 1 rows before it again (from L2) and the taps, and its CTA starts
    // with those waits.  FP32 waits for HBM either way and takes 16 rows: 16384 x 10240 205 us
    // (32 rows 209, 64 211), 256 rows 13 us (16, 19).  16-bit rows wait for their arithmetic
    // too and take the largest tile that leaves 4 CTAs per SM: 10240 channels, BF16, tiles of
    // 16 / 32 / 64 rows: 256 rows 13 / 13 / 18 us, 1024 20 / 18 / 20, 2048 28 / 26 / 25,
    // 16384 139 / 128 / 124.
    const int64_t rows_y = q.T * blocks_y, fill = int64_t{4} * sm_count;
    const int tile = sizeof(T) == 4 || rows_y < 32 * fill ? 16 : rows_y < 64 * fill ? 32 : 64;
    const dim3 grid(static_cast<unsigned>((q.T + tile - 1) / tile), blocks_y);
    if (vec == V)
        ssm_conv_kernel<T, K, V><<<grid, kThreads, 0, s>>>(p, q, tile);
    else
        ssm_conv_kernel<T, K, 1><<<grid, kThreads, 0, s>>>(p, q, tile);
}

template <class T>
void launch_t(const SsmConvParams& p, const SsmSeqs& q, int sm_count, cudaStream_t s) {
    if (p.width == 2) launch_k<T, 2>(p, q, sm_count, s);
    else if (p.width == 3) launch_k<T, 3>(p, q, sm_count, s);
    else launch_k<T, 4>(p, q, sm_count, s);
}

}  // namespace

cudaError_t launch_ssm_conv(const SsmConvParams& p, int sm_count, cudaStream_t s) {
    const SsmSeqs q{p.cu, p.slots, p.has_state, p.n_seq, p.n_slots, p.T};
    switch (p.dtype) {
        case GDN_F32: launch_t<float>(p, q, sm_count, s); break;
        case GDN_BF16: launch_t<__nv_bfloat16>(p, q, sm_count, s); break;
        default: launch_t<__half>(p, q, sm_count, s); break;
    }
    return cudaGetLastError();
}

}  // namespace gdn
