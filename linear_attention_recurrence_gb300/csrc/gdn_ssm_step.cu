// One token of the causal convolution and the selective scan for each request, one
// launch (the decode step of a layer):
//     u = act(conv_bias + sum_j conv_w[.][j] rows[j]),  rows = (history, this token's row)
//     the history's slot <- its last width - 1 rows;   (x, B, C) = u
//     S <- exp(-exp(A_log) dt) S + dt B x^T,  y = (S^T C + D x) silu(z)
//
// Bound by HBM: a request's state crosses it once each way (64 KB per head of 128 x 128).
// A cluster of CTAs takes one (request, group) and shares out the columns of the
// group's heads in tiles of 32; every CTA convolves the group's B and C channels and its
// own x channels into shared memory.  The x history belongs to one CTA each; the B and C
// history is read by all of the cluster, and its first CTA writes it after a cluster
// barrier behind those reads.  A tile's rows are shared by WPT warps (4, 2 or 1, see the
// launch), which load them in rounds of 16 rows; lanes hold 4 rows x 8 float4 columns per
// load instruction, and the sums over rows meet in two shuffles (and, with more than one
// warp, in shared memory in a fixed order).  48 heads of 128 x 128: 250 requests in FP32
// 281 us (5.9 TB/s), 64 in BF16 76 us (5.4 TB/s), one 13 us (the waits of one request's chain).
#include <cooperative_groups.h>

#include "gdn_ssm.cuh"
#include "gdn_ssm.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int COLS = 32;
constexpr int kMaxN = 128;
// Load instructions in flight per warp (4 rows each), and the next as many: with 4 CTAs per
// SM that is 5.8 TB/s at 250 requests; 8 with 2 CTAs 5.3, 16 with 2 4.2 (the latency of a
// CTA's start and of its convolution is hidden by the other CTAs, not by more loads).
constexpr int kBatchRows = 4;

template <class T>
__device__ __forceinline__ float conv_channel(const SsmStepParams& p, int64_t cw, const T* row, T* hist, bool owner, int64_t c,
                                              float (&old)[4]) {
    const int K = p.width;
    const float now = to_f<T>(row[c]);
    float acc = p.conv_bias ? __ldg(p.conv_bias + c) : 0.f;
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < K) w[j] = __ldg(p.conv_w + c * K + j);
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (j < K - 1) old[j] = to_f<T>(hist[j * cw + c]);
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (j < K - 1) {
            acc = fmaf(w[j], old[j], acc);
            if (owner && j > 0) hist[(j - 1) * cw + c] = from_f<T>(old[j]);
        }
    acc = fmaf(w[K - 1], now, acc);
    if (owner) hist[(K - 2) * cw + c] = from_f<T>(now);
    return p.activation ? ssm_silu(acc) : acc;
}

template <class T, int WPT>
__global__ void __launch_bounds__(kThreads, 4) ssm_step_kernel(const SsmStepParams p) {
    namespace cg = cooperative_groups;
    extern __shared__ float x_s[];  // this CTA's x columns
    __shared__ float B_s[kMaxN], C_s[kMaxN];
    __shared__ float4 part[kWarps][8];
    const int rank = blockIdx.x, ranks = gridDim.x, g = blockIdx.y, req = blockIdx.z;
    const int slot = p.slots ? __ldg(p.slots + req) : req;
    if (slot < 0 || slot >= p.n_slots) return;  // a padded request (the whole cluster returns)

    const int N = p.state_dim, P = p.head_dim, r = p.n_heads / p.n_groups;
    const int64_t cw = static_cast<int64_t>(p.n_heads) * P + 2 * static_cast<int64_t>(p.n_groups) * N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* row = static_cast<const T*>(p.xbc) + req * p.xbc_stride;
    T* hist = static_cast<T*>(p.hist) + static_cast<int64_t>(slot) * (p.width - 1) * cw;
    // the group's tiles of 32 columns, r heads x P / 32 each; this CTA's are [t0, t1)
    const int per_head = P / COLS, tiles = r * per_head;
    const int t0 = tiles * rank / ranks, t1 = tiles * (rank + 1) / ranks;

    // A warp's work is a list of rounds: 16 rows (4 load instructions of 4 rows x 8 float4
    // columns) of its share of a tile's rows, tile after tile.  The next round's loads are
    // issued before a round is worked on, the first ones before the convolution.
    const int sub = lane >> 3, quad = lane & 7;  // row within a load instruction, float4 column
    constexpr int kTilesPerPass = kWarps / WPT;
    const int share = N / WPT, rounds = (share + 4 * kBatchRows - 1) / (4 * kBatchRows);
    const int n0 = (warp % WPT) * share;
    const int passes = (t1 - t0 + kTilesPerPass - 1) / kTilesPerPass;
    auto state_at = [&](int tile, int k) {
        const int h = (tile / per_head) * p.n_groups + g, col = (tile % per_head) * COLS + 4 * quad;
        return p.states + ((static_cast<int64_t>(slot) * p.n_heads + h) * N + n0 + k + sub) * P + col;
    };
    float4 v[kBatchRows], next[kBatchRows];
    auto fetch = [&](int pass, int round) {
        const int tile = t0 + pass * kTilesPerPass + warp / WPT, k = round * 4 * kBatchRows;
        if (tile >= t1) return;
        const float* st = state_at(tile, k);
#pragma unroll
        for (int i = 0; i < kBatchRows; ++i)
            if (k + 4 * i < share) next[i] = __ldcs(reinterpret_cast<const float4*>(st + static_cast<int64_t>(4 * i) * P));
    };
    fetch(0, 0);

    float old[4];
    const int64_t bc = static_cast<int64_t>(p.n_heads) * P;
    // B and C channels of the group: 2 N <= 256 of them, one per thread
    const bool is_bc = tid < 2 * N;
    const int64_t c_bc = tid < N ? bc + static_cast<int64_t>(g) * N + tid
                                 : bc + static_cast<int64_t>(p.n_groups) * N + static_cast<int64_t>(g) * N + (tid - N);
    if (is_bc) {
        const float u = conv_channel<T>(p, cw, row, hist, false, c_bc, old);
        (tid < N ? B_s[tid] : C_s[tid - N]) = u;
    }
    for (int i = tid; i < (t1 - t0) * COLS; i += kThreads) {
        const int tile = t0 + i / COLS, h = (tile / per_head) * p.n_groups + g;
        const int64_t c = static_cast<int64_t>(h) * P + (tile % per_head) * COLS + (i % COLS);
        float mine[4];
        x_s[i] = conv_channel<T>(p, cw, row, hist, true, c, mine);
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (ranks > 1) cluster.barrier_arrive();  // this CTA has read the B and C history
    __syncthreads();

    for (int pass = 0; pass < passes; ++pass) {
        const int tile = t0 + pass * kTilesPerPass + warp / WPT;
        const bool live = tile < t1;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        int h = 0, col = 0;
        if (live) {
            h = (tile / per_head) * p.n_groups + g;
            col = (tile % per_head) * COLS + 4 * quad;
            const float dt = ssm_softplus(to_f<T>(static_cast<const T*>(p.a)[req * p.a_stride + h]) + __ldg(p.dt_bias + h));
            const float keep = expf(ssm_rate(__ldg(p.A_log + h)) * dt);
            const float4 x4 = *reinterpret_cast<const float4*>(&x_s[(tile - t0) * COLS + 4 * quad]);
            const float4 dx = make_float4(dt * x4.x, dt * x4.y, dt * x4.z, dt * x4.w);
            for (int round = 0; round < rounds; ++round) {
                const int k = round * 4 * kBatchRows;
#pragma unroll
                for (int i = 0; i < kBatchRows; ++i) v[i] = next[i];
                if (round + 1 < rounds) fetch(pass, round + 1);
                else if (pass + 1 < passes) fetch(pass + 1, 0);
                float* st = state_at(tile, k);
#pragma unroll
                for (int i = 0; i < kBatchRows; ++i) {
                    if (k + 4 * i >= share) break;
                    const float bn = B_s[n0 + k + 4 * i + sub], cn = C_s[n0 + k + 4 * i + sub];
                    v[i].x = fmaf(keep, v[i].x, bn * dx.x);
                    v[i].y = fmaf(keep, v[i].y, bn * dx.y);
                    v[i].z = fmaf(keep, v[i].z, bn * dx.z);
                    v[i].w = fmaf(keep, v[i].w, bn * dx.w);
                    acc.x = fmaf(cn, v[i].x, acc.x);
                    acc.y = fmaf(cn, v[i].y, acc.y);
                    acc.z = fmaf(cn, v[i].z, acc.z);
                    acc.w = fmaf(cn, v[i].w, acc.w);
                    __stcs(reinterpret_cast<float4*>(st + static_cast<int64_t>(4 * i) * P), v[i]);
                }
            }
#pragma unroll
            for (int off = 8; off < 32; off <<= 1) {
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
                acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
                acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
            }
        }
        if constexpr (WPT > 1) {
            if (lane < 8) part[warp][lane] = acc;
            __syncthreads();
            if (warp % WPT == 0) {
#pragma unroll
                for (int i = 1; i < WPT; ++i) {
                    const float4 o = part[warp + i][quad];
                    acc.x += o.x;
                    acc.y += o.y;
                    acc.z += o.z;
                    acc.w += o.w;
                }
            }
            __syncthreads();
        }
        if (live && warp % WPT == 0 && lane < 8) {
            const float D = p.D ? __ldg(p.D + h) : 0.f;
            const float4 x4 = *reinterpret_cast<const float4*>(&x_s[(tile - t0) * COLS + 4 * quad]);
            float o[4] = {fmaf(D, x4.x, acc.x), fmaf(D, x4.y, acc.y), fmaf(D, x4.z, acc.z), fmaf(D, x4.w, acc.w)};
            if (p.z) {
                const T* z = static_cast<const T*>(p.z) + req * p.z_stride + static_cast<int64_t>(h) * P + col;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] *= ssm_silu(to_f<T>(z[j]));
            }
            T* y = static_cast<T*>(p.y) + req * p.y_stride + static_cast<int64_t>(h) * P + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = from_f<T>(o[j]);
        }
    }
    if (ranks > 1) cluster.barrier_wait();
    if (rank == 0 && is_bc) {
        const int K = p.width;
#pragma unroll
        for (int j = 1; j < 3; ++j)
            if (j < K - 1) hist[(j - 1) * cw + c_bc] = from_f<T>(old[j]);
        hist[(K - 2) * cw + c_bc] = row[c_bc];
    }
}

template <class T, int WPT>
cudaError_t launch_w(const SsmStepParams& p, int ranks, cudaStream_t s) {
    const int tiles = p.n_heads / p.n_groups * (p.head_dim / COLS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, p.n_groups, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>((tiles + ranks - 1) / ranks) * COLS * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ssm_step_kernel<T, WPT>, p);
}

template <class T>
cudaError_t launch_t(const SsmStepParams& p, int sm_count, cudaStream_t s) {
    const int tiles = p.n_heads / p.n_groups * (p.head_dim / COLS);
    const int64_t all = static_cast<int64_t>(p.batch) * p.n_groups * tiles;
    // Warps to a tile.  With few tiles a lone request's loads should be in flight at once: 4,
    // or what 8 CTAs hold of a group in one pass (48 heads of 128 x 128, 12 tiles a group, 1
    // request: 1 / 2 / 4 warps 17.5 / 14.5 / 13.4 us; 32 tiles 16.5 / 13.4 / 13.4; 64 tiles
    // 15.5 / 16.6 / 17.6).  With many, as few as occupy a CTA's 8 warps (12 tiles, 64 requests:
    // 81 / 81 / 91 us; 4 tiles, 256: 64 / 56 / 64; 2 tiles, 256: 36 / 30 / 30).  They meet
    // between 8 requests of 12 tiles in 16 groups (22 / 20 / 22) and 16 (28 / 32 / 32).
    const bool few = all <= static_cast<int64_t>(sm_count) * 12;
    const int wpt = few ? (tiles <= 16 ? 4 : tiles <= 32 ? 2 : 1) : (tiles >= 8 ? 1 : tiles >= 3 ? 2 : 4);
    const int per_cta = kWarps / wpt, ranks = tiles >= 8 * per_cta ? 8 : (tiles + per_cta - 1) / per_cta;
    if (wpt == 4) return launch_w<T, 4>(p, ranks, s);
    if (wpt == 2) return launch_w<T, 2>(p, ranks, s);
    return launch_w<T, 1>(p, ranks, s);
}

}  // namespace

cudaError_t launch_ssm_step(const SsmStepParams& p, int sm_count, cudaStream_t s) {
    switch (p.dtype) {
        case GDN_F32: return launch_t<float>(p, sm_count, s);
        case GDN_BF16: return launch_t<__nv_bfloat16>(p, sm_count, s);
        default: return launch_t<__half>(p, sm_count, s);
    }
}

}  // namespace gdn
