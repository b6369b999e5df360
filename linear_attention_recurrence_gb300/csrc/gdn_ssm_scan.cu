// Selective state space scan over packed sequences, one token after the other.  Per
// head h, reading group h % n_groups, with S [state_dim][head_dim] in FP32:
//     dt = softplus(a[t][h] + dt_bias[h])
//     S <- exp(-exp(A_log[h]) dt) S + dt B_t x_t^T
//     y[t][h] = (S^T C_t + D[h] x_t) silu(z[t][h])
//
// This form takes every type and size; the tensor-core form (gdn_ssm_scan_tc.cu) takes
// long 16-bit prompts.  Bound by FP32 arithmetic: 3 packed operations per 2 state
// elements and token (decay, update, output), and by their latency where sequences x heads
// are few.  The columns of S are independent, so a CTA holds 32 columns of one head's state
// in registers: thread (row group rg, column pair cp) has 8 rows (4 or 2 of a small state)
// of 2 columns, packed along the rows, so B and C come as vectors from shared memory and
// serve both columns.  Tokens are staged in blocks of 16, double-buffered; there is no
// feedback from the output, so a block's partial sums over the row groups meet once per
// block (a shuffle, then one partial per warp in shared memory, in a fixed order).  A
// token's arithmetic does not depend on its place in the call: a sequence split over calls
// gives the same bits.  48 heads of 128 x 128 in FP32: 77 tokens 26 us, 2048 of one
// sequence 429 us, 8192 of 64 sequences 1066 us (30 TFLOP/s at 5 flop per state element
// and token).
#include "gdn_ssm.cuh"
#include "gdn_ssm.h"

namespace gdn {
namespace {

constexpr int TB = 16;   // tokens per staged block
constexpr int COLS = 32;  // state columns per CTA

// N consecutive elements: as vectors when ALIGNED, else one by one.
template <class T, int N, bool ALIGNED>
__device__ __forceinline__ void load_n(const T* p, float (&f)[N]) {
    constexpr int V = ALIGNED ? (N * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : N) : 1;
#pragma unroll
    for (int i = 0; i < N; i += V) {
        float g[V];
        load_vec<T, V>(p + i, g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[i + j] = g[j];
    }
}

// N: state_dim, NR: rows of it a thread holds.
template <class T, int N, int NR, bool ALIGNED>
__global__ void __launch_bounds__(N / NR * 16) ssm_scan_tokens_kernel(const SsmScanParams p, const SsmSeqs q) {
    constexpr int kThreads = N / NR * 16, kWarps = kThreads / 32;
    constexpr int TPT = kThreads / TB;               // threads that stage a token,
    constexpr int SN = N / TPT, SX = COLS / TPT;     // this many state rows and columns each
    static_assert(SN % 2 == 0 && SX % 2 == 0 && NR % 2 == 0, "staged and held in pairs");
    __shared__ __align__(16) float Bs[2][TB][N], Cs[2][TB][N], xs[2][TB][COLS], yp[kWarps][TB][COLS];
    __shared__ float2 gate[2][TB];  // decay, dt
    const int slices = p.head_dim / COLS;
    int64_t id = blockIdx.x;
    const int c0 = static_cast<int>(id % slices) * COLS;
    id /= slices;
    const int h = static_cast<int>(id % p.n_heads), s = static_cast<int>(id / p.n_heads);
    const int g = h % p.n_groups;
    int64_t b, e;
    seq_rows(q, s, b, e);
    if (b == e) return;  // a sequence without tokens leaves its slot as it is

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rg = tid >> 4, cp = tid & 15;
    const int lt = tid / TPT, lc = tid % TPT;
    const T* x = static_cast<const T*>(p.x) + static_cast<int64_t>(h) * p.head_dim + c0 + SX * lc;
    const T* z = p.z ? static_cast<const T*>(p.z) + static_cast<int64_t>(h) * p.head_dim + c0 + SX * lc : nullptr;
    T* y = static_cast<T*>(p.y) + static_cast<int64_t>(h) * p.head_dim + c0 + SX * lc;
    const T* Bp = static_cast<const T*>(p.B) + static_cast<int64_t>(g) * N + SN * lc;
    const T* Cp = static_cast<const T*>(p.C) + static_cast<int64_t>(g) * N + SN * lc;
    const T* ap = static_cast<const T*>(p.a) + h;
    const float A = ssm_rate(__ldg(p.A_log + h)), bias = __ldg(p.dt_bias + h), D = p.D ? __ldg(p.D + h) : 0.f;

    const int slot = p.states ? seq_slot(q, s) : -1;
    float* st = p.states + ((static_cast<int64_t>(slot) * p.n_heads + h) * N + NR * rg) * p.head_dim + c0 + 2 * cp;
    float2 S[2][NR / 2];
    const bool old = slot >= 0 && seq_has_state(q, s);
#pragma unroll
    for (int i = 0; i < NR / 2; ++i) {
        float2 u = make_float2(0.f, 0.f), v = u;
        if (old) {
            u = *reinterpret_cast<const float2*>(st + static_cast<int64_t>(2 * i) * p.head_dim);
            v = *reinterpret_cast<const float2*>(st + static_cast<int64_t>(2 * i + 1) * p.head_dim);
        }
        S[0][i] = make_float2(u.x, v.x);
        S[1][i] = make_float2(u.y, v.y);
    }

    float fb[SN], fc[SN], fx[SX], fz[SX];
    float2 fg = make_float2(1.f, 0.f);
    auto fetch = [&](int64_t t0) {
        const int64_t t = t0 + lt;
        if (t < e) {
            load_n<T, SN, ALIGNED>(Bp + t * p.b_stride, fb);
            load_n<T, SN, ALIGNED>(Cp + t * p.c_stride, fc);
            load_n<T, SX, ALIGNED>(x + t * p.x_stride, fx);
            if (z) load_n<T, SX, ALIGNED>(z + t * p.z_stride, fz);
        }
        if (tid < TB && t0 + tid < e) {
            const float dt = ssm_softplus(to_f<T>(ap[(t0 + tid) * p.a_stride]) + bias);
            fg = make_float2(expf(A * dt), dt);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < SN; i += 2) {
            *reinterpret_cast<float2*>(&Bs[buf][lt][SN * lc + i]) = make_float2(fb[i], fb[i + 1]);
            *reinterpret_cast<float2*>(&Cs[buf][lt][SN * lc + i]) = make_float2(fc[i], fc[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < SX; i += 2) *reinterpret_cast<float2*>(&xs[buf][lt][SX * lc + i]) = make_float2(fx[i], fx[i + 1]);
        if (tid < TB) gate[buf][tid] = fg;
    };
    fetch(b);
    stage(0);
    __syncthreads();
    int buf = 0;
    for (int64_t t0 = b; t0 < e; t0 += TB, buf ^= 1) {
        const int nv = e - t0 < TB ? static_cast<int>(e - t0) : TB;
        float dx[SX], zc[SX];  // this thread's outputs of the block: D x and z
#pragma unroll
        for (int j = 0; j < SX; ++j) {
            dx[j] = D * fx[j];
            zc[j] = fz[j];
        }
        const bool more = t0 + TB < e;
        if (more) fetch(t0 + TB);
        // one token: the state's update and this thread's part of its two outputs
        auto token = [&](int t, float& r0, float& r1) {
            const float2 gt = gate[buf][t];
            const float2 xv = *reinterpret_cast<const float2*>(&xs[buf][t][2 * cp]);
            const float2 a2 = make_float2(gt.x, gt.x);
            const float x0 = gt.y * xv.x, x1 = gt.y * xv.y;
            float2 y0 = make_float2(0.f, 0.f), y1 = y0;
            constexpr int W = NR >= 4 ? 4 : 2;  // rows per shared-memory load
#pragma unroll
            for (int i = 0; i < NR; i += W) {
                float bb[W], cc[W];
                if constexpr (W == 4) {
                    const float4 b4 = *reinterpret_cast<const float4*>(&Bs[buf][t][NR * rg + i]);
                    const float4 c4 = *reinterpret_cast<const float4*>(&Cs[buf][t][NR * rg + i]);
                    bb[0] = b4.x; bb[1] = b4.y; bb[2] = b4.z; bb[3] = b4.w;
                    cc[0] = c4.x; cc[1] = c4.y; cc[2] = c4.z; cc[3] = c4.w;
                } else {
                    const float2 b2 = *reinterpret_cast<const float2*>(&Bs[buf][t][NR * rg + i]);
                    const float2 c2 = *reinterpret_cast<const float2*>(&Cs[buf][t][NR * rg + i]);
                    bb[0] = b2.x; bb[1] = b2.y;
                    cc[0] = c2.x; cc[1] = c2.y;
                }
#pragma unroll
                for (int j = 0; j < W; j += 2) {
                    const float2 b2 = make_float2(bb[j], bb[j + 1]), c2 = make_float2(cc[j], cc[j + 1]);
                    float2 &s0 = S[0][(i + j) / 2], &s1 = S[1][(i + j) / 2];
                    s0 = ffma2(a2, s0, fmul2(b2, make_float2(x0, x0)));
                    s1 = ffma2(a2, s1, fmul2(b2, make_float2(x1, x1)));
                    y0 = ffma2(c2, s0, y0);
                    y1 = ffma2(c2, s1, y1);
                }
            }
            r0 = y0.x + y0.y;
            r1 = y1.x + y1.y;
        };
        // 4 tokens between the sums over the warp's two row groups, so that those overlap
        for (int t = 0; t < nv; t += 4) {
            float r0[4] = {}, r1[4] = {};
            if (t + 4 <= nv) {  // (no branch between the tokens: their loads move up)
#pragma unroll
                for (int k = 0; k < 4; ++k) token(t + k, r0[k], r1[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (t + k < nv) token(t + k, r0[k], r1[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                r0[k] += __shfl_xor_sync(0xffffffffu, r0[k], 16);
                r1[k] += __shfl_xor_sync(0xffffffffu, r1[k], 16);
                if (lane < 16) *reinterpret_cast<float2*>(&yp[warp][t + k][2 * cp]) = make_float2(r0[k], r1[k]);
            }
        }
        if (more) stage(buf ^ 1);
        __syncthreads();
        if (lt < nv) {
            float o[SX];
#pragma unroll
            for (int j = 0; j < SX; ++j) {
                const int k = SX * lc + j;
                float sum = yp[0][lt][k];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) sum += yp[w][lt][k];
                o[j] = sum + dx[j];
                if (z) o[j] *= ssm_silu(zc[j]);
            }
            T* out = y + (t0 + lt) * p.y_stride;
            if constexpr (ALIGNED) {
                store_vec<T, SX>(out, o);
            } else {
#pragma unroll
                for (int j = 0; j < SX; ++j) out[j] = from_f<T>(o[j]);
            }
        }
        __syncthreads();  // yp is read; the next block may overwrite it
    }
    if (slot >= 0) {
#pragma unroll
        for (int i = 0; i < NR / 2; ++i) {
            *reinterpret_cast<float2*>(st + static_cast<int64_t>(2 * i) * p.head_dim) = make_float2(S[0][i].x, S[1][i].x);
            *reinterpret_cast<float2*>(st + static_cast<int64_t>(2 * i + 1) * p.head_dim) =
                make_float2(S[0][i].y, S[1][i].y);
        }
    }
}

template <class T, int N, int NR>
void launch_n(const SsmScanParams& p, const SsmSeqs& q, cudaStream_t s) {
    // rows start on 16-byte boundaries: the pieces that threads stage are then aligned vectors
    auto fits = [](const void* ptr, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(ptr) | static_cast<uintptr_t>(stride * static_cast<int64_t>(sizeof(T)))) % 16 == 0;
    };
    const bool aligned = fits(p.x, p.x_stride) && fits(p.B, p.b_stride) && fits(p.C, p.c_stride) &&
                         fits(p.y, p.y_stride) && (!p.z || fits(p.z, p.z_stride));
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.n_seq) * p.n_heads * (p.head_dim / COLS));
    if (aligned)
        ssm_scan_tokens_kernel<T, N, NR, true><<<grid, N / NR * 16, 0, s>>>(p, q);
    else
        ssm_scan_tokens_kernel<T, N, NR, false><<<grid, N / NR * 16, 0, s>>>(p, q);
}

// Rows a thread holds of a large state: 8, so that a lone sequence's CTAs have 8 warps.  8 / 16
// rows (8 / 4 warps), FP32, 48 heads of 128 x 128, us: 77 tokens 26 / 32, 512 112 / 144, 2048
// 429 / 581, 2048 in 16 sequences 284 / 327, 8192 in 64 sequences 1066 / 1222.
constexpr int kRows = 8;
template <class T>
void launch_t(const SsmScanParams& p, const SsmSeqs& q, cudaStream_t s) {
    switch (p.state_dim) {
        case 16: launch_n<T, 16, 2>(p, q, s); break;
        case 32: launch_n<T, 32, 4>(p, q, s); break;
        case 64: launch_n<T, 64, kRows / 2>(p, q, s); break;
        default: launch_n<T, 128, kRows>(p, q, s); break;
    }
}

}  // namespace

cudaError_t launch_ssm_scan_tokens(const SsmScanParams& p, cudaStream_t s) {
    const SsmSeqs q{p.cu, p.slots, p.has_state, p.n_seq, p.n_slots, p.T};
    switch (p.dtype) {
        case GDN_F32: launch_t<float>(p, q, s); break;
        case GDN_BF16: launch_t<__nv_bfloat16>(p, q, s); break;
        default: launch_t<__half>(p, q, s); break;
    }
    return cudaGetLastError();
}

}  // namespace gdn
