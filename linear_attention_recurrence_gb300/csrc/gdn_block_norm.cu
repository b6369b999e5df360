// The norms around a block in one pass over the residual stream.  Per token:
//     u = b rsqrt(mean(b^2) + eps) w_post     (b itself without w_post)
//     r' = r + scale act(gate) u              (act: the sigmoid or none; gate 1 without it)
//     y = r' rsqrt(mean(r'^2) + eps) w_pre
//
// Bound by HBM: b, r and a per-token gate are read once, r' and y written once.  One CTA
// per token keeps its row in registers in FP32 (E elements a thread) across the two
// sums, which meet in a shuffle butterfly and one exchange between warps, in a fixed
// order.  y is formed from r' before r' is rounded to the stream's type.
#include "gdn_ssm.cuh"
#include "gdn_ssm.h"

namespace gdn {
namespace {

template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += red[i];
    }
    return v;
}

// T: block and output type, R: stream type; VEC elements per access, NV accesses a thread.
template <class T, class R, int VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const BlockNormParams p) {
    __shared__ float red[2][32];
    const int64_t t = blockIdx.x;
    const int d = p.dim;
    const T* b = static_cast<const T*>(p.b) + t * p.b_stride;
    const R* r = static_cast<const R*>(p.r) + t * p.r_stride;
    const T* gate = p.gate ? static_cast<const T*>(p.gate) + t * p.gate_stride : nullptr;
    R* r_out = static_cast<R*>(p.r_out) + t * p.r_out_stride;
    T* y = static_cast<T*>(p.y) + t * p.y_stride;
    const float inv_d = 1.0f / static_cast<float>(d);

    float u[NV][VEC], x[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * THREADS + threadIdx.x) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) u[i][v] = x[i][v] = 0.f;
        if (c < d) {
            load_vec<T, VEC>(b + c, u[i]);
            load_vec<R, VEC>(r + c, x[i]);
        }
    }
    float f = p.scale;
    if (p.w_post) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) ss = fmaf(u[i][v], u[i][v], ss);
        ss = block_sum<THREADS / 32>(ss, red[0]);
        f *= rsqrtf(fmaf(ss, inv_d, p.eps));
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * THREADS + threadIdx.x) * VEC;
        if (c < d) {
            float w[VEC], gt[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) w[v] = gt[v] = 1.f;
            if (p.w_post) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) w[v] = __ldg(p.w_post + c + v);
            }
            if (gate) {
                load_vec<T, VEC>(gate + c, gt);
                if (p.gate_sigmoid) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) gt[v] = __fdividef(1.0f, 1.0f + __expf(-gt[v]));
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                x[i][v] = fmaf(f * u[i][v], w[v] * gt[v], x[i][v]);
                ss = fmaf(x[i][v], x[i][v], ss);
            }
            store_vec<R, VEC>(r_out + c, x[i]);
        }
    }
    ss = block_sum<THREADS / 32>(ss, red[1]);
    const float q = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * THREADS + threadIdx.x) * VEC;
        if (c < d) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[i][v] *= q * __ldg(p.w_pre + c + v);
            store_vec<T, VEC>(y + c, x[i]);
        }
    }
}

template <class T, class R, int VEC, int THREADS>
void launch_n(const BlockNormParams& p, cudaStream_t s) {
    const int nv = (p.dim + VEC * THREADS - 1) / (VEC * THREADS);
    const unsigned grid = static_cast<unsigned>(p.T);
    // the number of accesses a thread makes, rounded up to an instance
    if (nv <= 1) block_norm_kernel<T, R, VEC, 1, THREADS><<<grid, THREADS, 0, s>>>(p);
    else if (nv <= 2) block_norm_kernel<T, R, VEC, 2, THREADS><<<grid, THREADS, 0, s>>>(p);
    else if (nv <= 3) block_norm_kernel<T, R, VEC, 3, THREADS><<<grid, THREADS, 0, s>>>(p);
    else if (VEC >= 4 || nv <= 4) block_norm_kernel<T, R, VEC, 4, THREADS><<<grid, THREADS, 0, s>>>(p);
    else if constexpr (VEC < 4) {
        // narrow rows' widest: 16 single elements or 8 pairs a thread (dim <= 16384)
        if (VEC == 2 || nv <= 8) block_norm_kernel<T, R, VEC, 8, THREADS><<<grid, THREADS, 0, s>>>(p);
        else block_norm_kernel<T, R, VEC, 16, THREADS><<<grid, THREADS, 0, s>>>(p);
    }
}

template <class T, class R, int VEC>
void launch_v(const BlockNormParams& p, cudaStream_t s) {
    // 4 accesses of a thread at most: 256 threads while they reach, then 1024
    if (p.dim <= VEC * 256 * 4) launch_n<T, R, VEC, 256>(p, s);
    else launch_n<T, R, VEC, 1024>(p, s);
}

template <class T, class R>
void launch_r(const BlockNormParams& p, cudaStream_t s) {
    if (p.vec >= 8) launch_v<T, R, 8>(p, s);
    else if (p.vec >= 4) launch_v<T, R, 4>(p, s);
    else if (p.vec >= 2) launch_v<T, R, 2>(p, s);
    else launch_v<T, R, 1>(p, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, cudaStream_t s) {
    const bool wide = p.stream_dtype == GDN_F32;
    switch (p.dtype) {
        case GDN_F32: launch_r<float, float>(p, s); break;
        case GDN_BF16:
            if (wide) launch_r<__nv_bfloat16, float>(p, s);
            else launch_r<__nv_bfloat16, __nv_bfloat16>(p, s);
            break;
        default:
            if (wide) launch_r<__half, float>(p, s);
            else launch_r<__half, __half>(p, s);
            break;
    }
    return cudaGetLastError();
}

}  // namespace gdn
