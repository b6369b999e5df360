// The norms around a block in one pass over the residual stream.  Per token:
//     u = b rsqrt(mean(b^2) + eps) w_post     (b itself without w_post)
//     r' = r + scale act(gate) u              (act: the sigmoid or none; gate 1 without it)
//     y = r' rsqrt(mean(r'^2) + eps) w_pre
//
// Bound by HBM: b, r and a per-token gate are read once, r' and y written once.  A CTA
// takes a token at a time and keeps its row in registers in FP32 across the two sums,
// which meet in a shuffle butterfly and one exchange between warps, in a fixed order.  y
// is formed from r' before r' is rounded to the stream's type.  The sums' order goes by the
// widest access that the rows allow and by the number of threads, which for rows of 513
// to 1024 accesses goes by T <= SMs: another T can give a token other last bits.  Two forms:
// one CTA per token reading its row itself (short rows, rows off 16-byte boundaries, rows
// longer than the other form holds), and CTAs that stay, the weights in registers, while
// bulk copies bring their next rows into shared memory (the two sums of a row leave memory
// idle otherwise).  8192 x 6144 (BF16, FP32 stream, a gate per token) takes 118 us, 6.0 TB/s.
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
                    for (int v = 0; v < VEC; ++v) gt[v] = ssm_sigmoid(gt[v]);
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

// Rows through shared memory.  `stages` rows are in flight per CTA; a stage holds a row
// of b, of r and (per-token gate) of the gate.
constexpr int kRowThreads = 256, kMaxStages = 8;
template <class T, class R, int NV>
__global__ void __launch_bounds__(kRowThreads, 2) block_norm_rows_kernel(const BlockNormParams p, int stages, uint32_t stage_bytes) {
    constexpr int VEC = 8;
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t full[kMaxStages];
    unsigned char* sm = aligned_dynamic_smem<unsigned char, 128>();
    const int tid = threadIdx.x, d = p.dim;
    const bool token_gate = p.gate && p.gate_stride != 0;
    const uint32_t b_bytes = d * sizeof(T), r_bytes = d * sizeof(R);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
        mbar_init_fence();
    }
    __syncthreads();
    auto fetch = [&](int64_t t, int s) {  // thread 0
        unsigned char* at = sm + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], b_bytes + r_bytes + (token_gate ? b_bytes : 0));
        bulk_load(at, static_cast<const T*>(p.b) + t * p.b_stride, b_bytes, &full[s]);
        bulk_load(at + b_bytes, static_cast<const R*>(p.r) + t * p.r_stride, r_bytes, &full[s]);
        if (token_gate) bulk_load(at + b_bytes + r_bytes, static_cast<const T*>(p.gate) + t * p.gate_stride, b_bytes, &full[s]);
    };
    if (tid == 0)
        for (int i = 0; i < stages; ++i) {
            const int64_t t = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
            if (t < p.T) fetch(t, i);
        }
    float wq[NV][VEC], wp[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * kRowThreads + tid) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            wq[i][v] = p.w_post && c < d ? __ldg(p.w_post + c + v) : 1.f;
            wp[i][v] = c < d ? __ldg(p.w_pre + c + v) : 0.f;
        }
    }
    const float inv_d = 1.0f / static_cast<float>(d);
    int s = 0;
    uint32_t phase = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        bool ok = false;
        for (uint32_t n = 0; n < kWaitPolls && !ok; ++n) ok = mbar_try_wait(&full[s], phase);
        if (!ok) {  // (threads that leave count as arrived at the barriers below)
            report_error(p.status, kDevErrBlockNorm);
            if (tid == 0)  // the copies in flight land before the CTA's shared memory is another's
                for (int i = 0; i < stages && t + i * static_cast<int64_t>(gridDim.x) < p.T; ++i) {
                    const bool wrapped = s + i >= stages;
                    mbar_wait(&full[wrapped ? s + i - stages : s + i], phase ^ (wrapped ? 1 : 0));
                }
            return;
        }
        const T* b = reinterpret_cast<const T*>(sm + s * stage_bytes);
        const R* r = reinterpret_cast<const R*>(sm + s * stage_bytes + b_bytes);
        const T* gate = token_gate ? reinterpret_cast<const T*>(sm + s * stage_bytes + b_bytes + r_bytes) : static_cast<const T*>(p.gate);
        R* r_out = static_cast<R*>(p.r_out) + t * p.r_out_stride;
        T* y = static_cast<T*>(p.y) + t * p.y_stride;
        float u[NV][VEC], x[NV][VEC];
        float ss = 0.f, f = p.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * kRowThreads + tid) * VEC;
#pragma unroll
            for (int v = 0; v < VEC; ++v) u[i][v] = 0.f;
            if (c < d) load_vec<T, VEC>(b + c, u[i]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) ss = fmaf(u[i][v], u[i][v], ss);
        }
        if (p.w_post) {
            ss = block_sum<kRowThreads / 32>(ss, red[0]);
            f *= rsqrtf(fmaf(ss, inv_d, p.eps));
        }
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * kRowThreads + tid) * VEC;
            if (c < d) {
                float gt[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) gt[v] = 1.f;
                if (gate) {
                    load_vec<T, VEC>(gate + c, gt);
                    if (p.gate_sigmoid) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) gt[v] = ssm_sigmoid(gt[v]);
                    }
                }
                load_vec<R, VEC>(r + c, x[i]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    x[i][v] = fmaf(f * u[i][v], wq[i][v] * gt[v], x[i][v]);
                    ss = fmaf(x[i][v], x[i][v], ss);
                }
                store_vec<R, VEC>(r_out + c, x[i]);
            }
        }
        ss = block_sum<kRowThreads / 32>(ss, red[1]);  // behind its barrier the stage is read
        if (tid == 0) {
            const int64_t next = t + static_cast<int64_t>(stages) * gridDim.x;
            if (next < p.T) fetch(next, s);
        }
        const float q = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * kRowThreads + tid) * VEC;
            if (c < d) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[i][v] *= q * wp[i][v];
                store_vec<T, VEC>(y + c, x[i]);
            }
        }
        if (!p.w_post) __syncthreads();  // red[1] is read before the next row writes it
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
}

template <class T, class R, int NV>
cudaError_t launch_rows(const BlockNormParams& p, int sm_count, cudaStream_t s) {
    const uint32_t bytes = static_cast<uint32_t>(p.dim) * (sizeof(T) * (p.gate && p.gate_stride ? 2 : 1) + sizeof(R));
    const uint32_t stage = (bytes + 127) / 128 * 128;
    int stages = static_cast<int>(100u * 1024 / stage);
    if (stages > kMaxStages) stages = kMaxStages;
    const int smem = static_cast<int>(stage) * stages + 128;
    const void* k = reinterpret_cast<const void*>(block_norm_rows_kernel<T, R, NV>);
    cudaError_t e = set_smem_once(k, 101 * 1024);
    if (e != cudaSuccess) return e;
    const int64_t grid = p.T < 2 * sm_count ? p.T : 2 * sm_count;
    block_norm_rows_kernel<T, R, NV><<<static_cast<unsigned>(grid), kRowThreads, smem, s>>>(p, stages, stage);
    return cudaGetLastError();
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
void launch_v(const BlockNormParams& p, int sm_count, cudaStream_t s) {
    // 4 accesses of a thread at most: 256 threads while they reach, then 1024; 1024 too where a
    // lone row would take 256 threads 3 or 4 accesses (8192 elements, BF16, FP32 stream, 256 /
    // 1024 threads: 1 token 14.5 / 10.4 us, 152 14.5 / 12.5, 304 16.6 / 19.6, 2432 87 / 95;
    // 4096 elements: 1 token 4.0 / 4.0).
    if (p.dim <= VEC * 256 * (p.T <= sm_count ? 2 : 4)) launch_n<T, R, VEC, 256>(p, s);
    else launch_n<T, R, VEC, 1024>(p, s);
}

template <class T, class R>
cudaError_t launch_r(const BlockNormParams& p, int sm_count, cudaStream_t s) {
    const int nv = (p.dim + 8 * kRowThreads - 1) / (8 * kRowThreads);
    // Rows of whole 16-byte pieces, at most 3 accesses of 8 elements a thread (the weights stay
    // in registers) and 1024 elements.  One CTA per token / this form, us, BF16, FP32 stream
    // and a gate per token: 512 elements: 1 token 2.3 / 2.7, 8192 32 / 32; 1024: 2.5 / 2.7,
    // 40 / 34; 2048: 2.8 / 2.8, 58 / 46; 6144: 5.0 / 4.7, 171 / 118.
    if (p.vec == 8 && p.dim >= 1024 && nv <= 3) {
        if (nv == 1) return launch_rows<T, R, 1>(p, sm_count, s);
        if (nv == 2) return launch_rows<T, R, 2>(p, sm_count, s);
        return launch_rows<T, R, 3>(p, sm_count, s);
    }
    if (p.vec >= 8) launch_v<T, R, 8>(p, sm_count, s);
    else if (p.vec >= 4) launch_v<T, R, 4>(p, sm_count, s);
    else if (p.vec >= 2) launch_v<T, R, 2>(p, sm_count, s);
    else launch_v<T, R, 1>(p, sm_count, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, int sm_count, cudaStream_t s) {
    const bool wide = p.stream_dtype == GDN_F32;
    switch (p.dtype) {
        case GDN_F32: return launch_r<float, float>(p, sm_count, s);
        case GDN_BF16:
            return wide ? launch_r<__nv_bfloat16, float>(p, sm_count, s) : launch_r<__nv_bfloat16, __nv_bfloat16>(p, sm_count, s);
        default: return wide ? launch_r<__half, float>(p, sm_count, s) : launch_r<__half, __half>(p, sm_count, s);
    }
}

}  // namespace gdn
