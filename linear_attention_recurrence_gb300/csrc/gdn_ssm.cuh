// Shared by the selective state space kernels and the block norm: the activation
// types, 16-byte (and narrower) vectors of them, the gate functions, and the reading
// of packed sequences and state slots.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "gdn_device.cuh"

namespace gdn {

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

// Round to nearest even, once, from FP32.
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// N elements of T that one access moves (N * sizeof(T) <= 32 bytes, a power of two;
// 32 bytes are two 16-byte accesses).
template <class T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Vec {
    T v[N];
};
template <class T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[N]) {
    const Vec<T, N> x = *reinterpret_cast<const Vec<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f<T>(x.v[i]);
}
template <class T, int N>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[N]) {
    Vec<T, N> x;
    if constexpr (N > 1 && sizeof(T) == 2) {  // two roundings per instruction
        uint32_t* u = reinterpret_cast<uint32_t*>(x.v);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(f[i], f[i + 1]);
                u[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[i], f[i + 1]);
                u[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x.v[i] = from_f<T>(f[i]);
    }
    *reinterpret_cast<Vec<T, N>*>(p) = x;
}

constexpr float kLog2e = 1.4426950408889634f;

// The hardware's 2^v and 1 / v (relative error below 2^-22 and 2^-23; subnormals are 0).
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// The hardware's log2 v (off by 2^-22, outside (0.5, 2) of itself; of a subnormal -infinity).
__device__ __forceinline__ float lg2(float v) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    return upk(r);
}
// sigmoid(z) = 1 / (1 + 2^(-z log2 e)) and silu(z) = z sigmoid(z) (an infinite divisor
// gives 0), and silu of two: the same operations, the same bits.
__device__ __forceinline__ float ssm_sigmoid(float z) { return rcp(1.0f + ex2(__fmul_rn(z, -kLog2e))); }
__device__ __forceinline__ float ssm_silu(float z) { return z * ssm_sigmoid(z); }
__device__ __forceinline__ float2 silu2(float2 z) {
    const float2 m = fmul2(z, make_float2(-kLog2e, -kLog2e));
    const float2 d = fadd2(make_float2(ex2(m.x), ex2(m.y)), make_float2(1.f, 1.f));
    return fmul2(z, make_float2(rcp(d.x), rcp(d.y)));
}

// softplus(v) = log(1 + e^v), accurate for small e^v too (log1p); v itself once e^-v
// is below half an FP32 ulp of v.
__device__ __forceinline__ float ssm_softplus(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

// -exp(A_log), finite (so that no step, dt = 0, stays no decay).
__device__ __forceinline__ float ssm_rate(float A_log) { return fmaxf(-expf(A_log), -3.402823466e38f); }

// A token's decay is e^g = 2^(g log2 e).  The exponent is held at -256 or above: such a
// factor is 0 in FP32 either way, and running sums of the exponents stay finite.
constexpr float kMinLog2Decay = -256.0f;

// The packed sequences of a call: sequence s has rows [begin, end) of the packed rows.
// A bound outside [0, T], or an end below its begin, gives an empty sequence, so every row
// that a sequence has is one of the arrays'.  Bounds that decrease between sequences can make
// them overlap or put them out of order, which no kernel looks for: what they leave is
// undefined, so each holds what it derives from other sequences' bounds (a window's rows, a
// unit's number) to its own arrays.
struct SsmSeqs {
    const int32_t* cu;         // [n_seq + 1], or nullptr: one sequence of T rows
    const int32_t* slots;      // [n_seq], or nullptr: sequence s has slot s
    const uint8_t* has_state;  // [n_seq], or nullptr: every sequence continues from its slot
    int n_seq;
    int n_slots;
    int64_t T;
};
__device__ __forceinline__ void seq_rows(const SsmSeqs& q, int s, int64_t& begin, int64_t& end) {
    begin = 0;
    end = q.T;
    if (q.cu) {
        begin = __ldg(q.cu + s);
        end = __ldg(q.cu + s + 1);
        if (begin < 0 || end > q.T || end < begin) end = begin = 0;
    }
}
// The slot of sequence s, or -1 if it has none (negative or out of range).
__device__ __forceinline__ int seq_slot(const SsmSeqs& q, int s) {
    const int slot = q.slots ? __ldg(q.slots + s) : s;
    return slot >= 0 && slot < q.n_slots ? slot : -1;
}
__device__ __forceinline__ bool seq_has_state(const SsmSeqs& q, int s) {
    return !q.has_state || __ldg(q.has_state + s) != 0;
}

}  // namespace gdn
