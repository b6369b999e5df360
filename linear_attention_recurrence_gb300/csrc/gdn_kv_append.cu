// Appending keys and values to a paged 4-bit cache, rotated by position (sm_103a).
//
// A unit is 32 elements of one row (head) of one token: two groups of 16.  For rotated rows
// in halves the groups are elements 16 j .. and rotary / 2 + 16 j .., so a pair's two elements
// and a group's maximum are one thread's; otherwise they are 32 neighbours.
//
// Rotation: the angle is position * inv_freq, which in FP32 is off by the position's size, so
// it is formed as a fixed-point fraction of a turn: inv_freq / 2 pi to 64 bits after the point,
// times the position modulo 2^64 (whole turns fall away), its top 32 bits to sincospif.  A
// token's angles are formed once and shared by its heads through shared memory.
//
// Quantisation has one right answer (nearest, ties to even, of the exact quotient).  The FP32
// arithmetic is off by a few 2^-24 of the pair's size; where the two ends of its error interval
// round to different scales or codes, those are decided in FP64 (one group in some thousands).
// Ties, which 16-bit values without a rotation hit often, need none of it: see `quantise`.
//
// What bounds it: the latency of a unit's loads behind one another at 16 to 24 warps a
// multiprocessor (registers), then instructions (640 a unit and warp, issued in half the cycles), then
// memory. 48 + 2 x 16 heads of 128: 8191 tokens, 16 bits, 94 us (3.8 TB/s); 64 + 2 x 8 of 64, 2048 tokens
// of FP32 32 us; one token 10 us from launch to end. With whole groups done again in FP64 148, 82 and, for 250 tokens,
// 61 us (now 14): FP64 runs at a sixty-fourth of FP32's rate.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

struct Item {
    int64_t row;    // of the packed rows; -1: none
    int64_t place;  // in the cache: byte offset of the token's codes in KV head 0's keys, or -1
    int64_t pos;    // rotation
    int in_page;
};

// The sequence of row t: the last whose begin is not after it (all lanes of a warp together).
__device__ int seq_of(const KvSeqs& q, int64_t t) {
    if (!q.cu) return static_cast<int>(t / q.per_seq);
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = q.n_seq;  // cu[lo] <= t < cu[hi] where the bounds are sound
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const uint32_t before = __ballot_sync(0xffffffffu, at < hi && __ldg(q.cu + at) <= t);
        const int n = __popc(before);
        lo += n * step;
        if (lo + step < hi) hi = lo + step;
    }
    int64_t b, e;
    kv_rows(q, lo, b, e);
    return t >= b && t < e ? lo : -1;
}

// x >= 0 rounded to e4m3 (as a value), in FP64.
__device__ double e4m3_exact(double x) {
    if (!(x < 1e300)) return x != x ? x : 448.0;
    if (x == 0) return 0;
    int e = ilogb(x);
    e = e < -6 ? -6 : e;
    const double step = scalbn(1.0, e - 3), r = rint(x / step) * step;
    return r > 448.0 ? 448.0 : r;
}
// |x| rounded to e2m1: the code without its sign, in FP64.
__device__ uint32_t e2m1_exact(double x) {
    if (x >= 6.0) return 7;
    if (x >= 4.0) return static_cast<uint32_t>(rint(x / 2)) + 4;  // 4 -> 6, 6 -> 7
    if (x >= 2.0) return static_cast<uint32_t>(rint(x)) + 2;      // 2 -> 4, 3 -> 5, 4 -> 6
    return static_cast<uint32_t>(rint(x * 2));
}

__device__ __forceinline__ uint32_t e4m3x2(float hi, float lo) {
    uint32_t r;
    asm("{\n .reg .b16 h;\n cvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n mov.b32 %0, {h, h};\n}" : "=r"(r) : "f"(hi), "f"(lo));
    return r & 0xffff;
}
__device__ __forceinline__ uint32_t e2m1x2(float hi, float lo) {
    uint32_t r;
    asm("{\n .reg .b8 b;\n .reg .b16 h;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n mov.b16 h, {b, b};\n mov.b32 %0, {h, h};\n}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r & 0xff;
}

// 2^64 times inv_freq / 2 pi, modulo 2^64: 1 / 2 pi as the sum of two FP64 numbers, the
// product with its rounding error.
__device__ uint64_t turns_per_position(float inv_freq) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double x = inv_freq, p = x * kHi, e = fma(x, kHi, -p) + x * kLo;
    const double up = (p - floor(p)) * 4294967296.0, hi = floor(up);
    const double rest = ((up - hi) + e * 4294967296.0) * 4294967296.0;
    return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(static_cast<int64_t>(rest));
}

// Where one group comes from, for the exact path.
template <class T>
struct Source {
    const T* row;
    const float* inv_freq;
    int64_t pos;
    int first, rotary, interleaved;  // rotary 0: no rotation
};
// Element i of the group in FP64 (the angle to 2^-64 of a turn a position).
template <class T>
__device__ double exact_element(const Source<T>& s, int i) {
    const int e = s.first + i;
    const double x = to_f<T>(s.row[e]);
    if (e >= s.rotary) return x;
    const int half = s.rotary / 2;
    const int pair = s.interleaved ? e / 2 : e % half;
    const bool second = s.interleaved ? (e & 1) : e >= half;
    const double other = to_f<T>(s.row[s.interleaved ? (e ^ 1) : second ? e - half : e + half]);
    double sn, cs;
    sincospi(static_cast<double>(static_cast<int64_t>(static_cast<uint64_t>(s.pos) * turns_per_position(s.inv_freq[pair]))) * 0x1p-63,
             &sn, &cs);
    return second ? __dadd_rn(__dmul_rn(x, cs), __dmul_rn(other, sn)) : __dsub_rn(__dmul_rn(x, cs), __dmul_rn(other, sn));
}
// The group's scale byte, where `mask` has the elements that may be its largest.
template <class T>
__device__ __noinline__ uint32_t exact_scale(const Source<T>& s, uint32_t mask, float head_scale) {
    double top = 0;
    for (; mask; mask &= mask - 1) {
        const double y = exact_element(s, __ffs(mask) - 1);
        if (y != y) return 0x7f;
        top = fmax(top, fabs(y));
    }
    const double sc = e4m3_exact(top / (6.0 * static_cast<double>(head_scale)));
    if (sc != sc) return 0x7f;
    if (sc < 0.015625) return static_cast<uint32_t>(sc * 512);
    const int e = ilogb(sc);
    return static_cast<uint32_t>((e + 7) * 8 + static_cast<int>(scalbn(sc, 3 - e)) - 8);
}
// `codes` with those that differ in `diff` made right.
template <class T>
__device__ __noinline__ uint64_t exact_codes(const Source<T>& s, uint64_t codes, uint64_t diff, float scale, float head_scale) {
    const double by = static_cast<double>(scale) * static_cast<double>(head_scale);
    while (diff) {
        const int i = (__ffsll(static_cast<long long>(diff)) - 1) / 4;
        const double y = exact_element(s, i);
        const uint64_t c = e2m1_exact(fabs(y) / by) | (y < 0 ? 8u : 0u);
        codes = (codes & ~(uint64_t{15} << (4 * i))) | c << (4 * i);
        diff &= ~(uint64_t{15} << (4 * i));
    }
    return codes;
}

struct Held {
    uint64_t codes;
    uint32_t scale;  // e4m3
};

// Rounded to 17 significant bits.
__device__ __forceinline__ float snap(float v) { return __uint_as_float((__float_as_uint(v) + 0x40) & ~0x7fu); }

// One group: y within `err` of the exact values.  A NaN gives the scale NaN; an infinity the
// largest scale.
// Where nothing was rotated and the elements have 11 significant bits at most and the head's
// scale 5, a quotient that is no tie is 2^-12 of it away from one, and a computed one is 2^-21
// off at most: rounded to 17 bits it is the tie itself, or on its own side of it.
template <class T>
__device__ __forceinline__ Held quantise(const float (&y)[kKvGroup], float err, const Source<T>& s, float head_scale,
                                         float inv_scale) {
    uint32_t most = 0, bits = 0;  // (as integers: a NaN is above all)
#pragma unroll
    for (int i = 0; i < kKvGroup; ++i) {
        const uint32_t b = __float_as_uint(y[i]);
        most = max(most, b & 0x7fffffffu);
        bits |= b;
    }
    const bool exact = err == 0 && most < 0x7f800000u && (bits & 0x1fff) == 0 && (__float_as_uint(head_scale) & 0x7ffff) == 0;
    // the quotients are off by err / scale and three roundings
    const float off = exact ? 0.f : 0x1p-21f;
    const float f = inv_scale * (1.0f / 6.0f), a0 = __uint_as_float(most) * f, a = exact ? snap(a0) : a0;
    const float ea = fmaf(a, off, err * f);
    const uint32_t two = e4m3x2(a + ea, fmaxf(a - ea, 0.f));
    Held h;
    h.scale = two & 0xff;
    // (a head's scale far from 1: FP32's quotients and their bounds would leave its normal range)
    const bool far = !(inv_scale > 0x1p-100f && inv_scale < 0x1p100f);
    const bool odd = far || !(a < 1e30f) || !(err < 1e30f);
    if ((two >> 8) != h.scale || odd) {
        const float least = __uint_as_float(most) - 2 * err;
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < kKvGroup; ++i) mask |= odd || fabsf(y[i]) >= least ? 1u << i : 0u;
        h.scale = exact_scale(s, mask, head_scale);
    }
    const uint32_t sc16 = e4m3_to_f16(h.scale);
    const float sc = __half2float(__ushort_as_half(static_cast<unsigned short>(sc16 & 0xffff)));
    const float inv = sc > 0 ? __fdividef(inv_scale, sc) : 0.f;
    const float e0 = err * inv;
    uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kKvGroup; i += 2) {
        float u = y[i] * inv, w = y[i + 1] * inv;
        if (exact) u = snap(u), w = snap(w);
        const float eu = fmaf(fabsf(u), off, e0), ew = fmaf(fabsf(w), off, e0);
        lo[i / 8] |= e2m1x2(w - ew, u - eu) << (4 * (i & 7));
        hi[i / 8] |= e2m1x2(w + ew, u + eu) << (4 * (i & 7));
    }
    h.codes = sc > 0 ? (static_cast<uint64_t>(lo[1]) << 32 | lo[0]) : 0;
    const uint64_t open = far ? ~uint64_t{0} : static_cast<uint64_t>(lo[1] ^ hi[1]) << 32 | (lo[0] ^ hi[0]);
    if (open && sc > 0) h.codes = exact_codes(s, h.codes, open, sc, head_scale);
    return h;
}

template <class T, int N>
__device__ __forceinline__ void load_n(const T* p, bool vector, float (&f)[N]) {
    constexpr int V = 16 / sizeof(T);
    if (vector) {
#pragma unroll
        for (int i = 0; i < N; i += V) {
            float g[V];
            load_vec<T, V>(p + i, g);
#pragma unroll
            for (int k = 0; k < V; ++k) f[i + k] = g[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f<T>(p[i]);
    }
}
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, bool vector, const float (&f)[N]) {
    constexpr int V = 16 / sizeof(T);
    if (vector) {
#pragma unroll
        for (int i = 0; i < N; i += V) {
            float g[V];
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = f[i + k];
            store_vec<T, V>(p + i, g);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = from_f<T>(f[i]);
    }
}

// A CTA takes `per_cta` tokens and the units [blockIdx.y, + gridDim.y, ...) x kThreads of each.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p, int per_cta) {
    extern __shared__ float2 turn[];  // [per_cta][rotary / 2]: cos, sin
    __shared__ Item items[8];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_cta;
    const int half = p.rotary / 2;
    if (warp < per_cta) {
        Item it{-1, -1, 0, 0};
        const int64_t t = t0 + warp;
        if (t < p.s.T) {
            const int s = seq_of(p.s, t);
            if (s >= 0) {
                int64_t b, e;
                kv_rows(p.s, s, b, e);
                const int64_t at = __ldg(p.s.kv_lens + s) - (e - t);
                const int64_t page = kv_page(p.s, s, at);
                it.row = t;
                it.pos = p.positions ? __ldg(p.positions + t) : at;
                it.in_page = static_cast<int>(at & ((int64_t{1} << p.s.page_log2) - 1));
                if (page >= 0) it.place = page * p.n_kv * 2 * kv_plane(p.s.page_log2, D);
            }
        }
        if ((tid & 31) == 0) items[warp] = it;
    }
    __syncthreads();
    for (int i = tid; i < per_cta * half; i += kThreads) {
        const int k = i / half, j = i - k * half;
        const uint64_t a = static_cast<uint64_t>(items[k].pos) * turns_per_position(__ldg(p.inv_freq + j));
        // the nearest 32-bit fraction of a turn, in [-1/2, 1/2), as an FP32 number and its rest
        const int32_t top = static_cast<int32_t>((a + 0x80000000ull) >> 32);
        const float near = static_cast<float>(top);
        const float rest = static_cast<float>(static_cast<int64_t>(top) - static_cast<int64_t>(near)) * (6.2831853f * 0x1p-32f);
        float sn, cs;
        sincospif(near * 0x1p-31f, &sn, &cs);
        turn[i] = make_float2(fmaf(-sn, rest, cs), fmaf(cs, rest, sn));
    }
    __syncthreads();
    constexpr int U = D / 32;  // units of a row
    const int q_units = p.q ? p.n_heads * U : 0, kv_units = p.n_kv * U;
    const int units = q_units + 2 * kv_units;
    for (int x = blockIdx.y * kThreads + tid; x < per_cta * units; x += gridDim.y * kThreads) {
        const int k = x / units;
        int u = x - k * units;
        const Item it = items[k];
        if (it.row < 0) continue;
        const int kind = u < q_units ? 0 : u < q_units + kv_units ? 1 : 2;  // q, k, v
        u -= kind == 0 ? 0 : q_units + (kind == 2 ? kv_units : 0);
        const int head = u / U, j = u - head * U;
        const T* src = kind == 0   ? static_cast<const T*>(p.q) + it.row * p.q_stride
                       : kind == 1 ? static_cast<const T*>(p.k) + it.row * p.k_stride
                                   : static_cast<const T*>(p.v) + it.row * p.v_stride;
        src += head * D;
        const int rotary = kind == 2 ? 0 : p.rotary;
        const bool in_halves = !p.interleaved && 32 * j < rotary;
        const int first[2] = {in_halves ? 16 * j : 32 * j, in_halves ? half + 16 * j : 32 * j + 16};
        float a[kKvGroup], b[kKvGroup];
        load_n<T>(src + first[0], p.vector, a);
        load_n<T>(src + first[1], p.vector, b);
        float err[2] = {0, 0};  // bounds of the rotation's error
        if (32 * j < rotary) {
            const float2* cs = turn + k * half;
            float size = 0;
            if (in_halves) {
#pragma unroll
                for (int i = 0; i < kKvGroup; ++i) {
                    const float2 c = cs[16 * j + i];
                    const float m = a[i], n = b[i];
                    a[i] = m * c.x - n * c.y;
                    b[i] = n * c.x + m * c.y;
                    size = fmaxf(size, fabsf(m) + fabsf(n));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kKvGroup; i += 2) {
                    const float2 c = cs[16 * j + i / 2], d = cs[16 * j + 8 + i / 2];
                    const float m = a[i], n = a[i + 1], r = b[i], s = b[i + 1];
                    a[i] = m * c.x - n * c.y;
                    a[i + 1] = n * c.x + m * c.y;
                    b[i] = r * d.x - s * d.y;
                    b[i + 1] = s * d.x + r * d.y;
                    size = fmaxf(size, fmaxf(fabsf(m) + fabsf(n), fabsf(r) + fabsf(s)));
                }
            }
            // the sine and cosine are good to 1 ulp of the function and half of one of the correction, the
            // angle to 2^-32 of a turn; products and sum are rounded: 2^-22.5 of the pair's size
            err[0] = err[1] = size * 0x1p-22f;
        }
        if (kind == 0) {
            T* dst = static_cast<T*>(p.q_out) + it.row * p.q_out_stride + head * D;
            store_n<T>(dst + first[0], p.vector, a);
            store_n<T>(dst + first[1], p.vector, b);
            continue;
        }
        const float* scales = kind == 1 ? p.k_scale : p.v_scale;
        const float hs = scales ? __ldg(scales + head) : 1.0f, inv = 1.0f / hs;
        const Source<T> sa{src, p.inv_freq, it.pos, first[0], rotary, p.interleaved};
        const Source<T> sb{src, p.inv_freq, it.pos, first[1], rotary, p.interleaved};
        const Held held[2] = {quantise(a, err[0], sa, hs, inv), quantise(b, err[1], sb, hs, inv)};
        if (it.place >= 0) {
            const int64_t plane = kv_plane(p.s.page_log2, D);
            uint8_t* at = p.cache + it.place + (2 * head + kind - 1) * plane;
            uint8_t* scale_at = at + ((int64_t{D / 2} << p.s.page_log2) + it.in_page * (D / kKvGroup));
            at += it.in_page * (D / 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<uint64_t*>(at + first[i] / 2) = held[i].codes;
                scale_at[first[i] / kKvGroup] = static_cast<uint8_t>(held[i].scale);
            }
        }
        void* kept = kind == 1 ? p.k_out : p.v_out;
        if (kept) {
            T* dst = static_cast<T*>(kept) + it.row * (kind == 1 ? p.k_out_stride : p.v_out_stride) + head * D;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t sc = e4m3_to_f16(held[i].scale);
                const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sc & 0xffff)));
                float f[kKvGroup];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t r[4];
                    e2m1_to_f16(static_cast<uint32_t>(held[i].codes >> (32 * w)), r);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r[n]));
                        f[8 * w + 2 * n] = v.x * s * hs;
                        f[8 * w + 2 * n + 1] = v.y * s * hs;
                    }
                }
                store_n<T>(dst + first[i], p.vector, f);
            }
        }
    }
}

template <class T, int D>
cudaError_t launch(const KvAppendParams& p, int sm_count, cudaStream_t s) {
    const int units = ((p.q ? p.n_heads : 0) + 2 * p.n_kv) * (D / 32);
    // several tokens a CTA where there are tokens for all multiprocessors, which share its start (2048
    // tokens of FP32: 4 a CTA 33 us, 1 41; 8191 of FP16: 4 96, 2 107), a token's units over several CTAs
    // where there are few
    int per = 1;
    while (per < 4 && p.s.T >= static_cast<int64_t>(sm_count) * 4 * per) per *= 2;
    const int64_t x = (p.s.T + per - 1) / per;
    const int pieces = (per * units + kThreads - 1) / kThreads;
    int y = 1;
    while (y < pieces && x * y < 2 * sm_count) ++y;
    kv_append_kernel<T, D><<<dim3(static_cast<unsigned>(x), y), kThreads, per * (p.rotary / 2) * sizeof(float2), s>>>(p, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int sm_count, cudaStream_t s) {
    const bool wide = p.head_dim == 128;
    if (p.dtype == GDN_F32) return wide ? launch<float, 128>(p, sm_count, s) : launch<float, 64>(p, sm_count, s);
    if (p.dtype == GDN_BF16)
        return wide ? launch<__nv_bfloat16, 128>(p, sm_count, s) : launch<__nv_bfloat16, 64>(p, sm_count, s);
    return wide ? launch<__half, 128>(p, sm_count, s) : launch<__half, 64>(p, sm_count, s);
}

}  // namespace gdn
