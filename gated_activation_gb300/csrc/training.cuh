// Internal helpers of the training operators (checkpoint.cu, layer_norm.cu,
// balance.cu): element types, the activations with their derivatives, the
// 8-bit block format, and the host side's argument checks.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "gated_act_training.h"

namespace gact {

// ---------------------------------------------------------------- elements

using bf16 = __nv_bfloat16;
using f16 = __half;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(f16 x) { return __half2float(x); }

template <class T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_float<bf16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ f16 from_float<f16>(float x) { return __float2half_rn(x); }

// ------------------------------------------------------------- activations

// Both activations are g sigma(a) with a = a(g), and their slope is
// sigma (1 + g (1 - sigma) a').  With t = e^{-|a|}, sigma and 1 - sigma are
// 1 / (1 + t) and t / (1 + t) in one order or the other: no cancellation.  t is
// the square of h = 2^{-|a| log2(e) / 2}, which the flushing hardware
// exponential (PTX ISA ex2.approx.ftz.f32, relative error about 2^-22) keeps
// normal for |a| < 174; 1 + t lies in [1, 2], where the hardware reciprocal
// is within one ulp.  sigma is handed on as the product s1 s2 (h / (1 + t)
// and h for a < 0), s2 to be multiplied last: then nothing but a result itself
// can fall below fp32's normal range.
struct Gate {
    float s1, s2;   // sigma = s1 s2
    float w;        // slope = sigma w
};
__device__ __forceinline__ Gate gate_of(float a, float g_slope) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fabsf(a) * (-0.5f * 1.4426950408889634f)));
    const float t = h * h;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    const bool up = a >= 0.f;
    Gate m;
    m.s2 = up ? 1.f : h;
    m.s1 = r * m.s2;
    m.w = fmaf(g_slope, up ? t * r : r, 1.f);
    return m;
}

struct Silu {
    __device__ static Gate gate(float g) { return gate_of(g, g); }
};

// a = 2 sqrt(2/pi) (g + 0.044715 g^3).  g a' is taken at most at |g| = 16,
// where it cannot overflow: past |g| = 11, t is 0 and so is its factor (a > 0)
// or sigma (a < 0).
struct Gelu {
    static constexpr float k2 = 2.0f * 0.7978845608028654f;
    static constexpr float k2c = 2.0f * 0.7978845608028654f * 0.044715f;
    __device__ static Gate gate(float g) {
        const float b = fminf(fmaxf(g, -16.f), 16.f);
        return gate_of(g * fmaf(k2c, g * g, k2), b * fmaf(3.f * k2c, b * b, k2));
    }
};

// gelu_tanh(s) u for s >= 0 or NaN.
__device__ __forceinline__ float gelu_mul(float s, float u) {
    const Gate m = Gelu::gate(s);
    return s * m.s1 * u;
}

// act(g) u
template <class Act> __device__ __forceinline__ float act_mul(float g, float u) {
    const Gate m = Act::gate(g);
    return g * m.s1 * u * m.s2;
}

// The gradients of act(g) u, and act(g) u itself.
struct GateGrad {
    float gate, up, out;
};
template <class Act> __device__ __forceinline__ GateGrad act_grad(float g, float u, float dy) {
    const Gate m = Act::gate(g);
    const float p = g * m.s1;
    return {dy * u * m.s1 * m.w * m.s2, p * dy * m.s2, p * u * m.s2};
}
// The same of gelu_tanh at s = max(delta, 0); gate is 0 where delta <= 0.
__device__ __forceinline__ GateGrad sparse_grad(float delta, float u, float dy) {
    float s;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(s) : "f"(delta));
    const Gate m = Gelu::gate(s);
    const float p = s * m.s1;
    return {delta <= 0.f ? 0.f : dy * u * m.s1 * m.w, p * dy, p * u};
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ------------------------------------------------------------ 8 elements

__device__ __forceinline__ uint2 ld_stream_u2(const void *p) {
    uint2 r;
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ void st_u2(void *p, uint2 v) {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 8 consecutive elements of a row, as loaded: four words of two 16-bit
// elements, or eight of one.  pair(i) is elements 2i and 2i + 1.
template <class T> struct Vec8 {
    static_assert(sizeof(T) == 2, "16-bit elements");
    uint4 q;
    __device__ static Vec8 zero() { return {make_uint4(0u, 0u, 0u, 0u)}; }
    __device__ static Vec8 load(const T *p) { return {ld_stream(p)}; }
    __device__ void store(T *p) const { st_vec_out(p, q); }
    __device__ float2 pair(int i) const {
        const uint32_t w = (&q.x)[i];
        if constexpr (std::is_same_v<T, bf16>)
            return make_float2(bf16_lo(w), bf16_hi(w));
        else
            return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ void put(int i, float2 f) {
        if constexpr (std::is_same_v<T, bf16>) {
            (&q.x)[i] = pack_bf16x2(f.x, f.y);
        } else {
            const __half2 h = __floats2half2_rn(f.x, f.y);
            (&q.x)[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    // Largest magnitude, as the bits of the element type: for values of one
    // type these order as the magnitudes do, infinity and NaN above all.
    __device__ uint32_t top() const {
        constexpr uint32_t m = 0x7FFF7FFFu;
        const uint32_t w = max_u16x2(max_u16x2(q.x & m, q.y & m), max_u16x2(q.z & m, q.w & m));
        return max(w >> 16, w & 0xFFFFu);
    }
};
template <> struct Vec8<float> {
    uint4 q[2];
    __device__ static Vec8 zero() {
        return {{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}};
    }
    __device__ static Vec8 load(const float *p) { return {{ld_stream(p), ld_stream(p + 4)}}; }
    __device__ void store(float *p) const {
        st_vec_out(p, q[0]);
        st_vec_out(p + 4, q[1]);
    }
    __device__ float2 pair(int i) const {
        const uint32_t *w = &q[i / 2].x + 2 * (i & 1);
        return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    }
    __device__ void put(int i, float2 f) {
        uint32_t *w = &q[i / 2].x + 2 * (i & 1);
        w[0] = __float_as_uint(f.x);
        w[1] = __float_as_uint(f.y);
    }
    __device__ uint32_t top() const {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            t = max(t, max(max(q[i].x & 0x7FFFFFFFu, q[i].y & 0x7FFFFFFFu),
                           max(q[i].z & 0x7FFFFFFFu, q[i].w & 0x7FFFFFFFu)));
        return t;
    }
};

// Bits of a largest magnitude (Vec8::top) as those of the fp32 value.
template <class T> __device__ __forceinline__ uint32_t top_as_float(uint32_t t) {
    if constexpr (std::is_same_v<T, float>)
        return t;
    else if constexpr (std::is_same_v<T, bf16>)
        return t << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(t))));
}

// ------------------------------------------------------- 8-bit block format

constexpr int kBlock = 32;   // elements that share a scale
constexpr uint32_t kBadScale = 255u;
constexpr uint32_t kTopScale = 248u;   // 2^121: the next one's codes would reach 2^128

// Scale byte of a block from the bits of its largest magnitude, m 2^E with
// m in [1, 2): the codes of k = E - 6 reach 64 m, which rounds past 127 from
// m = 127.5 / 64 on; adding 2^23 - 0x7F0000 to the bits carries into the
// exponent exactly then.  NaN and infinity give 255.  At kTopScale the largest
// magnitudes round to 128: clamp_top limits the values of such a block first.
__device__ __forceinline__ uint32_t scale_of(uint32_t top_bits) {
    if (top_bits >= 0x7F800000u)
        return kBadScale;
    const int e = static_cast<int>((top_bits + 0x10000u) >> 23) - 6;
    return static_cast<uint32_t>(min(max(e, 0), static_cast<int>(kTopScale)));
}
__device__ __forceinline__ float clamp_top(float v) {
    constexpr float top = 127.f * 0x1p121f;
    return fminf(fmaxf(v, -top), top);
}
// 2^-k, the factor from value to code (0 for a bad block), and 2^k, the step
// from code to value (NaN for a bad block, subnormal for scale 0).
__device__ __forceinline__ float code_factor(uint32_t scale) {
    return scale == kBadScale ? 0.f : __uint_as_float((254u - scale) << 23);
}
__device__ __forceinline__ float code_step(uint32_t scale) {
    return __uint_as_float(scale == kBadScale ? 0x7FC00000u : scale == 0 ? 0x00400000u : scale << 23);
}
// rint(v 2^-k): the product is exact, so the fused add of 1.5 2^23 rounds once,
// to nearest even, and leaves the code in the low byte.  v = NaN or infinity
// (only with factor 0) gives NaN bits; the caller masks bad blocks.
__device__ __forceinline__ int code_of(float v, float factor) {
    return __float_as_int(fmaf(v, factor, 12582912.f)) - 0x4B400000;
}

// The codes of 8 values of one block, for the block's scale.
template <bool KEEP_SIGN>
__device__ __forceinline__ uint2 codes_of(const float2 (&v)[4], uint32_t scale) {
    const float f = code_factor(scale);
    const float2 f2 = make_float2(f, f), magic = make_float2(12582912.f, 12582912.f);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 x = v[i];
        if (scale == kTopScale)
            x = make_float2(clamp_top(x.x), clamp_top(x.y));
        const float2 q = fma2(x, f2, magic);
        w[2 * i] = __float_as_uint(q.x);
        w[2 * i + 1] = __float_as_uint(q.y);
        if (KEEP_SIGN) {   // 12582912 + 1, the bits of code 1
            if (x.x > 0.f)
                w[2 * i] = max(w[2 * i], 0x4B400001u);
            if (x.y > 0.f)
                w[2 * i + 1] = max(w[2 * i + 1], 0x4B400001u);
        }
    }
    uint2 c;
    c.x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    c.y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
    return scale == kBadScale ? make_uint2(0u, 0u) : c;
}

// Codes 2i and 2i + 1 of 8 (biased: codes ^ 0x80808080) as values: the byte
// becomes the low bits of 2^23 + 128 + code; both steps are exact.
__device__ __forceinline__ float2 decode_pair(uint2 biased, int i, float step) {
    const uint32_t w = i < 2 ? biased.x : biased.y;
    const float2 f = make_float2(
        __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + 2 * (i & 1))),
        __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + 2 * (i & 1))));
    return mul2(sub2(f, make_float2(8388736.f, 8388736.f)), make_float2(step, step));
}
__device__ __forceinline__ uint2 bias_codes(uint2 c) {
    return make_uint2(c.x ^ 0x80808080u, c.y ^ 0x80808080u);
}

// ---------------------------------------------------------------- host side

// One buffer of a call: its checks, then the address kernels use for it.
struct Region {
    const void *p;
    uint64_t bytes;
    uintptr_t align;
    bool write;
    const void *dev = nullptr;
};

// Null, alignment, overlap (of two buffers of which one is written) and
// residence of every buffer; empty buffers (bytes = 0) are skipped.
int check_regions(Region *r, int n);

inline int64_t elem_size(int dtype) {
    return dtype == GATED_ACT_F32 ? 4 : dtype == GATED_ACT_BF16 || dtype == GATED_ACT_F16 ? 2 : 0;
}
inline int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes spanned by `rows` rows of `width` elements, `stride` elements apart.
inline uint64_t span_bytes(int64_t rows, int64_t stride, int64_t width, int64_t size) {
    return rows <= 0 ? 0 : static_cast<uint64_t>(((rows - 1) * stride + width) * size);
}

template <class T> inline T *as(const Region &r) {
    return static_cast<T *>(const_cast<void *>(r.dev));
}

// Calls f(T{}) with the element type of a checked dtype code.
template <class F> inline int with_type(int dtype, F f) {
    switch (dtype) {
    case GATED_ACT_BF16: return f(bf16{});
    case GATED_ACT_F16: return f(f16{});
    default: return f(float{});
    }
}

// Lets `kernel` launch with `bytes` of dynamic shared memory (and up to 1 KB
// of static).  Above the default 48 KB that takes an attribute of the kernel,
// set before each launch: a host-side call, with nothing kept per device or
// context.
inline cudaError_t allow_smem(const void *kernel, size_t bytes) {
    if (bytes <= 47 * 1024)
        return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(bytes));
}

inline int launched(cudaError_t e) {
    return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace gact
