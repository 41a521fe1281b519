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
// sigma (1 + g a' (1 - sigma)).  With y = a log2(e) / 2 and e = 2^-|y|,
//   sigma = r k,  r = 1 / (1 + e^2), k = 1 for y >= 0;  r = e / (1 + e^2), k = e for y < 0:
// no cancellation and no limit on y.  e and the reciprocal come from the flushing
// hardware functions (PTX ISA ex2.approx.ftz.f32, rcp.approx.ftz.f32, relative error
// about 2^-22); e stays normal down to a = -174, where sigma is 2^-251, and is 0 below.
// Neither factor is above 1, and k is multiplied last, so that a product with them
// falls below fp32's normal range only where the result does, or where what it
// multiplies is there already.  (The gate's gradient is the product of u r and dy k:
// one of these may lose bits below the normal range while the other is large.)  Two
// elements at a time: the paired fp32 instructions halve the issue slots.
struct Gate2 {
    float2 r, k;   // sigma = r k
};
__device__ __forceinline__ Gate2 gate_of(float2 y) {
    Gate2 m;
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-fabsf(y.x)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-fabsf(y.y)));
    m.k = make_float2(y.x < 0.f ? e.x : 1.f, y.y < 0.f ? e.y : 1.f);
    e = fma2(e, e, make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(m.r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(m.r.y) : "f"(e.y));
    m.r = mul2(m.r, m.k);
    return m;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// exponent(g) = y, lean(g) = g a'.
struct Silu {
    __device__ static float2 exponent(float2 g) { return mul2(g, both(0.5f * 1.4426950408889634f)); }
    __device__ static float2 lean(float2 g) { return g; }
};

// a = 2 sqrt(2/pi) (g + 0.044715 g^3).  g a' is taken at most at |g| = 16,
// where it cannot overflow: past |g| = 11, sigma or 1 - sigma is 0 beside it.
struct Gelu {
    static constexpr float k2 = 2.0f * 0.7978845608028654f;
    static constexpr float k2c = 2.0f * 0.7978845608028654f * 0.044715f;
    static constexpr float e = 0.5f * 1.4426950408889634f;
    __device__ static float2 exponent(float2 g) {
        return mul2(g, fma2(mul2(g, g), both(e * k2c), both(e * k2)));
    }
    __device__ static float2 lean(float2 g) {
        float2 b;
        asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(b.x) : "f"(g.x), "f"(16.f));
        asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(b.y) : "f"(g.y), "f"(16.f));
        return mul2(b, fma2(mul2(b, b), both(3.f * k2c), both(k2)));
    }
};

// act(g) u
template <class Act> __device__ __forceinline__ float2 act_mul(float2 g, float2 u) {
    const Gate2 m = gate_of(Act::exponent(g));
    return mul2(mul2(mul2(g, m.r), u), m.k);
}

// The gradients of act(g) u, and act(g) u itself.
struct GateGrad2 {
    float2 gate, up, out;
};
template <class Act>
__device__ __forceinline__ GateGrad2 act_grad(float2 g, float2 u, float2 dy) {
    const Gate2 m = gate_of(Act::exponent(g));
    const float2 p = mul2(g, m.r), q = mul2(dy, m.k);
    const float2 off = fma2(make_float2(-m.r.x, -m.r.y), m.k, both(1.f));   // 1 - sigma
    const float2 w = fma2(Act::lean(g), off, both(1.f));
    return {mul2(mul2(mul2(u, m.r), w), q), mul2(p, q), mul2(mul2(p, u), m.k)};
}
__device__ __forceinline__ float2 relu_nan2(float2 x) {
    float2 s;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(s.x) : "f"(x.x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(s.y) : "f"(x.y));
    return s;
}

// gelu_tanh at s >= 0 (or NaN), where sigma = 1 / (1 + e) with e = 2^{-2 y} <= 1
// takes one exponential less and no limit; 1 - sigma = e r.
__device__ __forceinline__ void gate_of_positive(float2 s, float2 *e, float2 *r) {
    const float2 y2 = mul2(s, fma2(mul2(s, s), both(-2.f * Gelu::e * Gelu::k2c),
                                   both(-2.f * Gelu::e * Gelu::k2)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e->x) : "f"(y2.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e->y) : "f"(y2.y));
    const float2 n = add2(*e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r->x) : "f"(n.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r->y) : "f"(n.y));
}
// gelu_tanh(max(delta, 0)) u, and its gradients; gate is 0 where delta <= 0.
__device__ __forceinline__ float2 sparse_mul(float2 delta, float2 u) {
    const float2 s = relu_nan2(delta);
    float2 e, r;
    gate_of_positive(s, &e, &r);
    return mul2(mul2(s, r), u);
}
__device__ __forceinline__ GateGrad2 sparse_grad(float2 delta, float2 u, float2 dy) {
    const float2 s = relu_nan2(delta);
    float2 e, r;
    gate_of_positive(s, &e, &r);
    const float2 p = mul2(s, r), w = fma2(Gelu::lean(s), mul2(e, r), both(1.f));
    GateGrad2 m = {mul2(mul2(mul2(u, r), w), dy), mul2(p, dy), mul2(p, u)};
    m.gate.x = delta.x <= 0.f ? 0.f : m.gate.x;
    m.gate.y = delta.y <= 0.f ? 0.f : m.gate.y;
    return m;
}

// max(t, |a|, |b|), NaN if one is NaN.
__device__ __forceinline__ float max_abs(float t, float2 v) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(t), "f"(v.x), "f"(v.y));
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

// 8 consecutive elements of a row, aligned to their size, as loaded: four words of two 16-bit
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
        using T2 = std::conditional_t<std::is_same_v<T, bf16>, __nv_bfloat162, __half2>;
        const T2 *h = reinterpret_cast<const T2 *>(&q);
        const T2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                 __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
        return max(w >> 16, w & 0xFFFFu);
    }
};
// Of fp32, 32 bytes in one access (PTX ISA ld/st.global.v8.b32, sm_100 and
// later): two 16-byte accesses of a warp would each touch every sector.
template <> struct Vec8<float> {
    uint4 q[2];
    __device__ static Vec8 zero() {
        return {{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}};
    }
    __device__ static Vec8 load(const float *p) {
        Vec8 v;
        asm("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(v.q[0].x), "=r"(v.q[0].y), "=r"(v.q[0].z), "=r"(v.q[0].w), "=r"(v.q[1].x),
              "=r"(v.q[1].y), "=r"(v.q[1].z), "=r"(v.q[1].w)
            : "l"(p));
        return v;
    }
    __device__ void store(float *p) const {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "r"(q[0].x), "r"(q[0].y), "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y),
                     "r"(q[1].z), "r"(q[1].w));
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
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = max_abs(t, pair(i));
        return __float_as_uint(t);
    }
};

// Asynchronous copies to shared memory, by the thread that will read them.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bits of a largest magnitude (Vec8::top) as those of the fp32 value.
template <class T> __device__ __forceinline__ uint32_t top_as_float(uint32_t t) {
    if constexpr (std::is_same_v<T, float>)
        return t;
    else if constexpr (std::is_same_v<T, bf16>)
        return t << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(t))));
}

// f(i0, full) for the groups i0, i0 + 4, ... < V of four columns t + NT i each that
// hold any; full: all of the group's columns are below d in the whole warp.
template <int NT, int V, class F> __device__ __forceinline__ void for_groups(int t, int d, F f) {
    const int last = t | 31;
#pragma unroll
    for (int i = 0; i < V; i += 4)
        if (NT * i + t - (t & 31) < d)
            f(i, last + NT * (i + 3) < d);
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
__device__ __forceinline__ uint2 pack_codes(const float2 (&v)[4], float factor) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = fma2(v[i], both(factor), both(12582912.f));
        w[2 * i] = __float_as_uint(q.x);
        w[2 * i + 1] = __float_as_uint(q.y);
        if (KEEP_SIGN) {   // 12582912 + 1, the bits of code 1
            if (v[i].x > 0.f)
                w[2 * i] = max(w[2 * i], 0x4B400001u);
            if (v[i].y > 0.f)
                w[2 * i + 1] = max(w[2 * i + 1], 0x4B400001u);
        }
    }
    return make_uint2(
        __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
        __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
}
template <bool KEEP_SIGN>
__device__ __forceinline__ uint2 codes_of(const float2 (&v)[4], uint32_t scale) {
    if (scale >= kTopScale) {   // a block at the very end of the range, or a bad one
        if (scale == kBadScale)
            return make_uint2(0u, 0u);
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(clamp_top(v[i].x), clamp_top(v[i].y));
        return pack_codes<KEEP_SIGN>(x, __uint_as_float((254u - kTopScale) << 23));
    }
    return pack_codes<KEEP_SIGN>(v, __uint_as_float((254u - scale) << 23));
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

// ------------------------------------------------------- CTAs and clusters

// Sum over the NT threads of a CTA that holds one row, the same bits in every thread;
// red holds NT / 32 floats.
template <int NT> __device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = v;
        __syncthreads();
        constexpr int NW = NT / 32;
        v = red[threadIdx.x & (NW - 1)];
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    return v;
}


// Rows of one value have that value as their mean, and no deviation.  A rounded sum would
// give them a deviation of its rounding: the sparse GELU then passes all or none of the
// row at z < 1, and layer norm multiplies the rounding by up to 1 / sqrt(eps).  So the
// kernels ask, with one logic instruction per word, whether all elements of a row have the
// bits of its first, where sums of one value can be rounded: fp32 holds the multiples up
// to 2^13 of an fp16 number and up to 2^16 of a bf16 one (11 and 8 bits).  (For 16-bit rows in
// vectors the test would cost 2 to 4%: sparse GELU forward 2048 x 16384 bf16 49.7 us against
// 48.5, 4000 x 8192 46.3 against 44.7.)
//
// N: the most elements, or whole vectors where every sum is of whole ones.
template <class T, int N>
constexpr bool kSumsRound = N > (std::is_same_v<T, float> ? 1
                                 : std::is_same_v<T, f16> ? 1 << 13
                                                          : 1 << 16);
// The word that repeats an element's bits, and nonzero where q differs from it.
template <class T> __device__ __forceinline__ uint32_t repeated(T first) {
    if constexpr (sizeof(T) == 4)
        return __float_as_uint(first);
    else
        return 0x10001u * *reinterpret_cast<const unsigned short *>(&first);
}
__device__ __forceinline__ uint32_t unlike(uint4 q, uint32_t word) {
    return (q.x ^ word) | (q.y ^ word) | (q.z ^ word) | (q.w ^ word);
}
template <class T> __device__ __forceinline__ uint32_t unlike(const Vec8<T> &v, T first) {
    uint32_t r = 0u;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
        r |= unlike(reinterpret_cast<const uint4 *>(&v)[i], repeated(first));
    return r;
}
__device__ __forceinline__ uint32_t unlike(float a, float b) {
    return __float_as_uint(a) ^ __float_as_uint(b);
}
// row_sum, and whether `other` is 0 in all threads: the barrier carries the answer.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *red, uint32_t other, bool *same) {
    v = warp_sum(v);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = v;
        *same = !__syncthreads_or(other != 0u);
        constexpr int NW = NT / 32;
        v = red[threadIdx.x & (NW - 1)];
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    } else {
        *same = !__any_sync(0xFFFFFFFFu, other != 0u);
    }
    return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Barrier of the cluster's threads: what each wrote before is seen by all after it.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A CTA's shared memory may be written by its peers once it has started: each says so on
// entry, and waits for the others before it first writes to them.
__device__ __forceinline__ void cluster_started() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- host side

// One buffer of a call: its checks, then the address kernels use for it.
struct Region {
    const void *p;
    uint64_t bytes;
    uintptr_t align;
    bool write;
    const void *dev = nullptr;
    bool host = false;   // set by check_regions: page-locked host memory
};

// Null, alignment, overlap (of two buffers of which one is written) and
// residence of every buffer; empty buffers (bytes = 0) are skipped.
int check_regions(Region *r, int n);

constexpr int64_t kMaxWidth = int64_t(1) << 30, kMaxRows = int64_t(1) << 40;

template <int N> using Const = std::integral_constant<int, N>;

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

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): with 2^(s-1) < d <= 2^s and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(m, n) + n) >> s.
struct FastDiv {
    uint32_t m, s;
    explicit FastDiv(uint32_t d) : s(0) {
        while (s < 32 && (uint64_t(1) << s) < d)
            ++s;
        m = static_cast<uint32_t>((((uint64_t(1) << s) - d) << 32) / d + 1);
    }
    __device__ uint32_t operator()(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

inline int launched(cudaError_t e) {
    return cuda_status(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace gact
