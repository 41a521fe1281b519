// 8-bit checkpoints of the gated activations, and the backward passes that
// read them (definitions in gated_act_training.h).
//
// Each op reads and writes every byte once and computes a few dozen
// instructions per element: HBM bandwidth bounds it.  Per gate/up pair of a
// 16-bit type the forward pass moves 4 + 2 bytes of rows and 2 + 1/16 of
// checkpoint, the backward pass 2 (+ 2 with the recomputed output) + 4 and
// the same 2 + 1/16.  Rates below are of GB300 and, in percent, of its copy
// rate, 6.79 TB/s; inputs larger than L2 in turn, backward passes with the
// recomputed output.
//
// A block of the 8-bit format is 32 elements of one half.  Its largest
// magnitude m = 1.f 2^E fixes k = E - 6 (or the next one, where 1.f would round
// to 128), a code is v 2^-k rounded, and both powers of two are exact.
#include <algorithm>

#include "training.cuh"

namespace gact {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t live_rows(int64_t M, const int32_t *n_rows) {
    if (!n_rows)
        return M;
    const int64_t n = *n_rows;
    return n < 0 ? 0 : n > M ? M : n;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One block of a half, one element per lane (`in`: the lane holds one): writes
// its code and, from lane 0, the scale.
template <bool KEEP_SIGN>
__device__ __forceinline__ void put_block(int8_t *codes, uint8_t *scale, float v, bool in, int lane) {
    const uint32_t s = scale_of(__reduce_max_sync(0xFFFFFFFFu, in ? abs_bits(v) : 0u));
    if (s == kTopScale)
        v = clamp_top(v);
    int q = code_of(v, code_factor(s));
    if (KEEP_SIGN && v > 0.f)
        q = max(q, 1);
    if (in)
        *codes = static_cast<int8_t>(s == kBadScale ? 0 : q);
    if (lane == 0)
        *scale = static_cast<uint8_t>(s);
}

// Four blocks of each half, whole, one element of each per lane: their codes at
// codes + i * es and codes + d + i * es, their scales at scales + i * ss and
// scales + B + i * ss.  The eight largest magnitudes are found together, halving
// the values at every exchange, so that lane 4 k ends with the k-th and each
// scale is computed once, not by every lane.
template <bool KEEP_SIGN>
__device__ __forceinline__ void put_blocks(int8_t *codes, int64_t d, int es, uint8_t *scales,
                                           int64_t B, int ss, const float (&g)[4],
                                           const float (&u)[4], int lane) {
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = abs_bits(g[i]);
        t[4 + i] = abs_bits(u[i]);
    }
#pragma unroll
    for (int n = 4; n >= 1; n >>= 1) {
        const bool up = lane & (4 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t keep = up ? t[i + n] : t[i], give = up ? t[i] : t[i + n];
            t[i] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 4 * n));
        }
    }
    t[0] = max(t[0], __shfl_xor_sync(0xFFFFFFFFu, t[0], 2));
    t[0] = max(t[0], __shfl_xor_sync(0xFFFFFFFFu, t[0], 1));
    const uint32_t s = scale_of(t[0]);
    const int k = lane >> 2;
    if ((lane & 3) == 0)
        scales[(k < 4 ? k * ss : B + (k - 4) * ss)] = static_cast<uint8_t>(s);
    const bool odd = __any_sync(0xFFFFFFFFu, s >= kTopScale);
    const float f = code_factor(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v = i < 4 ? g[i & 3] : u[i & 3];
        if (odd && __shfl_sync(0xFFFFFFFFu, s, 4 * i) >= kTopScale)
            v = __shfl_sync(0xFFFFFFFFu, s, 4 * i) == kBadScale ? 0.f : clamp_top(v);
        int q = code_of(v, __shfl_sync(0xFFFFFFFFu, f, 4 * i));
        if (KEEP_SIGN && i < 4 && v > 0.f)
            q = max(q, 1);
        codes[(i < 4 ? 0 : d) + (i & 3) * es] = static_cast<int8_t>(q);
    }
}

// n / d; a 32-bit n takes the multiplication.
template <class I> __device__ __forceinline__ I quotient(I n, I d, const FastDiv &by) {
    if constexpr (sizeof(I) == 4)
        return by(n);
    else
        return n / d;
}

// ------------------------------------------------- elementwise, any layout
//
// A warp takes kAnyBlocks consecutive blocks of a row of both halves, one element
// of each per lane, so that every access of a warp is one contiguous run
// whatever the alignment; J = ceil(B / kAnyBlocks) such jobs make a row.  Four
// blocks of two halves are the eight largest magnitudes that one exchange of
// lanes finds together (put_blocks).  The single bytes and half words that a
// lane moves make instructions the bound: 16384 x 767 bf16 takes 28.7 us forward
// (52%) and 30.5 us backward (61%), against 25.5 and 29.1 us at 768, where the
// vectors below take 17.2 and 20.7.

constexpr int kAnyBlocks = 4;

// Steps of the blocks b0, b0 + 1, ... of both halves, one per lane: lane i
// that of block i of the gate half, lane kAnyBlocks + i of the up half.
__device__ __forceinline__ float lane_step(const uint8_t *scales, int64_t b0, int64_t B, int lane) {
    const int i = lane % kAnyBlocks, up = lane / kAnyBlocks;
    return up < 2 && b0 + i < B ? code_step(__ldg(scales + up * B + b0 + i)) : 0.f;
}

template <class T, class Act, class I>
__global__ void __launch_bounds__(kThreads)
ckpt_forward_any(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                 const T *__restrict__ in, int64_t M, int64_t d, int64_t rs, int64_t B, I J,
                 FastDiv by_J, const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = kAnyBlocks;
    const int lane = threadIdx.x & 31;
    const I job = static_cast<I>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const I row = quotient(job, J, by_J);
    if (row >= live_rows(M, n_rows))      // the warp as a whole
        return;
    const int64_t r = row, b0 = static_cast<int64_t>(job - row * J) * U, c0 = b0 * kBlock + lane;
    const T *p = in + r * rs + c0;
    T *o = out + r * d + c0;
    int8_t *q = codes + r * 2 * d + c0;
    uint8_t *s = scales + r * 2 * B + b0;
    T graw[U], uraw[U];
    if (c0 - lane + kBlock * U <= d) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            graw[i] = __ldg(p + kBlock * i);
            uraw[i] = __ldg(p + d + kBlock * i);
        }
        float g[U], u[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            g[i] = to_float(graw[i]);
            u[i] = to_float(uraw[i]);
        }
#pragma unroll
        for (int i = 0; i < U; i += 2) {
            const float2 y = act_mul<Act>(make_float2(g[i], g[i + 1]), make_float2(u[i], u[i + 1]));
            o[kBlock * i] = from_float<T>(y.x);
            o[kBlock * (i + 1)] = from_float<T>(y.y);
        }
        put_blocks<false>(q, d, kBlock, s, B, 1, g, u, lane);
        return;
    }
    // the row's end
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (b0 + i >= B)
            break;
        const bool ok = c0 + kBlock * i < d;
        const float g = ok ? to_float(__ldg(p + kBlock * i)) : 0.f;
        const float u = ok ? to_float(__ldg(p + d + kBlock * i)) : 0.f;
        if (ok)
            o[kBlock * i] = from_float<T>(act_mul<Act>(both(g), both(u)).x);
        put_block<false>(q + kBlock * i, s + i, g, ok, lane);
        put_block<false>(q + d + kBlock * i, s + B + i, u, ok, lane);
    }
}

// A code as the low byte of 2^23 + 128 + code, and two such as values.
__device__ __forceinline__ uint32_t load_code(const int8_t *p) {
    return (__ldg(reinterpret_cast<const uint8_t *>(p)) ^ 0x80u) | 0x4B000000u;
}
__device__ __forceinline__ float2 code_pair(uint32_t a, uint32_t b) {
    return sub2(make_float2(__uint_as_float(a), __uint_as_float(b)), both(8388736.f));
}

template <class T, class Act, class I>
__global__ void __launch_bounds__(kThreads)
ckpt_backward_any(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                  const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t M,
                  int64_t d, int64_t gs, int64_t B, I J, FastDiv by_J, const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = kAnyBlocks;
    const int lane = threadIdx.x & 31;
    const I job = static_cast<I>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const I row = quotient(job, J, by_J);
    if (row >= live_rows(M, n_rows))
        return;
    const int64_t r = row, b0 = static_cast<int64_t>(job - row * J) * U, c0 = b0 * kBlock + lane;
    const T *dy = grad + r * gs + c0;
    const int8_t *q = codes + r * 2 * d + c0;
    if (c0 - lane + kBlock * U <= d) {
        T y[U];
        uint32_t g[U], u[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            y[i] = __ldg(dy + kBlock * i);
            g[i] = load_code(q + kBlock * i);
            u[i] = load_code(q + d + kBlock * i);
        }
        const float step = lane_step(scales + r * 2 * B, b0, B, lane);
        T *gi = grad_in + r * 2 * d + c0, *o = out + r * d + c0;
#pragma unroll
        for (int i = 0; i < U; i += 2) {
            const float2 sg = make_float2(__shfl_sync(0xFFFFFFFFu, step, i),
                                          __shfl_sync(0xFFFFFFFFu, step, i + 1));
            const float2 su = make_float2(__shfl_sync(0xFFFFFFFFu, step, U + i),
                                          __shfl_sync(0xFFFFFFFFu, step, U + i + 1));
            const GateGrad2 m = act_grad<Act>(mul2(code_pair(g[i], g[i + 1]), sg),
                                              mul2(code_pair(u[i], u[i + 1]), su),
                                              make_float2(to_float(y[i]), to_float(y[i + 1])));
            gi[kBlock * i] = from_float<T>(m.gate.x);
            gi[kBlock * (i + 1)] = from_float<T>(m.gate.y);
            gi[d + kBlock * i] = from_float<T>(m.up.x);
            gi[d + kBlock * (i + 1)] = from_float<T>(m.up.y);
            if (out) {
                o[kBlock * i] = from_float<T>(m.out.x);
                o[kBlock * (i + 1)] = from_float<T>(m.out.y);
            }
        }
        return;
    }
    T yraw[U];
    int8_t qg[U], qu[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (c0 + kBlock * i < d) {
            yraw[i] = __ldg(dy + kBlock * i);
            qg[i] = __ldg(q + kBlock * i);
            qu[i] = __ldg(q + d + kBlock * i);
        }
    const float step = lane_step(scales + r * 2 * B, b0, B, lane);
    T *gi = grad_in + r * 2 * d + c0, *o = out + r * d + c0;
#pragma unroll
    for (int i = 0; i < U; i += 2) {
        const bool in0 = c0 + kBlock * i < d, in1 = c0 + kBlock * (i + 1) < d;
        const float2 sg = make_float2(__shfl_sync(0xFFFFFFFFu, step, i),
                                      __shfl_sync(0xFFFFFFFFu, step, i + 1));
        const float2 su = make_float2(__shfl_sync(0xFFFFFFFFu, step, U + i),
                                      __shfl_sync(0xFFFFFFFFu, step, U + i + 1));
        const float2 g = mul2(make_float2(in0 ? qg[i] : 0, in1 ? qg[i + 1] : 0), sg);
        const float2 u = mul2(make_float2(in0 ? qu[i] : 0, in1 ? qu[i + 1] : 0), su);
        const float2 y = make_float2(in0 ? to_float(yraw[i]) : 0.f, in1 ? to_float(yraw[i + 1]) : 0.f);
        const GateGrad2 m = act_grad<Act>(g, u, y);
        if (in0) {
            gi[kBlock * i] = from_float<T>(m.gate.x);
            gi[d + kBlock * i] = from_float<T>(m.up.x);
            if (out)
                o[kBlock * i] = from_float<T>(m.out.x);
        }
        if (in1) {
            gi[kBlock * (i + 1)] = from_float<T>(m.gate.y);
            gi[d + kBlock * (i + 1)] = from_float<T>(m.up.y);
            if (out)
                o[kBlock * (i + 1)] = from_float<T>(m.out.y);
        }
    }
}

template <class T, class I>
__global__ void __launch_bounds__(kThreads)
ckpt_values_any(T *__restrict__ values, const int8_t *__restrict__ codes,
                const uint8_t *__restrict__ scales, int64_t M, int64_t d, int64_t B, I J,
                FastDiv by_J) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = kAnyBlocks;
    const int lane = threadIdx.x & 31;
    const I job = static_cast<I>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const I row = quotient(job, J, by_J);
    if (row >= M)
        return;
    const int64_t r = row, b0 = static_cast<int64_t>(job - row * J) * U, c0 = b0 * kBlock + lane;
    const int8_t *q = codes + r * 2 * d + c0;
    T *v = values + r * 2 * d + c0;
    int8_t qg[U], qu[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (c0 + kBlock * i < d) {
            qg[i] = __ldg(q + kBlock * i);
            qu[i] = __ldg(q + d + kBlock * i);
        }
    const float step = lane_step(scales + r * 2 * B, b0, B, lane);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float sg = __shfl_sync(0xFFFFFFFFu, step, i), su = __shfl_sync(0xFFFFFFFFu, step, U + i);
        if (c0 + kBlock * i < d) {
            v[kBlock * i] = from_float<T>(qg[i] * sg);
            v[d + kBlock * i] = from_float<T>(qu[i] * su);
        }
    }
}

// --------------------------------------------------- elementwise, vectors
//
// Rows in 16-byte vectors (pointers and strides allow it, d a multiple of 8):
// a thread takes 8 elements of the gate and the 8 of the up half beside them;
// four neighbouring lanes hold a block of each.  A row is 4 B slots of 8
// elements, B blocks, so that lane groups and blocks coincide in every row;
// the slots past d (a ragged last block) are empty.
//
// HBM bounds it: silu of 16384 x 768 bf16 takes 17.2 us forward (87%) and 20.7 us
// backward (90%), of 4000 x 2048 fp32 18.4 us (92%) and 23.4 us (93%).  One slot
// per thread and full occupancy hide the loads better than two per thread (20.8
// and 24.6 us); the values, with nothing to compute, take four (2048 x 16384:
// 31.5 us, 95%; one: 36.5 us).  Slots are found by a 32-bit multiplication while
// they number fewer than 2^31: by a 64-bit division the two passes take 18.5
// and 21.9 us.

// Largest magnitude over the four lanes of a block, of both halves at once.
template <class T>
__device__ __forceinline__ void block_tops(uint32_t *g, uint32_t *u) {
    if constexpr (sizeof(T) == 2) {
        uint32_t w = *g | (*u << 16);
        w = max_u16x2(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1));
        w = max_u16x2(w, __shfl_xor_sync(0xFFFFFFFFu, w, 2));
        *g = w & 0xFFFFu;
        *u = w >> 16;
    } else {
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            *g = max(*g, __shfl_xor_sync(0xFFFFFFFFu, *g, o));
            *u = max(*u, __shfl_xor_sync(0xFFFFFFFFu, *u, o));
        }
    }
}

template <class T, class Act, int VPT, class I>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && sizeof(I) == 4 ? 8 : 6)
ckpt_forward_vec(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                 const T *__restrict__ in, int64_t M, I d, int64_t rs, I B, FastDiv by_slots,
                 const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    const I slots = 4 * B;
    const I live = static_cast<I>(live_rows(M, n_rows));
    const I first = static_cast<I>(blockIdx.x) * (VPT * kThreads) + threadIdx.x;
    I row[VPT], col[VPT];
    Vec8<T> g[VPT], u[VPT];
    bool ok[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const I s = first + i * kThreads;
        row[i] = quotient(s, slots, by_slots);
        col[i] = (s - row[i] * slots) * 8;
        ok[i] = row[i] < live && col[i] < d;
        g[i] = u[i] = Vec8<T>::zero();
        if (ok[i]) {
            const T *p = in + static_cast<int64_t>(row[i]) * rs + col[i];
            g[i] = Vec8<T>::load(p);
            u[i] = Vec8<T>::load(p + d);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        uint32_t tg = g[i].top(), tu = u[i].top();
        block_tops<T>(&tg, &tu);
        if (!ok[i])
            continue;
        const uint32_t sg = scale_of(top_as_float<T>(tg)), su = scale_of(top_as_float<T>(tu));
        float2 gf[4], uf[4];
        Vec8<T> o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gf[j] = g[i].pair(j);
            uf[j] = u[i].pair(j);
            o.put(j, act_mul<Act>(gf[j], uf[j]));
        }
        const int64_t r = row[i];
        o.store(out + r * d + col[i]);
        int8_t *c = codes + r * 2 * d + col[i];
        st_u2(c, codes_of<false>(gf, sg));
        st_u2(c + d, codes_of<false>(uf, su));
        if (col[i] % kBlock == 0) {
            uint8_t *s = scales + r * 2 * B + col[i] / kBlock;
            s[0] = static_cast<uint8_t>(sg);
            s[B] = static_cast<uint8_t>(su);
        }
    }
}

template <class T, class Act, int VPT, class I>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && sizeof(I) == 4 ? 8 : 6)
ckpt_backward_vec(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                  const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t M,
                  I d, int64_t gs, I B, FastDiv by_nv, const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    const I nv = d / 8;
    const I live = static_cast<I>(live_rows(M, n_rows));
    const I first = static_cast<I>(blockIdx.x) * (VPT * kThreads) + threadIdx.x;
    I row[VPT], col[VPT];
    Vec8<T> dy[VPT];
    uint2 cg[VPT], cu[VPT];
    uint32_t sg[VPT], su[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const I s = first + i * kThreads;
        row[i] = quotient(s, nv, by_nv);
        col[i] = (s - row[i] * nv) * 8;
        if (row[i] < live) {
            const int64_t r = row[i];
            dy[i] = Vec8<T>::load(grad + r * gs + col[i]);
            const int8_t *c = codes + r * 2 * d + col[i];
            cg[i] = ld_stream_u2(c);
            cu[i] = ld_stream_u2(c + d);
            const uint8_t *q = scales + r * 2 * B + col[i] / kBlock;
            sg[i] = __ldg(q);
            su[i] = __ldg(q + B);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (row[i] >= live)
            continue;
        const uint2 bg = bias_codes(cg[i]), bu = bias_codes(cu[i]);
        const float stg = code_step(sg[i]), stu = code_step(su[i]);
        Vec8<T> og, ou, oo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 g = decode_pair(bg, j, stg), u = decode_pair(bu, j, stu);
            const float2 y = dy[i].pair(j);
            const GateGrad2 m = act_grad<Act>(g, u, y);
            og.put(j, m.gate);
            ou.put(j, m.up);
            oo.put(j, m.out);
        }
        const int64_t r = row[i];
        T *p = grad_in + r * 2 * d + col[i];
        og.store(p);
        ou.store(p + d);
        if (out)
            oo.store(out + r * d + col[i]);
    }
}

template <class T, int VPT, class I>
__global__ void __launch_bounds__(kThreads)
ckpt_values_vec(T *__restrict__ values, const int8_t *__restrict__ codes,
                const uint8_t *__restrict__ scales, I total, I nv, I B, FastDiv by_nv) {
    pdl_wait();
    pdl_trigger();
    const I first = static_cast<I>(blockIdx.x) * (VPT * kThreads) + threadIdx.x;
    uint2 c[VPT];
    uint32_t e[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const I s = first + i * kThreads;
        if (s < total) {
            const I h = quotient(s, nv, by_nv), v = s - h * nv;        // half-row, vector
            c[i] = ld_stream_u2(codes + static_cast<int64_t>(s) * 8);
            e[i] = __ldg(scales + static_cast<int64_t>(h) * B + v / 4);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const I s = first + i * kThreads;
        if (s >= total)
            continue;
        const float step = code_step(e[i]);
        const uint2 b = bias_codes(c[i]);
        Vec8<T> o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o.put(j, decode_pair(b, j, step));
        o.store(values + static_cast<int64_t>(s) * 8);
    }
}

// The mean of a row of n elements: `first` where all have its bits.
template <int NT>
__device__ __forceinline__ float row_mean(float v, float *red, uint32_t other, float first, float n) {
    bool same;
    const float sum = row_sum<NT>(v, red, other, &same);
    return same ? first : sum / n;
}

// ------------------------------------------------------ sparse, any layout
//
// One CTA per row, one element per lane: warp w holds the blocks w, w + NT / 32,
// ..., V of them, in registers.  Two things bound it: 89 and 105 instructions per
// element, which keep the issue slots 66 and 62% busy while the CTAs run, and the wait
// for a row's loads, since nothing of the next row is on its way during a row's sums
// and barriers.  2000 x 4097 bf16 takes 30.9 us forward (31%; 35.2 with registers for 1024
// threads per SM instead of 1536) and 37.8 us backward (32%; with 1536: 46.2), 43.3 and
// 76.6 us with the row read again for each pass, as the next section does.  Rows in
// vectors take half: 2000 x 4096 fp16 13.3 and 17.4 us.

template <class T, int NT, int V>
__global__ void __launch_bounds__(NT, 1536 / NT)
sparse_forward_any(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   float *__restrict__ std_out, const T *__restrict__ in, int d, int64_t rs,
                   int B, float z) {
    __shared__ float red[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x;
    const int t = threadIdx.x;
    const T *p = in + r * rs + t;
    // the up half is read last: to L2 meanwhile
    constexpr int kLine = 128 / sizeof(T);
    for (int c = kLine * t; c < d; c += kLine * NT)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + r * rs + d + c));
    constexpr bool kRound = kSumsRound<T, NT * V>;
    const float first = kRound ? to_float(__ldg(in + r * rs)) : 0.f;
    uint32_t other = 0u;
    float g[V], acc = 0.f;
    for_groups<NT, V>(t, d, [&](int i, bool full) {
#pragma unroll
        for (int j = i; j < i + 4; ++j)
            g[j] = full || t + NT * j < d ? to_float(__ldg(p + NT * j)) : 0.f;
    });
    for_groups<NT, V>(t, d, [&](int i, bool full) {
        acc += (g[i] + g[i + 1]) + (g[i + 2] + g[i + 3]);
        if constexpr (kRound)
#pragma unroll
            for (int j = i; j < i + 4; ++j)
                if (full || t + NT * j < d)
                    other |= unlike(g[j], first);
    });
    const float n = static_cast<float>(d);
    float mean;
    if constexpr (kRound)
        mean = row_mean<NT>(acc, red[0], other, first, n);
    else
        mean = row_sum<NT>(acc, red[0]) / n;
    acc = 0.f;
    for_groups<NT, V>(t, d, [&](int i, bool full) {
#pragma unroll
        for (int j = i; j < i + 4; ++j) {
            const float e = full || t + NT * j < d ? g[j] - mean : 0.f;
            acc = fmaf(e, e, acc);
        }
    });
    const float std = __fsqrt_rn(row_sum<NT>(acc, red[1]) / n);
    const float cutoff = fmaf(std, z, mean);
    if (t == 0)
        std_out[r] = std;
    T *o = out + r * d + t;
    int8_t *q = codes + r * 2 * d + t;
    uint8_t *s = scales + r * 2 * B + (t >> 5);
    for_groups<NT, V>(t, d, [&](int i, bool full) {
        float v[4], u[4];
        if (full) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = g[i + j] - cutoff;
                u[j] = to_float(__ldg(p + d + NT * (i + j)));
            }
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float2 y = sparse_mul(make_float2(v[j], v[j + 1]), make_float2(u[j], u[j + 1]));
                o[NT * (i + j)] = from_float<T>(y.x);
                o[NT * (i + j + 1)] = from_float<T>(y.y);
            }
            put_blocks<true>(q + NT * i, d, NT, s + NT / 32 * i, B, NT / 32, v, u, lane);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = t + NT * (i + j);
            if (c - lane >= d)       // the warp's block as a whole
                continue;
            const bool ok = c < d;
            v[j] = ok ? g[i + j] - cutoff : 0.f;
            u[j] = ok ? to_float(__ldg(p + d + NT * (i + j))) : 0.f;
            if (ok)
                o[NT * (i + j)] = from_float<T>(sparse_mul(both(v[j]), both(u[j])).x);
            put_block<true>(q + NT * (i + j), s + NT / 32 * (i + j), v[j], ok, lane);
            put_block<false>(q + d + NT * (i + j), s + B + NT / 32 * (i + j), u[j], ok, lane);
        }
    });
}

template <class T, int NT, int V>
__global__ void __launch_bounds__(NT, 1024 / NT)
sparse_backward_any(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                    const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    const float *__restrict__ std_in, int d, int64_t gs, int B, float z) {
    __shared__ float red[NT / 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const float std = std_in[r];
    const int t = threadIdx.x;
    const T *y = grad + r * gs + t;
    const int8_t *q = codes + r * 2 * d + t;
    const uint8_t *s = scales + r * 2 * B + (t >> 5);
    T *gi = grad_in + r * 2 * d + t, *o = out + r * d + t;
    float h[V], acc = 0.f;
    for_groups<NT, V>(t, d, [&](int i, bool full) {
        T dy[4];
        int8_t cg[4], cu[4];
        uint8_t sg[4], su[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (full || t + NT * (i + j) < d) {
                dy[j] = __ldg(y + NT * (i + j));
                cg[j] = __ldg(q + NT * (i + j));
                cu[j] = __ldg(q + d + NT * (i + j));
                sg[j] = __ldg(s + NT / 32 * (i + j));
                su[j] = __ldg(s + B + NT / 32 * (i + j));
            } else {
                dy[j] = from_float<T>(0.f);
                cg[j] = cu[j] = 0;
                sg[j] = su[j] = 0;
            }
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const GateGrad2 m = sparse_grad(
                make_float2(cg[j] * code_step(sg[j]), cg[j + 1] * code_step(sg[j + 1])),
                make_float2(cu[j] * code_step(su[j]), cu[j + 1] * code_step(su[j + 1])),
                make_float2(to_float(dy[j]), to_float(dy[j + 1])));
            h[i + j] = m.gate.x;
            h[i + j + 1] = m.gate.y;
            acc += m.gate.x + m.gate.y;
            const float up[2] = {m.up.x, m.up.y}, again[2] = {m.out.x, m.out.y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (full || t + NT * (i + j + k) < d) {
                    gi[d + NT * (i + j + k)] = from_float<T>(up[k]);
                    if (out)
                        o[NT * (i + j + k)] = from_float<T>(again[k]);
                }
        }
    });
    const float m = row_sum<NT>(acc, red) / static_cast<float>(d);
    const float inv = std == 0.f ? 0.f : z / std;
    for_groups<NT, V>(t, d, [&](int i, bool full) {
#pragma unroll
        for (int j = i; j < i + 4; ++j)
            if (full || t + NT * j < d) {      // the codes again, from L1 or L2
                const float v = __ldg(q + NT * j) * code_step(__ldg(s + NT / 32 * j));
                gi[NT * j] = from_float<T>(fmaf(-m, fmaf(inv, fmaf(z, std, v), 1.f), h[j]));
            }
    });
}

// ----------------------------------------- sparse, rows that no CTA holds

constexpr int kWideThreads = 1024, kWideWarps = kWideThreads / 32;

// One CTA per row; the gate is read again (from L1/L2) for each pass.  100 x 40000
// bf16: 41.0 us forward, 50.7 us backward (256 threads: 115.6 and 166.9): a row's
// latency bounds so few of them.
template <class T>
__global__ void __launch_bounds__(kWideThreads)
sparse_forward_wide(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   float *__restrict__ std_out, const T *__restrict__ in, int64_t rows, int64_t d,
                   int64_t rs, int64_t B, float z) {
    __shared__ float red[2][kWideWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *g = in + r * rs;
        const float first = to_float(g[0]);
        uint32_t other = 0u;
        float acc = 0.f;
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float x = to_float(g[c]);
            acc += x;
            other |= unlike(x, first);
        }
        const float mean =
            row_mean<kWideThreads>(acc, red[0], other, first, static_cast<float>(d));
        acc = 0.f;
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float e = to_float(g[c]) - mean;
            acc = fmaf(e, e, acc);
        }
        const float std = __fsqrt_rn(row_sum<kWideThreads>(acc, red[1]) / static_cast<float>(d));
        const float cutoff = fmaf(std, z, mean);
        if (threadIdx.x == 0)
            std_out[r] = std;
        for (int64_t b = warp; b < B; b += kWideWarps) {
            const int64_t c = b * kBlock + lane;
            const bool ok = c < d;
            const float v = ok ? to_float(g[c]) - cutoff : 0.f;
            const float u = ok ? to_float(g[d + c]) : 0.f;
            if (ok)
                out[r * d + c] = from_float<T>(sparse_mul(both(v), both(u)).x);
            put_block<true>(codes + r * 2 * d + c, scales + r * 2 * B + b, v, ok, lane);
            put_block<false>(codes + r * 2 * d + d + c, scales + r * 2 * B + B + b, u, ok, lane);
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kWideThreads)
sparse_backward_wide(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                    const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    const float *__restrict__ std_in, int64_t rows, int64_t d, int64_t gs,
                    int64_t B, float z) {
    __shared__ float red[2][kWideWarps];
    pdl_wait();
    pdl_trigger();
    int k = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, k ^= 1) {
        const float std = std_in[r];
        const float inv = std == 0.f ? 0.f : z / std;
        const int8_t *q = codes + r * 2 * d;
        const uint8_t *sc = scales + r * 2 * B;
        T *gi = grad_in + r * 2 * d;
        float acc = 0.f;
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float v = q[c] * code_step(sc[c / kBlock]);
            const float u = q[d + c] * code_step(sc[B + c / kBlock]);
            const float dy = to_float(grad[r * gs + c]);
            const GateGrad2 m = sparse_grad(both(v), both(u), both(dy));
            acc += m.gate.x;
            gi[d + c] = from_float<T>(m.up.x);
            if (out)
                out[r * d + c] = from_float<T>(m.out.x);
        }
        const float mean_h = row_sum<kWideThreads>(acc, red[k]) / static_cast<float>(d);
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float v = q[c] * code_step(sc[c / kBlock]);
            const float u = q[d + c] * code_step(sc[B + c / kBlock]);
            const float dy = to_float(grad[r * gs + c]);
            const float h = sparse_grad(both(v), both(u), both(dy)).gate.x;
            gi[c] = from_float<T>(fmaf(-mean_h, fmaf(inv, fmaf(z, std, v), 1.f), h));
        }
    }
}

// -------------------------------------------------------- sparse, vectors
//
// One CTA per row, the row in registers: thread t holds the 8-element vectors
// t, t + NT, ... (V of them) of both halves, so the gate is read once for its
// statistics and its codes, and four neighbouring lanes hold a block.  All
// loads are issued before the first sum.  The barriers of the statistics, at
// which a CTA neither reads nor writes, keep it from the copy rate: 4000 x 4096 bf16
// takes 22.6 us forward (86%), 500 x 32768 31.9 forward and 43.3 us backward (61 and
// 56%), 300 x 32768 fp32 33.9 us forward, 8 x 8192 fp32 2.7 and 3.9 us (launch and latency).

// The output and the codes of the 8 elements at column c of a row (nothing for
// c >= d, but the lane takes part in its block's largest magnitudes).
template <class T>
__device__ __forceinline__ void finish_vec(const Vec8<T> &g, const Vec8<T> &u, float cutoff, int c,
                                           int d, T *out, int8_t *codes, uint8_t *scales, int B) {
    float2 v[4], w[4];
    Vec8<T> o;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = sub2(g.pair(j), both(cutoff));
        w[j] = u.pair(j);
        top = max_abs(top, v[j]);
        o.put(j, sparse_mul(v[j], w[j]));
    }
    uint32_t tg = c < d ? __float_as_uint(top) : 0u, tu = c < d ? u.top() : 0u;
    block_tops<float>(&tg, &tu);   // 32-bit keys; u's own order is that of its type
    if (c >= d)
        return;
    const uint32_t sg = scale_of(tg), su = scale_of(top_as_float<T>(tu));
    o.store(out + c);
    st_u2(codes + c, codes_of<true>(v, sg));
    st_u2(codes + d + c, codes_of<false>(w, su));
    if (c % kBlock == 0) {
        uint8_t *s = scales + c / kBlock;
        s[0] = static_cast<uint8_t>(sg);
        s[B] = static_cast<uint8_t>(su);
    }
}

template <class T, int NT, int V>
__global__ void __launch_bounds__(NT)
sparse_forward_vec(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   float *__restrict__ std_out, const T *__restrict__ in, int d, int64_t rs,
                   int B, float z) {
    __shared__ float red[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const T *p = in + r * rs;
    constexpr bool kRound = kSumsRound<T, NT * V>;    // whole vectors: multiples of 8 elements
    const T first = kRound ? __ldg(p) : T{};
    Vec8<T> g[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        g[i] = c < d ? Vec8<T>::load(p + c) : Vec8<T>::zero();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        u[i] = c < d ? Vec8<T>::load(p + d + c) : Vec8<T>::zero();
    }
    float2 acc = make_float2(0.f, 0.f);
    uint32_t other = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = add2(acc, g[i].pair(j));
        if constexpr (kRound)
            if (8 * (threadIdx.x + NT * i) < d)
                other |= unlike(g[i], first);
    }
    const float n = static_cast<float>(d);
    float mean;
    if constexpr (kRound)
        mean = row_mean<NT>(acc.x + acc.y, red[0], other, to_float(first), n);
    else
        mean = row_sum<NT>(acc.x + acc.y, red[0]) / n;
    acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (8 * (threadIdx.x + NT * i) < d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 e = sub2(g[i].pair(j), make_float2(mean, mean));
                acc = fma2(e, e, acc);
            }
    const float std = __fsqrt_rn(row_sum<NT>(acc.x + acc.y, red[1]) / n);
    const float cutoff = fmaf(std, z, mean);
    if (threadIdx.x == 0)
        std_out[r] = std;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        finish_vec(g[i], u[i], cutoff, c, d, out + r * d, codes + r * 2 * d, scales + r * 2 * B, B);
    }
}

template <class T, int NT, int V>
__global__ void __launch_bounds__(NT)
sparse_backward_vec(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                    const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    const float *__restrict__ std_in, int d, int64_t gs, int B, float z) {
    __shared__ float red[NT / 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const float std = std_in[r];
    const T *y = grad + r * gs;
    const int8_t *q = codes + r * 2 * d;
    const uint8_t *sc = scales + r * 2 * B;
    T *gi = grad_in + r * 2 * d;
    Vec8<T> dy[V];
    uint2 cg[V], cu[V];
    uint32_t sg[V], su[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        if (c < d) {
            cg[i] = ld_stream_u2(q + c);
            cu[i] = ld_stream_u2(q + d + c);
            dy[i] = Vec8<T>::load(y + c);
            sg[i] = __ldg(sc + c / kBlock);
            su[i] = __ldg(sc + B + c / kBlock);
        }
    }
    // h, and the two outputs that do not wait for its sum
    float2 h[V][4], acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        if (c >= d)
            continue;
        const uint2 bg = bias_codes(cg[i]), bu = bias_codes(cu[i]);
        const float stg = code_step(sg[i]), stu = code_step(su[i]);
        Vec8<T> ou, oo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = decode_pair(bg, j, stg), u = decode_pair(bu, j, stu);
            const float2 t = dy[i].pair(j);
            const GateGrad2 m = sparse_grad(v, u, t);
            h[i][j] = m.gate;
            acc = add2(acc, m.gate);
            ou.put(j, m.up);
            oo.put(j, m.out);
        }
        ou.store(gi + d + c);
        if (out)
            oo.store(out + r * d + c);
    }
    // grad = h - m (1 + inv (delta + z std)), m the mean of h, inv = z / std
    const float m = row_sum<NT>(acc.x + acc.y, red) / static_cast<float>(d);
    const float inv = std == 0.f ? 0.f : z / std;
    const float2 zs = make_float2(z * std, z * std), inv2 = make_float2(inv, inv),
                 one = make_float2(1.f, 1.f), m2 = make_float2(-m, -m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        if (c >= d)
            continue;
        const uint2 bg = bias_codes(cg[i]);
        const float stg = code_step(sg[i]);
        Vec8<T> og;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            og.put(j, fma2(m2, fma2(inv2, add2(decode_pair(bg, j, stg), zs), one), h[i][j]));
        og.store(gi + c);
    }
}

// ----------------------------------------------------------- sparse, a ring
//
// The same with persistent CTAs: CTA b takes the rows b, b + G, ..., which
// reach it through a ring of S shared-memory slots that cp.async fills S - 1
// rows ahead, so that HBM keeps streaming while a row is summed and written.  A
// thread copies just the vectors it will read itself: its own wait_group is
// all the synchronization that the ring needs.  2048 x 16384 bf16: forward 48.6 us
// (82%), backward 57.3 us (87%); with_ring_cta has the figures without it.

template <class T, int NT, int V, int S>
__global__ void __launch_bounds__(NT, 1024 / NT)
sparse_forward_ring(T *__restrict__ out, int8_t *__restrict__ codes,
                    uint8_t *__restrict__ scales, float *__restrict__ std_out,
                    const T *__restrict__ in, int64_t rows, int d, int64_t rs, int B, float z) {
    constexpr int P = sizeof(T) / 2;                // 16-byte pieces of a vector
    extern __shared__ __align__(16) uint4 ring[];   // [S][2][V][P][NT]
    __shared__ float red[2][NT / 32];
    const int t = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int64_t G = gridDim.x;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16u * t;
    const auto fetch = [&](int64_t r, int slot) {
        if (r < rows) {
            const T *p = in + r * rs + 8 * t;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (8 * (t + NT * i) < d)
#pragma unroll
                        for (int k = 0; k < P; ++k)
                            copy16(base + 16u * NT * (((slot * 2 + h) * V + i) * P + k),
                                   p + h * d + 8 * NT * i + 16 / sizeof(T) * k);
        }
        copy_commit();
    };
    const auto held = [&](int slot, int h, int i) {
        Vec8<T> v = Vec8<T>::zero();
        if (8 * (t + NT * i) < d) {
            uint4 *q = reinterpret_cast<uint4 *>(&v);
#pragma unroll
            for (int k = 0; k < P; ++k)
                q[k] = ring[(((slot * 2 + h) * V + i) * P + k) * NT + t];
        }
        return v;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        fetch(blockIdx.x + k * G, k);
    int slot = 0;
    const float n = static_cast<float>(d);
    for (int64_t r = blockIdx.x; r < rows; r += G) {
        // the slot read in the round before: this thread is done with it
        fetch(r + (S - 1) * G, slot == 0 ? S - 1 : slot - 1);
        copy_wait<S - 1>();
        Vec8<T> g[V];
        float2 acc = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = held(slot, 0, i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = add2(acc, g[i].pair(j));
        }
        static_assert(!kSumsRound<T, NT * V>, "the mean of a constant row");
        const float mean = row_sum<NT>(acc.x + acc.y, red[0]) / n;
        acc = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (8 * (t + NT * i) < d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 e = sub2(g[i].pair(j), both(mean));
                    acc = fma2(e, e, acc);
                }
        const float std = __fsqrt_rn(row_sum<NT>(acc.x + acc.y, red[1]) / n);
        const float cutoff = fmaf(std, z, mean);
        if (t == 0)
            std_out[r] = std;
#pragma unroll
        for (int i = 0; i < V; ++i)
            finish_vec(g[i], held(slot, 1, i), cutoff, 8 * (t + NT * i), d, out + r * d,
                       codes + r * 2 * d, scales + r * 2 * B, B);
        slot = slot == S - 1 ? 0 : slot + 1;
    }
}

template <class T, int NT, int V, int S>
__global__ void __launch_bounds__(NT, 1024 / NT)
sparse_backward_ring(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                     const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                     const float *__restrict__ std_in, int64_t rows, int d, int64_t gs, int B,
                     float z) {
    constexpr int P = sizeof(T) / 2;
    extern __shared__ __align__(16) uint4 ring[];          // [S][V][P][NT], then the codes:
    uint2 *const ring8 = reinterpret_cast<uint2 *>(ring + S * V * P * NT);   // [S][2][V][NT]
    __shared__ float red[2][NT / 32];
    const int t = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int64_t G = gridDim.x;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16u * t;
    const uint32_t base8 = static_cast<uint32_t>(__cvta_generic_to_shared(ring8)) + 8u * t;
    const auto fetch = [&](int64_t r, int slot) {
        if (r < rows) {
            const T *y = grad + r * gs + 8 * t;
            const int8_t *q = codes + r * 2 * d + 8 * t;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (8 * (t + NT * i) < d) {
                    copy8(base8 + 8u * NT * ((slot * 2) * V + i), q + 8 * NT * i);
                    copy8(base8 + 8u * NT * ((slot * 2 + 1) * V + i), q + d + 8 * NT * i);
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        copy16(base + 16u * NT * ((slot * V + i) * P + k),
                               y + 8 * NT * i + 16 / sizeof(T) * k);
                }
        }
        copy_commit();
    };
    // the scales are read a row ahead too, into registers: bytes have no cp.async
    uint32_t sg[V], su[V];
    float std = 0.f;
    const auto fetch_scales = [&](int64_t r) {
        if (r >= rows)
            return;
        const uint8_t *sc = scales + r * 2 * B + t / 4;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (8 * (t + NT * i) < d) {
                sg[i] = __ldg(sc + NT / 4 * i);
                su[i] = __ldg(sc + B + NT / 4 * i);
            }
        std = __ldg(std_in + r);
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        fetch(blockIdx.x + k * G, k);
    fetch_scales(blockIdx.x);
    int slot = 0, k = 0;
    for (int64_t r = blockIdx.x; r < rows; r += G, k ^= 1) {
        fetch(r + (S - 1) * G, slot == 0 ? S - 1 : slot - 1);
        copy_wait<S - 1>();
        T *gi = grad_in + r * 2 * d;
        float2 h[V][4], acc = both(0.f);
        float step[V];
        const float dev = std;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + NT * i);
            if (c >= d)
                continue;
            step[i] = code_step(sg[i]);
            const float stu = code_step(su[i]);
            const uint2 bg = bias_codes(ring8[((slot * 2) * V + i) * NT + t]);
            const uint2 bu = bias_codes(ring8[((slot * 2 + 1) * V + i) * NT + t]);
            Vec8<T> dy, ou, oo;
            uint4 *q = reinterpret_cast<uint4 *>(&dy);
#pragma unroll
            for (int p = 0; p < P; ++p)
                q[p] = ring[((slot * V + i) * P + p) * NT + t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const GateGrad2 m = sparse_grad(decode_pair(bg, j, step[i]), decode_pair(bu, j, stu),
                                                dy.pair(j));
                h[i][j] = m.gate;
                acc = add2(acc, m.gate);
                ou.put(j, m.up);
                oo.put(j, m.out);
            }
            ou.store(gi + d + c);
            if (out)
                oo.store(out + r * d + c);
        }
        fetch_scales(r + G);
        // grad = h - m (1 + inv (delta + z std)), m the mean of h, inv = z / std
        const float m = row_sum<NT>(acc.x + acc.y, red[k]) / static_cast<float>(d);
        const float inv = dev == 0.f ? 0.f : z / dev;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + NT * i);
            if (c >= d)
                continue;
            const uint2 bg = bias_codes(ring8[((slot * 2) * V + i) * NT + t]);
            Vec8<T> og;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                og.put(j, fma2(both(-m), fma2(both(inv), add2(decode_pair(bg, j, step[i]), both(z * dev)),
                                              both(1.f)), h[i][j]));
            og.store(gi + c);
        }
        slot = slot == S - 1 ? 0 : slot + 1;
    }
}

// -------------------------------------------------------------- host side

int check_sizes(int64_t M, int64_t d, int64_t stride, int64_t width, int dtype) {
    if (M < 0 || d <= 0)
        return GATED_ACT_ERR_SIZE;
    if (stride < width)
        return GATED_ACT_ERR_STRIDE;
    if (!elem_size(dtype))
        return GATED_ACT_ERR_DTYPE;
    if (d > kMaxWidth || M > kMaxRows || stride > kMaxRows ||
        (M > 0 && std::max(stride, 2 * d) > (int64_t(1) << 60) / M))
        return GATED_ACT_ERR_TOO_LARGE;
    return GATED_ACT_OK;
}

dim3 grid_of(int64_t units, int64_t per_cta) {
    // grid-stride kernels: at most 64 CTAs per SM
    return dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div64(units, per_cta),
                                                        int64_t(device_sm_count()) * 64)));
}

// Calls f(I{}, grid) for `slots` slots, VPT per thread, with I the type that
// their indexes take: 32 bits where they fit.
template <class F> int with_index(int64_t slots, int vpt, F f) {
    const int64_t per = int64_t(kThreads) * vpt, grid = ceil_div64(slots, per);
    if (grid > 0x7FFFFFFF)
        return GATED_ACT_ERR_TOO_LARGE;
    const dim3 g(static_cast<unsigned>(grid));
    return slots + per < (int64_t(1) << 31) ? f(uint32_t{}, g) : f(int64_t{}, g);
}

// Calls f(I{}, grid) for `jobs` jobs of a warp each, as with_index.
template <class F> int with_jobs(int64_t jobs, F f) {
    const int64_t grid = ceil_div64(jobs, kWarps);
    if (grid > 0x7FFFFFFF)
        return GATED_ACT_ERR_TOO_LARGE;
    const dim3 g(static_cast<unsigned>(grid));
    return jobs + kWarps < (int64_t(1) << 31) ? f(uint32_t{}, g) : f(int64_t{}, g);
}

// The CTA that holds a row of d elements one by one, as with_row_cta.
template <class F> bool with_any_cta(int64_t d, int *rc, F f) {
    if (d <= 512)
        *rc = f(Const<64>{}, Const<8>{});
    else if (d <= 1024)
        *rc = f(Const<64>{}, Const<16>{});
    else if (d <= 2048)
        *rc = f(Const<128>{}, Const<16>{});
    else if (d <= 4096)
        *rc = f(Const<256>{}, Const<16>{});
    else if (d <= 8192)
        *rc = f(Const<512>{}, Const<16>{});
    else if (d <= 16384)
        *rc = f(Const<1024>{}, Const<16>{});
    else if (d <= 32768)
        *rc = f(Const<1024>{}, Const<32>{});
    else
        return false;
    return true;
}

// Calls f(integral constants NT, V) for rows of nv 8-element vectors held by
// one CTA, at most MAX of them per thread; false when no such CTA holds them.
template <int MAX, class F> bool with_row_cta(int64_t nv, int *rc, F f) {
    if (nv <= 128)
        *rc = f(Const<128>{}, Const<1>{});
    else if (nv <= 256)
        *rc = f(Const<256>{}, Const<1>{});
    else if (nv <= 512)
        *rc = f(Const<256>{}, Const<2>{});
    else if (nv <= 1024)
        *rc = f(Const<512>{}, Const<2>{});
    else if (nv <= 2048)
        *rc = f(Const<1024>{}, Const<2>{});
    else if constexpr (MAX < 4)
        return false;
    else if (nv <= 4096)
        *rc = f(Const<1024>{}, Const<4>{});
    else
        return false;
    return true;
}

// Persistent CTAs, 1024 threads per SM.
dim3 ring_grid(int nt) { return dim3(static_cast<unsigned>(device_sm_count() * (1024 / nt))); }

// Calls f(integral constant NT) for the ring over T rows of nv vectors, two per
// thread; false for rows that do not take it: those of more or fewer vectors, and
// batches of no more than two rows per CTA, where filling the ring costs what it
// hides (608 x 8192 bf16 forward 10.6 us in the ring and 9.9 without, 450 x 8192 backward
// 10.6 and 9.7; 1216 x 8192 16.6 and 17.7, 19.8 and 21.7).  In the ring and without, bf16:
//                  8000 x 2048   4000 x 4096   4000 x 8192   2048 x 16384
//   forward, us    22.8  25.1    23.2  22.5    44.8  50.2    48.5  62.4
//   backward, us   29.7  31.0    29.9  32.7    55.3  64.4    56.4  76.3
// The forward pass leaves out the class of its one loss, which loses at other sizes too
// (8000 x 2304 35.7 us against 32.8, 4000 x 3328 21.2 against 20.5).  It has two slots,
// with three 2048 x 16384 takes 49.0 us; the backward pass three, with two 65.3.  fp32
// rows that wide would not leave room for slots to fill ahead, and reach 91 to 94% of
// the copy rate without.
template <bool FORWARD, class F> bool with_ring_cta(int64_t T, int64_t nv, int *rc, F f) {
    if (nv <= 128 || nv > 2048 || (FORWARD && nv > 256 && nv <= 512))
        return false;
    const int nt = nv <= 256 ? 128 : nv <= 512 ? 256 : nv <= 1024 ? 512 : 1024;
    if (T <= int64_t(2) * device_sm_count() * (1024 / nt))
        return false;
    if (nt == 128)
        *rc = f(Const<128>{});
    else if (nt == 512)
        *rc = f(Const<512>{});
    else if (nt == 1024)
        *rc = f(Const<1024>{});
    else if constexpr (!FORWARD)
        *rc = f(Const<256>{});
    return true;
}

constexpr int kForwardVpt = 1, kBackwardVpt = 1, kValuesVpt = 4;   // slots per thread

template <class Act>
int forward(void *out, int8_t *codes, uint8_t *scales, const void *in, int64_t M, int64_t d,
            int64_t rs, int dtype, const int32_t *n_rows, cudaStream_t stream) {
    int rc = check_sizes(M, d, rs, 2 * d, dtype);
    if (rc != GATED_ACT_OK || M == 0)
        return rc;
    const int64_t B = ceil_div64(d, kBlock), size = elem_size(dtype);
    Region r[5] = {{out, static_cast<uint64_t>(M * d * size), uintptr_t(size), true},
                   {codes, static_cast<uint64_t>(M * 2 * d), 1, true},
                   {scales, static_cast<uint64_t>(M * 2 * B), 1, true},
                   {in, span_bytes(M, rs, 2 * d, size), uintptr_t(size), false},
                   {n_rows, n_rows ? 4u : 0u, 4, false}};
    if ((rc = check_regions(r, 5)) != GATED_ACT_OK)
        return rc;
    const bool vec = d % 8 == 0 && rs % 8 == 0 && aligned(r[0].dev, 8 * size) && aligned(r[1].dev, 8) &&
                     aligned(r[3].dev, 8 * size);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (vec) {
            constexpr int VPT = kForwardVpt;
            return with_index(M * 4 * B, VPT, [&](auto idx, dim3 grid) {
                using I = decltype(idx);
                return launched(launch_kernel(
                    ckpt_forward_vec<T, Act, VPT, I>, grid, dim3(kThreads), 0, stream, 1,
                    as<T>(r[0]), as<int8_t>(r[1]), as<uint8_t>(r[2]), as<const T>(r[3]), M,
                    static_cast<I>(d), rs, static_cast<I>(B), FastDiv(static_cast<uint32_t>(4 * B)),
                    as<const int32_t>(r[4])));
            });
        }
        const int64_t J = ceil_div64(B, kAnyBlocks);
        return with_jobs(M * J, [&](auto idx, dim3 grid) {
            using I = decltype(idx);
            return launched(launch_kernel(
                ckpt_forward_any<T, Act, I>, grid, dim3(kThreads), 0, stream, 1, as<T>(r[0]),
                as<int8_t>(r[1]), as<uint8_t>(r[2]), as<const T>(r[3]), M, d, rs, B,
                static_cast<I>(J), FastDiv(static_cast<uint32_t>(J)), as<const int32_t>(r[4])));
        });
    });
}

template <class Act>
int backward(void *grad_in, void *out, const void *grad, const int8_t *codes,
             const uint8_t *scales, int64_t M, int64_t d, int64_t gs, int dtype,
             const int32_t *n_rows, cudaStream_t stream) {
    int rc = check_sizes(M, d, gs, d, dtype);
    if (rc != GATED_ACT_OK || M == 0)
        return rc;
    const int64_t B = ceil_div64(d, kBlock), size = elem_size(dtype);
    Region r[6] = {{grad_in, static_cast<uint64_t>(M * 2 * d * size), uintptr_t(size), true},
                   {out, out ? static_cast<uint64_t>(M * d * size) : 0, uintptr_t(size), true},
                   {grad, span_bytes(M, gs, d, size), uintptr_t(size), false},
                   {codes, static_cast<uint64_t>(M * 2 * d), 1, false},
                   {scales, static_cast<uint64_t>(M * 2 * B), 1, false},
                   {n_rows, n_rows ? 4u : 0u, 4, false}};
    if ((rc = check_regions(r, 6)) != GATED_ACT_OK)
        return rc;
    const bool vec = d % 8 == 0 && gs % 8 == 0 && aligned(r[0].dev, 8 * size) && aligned(r[1].dev, 8 * size) &&
                     aligned(r[2].dev, 8 * size) && aligned(r[3].dev, 8);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (vec) {
            constexpr int VPT = kBackwardVpt;
            return with_index(M * (d / 8), VPT, [&](auto idx, dim3 grid) {
                using I = decltype(idx);
                return launched(launch_kernel(
                    ckpt_backward_vec<T, Act, VPT, I>, grid, dim3(kThreads), 0, stream, 1,
                    as<T>(r[0]), as<T>(r[1]), as<const T>(r[2]), as<const int8_t>(r[3]),
                    as<const uint8_t>(r[4]), M, static_cast<I>(d), gs, static_cast<I>(B),
                    FastDiv(static_cast<uint32_t>(d / 8)), as<const int32_t>(r[5])));
            });
        }
        const int64_t J = ceil_div64(B, kAnyBlocks);
        return with_jobs(M * J, [&](auto idx, dim3 grid) {
            using I = decltype(idx);
            return launched(launch_kernel(
                ckpt_backward_any<T, Act, I>, grid, dim3(kThreads), 0, stream, 1, as<T>(r[0]),
                as<T>(r[1]), as<const T>(r[2]), as<const int8_t>(r[3]), as<const uint8_t>(r[4]), M,
                d, gs, B, static_cast<I>(J), FastDiv(static_cast<uint32_t>(J)),
                as<const int32_t>(r[5])));
        });
    });
}

}  // namespace
}  // namespace gact

extern "C" int64_t gated_act_checkpoint_scales(int64_t d) {
    return d <= 0 ? 0 : 2 * ((d - 1) / gact::kBlock + 1);
}

extern "C" int silu_and_mul_checkpoint(void *out, int8_t *codes, uint8_t *scales, const void *in,
                                       int64_t M, int64_t d, int64_t row_stride, int dtype,
                                       const int32_t *n_rows, cudaStream_t stream) {
    return gact::forward<gact::Silu>(out, codes, scales, in, M, d, row_stride, dtype, n_rows,
                                     stream);
}

extern "C" int gelu_and_mul_checkpoint(void *out, int8_t *codes, uint8_t *scales, const void *in,
                                       int64_t M, int64_t d, int64_t row_stride, int dtype,
                                       const int32_t *n_rows, cudaStream_t stream) {
    return gact::forward<gact::Gelu>(out, codes, scales, in, M, d, row_stride, dtype, n_rows,
                                     stream);
}

extern "C" int silu_and_mul_backward(void *grad_in, void *out, const void *grad_out,
                                     const int8_t *codes, const uint8_t *scales, int64_t M,
                                     int64_t d, int64_t grad_stride, int dtype,
                                     const int32_t *n_rows, cudaStream_t stream) {
    return gact::backward<gact::Silu>(grad_in, out, grad_out, codes, scales, M, d, grad_stride,
                                      dtype, n_rows, stream);
}

extern "C" int gelu_and_mul_backward(void *grad_in, void *out, const void *grad_out,
                                     const int8_t *codes, const uint8_t *scales, int64_t M,
                                     int64_t d, int64_t grad_stride, int dtype,
                                     const int32_t *n_rows, cudaStream_t stream) {
    return gact::backward<gact::Gelu>(grad_in, out, grad_out, codes, scales, M, d, grad_stride,
                                      dtype, n_rows, stream);
}

extern "C" int gelu_and_mul_sparse_checkpoint(void *out, int8_t *codes, uint8_t *scales,
                                              float *std, const void *in, int64_t T, int64_t d,
                                              int64_t row_stride, double z, int dtype,
                                              cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, d, row_stride, 2 * d, dtype);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    const int64_t B = ceil_div64(d, kBlock), size = elem_size(dtype);
    Region r[5] = {{out, static_cast<uint64_t>(T * d * size), uintptr_t(size), true},
                   {codes, static_cast<uint64_t>(T * 2 * d), 1, true},
                   {scales, static_cast<uint64_t>(T * 2 * B), 1, true},
                   {std, static_cast<uint64_t>(T * 4), 4, true},
                   {in, span_bytes(T, row_stride, 2 * d, size), uintptr_t(size), false}};
    if ((rc = check_regions(r, 5)) != GATED_ACT_OK)
        return rc;
    const bool vec = d % 8 == 0 && row_stride % 8 == 0 && aligned(r[0].dev, 8 * size) &&
                     aligned(r[1].dev, 8) && aligned(r[4].dev, 8 * size) && T <= 0x7FFFFFFF;
    return with_type(dtype, [&](auto t) {
        using E = decltype(t);
        const auto go = [&](auto nt, auto v) {
            return launched(launch_kernel(
                sparse_forward_vec<E, nt(), v()>, dim3(static_cast<unsigned>(T)), dim3(nt()), 0,
                stream, 1, as<E>(r[0]), as<int8_t>(r[1]), as<uint8_t>(r[2]), as<float>(r[3]),
                as<const E>(r[4]), static_cast<int>(d), row_stride, static_cast<int>(B),
                static_cast<float>(z)));
        };
        int done;
        if constexpr (sizeof(E) == 2) {
            const auto ring = [&](auto nt) {
                constexpr int kSlots = 2;
                constexpr size_t smem = kSlots * 2 * nt() * 16 * sizeof(E);
                const auto kernel = sparse_forward_ring<E, nt(), 2, kSlots>;
                const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
                if (e != cudaSuccess)
                    return cuda_status(e);
                return launched(launch_kernel(
                    kernel, ring_grid(nt()), dim3(nt()), smem, stream, 1, as<E>(r[0]),
                    as<int8_t>(r[1]), as<uint8_t>(r[2]), as<float>(r[3]), as<const E>(r[4]), T,
                    static_cast<int>(d), row_stride, static_cast<int>(B), static_cast<float>(z)));
            };
            if (vec && with_ring_cta<true>(T, d / 8, &done, ring))
                return done;
        }
        if (vec && with_row_cta<4>(d / 8, &done, go))
            return done;
        const auto any = [&](auto nt, auto v) {
            return launched(launch_kernel(
                sparse_forward_any<E, nt(), v()>, dim3(static_cast<unsigned>(T)), dim3(nt()), 0,
                stream, 1, as<E>(r[0]), as<int8_t>(r[1]), as<uint8_t>(r[2]), as<float>(r[3]),
                as<const E>(r[4]), static_cast<int>(d), row_stride, static_cast<int>(B),
                static_cast<float>(z)));
        };
        if (T <= 0x7FFFFFFF && with_any_cta(d, &done, any))
            return done;
        return launched(launch_kernel(sparse_forward_wide<E>, grid_of(T, 1), dim3(kWideThreads), 0,
                                      stream, 1, as<E>(r[0]), as<int8_t>(r[1]), as<uint8_t>(r[2]),
                                      as<float>(r[3]), as<const E>(r[4]), T, d, row_stride, B,
                                      static_cast<float>(z)));
    });
}

extern "C" int gelu_and_mul_sparse_backward(void *grad_in, void *out, const void *grad_out,
                                            const int8_t *codes, const uint8_t *scales,
                                            const float *std, int64_t T, int64_t d,
                                            int64_t grad_stride, double z, int dtype,
                                            cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, d, grad_stride, d, dtype);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    const int64_t B = ceil_div64(d, kBlock), size = elem_size(dtype);
    Region r[6] = {{grad_in, static_cast<uint64_t>(T * 2 * d * size), uintptr_t(size), true},
                   {out, out ? static_cast<uint64_t>(T * d * size) : 0, uintptr_t(size), true},
                   {grad_out, span_bytes(T, grad_stride, d, size), uintptr_t(size), false},
                   {codes, static_cast<uint64_t>(T * 2 * d), 1, false},
                   {scales, static_cast<uint64_t>(T * 2 * B), 1, false},
                   {std, static_cast<uint64_t>(T * 4), 4, false}};
    if ((rc = check_regions(r, 6)) != GATED_ACT_OK)
        return rc;
    const bool vec = d % 8 == 0 && grad_stride % 8 == 0 && aligned(r[0].dev, 8 * size) &&
                     aligned(r[1].dev, 8 * size) && aligned(r[2].dev, 8 * size) && aligned(r[3].dev, 8) &&
                     T <= 0x7FFFFFFF;
    return with_type(dtype, [&](auto t) {
        using E = decltype(t);
        const auto go = [&](auto nt, auto v) {
            return launched(launch_kernel(
                sparse_backward_vec<E, nt(), v()>, dim3(static_cast<unsigned>(T)), dim3(nt()), 0,
                stream, 1, as<E>(r[0]), as<E>(r[1]), as<const E>(r[2]), as<const int8_t>(r[3]),
                as<const uint8_t>(r[4]), as<const float>(r[5]), static_cast<int>(d), grad_stride,
                static_cast<int>(B), static_cast<float>(z)));
        };
        int done;
        if constexpr (sizeof(E) == 2) {
            const auto ring = [&](auto nt) {
                constexpr int kSlots = 3;
                constexpr size_t smem = kSlots * 2 * nt() * (8 * sizeof(E) + 16);
                const auto kernel = sparse_backward_ring<E, nt(), 2, kSlots>;
                const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
                if (e != cudaSuccess)
                    return cuda_status(e);
                return launched(launch_kernel(
                    kernel, ring_grid(nt()), dim3(nt()), smem, stream, 1, as<E>(r[0]),
                    as<E>(r[1]), as<const E>(r[2]), as<const int8_t>(r[3]), as<const uint8_t>(r[4]),
                    as<const float>(r[5]), T, static_cast<int>(d), grad_stride,
                    static_cast<int>(B), static_cast<float>(z)));
            };
            if (vec && with_ring_cta<false>(T, d / 8, &done, ring))
                return done;
        }
        // fp32 rows of more than 16384 elements would spill: element by element they take
        // 49.8 us at 300 x 32768 against 69.4, at 2048 x 16384 the vectors 94.5 against 141.4
        if (vec && with_row_cta<sizeof(E) == 2 ? 4 : 2>(d / 8, &done, go))
            return done;
        const auto any = [&](auto nt, auto v) {
            return launched(launch_kernel(
                sparse_backward_any<E, nt(), v()>, dim3(static_cast<unsigned>(T)), dim3(nt()), 0,
                stream, 1, as<E>(r[0]), as<E>(r[1]), as<const E>(r[2]),
                as<const int8_t>(r[3]), as<const uint8_t>(r[4]), as<const float>(r[5]),
                static_cast<int>(d), grad_stride, static_cast<int>(B), static_cast<float>(z)));
        };
        if (T <= 0x7FFFFFFF && with_any_cta(d, &done, any))
            return done;
        return launched(launch_kernel(sparse_backward_wide<E>, grid_of(T, 1), dim3(kWideThreads), 0,
                                      stream, 1, as<E>(r[0]), as<E>(r[1]), as<const E>(r[2]),
                                      as<const int8_t>(r[3]), as<const uint8_t>(r[4]),
                                      as<const float>(r[5]), T, d, grad_stride, B,
                                      static_cast<float>(z)));
    });
}

extern "C" int gated_act_checkpoint_values(void *values, const int8_t *codes,
                                           const uint8_t *scales, int64_t M, int64_t d, int dtype,
                                           cudaStream_t stream) {
    using namespace gact;
    if (dtype == GATED_ACT_F16)
        return GATED_ACT_ERR_DTYPE;
    int rc = check_sizes(M, d, 2 * d, 2 * d, dtype);
    if (rc != GATED_ACT_OK || M == 0)
        return rc;
    const int64_t B = ceil_div64(d, kBlock), size = elem_size(dtype);
    Region r[3] = {{values, static_cast<uint64_t>(M * 2 * d * size), uintptr_t(size), true},
                   {codes, static_cast<uint64_t>(M * 2 * d), 1, false},
                   {scales, static_cast<uint64_t>(M * 2 * B), 1, false}};
    if ((rc = check_regions(r, 3)) != GATED_ACT_OK)
        return rc;
    return with_type(dtype, [&](auto t) {
        using E = decltype(t);
        if (d % 8 == 0 && aligned(r[0].dev, 8 * size) && aligned(r[1].dev, 8))
            return with_index(M * 2 * (d / 8), kValuesVpt, [&](auto idx, dim3 grid) {
                using I = decltype(idx);
                return launched(launch_kernel(
                    ckpt_values_vec<E, kValuesVpt, I>, grid, dim3(kThreads), 0, stream, 1, as<E>(r[0]),
                    as<const int8_t>(r[1]), as<const uint8_t>(r[2]), static_cast<I>(M * 2 * (d / 8)),
                    static_cast<I>(d / 8), static_cast<I>(B), FastDiv(static_cast<uint32_t>(d / 8))));
            });
        const int64_t J = ceil_div64(B, kAnyBlocks);
        return with_jobs(M * J, [&](auto idx, dim3 grid) {
            using I = decltype(idx);
            return launched(launch_kernel(
                ckpt_values_any<E, I>, grid, dim3(kThreads), 0, stream, 1, as<E>(r[0]),
                as<const int8_t>(r[1]), as<const uint8_t>(r[2]), M, d, B, static_cast<I>(J),
                FastDiv(static_cast<uint32_t>(J))));
        });
    });
}
