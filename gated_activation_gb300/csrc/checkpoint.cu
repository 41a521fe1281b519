// 8-bit checkpoints of the gated activations, and the backward passes that
// read them (definitions in gated_act_training.h).
//
// Each op reads and writes every byte once and computes a few dozen
// instructions per element: HBM bandwidth bounds it.  Per gate/up pair of a
// 16-bit type the forward pass moves 4 + 2 bytes of rows and 2 + 1/16 of
// checkpoint, the backward pass 2 (+ 2 with the recomputed output) + 4 and
// the same 2 + 1/16.
//
// Blocks: a block of the 8-bit format is 32 elements of one half.  The
// any-layout kernels give a block of the gate half and the block of the up
// half beside it to one warp, one element per lane, so every access of a warp
// is one contiguous run whatever the alignment, and the block's largest
// magnitude is one redux.
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

// ------------------------------------------------- elementwise, any layout

template <class T, class Act>
__global__ void __launch_bounds__(kThreads)
ckpt_forward_any(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                 const T *__restrict__ in, int64_t M, int64_t d, int64_t rs, int64_t B,
                 const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t total = live_rows(M, n_rows) * B;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < total;
         i += step) {
        const int64_t r = i / B, b = i - r * B, c = b * kBlock + lane;
        const bool ok = c < d;
        const float g = ok ? to_float(in[r * rs + c]) : 0.f;
        const float u = ok ? to_float(in[r * rs + d + c]) : 0.f;
        if (ok)
            out[r * d + c] = from_float<T>(act_mul<Act>(g, u));
        put_block<false>(codes + r * 2 * d + c, scales + r * 2 * B + b, g, ok, lane);
        put_block<false>(codes + r * 2 * d + d + c, scales + r * 2 * B + B + b, u, ok, lane);
    }
}

template <class T, class Act>
__global__ void __launch_bounds__(kThreads)
ckpt_backward_any(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                  const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t M,
                  int64_t d, int64_t gs, int64_t B, const int32_t *n_rows) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t total = live_rows(M, n_rows) * B;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < total;
         i += step) {
        const int64_t r = i / B, b = i - r * B, c = b * kBlock + lane;
        if (c >= d)
            continue;
        const float g = codes[r * 2 * d + c] * code_step(scales[r * 2 * B + b]);
        const float u = codes[r * 2 * d + d + c] * code_step(scales[r * 2 * B + B + b]);
        const float dy = to_float(grad[r * gs + c]);
        const GateGrad m = act_grad<Act>(g, u, dy);
        grad_in[r * 2 * d + c] = from_float<T>(m.gate);
        grad_in[r * 2 * d + d + c] = from_float<T>(m.up);
        if (out)
            out[r * d + c] = from_float<T>(m.out);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
ckpt_values_any(T *__restrict__ values, const int8_t *__restrict__ codes,
                const uint8_t *__restrict__ scales, int64_t M, int64_t d, int64_t B) {
    pdl_wait();
    pdl_trigger();
    const int64_t total = M * 2 * d, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += step) {
        const int64_t h = i / d, c = i - h * d;   // h: half-row
        values[i] = from_float<T>(codes[i] * code_step(scales[h * B + c / kBlock]));
    }
}

// --------------------------------------------------- elementwise, vectors
//
// Rows in 16-byte vectors (pointers and strides allow it, d a multiple of 8):
// a thread takes 8 elements of the gate and the 8 of the up half beside them;
// four neighbouring lanes hold a block of each.  A row is 4 B slots of 8
// elements, B blocks, so that lane groups and blocks coincide in every row;
// the slots past d (a ragged last block) are empty.

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
__global__ void __launch_bounds__(kThreads)
ckpt_forward_vec(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                 const T *__restrict__ in, int64_t M, I d, int64_t rs, I B,
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
        row[i] = s / slots;
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
            o.put(j, make_float2(act_mul<Act>(gf[j].x, uf[j].x), act_mul<Act>(gf[j].y, uf[j].y)));
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
__global__ void __launch_bounds__(kThreads)
ckpt_backward_vec(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                  const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t M,
                  I d, int64_t gs, I B, const int32_t *n_rows) {
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
        row[i] = s / nv;
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
            const GateGrad a = act_grad<Act>(g.x, u.x, y.x), b = act_grad<Act>(g.y, u.y, y.y);
            og.put(j, make_float2(a.gate, b.gate));
            ou.put(j, make_float2(a.up, b.up));
            oo.put(j, make_float2(a.out, b.out));
        }
        const int64_t r = row[i];
        T *p = grad_in + r * 2 * d + col[i];
        og.store(p);
        ou.store(p + d);
        if (out)
            oo.store(out + r * d + col[i]);
    }
}

template <class T, class I>
__global__ void __launch_bounds__(kThreads)
ckpt_values_vec(T *__restrict__ values, const int8_t *__restrict__ codes,
                const uint8_t *__restrict__ scales, I total, I nv, I B) {
    pdl_wait();
    pdl_trigger();
    const I s = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x;
    if (s >= total)
        return;
    const I h = s / nv, v = s - h * nv;                // half-row, vector
    const float step = code_step(__ldg(scales + static_cast<int64_t>(h) * B + v / 4));
    const uint2 b = bias_codes(ld_stream_u2(codes + static_cast<int64_t>(s) * 8));
    Vec8<T> o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o.put(j, decode_pair(b, j, step));
    o.store(values + static_cast<int64_t>(s) * 8);
}

// ------------------------------------------------------ sparse, any layout

// Sum over the CTA, the same bits in every thread; red holds kWarps floats
// and may be used again after the next barrier.
__device__ __forceinline__ float cta_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = red[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1)
        t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return t;
}

// One CTA per row; the gate is read again (from L1/L2) for each pass.
template <class T>
__global__ void __launch_bounds__(kThreads)
sparse_forward_any(T *__restrict__ out, int8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                   float *__restrict__ std_out, const T *__restrict__ in, int64_t rows, int64_t d,
                   int64_t rs, int64_t B, float z) {
    __shared__ float red[2][kWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *g = in + r * rs;
        float acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads)
            acc += to_float(g[c]);
        const float mean = cta_sum(acc, red[0]) / static_cast<float>(d);
        acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float e = to_float(g[c]) - mean;
            acc = fmaf(e, e, acc);
        }
        const float std = __fsqrt_rn(cta_sum(acc, red[1]) / static_cast<float>(d));
        const float cutoff = fmaf(std, z, mean);
        if (threadIdx.x == 0)
            std_out[r] = std;
        for (int64_t b = warp; b < B; b += kWarps) {
            const int64_t c = b * kBlock + lane;
            const bool ok = c < d;
            const float v = ok ? to_float(g[c]) - cutoff : 0.f;
            const float u = ok ? to_float(g[d + c]) : 0.f;
            if (ok)
                out[r * d + c] = from_float<T>(gelu_mul(max_nan(v, 0.f), u));
            put_block<true>(codes + r * 2 * d + c, scales + r * 2 * B + b, v, ok, lane);
            put_block<false>(codes + r * 2 * d + d + c, scales + r * 2 * B + B + b, u, ok, lane);
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
sparse_backward_any(T *__restrict__ grad_in, T *__restrict__ out, const T *__restrict__ grad,
                    const int8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    const float *__restrict__ std_in, int64_t rows, int64_t d, int64_t gs,
                    int64_t B, float z) {
    __shared__ float red[2][kWarps];
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
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float v = q[c] * code_step(sc[c / kBlock]);
            const float u = q[d + c] * code_step(sc[B + c / kBlock]);
            const float dy = to_float(grad[r * gs + c]);
            const GateGrad m = sparse_grad(v, u, dy);
            acc += m.gate;
            gi[d + c] = from_float<T>(m.up);
            if (out)
                out[r * d + c] = from_float<T>(m.out);
        }
        const float mean_h = cta_sum(acc, red[k]) / static_cast<float>(d);
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float v = q[c] * code_step(sc[c / kBlock]);
            const float u = q[d + c] * code_step(sc[B + c / kBlock]);
            const float dy = to_float(grad[r * gs + c]);
            const float h = sparse_grad(v, u, dy).gate;
            gi[c] = from_float<T>(fmaf(-mean_h, fmaf(inv, fmaf(z, std, v), 1.f), h));
        }
    }
}

// -------------------------------------------------------- sparse, vectors
//
// One CTA per row, the row in registers: thread t holds the 8-element vectors
// t, t + NT, ... (V of them) of both halves, so the gate is read once for its
// statistics and its codes, and four neighbouring lanes hold a block.  All
// loads are issued before the first sum.

template <int NT>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    constexpr int NW = NT / 32;
    float t = red[threadIdx.x & (NW - 1)];
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1)
        t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return t;
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
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = add2(acc, g[i].pair(j));
    const float n = static_cast<float>(d);
    const float mean = row_sum<NT>(acc.x + acc.y, red[0]) / n;
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
        float2 v[4], w[4];
        Vec8<T> o;
        uint32_t tg = 0, tu = u[i].top();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = sub2(g[i].pair(j), make_float2(cutoff, cutoff));
            w[j] = u[i].pair(j);
            tg = max(tg, max(abs_bits(v[j].x), abs_bits(v[j].y)));
            o.put(j, make_float2(gelu_mul(max_nan(v[j].x, 0.f), w[j].x),
                                 gelu_mul(max_nan(v[j].y, 0.f), w[j].y)));
        }
        if (c >= d)
            tg = 0;
        block_tops<float>(&tg, &tu);   // 32-bit keys; u's own order is that of its type
        if (c >= d)
            continue;
        const uint32_t sg = scale_of(tg), su = scale_of(top_as_float<T>(tu));
        o.store(out + r * d + c);
        int8_t *q = codes + r * 2 * d + c;
        st_u2(q, codes_of<true>(v, sg));
        st_u2(q + d, codes_of<false>(w, su));
        if (c % kBlock == 0) {
            uint8_t *s = scales + r * 2 * B + c / kBlock;
            s[0] = static_cast<uint8_t>(sg);
            s[B] = static_cast<uint8_t>(su);
        }
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
            const GateGrad a = sparse_grad(v.x, u.x, t.x), b = sparse_grad(v.y, u.y, t.y);
            h[i][j] = make_float2(a.gate, b.gate);
            acc = add2(acc, h[i][j]);
            ou.put(j, make_float2(a.up, b.up));
            oo.put(j, make_float2(a.out, b.out));
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

// -------------------------------------------------------------- host side

constexpr int64_t kMaxWidth = int64_t(1) << 30, kMaxRows = int64_t(1) << 40;

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

// Calls f(integral constants NT, V) for rows of nv 8-element vectors held by
// one CTA; false when no such CTA holds them.
template <int N> using Const = std::integral_constant<int, N>;
template <class F> bool with_row_cta(int64_t nv, int *rc, F f) {
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
    else if (nv <= 4096)
        *rc = f(Const<1024>{}, Const<4>{});
    else
        return false;
    return true;
}

constexpr int kForwardVpt = 1, kBackwardVpt = 1;

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
    const bool vec = d % 8 == 0 && rs % 8 == 0 && aligned(r[0].dev, 16) && aligned(r[1].dev, 8) &&
                     aligned(r[3].dev, 16);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (vec) {
            constexpr int VPT = kForwardVpt;
            return with_index(M * 4 * B, VPT, [&](auto idx, dim3 grid) {
                using I = decltype(idx);
                return launched(launch_kernel(
                    ckpt_forward_vec<T, Act, VPT, I>, grid, dim3(kThreads), 0, stream, 1,
                    as<T>(r[0]), as<int8_t>(r[1]), as<uint8_t>(r[2]), as<const T>(r[3]), M,
                    static_cast<I>(d), rs, static_cast<I>(B), as<const int32_t>(r[4])));
            });
        }
        return launched(launch_kernel(ckpt_forward_any<T, Act>, grid_of(M * B, kWarps),
                                      dim3(kThreads), 0, stream, 1, as<T>(r[0]), as<int8_t>(r[1]),
                                      as<uint8_t>(r[2]), as<const T>(r[3]), M, d, rs, B,
                                      as<const int32_t>(r[4])));
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
    const bool vec = d % 8 == 0 && gs % 8 == 0 && aligned(r[0].dev, 16) && aligned(r[1].dev, 16) &&
                     aligned(r[2].dev, 16) && aligned(r[3].dev, 8);
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
                    as<const int32_t>(r[5])));
            });
        }
        return launched(launch_kernel(ckpt_backward_any<T, Act>, grid_of(M * B, kWarps),
                                      dim3(kThreads), 0, stream, 1, as<T>(r[0]), as<T>(r[1]),
                                      as<const T>(r[2]), as<const int8_t>(r[3]),
                                      as<const uint8_t>(r[4]), M, d, gs, B,
                                      as<const int32_t>(r[5])));
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
    const bool vec = d % 8 == 0 && row_stride % 8 == 0 && aligned(r[0].dev, 16) &&
                     aligned(r[1].dev, 8) && aligned(r[4].dev, 16) && T <= 0x7FFFFFFF;
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
        if (vec && with_row_cta(d / 8, &done, go))
            return done;
        return launched(launch_kernel(sparse_forward_any<E>, grid_of(T, 1), dim3(kThreads), 0,
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
    const bool vec = d % 8 == 0 && grad_stride % 8 == 0 && aligned(r[0].dev, 16) &&
                     aligned(r[1].dev, 16) && aligned(r[2].dev, 16) && aligned(r[3].dev, 8) &&
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
        if (vec && with_row_cta(d / 8, &done, go))
            return done;
        return launched(launch_kernel(sparse_backward_any<E>, grid_of(T, 1), dim3(kThreads), 0,
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
        if (d % 8 == 0 && aligned(r[0].dev, 16) && aligned(r[1].dev, 8))
            return with_index(M * 2 * (d / 8), 1, [&](auto idx, dim3 grid) {
                using I = decltype(idx);
                return launched(launch_kernel(
                    ckpt_values_vec<E, I>, grid, dim3(kThreads), 0, stream, 1, as<E>(r[0]),
                    as<const int8_t>(r[1]), as<const uint8_t>(r[2]), static_cast<I>(M * 2 * (d / 8)),
                    static_cast<I>(d / 8), static_cast<I>(B)));
            });
        return launched(launch_kernel(ckpt_values_any<E>, grid_of(M * 2 * d, kThreads),
                                      dim3(kThreads), 0, stream, 1, as<E>(r[0]),
                                      as<const int8_t>(r[1]), as<const uint8_t>(r[2]), M, d, B));
    });
}
