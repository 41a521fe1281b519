// A router's balance loss, its per-expert counts and the gradient of its
// logits (definitions in gated_act_training.h).
//
// The forward pass reads the logits and the chosen ids once, the backward
// pass reads the logits again (a softmax is recomputed in registers rather
// than stored) and writes their gradient: HBM or L2 bandwidth bounds long
// batches, launch latency short ones.  One warp takes a token: lane l holds
// the logits l, l + 32, ... so any row start is one contiguous run per
// access.  The sums over tokens are kept per lane in registers, joined per CTA
// in shared memory in warp order, and over the CTAs by a second kernel in
// CTA order; the counts are integers, so their atomics give the same result
// in any order.
#include <algorithm>

#include "training.cuh"

namespace gact {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxExperts = 1024;

// Softmax of one token's logits, held V per lane; a row with no finite
// maximum above -infinity gives 0 everywhere.
template <int V>
__device__ __forceinline__ void softmax_row(float (&p)[V]) {
    float top = p[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        top = fmaxf(top, p[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // fmaxf skips NaN; exp of a NaN logit stays NaN and reaches the sum
    const float shift = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        p[i] = __expf(p[i] - shift);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i)
        p[i] *= inv;
}

template <class T, int V>
__device__ __forceinline__ void load_row(float (&p)[V], const T *row, int E, int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? to_float(row[e]) : -INFINITY;
    }
}

// CTA b takes the tokens [b * per, (b + 1) * per).  part_p [G][E] fp32,
// part_c [G][E + 1] int32 (the last: live tokens).
template <class T, class I, int V>
__global__ void __launch_bounds__(kThreads)
balance_rows(float *__restrict__ part_p, int32_t *__restrict__ part_c,
             const T *__restrict__ logits, const I *__restrict__ ids,
             const uint8_t *__restrict__ live, int64_t tokens, int64_t per, int E, int64_t k,
             int64_t ls) {
    extern __shared__ float sums[];                              // [kWarps][E]
    int *hist = reinterpret_cast<int *>(sums + kWarps * E);      // [E + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e <= E; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = blockIdx.x * per, t1 = min(tokens, t0 + per);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.f;
    int mine = 0;
    for (int64_t t = t0 + warp; t < t1; t += kWarps) {
        if (live && !live[t])
            continue;
        ++mine;
        float p[V];
        load_row<T, V>(p, logits + t * ls, E, lane);
        softmax_row<V>(p);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] += p[i];
        for (int64_t j = lane; j < k; j += 32) {
            const int64_t e = static_cast<int64_t>(ids[t * k + j]);
            if (e >= 0 && e < E)
                atomicAdd(hist + e, 1);
        }
    }
    if (lane == 0)
        atomicAdd(hist + E, mine);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < E)
            sums[warp * E + lane + 32 * i] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        part_c[static_cast<int64_t>(blockIdx.x) * (E + 1) + e] = hist[e];
        if (e < E) {
            float s = 0.f;
            for (int w = 0; w < kWarps; ++w)
                s += sums[w * E + e];
            part_p[static_cast<int64_t>(blockIdx.x) * E + e] = s;
        }
    }
}

// Joins the G partial sums: one CTA, thread e the expert e.
__global__ void __launch_bounds__(kMaxExperts)
balance_join(float *__restrict__ loss, int32_t *__restrict__ counts, int32_t *__restrict__ tokens,
             float *__restrict__ mean_p, const float *__restrict__ part_p,
             const int32_t *__restrict__ part_c, int G, int E, float k, float coef) {
    __shared__ float red[32];
    __shared__ int live;
    pdl_wait();
    pdl_trigger();
    const int e = threadIdx.x, lane = e & 31;
    if (e == 0)
        live = 0;
    __syncthreads();
    int n = 0;
    for (int g = e; g < G; g += blockDim.x)
        n += part_c[static_cast<int64_t>(g) * (E + 1) + E];
    if (n)
        atomicAdd(&live, n);
    float p = 0.f;
    int c = 0;
    if (e < E)
        for (int g = 0; g < G; ++g) {
            p += part_p[static_cast<int64_t>(g) * E + e];
            c += part_c[static_cast<int64_t>(g) * (E + 1) + e];
        }
    __syncthreads();
    n = live;
    const float nf = static_cast<float>(n > 0 ? n : 1);
    p /= nf;
    if (e < E) {
        counts[e] = c;
        mean_p[e] = p;
    }
    float s = warp_sum(e < E ? static_cast<float>(c) / (nf * k) * p : 0.f);
    if (lane == 0)
        red[e >> 5] = s;
    __syncthreads();
    if (e < 32) {
        s = warp_sum(e < static_cast<int>(blockDim.x) / 32 ? red[e] : 0.f);
        if (e == 0) {
            loss[0] = coef * static_cast<float>(E) * s;
            tokens[0] = n;
        }
    }
}

// Counts enter as c_j - C/E, C their sum: the same gradient, since p sums to
// 1, without the cancellation of nearly equal counts.
template <class T, int V>
__global__ void __launch_bounds__(kThreads)
balance_backward(T *__restrict__ grad, const float *__restrict__ grad_loss,
                 const T *__restrict__ logits, const int32_t *__restrict__ counts,
                 const int32_t *__restrict__ tokens_live, const uint8_t *__restrict__ live,
                 int64_t tokens, int E, float k, int64_t ls, float coef) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    float c[V], total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        c[i] = e < E ? static_cast<float>(counts[e]) : 0.f;
        total += c[i];
    }
    const float mid = rintf(warp_sum(total) / static_cast<float>(E));
#pragma unroll
    for (int i = 0; i < V; ++i)
        c[i] -= mid;
    const int n = *tokens_live;
    const float nf = static_cast<float>(n > 0 ? n : 1);
    const float scale = *grad_loss * (coef * static_cast<float>(E) / (nf * nf * k));
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < tokens;
         t += step) {
        const bool on = !live || live[t];
        float p[V], mixed = 0.f;
        if (on) {
            load_row<T, V>(p, logits + t * ls, E, lane);
            softmax_row<V>(p);
#pragma unroll
            for (int i = 0; i < V; ++i)
                mixed = fmaf(p[i], c[i], mixed);
            mixed = warp_sum(mixed);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < E)
                grad[t * E + lane + 32 * i] =
                    from_float<T>(on ? scale * p[i] * (c[i] - mixed) : 0.f);
    }
}

int check_sizes(int64_t T, int64_t E, int64_t k, int64_t ls, int dtype) {
    if (T < 0 || E <= 0 || k <= 0)
        return GATED_ACT_ERR_SIZE;
    if (ls < E)
        return GATED_ACT_ERR_STRIDE;
    if (!elem_size(dtype))
        return GATED_ACT_ERR_DTYPE;
    if (E > kMaxExperts || T > 0x7FFFFFFF || k > 0x7FFFFFFF || T * k > 0x7FFFFFFF ||
        ls > (int64_t(1) << 30))
        return GATED_ACT_ERR_TOO_LARGE;
    return GATED_ACT_OK;
}

// Calls f(integral_constant<V>) with the smallest V in 1, 2, 4, .. for which
// 32 V >= E.
template <int V> struct Lanes {
    static constexpr int value = V;
};
template <class F> int with_lanes(int64_t E, F f) {
    return E <= 32    ? f(Lanes<1>{})
           : E <= 64  ? f(Lanes<2>{})
           : E <= 128 ? f(Lanes<4>{})
           : E <= 256 ? f(Lanes<8>{})
           : E <= 512 ? f(Lanes<16>{})
                      : f(Lanes<32>{});
}

int64_t parts(int64_t T) {
    return std::max<int64_t>(1, std::min<int64_t>(ceil_div64(T, kWarps * 4),
                                                  device_sm_count()));
}

}  // namespace
}  // namespace gact

extern "C" size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t E) {
    if (T < 0 || E <= 0 || E > gact::kMaxExperts)
        return 16;
    return static_cast<size_t>((gact::parts(T) * (2 * E + 1) * 4 + 15) / 16 * 16);
}

extern "C" int moe_balance_loss(float *loss, int32_t *counts, int32_t *tokens, float *mean_p,
                                const void *logits, const void *ids, const uint8_t *live,
                                int64_t T, int64_t E, int64_t k, int64_t logits_stride, int dtype,
                                int ids64, double coef, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, E, k, logits_stride, dtype);
    if (rc != GATED_ACT_OK)
        return rc;
    const size_t need = moe_balance_loss_workspace_bytes(T, E);
    if (workspace && workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    const int64_t size = elem_size(dtype), isize = ids64 ? 8 : 4;
    Region r[8] = {{loss, 4, 4, true},
                   {counts, static_cast<uint64_t>(E * 4), 4, true},
                   {tokens, 4, 4, true},
                   {mean_p, static_cast<uint64_t>(E * 4), 4, true},
                   {workspace, need, 16, true},
                   {logits, span_bytes(T, logits_stride, E, size), uintptr_t(size), false},
                   {ids, static_cast<uint64_t>(T * k * isize), uintptr_t(isize), false},
                   {live, live ? static_cast<uint64_t>(T) : 0, 1, false}};
    if ((rc = check_regions(r, 8)) != GATED_ACT_OK)
        return rc;
    const int64_t per = std::max<int64_t>(1, ceil_div64(T, parts(T)));
    const int64_t G = ceil_div64(T, per);
    float *part_p = as<float>(r[4]);
    int32_t *part_c = reinterpret_cast<int32_t *>(part_p + G * E);
    if (G > 0) {
        rc = with_type(dtype, [&](auto t) {
            return with_lanes(E, [&](auto lanes) {
                using Elem = decltype(t);
                constexpr int V = decltype(lanes)::value;
                const size_t smem = (kWarps * E + E + 1) * 4;
                const auto go = [&](auto id) {
                    using I = decltype(id);
                    return launched(launch_kernel(
                        balance_rows<Elem, I, V>, dim3(static_cast<unsigned>(G)), dim3(kThreads),
                        smem, stream, 1, part_p, part_c, as<const Elem>(r[5]), as<const I>(r[6]),
                        as<const uint8_t>(r[7]), T, per, static_cast<int>(E), k, logits_stride));
                };
                return ids64 ? go(int64_t{}) : go(int32_t{});
            });
        });
        if (rc != GATED_ACT_OK)
            return rc;
    }
    return launched(launch_kernel(
        balance_join, dim3(1), dim3(static_cast<unsigned>(ceil_div64(E, 32) * 32)), 0, stream, 1,
        as<float>(r[0]), as<int32_t>(r[1]), as<int32_t>(r[2]), as<float>(r[3]),
        static_cast<const float *>(part_p), static_cast<const int32_t *>(part_c),
        static_cast<int>(G), static_cast<int>(E), static_cast<float>(k),
        static_cast<float>(coef)));
}

extern "C" int moe_balance_loss_backward(void *grad_logits, const float *grad_loss,
                                         const void *logits, const int32_t *counts,
                                         const int32_t *tokens, const uint8_t *live, int64_t T,
                                         int64_t E, int64_t k, int64_t logits_stride, int dtype,
                                         double coef, cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, E, k, logits_stride, dtype);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    const int64_t size = elem_size(dtype);
    Region r[6] = {{grad_logits, static_cast<uint64_t>(T * E * size), uintptr_t(size), true},
                   {grad_loss, 4, 4, false},
                   {logits, span_bytes(T, logits_stride, E, size), uintptr_t(size), false},
                   {counts, static_cast<uint64_t>(E * 4), 4, false},
                   {tokens, 4, 4, false},
                   {live, live ? static_cast<uint64_t>(T) : 0, 1, false}};
    if ((rc = check_regions(r, 6)) != GATED_ACT_OK)
        return rc;
    const int64_t grid = std::min<int64_t>(ceil_div64(T, kWarps), int64_t(device_sm_count()) * 8);
    return with_type(dtype, [&](auto t) {
        return with_lanes(E, [&](auto lanes) {
            using Elem = decltype(t);
            constexpr int V = decltype(lanes)::value;
            return launched(launch_kernel(
                balance_backward<Elem, V>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                stream, 1, as<Elem>(r[0]), as<const float>(r[1]), as<const Elem>(r[2]),
                as<const int32_t>(r[3]), as<const int32_t>(r[4]), as<const uint8_t>(r[5]), T,
                static_cast<int>(E), static_cast<float>(k), logits_stride,
                static_cast<float>(coef)));
        });
    });
}
