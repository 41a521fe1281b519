// Layer norm, forward and backward (definitions in gated_act_training.h).
//
// HBM bandwidth bounds both: the forward pass reads and writes each row once,
// the backward pass reads two and writes one.  The parameters' gradients are
// sums over the rows: each CTA adds up its own rows' share of every column,
// and a second kernel adds the CTAs' shares in a fixed order, so results do
// not depend on how the blocks were scheduled.
#include <algorithm>

#include "training.cuh"

namespace gact {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// Any layout: one CTA per row, the row read again (from L1/L2) for each pass.
template <class T, class W>
__global__ void __launch_bounds__(kThreads)
ln_forward_any(T *__restrict__ out, float *__restrict__ mean_out, float *__restrict__ rstd_out,
               const T *__restrict__ in, const W *__restrict__ weight, const W *__restrict__ bias,
               int64_t rows, int64_t d, int64_t rs, float eps) {
    __shared__ float red[2][kWarps];
    pdl_wait();
    pdl_trigger();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *x = in + r * rs;
        float acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads)
            acc += to_float(x[c]);
        const float mean = cta_sum(acc, red[0]) / static_cast<float>(d);
        acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float e = to_float(x[c]) - mean;
            acc = fmaf(e, e, acc);
        }
        const float var = cta_sum(acc, red[1]) / static_cast<float>(d);
        const float rstd = 1.0f / __fsqrt_rn(var + eps);
        if (threadIdx.x == 0) {
            mean_out[r] = mean;
            rstd_out[r] = rstd;
        }
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float h = (to_float(x[c]) - mean) * rstd;
            const float w = to_float(weight[c]);
            out[r * d + c] = from_float<T>(bias ? fmaf(h, w, to_float(bias[c])) : h * w);
        }
    }
}

template <class T, class W>
__global__ void __launch_bounds__(kThreads)
ln_backward_rows_any(T *__restrict__ grad_in, const T *__restrict__ grad, const T *__restrict__ in,
                     const W *__restrict__ weight, const float *__restrict__ mean_in,
                     const float *__restrict__ rstd_in, int64_t rows, int64_t d, int64_t rs,
                     int64_t gs) {
    __shared__ float red[2][2][kWarps];
    pdl_wait();
    pdl_trigger();
    int k = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, k ^= 1) {
        const T *x = in + r * rs, *dy = grad + r * gs;
        const float mean = mean_in[r], rstd = rstd_in[r];
        float a = 0.f, b = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = to_float(dy[c]) * to_float(weight[c]);
            a += g;
            b = fmaf(g, (to_float(x[c]) - mean) * rstd, b);
        }
        const float ma = cta_sum(a, red[k][0]) / static_cast<float>(d);
        const float mb = cta_sum(b, red[k][1]) / static_cast<float>(d);
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = to_float(dy[c]) * to_float(weight[c]);
            const float h = (to_float(x[c]) - mean) * rstd;
            grad_in[r * d + c] = from_float<T>(rstd * (g - ma - h * mb));
        }
    }
}

// Columns' shares of the rows [y * per, (y + 1) * per), y = blockIdx.y: one
// column per thread.  part: [2][gridDim.y][d].
template <class T>
__global__ void __launch_bounds__(kThreads)
ln_backward_columns_any(float *__restrict__ part, const T *__restrict__ grad,
                        const T *__restrict__ in, const float *__restrict__ mean_in,
                        const float *__restrict__ rstd_in, int64_t rows, int64_t per, int64_t d,
                        int64_t rs, int64_t gs) {
    pdl_wait();
    pdl_trigger();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    if (c >= d)
        return;
    float w = 0.f, b = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = to_float(grad[r * gs + c]);
        w = fmaf(dy, (to_float(in[r * rs + c]) - mean_in[r]) * rstd_in[r], w);
        b += dy;
    }
    part[blockIdx.y * d + c] = w;
    part[(gridDim.y + blockIdx.y) * d + c] = b;
}

// Adds the n shares of every column: thread x a column, the kReduceY threads y
// of a column every kReduceY-th share.
constexpr int kReduceX = 32, kReduceY = 8;
__global__ void __launch_bounds__(kReduceX *kReduceY)
ln_backward_reduce(float *__restrict__ grad_weight, float *__restrict__ grad_bias,
                   const float *__restrict__ part, int64_t n, int64_t d) {
    __shared__ float sum[2][kReduceY][kReduceX];
    pdl_wait();
    pdl_trigger();
    const int x = threadIdx.x % kReduceX, y = threadIdx.x / kReduceX;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kReduceX + x;
    float w = 0.f, b = 0.f;
    if (c < d)
        for (int64_t i = y; i < n; i += kReduceY) {
            w += part[i * d + c];
            if (grad_bias)
                b += part[(n + i) * d + c];
        }
    sum[0][y][x] = w;
    sum[1][y][x] = b;
    __syncthreads();
    if (y == 0 && c < d) {
        for (int i = 1; i < kReduceY; ++i) {
            w += sum[0][i][x];
            b += sum[1][i][x];
        }
        grad_weight[c] = w;
        if (grad_bias)
            grad_bias[c] = b;
    }
}

constexpr int64_t kMaxWidth = int64_t(1) << 30, kMaxRows = int64_t(1) << 40;

int check_sizes(int64_t T, int64_t d, int64_t rs, int64_t gs, int dtype, int param_dtype) {
    if (T < 0 || d <= 0)
        return GATED_ACT_ERR_SIZE;
    if (rs < d || gs < d)
        return GATED_ACT_ERR_STRIDE;
    if (!elem_size(dtype) || (param_dtype != dtype && param_dtype != GATED_ACT_F32))
        return GATED_ACT_ERR_DTYPE;
    const int64_t widest = std::max(rs, gs);
    if (d > kMaxWidth || T > kMaxRows || widest > kMaxRows ||
        (T > 0 && widest > (int64_t(1) << 60) / T))
        return GATED_ACT_ERR_TOO_LARGE;
    return GATED_ACT_OK;
}

// Calls f(T{}, W{}) with the element types of the rows and the parameters.
template <class F> int with_types(int dtype, int param_dtype, F f) {
    return with_type(dtype, [&](auto t) {
        return param_dtype == dtype ? f(t, t) : f(t, float{});
    });
}

// Rows whose shares are added up apart before the second kernel joins them.
int64_t shares(int64_t T, int64_t d) {
    (void)d;
    return std::min<int64_t>(T, int64_t(device_sm_count()) * 2);
}

}  // namespace
}  // namespace gact

extern "C" int layer_norm(void *out, float *mean, float *rstd, const void *in, const void *weight,
                          const void *bias, int64_t T, int64_t d, int64_t row_stride, double eps,
                          int dtype, int param_dtype, cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, d, row_stride, d, dtype, param_dtype);
    if (rc == GATED_ACT_OK && !(eps >= 0.0))
        rc = GATED_ACT_ERR_SIZE;
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    const int64_t size = elem_size(dtype), wsize = elem_size(param_dtype);
    Region r[6] = {{out, static_cast<uint64_t>(T * d * size), uintptr_t(size), true},
                   {mean, static_cast<uint64_t>(T * 4), 4, true},
                   {rstd, static_cast<uint64_t>(T * 4), 4, true},
                   {in, span_bytes(T, row_stride, d, size), uintptr_t(size), false},
                   {weight, static_cast<uint64_t>(d * wsize), uintptr_t(wsize), false},
                   {bias, bias ? static_cast<uint64_t>(d * wsize) : 0, uintptr_t(wsize), false}};
    if ((rc = check_regions(r, 6)) != GATED_ACT_OK)
        return rc;
    const int64_t grid = std::min<int64_t>(T, int64_t(device_sm_count()) * 64);
    return with_types(dtype, param_dtype, [&](auto t, auto w) {
        using E = decltype(t);
        using W = decltype(w);
        return launched(launch_kernel(ln_forward_any<E, W>, dim3(static_cast<unsigned>(grid)),
                                      dim3(kThreads), 0, stream, 1, as<E>(r[0]), as<float>(r[1]),
                                      as<float>(r[2]), as<const E>(r[3]), as<const W>(r[4]),
                                      as<const W>(r[5]), T, d, row_stride,
                                      static_cast<float>(eps)));
    });
}

extern "C" size_t layer_norm_backward_workspace_bytes(int64_t T, int64_t d) {
    if (T <= 0 || d <= 0 || d > gact::kMaxWidth)
        return 16;
    return static_cast<size_t>(std::max<int64_t>(16, gact::shares(T, d) * d * 8));
}

extern "C" int layer_norm_backward(void *grad_in, float *grad_weight, float *grad_bias,
                                   const void *grad_out, const void *in, const void *weight,
                                   const float *mean, const float *rstd, int64_t T, int64_t d,
                                   int64_t row_stride, int64_t grad_stride, int dtype,
                                   int param_dtype, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
    using namespace gact;
    int rc = check_sizes(T, d, row_stride, grad_stride, dtype, param_dtype);
    if (rc != GATED_ACT_OK)
        return rc;
    const size_t need = layer_norm_backward_workspace_bytes(T, d);
    if (T > 0 && workspace && workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    const int64_t size = elem_size(dtype), wsize = elem_size(param_dtype);
    Region r[9] = {{grad_in, static_cast<uint64_t>(T * d * size), uintptr_t(size), true},
                   {grad_weight, static_cast<uint64_t>(d * 4), 4, true},
                   {grad_bias, grad_bias ? static_cast<uint64_t>(d * 4) : 0, 4, true},
                   {workspace, T > 0 ? need : 0, 16, true},
                   {grad_out, span_bytes(T, grad_stride, d, size), uintptr_t(size), false},
                   {in, span_bytes(T, row_stride, d, size), uintptr_t(size), false},
                   {weight, T > 0 ? static_cast<uint64_t>(d * wsize) : 0, uintptr_t(wsize), false},
                   {mean, static_cast<uint64_t>(T * 4), 4, false},
                   {rstd, static_cast<uint64_t>(T * 4), 4, false}};
    if ((rc = check_regions(r, 9)) != GATED_ACT_OK)
        return rc;
    float *part = as<float>(r[3]);
    int64_t n = 0;
    if (T > 0) {
        const int64_t per = ceil_div64(T, shares(T, d));
        n = ceil_div64(T, per);
        const int64_t grid = std::min<int64_t>(T, int64_t(device_sm_count()) * 64);
        rc = with_types(dtype, param_dtype, [&](auto t, auto w) {
            using E = decltype(t);
            using W = decltype(w);
            return launched(launch_kernel(
                ln_backward_rows_any<E, W>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                stream, 1, as<E>(r[0]), as<const E>(r[4]), as<const E>(r[5]), as<const W>(r[6]),
                as<const float>(r[7]), as<const float>(r[8]), T, d, row_stride, grad_stride));
        });
        if (rc != GATED_ACT_OK)
            return rc;
        rc = with_type(dtype, [&](auto t) {
            using E = decltype(t);
            return launched(launch_kernel(
                ln_backward_columns_any<E>,
                dim3(static_cast<unsigned>(ceil_div64(d, kThreads)), static_cast<unsigned>(n)),
                dim3(kThreads), 0, stream, 1, part, as<const E>(r[4]), as<const E>(r[5]),
                as<const float>(r[7]), as<const float>(r[8]), T, per, d, row_stride, grad_stride));
        });
        if (rc != GATED_ACT_OK)
            return rc;
    }
    return launched(launch_kernel(ln_backward_reduce,
                                  dim3(static_cast<unsigned>(ceil_div64(d, kReduceX))),
                                  dim3(kReduceX * kReduceY), 0, stream, 1, as<float>(r[1]),
                                  as<float>(r[2]), static_cast<const float *>(part), n, d));
}
