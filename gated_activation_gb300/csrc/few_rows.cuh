// Gated projections of a few rows (up to 16): reading the weight is all the time there is.
//
// A warp holds the sums of 8 columns, gate and up, for every row: the tensor cores' 16 x 8 x 16
// product (mma.sync) takes 8 gate rows of the weight as its first eight rows and the same 8 up rows
// as its last, and 8 rows of the input as its columns, so that a thread ends with g and u of the same
// column and rows.  (The big tiles of tcgen05 would be empty in all but a few of their 256 rows and
// leave most SMs without a tile: 1 x 768 x 2048 takes 3 pairs.)  No weight passes through shared
// memory: since the order of a sum does not matter to it, each thread takes 8 consecutive elements
// of its row, one 16-byte load, as the operand's elements that the instruction wants from it.
//
// `split` warps of a block share the sum; they add up through shared memory, in a fixed order.
//
// Measured: 1 row of 2048 -> 768 in 4.5 us a call (5.3 us alone; the big tiles took 13.6), of which the 6 MB are
// 0.9 us and the rest launch, one chain of loads and the host.  It stands back where there are more rows or turned tiles
// (`few` in linear_act.cu has the figures): every warp reads the rows through L1 again, at 16 rows as many bytes as of
// its weight, and 16 rows of 4096 -> 16384 took 80 us here and 44 us there.
#pragma once

#include "product.cuh"

namespace gact {

constexpr int kFewRows = 16;
constexpr int kFewUnroll = 4;   // 16-byte loads of a row on their way per thread: 256 bytes a warp

template <class T> struct FewArgs {
    const T *in, *weight;
    T *out;
    const int32_t *live;
    int64_t in_stride, in_batch, weight_stride, weight_batch;
    int rows, k, d, split;
};

template <class T>
__device__ __forceinline__ void few_product(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, bf16>)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Up to eight elements of a row from p on; those past n (and all of a row that is not there) are 0.
template <bool VEC, class T> __device__ __forceinline__ uint4 few_load(const T *p, int n) {
    if (VEC && n >= 8)
        return ld_stream(p);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < n ? ld_stream_u16(reinterpret_cast<const uint16_t *>(p) + i) : 0;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}
// The same of the input, which the other warps of the SM read too: through L1.
template <bool VEC, class T> __device__ __forceinline__ uint4 few_load_in(const T *p, int n) {
    if (VEC && n >= 8)
        return *reinterpret_cast<const uint4 *>(p);
    return few_load<false>(p, n);
}

// NT: eights of rows.
template <class Act, class T, int NT, bool VEC>
__global__ void __launch_bounds__(256) few_rows(FewArgs<T> g) {
    __shared__ float4 share[8][NT][32];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y, live = g.live ? min(max(g.live[e], 0), g.rows) : g.rows;
    if (live == 0)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane >> 2, tig = lane & 3;
    const int part = warp % g.split, col = (blockIdx.x * (8 / g.split) + warp / g.split) * 8 + quad;
    const T *gate = g.weight + e * g.weight_batch + int64_t(col) * g.weight_stride,
            *up = gate + int64_t(g.d) * g.weight_stride;
    const T *in = g.in + e * g.in_batch + int64_t(quad) * g.in_stride;
    float sums[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[t][i] = 0.f;
    for (int k0 = part * (32 * kFewUnroll); k0 < g.k; k0 += g.split * (32 * kFewUnroll)) {
        uint4 a[kFewUnroll], b[kFewUnroll];
#pragma unroll
        for (int u = 0; u < kFewUnroll; ++u) {
            const int k = k0 + 32 * u + 8 * tig, n = col < g.d ? g.k - k : 0;
            a[u] = few_load<VEC>(gate + k, n);
            b[u] = few_load<VEC>(up + k, n);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= live)
                break;
#pragma unroll
            for (int u = 0; u < kFewUnroll; ++u) {
                const int k = k0 + 32 * u + 8 * tig;
                const uint4 x = few_load_in<VEC>(in + int64_t(8 * t) * g.in_stride + k,
                                                 8 * t + quad < live ? g.k - k : 0);
                few_product<T>(sums[t], a[u].x, b[u].x, a[u].y, b[u].y, x.x, x.y);
                few_product<T>(sums[t], a[u].z, b[u].z, a[u].w, b[u].w, x.z, x.w);
            }
        }
    }
    if (g.split > 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
            share[warp][t][lane] = make_float4(sums[t][0], sums[t][1], sums[t][2], sums[t][3]);
        __syncthreads();
        if (part)
            return;
        for (int i = 1; i < g.split; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float4 v = share[warp + i][t][lane];
                sums[t][0] += v.x;
                sums[t][1] += v.y;
                sums[t][2] += v.z;
                sums[t][3] += v.w;
            }
    }
    if (col >= g.d)
        return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float2 y = act_mul<Act>({sums[t][0], sums[t][1]}, {sums[t][2], sums[t][3]});
        const int row = 8 * t + 2 * tig;
        T *to = g.out + (int64_t(e) * g.rows + row) * g.d + col;
        if (row < live)
            to[0] = from_float<T>(y.x);
        if (row + 1 < live)
            to[g.d] = from_float<T>(y.y);
    }
}

template <class Act, class T>
int launch_few_rows(const FewArgs<T> &args, int64_t E, bool vec, cudaStream_t stream) {
    FewArgs<T> g = args;
    // Warps that share a sum: enough that every SM has 32 warps (eight SM-wide loads of 8 KB each on
    // their way), no more than the sum has turns.
    const int64_t groups = ceil_div64(g.d, 8), want = int64_t(32) * device_sm_count();
    g.split = 1;
    while (g.split < 8 && groups * E * g.split < want && g.split * 32 * kFewUnroll < g.k)
        g.split *= 2;
    const dim3 grid(static_cast<unsigned>(ceil_div64(groups, 8 / g.split)), static_cast<unsigned>(E));
    const auto go = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        auto kernel = vec ? few_rows<Act, T, NT, true> : few_rows<Act, T, NT, false>;
        return cuda_status(launch_kernel(kernel, grid, dim3(256), 0, stream, 1, g));
    };
    return g.rows <= 8 ? go(Const<1>{}) : go(Const<2>{});
}

}  // namespace gact
