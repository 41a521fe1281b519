// Gated projections: both products of a gated MLP's up half with the activation as
// their epilogue, and their backward pass.
//
//   forward   (g, u) = in (Wg, Wu)',  out = act(g) u: one product kernel.  A pair's tile
//             holds 128 columns of g and the same 128 of u, so that a thread has both.
//   backward  dg = grad_out u act'(g), du = grad_out act(g) from the kept g and u (one pass
//             over memory; in fp16 under a power of two, from a pass before), then grad_in = (dg, du) W and grad_weight = (dg, du)' in.
#include <cfloat>

#include "few_rows.cuh"

#include "gated_act_linear.h"

namespace gact {
namespace {

constexpr int kBlock = 32;   // elements under one scale

// ------------------------------------------------------- 16-bit checkpoints

// The scale byte of a block whose largest magnitude is `top`: 2^(e - 127) is the smallest
// power of two of which `top` is at most 32767 multiples, after rounding.  Adding 2^8 to
// the bits carries a mantissa of 2 - 2^-15 or more, which would round to 2^15 multiples,
// into the exponent.
__device__ __forceinline__ uint32_t scale_of(float top) {
    const uint32_t e = (__float_as_uint(top) + 0x100u) >> 23;   // 255: infinity or NaN
    return e >= 255 ? 255u : e <= 15 ? 1u : e - 14;
}
__device__ __forceinline__ float inverse_scale(uint32_t e) {
    return e == 255 ? 0.f : __uint_as_float((254u - e) << 23);
}

// Two codes of a word.  2^23 + 2^15 + q has q + 2^15 in its last mantissa bits, so that no
// conversion is needed (those run at a quarter of the exponentials' already small rate, in the same unit).
__device__ __forceinline__ float2 decode2(uint32_t w) {
    const uint32_t u = w ^ 0x80008000u;
    return sub2({__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7610)),
                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7632))},
                both(8388608.f + 32768.f));
}

// The codes of 32 values, two to a word; returns the scale byte.
__device__ __forceinline__ uint32_t encode32(uint32_t (&w)[16], const float (&v)[32]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        top = max_abs(top, make_float2(v[i], v[i + 1]));
    const uint32_t e = scale_of(top);
    const float inverse = inverse_scale(e);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        // 1.5 2^23 + x is rounded to whole numbers, ties to even, and x's 16 bits are its last ones:
        // no conversion, as in decode2
        const float2 x = fma2({v[2 * i], v[2 * i + 1]}, both(inverse), both(12582912.f));
        w[i] = e == 255 ? 0u : __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x5410);
    }
    return e;
}

// ------------------------------------------------------------------- products

// The forward product.  4 T k d operations; bound by the tensor cores where k is long (2048 x 4096 -> 16384:
// 285 us alone, cuBLAS's rate and more), by the epilogue where it is short: per element one exponential, one
// reciprocal and, for the checkpoint, a maximum, a product and three rounds through shared memory, 4 to
// 5 us for a tile of 128 x 128 per CTA (8 warps), against 5 ns per summed element in the main loop.
template <class Act, class T, int N, bool KEEP> struct Forward {
    using Elem = T;
    static constexpr bool kBAcross = false, kSecond = false;
    static constexpr int kN = N, kRows = kTile;
    static constexpr int kClosed = 0;
    static constexpr Live kLive = Live::Rows;
    struct Args {
        T *out;
        int16_t *codes;
        uint8_t *scales;
        int d;
        bool vec;
    };
    using G = Product<Forward>;
    __device__ static int batch_of(const G &, int b, bool) { return b; }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        load_along(a, &g.a, bar, step * kStep, t.m0 + static_cast<int>(rank) * kHalf, 0, t.b);
        // the first CTA brings the gate's rows of the weight, the second the up half's
        load_along(b, &g.b, bar, step * kStep, t.n0 * (N / 2), static_cast<int>(rank), t.b);
    }
    __device__ static int steps_of(const G &g, const Tile &) { return g.steps; }
    __device__ static void finish(const G &g, const Tile &t, int row, uint32_t sums, const Stage &stage) {
        const int d = g.j.d, r = t.m0 + row, blocks = (d + kBlock - 1) / kBlock;
        const bool mine = r < t.rows;
        const int lane = threadIdx.x & 31, rows = t.rows - (r - lane);   // of the warp
        const int64_t at = int64_t(t.b) * g.capacity + r, top = at - lane;
        for (int c = 32 * stage.part; c < N / 2 && t.n0 * (N / 2) + c < d; c += 64) {
            const int col = t.n0 * (N / 2) + c, n = d - col;
            float gate[32], up[32];
            sums_load32(sums + c, gate);
            sums_load32(sums + N / 2 + c, up);
            sums_ready(gate);
            sums_ready(up);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = pack2<T>(act_mul<Act>({gate[2 * i], gate[2 * i + 1]}, {up[2 * i], up[2 * i + 1]}));
            stage.flush(w, g.j.out + top * d + col, d, rows, n, g.j.vec);
            if (KEEP) {
                uint8_t *scale = g.j.scales + at * 2 * blocks + col / kBlock;
                int16_t *codes = g.j.codes + top * 2 * d + col;
                uint32_t e = encode32(w, gate);
                if (mine)
                    scale[0] = static_cast<uint8_t>(e);
                stage.flush(w, codes, 2 * int64_t(d), rows, n, g.j.vec);
                e = encode32(w, up);
                if (mine)
                    scale[blocks] = static_cast<uint8_t>(e);
                stage.flush(w, codes + d, 2 * int64_t(d), rows, n, g.j.vec);
            }
        }
    }
};

// The same product with the roles turned round, for up to N rows that would leave most of a
// 256-row tile empty: the weight's rows are the tile's (64 of g and the same 64 of u per CTA), the
// input's its columns.  Of four epilogue warps two hold g and two the u of the same columns, which
// they hand over through shared memory.  Bound by reading the weight: 16 rows of 4096 -> 16384 43.5 us (268 MB, 91%
// of the copy rate; upright 51 us), 128 experts of 2048 -> 768 with 0 to 4 rows 104 us (the copy rate;
// upright 117 us).
template <class Act, class T, int N> struct Swapped {
    using Elem = T;
    static constexpr bool kBAcross = false, kSecond = false;
    static constexpr int kN = N, kRows = kHalf;
    static constexpr int kClosed = 0;
    static constexpr Live kLive = Live::Columns;
    struct Args {
        T *out;
    };
    using G = Product<Swapped>;
    __device__ static int batch_of(const G &, int b, bool) { return b; }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static int steps_of(const G &g, const Tile &) { return g.steps; }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        const int col = t.m0 + static_cast<int>(rank) * 64;
        load_along(a, &g.a, bar, step * kStep, col, 0, t.b);
        load_along(a + kRowBytes / 2, &g.a, bar, step * kStep, col, 1, t.b);
        load_along(b, &g.b, bar, step * kStep, static_cast<int>(rank) * (N / 2), 0, t.b);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, uint32_t sums, const Stage &stage) {
        // [32 rows, 64 columns] of each part
        float *held = reinterpret_cast<float *>(stage.s.stage[4 * stage.part]);
        const uint32_t full = smem_address(&stage.s.swap_full[stage.part]),
                       empty = smem_address(&stage.s.swap_empty[stage.part]);
        const int lane = threadIdx.x & 31, at = row & 63;
        const bool up = row & 64;
        const int col = t.m0 + (row >> 7) * 64 + at, d = g.rows;
        T *out = g.j.out + int64_t(t.b) * g.capacity * d + col;
        for (int c = 32 * stage.part; c < N && c < t.live; c += 64) {
            const uint32_t use = stage.uses++;
            float v[32];
            sums_load32(sums + c, v);
            sums_ready(v);
            if (up) {
                if (!barrier_wait(empty, (use & 1) ^ 1, &stage.s.gave_up))
                    return;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    held[i * 64 + at] = v[i];
                __syncwarp();
                if (lane == 0)
                    barrier_arrive(full);
                continue;
            }
            if (!barrier_wait(full, use & 1, &stage.s.gave_up))
                return;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 y = act_mul<Act>({v[i], v[i + 1]}, {held[i * 64 + at], held[i * 64 + 64 + at]});
                if (col < d && c + i < t.live)
                    out[int64_t(c + i) * d] = from_float<T>(y.x);
                if (col < d && c + i + 1 < t.live)
                    out[int64_t(c + i + 1) * d] = from_float<T>(y.y);
            }
            __syncwarp();
            if (lane == 0)
                barrier_arrive(empty);
        }
    }
};

// grad_in: A = (dg, du) along the sum over 2d, B = the weight across it.
// Second, grad_weight: A = (dg, du) across the sum over the rows, B = in across it; batch 2e + half.
// Past the live rows dg and du are zeros up to a whole step; the last rows of `in` come from
// a copy with zeros there, as what lies past the live rows may be anything.
// SPLIT: the first product's sums are divided into shares, fp32 tiles as the threads hold them (256 x 256,
// column after column), which join_shares adds up.
// 8 T k d operations in one launch: 4096 rows of 4096 -> 8192 in 566 us alone (1.94 PFLOP/s; two launches 620),
// 32 experts of 2048 -> 768, 70% of 1024 rows, 167 us (1.73 PFLOP/s of the live rows).
template <class T, int N, bool SPLIT> struct Gradients {
    using Elem = T;
    static constexpr bool kBAcross = true, kSecond = true;
    static constexpr int kN = N, kRows = kTile;
    static constexpr int kClosed = 0;
    static constexpr Live kLive = Live::Rows;
    struct Args {
        CUtensorMap rows, in, tail;   // of the second product
        T *grad_in, *grad_weight;
        float *sums;                  // SPLIT: [E, shares, tile rows, tile columns, 256, 256]
        const float *power;           // fp16: [E] what dg and du were divided by
        int k, half_steps, shares;    // ring steps of one half of the first sum
        bool vec_in, vec_weight;
    };
    using G = Product<Gradients>;
    __device__ static int batch_of(const G &g, int b, bool second) {
        return second ? b >> 1 : SPLIT ? b / g.j.shares : b;
    }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static int second_steps(const G &, int live) { return (live + kStep - 1) / kStep; }
    // shares of whole steps, as even as they get
    __device__ static int first_step(const G &g, int b) {
        return SPLIT ? static_cast<int>(int64_t(g.steps) * (b % g.j.shares) / g.j.shares) : 0;
    }
    __device__ static int steps_of(const G &g, const Tile &t) {
        return SPLIT ? (t.b % g.j.shares == g.j.shares - 1 ? g.steps : first_step(g, t.b + 1)) - first_step(g, t.b)
                     : g.steps;
    }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        const int row = t.m0 + static_cast<int>(rank) * kHalf, col = t.n0 * N + static_cast<int>(rank) * (N / 2);
        if (!t.second) {
            const int at = first_step(g, t.b) + step, e = batch_of(g, t.b, false);
            const int half = at >= g.j.half_steps, x = (at - half * g.j.half_steps) * kStep;
            load_along(a, &g.a, bar, x, row, half, e);
            load_across<N / 2>(b, &g.b, bar, x, col, half, e);
            return;
        }
        const int x = step * kStep, e = t.b >> 1;
        load_across(a, &g.j.rows, bar, x, row, t.b & 1, e);
        const bool tail = x + kStep > t.live && t.live < g.capacity;
        load_across<N / 2>(b, tail ? &g.j.tail : &g.j.in, bar, tail ? 0 : x, col, 0, e);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, uint32_t sums, const Stage &stage) {
        const int k = g.j.k, top = t.m0 + (row & ~31), col = t.n0 * N;   // the warp's first row
        if (SPLIT && !t.second) {
            const int64_t tall = (g.capacity + kTile - 1) / kTile;
            const int64_t tile = (t.b * tall + t.m0 / kTile) * g.n_tiles + t.n0;
            float *held = g.j.sums + tile * (kTile * kTile) + 32 * stage.part * kTile + row;
            for (int c = 32 * stage.part; c < kTile && col + c < k; c += 64, held += 64 * kTile) {
                float v[32];
                sums_load32(sums + c, v);
                sums_ready(v);
                if (t.m0 + row < t.rows)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        held[i * kTile] = v[i];
            }
            return;
        }
        T *to = t.second ? g.j.grad_weight + (int64_t(t.b) * g.second.rows + top) * k + col
                         : g.j.grad_in + (int64_t(t.b) * g.capacity + top) * k + col;
        const float power = std::is_same_v<T, f16> ? g.j.power[t.second ? t.b >> 1 : t.b] : 1.f;
        store_tile<N>(sums, stage, to, k, t.rows - top, k - col, t.second ? g.j.vec_weight : g.j.vec_in,
                      power, t.steps == 0);
    }
};

template <class T> struct ShareArgs {
    const float *sums, *power;   // power: fp16
    T *out;
    const int32_t *live;
    int capacity, k, shares;
};

// grad_in's rows from the shares of their sums: a block takes 32 rows x 64 columns of a tile, reads columns
// (32 loads on their way per thread) and writes rows.
template <class T> __global__ void __launch_bounds__(256) join_shares(ShareArgs<T> g) {
    __shared__ float held[64][33];
    pdl_wait();
    pdl_trigger();
    const int wide = (g.k + 63) / 64, high = (g.capacity + 31) / 32;
    const int e = static_cast<int>(blockIdx.x / (wide * high)), at = static_cast<int>(blockIdx.x % (wide * high));
    const int r0 = at / wide * 32, c0 = at % wide * 64;
    const int live = g.live ? min(max(g.live[e], 0), g.capacity) : g.capacity;
    if (r0 >= live)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tall = (g.capacity + kTile - 1) / kTile, tiles = tall * ((g.k + kTile - 1) / kTile);
    const int64_t part = int64_t(tiles) * (kTile * kTile);
    const float *from = g.sums + e * g.shares * part +
                        (int64_t(r0 / kTile) * ((g.k + kTile - 1) / kTile) + c0 / kTile) * (kTile * kTile) +
                        (c0 % kTile) * kTile + r0 % kTile + lane;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < g.shares; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = warp + 8 * i;
            if (r0 + lane < live && c0 + c < g.k)
                v[i] += from[s * part + c * kTile];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        held[warp + 8 * i][lane] = v[i];
    __syncthreads();
    const float power = std::is_same_v<T, f16> ? g.power[e] : 1.f;
    for (int i = warp; i < 32 && r0 + i < live; i += 8) {
        T *to = g.out + (int64_t(e) * g.capacity + r0 + i) * g.k + c0;
        for (int c = lane; c < 64 && c0 + c < g.k; c += 32)
            to[c] = from_float<T>(held[c][i] * power);
    }
}

// ------------------------------------------------- the gradients of g and u

template <class T> struct GateGradArgs {
    const T *grad;
    const int16_t *codes;
    const uint8_t *scales;
    const T *in;          // with live counts: its last, partly live, step of rows goes to `tail`
    T *rows;              // [E, 2, padded, dp]
    T *tail;              // [E, 64, kp]
    const int32_t *live;
    float *tops, *power;  // fp16: [E, n_tops] the blocks' shares of gradient_tops, [E] what dg and du are divided by
    int64_t grad_stride, grad_batch, in_stride, in_batch;
    int T_, d, dp, k, kp, padded, n_tops, top_pieces;
};

// fp16's range is too short for dg and du as they come: they lost bits below 2^-14 and were infinite past 65504, where
// the gradients, sums of products with them, need do neither.  So they are divided by a power of two per expert that puts
// the largest just below 2^15.  A bound is enough for it: |act(g)| <= |g| and |act'(g)| < 1.13, and the scales bound g and
// u by 2^15 steps.  (They are 2^14 at least in a block's largest element, so that the bound is a few times the
// largest product; fp16's normal numbers reach 2^-29 of it.)  One pass over grad_out alone, whose rows are read as the
// aligned vectors that hold them, four of a lane on their way; the columns of one may lie in two blocks (1001 x 2731
// 5.3 us, element by element 12; 4096 x 8192 22 us, of which the bytes are 10).
constexpr int kTops = 1024, kTopVectors = 4 * 32;   // blocks of an expert; vectors of a warp's piece of a row
__global__ void __launch_bounds__(256) gradient_tops(GateGradArgs<f16> g) {
    __shared__ float red[8];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = (g.d + kBlock - 1) / kBlock;
    const int e = blockIdx.y, live = g.live ? min(max(g.live[e], 0), g.T_) : g.T_;
    const int pieces = g.top_pieces;
    const int64_t items = int64_t(live) * pieces;
    float top = 0.f;
    for (int64_t item = blockIdx.x * 8 + warp; item < items; item += gridDim.x * 8) {
        const int i = static_cast<int>(item / pieces), piece = static_cast<int>(item - int64_t(i) * pieces);
        const f16 *grad = g.grad + e * g.grad_batch + i * g.grad_stride;
        const int before = before_row(grad);
        const uint8_t *scale = g.scales + (int64_t(e) * g.T_ + i) * 2 * blocks;
        uint4 v[4];
        float step[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (piece * kTopVectors + 32 * j + lane) * 8 - before;   // of the vector's first element
            v[j] = eight_around(grad, c, g.d);
            step[j] = 0.f;
            if (c >= g.d || c + 8 <= 0)
                continue;
            const int first = max(c, 0), last = min(c + 8, g.d) - 1;
#pragma unroll
            for (int q = 0; q < 2; ++q) {   // a NaN's block is NaN whatever it is divided by
                const int b = (q ? last : first) / kBlock;
                const uint32_t sg = scale[b], su = scale[blocks + b];
                step[j] = fmaxf(step[j], fmaxf(sg == 255 ? 0.f : __uint_as_float(sg << 23),
                                               su == 255 ? 0.f : 1.13f * __uint_as_float(su << 23)));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)   // infinities and NaN stay what they are
            top = fmaxf(top, fminf(top_of_eight(v[j]) * step[j] * 32768.f, FLT_MAX));
    }
    const int bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(top));   // top >= 0
    if (lane == 0)
        red[warp] = __int_as_float(bits);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, red[i]);
        g.tops[e * g.n_tops + blockIdx.x] = top;
    }
}
// The power of two of an expert, for all threads of a block of 8 warps.
__device__ __forceinline__ float gradient_power(const GateGradArgs<f16> &g, int e) {
    __shared__ int red[8];
    const int thread = threadIdx.y * 32 + threadIdx.x;
    int top = 0;
#pragma unroll
    for (int i = 0; i < kTops / 256; ++i)
        if (thread + 256 * i < g.n_tops)
            top = max(top, __float_as_int(g.tops[e * g.n_tops + thread + 256 * i]));
    const int warps = __reduce_max_sync(0xFFFFFFFFu, top);
    if (threadIdx.x == 0)
        red[threadIdx.y] = warps;
    __syncthreads();
    const int most = __reduce_max_sync(0xFFFFFFFFu, red[threadIdx.x & 7]);
    const float power = most ? __int_as_float(max((most >> 23) + 1 - 15, 1) << 23) : 1.f;
    if (blockIdx.x == 0 && blockIdx.y == 0 && thread == 0)
        g.power[e] = power;
    return power;
}

// Eight columns of a row: what the gradients there are computed from.
template <class T> struct GateGradIn {
    uint4 dy, gate, up;
    float sg, su;
};

constexpr int kGradRows = 2;   // rows of a thread: six 16-byte loads on their way

// (dg, du) of eight columns of two rows per thread, zeros from the live rows to a whole step.
// One pass: 6 bytes and the scales in, 4 out per pair of elements; 4096 x 8192 in 53.5 us, 93% of the copy
// rate (four rows a thread in 128 registers: 71 us; two in 64, twice the warps).
template <class Act, class T, bool VEC>
__global__ void __launch_bounds__(256, 4) gate_gradients(GateGradArgs<T> g) {
    pdl_wait();
    pdl_trigger();
    const int x = (blockIdx.x * 32 + threadIdx.x) * 8;
    const int blocks = (g.d + kBlock - 1) / kBlock;
    const int e = blockIdx.z, live = g.live ? min(max(g.live[e], 0), g.T_) : g.T_;
    const int end = (live + kStep - 1) / kStep * kStep;
    float inverse = 1.f;   // exact
    if constexpr (std::is_same_v<T, f16>)
        inverse = 1.f / gradient_power(g, e);
    // the partly live step of `in`, eight elements at a time over all of the expert's threads (32 experts of 717 x
    // 768 with k = 2048: 26 us; with an element at a time in the blocks of its rows 36.5)
    if (g.live && live % kStep) {
        const int first = live / kStep * kStep, eights = g.kp / 8;
        for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.y * 32 + threadIdx.x; i < kStep * eights;
             i += gridDim.x * gridDim.y * 256) {
            const int row = i / eights, c = (i - row * eights) * 8;
            const T *from = g.in + e * g.in_batch + int64_t(first + row) * g.in_stride + c;
            const bool vec = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
            st_vec_out(g.tail + (int64_t(e) * kStep + row) * g.kp + c,
                       first + row < live ? eight(from, g.k - c, vec) : make_uint4(0, 0, 0, 0));
        }
    }
    for (int i0 = (blockIdx.y * kGradRows) * 8 + threadIdx.y; i0 < end && x < g.dp;
         i0 += gridDim.y * kGradRows * 8) {
        GateGradIn<T> in[kGradRows];
#pragma unroll
        for (int j = 0; j < kGradRows; ++j) {
            const int i = i0 + 8 * j;
            in[j].dy = in[j].gate = in[j].up = make_uint4(0, 0, 0, 0);
            in[j].sg = in[j].su = 0.f;
            if (i >= live)
                continue;
            const int64_t at = int64_t(e) * g.T_ + i;
            const T *grad = g.grad + e * g.grad_batch + i * g.grad_stride + x;
            const int16_t *gate = g.codes + at * 2 * g.d + x, *up = gate + g.d;
            const uint8_t *scale = g.scales + at * 2 * blocks + x / kBlock;
            if (VEC) {
                in[j].dy = ld_stream(grad);
                in[j].gate = ld_stream(gate);
                in[j].up = ld_stream(up);
            } else {
                uint32_t v[3][8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const bool here = x + c < g.d;
                    v[0][c] = here ? ld_stream_u16(reinterpret_cast<const uint16_t *>(grad) + c) : 0;
                    v[1][c] = here ? ld_stream_u16(reinterpret_cast<const uint16_t *>(gate) + c) : 0;
                    v[2][c] = here ? ld_stream_u16(reinterpret_cast<const uint16_t *>(up) + c) : 0;
                }
                const auto join = [](const uint32_t (&u)[8]) {
                    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16,
                                      u[6] | u[7] << 16);
                };
                in[j].dy = join(v[0]);
                in[j].gate = join(v[1]);
                in[j].up = join(v[2]);
            }
            in[j].sg = __uint_as_float(uint32_t(scale[0]) << 23);
            in[j].su = __uint_as_float(uint32_t(scale[blocks]) << 23);
        }
#pragma unroll
        for (int j = 0; j < kGradRows; ++j) {
            const int i = i0 + 8 * j;
            if (i >= end)
                break;
            const T *dy = reinterpret_cast<const T *>(&in[j].dy);
            const uint32_t *a = &in[j].gate.x, *b = &in[j].up.x;
            uint32_t dg[4], du[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                GateGrad2 m = act_grad<Act>(mul2(decode2(a[p]), both(in[j].sg)),
                                            mul2(decode2(b[p]), both(in[j].su)),
                                            {to_float(dy[2 * p]), to_float(dy[2 * p + 1])});
                if constexpr (std::is_same_v<T, f16>) {
                    m.gate = mul2(m.gate, both(inverse));
                    m.up = mul2(m.up, both(inverse));
                }
                dg[p] = i < live ? pack2<T>(m.gate) : 0;
                du[p] = i < live ? pack2<T>(m.up) : 0;
            }
            T *to = g.rows + (int64_t(e) * 2 * g.padded + i) * g.dp + x;
            st_vec(to, make_uint4(dg[0], dg[1], dg[2], dg[3]));
            st_vec(to + int64_t(g.padded) * g.dp, make_uint4(du[0], du[1], du[2], du[3]));
        }
    }
}

// ------------------------------------------------------------------ host side

struct Operands {
    Layout in, weight;   // as given
};

Operands operands(const gated_act_linear &a) {
    return {{a.in, {a.k, a.T, 1, a.E}, {1, a.in_stride, 0, a.in_batch}},
            {a.weight,
             {a.k, a.d, 2, a.E},
             {1, a.weight_stride, a.d * a.weight_stride, a.weight_batch}}};
}

int check_sizes(const gated_act_linear &a) {
    if (a.E < 0 || a.T < 0 || a.d <= 0 || a.k <= 0)
        return GATED_ACT_ERR_SIZE;
    if (a.dtype != GATED_ACT_BF16 && a.dtype != GATED_ACT_F16)
        return GATED_ACT_ERR_DTYPE;
    if (a.d > kMaxWidth || a.k > kMaxWidth || a.T > kMaxWidth || a.E > GATED_ACT_MAX_EXPERTS ||
        a.in_stride > kMaxRows || a.in_batch > kMaxRows || a.weight_stride > kMaxRows ||
        a.weight_batch > kMaxRows)
        return GATED_ACT_ERR_TOO_LARGE;
    if (a.in_stride < a.k || a.weight_stride < a.k ||
        (a.E > 1 && a.T > 0 && a.in_batch < (a.T - 1) * a.in_stride + a.k) ||
        (a.E > 1 && a.weight_batch < (2 * a.d - 1) * a.weight_stride + a.k))
        return GATED_ACT_ERR_STRIDE;
    // 32-bit tile numbers in each of the three products, 63-bit byte counts
    const int64_t most = (int64_t(1) << 31) - 4096;
    const auto tiles = [&](int64_t rows, int64_t cols, int64_t width) {
        return static_cast<double>(a.E) * static_cast<double>(ceil_div64(rows, kTile)) *
                   static_cast<double>(ceil_div64(cols, width)) <
               static_cast<double>(most);
    };
    if (!tiles(a.T, a.d, 64) || !tiles(a.T + 2 * a.d + kTile, a.k, kHalf) ||
        static_cast<double>(a.E) * static_cast<double>(a.T + kStep) *
                static_cast<double>(2 * a.d + a.k) > 1e17)
        return GATED_ACT_ERR_TOO_LARGE;
    return GATED_ACT_OK;
}

Region in_region(const gated_act_linear &a) {
    return {a.in, span_bytes(a.E, a.in_batch, span_bytes(a.T, a.in_stride, a.k, 1), 2), 2, false};
}
Region weight_region(const gated_act_linear &a) {
    return {a.weight, span_bytes(a.E, a.weight_batch, span_bytes(2 * a.d, a.weight_stride, a.k, 1), 2),
            2, false};
}

// Operands that TMA can address: as they are, or copies in the workspace.
int addressable(Operands *o, Carve *ws, cudaStream_t stream) {
    const bool in = !tma_addressable(o->in), weight = !tma_addressable(o->weight);
    const Layout none = {};
    Layout to[2] = {none, none}, from[2] = {none, none};
    int n = 0;
    for (Layout *t : {in ? &o->in : nullptr, weight ? &o->weight : nullptr}) {
        if (!t)
            continue;
        from[n] = *t;
        to[n] = packed_layout(*t, ws->take<void>(packed_bytes(*t)));
        *t = to[n++];
    }
    return n && ws->start ? launch_pack(to[0], from[0], to[1], from[1], stream) : GATED_ACT_OK;
}

// Rows without a checkpoint have other kernels where they are few: up to 16 of a weight of few turned tiles the one
// that streams it through registers, else up to 128 the turned product.  A turned tile is one long chain of copies, and a
// pair of SMs without a tile idles; the streaming kernel has warps on every SM, but its time grows with the
// rows, and in steps with its rounds of blocks: up to 25 tiles, a third of the pairs, are one round.  Weights off 16-byte
// boundaries are read in place there and copied first for the turned product: any number of tiles below the pairs'.
// Measured in us for 8, 16 and 32 rows (the streaming kernel's third figure is of a form that was not kept):
//                 tiles  floor  streaming         turned
//   256  -> 1024      8    0.2   2.5  3.4  5.1     4.3  4.3  4.4
//   2048 -> 768       6    0.9   4.7  6.4  9.9     8.3  8.3  8.4
//   2048 -> 2048     16    2.5   6.3  8.0 11.4     8.4  8.5  8.5
//   4096 -> 2560     20    6.2  11.8 15.4 36.2    13.0 13.0 13.1
//   2048 -> 4096     32    5.0  11.6 15.0 21.0     9.6  9.7  9.7
//   4096 -> 8192     64   19.8  32.4 42.5 74.4    23.5 23.7 23.7
//   2049 -> 2045     16    2.5  13.5 16.4 19.8    18.8 19.1 19.2   (off 16-byte boundaries)
//   4097 -> 4093     32    9.9  39.0 50.7 69.2    46.4 46.9 47.0
bool few(const gated_act_linear &a, bool keep) {
    const Operands o = operands(a);
    const int64_t tiles = a.E * ceil_div64(a.d, kHalf);
    const bool in_place = tma_addressable(o.in) && tma_addressable(o.weight);
    return !keep && a.T <= kFewRows && (in_place ? tiles <= sm_pairs() / 3 : tiles < sm_pairs());
}

uint64_t forward_bytes(const gated_act_linear &a, bool keep) {
    if (few(a, keep))
        return 0;
    Operands o = operands(a);
    Carve ws(nullptr);
    addressable(&o, &ws, nullptr);
    return ws.used;
}

// Columns of a tile, 256 or 128: those for which the pair of SMs with the most work has less of it.  Work is
// counted in ring steps of 256 columns (0.30 us); a step of 128 is 0.59 of one in the forward product and
// 0.68 in the gradients', both operands of which lie across the sum (2048 x 4096 -> 16384, both in one
// session: 274 and 323 us forward, 560 and 780 backward).  A tile is not done before the one in front of it has left through
// its epilogue: 11 steps of 256 columns (with the checkpoint 21, a gradient 9), 7.4 (11, 6) of 128.
// Measured where it decides: 512 x 4096 -> 2048 forward 23.2 us with 256 columns and 14.8 with 128, 256 x 2048 -> 9728
// 16.5 and 17.5, backward 98.5 and 70.6, 512 x 4096 -> 2048 backward 29.2 and 40.8.
double tile_steps(int64_t steps, double share, double epilogue) {
    const double n = share * static_cast<double>(steps);
    return n < epilogue ? epilogue : n;
}

int forward_columns(const gated_act_linear &a, bool keep) {
    const int64_t tall = a.E * ceil_div64(a.T, kTile), steps = ceil_div64(a.k, kStep), pairs = sm_pairs();
    const auto turns = [&](int64_t n) {
        return static_cast<double>(ceil_div64(tall * ceil_div64(2 * a.d, n), pairs));
    };
    return turns(128) * tile_steps(steps, 0.59, keep ? 11 : 7.4) < turns(256) * tile_steps(steps, 1, keep ? 21 : 11)
               ? 128
               : 256;
}

// How the gradients' products are divided: the columns of a tile, and shares of the first one's sums.
// A few long sums (2d terms, over the tiles of few rows) are as slow as their longest; shares of them cost
// their way through L2 as fp32 (a tile 0.4 of a step, on all pairs) and a second kernel (8 steps).
struct Division {
    int columns, shares;
};
Division division_of(const gated_act_linear &a) {
    const int64_t pairs = sm_pairs(), in_steps = 2 * ceil_div64(a.d, kStep), w_steps = ceil_div64(a.T, kStep);
    // the walk's own division of the two products' tiles among the pairs
    const auto busiest = [&](int64_t n, int64_t shares, double share, double epilogue) {
        const int64_t wide = ceil_div64(a.k, n), first = a.E * shares * ceil_div64(a.T, kTile) * wide;
        const int64_t second = 2 * a.E * ceil_div64(a.d, kTile) * wide, steps = ceil_div64(in_steps, shares);
        const int64_t left = first % pairs, others = left ? pairs - left : 0, ahead = steps / w_steps;
        const int64_t taken = second < ahead * others ? second : ahead * others, rest = second - taken;
        const double f = tile_steps(steps, share, epilogue), w = tile_steps(w_steps, share, epilogue);
        // the pairs in the order in which they take the rest: those with fewer first tiles in front
        const auto load = [&](int64_t firsts, int64_t place, int64_t before) {
            return static_cast<double>(firsts) * f +
                   static_cast<double>(before + rest / pairs + (place < rest % pairs)) * w;
        };
        double most = load(first / pairs, 0, others ? ceil_div64(taken, others) : 0);
        if (left) {
            const double more = load(first / pairs + 1, others, 0);
            most = more > most ? more : most;
        }
        return most + (shares > 1 ? 8 + 0.4 * static_cast<double>(first) / static_cast<double>(pairs) : 0);
    };
    const double narrow = busiest(128, 1, 0.68, 6), wide = busiest(256, 1, 1, 9);
    Division best = {narrow < wide ? 128 : 256, 1};
    double least = 0.85 * (narrow < wide ? narrow : wide);
    for (const int n : {2, 3, 4, 6, 8, 12, 16, 24, 32})
        if (n * 8 <= in_steps && n * a.E <= kMaxBatches && busiest(256, n, 1, 9) < least) {
            least = busiest(256, n, 1, 9);
            best = {256, n};
        }
    return best;
}

// The parts of a forward product that its jobs share.
template <class J> void set_forward(Product<J> *g, const gated_act_linear &a, const int32_t *live) {
    g->live = live;
    g->batches = static_cast<int>(a.E);
    g->capacity = static_cast<int>(a.T);
    g->steps = static_cast<int>(ceil_div64(a.k, kStep));
}

template <class Act, class T, int N, bool KEEP>
int run_product(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear &a, const Operands &o,
                const int32_t *live, cudaStream_t stream) {
    constexpr bool is_bf16 = std::is_same_v<T, bf16>;
    Product<Forward<Act, T, N, KEEP>> g;
    int rc = encode_map(&g.a, o.in, kHalf, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.b, o.weight, N / 2, is_bf16);
    if (rc != GATED_ACT_OK)
        return rc;
    set_forward(&g, a, live);
    g.rows = static_cast<int>(a.T);
    g.n_tiles = static_cast<int>(ceil_div64(a.d, N / 2));
    g.j = {static_cast<T *>(out), codes, scales, static_cast<int>(a.d),
           a.d % 8 == 0 && aligned(out, 16) && aligned(codes, 16)};
    return launch_product(g, a.E * ceil_div64(a.T, kTile) * g.n_tiles, stream);
}

template <class Act, class T, int N>
int run_swapped(void *out, const gated_act_linear &a, const Operands &o, const int32_t *live,
                cudaStream_t stream) {
    constexpr bool is_bf16 = std::is_same_v<T, bf16>;
    Product<Swapped<Act, T, N>> g;
    int rc = encode_map(&g.a, o.weight, 64, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.b, o.in, N / 2, is_bf16);
    if (rc != GATED_ACT_OK)
        return rc;
    set_forward(&g, a, live);
    g.rows = static_cast<int>(a.d);
    g.n_tiles = 1;
    g.j = {static_cast<T *>(out)};
    return launch_product(g, a.E * ceil_div64(a.d, kHalf), stream);
}

template <class Act, class T, bool KEEP>
int run_forward(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear &a,
                const int32_t *live, void *workspace, cudaStream_t stream) {
    Operands o = operands(a);
    if constexpr (!KEEP)
        if (few(a, KEEP))
            return launch_few_rows<Act, T>(
                {static_cast<const T *>(a.in), static_cast<const T *>(a.weight), static_cast<T *>(out),
                 live, a.in_stride, a.in_batch, a.weight_stride, a.weight_batch, static_cast<int>(a.T),
                 static_cast<int>(a.k), static_cast<int>(a.d), 1},
                a.E, tma_addressable(o.in) && tma_addressable(o.weight), stream);
    Carve ws(workspace);
    const int rc = addressable(&o, &ws, stream);
    if (rc != GATED_ACT_OK)
        return rc;
    if constexpr (!KEEP) {
        if (a.T <= 32)
            return run_swapped<Act, T, 32>(out, a, o, live, stream);
        if (a.T <= 128)
            return run_swapped<Act, T, 128>(out, a, o, live, stream);
    }
    return forward_columns(a, KEEP) == 256
               ? run_product<Act, T, 256, KEEP>(out, codes, scales, a, o, live, stream)
               : run_product<Act, T, 128, KEEP>(out, codes, scales, a, o, live, stream);
}

template <class Act>
int forward(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear *a, void *workspace,
            size_t workspace_bytes, cudaStream_t stream) {
    if (!a)
        return GATED_ACT_ERR_NULL;
    int rc = check_sizes(*a);
    if (rc != GATED_ACT_OK || a->T == 0 || a->E == 0)
        return rc;
    const uint64_t need = forward_bytes(*a, codes != nullptr), rows = a->E * a->T;
    if (workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    if (!codes != !scales)
        return GATED_ACT_ERR_NULL;
    Region r[] = {{out, rows * a->d * 2, 2, true},
                  in_region(*a),
                  weight_region(*a),
                  {workspace, need, 16, true},
                  {codes, codes ? rows * 4 * a->d : 0, 2, true},
                  {scales, codes ? rows * 2 * ceil_div64(a->d, kBlock) : 0, 1, true},
                  {a->n_rows, a->n_rows ? uint64_t(a->E) * 4 : 0, 4, false}};
    rc = check_device_regions(r, 7);
    if (rc != GATED_ACT_OK)
        return rc;
    const auto go = [&](auto type, auto keep) {
        using T = decltype(type);
        return run_forward<Act, T, decltype(keep)::value>(out, codes, scales, *a, a->n_rows,
                                                          workspace, stream);
    };
    const auto with_keep = [&](auto type) {
        return codes ? go(type, std::true_type{}) : go(type, std::false_type{});
    };
    return a->dtype == GATED_ACT_BF16 ? with_keep(bf16{}) : with_keep(f16{});
}

// What the backward pass keeps in its workspace.
struct BackwardParts {
    Operands o;
    int64_t dp, kp, padded;
    void *rows, *tail;
    Division division;
    float *sums, *tops, *power;
    int rc;
    BackwardParts(const gated_act_linear &a, void *workspace, cudaStream_t stream) : o(operands(a)) {
        dp = ceil_div64(a.d, 8) * 8;
        kp = ceil_div64(a.k, 8) * 8;
        padded = ceil_div64(a.T, kStep) * kStep;
        Carve ws(workspace);
        rows = ws.take<void>(uint64_t(a.E) * 2 * padded * dp * 2);
        tail = ws.take<void>(a.n_rows ? uint64_t(a.E) * kStep * kp * 2 : 0);
        division = division_of(a);
        sums = ws.take<float>(division.shares > 1 ? uint64_t(4) * kTile * kTile * a.E * division.shares *
                                                        ceil_div64(a.T, kTile) * ceil_div64(a.k, kTile)
                                                  : 0);
        const bool lifted = a.dtype == GATED_ACT_F16;
        tops = ws.take<float>(lifted ? uint64_t(4) * kTops * a.E : 0);
        power = ws.take<float>(lifted ? uint64_t(4) * a.E : 0);
        rc = addressable(&o, &ws, stream);
        bytes = ws.used;
    }
    uint64_t bytes;
};

template <class T, int N, bool SPLIT>
int run_gradients(void *grad_in, void *grad_weight, const gated_act_linear &a, const Layout &rows,
                  const BackwardParts &w, const Layout &tail, cudaStream_t stream) {
    constexpr bool is_bf16 = std::is_same_v<T, bf16>;
    const Operands &o = w.o;
    const int shares = w.division.shares;
    Product<Gradients<T, N, SPLIT>> g;
    int rc = encode_map(&g.a, rows, kHalf, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.b, o.weight, kStep, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.j.rows, rows, kStep, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.j.in, o.in, kStep, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.j.tail, a.n_rows ? tail : o.in, kStep, is_bf16);
    if (rc != GATED_ACT_OK)
        return rc;
    g.live = a.n_rows;
    g.batches = static_cast<int>(a.E) * shares;
    g.capacity = g.rows = static_cast<int>(a.T);
    g.n_tiles = static_cast<int>(ceil_div64(a.k, N));
    g.j.half_steps = static_cast<int>(ceil_div64(a.d, kStep));
    g.steps = 2 * g.j.half_steps;
    g.second.batches = static_cast<int>(2 * a.E);
    g.second.m_tiles = static_cast<int>(ceil_div64(a.d, kTile));
    g.second.n_tiles = g.n_tiles;
    g.second.rows = static_cast<int>(a.d);
    g.j.grad_in = static_cast<T *>(grad_in);
    g.j.grad_weight = static_cast<T *>(grad_weight);
    g.j.sums = w.sums;
    g.j.power = w.power;
    g.j.shares = shares;
    g.j.k = static_cast<int>(a.k);
    g.j.vec_in = a.k % 8 == 0 && aligned(grad_in, 16);
    g.j.vec_weight = a.k % 8 == 0 && aligned(grad_weight, 16);
    rc = launch_product(g, a.E * (shares * ceil_div64(a.T, kTile) + 2 * g.second.m_tiles) * g.n_tiles, stream);
    if (!SPLIT || rc != GATED_ACT_OK)
        return rc;
    const ShareArgs<T> j = {w.sums, w.power, static_cast<T *>(grad_in), a.n_rows, static_cast<int>(a.T),
                            static_cast<int>(a.k), shares};
    const int64_t blocks = a.E * ceil_div64(a.T, 32) * ceil_div64(a.k, 64);
    return cuda_status(launch_kernel(join_shares<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                     stream, 1, j));
}

template <class Act, class T>
int run_backward(void *grad_in, void *grad_weight, const void *grad_out, int64_t grad_stride,
                 int64_t grad_batch, const int16_t *codes, const uint8_t *scales,
                 const gated_act_linear &a, void *workspace, cudaStream_t stream) {
    const int E = static_cast<int>(a.E), d = static_cast<int>(a.d), k = static_cast<int>(a.k);
    const BackwardParts w(a, workspace, stream);
    if (w.rc != GATED_ACT_OK)
        return w.rc;

    GateGradArgs<T> e;
    e.grad = static_cast<const T *>(grad_out);
    e.codes = codes;
    e.scales = scales;
    e.in = static_cast<const T *>(a.in);
    e.rows = static_cast<T *>(w.rows);
    e.tail = static_cast<T *>(w.tail);
    e.live = a.n_rows;
    e.grad_stride = grad_stride;
    e.grad_batch = grad_batch;
    e.in_stride = a.in_stride;
    e.in_batch = a.in_batch;
    e.T_ = static_cast<int>(a.T);
    e.d = d;
    e.dp = static_cast<int>(w.dp);
    e.k = k;
    e.kp = static_cast<int>(w.kp);
    e.padded = static_cast<int>(w.padded);
    e.tops = w.tops;
    e.power = w.power;
    e.n_tops = e.top_pieces = 0;
    if constexpr (std::is_same_v<T, f16>) {
        // rows off 16-byte boundaries begin up to seven elements into their first vector
        const bool whole = aligned(grad_out, 16) && grad_stride % 8 == 0 && grad_batch % 8 == 0;
        e.top_pieces = static_cast<int>(ceil_div64(a.d + (whole ? 0 : 7), 8 * kTopVectors));
        const int64_t want = ceil_div64(int64_t(8) * device_sm_count(), E), most = ceil_div64(a.T * e.top_pieces, 8);
        const int64_t blocks = want < most ? want : most;
        e.n_tops = static_cast<int>(blocks < kTops ? blocks : kTops);
        const int rc = cuda_status(launch_kernel(gradient_tops, dim3(static_cast<unsigned>(e.n_tops), static_cast<unsigned>(E)),
                                                 dim3(256), 0, stream, 1, e));
        if (rc != GATED_ACT_OK)
            return rc;
    }
    const bool vec = d % 8 == 0 && aligned(grad_out, 16) && aligned(codes, 16) &&
                     grad_stride % 8 == 0 && grad_batch % 8 == 0;
    const int64_t wide = ceil_div64(w.dp, 256), most = ceil_div64(w.padded, 8 * kGradRows);
    // eight blocks per SM, each over several rows: 4096 x 8192 in 53.5 us (a block for every 16 rows 57.6, two
    // per SM 70.8)
    int64_t high = ceil_div64(int64_t(8) * device_sm_count(), wide * E);
    high = high < most ? high : most;
    const dim3 grid(static_cast<unsigned>(wide), static_cast<unsigned>(high < 32768 ? high : 32768),
                    static_cast<unsigned>(E));
    auto kernel = vec ? gate_gradients<Act, T, true> : gate_gradients<Act, T, false>;
    int rc = cuda_status(launch_kernel(kernel, grid, dim3(32, 8), 0, stream, 1, e));
    if (rc != GATED_ACT_OK)
        return rc;

    const Layout rows = {w.rows,
                         {a.d, w.padded, 2, a.E},
                         {1, w.dp, w.padded * w.dp, 2 * w.padded * w.dp}};
    const Layout tail = {w.tail, {a.k, kStep, 1, a.E}, {1, w.kp, 0, kStep * w.kp}};

    return w.division.shares > 1
               ? run_gradients<T, 256, true>(grad_in, grad_weight, a, rows, w, tail, stream)
           : w.division.columns == 256
               ? run_gradients<T, 256, false>(grad_in, grad_weight, a, rows, w, tail, stream)
               : run_gradients<T, 128, false>(grad_in, grad_weight, a, rows, w, tail, stream);
}

template <class Act>
int backward(void *grad_in, void *grad_weight, const void *grad_out, int64_t grad_stride,
             int64_t grad_batch, const int16_t *codes, const uint8_t *scales,
             const gated_act_linear *a, void *workspace, size_t workspace_bytes,
             cudaStream_t stream) {
    if (!a)
        return GATED_ACT_ERR_NULL;
    int rc = check_sizes(*a);
    if (rc != GATED_ACT_OK)
        return rc;
    if (grad_stride > kMaxRows || grad_batch > kMaxRows)
        return GATED_ACT_ERR_TOO_LARGE;
    if (grad_stride < a->d ||
        (a->E > 1 && a->T > 0 && grad_batch < (a->T - 1) * grad_stride + a->d))
        return GATED_ACT_ERR_STRIDE;
    if (a->E == 0)
        return GATED_ACT_OK;
    const uint64_t need = a->T ? BackwardParts(*a, nullptr, nullptr).bytes : 0, rows = a->E * a->T;
    if (workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    const uint64_t weight_bytes = uint64_t(a->E) * 4 * a->d * a->k;
    Region r[] = {{grad_in, rows * a->k * 2, 2, true},
                  {grad_weight, weight_bytes, 2, true},
                  {grad_out,
                   span_bytes(a->E, grad_batch, span_bytes(a->T, grad_stride, a->d, 1), 2), 2, false},
                  {codes, rows * 4 * a->d, 2, false},
                  {scales, rows * 2 * ceil_div64(a->d, kBlock), 1, false},
                  in_region(*a),
                  weight_region(*a),
                  {workspace, need, 16, true},
                  {a->n_rows, a->n_rows ? uint64_t(a->E) * 4 : 0, 4, false}};
    rc = check_device_regions(r, 9);
    if (rc != GATED_ACT_OK)
        return rc;
    if (a->T == 0)   // sums over no rows
        return cuda_status(cudaMemsetAsync(grad_weight, 0, weight_bytes, stream));
    if (a->dtype == GATED_ACT_BF16)
        return run_backward<Act, bf16>(grad_in, grad_weight, grad_out, grad_stride, grad_batch,
                                       codes, scales, *a, workspace, stream);
    return run_backward<Act, f16>(grad_in, grad_weight, grad_out, grad_stride, grad_batch, codes,
                                  scales, *a, workspace, stream);
}

}  // namespace

cudaError_t take_linear_act_status(unsigned int *flags) { return take_product_status(flags); }

}  // namespace gact

extern "C" {

size_t linear_and_mul_workspace_bytes(const gated_act_linear *a) {
    if (!a || gact::check_sizes(*a) != GATED_ACT_OK || a->E == 0 || a->T == 0)
        return 0;
    return gact::forward_bytes(*a, true);
}
size_t linear_and_mul_backward_workspace_bytes(const gated_act_linear *a) {
    if (!a || gact::check_sizes(*a) != GATED_ACT_OK || a->E == 0 || a->T == 0)
        return 0;
    return gact::BackwardParts(*a, nullptr, nullptr).bytes;
}
int linear_silu_and_mul(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear *a,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gact::forward<gact::Silu>(out, codes, scales, a, workspace, workspace_bytes, stream);
}
int linear_gelu_and_mul(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear *a,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gact::forward<gact::Gelu>(out, codes, scales, a, workspace, workspace_bytes, stream);
}
int linear_silu_and_mul_backward(void *grad_in, void *grad_weight, const void *grad_out,
                                 int64_t grad_stride, int64_t grad_batch, const int16_t *codes,
                                 const uint8_t *scales, const gated_act_linear *a, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    return gact::backward<gact::Silu>(grad_in, grad_weight, grad_out, grad_stride, grad_batch, codes,
                                      scales, a, workspace, workspace_bytes, stream);
}
int linear_gelu_and_mul_backward(void *grad_in, void *grad_weight, const void *grad_out,
                                 int64_t grad_stride, int64_t grad_batch, const int16_t *codes,
                                 const uint8_t *scales, const gated_act_linear *a, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    return gact::backward<gact::Gelu>(grad_in, grad_weight, grad_out, grad_stride, grad_batch, codes,
                                      scales, a, workspace, workspace_bytes, stream);
}

}  // extern "C"
