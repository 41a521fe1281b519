// Cross entropy of in W' over a large vocabulary, the logits never kept.
//
//   slope_tops    fp16, backward: the largest slope times input, by which live_tokens scales the inputs.
//   live_tokens   numbers the tokens that take part; where some do not, copies their
//                 rows side by side, so that the products run over live rows alone.
//   forward       one product kernel whose epilogue leaves each row's maximum and sum of
//                 exponentials over a tile's 256 columns, the target's column left out; a second
//                 kernel joins them with the target's logit.
//   backward      for each piece of the vocabulary: the logits again, with y = (p - [target]) /
//                 (1 - p_target) as the epilogue; y W added to grad_in's sums; y' and the rows times
//                 their slopes as the piece's rows of grad_weight.  Last, grad_in from its sums.
#include <cfloat>

#include "product.cuh"

#include "gated_act_linear.h"

namespace gact {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Ring steps (64 terms each) after which the sum of a logit is closed.  The tensor cores cut their fp32 sums off
// towards 0 after every instruction (16 terms), half a unit in the last place on average: a sum of k dense terms,
// whose partial sums are half of it on average, loses a share of it that grows as k.  (Expected, with 24 bits:
// k / 16 cuts x 2^-24 x 0.72, the mean of 1 / m over mantissas m in [1, 2), x 1/2 = 1.3e-9 k.  Measured on GB300,
// 65536 sums of N(0, 16) each: 0.93e-9 to 0.97e-9 k in bf16 and 1.03e-9 to 1.12e-9 k in fp16 for k from 1024 to
// 8192.)  Closed sums lose the share of their own terms alone, 5e-7, and are added with rounding; a sum that fp32
// holds exactly stays exact.  For the gradients, which are rounded to 16 bits, twice as many.
// What it costs, 4096 tokens over 32768: k = 640 102 us for 93 (the epilogue no longer hides), 1024 167 for 165,
// 2048 and 8192 nothing; sums closed after 4 steps cost 8% at every k.  Up to 8 (16) steps a kernel without closed
// sums is taken: with them k = 256 took 77 us for 57, as 128 registers of sums leave few for the exponentials.
constexpr int kLossSteps = 8, kSlopeSteps = 16;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger of two, NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The targets as given: a token's, or -1 where it lies outside the vocabulary.
struct Targets {
    const void *data;
    bool wide;
    int V;
    __device__ __forceinline__ int operator[](int i) const {
        const int64_t v = wide ? static_cast<const int64_t *>(data)[i] : static_cast<const int32_t *>(data)[i];
        return v >= 0 && v < V ? static_cast<int>(v) : -1;
    }
};

// ------------------------------------------------------------------ live tokens

// What live_tokens writes; `row` counts live tokens.
struct Tokens {
    int32_t *count;     // [1] live tokens
    int32_t *token;     // [T] the token of a row
    int32_t *goal;      // [T] its target
    // backward: with c = 1 - p_target = -expm1(-loss) and f = grad_loss c,
    float *shift;       // [T] lse and log c, in powers of two
    float *factor;      // [T] f
    float *power;       // [1] 2^e, above every |f| (fp16: that puts the largest |f x| into the type's top binades)
};

template <class T> struct TokenArgs {
    Targets target;
    const T *in;
    const float *grad_loss, *loss, *lse;   // backward
    float *loss_out, *lse_out;      // forward: 0 at dead tokens
    T *grad_in;                     // backward: 0 at dead tokens
    T *rows;                        // copies of live rows, zeros up to a whole step
    T *scaled;                      // backward: the same, times f / 2^e
    const float *tops;              // backward, fp16: [n_tops] each block's largest |f x| of slope_tops
    int64_t low;                    // where what that rounded off lies behind it; 0: nowhere
    Tokens t;
    int64_t in_stride;
    int n, k, kp, segment, n_tops;
    bool copy;                      // also where every token is live
};

constexpr int kTokenThreads = 1024, kTokenWarps = kTokenThreads / 32;
constexpr int kTokenColumns = 4 * 256;   // of a row that a warp takes at a time: four 16-byte loads a thread

__device__ __forceinline__ int block_sum_int(int v, int *red) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xFFFFFFFFu, red[threadIdx.x & 31]);
}

// fp16: the largest finite |f x| of the live tokens, one of each block.  Below a power of two above every |f| alone, f x
// left fp16's upper binades empty, and a token whose slope is 2^-14 of the largest lost bits to the type's lower end
// (its remainder all of them); next to the largest |f x|, 2^-29.  bf16 has fp32's range.  One pass over the rows,
// read as the aligned vectors that hold them (a step of 777 tokens of 1001 over 50001 takes 4.4 us more with it, 348).
constexpr int kTops = 1024;
__global__ void __launch_bounds__(256) slope_tops(TokenArgs<f16> g, float *tops) {
    __shared__ float red[8];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float top = 0.f;
    for (int i = blockIdx.x * 8 + warp; i < g.n; i += gridDim.x * 8) {
        if (g.target[i] < 0)
            continue;
        const float f = fabsf(g.grad_loss[i] * -expm1f(-g.loss[i]));
        if (!(f < INFINITY))   // an infinity or a NaN, whatever it is divided by
            continue;
        const f16 *row = g.in + i * g.in_stride;
        float most = 0.f;
        const int before = before_row(row);
#pragma unroll 4
        for (int c = lane * 8 - before; c < g.k; c += 256)
            most = fmaxf(most, top_of_eight(eight_around(row, c, g.k)));
        top = fmaxf(top, fminf(f * most, FLT_MAX));
    }
    top = __int_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_int(top)));   // top >= 0
    if (lane == 0)
        red[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i)
            top = fmaxf(top, red[i]);
        tops[blockIdx.x] = top;
    }
}

// Each block numbers a segment of the tokens.  It counts those in front of it itself (the
// targets are few bytes and stay in L2), so that no block waits for another.  Bound by its chain of
// loads: the counts, the segment's tokens, their rows; hence one block of 32 warps per SM, with all of a
// segment's rows on their way at once (4096 tokens of 2048 in the backward pass 11.8 us, two blocks of 8 warps,
// each with a row at a time, 30).
template <class T> __global__ void __launch_bounds__(kTokenThreads) live_tokens(TokenArgs<T> g) {
    __shared__ int red[kTokenWarps];
    __shared__ int list[kTokenThreads];
    __shared__ float times[kTokenThreads];
    pdl_wait();
    pdl_trigger();
    const Targets &target = g.target;
    const int begin = blockIdx.x * g.segment, end = min(begin + g.segment, g.n);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int before = 0, all = 0;
    float top = 0.f;
    for (int i0 = threadIdx.x; i0 < g.n; i0 += 4 * kTokenThreads) {   // twelve loads on their way
        int goal[4];
        float weight[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + kTokenThreads * j;
            goal[j] = i < g.n ? target[i] : -1;
            weight[j] = g.grad_loss && !g.tops && i < g.n ? g.grad_loss[i] * -expm1f(-g.loss[i]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            all += goal[j] >= 0;
            before += goal[j] >= 0 && i0 + kTokenThreads * j < begin;
            top = goal[j] >= 0 ? fmaxf(top, fabsf(weight[j])) : top;
        }
    }
    all = block_sum_int(all, red);
    before = block_sum_int(before, red);
    float power = 1.f;
    if (g.tops)
        top = static_cast<int>(threadIdx.x) < g.n_tops ? g.tops[threadIdx.x] : 0.f;
    if (g.grad_loss) {
        const int bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(top));   // top >= 0
        __syncthreads();
        if (lane == 0)
            red[warp] = bits;
        __syncthreads();
        const int most = __reduce_max_sync(0xFFFFFFFFu, red[lane]);
        // the next power of two, a normal number (fp16: 2^-15 of it, below which 2^15 is rounded to at most); 1 for
        // 0 and infinity
        const int e = g.tops ? max((most >> 23) + 1 - 15, 1) : min((most >> 23) + 1, 254);
        power = most == 0 || most >= 0x7F800000 ? 1.f : __int_as_float(e << 23);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *g.t.count = all;
        if (g.grad_loss)
            *g.t.power = power;
    }
    const bool copy = g.copy || all < g.n;
    const int pieces = (g.k + kTokenColumns - 1) / kTokenColumns;
    for (int i0 = begin; i0 < end; i0 += kTokenThreads) {
        const int i = i0 + threadIdx.x, goal = i < end ? target[i] : -1;
        const bool live = goal >= 0;
        // the rank of a live token among this turn's
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, live);
        __syncthreads();
        if (lane == 0)
            red[warp] = __popc(votes);
        list[threadIdx.x] = -1;
        __syncthreads();
        const int count = red[lane], turn = __reduce_add_sync(0xFFFFFFFFu, count);
        const int row = before + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? count : 0) +
                        __popc(votes & ((1u << lane) - 1));
        if (live) {
            list[threadIdx.x] = row;
            g.t.token[row] = i;
            g.t.goal[row] = goal;
            if (g.grad_loss) {
                const float c = -expm1f(-g.loss[i]), f = g.grad_loss[i] * c;
                // c = 0: no slope; infinity makes every y 0 but the target's, and f is 0
                g.t.shift[row] = c > 0.f ? fmaf(g.lse[i], kLog2e, log2f(c)) : INFINITY;
                g.t.factor[row] = f;
                // a row of zeros beside small |f x| may have any slope
                const float y = f / power;
                times[threadIdx.x] = isinf(y) && !isinf(f) ? copysignf(FLT_MAX, f) : y;
            }
        } else if (i < end && g.loss_out) {
            g.loss_out[i] = 0.f;
            g.lse_out[i] = 0.f;
        }
        __syncthreads();
        // rows: copied where they are packed, zero gradients where they are dead
        const int items = copy || g.grad_in ? min(end - i0, kTokenThreads) * pieces : 0;
        for (int item = warp; item < items; item += kTokenWarps) {
            const int j = item / pieces, x = (item - j * pieces) * kTokenColumns + lane * 8, at = list[j];
            if (at >= 0) {
                const T *from = g.in + (i0 + j) * g.in_stride;
                T *to = g.rows + int64_t(at) * g.kp, *scaled = g.scaled + int64_t(at) * g.kp;
                const float f = times[j];
                const bool vec = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
                uint4 v[4];
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    v[p] = x + 256 * p < g.k ? eight(from + x + 256 * p, g.k - x - 256 * p, vec) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int c = x + 256 * p;
                    if (c >= g.k)
                        break;
                    if (copy)
                        st_vec_out(to + c, v[p]);   // rows are padded to eight
                    if (g.scaled) {
                        const T *e = reinterpret_cast<const T *>(&v[p]);
                        uint32_t w[4], rest[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 y = {to_float(e[2 * q]) * f, to_float(e[2 * q + 1]) * f};
                            w[q] = pack2<T>(y);
                            const T *high = reinterpret_cast<const T *>(&w[q]);
                            rest[q] = pack2<T>({y.x - to_float(high[0]), y.y - to_float(high[1])});
                        }
                        st_vec_out(scaled + c, make_uint4(w[0], w[1], w[2], w[3]));
                        if (g.low)
                            st_vec_out(scaled + g.low + c, make_uint4(rest[0], rest[1], rest[2], rest[3]));
                    }
                }
            } else if (g.grad_in) {
                T *to = g.grad_in + int64_t(i0 + j) * g.k;
                const bool vec = (reinterpret_cast<uintptr_t>(to) & 15) == 0;
                for (int c = x; c < x + kTokenColumns && c < g.k; c += 256) {
                    if (vec && c + 8 <= g.k)
                        st_vec(to + c, make_uint4(0, 0, 0, 0));
                    else
                        for (int q = c; q < c + 8 && q < g.k; ++q)
                            to[q] = from_float<T>(0.f);
                }
            }
        }
        before += turn;
        __syncthreads();
    }
    // zeros from the live rows to a whole step of a sum over them
    if (blockIdx.x == 0) {
        const int64_t from = int64_t(all) * g.kp, to = int64_t((all + kStep - 1) / kStep * kStep) * g.kp;
        for (int64_t c = from + 8 * threadIdx.x; c < to; c += 8 * kTokenThreads) {
            if (copy)
                st_vec(g.rows + c, make_uint4(0, 0, 0, 0));
            if (g.scaled)
                st_vec(g.scaled + c, make_uint4(0, 0, 0, 0));
            if (g.scaled && g.low)
                st_vec(g.scaled + g.low + c, make_uint4(0, 0, 0, 0));
        }
    }
}

// ------------------------------------------------------------- products of logits

// Copies of the operands of logits [rows, from `first` on]: packed rows where some token is dead.
template <class G>
__device__ __forceinline__ void load_logits(const G &g, const Tile &t, int first, int step, uint32_t rank,
                                            uint32_t a, uint32_t b, uint32_t bar) {
    load_along(a, t.rows < g.capacity ? &g.j.packed : &g.a, bar, step * kStep,
               t.m0 + static_cast<int>(rank) * kHalf, 0, 0);
    load_along(b, &g.b, bar, step * kStep, first + t.n0 * kTile + static_cast<int>(rank) * kHalf, 0, 0);
}

// Maximum (in powers of two) and sum of exponentials of each row over a tile's columns.  2 T V k operations,
// bound by the tensor cores: 8192 x 65536 x 2048 in 1.11 ms alone (1.98 PFLOP/s), 1.25 ms in a stream of such
// calls (the power limit).  A tile's exponentials take 1.7 us, hidden from k = 384 on.
template <class T, int CLOSED> struct Statistics {
    using Elem = T;
    static constexpr bool kBAcross = false, kSecond = false;
    static constexpr int kN = kTile, kRows = kTile, kClosed = CLOSED;
    static constexpr Live kLive = Live::Rows;
    struct Args {
        CUtensorMap packed;  // the live rows, where some token is dead
        const int32_t *goal;
        float2 *part;        // [capacity, 2 tiles]: maximum, sum of each warp's columns
        int V;
    };
    using G = Product<Statistics>;
    __device__ static int batch_of(const G &, int, bool) { return 0; }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static int steps_of(const G &g, const Tile &) { return g.steps; }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        load_logits(g, t, 0, step, rank, a, b, bar);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, Sums<CLOSED, kN> &sums,
                                  const Stage &stage) {
        const int r = t.m0 + row;
        const bool mine = r < t.rows;
        const int first = t.n0 * kTile, goal = mine ? g.j.goal[r] - first : -1;
        float top = -INFINITY, sum = 0.f;
        for_columns<CLOSED, kN>(sums, stage.part, g.j.V - first, [&](int c, float (&v)[32]) {
            const int n = g.j.V - first - c;
            if (n < 32 || (goal >= c && goal < c + 32)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = i < n && goal - c != i ? v[i] : -INFINITY;
            }
            float most[4] = {-INFINITY, v[0], v[1], v[2]};
#pragma unroll
            for (int i = 3; i < 32; ++i)
                most[i & 3] = max_nan(most[i & 3], v[i]);
            const float here = max_nan(max_nan(most[0], most[1]), max_nan(most[2], most[3]));
            const float now = max_nan(top, here * kLog2e);
            // a row of -infinity alone has no exponential: its maximum is taken as 0
            const float base = now == -INFINITY ? 0.f : now;
            float2 part[2] = {{sum * exp2_fast(top - base), 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 y = fma2({v[i], v[i + 1]}, both(kLog2e), both(-base));
                part[i >> 1 & 1] = add2(part[i >> 1 & 1], {exp2_fast(y.x), exp2_fast(y.y)});
            }
            part[0] = add2(part[0], part[1]);
            sum = part[0].x + part[0].y;
            top = now;
        });
        if (mine)
            g.j.part[int64_t(r) * 2 * g.n_tiles + 2 * t.n0 + stage.part] = make_float2(top, sum);
    }
};

// The same for up to N tokens, which would leave most of a 256-row tile empty, with the roles turned
// round: the vocabulary's rows are the tile's, the tokens its columns (64 x 32000 x 1024: 12.9 us, upright 17.3).  A warp turns its 32 rows of 16
// tokens in shared memory; two lanes then take half of the rows of a token each.
template <class T, int N, int CLOSED> struct TurnedStatistics {
    using Elem = T;
    static constexpr bool kBAcross = false, kSecond = false;
    static constexpr int kN = N, kRows = kTile, kClosed = CLOSED;
    static constexpr Live kLive = Live::Columns;
    struct Args {
        Targets target;
        float2 *part;        // [capacity, 8 tiles]: maximum, sum of 32 columns
        int tiles;
    };
    using G = Product<TurnedStatistics>;
    __device__ static int batch_of(const G &, int, bool) { return 0; }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static int steps_of(const G &g, const Tile &) { return g.steps; }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        load_along(a, &g.a, bar, step * kStep, t.m0 + static_cast<int>(rank) * kHalf, 0, 0);
        load_along(b, &g.b, bar, step * kStep, static_cast<int>(rank) * (N / 2), 0, 0);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, Sums<CLOSED, N> &sums,
                                  const Stage &stage) {
        static_assert(32 * 17 * 4 <= 32 * kStageRow);
        float *held = reinterpret_cast<float *>(stage.p);   // [32 rows, 16 tokens], 17 apart
        const int lane = threadIdx.x & 31, first = t.m0 + (row & ~31), from = (lane >> 4) * 16;
        for_columns<CLOSED, N>(sums, stage.part, t.live, [&](int c, float (&v)[32]) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    held[lane * 17 + i] = t.m0 + row < t.rows ? v[16 * half + i] : -INFINITY;
                __syncwarp();
                const int token = c + 16 * half + (lane & 15);
                const bool mine = token < t.live;
                const int goal = (mine ? g.j.target[token] : -1) - first - from;
                float x[16], top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = held[(from + i) * 17 + (lane & 15)] * kLog2e;
                    x[i] = goal == i ? -INFINITY : x[i];
                    top = max_nan(top, x[i]);
                }
                top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum += exp2_fast(x[i] - base);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
                if (mine && lane < 16)
                    g.j.part[int64_t(token) * 8 * g.j.tiles + (first >> 5)] = make_float2(top, sum);
                __syncwarp();
            }
        });
    }
};

// y = (p - [target]) / c, c = 1 - p_target: the target's is -1, exactly, and the others' sum is 1.  A token's slope
// f = grad_loss c stands outside: grad_in = f (y W) in fp32, grad_weight = y' (f in).  (With the slope inside, the rounding
// of the target's y, half of a row's gradient in one number, was in all of the row: with a few dozen
// tokens the error could be 1.5 of the results' own.)  Times 2^14 in fp16, whose smallest normal number, 2^-14, a
// probability in a large vocabulary often falls below.
template <class T> constexpr float kLift = std::is_same_v<T, f16> ? 16384.f : 1.f;

// The product again, y written as the operand that the next one reads along the sum and across it: 4096 x
// 38912 x 2048 in 337 us (1.94 PFLOP/s).
template <class T, int CLOSED> struct Slopes {
    using Elem = T;
    static constexpr bool kBAcross = false, kSecond = false;
    static constexpr int kN = kTile, kRows = kTile, kClosed = CLOSED;
    static constexpr Live kLive = Live::Rows;
    struct Args {
        CUtensorMap packed;
        Tokens t;
        T *y;              // [padded, piece]
        int V, first, piece;
    };
    using G = Product<Slopes>;
    __device__ static int batch_of(const G &, int, bool) { return 0; }
    __device__ static int batches(const G &g) { return g.batches; }
    __device__ static int steps_of(const G &g, const Tile &) { return g.steps; }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        load_logits(g, t, g.j.first, step, rank, a, b, bar);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, Sums<CLOSED, kN> &sums,
                                  const Stage &stage) {
        const int r = t.m0 + row;
        const bool mine = r < t.rows;
        const int first = g.j.first + t.n0 * kTile;
        const int goal = mine ? g.j.t.goal[r] - first : -1;
        const float shift = mine ? g.j.t.shift[r] : 0.f;
        const int top = t.m0 + (row & ~31), whole = (t.rows + kStep - 1) / kStep * kStep;
        T *y = g.j.y + int64_t(top) * g.j.piece + t.n0 * kTile;   // the warp's first row
        for_columns<CLOSED, kN>(sums, stage.part, g.j.piece - t.n0 * kTile, [&](int c, float (&v)[32]) {
            const int n = mine ? g.j.V - first - c : 0;
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 x = fma2({v[i], v[i + 1]}, both(kLog2e), both(-shift));
                v[i] = exp2_fast(x.x);
                v[i + 1] = exp2_fast(x.y);
            }
            if (goal >= c && goal < c + 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = goal - c == i ? -1.f : v[i];
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = i < n ? v[i] * kLift<T> : 0.f;
            pack32<T>(w, v);
            stage.flush(w, y + c, g.j.piece, whole - top, 32, true);
        });
    }
};

// Shares that grad_in's sums over a piece are split into, so that the longest tile is at most half of
// what each pair of SMs has to do.  The number follows from the live rows: it is taken on the device,
// and from the numbers of a whole piece, so that it is the same for all.
constexpr int kShares = 32;
struct Shares {
    int n_tiles, piece_steps, w_tiles, pairs;   // column tiles of grad_in; the piece's steps; tiles of grad_weight
    __host__ __device__ int operator()(int64_t live) const {
        const int64_t tiles = (live + kTile - 1) / kTile * n_tiles, w_steps = (live + kStep - 1) / kStep;
        const int64_t each = (tiles * piece_steps + w_tiles * w_steps) / pairs + 1;
        int64_t n = (2 * piece_steps + each - 1) / each;
        n = n < piece_steps / 8 ? n : piece_steps / 8;
        return n < 1 ? 1 : n > kShares ? kShares : static_cast<int>(n);
    }
};

// grad_in's sums += y W over one piece: A = y along the sum, B = the weight across it; each batch
// sums a share of the piece's columns.  The sums lie as the threads hold them, 256 x 256 to a tile,
// column after column: a warp writes 128 bytes at once.
// Second, the piece's rows of grad_weight: A = y across the sum over the live rows, B = in across it.
// 4096 x 38912 x 2048 in 665 us (1.96 PFLOP/s); 4096 x 8192 x 2048 in 168 us, as two launches 182.
template <class T> struct PieceGradients {
    using Elem = T;
    static constexpr bool kBAcross = true, kSecond = true;
    static constexpr int kN = kTile, kRows = kTile, kClosed = 0;
    static constexpr Live kLive = Live::Rows;
    struct Args {
        CUtensorMap y, scaled;       // of the second product
        float *sums;
        const float *power;
        T *grad_weight;              // the piece's first row
        Shares shares;
        int k, first, low;           // rows from a scaled row to what it rounded off; 0: not kept
        bool begin, vec;
    };
    using G = Product<PieceGradients>;
    __device__ static int second_steps(const G &g, int live) {
        return (live + kStep - 1) / kStep * (g.j.low ? 2 : 1);
    }
    __device__ static int batch_of(const G &, int, bool) { return 0; }
    __device__ static int batches(const G &g) { return g.j.shares(g.live_of(0)); }
    // shares of whole steps, as even as they get
    __device__ static int first_step(const G &g, const Tile &t, int b) {
        return static_cast<int>(int64_t(g.steps) * b / t.batches);
    }
    __device__ static int steps_of(const G &g, const Tile &t) {
        return first_step(g, t, t.b + 1) - first_step(g, t, t.b);
    }
    __device__ static void load(const G &g, const Tile &t, int step, uint32_t rank, uint32_t a,
                                uint32_t b, uint32_t bar) {
        const int row = t.m0 + static_cast<int>(rank) * kHalf;
        const int col = t.n0 * kTile + static_cast<int>(rank) * kHalf;
        if (!t.second) {
            const int x = (first_step(g, t, t.b) + step) * kStep;
            load_along(a, &g.a, bar, x, row, 0, 0);
            load_across(b, &g.b, bar, g.j.first + x, col, 0, 0);
            return;
        }
        const int whole = (t.live + kStep - 1) / kStep, low = step >= whole;
        const int x = (step - low * whole) * kStep;
        load_across(a, &g.j.y, bar, x, row, 0, 0);
        load_across(b, &g.j.scaled, bar, x + low * g.j.low, col, 0, 0);
    }
    __device__ static void finish(const G &g, const Tile &t, int row, uint32_t sums, const Stage &stage) {
        const int k = g.j.k, r = t.m0 + row, col = t.n0 * kTile;
        const bool mine = r < t.rows;
        if (t.second) {
            const int top = t.m0 + (row & ~31);
            store_tile<kTile>(sums, stage, g.j.grad_weight + int64_t(top) * k + col, k, t.rows - top, k - col,
                              g.j.vec, *g.j.power * (1.f / kLift<T>), t.steps == 0);
            return;
        }
        const int64_t m_tiles = (t.live + kTile - 1) / kTile;
        const int64_t tile = (t.b * m_tiles + t.m0 / kTile) * g.n_tiles + t.n0;
        float *held = g.j.sums + tile * (kTile * kTile) + 32 * stage.part * kTile + row;
        for (int c = 32 * stage.part; c < kTile && col + c < k; c += 64, held += 64 * kTile) {
            float v[32];
            sums_load32(sums + c, v);
            sums_ready(v);
            if (!mine)
                continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float x = t.steps ? v[i] : 0.f;
                if (g.j.begin)
                    held[i * kTile] = x;
                else   // one addition per element and launch: no order to depend on, no load to wait for
                    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(held + i * kTile), "f"(x)
                                 : "memory");
            }
        }
    }
};

// ---------------------------------------------------------------------- the joins

template <class T> struct JoinArgs {
    const float2 *part;
    const T *in, *weight;     // as given: rows in_stride and weight_stride apart
    Tokens t;                 // count null: every token has a row
    Targets target;
    float *loss, *lse;
    int64_t in_stride, weight_stride;
    int parts, k;
};

// WARPS warps per live row: one, or eight where there are few.  The target's logit is summed here in fp32 with rounding: the tensor cores cut
// sums off, 5e-7 of its size even where they are closed.  With the other columns' sum s of
// 2^(l - m), loss = log(1 + s 2^(m - l_target)) where the target is above them, so that a confident
// token's small loss keeps its bits.
template <class T, int WARPS> __global__ void __launch_bounds__(256) join_statistics(JoinArgs<T> g) {
    __shared__ float share[3][8];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = (blockIdx.x * 8 + warp) / WARPS;
    const int thread = warp % WARPS * 32 + lane;
    if (g.t.count && r >= *g.t.count)
        return;
    const int token = g.t.count ? g.t.token[r] : r, target = g.t.count ? g.t.goal[r] : g.target[r];
    if (target < 0) {
        if (thread == 0)
            g.loss[token] = g.lse[token] = 0.f;
        return;
    }
    const T *x = g.in + token * g.in_stride, *w = g.weight + target * g.weight_stride;
    float2 dot[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
    const int from = g.k & ~7;
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15) == 0;
#pragma unroll 4
    for (int c = thread * 8; c < from; c += 256 * WARPS) {   // in one order, whatever the alignment
        const uint4 vx = eight(x + c, 8, vec), vw = eight(w + c, 8, vec);
        const T *px = reinterpret_cast<const T *>(&vx), *pw = reinterpret_cast<const T *>(&vw);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dot[i] = fma2({to_float(px[2 * i]), to_float(px[2 * i + 1])},
                          {to_float(pw[2 * i]), to_float(pw[2 * i + 1])}, dot[i]);
    }
    for (int c = from + thread; c < g.k; c += 32 * WARPS)
        dot[0].x = fmaf(to_float(x[c]), to_float(w[c]), dot[0].x);
    dot[0] = add2(add2(dot[0], dot[1]), add2(dot[2], dot[3]));
    float at = warp_sum(dot[0].x + dot[0].y);

    float top = -INFINITY, sum = 0.f;
    const auto add = [&](float2 p) {
        const float most = max_nan(top, p.x), base = most == -INFINITY ? 0.f : most;
        sum = sum * exp2_fast(top - base) + p.y * exp2_fast(p.x - base);
        top = most;
    };
    constexpr int kAhead = 8;   // of a thread's parts on their way; one exponential each
    for (int i0 = thread; i0 < g.parts; i0 += kAhead * 32 * WARPS) {
        float2 p[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * 32 * WARPS;
            p[j] = i < g.parts ? g.part[int64_t(r) * g.parts + i] : make_float2(-INFINITY, 0.f);
        }
        float most = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            most = max_nan(most, p[j].x);
        const float base = most == -INFINITY ? 0.f : most;
        sum *= exp2_fast(top - base);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            sum = fmaf(p[j].y, exp2_fast(p[j].x - base), sum);
        top = most;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float2 p = {__shfl_xor_sync(0xFFFFFFFFu, top, o), __shfl_xor_sync(0xFFFFFFFFu, sum, o)};
        add(p);
    }
    if (WARPS > 1) {   // a block is one row
        if (lane == 0) {
            share[0][warp] = at;
            share[1][warp] = top;
            share[2][warp] = sum;
        }
        __syncthreads();
        if (thread == 0)
            for (int i = 1; i < WARPS; ++i) {
                at += share[0][i];
                add({share[1][i], share[2][i]});
            }
    }
    if (thread)
        return;
    const float goal = at * kLog2e;
    float lse, loss;
    if (goal >= top) {
        loss = goal == INFINITY ? NAN : log1pf(sum * exp2f(top - goal));
        lse = at + loss;
    } else {
        lse = top * kLn2 + logf(sum + exp2f(goal - top));
        loss = lse - at;
    }
    g.lse[token] = lse;
    g.loss[token] = loss;
}

template <class T> struct GradInArgs {
    const float *sums;
    Tokens t;
    T *out;
    Shares shares;
    int k;
};

// grad_in's rows from the shares of their sums: a block takes 32 rows x 64 columns of a tile, reads
// columns (32 loads on their way per thread) and writes rows.
template <class T> __global__ void __launch_bounds__(256) join_grad_in(GradInArgs<T> g) {
    __shared__ float held[64][33];
    pdl_wait();
    pdl_trigger();
    const int wide = (g.k + 63) / 64, count = *g.t.count;
    const int r0 = static_cast<int>(blockIdx.x / wide) * 32, c0 = static_cast<int>(blockIdx.x % wide) * 64;
    if (r0 >= count)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool mine = r0 + lane < count;   // the lane's row: its place and slope, for the end
    const int token = mine ? g.t.token[r0 + lane] : 0;
    const float slope = mine ? g.t.factor[r0 + lane] * (1.f / kLift<T>) : 0.f;
    const int shares = g.shares(count);
    const int64_t part = int64_t((count + kTile - 1) / kTile) * g.shares.n_tiles * (kTile * kTile);
    const float *from = g.sums + (int64_t(r0 / kTile) * g.shares.n_tiles + c0 / kTile) * (kTile * kTile) +
                        (c0 % kTile) * kTile + r0 % kTile + lane;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < shares; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = warp + 8 * i;
            if (mine && c0 + c < g.k)
                v[i] += from[s * part + c * kTile];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        held[warp + 8 * i][lane] = v[i];
    __syncthreads();
    for (int i = warp; i < 32 && r0 + i < count; i += 8) {
        const float f = __shfl_sync(0xFFFFFFFFu, slope, i);
        T *to = g.out + int64_t(__shfl_sync(0xFFFFFFFFu, token, i)) * g.k + c0;
        for (int c = lane; c < 64 && c0 + c < g.k; c += 32)
            to[c] = from_float<T>(held[c][i] * f);
    }
}

// ------------------------------------------------------------------ host side

int check_sizes(const gated_act_vocabulary &a) {
    if (a.T < 0 || a.k <= 0 || a.V <= 0)
        return GATED_ACT_ERR_SIZE;
    if (a.dtype != GATED_ACT_BF16 && a.dtype != GATED_ACT_F16)
        return GATED_ACT_ERR_DTYPE;
    if (a.T > kMaxWidth || a.k > kMaxWidth || a.V > kMaxWidth || a.in_stride > kMaxRows ||
        a.weight_stride > kMaxRows)
        return GATED_ACT_ERR_TOO_LARGE;
    if (a.in_stride < a.k || a.weight_stride < a.k)
        return GATED_ACT_ERR_STRIDE;
    const double most = 2147479552.0;   // 32-bit tile numbers
    const auto tiles = [&](int64_t x, int64_t y) {
        return static_cast<double>(ceil_div64(x, kTile)) * static_cast<double>(ceil_div64(y, kTile));
    };
    if (tiles(a.T, a.V) >= most || 32 * tiles(a.T, a.k) >= most || tiles(a.V, a.k) >= most)
        return GATED_ACT_ERR_TOO_LARGE;
    return GATED_ACT_OK;
}

Region in_region(const gated_act_vocabulary &a) {
    return {a.in, span_bytes(a.T, a.in_stride, a.k, 2), 2, false};
}
Region weight_region(const gated_act_vocabulary &a) {
    return {a.weight, span_bytes(a.V, a.weight_stride, a.k, 2), 2, false};
}
Region target_region(const gated_act_vocabulary &a) {
    const int64_t size = a.targets64 ? 8 : 4;
    return {a.targets, static_cast<uint64_t>(a.T * size), static_cast<uintptr_t>(size), false};
}

Targets targets_of(const gated_act_vocabulary &a) {
    return {a.targets, a.targets64 != 0, static_cast<int>(a.V)};
}

// Up to 128 tokens are few: the forward product is turned round, and dead tokens, columns of their own, are
// left in (nothing of theirs reaches another), so that no kernel has to count them first.
bool few(const gated_act_vocabulary &a) { return a.T <= 128; }

// Columns of one piece of the vocabulary: as many as give y 256 MB (of which the products that read
// it find half in L2), but at least 8192, so that adding to grad_in's sums (8 bytes per row and column of it)
// stays small beside the products; of those a quarter fewer to a quarter more, the number whose tiles come
// nearest to a whole number of turns of the SM pairs.  (Pieces of 48 MB, which L2 holds, measured a
// third slower at 4096 x 65536 x 1024, 40% live: 945 us against 710 with 64 MB.)
int64_t piece_of(const gated_act_vocabulary &a) {
    const int64_t rows = ceil_div64(a.T, kStep) * kStep, m = ceil_div64(a.T, kTile);
    const int64_t pairs = sm_pairs(), all = ceil_div64(a.V, kTile);
    int64_t n = (int64_t(128) << 20) / rows / kTile;
    n = n < 32 ? 32 : n;
    if (n >= all)
        return all * kTile;
    int64_t best = n;
    double most = 0;
    for (int64_t i = n - n / 4; i <= n + n / 4; ++i) {
        const double full = static_cast<double>(m * i) / static_cast<double>(ceil_div64(m * i, pairs) * pairs);
        if (full >= most) {
            most = full;
            best = i;
        }
    }
    return (best < all ? best : all) * kTile;
}

// The parts of a workspace.
struct Parts {
    Layout in, packed, scaled = {}, weight;
    Tokens t = {};
    float2 *part = nullptr;
    float *sums = nullptr, *tops = nullptr;
    void *y = nullptr;
    int64_t kp, padded, piece, low = 0;
    Shares shares = {};
    bool copy;
    uint64_t bytes;
    int rc;
    Parts(const gated_act_vocabulary &a, bool backward, void *workspace, cudaStream_t stream)
        : in{a.in, {a.k, a.T, 1, 1}, {1, a.in_stride, 0, 0}},
          weight{a.weight, {a.k, a.V, 1, 1}, {1, a.weight_stride, 0, 0}} {
        kp = ceil_div64(a.k, 8) * 8;
        padded = ceil_div64(a.T, kStep) * kStep;
        piece = piece_of(a);
        copy = !tma_addressable(in);
        Carve ws(workspace);
        t.count = ws.take<int32_t>(4);
        t.token = ws.take<int32_t>(4 * a.T);
        t.goal = ws.take<int32_t>(4 * a.T);
        packed = {ws.take<void>(2 * padded * kp), {a.k, padded, 1, 1}, {1, kp, 0, 0}};
        if (backward) {
            t.shift = ws.take<float>(4 * a.T);
            t.factor = ws.take<float>(4 * a.T);
            t.power = ws.take<float>(4);
            tops = ws.take<float>(a.dtype == GATED_ACT_F16 ? 4 * kTops : 0);
            // With a few dozen tokens there is no average over the roundings of f in: what they take off is
            // kept, a second operand of the same size.
            low = a.T <= 256 ? padded : 0;
            scaled = packed;
            scaled.size[1] += low;
            scaled.data = ws.take<void>(2 * (padded + low) * kp);
            y = ws.take<void>(2 * padded * piece);
            shares = {static_cast<int>(ceil_div64(a.k, kTile)),
                      static_cast<int>(ceil_div64(piece < a.V ? piece : a.V, kStep)),
                      static_cast<int>(ceil_div64(piece < a.V ? piece : a.V, kTile) * ceil_div64(a.k, kTile)),
                      sm_pairs()};
            // the most tiles of sums that any number of live rows takes: with more rows there are
            // more tiles and no more shares, and past kShares x pairs tiles the last count has the most
            int64_t most = 0;
            const int64_t m_tiles = ceil_div64(a.T, kTile);
            for (int64_t m = 1; m <= m_tiles; ++m) {
                const int64_t n = m * shares.n_tiles;
                if (n > int64_t(kShares) * shares.pairs)
                    m = m_tiles;
                // fewer rows of the last tile mean fewer steps of grad_weight, and more shares
                const int64_t s = shares((m - 1) * kTile + 1);
                most = m * shares.n_tiles * s > most ? m * shares.n_tiles * s : most;
            }
            sums = ws.take<float>(4 * kTile * kTile * most);
        } else {
            // two warps' shares of a tile's columns, or eight of the turned form's
            part = ws.take<float2>((few(a) ? 64 : 16) * ceil_div64(a.V, kTile) * a.T);
        }
        rc = GATED_ACT_OK;
        if (!tma_addressable(weight)) {
            const Layout to = packed_layout(weight, ws.take<void>(packed_bytes(weight)));
            if (workspace)
                rc = launch_pack(to, weight, stream);
            weight = to;
        }
        bytes = ws.used;
    }
};

template <class T>
int run_live_tokens(const Parts &w, const gated_act_vocabulary &a, const float *grad_loss,
                    const float *loss, const float *lse, float *loss_out, float *lse_out, void *grad_in,
                    cudaStream_t stream) {
    TokenArgs<T> g;
    g.target = targets_of(a);
    g.in = static_cast<const T *>(a.in);
    g.grad_loss = grad_loss;
    g.loss = loss;
    g.lse = lse;
    g.loss_out = loss_out;
    g.lse_out = lse_out;
    g.grad_in = static_cast<T *>(grad_in);
    g.rows = static_cast<T *>(const_cast<void *>(w.packed.data));
    g.scaled = static_cast<T *>(const_cast<void *>(w.scaled.data));
    g.low = w.low * w.kp;
    g.t = w.t;
    g.in_stride = a.in_stride;
    g.n = static_cast<int>(a.T);
    g.k = static_cast<int>(a.k);
    g.kp = static_cast<int>(w.kp);
    g.copy = w.copy;
    g.tops = nullptr;
    g.n_tops = 0;
    if constexpr (std::is_same_v<T, f16>)
        if (grad_loss) {
            const int64_t blocks = ceil_div64(a.T, 8);
            g.n_tops = static_cast<int>(blocks < kTops ? blocks : kTops);
            const int rc = cuda_status(launch_kernel(slope_tops, dim3(static_cast<unsigned>(g.n_tops)), dim3(256), 0,
                                                     stream, 1, g, w.tops));
            if (rc != GATED_ACT_OK)
                return rc;
            g.tops = w.tops;
        }
    const int64_t segment = ceil_div64(a.T, device_sm_count());
    g.segment = static_cast<int>(segment < 8 ? 8 : segment);
    const unsigned grid = static_cast<unsigned>(ceil_div64(a.T, g.segment));
    return cuda_status(launch_kernel(live_tokens<T>, dim3(grid), dim3(kTokenThreads), 0, stream, 1, g));
}

template <class J>
void set_rows(Product<J> *g, const Parts &w, const gated_act_vocabulary &a) {
    g->live = w.t.count;
    g->batches = 1;
    g->capacity = g->rows = static_cast<int>(a.T);
}

// Maps of the live rows: in place, and packed.
template <class T> int encode_rows(CUtensorMap *place, CUtensorMap *packed, const Parts &w, int rows) {
    constexpr bool is_bf16 = std::is_same_v<T, bf16>;
    const int rc = encode_map(packed, w.packed, rows, is_bf16);
    if (rc != GATED_ACT_OK)
        return rc;
    if (w.copy) {
        *place = *packed;
        return rc;
    }
    return encode_map(place, w.in, rows, is_bf16);
}

// The two forms of the statistics' product.
template <class T, int CLOSED> struct Upright {
    static int set(Product<Statistics<T, CLOSED>> *g, const Parts &w, const gated_act_vocabulary &a) {
        g->n_tiles = static_cast<int>(ceil_div64(a.V, kTile));
        g->j.goal = w.t.goal;
        g->j.part = w.part;
        g->j.V = static_cast<int>(a.V);
        const int rc = encode_rows<T>(&g->a, &g->j.packed, w, kHalf);
        return rc == GATED_ACT_OK ? encode_map(&g->b, w.weight, kHalf, std::is_same_v<T, bf16>) : rc;
    }
    using Job = Statistics<T, CLOSED>;
    static int64_t tiles(const gated_act_vocabulary &a) { return ceil_div64(a.T, kTile) * ceil_div64(a.V, kTile); }
};
template <class T, int N, int CLOSED> struct Turned {
    static int set(Product<TurnedStatistics<T, N, CLOSED>> *g, const Parts &w, const gated_act_vocabulary &a) {
        g->live = nullptr;
        g->n_tiles = 1;
        g->rows = static_cast<int>(a.V);
        g->j = {targets_of(a), w.part, static_cast<int>(ceil_div64(a.V, kTile))};
        const int rc = encode_map(&g->b, w.copy ? w.packed : w.in, N / 2, std::is_same_v<T, bf16>);
        return rc == GATED_ACT_OK ? encode_map(&g->a, w.weight, kHalf, std::is_same_v<T, bf16>) : rc;
    }
    using Job = TurnedStatistics<T, N, CLOSED>;
    static int64_t tiles(const gated_act_vocabulary &a) { return ceil_div64(a.V, kTile); }
};
template <class Form>
int run_statistics(Form, const Parts &w, const gated_act_vocabulary &a, cudaStream_t stream) {
    Product<typename Form::Job> g;
    set_rows(&g, w, a);
    g.steps = static_cast<int>(ceil_div64(a.k, kStep));
    const int rc = Form::set(&g, w, a);
    return rc == GATED_ACT_OK ? launch_product(g, Form::tiles(a), stream) : rc;
}

template <class T>
int run_forward(float *loss, float *lse, const gated_act_vocabulary &a, void *workspace,
                cudaStream_t stream) {
    const Parts w(a, false, workspace, stream);
    int rc = w.rc;
    const bool turned = few(a);
    if (rc == GATED_ACT_OK && !turned)
        rc = run_live_tokens<T>(w, a, nullptr, nullptr, nullptr, loss, lse, nullptr, stream);
    if (rc == GATED_ACT_OK && turned && w.copy)
        rc = launch_pack(packed_layout(w.in, const_cast<void *>(w.packed.data)), w.in, stream);
    if (rc != GATED_ACT_OK)
        return rc;
    const auto statistics = [&](auto closed) {
        constexpr int CLOSED = decltype(closed)::value;
        return a.T <= 32 ? run_statistics(Turned<T, 32, CLOSED>{}, w, a, stream)
               : turned  ? run_statistics(Turned<T, 128, CLOSED>{}, w, a, stream)
                         : run_statistics(Upright<T, CLOSED>{}, w, a, stream);
    };
    rc = a.k > kLossSteps * kStep ? statistics(Const<kLossSteps>{}) : statistics(Const<0>{});
    if (rc != GATED_ACT_OK)
        return rc;
    const int parts = static_cast<int>((turned ? 8 : 2) * ceil_div64(a.V, kTile));
    const JoinArgs<T> j = {w.part, static_cast<const T *>(a.in), static_cast<const T *>(a.weight),
                           turned ? Tokens{} : w.t, targets_of(a), loss, lse, a.in_stride,
                           a.weight_stride, parts, static_cast<int>(a.k)};
    // with up to 1024 rows, a block each fills the SMs no better with a warp each
    const bool wide = a.T <= 1024;
    return cuda_status(launch_kernel(wide ? join_statistics<T, 8> : join_statistics<T, 1>,
                                     dim3(static_cast<unsigned>(wide ? a.T : ceil_div64(a.T, 8))), dim3(256),
                                     0, stream, 1, j));
}

template <class T, int CLOSED>
int run_backward(void *grad_in, void *grad_weight, const float *grad_loss, const float *loss,
                 const float *lse, const gated_act_vocabulary &a, void *workspace, cudaStream_t stream) {
    constexpr bool is_bf16 = std::is_same_v<T, bf16>;
    const Parts w(a, true, workspace, stream);
    int rc = w.rc;
    if (rc == GATED_ACT_OK)
        rc = run_live_tokens<T>(w, a, grad_loss, loss, lse, nullptr, nullptr, grad_in, stream);
    const int k = static_cast<int>(a.k);
    const bool vec = a.k % 8 == 0 && aligned(grad_weight, 16);

    Product<Slopes<T, CLOSED>> s;
    Product<PieceGradients<T>> g;
    if (rc == GATED_ACT_OK)
        rc = encode_rows<T>(&s.a, &s.j.packed, w, kHalf);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&s.b, w.weight, kHalf, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.b, w.weight, kStep, is_bf16);
    if (rc == GATED_ACT_OK)
        rc = encode_map(&g.j.scaled, w.scaled, kStep, is_bf16);
    for (int64_t first = 0; first < a.V && rc == GATED_ACT_OK; first += w.piece) {
        const int64_t cols = a.V - first < w.piece ? a.V - first : w.piece;
        const Layout y = {w.y, {cols, w.padded, 1, 1}, {1, w.piece, 0, 0}};
        set_rows(&s, w, a);
        s.n_tiles = static_cast<int>(ceil_div64(cols, kTile));
        s.steps = static_cast<int>(ceil_div64(a.k, kStep));
        s.j.t = w.t;
        s.j.y = static_cast<T *>(w.y);
        s.j.V = static_cast<int>(a.V);
        s.j.first = static_cast<int>(first);
        s.j.piece = static_cast<int>(w.piece);
        rc = launch_product(s, ceil_div64(a.T, kTile) * s.n_tiles, stream);
        if (rc == GATED_ACT_OK)
            rc = encode_map(&g.a, y, kHalf, is_bf16);
        if (rc == GATED_ACT_OK)
            rc = encode_map(&g.j.y, y, kStep, is_bf16);
        if (rc != GATED_ACT_OK)
            return rc;
        set_rows(&g, w, a);
        g.batches = kShares;
        g.n_tiles = w.shares.n_tiles;
        g.steps = static_cast<int>(ceil_div64(cols, kStep));
        g.second.batches = 1;
        g.second.m_tiles = static_cast<int>(ceil_div64(cols, kTile));
        g.second.n_tiles = g.n_tiles;
        g.second.rows = static_cast<int>(cols);
        g.j.sums = w.sums;
        g.j.power = w.t.power;
        g.j.grad_weight = static_cast<T *>(grad_weight) + first * a.k;
        g.j.shares = w.shares;
        g.j.k = k;
        g.j.first = static_cast<int>(first);
        g.j.low = static_cast<int>(w.low);
        g.j.begin = first == 0;
        g.j.vec = vec;
        rc = launch_product(g, (ceil_div64(a.T, kTile) + g.second.m_tiles) * g.n_tiles, stream);
    }
    if (rc != GATED_ACT_OK)
        return rc;
    const GradInArgs<T> j = {w.sums, w.t, static_cast<T *>(grad_in), w.shares, k};
    const int64_t blocks = ceil_div64(a.k, 64) * ceil_div64(a.T, 32);
    return cuda_status(launch_kernel(join_grad_in<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                     stream, 1, j));
}

}  // namespace

cudaError_t take_cross_entropy_status(unsigned int *flags) { return take_product_status(flags); }

}  // namespace gact

using gact::check_sizes;
using gact::Region;

extern "C" {

size_t linear_cross_entropy_workspace_bytes(const gated_act_vocabulary *a) {
    if (!a || check_sizes(*a) != GATED_ACT_OK || a->T == 0)
        return 0;
    return gact::Parts(*a, false, nullptr, nullptr).bytes;
}

size_t linear_cross_entropy_backward_workspace_bytes(const gated_act_vocabulary *a) {
    if (!a || check_sizes(*a) != GATED_ACT_OK || a->T == 0)
        return 0;
    return gact::Parts(*a, true, nullptr, nullptr).bytes;
}

int linear_cross_entropy(float *loss, float *lse, const gated_act_vocabulary *a, void *workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
    if (!a)
        return GATED_ACT_ERR_NULL;
    int rc = check_sizes(*a);
    if (rc != GATED_ACT_OK || a->T == 0)
        return rc;
    const size_t need = linear_cross_entropy_workspace_bytes(a);
    if (workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    const uint64_t each = static_cast<uint64_t>(a->T) * 4;
    Region r[] = {{loss, each, 4, true},     {lse, each, 4, true},
                  gact::in_region(*a),       gact::weight_region(*a),
                  gact::target_region(*a),   {workspace, need, 16, true}};
    rc = gact::check_device_regions(r, 6);
    if (rc != GATED_ACT_OK)
        return rc;
    return a->dtype == GATED_ACT_BF16
               ? gact::run_forward<gact::bf16>(loss, lse, *a, workspace, stream)
               : gact::run_forward<gact::f16>(loss, lse, *a, workspace, stream);
}

int linear_cross_entropy_backward(void *grad_in, void *grad_weight, const float *grad_loss,
                                  const float *loss, const float *lse, const gated_act_vocabulary *a,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!a)
        return GATED_ACT_ERR_NULL;
    int rc = check_sizes(*a);
    if (rc != GATED_ACT_OK)
        return rc;
    const size_t need = linear_cross_entropy_backward_workspace_bytes(a);
    if (workspace_bytes < need)
        return GATED_ACT_ERR_SCRATCH;
    const uint64_t each = static_cast<uint64_t>(a->T) * 4;
    const uint64_t weight_bytes = static_cast<uint64_t>(a->V * a->k) * 2;
    Region r[] = {{grad_in, static_cast<uint64_t>(a->T * a->k) * 2, 2, true},
                  {grad_weight, weight_bytes, 2, true},
                  {grad_loss, each, 4, false},
                  {loss, each, 4, false},
                  {lse, each, 4, false},
                  gact::in_region(*a),
                  gact::weight_region(*a),
                  gact::target_region(*a),
                  {workspace, need, 16, true}};
    rc = gact::check_device_regions(r, 9);
    if (rc != GATED_ACT_OK)
        return rc;
    if (a->T == 0)   // sums over no tokens
        return gact::cuda_status(cudaMemsetAsync(grad_weight, 0, weight_bytes, stream));
    const auto go = [&](auto type) {
        using T = decltype(type);
        return a->k > gact::kSlopeSteps * gact::kStep
                   ? gact::run_backward<T, gact::kSlopeSteps>(grad_in, grad_weight, grad_loss, loss, lse, *a, workspace, stream)
                   : gact::run_backward<T, 0>(grad_in, grad_weight, grad_loss, loss, lse, *a, workspace, stream);
    };
    return a->dtype == GATED_ACT_BF16 ? go(gact::bf16{}) : go(gact::f16{});
}

}  // extern "C"
