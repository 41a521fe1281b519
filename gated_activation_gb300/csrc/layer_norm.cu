// Layer norm, forward and backward (definitions in gated_act_training.h).
//
// HBM bandwidth bounds both: the forward pass reads and writes each row once,
// the backward pass reads two and writes one.  The parameters' gradients are
// sums over the rows: each CTA adds up its own rows' share of every column,
// and a second kernel adds the CTAs' shares in a fixed order, so results do
// not depend on how the blocks were scheduled.  Rates below are of GB300 and, in
// percent, of its copy rate, 6.79 TB/s; inputs larger than L2 in turn.
#include <algorithm>

#include "training.cuh"

namespace gact {
namespace {

constexpr int kThreads = 256;

// -------------------------------------------------- rows that no CTA holds

// Sums over the CTA, the same bits in every thread; red holds 32 values.
__device__ __forceinline__ float2 cta_sum2(float2 v, float2 *red) {
    v = make_float2(warp_sum(v.x), warp_sum(v.y));
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// One CTA per row, the row read again (from L1/L2) for each pass, one element per
// access: rows wider than the rings hold, and rows whose buffers lie at different
// offsets.  1000 x 12345 fp16 takes 27.0 us forward and 50.8 us backward (rings: 17.1
// and 33.2), 100 x 40000 bf16 14.8 and 43.3 us (with 256 threads 52.2 and 97.2).
template <class T, class W, int NT>
__global__ void __launch_bounds__(NT)
ln_forward_wide(T *__restrict__ out, float *__restrict__ mean_out, float *__restrict__ rstd_out,
                const T *__restrict__ in, const W *__restrict__ weight, const W *__restrict__ bias,
                int64_t rows, int64_t d, int64_t rs, float eps) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_trigger();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *x = in + r * rs;
        const float first = to_float(x[0]);
        uint32_t other = 0u;
        bool same;
        float acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += NT) {
            const float v = to_float(x[c]);
            acc += v;
            other |= unlike(v, first);
        }
        const float sum = row_sum<NT>(acc, red[0], other, &same);
        const float mean = same ? first : sum / static_cast<float>(d);
        acc = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += NT) {
            const float e = to_float(x[c]) - mean;
            acc = fmaf(e, e, acc);
        }
        const float var = row_sum<NT>(acc, red[1]) / static_cast<float>(d);
        const float rstd = 1.0f / __fsqrt_rn(var + eps);
        if (threadIdx.x == 0) {
            mean_out[r] = mean;
            rstd_out[r] = rstd;
        }
        for (int64_t c = threadIdx.x; c < d; c += NT) {
            const float h = (to_float(x[c]) - mean) * rstd;
            const float w = to_float(weight[c]);
            out[r * d + c] = from_float<T>(bias ? fmaf(h, w, to_float(bias[c])) : h * w);
        }
    }
}

template <class T, class W, int NT>
__global__ void __launch_bounds__(NT)
ln_backward_rows(T *__restrict__ grad_in, const T *__restrict__ grad, const T *__restrict__ in,
                 const W *__restrict__ weight, const float *__restrict__ mean_in,
                 const float *__restrict__ rstd_in, int64_t rows, int64_t d, int64_t rs,
                 int64_t gs) {
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    int k = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, k ^= 1) {
        const T *x = in + r * rs, *dy = grad + r * gs;
        const float mean = mean_in[r], rstd = rstd_in[r];
        float2 s = make_float2(0.f, 0.f);
        for (int64_t c = threadIdx.x; c < d; c += NT) {
            const float g = to_float(dy[c]) * to_float(weight[c]);
            s.x += g;
            s.y = fmaf(g, (to_float(x[c]) - mean) * rstd, s.y);
        }
        s = cta_sum2(s, red[k]);
        const float ma = s.x / static_cast<float>(d), mb = s.y / static_cast<float>(d);
        for (int64_t c = threadIdx.x; c < d; c += NT) {
            const float g = to_float(dy[c]) * to_float(weight[c]);
            const float h = (to_float(x[c]) - mean) * rstd;
            grad_in[r * d + c] = from_float<T>(rstd * (g - ma - h * mb));
        }
    }
}

// Floats from one share of the d columns to the next: whole 16-byte vectors.
// What lies past column d is not written, and summed into no result.
__host__ __device__ constexpr int64_t share_width(int64_t d) { return (d + 3) / 4 * 4; }

// Columns' shares of the rows [y * per, (y + 1) * per), y = blockIdx.y: one
// column per thread.  part: [2][gridDim.y][share_width(d)].
template <class T>
__global__ void __launch_bounds__(kThreads)
ln_backward_columns(float *__restrict__ part, const T *__restrict__ grad,
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
    part[blockIdx.y * share_width(d) + c] = w;
    part[(gridDim.y + blockIdx.y) * share_width(d) + c] = b;
}

// Adds the n shares of every column, of the weight (blockIdx.y = 0) or the bias:
// a warp reads 128 columns of every kReduceWarps-th share, four per lane.  L2's
// latency bounds it, so the loads are issued together: one CTA per SM leaves them
// the registers, and where there are more CTAs than SMs two share one (whole backward
// pass, one and two: 16384 x 2048 bf16 38.0 and 38.9 us, 800 x 32768 52.3 and 49.6).
constexpr int kReduceWarps = 16, kReduceLoads = 10, kReduceColumns = 128;
template <int PER_SM>
__global__ void __launch_bounds__(32 * kReduceWarps, PER_SM)
ln_backward_reduce(float *__restrict__ grad_weight, float *__restrict__ grad_bias,
                   const float *__restrict__ part, int64_t n, int64_t d) {
    __shared__ float4 sum[kReduceWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kReduceColumns + 4 * lane;
    const int64_t ps = share_width(d);
    const float *p = part + blockIdx.y * n * ps;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d)
        for (int64_t i = warp; i < n; i += kReduceWarps * kReduceLoads) {
            float4 v[kReduceLoads];       // on their way together; past the last, that one
#pragma unroll
            for (int j = 0; j < kReduceLoads; ++j)
                v[j] = __ldcg(reinterpret_cast<const float4 *>(
                    p + min(i + j * kReduceWarps, n - 1) * ps + c));
#pragma unroll
            for (int j = 0; j < kReduceLoads; ++j)
                if (i + j * kReduceWarps < n) {
                    s.x += v[j].x;
                    s.y += v[j].y;
                    s.z += v[j].z;
                    s.w += v[j].w;
                }
        }
    sum[warp][lane] = s;
    __syncthreads();
    const int64_t to = static_cast<int64_t>(blockIdx.x) * kReduceColumns + threadIdx.x;
    if (threadIdx.x < kReduceColumns && to < d) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kReduceWarps; ++w)
            t += reinterpret_cast<const float *>(sum[w])[threadIdx.x];
        (blockIdx.y ? grad_bias : grad_weight)[to] = t;
    }
}

// 8 parameters.
template <class W> __device__ __forceinline__ Vec8<W> load_params(const W *p) {
    Vec8<W> v;
    uint4 *q = reinterpret_cast<uint4 *>(&v);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
        q[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    return v;
}

// ------------------------------------------------------- vectors, a ring
//
// Persistent CTAs, each row held by TPR threads, thread t with the 8-element
// vectors t, t + TPR, ..., V of them; the parameters stay in registers.  Rows
// reach their threads through a ring of S shared-memory slots that cp.async
// fills S - 1 rows ahead, so that HBM keeps streaming while a row is summed
// and written.  A thread copies just the vectors it will read itself: its own
// wait_group is all the synchronization that the ring needs.
//
// EDGES: rows that start or end off a 16-byte boundary.  The ring holds the
// vectors of the row that lie on it; the up to 7 elements before and after them
// are `edges`, one per thread of the row's first warp, read a row ahead into a
// register.  Rows of one kind of offset go to one CTA (its rows are a multiple
// of kKinds apart), so that its threads keep their columns.
//
// 16384 x 2048 bf16 with fp32 parameters takes 22.8 us (87%), 4004 x 4096 fp32 22.8 us
// (85%), 2048 x 16384 bf16 26.6 us (74%: the two barriers of a row that fills the
// CTA).  EDGES costs tests and a dependent load per row: aligned rows through it
// took 29.6 us at 16384 x 2048; 5000 x 2047 bf16 takes 13.0 us (46%).

constexpr int kKinds = 8;      // rows this far apart have the same offset

// Where the vectors of a row of d elements begin, and how many elements they hold.
struct Span8 {
    int head, width;
};
template <class T, bool EDGES> __device__ __forceinline__ Span8 span_of(const T *row, int d) {
    if constexpr (!EDGES)
        return {0, d};
    const int head = min(d, static_cast<int>((-reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)));
    return {head, (d - head) / 8 * 8};
}
// The column of thread t's edge, or -1.
template <bool EDGES> __device__ __forceinline__ int edge_of(const Span8 &s, int d, int t) {
    if constexpr (!EDGES)
        return -1;
    if (t < 8)
        return t < s.head ? t : -1;
    const int c = s.head + s.width + t - 8;
    return t < 16 && c < d ? c : -1;
}

// This thread's part of the ring: `which` counts the rows of a slot (the
// input, and in the backward pass the gradient).  Columns from the span's head.
// A vector is P pieces of 16 bytes, and neighbouring lanes have neighbouring
// pieces: of 16-bit elements a vector is 8 consecutive columns, of 32-bit ones
// twice 4 of them, 4 TPR apart (two pieces side by side would have each access
// of a warp fetch half of every sector that it touches).
template <class T, int NT, int TPR, int V, int ROWS> struct Ring {
    static constexpr int P = sizeof(T) / 2;
    static constexpr int kPiece = 16 / sizeof(T);     // elements of a piece
    uint4 *mine;                                      // [S][ROWS][V][P][NT]
    uint32_t at;
    int t, d;
    __device__ Ring(uint4 *ring, int t_, int d_)
        : mine(ring + threadIdx.x),
          at(static_cast<uint32_t>(__cvta_generic_to_shared(ring + threadIdx.x))), t(t_), d(d_) {}
    __device__ static int index(int slot, int which, int i, int p) {
        return (((slot * ROWS + which) * V + i) * P + p) * NT;
    }
    // Column of element e (0 to 7) of vector i.
    __device__ int column(int i, int e) const {
        return kPiece * (t + TPR * (P * i + e / kPiece)) + e % kPiece;
    }
    __device__ bool in(int i, int e = 0) const { return column(i, e) < d; }
    __device__ void fetch(int slot, int which, const T *row) const {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (in(i, kPiece * p))
                    copy16(at + 16u * index(slot, which, i, p), row + column(i, kPiece * p));
    }
    // Zero past the span's end.
    __device__ Vec8<T> held(int slot, int which, int i) const {
        Vec8<T> v = Vec8<T>::zero();
        uint4 *q = reinterpret_cast<uint4 *>(&v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (in(i, kPiece * p))
                q[p] = mine[index(slot, which, i, p)];
        return v;
    }
    // Nonzero where an element of vector i has other bits than `first`.
    __device__ uint32_t unlike(const Vec8<T> &v, int i, T first) const {
        const uint4 *q = reinterpret_cast<const uint4 *>(&v);
        uint32_t r = 0u;
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (in(i, kPiece * p))
                r |= gact::unlike(q[p], repeated(first));
        return r;
    }
    __device__ void store(const Vec8<T> &v, T *row, int i) const {
        const uint4 *q = reinterpret_cast<const uint4 *>(&v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (in(i, kPiece * p))
                st_vec_out(row + column(i, kPiece * p), q[p]);
    }
    // The parameters of vector i; one by one where they are not aligned.
    template <bool EDGES, class W> __device__ Vec8<W> params(const W *w, int i) const {
        Vec8<W> v = Vec8<W>::zero();
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (in(i, kPiece * p)) {
                const W *from = w + column(i, kPiece * p);
                W *to = reinterpret_cast<W *>(&v) + kPiece * p;
                if constexpr (EDGES) {
#pragma unroll
                    for (int j = 0; j < kPiece; ++j)
                        to[j] = __ldg(from + j);
                } else {
#pragma unroll
                    for (int j = 0; j < kPiece * static_cast<int>(sizeof(W)) / 16; ++j)
                        reinterpret_cast<uint4 *>(to)[j] =
                            __ldg(reinterpret_cast<const uint4 *>(from) + j);
                }
            }
        return v;
    }
};

// Barrier of the TPR threads of one row: the CTA's, or one of its named ones.
template <int NT, int TPR> __device__ __forceinline__ void row_barrier() {
    if constexpr (TPR == NT)
        __syncthreads();
    else if constexpr (TPR > 32)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / TPR), "n"(TPR) : "memory");
}

template <class T, class W, int NT, int V, int S, bool EDGES>
__global__ void __launch_bounds__(NT, 1024 / NT)
ln_forward_ring(T *__restrict__ out, float *__restrict__ mean_out, float *__restrict__ rstd_out,
                const T *__restrict__ in, const W *__restrict__ weight, const W *__restrict__ bias,
                int64_t rows, int d, int64_t rs, float eps) {
    extern __shared__ __align__(16) uint4 slots[];
    __shared__ float red[2][NT / 32];
    const int t = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int64_t G = gridDim.x;
    const Span8 span = span_of<T, EDGES>(in + blockIdx.x * rs, d);
    const int edge = edge_of<EDGES>(span, d, t);
    const Ring<T, NT, NT, V, 1> ring(slots, t, span.width);
    const auto fetch = [&](int64_t r, int slot) {
        if (r < rows)
            ring.fetch(slot, 0, in + r * rs + span.head);
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        fetch(blockIdx.x + k * G, k);
    Vec8<W> w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i] = ring.template params<EDGES>(weight + span.head, i);
        b[i] = bias ? ring.template params<EDGES>(bias + span.head, i) : Vec8<W>::zero();
    }
    float we = 0.f, be = 0.f;
    T next{};      // as loaded: its conversion would wait for it
    if (EDGES && edge >= 0) {
        we = to_float(__ldg(weight + edge));
        be = bias ? to_float(__ldg(bias + edge)) : 0.f;
        if (blockIdx.x < rows)
            next = __ldg(in + blockIdx.x * rs + edge);
    }
    // the sums are of whole vectors, or of any number of elements with EDGES
    constexpr bool kRound = EDGES ? kSumsRound<T, 8 * NT * V + 7> : kSumsRound<T, NT * V>;
    T next_first = kRound && blockIdx.x < rows ? __ldg(in + blockIdx.x * rs) : T{};
    int slot = 0;
    const float inv = 1.0f / static_cast<float>(d);
    for (int64_t r = blockIdx.x; r < rows; r += G) {
        // the slot read in the round before: this thread is done with it
        fetch(r + (S - 1) * G, slot == 0 ? S - 1 : slot - 1);
        const T first = next_first;
        if (kRound && r + G < rows)
            next_first = __ldg(in + (r + G) * rs);
        const float xe = EDGES ? to_float(next) : 0.f;
        if (EDGES && edge >= 0 && r + G < rows)
            next = __ldg(in + (r + G) * rs + edge);
        copy_wait<S - 1>();
        uint32_t other = kRound && EDGES && edge >= 0 ? unlike(xe, to_float(first)) : 0u;
        float2 acc = make_float2(xe, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Vec8<T> x = ring.held(slot, 0, i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = add2(acc, x.pair(j));
            if constexpr (kRound)
                other |= ring.unlike(x, i, first);
        }
        bool same = false;
        float sum;
        if constexpr (kRound)
            sum = row_sum<NT>(acc.x + acc.y, red[0], other, &same);
        else
            sum = row_sum<NT>(acc.x + acc.y, red[0]);
        // the quotient by a product and its residual, which gives the value of a row of one
        // where the sum is exact
        float mean = sum * inv;
        mean = fmaf(fmaf(-mean, static_cast<float>(d), sum), inv, mean);
        if (kRound && same)
            mean = to_float(first);
        const float2 m2 = make_float2(mean, mean);
        acc = make_float2(0.f, 0.f);
        if (EDGES && edge >= 0)
            acc.x = (xe - mean) * (xe - mean);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (ring.in(i)) {
                const Vec8<T> x = ring.held(slot, 0, i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (ring.in(i, 2 * j)) {
                        const float2 e = sub2(x.pair(j), m2);
                        acc = fma2(e, e, acc);
                    }
            }
        const float var = row_sum<NT>(acc.x + acc.y, red[1]) * inv;
        const float rstd = rsqrtf(var + eps);
        const float2 r2 = make_float2(rstd, rstd);
        if (t == 0) {
            mean_out[r] = mean;
            rstd_out[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!ring.in(i))
                continue;
            const Vec8<T> x = ring.held(slot, 0, i);
            Vec8<T> o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o.put(j, fma2(mul2(sub2(x.pair(j), m2), r2), w[i].pair(j), b[i].pair(j)));
            ring.store(o, out + r * d + span.head, i);
        }
        if (EDGES && edge >= 0)
            out[r * d + edge] = from_float<T>(fmaf((xe - mean) * rstd, we, be));
        slot = slot == S - 1 ? 0 : slot + 1;
    }
}

// ------------------------------------------------- forward, wider rows
//
// One CTA per row, which its registers hold; the parameters through L1, which
// the row's loads bypass.  800 x 32768 bf16: 29.7 us (52%), against 65.0 with the row
// read again for each pass.

template <class T, class W, int NT, int V>
__global__ void __launch_bounds__(NT)
ln_forward_vec(T *__restrict__ out, float *__restrict__ mean_out, float *__restrict__ rstd_out,
               const T *__restrict__ in, const W *__restrict__ weight, const W *__restrict__ bias,
               int d, int64_t rs, float eps) {
    __shared__ float red[2][NT / 32];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x;
    const int64_t r = blockIdx.x;
    const T *p = in + r * rs;
    constexpr bool kRound = kSumsRound<T, NT * V>;    // sums of whole vectors
    const T first = kRound ? __ldg(p) : T{};
    Vec8<T> x[V];
    float2 acc = make_float2(0.f, 0.f);
    uint32_t other = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + NT * i);
        x[i] = c < d ? Vec8<T>::load(p + c) : Vec8<T>::zero();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = add2(acc, x[i].pair(j));
        if constexpr (kRound)
            if (8 * (t + NT * i) < d)
                other |= unlike(x[i], first);
    }
    const float n = static_cast<float>(d);
    bool same = false;
    float mean;
    if constexpr (kRound) {
        mean = row_sum<NT>(acc.x + acc.y, red[0], other, &same) / n;
        mean = same ? to_float(first) : mean;
    } else {
        mean = row_sum<NT>(acc.x + acc.y, red[0]) / n;
    }
    const float2 m2 = make_float2(mean, mean);
    acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (8 * (t + NT * i) < d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 e = sub2(x[i].pair(j), m2);
                acc = fma2(e, e, acc);
            }
    const float var = row_sum<NT>(acc.x + acc.y, red[1]) / n;
    const float rstd = 1.0f / __fsqrt_rn(var + eps);
    const float2 r2 = make_float2(rstd, rstd);
    if (t == 0) {
        mean_out[r] = mean;
        rstd_out[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + NT * i);
        if (c >= d)
            continue;
        const Vec8<W> w = load_params(weight + c);
        Vec8<T> o;
        if (bias) {
            const Vec8<W> b = load_params(bias + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o.put(j, fma2(mul2(sub2(x[i].pair(j), m2), r2), w.pair(j), b.pair(j)));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o.put(j, mul2(mul2(sub2(x[i].pair(j), m2), r2), w.pair(j)));
        }
        o.store(out + r * d + c);
    }
}

// ------------------------------------------------------ backward, a ring
//
// CTAs of NT threads, NT / TPR rows at a time, each row's TPR threads with a
// barrier of their own.  A thread holds its columns' shares of the
// parameters' gradients, and the weight, in registers; at the end the CTA
// joins its rows' shares in shared memory and writes one share per column.
// With h = (x - mean) rstd and g = dy w, the gradient is
//   rstd (g - A - h B) = dy (w rstd) + h (-B rstd) - A rstd;
// (x - mean) (-B rstd^2) would be one product less, but rstd^2 leaves fp32's
// range where the deviation is below 1e-19 or above 1e19.
// Rows that one CTA's registers and ring cannot hold are split over a cluster
// of CL CTAs, `chunk` columns each; the row's two sums are then joined through
// distributed shared memory, after a barrier that every CTA has started.
//
// With the second kernel, 16384 x 2048 bf16 with fp32 parameters takes 37.9 us (78%),
// 4004 x 4096 fp32 33.6 us (86%), 2048 x 16384 bf16 43.0 us (69%), 800 x 32768 bf16
// 49.5 us over clusters of two (140.0 with the row read again for each pass), 800 x 16384
// fp32 40.5 us over clusters of two; 5000 x 2047 bf16 22.7 us.  The shares, one per SM and column, are written and read
// again: with few rows they are the larger part (16 x 2048: 4.9 us, two launches).

constexpr int kBackThreads = 512;

// A float2 into the same shared-memory variable of another CTA of the cluster.
__device__ __forceinline__ void put_peer(float2 *p, uint32_t rank, float2 v) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

template <class T, class W, int TPR, int V, int S, int CL, bool EDGES>
__global__ void __launch_bounds__(kBackThreads, 1)
ln_backward_ring(T *__restrict__ grad_in, float *__restrict__ part, const T *__restrict__ grad,
                 const T *__restrict__ in, const W *__restrict__ weight,
                 const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                 int64_t rows, int width, int chunk, int64_t rs, int64_t gs) {
    constexpr int NT = kBackThreads, R = NT / TPR, NW = TPR / 32;
    static_assert(CL == 1 || (R == 1 && !EDGES), "a cluster takes one row at a time");
    extern __shared__ __align__(16) uint4 slots[];
    __shared__ float2 red[2][NT / 32];
    __shared__ float2 peers[2][CL];
    if constexpr (CL > 1)
        cluster_started();
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    // this CTA's columns: d of them from `from` on
    const int rank = CL == 1 ? 0 : blockIdx.x % CL, from = rank * chunk;
    const int d = CL == 1 ? width : max(0, min(chunk, width - from));
    in += from;
    grad += from;
    weight += from;
    grad_in += from;
    part += from;
    pdl_wait();
    pdl_trigger();
    const int64_t share = blockIdx.x / CL, count = gridDim.x / CL;
    const int64_t G = count * R, first = share * R + group;
    const Span8 span = span_of<T, EDGES>(in + first * rs, d);
    const int edge = edge_of<EDGES>(span, d, t);
    const Ring<T, NT, TPR, V, 2> ring(slots, t, span.width);
    const auto fetch = [&](int64_t r, int slot) {
        if (r < rows) {
            ring.fetch(slot, 0, in + r * rs + span.head);
            ring.fetch(slot, 1, grad + r * gs + span.head);
        }
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        fetch(first + k * G, k);
    Vec8<W> w[V];
    float2 dw[V][4], db[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        w[i] = ring.template params<EDGES>(weight + span.head, i);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dw[i][j] = db[i][j] = make_float2(0.f, 0.f);
    }
    float we = 0.f, dwe = 0.f, dbe = 0.f, next_x = 0.f, next_y = 0.f;
    const auto fetch_edge = [&](int64_t r) {
        if (EDGES && edge >= 0 && r < rows) {
            next_x = to_float(__ldg(in + r * rs + edge));
            next_y = to_float(__ldg(grad + r * gs + edge));
        }
    };
    if (EDGES && edge >= 0)
        we = to_float(__ldg(weight + edge));
    fetch_edge(first);
    int slot = 0, k = 0;
    float mean = first < rows ? mean_in[first] : 0.f, rstd = first < rows ? rstd_in[first] : 0.f;
    const float inv = 1.0f / static_cast<float>(width);
    if constexpr (CL > 1) {
        cluster_wait_started();      // the first rows are on their way
    }
    for (int64_t r = first; r < rows; r += G, k ^= 1) {
        // the slot read in the round before: this thread is done with it
        fetch(r + (S - 1) * G, slot == 0 ? S - 1 : slot - 1);
        const float r1 = rstd;
        const float2 r2 = make_float2(r1, r1), m2 = make_float2(mean, mean);
        if (r + G < rows) {
            mean = mean_in[r + G];
            rstd = rstd_in[r + G];
        }
        const float xe = (next_x - m2.x) * r1, ye = next_y;   // an edge's h and gradient
        fetch_edge(r + G);
        copy_wait<S - 1>();
        float2 a2 = make_float2(0.f, 0.f), b2 = a2;
        if (EDGES && edge >= 0) {
            dbe += ye;
            dwe = fmaf(ye, xe, dwe);
            a2.x = ye * we;
            b2.x = ye * we * xe;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Vec8<T> x = ring.held(slot, 0, i), y = ring.held(slot, 1, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 dy = y.pair(j), h = mul2(sub2(x.pair(j), m2), r2);
                db[i][j] = add2(db[i][j], dy);
                dw[i][j] = fma2(dy, h, dw[i][j]);
                const float2 g = mul2(dy, w[i].pair(j));
                a2 = add2(a2, g);
                b2 = fma2(g, h, b2);
            }
        }
        float a = warp_sum(a2.x + a2.y), b = warp_sum(b2.x + b2.y);
        if constexpr (NW > 1) {
            if ((t & 31) == 0)
                red[k][threadIdx.x >> 5] = make_float2(a, b);
            row_barrier<NT, TPR>();
            const float2 s = red[k][group * NW + (t & (NW - 1))];
            a = s.x;
            b = s.y;
#pragma unroll
            for (int o = NW / 2; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
        }
        if constexpr (CL > 1) {
            if (threadIdx.x < CL)
                put_peer(&peers[k][rank], threadIdx.x, make_float2(a, b));
            cluster_barrier();
            a = b = 0.f;
#pragma unroll
            for (int q = 0; q < CL; ++q) {
                a += peers[k][q].x;
                b += peers[k][q].y;
            }
        }
        a *= inv;
        b *= inv;
        const float hs = -b * r1, off = -a * r1;
        const float2 hs2 = make_float2(hs, hs), off2 = make_float2(off, off);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!ring.in(i))
                continue;
            const Vec8<T> x = ring.held(slot, 0, i), y = ring.held(slot, 1, i);
            Vec8<T> o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o.put(j, fma2(y.pair(j), mul2(w[i].pair(j), r2),
                              fma2(mul2(sub2(x.pair(j), m2), r2), hs2, off2)));
            ring.store(o, grad_in + r * width + span.head, i);
        }
        if (EDGES && edge >= 0)
            grad_in[r * width + edge] = from_float<T>(r1 * (ye * we - a - xe * b));
        slot = slot == S - 1 ? 0 : slot + 1;
    }
    if constexpr (CL > 1)
        cluster_barrier();      // no CTA leaves while another writes to it
    // columns' shares: over the CTA's rows in shared memory, group by group
    float *pw = part + share * share_width(width), *pb = pw + count * share_width(width);
    if constexpr (R == 1 && !EDGES) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                if (ring.in(i, 2 * j)) {
                    const int c = ring.column(i, 2 * j);
                    *reinterpret_cast<float4 *>(pw + c) =
                        make_float4(dw[i][j].x, dw[i][j].y, dw[i][j + 1].x, dw[i][j + 1].y);
                    *reinterpret_cast<float4 *>(pb + c) =
                        make_float4(db[i][j].x, db[i][j].y, db[i][j + 1].x, db[i][j + 1].y);
                }
    } else {
        // [R][kCols] for the weight, then, once read, for the bias
        constexpr int kCols = 8 * V * TPR + 16;
        float *sum = reinterpret_cast<float *>(slots);
        copy_wait<0>();
        __syncthreads();      // every group is done with the ring
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float *to = sum + group * kCols;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (ring.in(i, 2 * j)) {
                        const float2 v = which ? db[i][j] : dw[i][j];
                        const int c = span.head + ring.column(i, 2 * j);
                        to[c] = v.x;
                        to[c + 1] = v.y;
                    }
            if (EDGES && edge >= 0)
                to[edge] = which ? dbe : dwe;
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += NT) {
                float v = sum[c];
#pragma unroll
                for (int q = 1; q < R; ++q)
                    v += sum[q * kCols + c];
                (which ? pb : pw)[c] = v;
            }
            __syncthreads();
        }
    }
}

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

// Calls f(integral constant NT): the threads of a row that no ring takes.  1024
// for wide ones: 100 x 12345 fp16 forward 6.4 us against 17.0 with 256 and backward 17.3
// against 35.1, 1000 of them 27.0 against 24.2 and 50.8 against 54.9.
template <class F> int with_threads(int64_t d, F f) {
    return d > 8192 ? f(Const<1024>{}) : f(Const<kThreads>{});
}

// Shares of the parameters' gradients that the second kernel joins: one per
// SM, or per row where there are fewer rows; a multiple of kKinds of them.
int64_t shares(int64_t T) {
    return std::min<int64_t>(ceil_div64(T, kKinds), std::max(1, device_sm_count() / kKinds)) * kKinds;
}

// Calls f(integral constants NT, V, S) for the forward ring over rows of nv
// vectors, 1024 threads per SM; false when it holds no such row.  Two slots, one
// row ahead, are enough: with four 16384 x 2048 bf16 takes 23.5 us against 22.7,
// 16384 x 512 8.2 against 7.0 (the first rows reach the SM as one burst).
template <class F> bool with_forward_ring(int64_t nv, int *rc, F f) {
    constexpr int S = 2;
    if (nv <= 32)
        *rc = f(Const<32>{}, Const<1>{}, Const<S>{});
    else if (nv <= 64)
        *rc = f(Const<32>{}, Const<2>{}, Const<S>{});
    else if (nv <= 128)
        *rc = f(Const<64>{}, Const<2>{}, Const<S>{});
    else if (nv <= 256)
        *rc = f(Const<128>{}, Const<2>{}, Const<S>{});
    else if (nv <= 512)
        *rc = f(Const<256>{}, Const<2>{}, Const<S>{});
    else if (nv <= 1024)
        *rc = f(Const<512>{}, Const<2>{}, Const<S>{});
    else if (nv <= 2048)
        *rc = f(Const<1024>{}, Const<2>{}, Const<S>{});
    else
        return false;
    return true;
}

// Calls f(integral constants TPR, V, S, CL) for the backward ring.  Two slots are
// enough here, too: with six, 192 KB, 16384 x 2048 bf16 takes 40.0 us, with four 39.6,
// with two 38.0.  At four vectors per thread the CTA holds one row, and three are
// better: 2048 x 16384 bf16 43.1 us against 43.9.
template <int SIZE, class F> bool with_backward_ring(int64_t nv, int *rc, F f) {
    constexpr int S2 = 2;    // slots at two vectors per thread
    constexpr Const<1> one{};
    if (nv <= 32)
        *rc = f(Const<32>{}, Const<1>{}, Const<S2>{}, one);
    else if (nv <= 64)
        *rc = f(Const<32>{}, Const<2>{}, Const<S2>{}, one);
    else if (nv <= 128)
        *rc = f(Const<64>{}, Const<2>{}, Const<S2>{}, one);
    else if (nv <= 256)
        *rc = f(Const<128>{}, Const<2>{}, Const<S2>{}, one);
    else if (nv <= 512)
        *rc = f(Const<256>{}, Const<2>{}, Const<S2>{}, one);
    else if (nv <= 1024)
        *rc = f(Const<512>{}, Const<2>{}, Const<S2>{}, one);
    else if constexpr (SIZE == 2) {
        if (nv <= 2048)
            *rc = f(Const<512>{}, Const<4>{}, Const<3>{}, one);
        else if (nv <= 4096)
            *rc = f(Const<512>{}, Const<4>{}, Const<3>{}, Const<2>{});
        else
            return false;
    } else {
        if (nv <= 2048)
            *rc = f(Const<512>{}, Const<2>{}, Const<S2>{}, Const<2>{});
        else if (nv <= 4096)
            *rc = f(Const<512>{}, Const<2>{}, Const<S2>{}, Const<4>{});
        else
            return false;
    }
    return true;
}

// Whether the rows of two buffers, a and b elements apart, start at the same
// offset from a 16-byte boundary, and rows kKinds apart at the same one.
inline bool same_offsets(const Region &x, int64_t a, const Region &y, int64_t b, int64_t size) {
    return (reinterpret_cast<uintptr_t>(x.dev) - reinterpret_cast<uintptr_t>(y.dev)) % 16 == 0 &&
           ((a - b) * size) % 16 == 0;
}
// Vectors of 8 elements that a row of d elements off a boundary holds at most.
inline int64_t vectors_of(int64_t d) { return std::max<int64_t>(1, d / 8); }

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
    const bool vec = d % 8 == 0 && row_stride % 8 == 0 && aligned(r[0].dev, 16) &&
                     aligned(r[3].dev, 16) && aligned(r[4].dev, 16) && aligned(r[5].dev, 16) &&
                     T <= 0x7FFFFFFF;
    return with_types(dtype, param_dtype, [&](auto t, auto w) {
        using E = decltype(t);
        using W = decltype(w);
        const auto ring = [&](auto edges) {
            return [&](auto nt, auto v, auto slots) {
                constexpr size_t smem = slots() * v() * nt() * 8 * sizeof(E);
                const auto kernel = ln_forward_ring<E, W, nt(), v(), slots(), edges()>;
                const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
                if (e != cudaSuccess)
                    return cuda_status(e);
                const int64_t most = std::max(1, device_sm_count() / kKinds) * (1024 / nt());
                const int64_t ctas = std::min<int64_t>(ceil_div64(T, kKinds), most) * kKinds;
                return launched(launch_kernel(
                    kernel, dim3(static_cast<unsigned>(edges() ? ctas : std::min(T, ctas))),
                    dim3(nt()), smem, stream, 1, as<E>(r[0]), as<float>(r[1]), as<float>(r[2]),
                    as<const E>(r[3]), as<const W>(r[4]), as<const W>(r[5]), T,
                    static_cast<int>(d), row_stride, static_cast<float>(eps)));
            };
        };
        int done;
        if (vec && with_forward_ring(d / 8, &done, ring(std::false_type{})))
            return done;
        if (vec && d / 8 <= 4096 && aligned(r[0].dev, 8 * size) && aligned(r[3].dev, 8 * size))
            return launched(launch_kernel(
                ln_forward_vec<E, W, 1024, 4>, dim3(static_cast<unsigned>(T)), dim3(1024), 0,
                stream, 1, as<E>(r[0]), as<float>(r[1]), as<float>(r[2]), as<const E>(r[3]),
                as<const W>(r[4]), as<const W>(r[5]), static_cast<int>(d), row_stride,
                static_cast<float>(eps)));
        if (!vec && same_offsets(r[0], d, r[3], row_stride, size) &&
            with_forward_ring(vectors_of(d), &done, ring(std::true_type{})))
            return done;
        const int64_t grid = std::min<int64_t>(T, int64_t(device_sm_count()) * 64);
        return with_threads(d, [&](auto nt) {
            return launched(launch_kernel(
                ln_forward_wide<E, W, nt()>, dim3(static_cast<unsigned>(grid)), dim3(nt()), 0,
                stream, 1, as<E>(r[0]), as<float>(r[1]), as<float>(r[2]), as<const E>(r[3]),
                as<const W>(r[4]), as<const W>(r[5]), T, d, row_stride, static_cast<float>(eps)));
        });
    });
}

extern "C" size_t layer_norm_backward_workspace_bytes(int64_t T, int64_t d) {
    if (T <= 0 || d <= 0 || d > gact::kMaxWidth)
        return 16;
    return static_cast<size_t>(std::max<int64_t>(16, gact::shares(T) * gact::share_width(d) * 8));
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
        const bool vec = d % 8 == 0 && row_stride % 8 == 0 && grad_stride % 8 == 0 &&
                         aligned(r[0].dev, 16) && aligned(r[4].dev, 16) && aligned(r[5].dev, 16) &&
                         aligned(r[6].dev, 16);
        rc = with_types(dtype, param_dtype, [&](auto t, auto w) {
            using E = decltype(t);
            using W = decltype(w);
            const auto ring = [&](auto edges) {
                return [&](auto tpr, auto v, auto slots, auto cl) {
                    constexpr bool kEdges = edges() && cl() == 1;
                    if (edges() && !kEdges)      // rows that wide are not sent here
                        return static_cast<int>(GATED_ACT_ERR_VARIANT);
                    constexpr size_t smem = 2 * slots() * v() * kBackThreads * 8 * sizeof(E);
                    const auto kernel = ln_backward_ring<E, W, tpr(), v(), slots(), cl(), kEdges>;
                    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
                    if (e != cudaSuccess)
                        return cuda_status(e);
                    const int64_t chunk = ceil_div64(d / 8, cl()) * 8;
                    n = std::min<int64_t>(ceil_div64(T, kBackThreads / tpr()),
                                          std::max<int64_t>(1, shares(T) / cl()));
                    if (kEdges)
                        n = std::min(ceil_div64(n, kKinds) * kKinds, shares(T));
                    return launched(launch_kernel(
                        kernel, dim3(static_cast<unsigned>(n * cl())), dim3(kBackThreads), smem,
                        stream, cl(), as<E>(r[0]), part, as<const E>(r[4]), as<const E>(r[5]),
                        as<const W>(r[6]), as<const float>(r[7]), as<const float>(r[8]), T,
                        static_cast<int>(d), static_cast<int>(chunk), row_stride, grad_stride));
                };
            };
            int done;
            if (vec && with_backward_ring<sizeof(E)>(d / 8, &done, ring(std::false_type{})))
                return done;
            if (!vec && same_offsets(r[0], d, r[5], row_stride, size) &&
                same_offsets(r[0], d, r[4], grad_stride, size) &&
                vectors_of(d) <= (size == 2 ? 2048 : 1024) &&
                with_backward_ring<sizeof(E)>(vectors_of(d), &done, ring(std::true_type{})))
                return done;
            const int64_t grid = std::min<int64_t>(T, int64_t(device_sm_count()) * 64);
            done = with_threads(d, [&](auto nt) {
                return launched(launch_kernel(
                    ln_backward_rows<E, W, nt()>, dim3(static_cast<unsigned>(grid)), dim3(nt()),
                    0, stream, 1, as<E>(r[0]), as<const E>(r[4]), as<const E>(r[5]),
                    as<const W>(r[6]), as<const float>(r[7]), as<const float>(r[8]), T, d,
                    row_stride, grad_stride));
            });
            if (done != GATED_ACT_OK)
                return done;
            const int64_t per = ceil_div64(T, shares(T));
            n = ceil_div64(T, per);
            return launched(launch_kernel(
                ln_backward_columns<E>,
                dim3(static_cast<unsigned>(ceil_div64(d, kThreads)), static_cast<unsigned>(n)),
                dim3(kThreads), 0, stream, 1, part, as<const E>(r[4]), as<const E>(r[5]),
                as<const float>(r[7]), as<const float>(r[8]), T, per, d, row_stride, grad_stride));
        });
        if (rc != GATED_ACT_OK)
            return rc;
    }
    const dim3 grid(static_cast<unsigned>(ceil_div64(d, kReduceColumns)), grad_bias ? 2 : 1);
    const auto reduce = int64_t(grid.x) * grid.y <= device_sm_count() ? ln_backward_reduce<1>
                                                                      : ln_backward_reduce<2>;
    return launched(launch_kernel(reduce, grid, dim3(32 * kReduceWarps), 0, stream, 1,
                                  as<float>(r[1]), as<float>(r[2]),
                                  static_cast<const float *>(part), n, d));
}
