// A router's balance loss, its per-expert counts and the gradient of its
// logits (definitions in gated_act_training.h).
//
// The forward pass reads the logits and the chosen ids once, the backward
// pass reads the logits again (a softmax is recomputed in registers rather
// than stored) and writes their gradient.  65536 x 128 bf16, k = 8, takes 11.3 us
// forward and 8.7 us backward on GB300 (27% and 57% of the copy rate, 6.79 TB/s).
// Latency bounds both: with 22.8 and 19.2 instructions per logit the issue slots are
// 57% busy while a CTA runs (40 and 34% of the whole launch), and a warp waits for its
// next tokens, the exchanges between a token's lanes and, forward, the CTA's barriers
// while the warps' sums are added.  The forward pass's second launch is 2.5 us of it, the counts
// 1 us.  Of 64 tokens both take the latency of a launch, 3.3 and 1.8 us.
//
// Tokens: L lanes share a token, each holding V groups of kLane elements of
// its logits (rows in 16-byte vectors: 8 consecutive elements per group; any
// other layout: one, and L = 32, so that every access of a warp is one
// contiguous run).  The probabilities are summed over tokens per lane in
// registers, over the lanes and warps of a CTA in shared memory, and over the
// CTAs in CTA order; the counts are integers, whose atomics give the same
// result in any order.
//
// Up to kClusterTokens tokens take one launch, a cluster of 8 CTAs that joins its
// sums through distributed shared memory; longer batches write each CTA's
// sums to the workspace, and a second kernel, one such cluster, joins them.
#include <algorithm>

#include "training.cuh"

namespace gact {
namespace {

constexpr int kThreads = 256;             // of the cluster, and of the backward pass
constexpr int kMaxExperts = 1024;
constexpr int kSumRows = 8;               // rows of the shared sums, each for every 8th warp
constexpr int kCluster = 8;

// ------------------------------------------------------------------- tokens

// The logits of one token held by one lane, V groups of N: group i starts at
// element (i * L + lane) * N.  As loaded, so that the next token's can be on
// their way while this one is computed; 0 past the row's end.
template <class T, int L, int V, int N> struct Raw {
    std::conditional_t<N == 8, Vec8<T>, T> v[V];
    __device__ void load(const T *row, int E, int lane) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * L + lane) * N;
            if constexpr (N == 8)
                v[i] = c < E ? Vec8<T>::load(row + c) : Vec8<T>::zero();
            else
                v[i] = c < E ? __ldg(row + c) : from_float<T>(0.f);
        }
    }
};

// A token's softmax, e * inv: e = exp(logit - largest).  A token whose logits
// are all -infinity, and one with E = 0, has e = 0 and inv = 0.
template <class T, int L, int V, int N> struct Row {
    static constexpr int M = V * N, P = (M + 1) / 2;
    float2 e[P];      // M = 1: the second half is 0
    float inv;

    __device__ static int column(int lane, int i) { return (i / N * L + lane) * N + i % N; }
    __device__ static float total(float v) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }

    __device__ Row(const Raw<T, L, V, N> &raw, int E, int lane) {
        float top = -INFINITY;
        if constexpr (N == 8) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float m = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[4 * i + j] = raw.v[i].pair(j);
                    m = fmaxf(m, fmaxf(e[4 * i + j].x, e[4 * i + j].y));
                }
                top = fmaxf(top, (i * L + lane) * N < E ? m : -INFINITY);
            }
        } else {
            e[P - 1].y = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = to_float(raw.v[i]);
                (i & 1 ? e[i / 2].y : e[i / 2].x) = x;
                top = fmaxf(top, i * L + lane < E ? x : -INFINITY);
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // e = (2^y)^2, y = (logit - top) log2(e) / 2: the square carries e down to
        // the subnormal numbers that the flushing exponential would drop.  The
        // difference comes first: it is 0 at the largest logit however far that is
        // from 0, where a product of each alone would leave its rounding.  fmaxf
        // skips a NaN; the exponential of a NaN logit brings it back.
        constexpr float half = 0.5f * 1.4426950408889634f;
        const float from = top == -INFINITY ? 0.f : top;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            // past the row's end 2^-infinity
            const float fx = column(lane, 2 * i) < E ? from : INFINITY;
            const float fy = N == 8 ? fx : column(lane, 2 * i + 1) < E && 2 * i + 1 < M ? from : INFINITY;
            float2 y = mul2(sub2(e[i], make_float2(fx, fy)), both(half));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y.x));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y.y));
            e[i] = mul2(y, y);
            sum = add2(sum, e[i]);
        }
        const float s = total(sum.x + sum.y);
        inv = s == 0.f ? 0.f : 1.0f / s;
    }
};

// The chosen ids, int32 or int64.
struct Ids {
    const void *p;
    int wide;
    __device__ int64_t at(int64_t i) const {
        return wide ? __ldg(static_cast<const long long *>(p) + i)
                    : static_cast<int64_t>(__ldg(static_cast<const int *>(p) + i));
    }
};

// Nonzero for a live token t of those before `end`.
__device__ __forceinline__ uint8_t live_at(const uint8_t *live, uint32_t t, uint32_t end) {
    return t >= end ? uint8_t(0) : live ? __ldg(live + t) : uint8_t(1);
}

constexpr int kIdLoads = 4;               // ids of a thread on their way together

// Sums of the tokens [t0, t1) into shared memory: sums [kSumRows][E], of which
// row r holds every kSumRows-th warp's, hist [E + 1] counts and live tokens.
// NT threads; ends with a barrier.
template <class T, int NT, int L, int V, int N>
__device__ __forceinline__ void sum_tokens(float *sums, int *hist, const T *logits, Ids ids,
                                           const uint8_t *live, uint32_t t0, uint32_t t1, int E,
                                           int k, int64_t ls) {
    constexpr int kTokens = 32 / L;       // tokens of a warp at a time
    constexpr int kWarps = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = lane / L, sub = lane % L;
    using R = Row<T, L, V, N>;
    // two tokens on their way, and whether the two after them are live
    Raw<T, L, V, N> raw[2];
    uint8_t on[2], next[2];
    constexpr uint32_t step = kWarps * kTokens;
    const auto fetch = [&](uint32_t t, int slot) {
        on[slot] = next[slot];
        raw[slot].load(logits + (t + part) * ls, on[slot] ? E : 0, sub);
        next[slot] = live_at(live, t + part + 2 * step, t1);
    };
    uint32_t t = t0 + warp * kTokens;
    next[0] = live_at(live, t + part, t1);
    next[1] = live_at(live, t + part + step, t1);
    fetch(t, 0);
    fetch(t + step, 1);
    // the counts, while the first tokens arrive
    const uint32_t kn = static_cast<uint32_t>(k), n = (t1 - t0) * kn;
    const int64_t first = static_cast<int64_t>(t0) * k;
    for (uint32_t j = threadIdx.x; j < n; j += NT * kIdLoads) {
        int64_t e[kIdLoads];
        uint8_t in[kIdLoads];
#pragma unroll
        for (int i = 0; i < kIdLoads; ++i) {
            const uint32_t at = j + i * NT;
            e[i] = at < n ? ids.at(first + at) : -1;
            in[i] = at < n ? live_at(live, t0 + at / kn, t1) : uint8_t(0);
        }
#pragma unroll
        for (int i = 0; i < kIdLoads; ++i)
            if (in[i] && e[i] >= 0 && e[i] < E)
                atomicAdd(hist + e[i], 1);
    }
    float2 acc2[R::P];
#pragma unroll
    for (int i = 0; i < R::P; ++i)
        acc2[i] = make_float2(0.f, 0.f);
    int mine = 0;
    // every lane takes part in the shuffles of every round; a token that is not
    // live adds zeros
    const auto take = [&](int slot) {
        const R p(raw[slot], on[slot] ? E : 0, sub);
        mine += on[slot] != 0 && sub == 0;
        fetch(t + 2 * step, slot);
#pragma unroll
        for (int i = 0; i < R::P; ++i)
            acc2[i] = fma2(p.e[i], both(p.inv), acc2[i]);
        t += step;
    };
    while (t < t1) {
        take(0);
        if (t < t1)
            take(1);
    }
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    if (lane == 0 && mine)
        atomicAdd(hist + E, mine);
    float acc[V * N];
#pragma unroll
    for (int i = 0; i < V * N; ++i)
        acc[i] = i & 1 ? acc2[i / 2].y : acc2[i / 2].x;
#pragma unroll
    for (int i = 0; i < V * N; ++i)
#pragma unroll
        for (int o = L; o < 32; o <<= 1)
            acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    // the rows of sums take the warps in turn: a fixed order
#pragma unroll
    for (int w = 0; w < kWarps; w += kSumRows) {
        if (part == 0 && warp >= w && warp < w + kSumRows) {
            float *row = sums + (warp - w) * E;
#pragma unroll
            for (int i = 0; i < V * N; ++i) {
                const int c = R::column(sub, i);
                if (c < E)
                    row[c] = w == 0 ? acc[i] : row[c] + acc[i];
            }
        }
        __syncthreads();
    }
}

__device__ __forceinline__ float rows_sum(const float *sums, int E, int e) {
    float s = sums[e];
#pragma unroll
    for (int w = 1; w < kSumRows; ++w)
        s += sums[w * E + e];
    return s;
}

// ------------------------------------------------------------- the cluster

// A word of the same shared-memory variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer(const void *p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// The CTA's share of sum_e c_e p_e, joined over the cluster: rank 0 writes
// the loss.  `mine`: the thread's term; red: a float per warp.
template <int NT>
__device__ __forceinline__ void write_loss(float *loss, float *share, float *red, float mine,
                                           float scale, uint32_t rank) {
    mine = warp_sum(mine);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
            s += red[w];
        *share = s;
    }
    cluster_barrier();
    if (rank == 0 && threadIdx.x == 0) {
        float s = 0.f;
        for (int c = 0; c < kCluster; ++c)
            s += __uint_as_float(peer(share, c));
        loss[0] = s * scale;
    }
    cluster_barrier();   // no CTA leaves while its share is read
}

// One launch: the cluster's CTAs take `per` tokens each, then E / 8 experts.
template <class T, int L, int V, int N>
__global__ void __launch_bounds__(kThreads)
balance_cluster(float *__restrict__ loss, int32_t *__restrict__ counts,
                int32_t *__restrict__ tokens, float *__restrict__ mean_p,
                const T *__restrict__ logits, Ids ids,
                const uint8_t *__restrict__ live, int64_t T_, int64_t per, int E, int k,
                int64_t ls, float coef) {
    extern __shared__ float sums[];                              // [kSumRows][E]
    int *hist = reinterpret_cast<int *>(sums + kSumRows * E);    // [E + 1]
    __shared__ float share, red[kThreads / 32];
    for (int e = threadIdx.x; e <= E; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint32_t rank = cluster_rank();
    const uint32_t t0 = min(T_, rank * per), t1 = min(T_, t0 + per);
    sum_tokens<T, kThreads, L, V, N>(sums, hist, logits, ids, live, t0, t1, E, k, ls);
    for (int e = threadIdx.x; e < E; e += kThreads)
        sums[e] = rows_sum(sums, E, e);                       // only this thread reads column e
    cluster_barrier();
    int n = 0;
    for (int c = 0; c < kCluster; ++c)
        n += static_cast<int>(peer(hist + E, c));
    const float nf = static_cast<float>(n > 0 ? n : 1);
    float mine = 0.f;
    for (int e = rank + kCluster * threadIdx.x; e < E; e += kCluster * kThreads) {
        float p = 0.f;
        int c = 0;
        for (int r = 0; r < kCluster; ++r) {
            p += __uint_as_float(peer(sums + e, r));
            c += static_cast<int>(peer(hist + e, r));
        }
        p /= nf;
        counts[e] = c;
        mean_p[e] = p;
        mine = fmaf(static_cast<float>(c), p, mine);
    }
    if (rank == 0 && threadIdx.x == 0)
        tokens[0] = n;
    write_loss<kThreads>(loss, &share, red, mine,
               coef * static_cast<float>(E) / (nf * static_cast<float>(k)), rank);
}

// Long batches: CTA b of G takes the tokens [b * per, (b + 1) * per) and leaves
// its sums in the workspace, an expert's G of them side by side:
// part_p [E][G] fp32, part_c [E + 1][G] int32 (the last: live tokens).
template <class T, int NT, int L, int V, int N>
__global__ void __launch_bounds__(NT)
balance_tokens(float *__restrict__ part_p, int32_t *__restrict__ part_c,
               const T *__restrict__ logits, Ids ids,
               const uint8_t *__restrict__ live, int64_t T_, int64_t per, int E, int k,
               int64_t ls) {
    extern __shared__ float sums[];
    int *hist = reinterpret_cast<int *>(sums + kSumRows * E);
    for (int e = threadIdx.x; e <= E; e += NT)
        hist[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint32_t t0 = min(T_, blockIdx.x * per), t1 = min(T_, t0 + per);
    sum_tokens<T, NT, L, V, N>(sums, hist, logits, ids, live, t0, t1, E, k, ls);
    const int64_t G = gridDim.x;
    for (int e = threadIdx.x; e <= E; e += NT) {
        part_c[e * G + blockIdx.x] = hist[e];
        if (e < E)
            part_p[e * G + blockIdx.x] = rows_sum(sums, E, e);
    }
}

// Joins the G sums of every expert, G <= 32 kJoinLoads: a warp takes an expert.
constexpr int kJoinThreads = 512;
constexpr int kJoinLoads = 8;
__global__ void __launch_bounds__(kJoinThreads, 1)
balance_join(float *__restrict__ loss, int32_t *__restrict__ counts, int32_t *__restrict__ tokens,
             float *__restrict__ mean_p, const float *__restrict__ part_p,
             const int32_t *__restrict__ part_c, int G, int E, float k, float coef) {
    constexpr int kWarps = kJoinThreads / 32;
    __shared__ float share, red[kWarps];
    pdl_wait();
    pdl_trigger();
    const uint32_t rank = cluster_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int e = rank * kWarps + warp;
    float p[kJoinLoads];
    int c[kJoinLoads], n = 0;
    const auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i) {
            const bool in = e < E && lane + 32 * i < G;
            p[i] = in ? part_p[e * G + lane + 32 * i] : 0.f;
            c[i] = in ? part_c[e * G + lane + 32 * i] : 0;
        }
    };
    fetch();
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i)
        n += lane + 32 * i < G ? part_c[E * G + lane + 32 * i] : 0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    const float nf = static_cast<float>(n > 0 ? n : 1);
    float mine = 0.f;
    while (e < E) {
        float ps = 0.f;
        int cs = 0;
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i) {
            ps += p[i];
            cs += c[i];
        }
        const int at = e;
        e += kCluster * kWarps;
        fetch();
        ps = warp_sum(ps) / nf;
        cs = __reduce_add_sync(0xFFFFFFFFu, cs);
        if (lane == 0) {
            counts[at] = cs;
            mean_p[at] = ps;
            mine = fmaf(static_cast<float>(cs), ps, mine);
        }
    }
    if (rank == 0 && threadIdx.x == 0)
        tokens[0] = n;
    write_loss<kJoinThreads>(loss, &share, red, mine, coef * static_cast<float>(E) / (nf * k), rank);
}

// Counts enter as c_j - C / E, C their sum, rounded to an integer: the same
// gradient, since p sums to 1, without the cancellation of nearly equal counts.  The
// difference is one of integers: fp32 does not hold a count past 2^24.
template <class T, int L, int V, int N>
__global__ void __launch_bounds__(kThreads)
balance_backward(T *__restrict__ grad, const float *__restrict__ grad_loss,
                 const T *__restrict__ logits, const int32_t *__restrict__ counts,
                 const int32_t *__restrict__ tokens, const uint8_t *__restrict__ live, int64_t T_,
                 int E, float k, int64_t ls, float coef) {
    using R = Row<T, L, V, N>;
    constexpr int kTokens = 32 / L, kWarps = kThreads / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, part = lane / L, sub = lane % L;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens + part;
    Raw<T, L, V, N> raw;
    bool on;
    const auto fetch = [&](int64_t at) {
        on = at < T_ && (!live || live[at]);
        raw.load(logits + at * ls, on ? E : 0, sub);
    };
    fetch(t);
    int chosen[2 * R::P];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * R::P; ++i) {
        const int e = R::column(sub, i);
        chosen[i] = i < R::M && e < E ? __ldg(counts + e) : 0;
        sum += static_cast<float>(chosen[i]);
    }
    const int n = *tokens;
    const float up = *grad_loss;
    const int mid = static_cast<int>(rintf(R::total(sum) / static_cast<float>(E)));
    float2 c[R::P];
#pragma unroll
    for (int i = 0; i < R::P; ++i)
        c[i] = make_float2(static_cast<float>(chosen[2 * i] - mid),
                           static_cast<float>(chosen[2 * i + 1] - mid));
    const float nf = static_cast<float>(n > 0 ? n : 1);
    const float scale = up * (coef * static_cast<float>(E) / (nf * nf * k));
    // every lane takes part in the shuffles of every round
    for (; t - part < T_; t += step) {
        const R p(raw, on ? E : 0, sub);
        const float up_row = on ? scale : 0.f;      // no product of 0 and a scale that overflowed
        fetch(t + step);
        float2 mix = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R::P; ++i)
            mix = fma2(p.e[i], c[i], mix);
        const float mixed = R::total(mix.x + mix.y) * p.inv, s = up_row * p.inv;
        if (t >= T_)
            continue;
        T *row = grad + t * E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = (i * L + sub) * N;
            if (at >= E)
                continue;
            if constexpr (N == 8) {
                Vec8<T> o;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o.put(j, mul2(mul2(p.e[4 * i + j], both(s)), sub2(c[4 * i + j], both(mixed))));
                o.store(row + at);
            } else {
                const float e = i & 1 ? p.e[i / 2].y : p.e[i / 2].x;
                row[at] = from_float<T>(e * s * ((i & 1 ? c[i / 2].y : c[i / 2].x) - mixed));
            }
        }
    }
}

// -------------------------------------------------------------- host side

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

// Calls f(integral constants L, V, N) for E experts: two vectors of 8 per lane, or
// single elements.  One vector per lane exchanges more in the backward pass, four keep
// fewer tokens on their way.  Forward and backward, us, with one, two and four:
//   65536 x 128 bf16   11.0 11.6    11.2  8.7    10.7  9.2
//   32768 x 64 fp32     7.7  5.2     7.4  5.2     8.4  4.5
template <class F> int with_lanes(int64_t E, bool vec, F f) {
    if (vec)
        return E <= 8     ? f(Const<1>{}, Const<1>{}, Const<8>{})
               : E <= 16  ? f(Const<1>{}, Const<2>{}, Const<8>{})
               : E <= 32  ? f(Const<2>{}, Const<2>{}, Const<8>{})
               : E <= 64  ? f(Const<4>{}, Const<2>{}, Const<8>{})
               : E <= 128 ? f(Const<8>{}, Const<2>{}, Const<8>{})
               : E <= 256 ? f(Const<16>{}, Const<2>{}, Const<8>{})
               : E <= 512 ? f(Const<32>{}, Const<2>{}, Const<8>{})
                          : f(Const<32>{}, Const<4>{}, Const<8>{});
    return E <= 32    ? f(Const<32>{}, Const<1>{}, Const<1>{})
           : E <= 64  ? f(Const<32>{}, Const<2>{}, Const<1>{})
           : E <= 128 ? f(Const<32>{}, Const<4>{}, Const<1>{})
           : E <= 256 ? f(Const<32>{}, Const<8>{}, Const<1>{})
           : E <= 512 ? f(Const<32>{}, Const<16>{}, Const<1>{})
                      : f(Const<32>{}, Const<32>{}, Const<1>{});
}

// Batches of up to this many tokens take the one-launch cluster: 128 experts, bf16,
// 512 tokens 4.0 us against 5.7 with two launches, 768 4.7 against 5.7, 1024 5.4 against
// 5.8, 2048 7.8 against 5.8; 512 experts, 512 tokens 8.1 against 10.2, 1024 12.6 against 8.4.
constexpr int64_t kClusterTokens = 768;

// CTAs that a longer batch's tokens are split over: one per SM, of at least 32
// tokens each.  The join reads up to 32 kJoinLoads of them.
int64_t parts(int64_t T) {
    return std::max<int64_t>(1, std::min<int64_t>({ceil_div64(T, 32), device_sm_count(),
                                                   int64_t(32) * kJoinLoads}));
}

}  // namespace
}  // namespace gact

extern "C" size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t E) {
    if (T <= gact::kClusterTokens || E <= 0 || E > gact::kMaxExperts)
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
    const bool vec = E % 8 == 0 && logits_stride % 8 == 0 && aligned(r[5].dev, 8 * size);
    const bool cluster = T <= kClusterTokens;
    const int64_t G = cluster ? kCluster : parts(T), per = ceil_div64(T, G);
    float *part_p = as<float>(r[4]);
    int32_t *part_c = reinterpret_cast<int32_t *>(part_p + G * E);
    const int Ei = static_cast<int>(E), ki = static_cast<int>(k);
    const float c = static_cast<float>(coef);
    const Ids chosen = {r[6].dev, ids64};
    rc = with_type(dtype, [&](auto t) {
        return with_lanes(E, vec, [&](auto l, auto v, auto n) {
            using Elem = decltype(t);
            const size_t smem = (kSumRows * E + E + 1) * 4;
            if (cluster)
                return launched(launch_kernel(
                    balance_cluster<Elem, l(), v(), n()>, dim3(kCluster), dim3(kThreads), smem,
                    stream, kCluster, as<float>(r[0]), as<int32_t>(r[1]), as<int32_t>(r[2]),
                    as<float>(r[3]), as<const Elem>(r[5]), chosen, as<const uint8_t>(r[7]), T,
                    per, Ei, ki, logits_stride, c));
            // 32 warps per SM; 16 where the registers of a lane's logits forbid it, and
            // where the warps' sums, added up a few warps at a time, are long: 16384 x
            // 512 bf16 13.4 us against 15.3, 32768 x 64 fp32 7.4 against 9.2 (65536 x 128
            // bf16: 14.4 against 11.2 with 32)
            constexpr int NT = l() * v() * n() > 256 || sizeof(Elem) * v() * n() > 32 ? 512 : 1024;
            return launched(launch_kernel(
                balance_tokens<Elem, NT, l(), v(), n()>, dim3(static_cast<unsigned>(G)),
                dim3(NT), smem, stream, 1, part_p, part_c, as<const Elem>(r[5]), chosen,
                as<const uint8_t>(r[7]), T, per, Ei, ki, logits_stride));
        });
    });
    if (rc != GATED_ACT_OK || cluster)
        return rc;
    return launched(launch_kernel(
        balance_join, dim3(kCluster), dim3(kJoinThreads), 0, stream, kCluster, as<float>(r[0]),
        as<int32_t>(r[1]), as<int32_t>(r[2]), as<float>(r[3]), static_cast<const float *>(part_p),
        static_cast<const int32_t *>(part_c), static_cast<int>(G), Ei, static_cast<float>(k), c));
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
    const bool vec = E % 8 == 0 && logits_stride % 8 == 0 && aligned(r[0].dev, 8 * size) &&
                     aligned(r[2].dev, 8 * size);
    return with_type(dtype, [&](auto t) {
        return with_lanes(E, vec, [&](auto l, auto v, auto n) {
            using Elem = decltype(t);
            // up to 4 CTAs per SM, as the registers of 16 logits per lane allow, or 8
            // (60000 x 60 fp32 11.3 us against 13.0 with 4), all with the same number of
            // rounds
            const int64_t rounds = ceil_div64(T, kThreads / l());
            const int64_t most = device_sm_count() * (v() * n() > 8 ? 4 : 8);
            const int64_t grid = ceil_div64(rounds, ceil_div64(rounds, most));
            return launched(launch_kernel(
                balance_backward<Elem, l(), v(), n()>, dim3(static_cast<unsigned>(grid)),
                dim3(kThreads), 0, stream, 1, as<Elem>(r[0]), as<const float>(r[1]),
                as<const Elem>(r[2]), as<const int32_t>(r[3]), as<const int32_t>(r[4]),
                as<const uint8_t>(r[5]), T, static_cast<int>(E), static_cast<float>(k),
                logits_stride, static_cast<float>(coef)));
        });
    });
}
