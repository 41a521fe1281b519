// gelu_and_mul_sparse for sm_103a: Gemma3n's sparse GELU gate, fused into one
// pass over HBM.
//
// Definition (vLLM PR "[Performance] Add Triton kernel for Gemma3n sparse
// GELU", section "Purpose", which lists the fused stages: row statistics, a
// threshold derived from them, the tanh form of GELU and the product with the
// up half), per row with gate g = [0, d), up u = [d, 2d):
//   mean = sum g / d,  std = sqrt(sum (g - mean)^2 / d),  cutoff = mean + std z,
//   out  = gelu_tanh(max(g - cutoff, 0)) * u,  fp32 math, one bf16 rounding.
//
// Every geometry reads each input element from HBM exactly once and keeps the
// row on chip between the statistics and the epilogue:
//   * tma rows    -- persistent CTAs; each streams its rows' gate and up halves
//                    through a ring of shared-memory slots with 1-D bulk copies
//                    (cp.async.bulk, completion on mbarriers), so HBM keeps
//                    streaming while earlier rows are reduced and written.
//                    Rows go round-robin, or, given a workspace, to whichever
//                    CTA takes the next ticket of an atomic counter;
//   * pipe rows   -- as tma rows, warp-specialised: one lane of a producer
//                    warp issues every copy and takes every ticket, the other
//                    warps finish rows; full/empty mbarriers per slot.  With
//                    tickets, the last wave of the widest rows runs as half
//                    jobs that both copy the row's gate half (the second
//                    copy is normally still in L2) and split its columns;
//   * warp rows   -- one warp per row, shuffles only (d <= 2048);
//   * CTA row     -- one CTA per row, or a cluster of C CTAs per row, each CTA
//                    holding a column slice in registers; in a cluster every
//                    warp's partials (count, sum, M2) are exchanged through
//                    distributed shared memory and combined with the
//                    parallel form of the variance of Chan, Golub and
//                    LeVeque (1979), M2 = sum M2_p + sum n_p (mean_p -
//                    mean)^2, so one cluster barrier serves mean and variance;
//   * scalar      -- any alignment or width: 2-byte loads, gate re-read from
//                    L1/L2 for each pass.
// The fp32 arithmetic uses Blackwell's paired-lane instructions (add/sub/mul/
// fma .f32x2), one instruction per two elements.
#include <algorithm>
#include <mutex>

#include <cuda.h>

#include "common.cuh"
#include "gated_act_testing.h"

namespace gact {

// Device status word of this library (bit 0: a bounded wait for a bulk copy
// gave up).  Read and cleared by gated_act_device_status().
__device__ unsigned int g_device_status;

namespace {

constexpr float kSqrt2OverPi = 0.7978845608028654f;        // sqrt(2/pi)
constexpr float kCubicCoef = 0.7978845608028654f * 0.044715f;

constexpr int kWarpRowsThreads = 128;      // 4 rows per CTA in the warp-rows geometry
constexpr int kMaxCluster = 8;             // portable cluster size
constexpr int kMaxSliceVec = 4096;         // 16-byte gate vectors one CTA can hold (1024 x 4)
constexpr int kMinSliceVec = 256;          // slices up to this use 2 vectors per thread
constexpr int kFewRows = 8;                // the "few rows" unit of the cluster rules
constexpr int kScalarThreads = 256;

constexpr int kTmaMaxStages = 8;
constexpr int kTmaSmemPerSm = 228 * 1024;  // shared memory of one SM (1 KB per CTA is reserved)
constexpr int kTmaSmemPerCta = 227 * 1024; // largest opt-in shared memory of one CTA
constexpr unsigned long long kWaitLimitNs = 1000000000ull;   // 1 s bound on every mbarrier wait
// With a workspace, the bulk-copy geometry hands rows out dynamically from
// this many rows per CTA on (measured on GB300: below it the static
// round-robin is as fast, since a CTA takes its next row about one row ahead
// of need and the last claims can then leave one CTA a row behind).
constexpr int64_t kDynamicRowsPerCta = 6;
constexpr size_t kWorkspaceBytes = 16;   // a 64-bit row-ticket counter and 8 reserved bytes

// max(x, 0) that returns NaN for a NaN input (fmaxf would return 0).
__device__ __forceinline__ float relu_nan(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
// bf16x2 word -> (low element, high element) as fp32
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// tanh via the hardware approximation (PTX ISA tanh.approx.f32, maximum
// relative error about 2^-11).  In gelu_tanh the argument is never negative,
// so 1 + tanh lies in [1, 2] and its relative error stays below 2^-12.
__device__ __forceinline__ float tanh_approx(float x) {
    float y;
    asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// gelu_tanh(s) = 0.5 s (1 + tanh(y)) = s / (1 + e^{-2y}) for fp32 outputs,
// y >= 0: e^{-2y} in (0, 1] from the flushing hardware exponential (PTX ISA
// ex2.approx.ftz.f32, relative error about 2^-22; below 2^-126, past y = 43.7,
// it flushes to 0 and the result is s, the exact limit), 1 + e^{-2y} in (1, 2]
// inverted by the flushing hardware reciprocal (rcp.approx.ftz.f32, within
// one ulp there).  Relative error about 2^-21, with no cancellation since
// nothing is subtracted.
__device__ __forceinline__ float gelu_exp_form(float s, float y) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * (-2.0f * 1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return s * r;
}

// ------------------------------------------------------------ element formats
// A 16-byte vector holds kPairs pairs of elements: pair(v, i) reads pair i as
// fp32, put_pair writes pair i rounded to the format (nearest even).
// gelu_a(s, y, h) is gelu_tanh(s) for a pair (y = sqrt(2/pi)(s + 0.044715 s^3),
// h = s/2): h + h tanh(y) on the hardware tanh for the 16-bit formats (its
// 2^-12 relative error in 1 + tanh is below their rounding), the exponential
// form above for fp32 outputs.
struct FmtBf16 {
    static constexpr int kElem = 2, kPairs = 4, kLut = 0;   // kLut: native table index
    __device__ static float2 pair(const uint4 &v, int i) { return unpack2((&v.x)[i]); }
    __device__ static void put_pair(uint4 &v, int i, float2 f) {
        (&v.x)[i] = pack_bf16x2(f.x, f.y);
    }
    __device__ static float2 gelu_a(float2 s, float2 y, float2 h) {
        return fma2(h, make_float2(tanh_approx(y.x), tanh_approx(y.y)), h);
    }
    __device__ static float load1(const uint8_t *p) {
        return __uint_as_float(static_cast<uint32_t>(ld_stream_u16(reinterpret_cast<const uint16_t *>(p))) << 16);
    }
    __device__ static void store1(uint8_t *p, float f) {
        *reinterpret_cast<uint16_t *>(p) = __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
};

struct FmtF16 {
    static constexpr int kElem = 2, kPairs = 4, kLut = 1;
    __device__ static float2 pair(const uint4 &v, int i) {
        const uint32_t w = (&v.x)[i];
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ static void put_pair(uint4 &v, int i, float2 f) {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        (&v.x)[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static float2 gelu_a(float2 s, float2 y, float2 h) {
        return fma2(h, make_float2(tanh_approx(y.x), tanh_approx(y.y)), h);
    }
    __device__ static float load1(const uint8_t *p) {
        return __half2float(__ushort_as_half(ld_stream_u16(reinterpret_cast<const uint16_t *>(p))));
    }
    __device__ static void store1(uint8_t *p, float f) {
        *reinterpret_cast<uint16_t *>(p) = __half_as_ushort(__float2half_rn(f));
    }
};

struct FmtF32 {
    static constexpr int kElem = 4, kPairs = 2;   // no native mode, so no kLut
    __device__ static float2 pair(const uint4 &v, int i) {
        return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static void put_pair(uint4 &v, int i, float2 f) {
        if (i == 0) {
            v.x = __float_as_uint(f.x);
            v.y = __float_as_uint(f.y);
        } else {
            v.z = __float_as_uint(f.x);
            v.w = __float_as_uint(f.y);
        }
    }
    __device__ static float2 gelu_a(float2 s, float2 y, float2) {
        return make_float2(gelu_exp_form(s.x, y.x), gelu_exp_form(s.y, y.y));
    }
    __device__ static float load1(const uint8_t *p) {
        return __uint_as_float(ld_stream_u32(reinterpret_cast<const uint32_t *>(p)));
    }
    __device__ static void store1(uint8_t *p, float f) { *reinterpret_cast<float *>(p) = f; }
};

// gelu_tanh(max(g - cutoff, 0)) * u for every element of one 16-byte vector.
template <class F>
__device__ __forceinline__ uint4 epi_vec(const uint4 &g, const uint4 &u, float cutoff) {
    const float2 c2 = make_float2(cutoff, cutoff);
    uint4 o;
#pragma unroll
    for (int i = 0; i < F::kPairs; ++i) {
        float2 s = sub2(F::pair(g, i), c2);
        s.x = relu_nan(s.x);
        s.y = relu_nan(s.y);
        const float2 y = mul2(s, fma2(mul2(s, s), make_float2(kCubicCoef, kCubicCoef),
                                      make_float2(kSqrt2OverPi, kSqrt2OverPi)));
        const float2 h = mul2(s, make_float2(0.5f, 0.5f));
        const float2 a = F::gelu_a(s, y, h);
        F::put_pair(o, i, mul2(a, F::pair(u, i)));
    }
    return o;
}

// Round an fp32 value to the format and back (nearest even).
template <class F> __device__ __forceinline__ float round_t(float x);
template <> __device__ __forceinline__ float round_t<FmtBf16>(float x) {
    return __bfloat162float(__float2bfloat16_rn(x));
}
template <> __device__ __forceinline__ float round_t<FmtF16>(float x) {
    return __half2float(__float2half_rn(x));
}
template <> __device__ __forceinline__ float round_t<FmtF32>(float x) { return x; }

// Native-rounding epilogue: each op of the composition computed in fp32 and
// rounded to the format -- s = R(g - c), relu, a = R(gelu_tanh(s)), out =
// R(a * u).  gelu_tanh follows the op order of PyTorch's own tanh-GELU kernel
// (the composition this mode reproduces): x3 = (s s) s, inner = sqrt(2/pi)
// fma(0.044715, x3, s), a = (0.5 s)(1 + tanh(inner)), with the accurate
// tanhf.  a depends only on the 16-bit pattern of s.
template <class F>
__device__ __forceinline__ float native_a(float s) {
    const float x3 = __fmul_rn(__fmul_rn(s, s), s);
    const float inner = __fmul_rn(kSqrt2OverPi, fmaf(0.044715f, x3, s));
    return round_t<F>(__fmul_rn(__fmul_rn(0.5f, s), __fadd_rn(1.0f, tanhf(inner))));
}

template <class F>
__device__ __forceinline__ float native_gelu_mul(float g, float u, float c) {
    return native_a<F>(relu_nan(round_t<F>(g - c))) * u;   // rounded by the caller's store
}

// a = R(gelu_tanh(s)) for every non-negative 16-bit pattern of s, one table
// per format (64 KB each: [0] bf16, [1] fp16), built once per device by the
// first native launch that finds it missing (its CTA 0, after which it sets
// the ready word with release semantics) and read through the read-only cache
// by later launches.  Entries come from native_a, so a launch that computes a
// directly (its table not ready yet) gives the same bits.
__device__ __align__(16) uint16_t g_native_lut[2][32768];
__device__ unsigned int g_native_lut_ready[2];

template <class F> __device__ __forceinline__ float from_bits(uint32_t p);
template <> __device__ __forceinline__ float from_bits<FmtBf16>(uint32_t p) {
    return __uint_as_float(p << 16);
}
template <> __device__ __forceinline__ float from_bits<FmtF16>(uint32_t p) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(p)));
}
template <class F> __device__ __forceinline__ uint32_t to_bits(float x);
template <> __device__ __forceinline__ uint32_t to_bits<FmtBf16>(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <> __device__ __forceinline__ uint32_t to_bits<FmtF16>(float x) {
    return __half_as_ushort(__float2half_rn(x));
}

// R(x.x), R(x.y) packed as the format's 16-bit pair (low element first), and
// max(pair, 0) on it with NaN kept (the relu of the composition).
template <class F> __device__ __forceinline__ uint32_t round_pair(float2 x);
template <> __device__ __forceinline__ uint32_t round_pair<FmtBf16>(float2 x) {
    return pack_bf16x2(x.x, x.y);
}
template <> __device__ __forceinline__ uint32_t round_pair<FmtF16>(float2 x) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <class F> __device__ __forceinline__ uint32_t relu_pair(uint32_t w);
template <> __device__ __forceinline__ uint32_t relu_pair<FmtBf16>(uint32_t w) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0u));
    return r;
}
template <> __device__ __forceinline__ uint32_t relu_pair<FmtF16>(uint32_t w) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0u));
    return r;
}

// Packed products of a format's pairs, each correctly rounded (nearest even).
template <class F> __device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t mul_pair<FmtBf16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t mul_pair<FmtF16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The table of format F, or nullptr while this launch must compute a directly.
// CTA 0 of a launch that finds the table missing builds it (every thread a
// strided share), fences, and publishes it; it still computes directly itself,
// since the read-only cache must not serve data written in the same launch.
// The ready word is read relaxed, not with acquire: the table is written once,
// every writer fences, and the word is published with a release store after
// that; a reader issues its table reads (read-only path) only after the word's
// value has decided its branch, and no SM holds earlier copies of table lines
// (nothing reads the table before it is published).  An acquire at GPU scope
// would also invalidate the SM's L1 at every CTA start, evicting the table's
// hot lines: measured on GB300, 1.5% slower at 2048 x 16384.
template <class F>
__device__ const uint16_t *native_table() {
    __shared__ unsigned int ready;
    constexpr int k = F::kLut;
    if (threadIdx.x == 0) {
        unsigned int v;
        asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(&g_native_lut_ready[k])
                     : "memory");
        ready = v;
    }
    __syncthreads();
    const unsigned int ok = ready;
    if (ok)
        return g_native_lut[k];
    if (blockIdx.x == 0) {
        for (uint32_t p = threadIdx.x; p < 32768u; p += blockDim.x)
            g_native_lut[k][p] = static_cast<uint16_t>(to_bits<F>(native_a<F>(from_bits<F>(p))));
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(&g_native_lut_ready[k]), "r"(1u)
                         : "memory");
    }
    return nullptr;
}

// One 16-byte vector of the native epilogue.  With the table: R(g - c) of a
// pair in one conversion, the relu on the packed pair, two table reads, and
// R(a u) at the store; without: native_gelu_mul per element.
template <class F>
__device__ __forceinline__ uint4 epi_vec_native(const uint4 &g, const uint4 &u, float cutoff,
                                                const uint16_t *__restrict__ lut) {
    uint4 o;
    if (lut) {
        const float2 c2 = make_float2(cutoff, cutoff);
#pragma unroll
        for (int i = 0; i < F::kPairs; ++i) {
            // after the relu both sign bits are clear, so the high index is s >> 16
            const uint32_t s = relu_pair<F>(round_pair<F>(sub2(F::pair(g, i), c2)));
            const uint32_t a = static_cast<uint32_t>(__ldg(lut + (s & 0x7FFFu))) |
                               (static_cast<uint32_t>(__ldg(lut + (s >> 16))) << 16);
            // R(a u): the product of two 16-bit values is exact in fp32, so
            // rounding it once is the packed multiply's own rounding
            (&o.x)[i] = mul_pair<F>(a, (&u.x)[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < F::kPairs; ++i) {
            const float2 gp = F::pair(g, i), up = F::pair(u, i);
            F::put_pair(o, i, make_float2(native_gelu_mul<F>(gp.x, up.x, cutoff),
                                          native_gelu_mul<F>(gp.y, up.y, cutoff)));
        }
    }
    return o;
}

// The native composition's cutoff from the fp32 row statistics:
// c = R(R(mean) + R(R(std) * z)).
template <class F>
__device__ __forceinline__ float native_cutoff(float mean, float var, float z) {
    const float m = round_t<F>(mean);
    const float sd = round_t<F>(__fsqrt_rn(var));
    return round_t<F>(m + round_t<F>(sd * z));
}

// Running pair sums over one vector of gate values.
template <class F>
__device__ __forceinline__ float2 sum_vec(float2 acc, const uint4 &g) {
#pragma unroll
    for (int i = 0; i < F::kPairs; ++i)
        acc = add2(acc, F::pair(g, i));
    return acc;
}
template <class F>
__device__ __forceinline__ float2 ssd_vec(float2 acc, const uint4 &g, float2 m2) {
#pragma unroll
    for (int i = 0; i < F::kPairs; ++i) {
        const float2 e = sub2(F::pair(g, i), m2);
        acc = fma2(e, e, acc);
    }
    return acc;
}

// CTA-wide sum; every thread returns the same bits.  NARROW: every lane
// takes the partial of warp (lane mod NW), and a butterfly over NW lanes
// leaves the total in all 32 lanes (log2 NW shuffles instead of 5).
// Measured on GB300: 1-6% faster for CTAs of two vectors per thread
// (decode rows), 2-7% slower for four-vector CTAs, which keep the full tree.
template <int NW, bool NARROW = false>
__device__ __forceinline__ float block_sum(float v, float *red, int lane, int warp) {
    static_assert(NW >= 1 && NW <= 32 && (NW & (NW - 1)) == 0, "warps per CTA: a power of two");
    v = warp_sum(v);
    if (NW == 1)
        return v;
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    if constexpr (NARROW) {
        float t = red[lane & (NW - 1)];
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1)
            t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        return t;
    } else {
        return warp_sum(lane < NW ? red[lane] : 0.f);
    }
}

// ------------------------------------------------------------ cluster helpers
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// Arrive without release: for a CTA whose only claim is that its own reads
// of its peers' shared memory are done (their values already consumed).
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Load a float from the same shared-memory variable in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_peer(const float *local, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}

// ------------------------------------------------------------ mbarrier + bulk copy
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// An arrive with no transaction bytes: completes the phase of a count-1 barrier.
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 1-D bulk copy global -> this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long globaltimer_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Wait for the phase `parity` of `bar`, giving up after limit_ns.
__device__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    if (mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 255u) == 0 && globaltimer_ns() - t0 > limit_ns)
            return false;
    }
}

// ------------------------------------------------------------ tma rows
// Persistent CTAs.  Each CTA's j-th row contributes chunk 2j (gate, 2d bytes)
// and chunk 2j+1 (up); chunk c lands in slot c mod S, guarded by mbarrier
// c mod S at phase parity (c / S) mod 2.  Thread 0 picks a CTA's rows as it
// issues their gate chunks and records each in slot_row[] beside the data:
//   * static  (sched == nullptr): rows b, b + G, b + 2G, ... (G = gridDim.x);
//   * dynamic (sched = a zeroed workspace): row b first, then G + the next
//     ticket of the counter sched[0], so SMs that stream faster take more
//     rows and the launch ends evenly;
// a row >= T ends the CTA: thread 0 completes that slot's phase with a plain
// arrive and slot_row = -1 tells every thread to stop.  Thread 0 refills a
// slot once every thread is past the barrier that follows the slot's last
// read: at the first CTA barrier of row j, chunks up to 2j are consumed (gate
// j is in registers, up j-1 was consumed by row j-1's epilogue), so chunks
// up to 2j + S may be in flight.  Thread 0 takes row j + 1's ticket at that
// barrier and issues its copies after the second one, so the atomic's round
// trip overlaps the variance reduction.
// Dynamic mode resets its own counter with no exit protocol: every CTA stops
// at its first failing ticket (G + t >= T), so a launch hands out exactly T
// tickets, T - G of them rows and G of them stops, and the CTA that draws
// ticket T - 1 is the last one to touch the counter; it sets it back to zero.
// withhold >= 0 (failure-handling tests only): every CTA skips issuing its
// chunk number `withhold`, so the wait for it runs out after wait_ns.
template <int NT, int V>
__global__ void __launch_bounds__(NT, (1024 / NT) > 0 ? (1024 / NT) : 1)
gelu_tma_rows(uint16_t *__restrict__ out, const uint16_t *__restrict__ in, int64_t T, int d,
              int64_t rs, float z, int S, unsigned long long *__restrict__ sched,
              int64_t withhold, unsigned long long wait_ns) {
    constexpr int NW = NT / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][NW];
    __shared__ int64_t slot_row[kTmaMaxStages];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t chunk = 2u * static_cast<uint32_t>(d);
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + static_cast<uint32_t>(S) * chunk;
    const int64_t G = gridDim.x;
    const int nvec = d >> 3;

    if (tid == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(bars + 8u * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // Ring positions advance one chunk at a time (slot = c mod S, parity =
    // (c / S) mod 2), kept as counters instead of divisions.
    const uint32_t nslots = static_cast<uint32_t>(S);
    int64_t issued = 0;     // thread 0: next chunk to issue ...
    uint32_t islot = 0;     // ... and its slot
    int64_t claimed = 0;    // thread 0: rows taken so far ...
    int64_t row_i = 0;      // ... the last of them ...
    bool more = true;       // ... and whether another may follow
    // thread 0, dynamic mode: a ticket taken ahead of the copy that needs it
    // (kNoTicket: none)
    constexpr unsigned long long kNoTicket = ~0ull;
    unsigned long long ticket = kNoTicket;
    // Dynamic mode: the ticket that stops this CTA is the launch's last one
    // (T - 1) for exactly one CTA, which sets the counter back to zero.
    auto stop_ticket = [&](int64_t r) {
        if (sched && r == G + T - 1)
            asm volatile("red.relaxed.gpu.global.and.b64 [%0], %1;" ::"l"(sched), "l"(0ull)
                         : "memory");
    };
    auto take_ticket = [&]() {
        if (tid == 0 && sched && more && claimed > 0 && ticket == kNoTicket)
            ticket = atomicAdd(sched, 1ull);
    };
    auto issue_upto = [&](int64_t last) {
        if (tid != 0)
            return;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (; more && issued <= last; ++issued) {
            const uint32_t slot = islot;
            islot = islot + 1 == nslots ? 0u : islot + 1;
            if ((issued & 1) == 0) {   // a gate chunk: the CTA's next row
                if (claimed == 0) {
                    row_i = static_cast<int64_t>(blockIdx.x);
                } else if (sched) {
                    take_ticket();
                    row_i = G + static_cast<int64_t>(ticket);
                    ticket = kNoTicket;
                } else {
                    row_i = static_cast<int64_t>(blockIdx.x) + claimed * G;
                }
                ++claimed;
                if (row_i >= T) {
                    slot_row[slot] = -1;
                    mbar_arrive(bars + 8u * slot);
                    more = false;
                    stop_ticket(row_i);
                    continue;
                }
                slot_row[slot] = row_i;
            }
            if (issued == withhold)
                continue;
            const uint16_t *src = in + row_i * rs + ((issued & 1) ? d : 0);
            mbar_expect_tx(bars + 8u * slot, chunk);
            bulk_load(base + slot * chunk, src, chunk, bars + 8u * slot);
        }
    };
    issue_upto(S - 1);

    bool bad = false;
    uint32_t cslot = 0, cpar = 0;   // every thread: the next chunk to consume
    auto consume = [&](uint32_t *slot, uint32_t *par) {
        *slot = cslot;
        *par = cpar;
        if (++cslot == nslots) {
            cslot = 0;
            cpar ^= 1u;
        }
    };
    int64_t k = 0;
    for (;; ++k) {
        const int64_t cg = 2 * k;
        uint32_t sg, pg, su, pu;
        consume(&sg, &pg);
        consume(&su, &pu);
        bad |= !mbar_wait(bars + 8u * sg, pg, wait_ns);
        const int64_t row = slot_row[sg];

        const uint4 *gs = reinterpret_cast<const uint4 *>(smem + static_cast<size_t>(sg) * chunk);
        uint4 g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + NT * i;
            g[i] = v < nvec ? gs[v] : make_uint4(0u, 0u, 0u, 0u);
        }
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc = sum_vec<FmtBf16>(acc, g[i]);
        float s = warp_sum(acc.x + acc.y);
        if (lane == 0)
            red[0][warp] = s;
        // Both exits are CTA-uniform: the vote, and the end mark that every
        // thread read after the same completed phase.
        if (__syncthreads_or(bad) || row < 0)
            break;
        s = warp_sum(lane < NW ? red[0][lane] : 0.f);
        take_ticket();   // its round trip overlaps the variance reduction

        const float mean = __fdiv_rn(s, static_cast<float>(d));
        const float2 m2 = make_float2(mean, mean);
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + NT * i < nvec)
                acc = ssd_vec<FmtBf16>(acc, g[i], m2);
        const float q = block_sum<NW>(acc.x + acc.y, red[1], lane, warp);
        issue_upto(cg + S);
        const float sd = __fsqrt_rn(__fdiv_rn(q, static_cast<float>(d)));
        const float cutoff = fmaf(sd, z, mean);

        bad |= !mbar_wait(bars + 8u * su, pu, wait_ns);
        if (!bad) {
            const uint4 *us = reinterpret_cast<const uint4 *>(smem + static_cast<size_t>(su) * chunk);
            uint16_t *op = out + row * static_cast<int64_t>(d);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + NT * i;
                if (v < nvec)
                    st_vec(op + 8 * v, epi_vec<FmtBf16>(g[i], us[v], cutoff));
            }
        }
    }
    // Every thread reaches this vote.  If a wait gave up, record it and let
    // thread 0 wait, bounded again, for every copy it issued that was not
    // consumed (from the up half of the row before the one in progress), so
    // none is in flight when the CTA exits.
    if (__syncthreads_or(bad) && tid == 0) {
        atomicOr(&g_device_status, 1u);
        for (int64_t c = k > 0 ? 2 * k - 1 : 0; c < issued; ++c)
            mbar_wait(bars + 8u * static_cast<uint32_t>(c % S),
                      static_cast<uint32_t>((c / S) & 1), wait_ns);
    }
    // Dynamic mode, a CTA that stopped before its failing ticket (it gave
    // up): it draws tickets until one fails, so the launch still hands out
    // exactly T and the counter is reset by whichever CTA draws T - 1.
    if (sched && tid == 0 && more) {
        int64_t r = ticket != kNoTicket ? G + static_cast<int64_t>(ticket) : -1;
        while (r < T)
            r = G + static_cast<int64_t>(atomicAdd(sched, 1ull));
        stop_ticket(r);
    }
}

// ------------------------------------------------------------ pipe rows
// Persistent CTAs with one producer lane and NCW consumer warps.  The
// consumers hold a row's gate in registers (V 16-byte vectors per thread)
// and finish the row; lane 0 of the last warp streams gate and up half-rows
// into a ring of S shared-memory slots with bulk copies and picks the CTA's
// rows (round-robin, or tickets from the workspace counter as in tma rows).
// Slot s has a "full" mbarrier (the producer's arrive plus the copy's bytes)
// and an "empty" one (one arrive per consumer warp once the slot has been
// read), so copy issue and ticket round trips run beside the consumers, who
// synchronise among themselves with a named barrier only.  Chunk c (gate of
// the CTA's job c/2 for even c, up for odd c) uses slot c mod S.
// A job is a row, or with dynamic rows one half of one of the last `split`
// rows: its CTA reads the whole gate half-row (the statistics need it; both
// halves compute the same bits) but only its half of the up half-row, and
// writes that half of the output row.  Splitting the last wave of rows
// halves the epilogue that ends the launch on the SMs that finish last.
// Failure handling: every wait is bounded.  Consumers that give up vote to
// stop together and leave their slots unreleased; the producer notices
// (cons_done), stops issuing, and waits (bounded) for its own copies in
// flight -- the latest use of each slot -- before it exits.
template <int NCW>
__device__ __forceinline__ void cons_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory");
}
template <int NCW>
__device__ __forceinline__ bool cons_sync_or(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, %2, q;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "n"(NCW * 32)
        : "memory");
    return r != 0;
}
template <int NCW>
__device__ __forceinline__ float cons_sum(float v, float *red, int lane, int warp) {
    v = warp_sum(v);
    if (lane == 0)
        red[warp] = v;
    cons_sync<NCW>();
    return warp_sum(lane < NCW ? red[lane] : 0.f);
}

constexpr int kPipeMaxStages = 16;
// Half jobs for the last rows of a pipe-rows launch with dynamic rows: one
// row per CTA, from 3 rows per CTA at d >= 32768.  Measured on GB300 at
// d = 32768: 1024 rows 32.66 -> 32.34 us, 2048 rows 60.67 -> 59.77, 4096
// rows 115.86 -> 114.65; splitting half or a quarter as many rows gained
// nothing; at 256 and 384 rows, and at d = 16384 and 20480, splitting lost
// 2-6% (the second read of the gate half-row costs more than it saves).
constexpr int64_t kPipeSplitDiv = 1;           // split rows: grid / this
constexpr int64_t kPipeSplitMinVec = 4096;
constexpr int64_t kPipeSplitMinRowsPerCta = 3;

template <int NCW, int V>
__global__ void __launch_bounds__((NCW + 1) * 32, (NCW >= 16 ? 1 : NCW >= 8 ? 2 : 4))
gelu_pipe_rows(uint16_t *__restrict__ out, const uint16_t *__restrict__ in, int64_t T, int d,
               int64_t rs, float z, int S, unsigned long long *__restrict__ sched, int64_t split,
               int64_t withhold, unsigned long long wait_ns) {
    constexpr int NC = NCW * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][NCW];
    __shared__ int cons_done;   // consumers have left their loop

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t chunk = 2u * static_cast<uint32_t>(d);
    const uint32_t base = smem_addr(smem);
    const uint32_t full = base + static_cast<uint32_t>(S) * chunk;
    const uint32_t empty = full + 8u * static_cast<uint32_t>(S);
    int64_t *slot_row = reinterpret_cast<int64_t *>(smem + static_cast<size_t>(S) * chunk +
                                                    16u * static_cast<uint32_t>(S));
    const uint32_t nslots = static_cast<uint32_t>(S);
    const int nvec = d >> 3;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8u * s, 1);
            mbar_init(empty + 8u * s, NCW);
        }
        cons_done = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    if (warp == NCW) {
        // ---------------- producer (one lane)
        if (lane != 0)
            return;
        const int64_t G = gridDim.x;
        volatile int *done = &cons_done;
        // the consumers' release of a slot, or false once they have stopped
        // (or after a limit well past theirs)
        auto wait_empty = [&](uint32_t bar, uint32_t par) -> bool {
            if (mbar_try_wait(bar, par))
                return true;
            const unsigned long long t0 = globaltimer_ns();
            for (uint32_t i = 1;; ++i) {
                if (mbar_try_wait(bar, par))
                    return true;
                if ((i & 63u) == 0 && (*done || globaltimer_ns() - t0 > 3 * wait_ns))
                    return false;
            }
        };
        // jobs: rows 0 .. T - split - 1 whole, then each of the last `split`
        // rows as two half jobs (both CTAs read the whole gate half-row for
        // the statistics; each reads, computes and writes half of the up
        // and output columns)
        const int64_t J = T + split, whole = T - split;
        int64_t c = 0, row = 0, claimed = 0;
        int half = -1;   // -1: the whole row, else which half of it
        uint32_t slot = 0, round = 0;
        bool ended = false, bad = false;
        for (;; ++c) {
            if (round > 0 && !wait_empty(empty + 8u * slot, (round - 1) & 1u)) {
                bad = true;
                break;
            }
            if ((c & 1) == 0) {   // a gate chunk: the CTA's next job
                const int64_t j = claimed == 0 ? static_cast<int64_t>(blockIdx.x)
                                  : sched      ? G + static_cast<int64_t>(atomicAdd(sched, 1ull))
                                               : static_cast<int64_t>(blockIdx.x) + claimed * G;
                ++claimed;
                if (j >= J) {
                    slot_row[slot] = -1;
                    mbar_arrive(full + 8u * slot);
                    if (sched && j == G + J - 1)   // ticket J - 1: reset the counter
                        asm volatile("red.relaxed.gpu.global.and.b64 [%0], %1;" ::"l"(sched),
                                     "l"(0ull)
                                     : "memory");
                    ended = true;
                    break;
                }
                row = j < whole ? j : whole + ((j - whole) >> 1);
                half = j < whole ? -1 : static_cast<int>((j - whole) & 1);
                slot_row[slot] = 4 * row + (half + 1);
            }
            if (c != withhold) {
                // an up chunk of a half job: d bytes (half the up half-row)
                const uint32_t bytes = ((c & 1) && half >= 0) ? chunk / 2 : chunk;
                const int64_t col = (c & 1) ? d + (half > 0 ? d / 2 : 0) : 0;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_expect_tx(full + 8u * slot, bytes);
                bulk_load(base + slot * chunk, in + row * rs + col, bytes, full + 8u * slot);
            }
            if (++slot == nslots) {
                slot = 0;
                ++round;
            }
        }
        // No copy may be in flight when the CTA exits: wait for the latest
        // copy into each slot (chunks c - S .. c - 1; after a normal end,
        // chunk c - S was released before the end mark took its slot).
        for (int64_t x = c - S + (ended ? 1 : 0); x < c; ++x)
            if (x >= 0 && x != withhold)
                bad |= !mbar_wait(full + 8u * static_cast<uint32_t>(x % S),
                                  static_cast<uint32_t>((x / S) & 1), wait_ns);
        if (bad)
            atomicOr(&g_device_status, 1u);
        // dynamic rows, stopped early: draw tickets until the first failing
        // one, so the launch hands out exactly T and one CTA resets the counter
        if (sched && !ended) {
            int64_t r = -1;
            while (r < J)
                r = G + static_cast<int64_t>(atomicAdd(sched, 1ull));
            if (r == G + J - 1)
                asm volatile("red.relaxed.gpu.global.and.b64 [%0], %1;" ::"l"(sched), "l"(0ull)
                             : "memory");
        }
        return;
    }

    // ---------------- consumers
    bool bad = false;
    uint32_t cslot = 0, cpar = 0;
    auto next = [&](uint32_t *s, uint32_t *p) {
        *s = cslot;
        *p = cpar;
        if (++cslot == nslots) {
            cslot = 0;
            cpar ^= 1u;
        }
    };
    for (;;) {
        uint32_t sg, pg, su, pu;
        next(&sg, &pg);
        next(&su, &pu);
        bad |= !mbar_wait(full + 8u * sg, pg, wait_ns);
        const int64_t tag = slot_row[sg];   // 4 row + (half + 1), or -1 at the end
        const uint4 *gs = reinterpret_cast<const uint4 *>(smem + static_cast<size_t>(sg) * chunk);
        uint4 g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + NC * i;
            g[i] = v < nvec ? gs[v] : make_uint4(0u, 0u, 0u, 0u);
        }
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc = sum_vec<FmtBf16>(acc, g[i]);
        float s = warp_sum(acc.x + acc.y);
        if (lane == 0)
            red[0][warp] = s;
        // both exits are uniform over the consumers: the vote, and the end
        // mark every consumer read after the same completed phase
        if (cons_sync_or<NCW>(bad) || tag < 0)
            break;
        const int64_t row = tag >> 2;
        const int half = static_cast<int>(tag & 3) - 1;
        if (lane == 0)
            mbar_arrive(empty + 8u * sg);   // the gate half-row is in registers
        s = warp_sum(lane < NCW ? red[0][lane] : 0.f);

        const float mean = __fdiv_rn(s, static_cast<float>(d));
        const float2 m2 = make_float2(mean, mean);
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + NC * i < nvec)
                acc = ssd_vec<FmtBf16>(acc, g[i], m2);
        const float q = cons_sum<NCW>(acc.x + acc.y, red[1], lane, warp);
        const float sd = __fsqrt_rn(__fdiv_rn(q, static_cast<float>(d)));
        const float cutoff = fmaf(sd, z, mean);

        bad |= !mbar_wait(full + 8u * su, pu, wait_ns);
        if (!bad) {
            const uint4 *us = reinterpret_cast<const uint4 *>(smem + static_cast<size_t>(su) * chunk);
            uint16_t *op = out + row * static_cast<int64_t>(d);
            // the columns of this job: all, or one half (nvec is even then)
            const int vlo = half > 0 ? nvec >> 1 : 0;
            const int vhi = half == 0 ? nvec >> 1 : nvec;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + NC * i;
                if (v >= vlo && v < vhi)
                    st_vec(op + 8 * v, epi_vec<FmtBf16>(g[i], us[v - vlo], cutoff));
            }
        }
        // a warp that missed the up half-row keeps its slot (its copy may
        // still land); the vote at the next row stops everyone
        if (!__any_sync(0xFFFFFFFFu, bad) && lane == 0)
            mbar_arrive(empty + 8u * su);
    }
    if (tid == 0) {
        if (bad)
            atomicOr(&g_device_status, 1u);
        *static_cast<volatile int *>(&cons_done) = 1;
    }
}

// ------------------------------------------------------------ warp rows
// One warp per row; lane l holds gate/up vectors l, l+32, ..., l+32(V-1).
template <int V>
__global__ void __launch_bounds__(kWarpRowsThreads, 4)
gelu_warp_rows(uint16_t *__restrict__ out, const uint16_t *__restrict__ in, int64_t T,
               int d, int64_t rs, float z) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kWarpRowsThreads / 32) +
                        (threadIdx.x >> 5);
    if (row >= T)
        return;
    pdl_wait();
    pdl_trigger();
    const int nvec = d >> 3;
    const uint16_t *gp = in + row * rs;
    const uint16_t *up = gp + d;

    uint4 g[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = lane + 32 * i;
        if (v < nvec) {
            g[i] = ld_stream(gp + 8 * v);
            u[i] = ld_stream(up + 8 * v);
        } else {
            g[i] = make_uint4(0u, 0u, 0u, 0u);   // +0 leaves the sum unchanged
            u[i] = g[i];
        }
    }
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc = sum_vec<FmtBf16>(acc, g[i]);
    const float mean = __fdiv_rn(warp_sum(acc.x + acc.y), static_cast<float>(d));
    const float2 m2 = make_float2(mean, mean);
    acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < nvec)
            acc = ssd_vec<FmtBf16>(acc, g[i], m2);
    const float q = warp_sum(acc.x + acc.y);
    const float sd = __fsqrt_rn(__fdiv_rn(q, static_cast<float>(d)));
    const float cutoff = fmaf(sd, z, mean);

    uint16_t *op = out + row * static_cast<int64_t>(d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = lane + 32 * i;
        if (v < nvec)
            st_vec(op + 8 * v, epi_vec<FmtBf16>(g[i], u[i], cutoff));
    }
}

// ------------------------------------------------------------ CTA / cluster rows
// A cluster of C CTAs (C = 1: a lone CTA) owns one row at a time; CTA k of
// the cluster holds gate/up vectors [k sv, min((k+1) sv, nvec)) of 16 bytes,
// thread t the vectors k sv + t + NT i.  Rows advance by the number of
// clusters in the grid.  CL = false: C must be 1 (no cluster code is
// compiled in).  F is the element format.
// NATIVE: the native-rounding composition (cutoff and epilogue rounded to the
// format after every op).
template <int NT, int V, bool CL, class F, bool NATIVE>
__global__ void __launch_bounds__(NT, (1024 / NT) > 0 ? (1024 / NT) : 1)
gelu_cta_rows(void *__restrict__ out_, const void *__restrict__ in_, int64_t T, int d,
              int64_t rs, float z, int C, int sv) {
    constexpr int NW = NT / 32;
    constexpr int kEpv = 16 / F::kElem;   // elements per 16-byte vector
    __shared__ float red[2][NW];
    __shared__ float xch[3];   // this CTA's (element count, sum, M2) for its peers
    // per-warp (element count, sum, M2) for the cluster, double-buffered by
    // row parity
    __shared__ float xw[2][3][NW];

    if (!CL)
        C = 1;
    const uint8_t *in = static_cast<const uint8_t *>(in_);
    uint8_t *out = static_cast<uint8_t *>(out_);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CL ? static_cast<int>(cluster_ctarank()) : 0;
    const int nvec = d / kEpv;
    const int v0 = rank * sv;
    const int v1 = min(nvec, v0 + sv);
    const int nk = max(v1 - v0, 0) * kEpv;
    const int64_t nclusters = gridDim.x / C;
    const int64_t rs_bytes = rs * F::kElem, d_bytes = static_cast<int64_t>(d) * F::kElem;
    pdl_wait();
    pdl_trigger();
    const uint16_t *lut = nullptr;   // native mode: the table of a, once built
    if constexpr (NATIVE)
        lut = native_table<F>();

    int it = 0;   // rows done by this CTA: the parity picks the exchange buffer
    for (int64_t row = blockIdx.x / C; row < T; row += nclusters, ++it) {
        const uint8_t *gp = in + row * rs_bytes;
        const uint8_t *up = gp + d_bytes;
        uint4 g[V], u[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = v0 + tid + NT * i;
            if (v < v1) {
                g[i] = ld_stream(gp + 16 * v);
                u[i] = ld_stream(up + 16 * v);
            } else {
                g[i] = make_uint4(0u, 0u, 0u, 0u);   // +0 in every format
                u[i] = g[i];
            }
        }
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc = sum_vec<F>(acc, g[i]);

        float mean, var;
        if constexpr (!NATIVE && CL) {
            // Two-pass statistics of each warp's elements in registers, then
            // one exchange of every warp's (count, sum, M2) across the cluster
            // through distributed shared memory, merged by every warp in the
            // same order: one cluster barrier per row and no CTA barrier.
            // (Measured on GB300: 7-11% faster for a few rows of d >= 16384;
            // without a cluster the same scheme was up to 14% slower than two
            // CTA-wide reductions, so lone CTAs keep those.)
            int cnt = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                cnt += (v0 + tid + NT * i < v1) ? 1 : 0;
            const float wn = static_cast<float>(__reduce_add_sync(0xFFFFFFFFu, cnt) * kEpv);
            const float ws = warp_sum(acc.x + acc.y);
            const float wm = wn > 0.f ? __fdiv_rn(ws, wn) : 0.f;
            const float2 m2 = make_float2(wm, wm);
            acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (v0 + tid + NT * i < v1)
                    acc = ssd_vec<F>(acc, g[i], m2);
            const float wq = warp_sum(acc.x + acc.y);
            float(&x)[3][NW] = xw[it & 1];
            if (lane == 0) {
                x[0][warp] = wn;
                x[1][warp] = ws;
                x[2][warp] = wq;
            }
            cluster_arrive_release();
            cluster_wait_acquire();
            // lane j takes partials j, j + 32, ... (partial p: CTA p / NW,
            // warp p % NW); M2 = sum_p M2_p + sum_p n_p (mean_p - mean)^2, each
            // sum a warp reduction over the lanes' shares.  Up to two partials
            // per lane stay in registers; more are read again after the mean.
            // (K: the most partials a lane can hold; when the cluster has at
            // most 32 partials, lane j's single one is also kept.)
            constexpr int K = (kMaxCluster * NW + 31) / 32;
            constexpr int KR = K <= 2 ? K : 1;                 // kept in registers
            const bool one = C * NW <= 32;
            float n_l[KR], s_l[KR], q_l[KR];
            float s_sum = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int p = lane + 32 * k;
                const bool keep = K <= 2 || k == 0;
                if (p < C * NW) {
                    const int c = p / NW, w = p - c * NW;
                    const float sp = ld_peer(&x[1][w], c);
                    if (keep) {
                        n_l[k < KR ? k : 0] = ld_peer(&x[0][w], c);
                        s_l[k < KR ? k : 0] = sp;
                        q_l[k < KR ? k : 0] = ld_peer(&x[2][w], c);
                    }
                    s_sum += sp;
                } else if (keep) {
                    n_l[k < KR ? k : 0] = s_l[k < KR ? k : 0] = q_l[k < KR ? k : 0] = 0.f;
                }
            }
            mean = __fdiv_rn(warp_sum(s_sum), static_cast<float>(d));
            float q_sum = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float np, sp, qp;
                if (K <= 2 || k == 0) {
                    np = n_l[k < KR ? k : 0];
                    sp = s_l[k < KR ? k : 0];
                    qp = q_l[k < KR ? k : 0];
                } else {
                    if (one)
                        break;   // every partial was lane j's first
                    const int p = lane + 32 * k;
                    np = sp = qp = 0.f;
                    if (p < C * NW) {
                        const int c = p / NW, w = p - c * NW;
                        np = ld_peer(&x[0][w], c);
                        sp = ld_peer(&x[1][w], c);
                        qp = ld_peer(&x[2][w], c);
                    }
                }
                if (np > 0.f) {
                    const float dm = __fdiv_rn(sp, np) - mean;
                    q_sum += qp + np * (dm * dm);
                }
            }
            var = __fdiv_rn(warp_sum(q_sum), static_cast<float>(d));
            // This CTA is done reading its peers.  No release is needed: the
            // values read are already consumed, the next exchange barrier (a
            // release) orders these reads before any peer rewrites this
            // buffer (double buffering), and this arrive only keeps the
            // peers resident until the reads are done.  (Measured on GB300:
            // 3-6% faster than a release arrive for 1-32 rows of d >= 16384.)
            cluster_arrive_relaxed();
        } else if (!CL) {
            const float s = block_sum<NW, V == 2>(acc.x + acc.y, red[0], lane, warp);
            mean = __fdiv_rn(s, static_cast<float>(d));
            const float2 m2 = make_float2(mean, mean);
            acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (v0 + tid + NT * i < v1)
                    acc = ssd_vec<F>(acc, g[i], m2);
            var = __fdiv_rn(block_sum<NW, V == 2>(acc.x + acc.y, red[1], lane, warp),
                            static_cast<float>(d));
        } else {
            const float s = block_sum<NW>(acc.x + acc.y, red[0], lane, warp);
            // local two-pass statistics of this CTA's slice ...
            const float mk = nk > 0 ? __fdiv_rn(s, static_cast<float>(nk)) : 0.f;
            const float2 m2 = make_float2(mk, mk);
            acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (v0 + tid + NT * i < v1)
                    acc = ssd_vec<F>(acc, g[i], m2);
            const float q = block_sum<NW>(acc.x + acc.y, red[1], lane, warp);
            if (tid == 0) {
                xch[0] = static_cast<float>(nk);
                xch[1] = s;
                xch[2] = q;
            }
            cluster_arrive_release();
            cluster_wait_acquire();
            // ... merged over the cluster in rank order (lane k reads CTA k):
            // M2 = sum_k M2_k + sum_k n_k (mean_k - mean)^2.
            float n_k = 0.f, s_k = 0.f, q_k = 0.f;
            if (lane < C) {
                n_k = ld_peer(&xch[0], lane);
                s_k = ld_peer(&xch[1], lane);
                q_k = ld_peer(&xch[2], lane);
            }
            mean = __fdiv_rn(warp_sum(s_k), static_cast<float>(d));
            float between = 0.f;
            if (n_k > 0.f) {
                const float dm = __fdiv_rn(s_k, n_k) - mean;
                between = n_k * (dm * dm);
            }
            var = __fdiv_rn(warp_sum(q_k + between), static_cast<float>(d));
            cluster_arrive_release();   // this CTA is done reading its peers
        }
        const float cutoff = NATIVE ? native_cutoff<F>(mean, var, z)
                                    : fmaf(__fsqrt_rn(var), z, mean);

        uint8_t *op = out + row * d_bytes;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = v0 + tid + NT * i;
            if (v < v1) {
                if constexpr (NATIVE)
                    st_vec_out(op + 16 * v, epi_vec_native<F>(g[i], u[i], cutoff, lut));
                else
                    st_vec(op + 16 * v, epi_vec<F>(g[i], u[i], cutoff));
            }
        }
        if (CL)
            cluster_wait_acquire();   // peers are done with xch before it changes
    }
}

// ------------------------------------------------------------ split rows
// A few wide rows, C independent CTAs per row (no cluster).  Each CTA reads
// the row's whole gate half and computes the row's statistics itself, in the
// same order as the other CTAs of the row, so all of them hold the same bits;
// then it does the epilogue of its slice [k sv, (k+1) sv) of the columns.
// The C reads of a gate half-row arrive together and L2 serves all but the
// first, so nothing is exchanged between CTAs: measured on GB300 this beats
// the cluster exchange (0.6-1.2 us per row) from 9 rows on while all CTAs fit
// one wave.  Thread t holds gate vectors t + NT i (i < V, the whole row) for
// the statistics and, for the epilogue, the slice's vectors v0 + t + NT j
// (j < U) of gate and up.  NATIVE: the native-rounding composition (cutoff
// and epilogue rounded to the format after every op, a from the table).
// The two CTA sums take the narrow butterfly (measured on GB300: 1-3% faster
// at 1-64 rows of d = 8192 ... 32768; it adds the same partials in the same
// pairs).  One CTA barrier
// instead of two -- per-warp two-pass statistics merged in the pairwise form
// of Chan, Golub and LeVeque -- was 6-12% slower (1 x 8192: 2.15 against
// 2.03 us; 8 x 20480: 3.03 against 2.73).
template <int NT, int V, int U, class F, bool NATIVE>
__global__ void __launch_bounds__(NT, 1)
gelu_split_rows(void *__restrict__ out_, const void *__restrict__ in_, int64_t T, int d,
                int64_t rs, float z, int C, int sv) {
    constexpr int NW = NT / 32;
    constexpr int kEpv = 16 / F::kElem;
    __shared__ float red[2][NW];
    const uint8_t *in = static_cast<const uint8_t *>(in_);
    uint8_t *out = static_cast<uint8_t *>(out_);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nvec = d / kEpv;
    const int64_t rs_bytes = rs * F::kElem, d_bytes = static_cast<int64_t>(d) * F::kElem;
    pdl_wait();
    pdl_trigger();
    const uint16_t *lut = nullptr;   // native mode: the table of a, once built
    if constexpr (NATIVE)
        lut = native_table<F>();
    for (int64_t b = blockIdx.x; b < T * C; b += gridDim.x) {
        const int64_t row = b / C;
        const int v0 = static_cast<int>(b - row * C) * sv;
        const int v1 = min(nvec, v0 + sv);
        const uint8_t *gp = in + row * rs_bytes;
        const uint8_t *up = gp + d_bytes;
        uint4 g[V], gs[U], u[U];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + NT * i;
            g[i] = v < nvec ? ld_stream(gp + 16 * v) : make_uint4(0u, 0u, 0u, 0u);   // +0
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int v = v0 + tid + NT * j;
            if (v < v1) {
                gs[j] = ld_stream(gp + 16 * v);
                u[j] = ld_stream(up + 16 * v);
            } else {
                gs[j] = u[j] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc = sum_vec<F>(acc, g[i]);
        const float mean =
            __fdiv_rn(block_sum<NW, true>(acc.x + acc.y, red[0], lane, warp), static_cast<float>(d));
        const float2 m2 = make_float2(mean, mean);
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (tid + NT * i < nvec)
                acc = ssd_vec<F>(acc, g[i], m2);
        const float var =
            __fdiv_rn(block_sum<NW, true>(acc.x + acc.y, red[1], lane, warp), static_cast<float>(d));
        const float cutoff =
            NATIVE ? native_cutoff<F>(mean, var, z) : fmaf(__fsqrt_rn(var), z, mean);
        uint8_t *op = out + row * d_bytes;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int v = v0 + tid + NT * j;
            if (v < v1) {
                if constexpr (NATIVE)
                    st_vec_out(op + 16 * v, epi_vec_native<F>(gs[j], u[j], cutoff, lut));
                else
                    st_vec(op + 16 * v, epi_vec<F>(gs[j], u[j], cutoff));
            }
        }
        __syncthreads();   // red[] is rewritten by the next row
    }
}

// ------------------------------------------------------------ scalar rows
// Any layout: one CTA per row, one element per access; each pass re-reads
// the gate (from L1/L2 after the first pass).
__device__ __forceinline__ float sparse_gelu_mul(float g, float u, float cutoff, bool exp_form) {
    const float s = relu_nan(g - cutoff);
    const float y = s * fmaf(kCubicCoef, s * s, kSqrt2OverPi);
    const float h = 0.5f * s;
    return (exp_form ? gelu_exp_form(s, y) : fmaf(h, tanh_approx(y), h)) * u;
}

template <class F, bool NATIVE>
__global__ void __launch_bounds__(kScalarThreads)
gelu_scalar_rows(void *__restrict__ out_, const void *__restrict__ in_, int64_t T, int64_t d,
                 int64_t rs, float z) {
    constexpr int NW = kScalarThreads / 32;
    constexpr int64_t E = F::kElem;
    __shared__ float red[2][NW];
    const uint8_t *in = static_cast<const uint8_t *>(in_);
    uint8_t *out = static_cast<uint8_t *>(out_);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
        const uint8_t *gp = in + row * rs * E;
        const uint8_t *up = gp + d * E;
        float s = 0.f;
        for (int64_t j = tid; j < d; j += kScalarThreads)
            s += F::load1(gp + j * E);
        s = block_sum<NW>(s, red[0], lane, warp);
        const float mean = __fdiv_rn(s, static_cast<float>(d));
        float q = 0.f;
        for (int64_t j = tid; j < d; j += kScalarThreads) {
            const float e = F::load1(gp + j * E) - mean;
            q = fmaf(e, e, q);
        }
        q = block_sum<NW>(q, red[1], lane, warp);
        const float var = __fdiv_rn(q, static_cast<float>(d));
        const float cutoff = NATIVE ? native_cutoff<F>(mean, var, z)
                                    : fmaf(__fsqrt_rn(var), z, mean);
        uint8_t *op = out + row * d * E;
        for (int64_t j = tid; j < d; j += kScalarThreads) {
            const float g = F::load1(gp + j * E), u = F::load1(up + j * E);
            F::store1(op + j * E, NATIVE ? native_gelu_mul<F>(g, u, cutoff)
                                         : sparse_gelu_mul(g, u, cutoff, E == 4));
        }
    }
}

// ------------------------------------------------------------ host side
using WarpFn = void (*)(uint16_t *, const uint16_t *, int64_t, int, int64_t, float);
using CtaFn = void (*)(void *, const void *, int64_t, int, int64_t, float, int, int);
using ScalarFn = void (*)(void *, const void *, int64_t, int64_t, int64_t, float);
using TmaFn = void (*)(uint16_t *, const uint16_t *, int64_t, int, int64_t, float, int,
                      unsigned long long *, int64_t, unsigned long long);
using PipeFn = void (*)(uint16_t *, const uint16_t *, int64_t, int, int64_t, float, int,
                        unsigned long long *, int64_t, int64_t, unsigned long long);

WarpFn warp_fn(int v) {
    switch (v) {
    case 1: return gelu_warp_rows<1>;
    case 2: return gelu_warp_rows<2>;
    case 4: return gelu_warp_rows<4>;
    case 8: return gelu_warp_rows<8>;
    default: return nullptr;
    }
}

template <bool CL, class F, bool N>
CtaFn cta_fn_t(int nt, int v) {
    if (v == 2) {
        switch (nt) {
        case 64: return gelu_cta_rows<64, 2, CL, F, N>;
        case 128: return gelu_cta_rows<128, 2, CL, F, N>;
        // the few-rows shapes (cta_shape, few_rows): lone CTAs, and CTAs of
        // 8-CTA clusters
        case 256: return gelu_cta_rows<256, 2, CL, F, N>;
        default: break;
        }
        if constexpr (!CL) {
            if (nt == 512)
                return gelu_cta_rows<512, 2, false, F, N>;
        }
        return nullptr;
    }
    if (v == 4) {
        switch (nt) {
        case 64: return gelu_cta_rows<64, 4, CL, F, N>;
        case 128: return gelu_cta_rows<128, 4, CL, F, N>;
        case 256: return gelu_cta_rows<256, 4, CL, F, N>;
        case 512: return gelu_cta_rows<512, 4, CL, F, N>;
        case 1024: return gelu_cta_rows<1024, 4, CL, F, N>;
        default: return nullptr;
        }
    }
    return nullptr;
}

template <class F, bool N>
CtaFn cta_fn_f(int nt, int v, int cluster) {
    return cluster > 1 ? cta_fn_t<true, F, N>(nt, v) : cta_fn_t<false, F, N>(nt, v);
}

// native: the native-rounding composition (bf16 and fp16 only)
CtaFn cta_fn(int nt, int v, int cluster, int dtype, bool native) {
    switch (dtype) {
    case GATED_ACT_F16:
        return native ? cta_fn_f<FmtF16, true>(nt, v, cluster)
                      : cta_fn_f<FmtF16, false>(nt, v, cluster);
    case GATED_ACT_F32: return native ? nullptr : cta_fn_f<FmtF32, false>(nt, v, cluster);
    default:
        return native ? cta_fn_f<FmtBf16, true>(nt, v, cluster)
                      : cta_fn_f<FmtBf16, false>(nt, v, cluster);
    }
}

// Split rows: NT threads of 8 gate vectors, U slice vectors per thread.
template <class F, bool N>
CtaFn split_fn_f(int nt, int u) {
    switch (nt * 8 + u) {
    case 128 * 8 + 1: return gelu_split_rows<128, 8, 1, F, N>;
    case 128 * 8 + 2: return gelu_split_rows<128, 8, 2, F, N>;
    case 128 * 8 + 4: return gelu_split_rows<128, 8, 4, F, N>;
    case 256 * 8 + 1: return gelu_split_rows<256, 8, 1, F, N>;
    case 256 * 8 + 2: return gelu_split_rows<256, 8, 2, F, N>;
    case 256 * 8 + 4: return gelu_split_rows<256, 8, 4, F, N>;
    case 512 * 8 + 1: return gelu_split_rows<512, 8, 1, F, N>;
    case 512 * 8 + 2: return gelu_split_rows<512, 8, 2, F, N>;
    case 512 * 8 + 4: return gelu_split_rows<512, 8, 4, F, N>;
    default: return nullptr;
    }
}
// native: the native-rounding composition (bf16 and fp16 only)
CtaFn split_fn(int nt, int u, int dtype, bool native) {
    switch (dtype) {
    case GATED_ACT_F16:
        return native ? split_fn_f<FmtF16, true>(nt, u) : split_fn_f<FmtF16, false>(nt, u);
    case GATED_ACT_F32: return native ? nullptr : split_fn_f<FmtF32, false>(nt, u);
    default:
        return native ? split_fn_f<FmtBf16, true>(nt, u) : split_fn_f<FmtBf16, false>(nt, u);
    }
}

ScalarFn scalar_fn(int dtype, bool native) {
    switch (dtype) {
    case GATED_ACT_F16:
        return native ? gelu_scalar_rows<FmtF16, true> : gelu_scalar_rows<FmtF16, false>;
    case GATED_ACT_F32: return native ? nullptr : gelu_scalar_rows<FmtF32, false>;
    default:
        return native ? gelu_scalar_rows<FmtBf16, true> : gelu_scalar_rows<FmtBf16, false>;
    }
}

int elem_bytes(int dtype) { return dtype == GATED_ACT_F32 ? 4 : 2; }

TmaFn tma_fn(int nt) {
    switch (nt) {
    case 32: return gelu_tma_rows<32, 4>;
    case 64: return gelu_tma_rows<64, 4>;
    case 128: return gelu_tma_rows<128, 4>;
    case 256: return gelu_tma_rows<256, 4>;
    case 512: return gelu_tma_rows<512, 4>;
    case 1024: return gelu_tma_rows<1024, 4>;
    default: return nullptr;
    }
}

// Pipe rows: NCW consumer warps x V gate vectors per consumer thread.
PipeFn pipe_fn(int ncw, int v) {
    switch (ncw * 16 + v) {
    case 16 * 16 + 8: return gelu_pipe_rows<16, 8>;
    case 16 * 16 + 4: return gelu_pipe_rows<16, 4>;
    case 8 * 16 + 8: return gelu_pipe_rows<8, 8>;
    case 8 * 16 + 4: return gelu_pipe_rows<8, 4>;
    case 4 * 16 + 8: return gelu_pipe_rows<4, 8>;
    case 4 * 16 + 4: return gelu_pipe_rows<4, 4>;
    case 4 * 16 + 2: return gelu_pipe_rows<4, 2>;
    default: return nullptr;
    }
}

int pow2_ceil(int64_t x) {
    int p = 1;
    while (p < x)
        p <<= 1;
    return p;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
    gated_act_plan pub;
    int sv;        // vectors per CTA slice (CTA rows, split rows)
    int su;        // slice vectors per thread (split rows)
    int dtype;     // gated_act_dtype of in and out
    bool native;   // native-rounding composition
};

// Threads and vectors per thread for a CTA slice of sv vectors.
// few_rows (a lone CTA per row, and the two-vector CTAs of all rows within
// one wave of 1024 threads per SM): two vectors per thread up to 1024
// vectors, so a row spreads over more threads.  Measured on GB300:
// 6-14% faster at d = 4096 up to T = 608 and at d = 8192 up to T = 304
// (T = 64, d = 8192: 2.73 against 2.99 us), but 8-23% slower beyond, where
// four vectors per thread let more rows share an SM.
void cta_shape(int64_t sv, int *nt, int *v, bool few_rows = false) {
    if (sv <= kMinSliceVec || (few_rows && sv <= 4 * kMinSliceVec)) {
        *v = 2;
        *nt = std::max(64, pow2_ceil(ceil_div(sv, 2)));
    } else {
        *v = 4;
        *nt = std::max(64, pow2_ceil(ceil_div(sv, 4)));
    }
}

// TMA rows geometry for a row of nvec gate vectors.  An SM runs 1024
// threads (64 registers each) split into cps CTAs of NT = 1024 / cps threads
// (fewer when the row is short), so cps rows are in progress per SM and one
// row's reduce/barrier latency overlaps the others' arithmetic.  Each CTA
// gets 1/cps of the SM's shared memory and at least three slots (the next
// row's gate and up stream in while a row is finished; two when a single CTA
// holds the widest rows).  want_cps = 0 picks cps; otherwise it is forced.
// Returns false when the row does not fit.
bool tma_shape_for(int64_t nvec, int c, int *nt, int *stages, int64_t *smem) {
    const int64_t chunk = 16 * nvec;                        // bytes of a gate (or up) half-row
    const int n = std::min(1024 / c, std::max(32, pow2_ceil(nvec)));
    if (n < 32 || ceil_div(nvec, n) > 4)
        return false;
    const int64_t per_cta = std::min<int64_t>(kTmaSmemPerSm / c, kTmaSmemPerCta) - 1536;
    const int64_t s = std::min<int64_t>(kTmaMaxStages, (per_cta - 8 * kTmaMaxStages) / chunk);
    if (s < 3 && !(c == 1 && s >= 2))
        return false;
    *nt = n;
    *stages = static_cast<int>(s);
    *smem = s * chunk + 8 * s;
    return true;
}

// Pipe rows geometry for a row of nvec gate vectors at cps CTAs per SM:
// consumer warps and vectors per thread from the instantiated set (four
// vectors per thread preferred), no more CTAs per SM than the kernel's
// register budget allows (its launch bounds), and at least three ring slots
// in 1/cps of the SM's shared memory.
bool pipe_shape_for(int64_t nvec, int cps, int *ncw, int *v, int *stages, int64_t *smem) {
    static const int kShapes[][2] = {{4, 4}, {8, 4}, {16, 4}, {4, 8}, {8, 8}, {16, 8}, {4, 2}};
    for (const auto &sh : kShapes) {
        const int w = sh[0], vv = sh[1];
        const int64_t cap = int64_t(w) * 32 * vv;
        if (cap < nvec || (w > 4 && cap / 2 >= nvec))
            continue;   // too small, or a smaller CTA would do
        if (cps > (w >= 16 ? 1 : w >= 8 ? 2 : 4))
            continue;   // the register budget each kernel is compiled for
        const int64_t chunk = 16 * nvec;
        const int64_t per_cta = std::min<int64_t>(kTmaSmemPerSm / cps, kTmaSmemPerCta) - 1536;
        // Ring depth, measured on GB300: about two rows ahead (four slots at
        // one CTA per SM, five at two) beats a deeper ring, which takes its
        // rows further ahead and so starts and ends the launch later
        // (2048 x 16384 at one CTA per SM: 31.3 us with 4 slots, 32.5 with 7).
        const int64_t depth = cps == 1 ? 4 : cps == 2 ? 5 : kPipeMaxStages;
        const int64_t s = std::min<int64_t>(depth, per_cta / (chunk + 24));
        if (s < 3)
            continue;
        *ncw = w;
        *v = vv;
        *stages = static_cast<int>(s);
        *smem = s * (chunk + 24);
        return true;
    }
    return false;
}

bool pipe_shape(int64_t nvec, int want_cps, int *cps, int *ncw, int *v, int *stages,
                int64_t *smem) {
    if (want_cps > 0) {
        if (want_cps > 8 || (want_cps & (want_cps - 1)) != 0)
            return false;
        *cps = want_cps;
        return pipe_shape_for(nvec, want_cps, ncw, v, stages, smem);
    }
    // default: as many CTAs per SM as keep the gate half-rows of the rows
    // in progress on an SM within 32 KB (one CTA per SM from d = 12288 on)
    for (int c = 8; c >= 1; c /= 2) {
        if (16 * nvec * c > 32 * 1024 && c > 1)
            continue;
        if (pipe_shape_for(nvec, c, ncw, v, stages, smem)) {
            *cps = c;
            return true;
        }
    }
    return false;
}

bool tma_shape(int64_t nvec, int want_cps, int *cps, int *nt, int *stages, int64_t *smem) {
    if (want_cps > 0) {
        if (want_cps > 16 || (want_cps & (want_cps - 1)) != 0)
            return false;
        *cps = want_cps;
        return tma_shape_for(nvec, want_cps, nt, stages, smem);
    }
    // default: four 16-byte gate vectors per thread (the most cps that fits)
    for (int c = 16; c >= 1; c /= 2) {
        if (1024 / c < ceil_div(nvec, 4))
            continue;
        if (tma_shape_for(nvec, c, nt, stages, smem)) {
            *cps = c;
            return true;
        }
    }
    return false;
}

// check_ptrs = false (plan queries): pointers are only inspected for alignment.
int validate(const void *out, const void *in, int64_t T, int64_t d, int64_t rs, int elem,
             bool check_ptrs) {
    if (T < 0 || d <= 0)
        return GATED_ACT_ERR_SIZE;
    if (rs < 2 * d)
        return GATED_ACT_ERR_STRIDE;
    if (d > (int64_t(1) << 30) || rs > (int64_t(1) << 40) || T > (int64_t(1) << 40))
        return GATED_ACT_ERR_TOO_LARGE;
    if (T == 0 || !check_ptrs)
        return GATED_ACT_OK;
    if (!out || !in)
        return GATED_ACT_ERR_NULL;
    if (!aligned(out, elem) || !aligned(in, elem))
        return GATED_ACT_ERR_ALIGN;
    const uint64_t in_bytes = elem * static_cast<uint64_t>((T - 1) * rs + 2 * d);
    const uint64_t out_bytes = elem * static_cast<uint64_t>(T * d);
    if (ranges_overlap(out, out_bytes, in, in_bytes))
        return GATED_ACT_ERR_OVERLAP;
    return GATED_ACT_OK;
}

// host_mem: in or out lives in host memory; only register-load kernels run.
int make_plan(const void *out, const void *in, int64_t T, int64_t d, int64_t rs, int dtype,
              int variant, int cluster, int sm_count, bool check_ptrs, Plan *p,
              bool native = false, bool host_mem = false, bool has_ws = false) {
    if (dtype < GATED_ACT_BF16 || dtype > GATED_ACT_F32 || (native && dtype == GATED_ACT_F32))
        return GATED_ACT_ERR_DTYPE;
    const int elem = elem_bytes(dtype), epv = 16 / elem;
    const int rc = validate(out, in, T, d, rs, elem, check_ptrs);
    if (rc != GATED_ACT_OK)
        return rc;
    if (variant < GATED_ACT_VARIANT_AUTO || variant > GATED_ACT_VARIANT_SPLIT_ROWS)
        return GATED_ACT_ERR_VARIANT;
    const bool forced = variant != GATED_ACT_VARIANT_AUTO;
    // the warp-rows and bulk-copy kernels exist for plain bf16 only; bulk
    // copies from host memory are not used
    const bool cta_only = dtype != GATED_ACT_BF16 || native;
    const bool bulk = variant == GATED_ACT_VARIANT_TMA_ROWS || variant == GATED_ACT_VARIANT_PIPE_ROWS;
    if (cta_only && (variant == GATED_ACT_VARIANT_WARP_ROWS || bulk))
        return GATED_ACT_ERR_VARIANT;
    if (host_mem && bulk)
        return GATED_ACT_ERR_VARIANT;
    // split rows read the gate half-row once per CTA: not from host memory
    if (variant == GATED_ACT_VARIANT_SPLIT_ROWS && host_mem)
        return GATED_ACT_ERR_VARIANT;
    gated_act_plan &q = p->pub;
    q = gated_act_plan{};
    p->sv = 0;
    p->su = 0;
    p->dtype = dtype;
    p->native = native;
    const bool vec_ok = aligned(in, 16) && aligned(out, 16) && d % epv == 0 && rs % epv == 0;
    const int64_t nvec = d / epv;
    const int sms = sm_count > 0 ? sm_count : (T > 0 ? device_sm_count() : 1);
    int t_cps = 0, t_nt = 0, t_stages = 0;
    int64_t t_smem = 0;
    const int want_cps = variant == GATED_ACT_VARIANT_TMA_ROWS ? cluster : 0;
    const bool tma_ok = vec_ok && !cta_only && !host_mem &&
                        tma_shape(nvec, want_cps, &t_cps, &t_nt, &t_stages, &t_smem);
    int p_cps = 0, p_ncw = 0, p_v = 0, p_stages = 0;
    int64_t p_smem = 0;
    const bool pipe_ok =
        vec_ok && !cta_only && !host_mem &&
        pipe_shape(nvec, variant == GATED_ACT_VARIANT_PIPE_ROWS ? cluster : 0, &p_cps, &p_ncw,
                   &p_v, &p_stages, &p_smem);

    // Measured on GB300 (every geometry timed per T x d, graph-replayed over
    // rotating buffers):
    //  * rows wider than 16384 from about 1.6 rows per SM at d = 32768 on:
    //    pipe rows; with a workspace (dynamic rows) at any T, without one
    //    while round-robin rows stay below 8 per CTA for d >= 28672 (beyond
    //    that a slow SM holds the static split back more than in tma rows:
    //    2048 x 28672, 59.6 against 56.7 us; at d = 24576 the two are within
    //    2%, at d = 20480 pipe rows stay ahead, 40.5 against 45.9);
    //  * d in [14336, 16384]: pipe rows from 8 rows per SM on, with or
    //    without a workspace (from 6 rows per SM a single launch is faster
    //    too, but among other activation kernels the switch of the SM's
    //    shared-memory split around it costs more than it gains);
    //  * tma rows for the widest rows at many rows per SM;
    //  * one CTA per row everywhere else, except up to 64 rows wider than
    //    8192, where clusters put more SMs on each row.
    // Split rows, measured on GB300 against cluster rows and one CTA per row
    // at T = 1 ... 192 and d = 4096 ... 32768, with the most CTAs per row that
    // fit one wave:
    //  * 8192 < d <= 16384, any T: 8, 4 or 2 per row (1 x 16384: 2.03 against
    //    2.16 us in 8-CTA clusters; 16 x 11008: 2.42 against 2.89; 64 x 16384:
    //    3.34 against 3.66 with one CTA per row);
    //  * d = 8192, 8 or 4 per row only (1 x 8192: 1.79 against 1.96 us with
    //    one CTA of 512 threads; 2-5% ahead from 8 rows on, within 1% at 2
    //    and 4 rows; with two per row one CTA wins);
    //  * wider rows up to d = 32768: 8 or 4 per row at 9-32 rows (16 x 32768:
    //    3.13 against 3.45 in 4-CTA clusters), 2 per row at 33 and more (64 x
    //    32768: 4.50 against 5.14 in 2-CTA clusters), and at up to 8 rows 8
    //    per row up to d = 20480 only (at d = 32768 8-CTA clusters stay 4-5%
    //    ahead);
    //  * d = 4096, and beyond one wave: split rows lose.
    // Native rounding (the table-read epilogue) gains more from split rows
    // (1 x 16384: 2.61 against 3.47 us in 8-CTA clusters; 64 x 32768: 5.62
    // against 6.78) but keeps one CTA per row where two or four CTAs per row
    // of d <= 16384 would take it (64 x 16384: 4.01 against 4.46 split in two)
    // -- at d = 8192 it takes 8 per row only.
    int split_c = 0;
    if (vec_ok && !host_mem && nvec >= 1024 && nvec <= 4096) {
        int cmin = 2, cmax = kMaxCluster;
        if (nvec == 1024)
            cmin = native ? kMaxCluster : 4;
        else if (nvec > 2048 && T <= kFewRows)
            cmin = nvec <= 2560 ? kMaxCluster : 2 * kMaxCluster;
        else if (nvec > 2048 && T <= 4 * kFewRows)
            cmin = 4;
        else if (nvec > 2048)
            cmax = 2;
        else if (native)
            cmin = 4;
        for (int c = cmax; c >= cmin && !split_c; c /= 2)
            if (T * c <= sms)
                split_c = c;
    }

    if (variant == GATED_ACT_VARIANT_AUTO) {
        const int64_t sm = static_cast<int64_t>(sms);
        if (!vec_ok || nvec > int64_t(kMaxSliceVec) * kMaxCluster)
            variant = GATED_ACT_VARIANT_SCALAR;
        else if (pipe_ok && nvec > 2048 && 10 * T * nvec >= 16 * sm * 4096 &&
                 (has_ws || nvec < 3584 || T < 8 * sm))
            variant = GATED_ACT_VARIANT_PIPE_ROWS;
        else if (pipe_ok && nvec >= 1792 && nvec <= 2048 && T >= 8 * sm)
            variant = GATED_ACT_VARIANT_PIPE_ROWS;
        else if (tma_ok && ((nvec >= 3584 && T >= 3 * sm) || (nvec >= 2048 && T >= 12 * sm)))
            variant = GATED_ACT_VARIANT_TMA_ROWS;
        else if (nvec <= 64 && !cta_only)
            variant = GATED_ACT_VARIANT_WARP_ROWS;
        else if (split_c > 0)
            variant = GATED_ACT_VARIANT_SPLIT_ROWS;
        else
            variant = GATED_ACT_VARIANT_CTA_ROW;
        cluster = variant == GATED_ACT_VARIANT_SPLIT_ROWS ? split_c : 0;
    }

    if (variant == GATED_ACT_VARIANT_SPLIT_ROWS) {
        // C CTAs per row (2, 4 or 8), 8 gate vectors per thread for the whole
        // row: 256 threads up to 2048 vectors, 512 up to 4096; 128 up to 1024
        // vectors in 8 CTAs per row (measured on GB300 at d = 8192: 1 row
        // 1.80 against 1.89 us with 256 threads, 8 rows 2.19 against 2.28; in
        // 4 CTAs per row 2% slower)
        const int C = cluster;
        if (!vec_ok || (C != 2 && C != 4 && C != 8) || nvec > 4096)
            return GATED_ACT_ERR_VARIANT;
        const int nt = (nvec <= 1024 && C == 8) ? 128 : nvec <= 2048 ? 256 : 512;
        const int64_t sv = ceil_div(nvec, C);
        const int su = pow2_ceil(ceil_div(sv, nt));
        if (su > 4)
            return GATED_ACT_ERR_VARIANT;
        q.variant = variant;
        q.cluster = C;
        q.threads = nt;
        q.vec_per_thread = 8;
        q.rows_per_cta = 1;
        q.grid = std::min<int64_t>(T, 0x7FFFFFFF / C) * C;
        p->sv = static_cast<int>(sv);
        p->su = su;
        return GATED_ACT_OK;
    }

    if (variant == GATED_ACT_VARIANT_TMA_ROWS) {
        if (!tma_ok)
            return GATED_ACT_ERR_VARIANT;
        q.variant = variant;
        q.cluster = 1;
        q.threads = t_nt;
        q.vec_per_thread = static_cast<int32_t>(ceil_div(nvec, t_nt));
        q.rows_per_cta = 1;
        q.ctas_per_sm = t_cps;
        q.stages = t_stages;
        q.smem_bytes = t_smem;
        q.grid = std::min<int64_t>(T, static_cast<int64_t>(sms) * t_cps);
        q.dynamic_rows = (forced || T >= kDynamicRowsPerCta * q.grid) ? 1 : 0;
        return GATED_ACT_OK;
    }

    if (variant == GATED_ACT_VARIANT_PIPE_ROWS) {
        if (!pipe_ok)
            return GATED_ACT_ERR_VARIANT;
        q.variant = variant;
        q.cluster = 1;
        q.threads = (p_ncw + 1) * 32;
        q.vec_per_thread = p_v;
        q.rows_per_cta = 1;
        q.ctas_per_sm = p_cps;
        q.stages = p_stages;
        q.smem_bytes = p_smem;
        q.grid = std::min<int64_t>(T, static_cast<int64_t>(sms) * p_cps);
        q.dynamic_rows = 1;   // measured: never slower than round-robin here
        return GATED_ACT_OK;
    }

    if (variant == GATED_ACT_VARIANT_WARP_ROWS) {
        if (!vec_ok || nvec > 256)
            return GATED_ACT_ERR_VARIANT;
        q.variant = variant;
        q.cluster = 1;
        q.threads = kWarpRowsThreads;
        q.vec_per_thread = pow2_ceil(ceil_div(nvec, 32));
        q.rows_per_cta = kWarpRowsThreads / 32;
        q.grid = ceil_div(T, q.rows_per_cta);
        if (q.grid > 0x7FFFFFFF)
            return GATED_ACT_ERR_TOO_LARGE;
        return GATED_ACT_OK;
    }

    if (variant == GATED_ACT_VARIANT_CTA_ROW) {
        if (!vec_ok)
            return GATED_ACT_ERR_VARIANT;
        int C = cluster;
        if (C == 0) {
            C = 1;
            while (ceil_div(nvec, C) > kMaxSliceVec && C < kMaxCluster)
                C *= 2;
            // measured on GB300 (every cluster size at T = 1...96 for d =
            // 8192 ... 32768): 8-CTA clusters for up to 8 rows wider than
            // 8192 (d = 9216, T = 1: 2.29 against 2.72 us with one CTA per
            // row, whose CTA then has 1024 threads; at d = 8192 one CTA of
            // 512 threads is 2-5% faster), up to 16 rows of d <= 16384
            // (d = 11008, T = 16: 2.89 against 2.99) and up to 32 rows of
            // d = 14336 ... 16384 (d = 16384, T = 32: 3.28 against 3.40;
            // T = 40: 3.50 against 3.44); 4-CTA clusters for 9-32 rows of
            // wider rows (d = 32768, T = 16: 3.84 against 4.59 us with one
            // CTA per row; d = 20480 and 24576, T = 16: 3.12 and 3.20 against
            // 3.36 and 3.41 in 8-CTA clusters, 3.81 and 4.04 with one CTA per
            // row), 2-CTA clusters for 33-64 of them (d = 32768, T = 64: 5.36
            // against 5.54 us; d = 24576, T = 48: 4.27 against 4.45; from 96
            // rows one CTA per row is 10% faster)
            const bool eight =
                nvec > 1024 &&
                (T <= kFewRows ||
                 (nvec <= 2048 && (T <= 2 * kFewRows || (nvec >= 1792 && T <= 4 * kFewRows))));
            if (eight)
                C = kMaxCluster;
            else if (T <= 4 * kFewRows && nvec > 2048)
                C = std::max(C, 4);
            else if (T <= 8 * kFewRows && nvec > 2048)
                C = std::max(C, 2);
        }
        if (C < 1 || C > kMaxCluster || (C & (C - 1)) != 0)
            return GATED_ACT_ERR_VARIANT;
        const int64_t sv = ceil_div(nvec, C);
        if (sv > kMaxSliceVec)
            return GATED_ACT_ERR_VARIANT;
        int nt, v;
        // few rows: the two-vector CTAs of all rows fit in one wave of 1024
        // threads per SM; and slices of 8-CTA clusters up to 512 vectors
        // (d = 32768 at T <= 8: 256 threads of two vectors, measured on
        // GB300 1-4% faster than 128 threads of four)
        const bool few_rows =
            (C == 1 && T * pow2_ceil(ceil_div(sv, 2)) <= 1024 * static_cast<int64_t>(sms)) ||
            (C == kMaxCluster && sv <= 2 * kMinSliceVec);
        cta_shape(sv, &nt, &v, few_rows);
        q.variant = variant;
        q.cluster = C;
        q.threads = nt;
        q.vec_per_thread = v;
        q.rows_per_cta = 1;
        const int64_t max_clusters = 0x7FFFFFFF / C;
        q.grid = std::min<int64_t>(T, max_clusters) * C;
        p->sv = static_cast<int>(sv);
        return GATED_ACT_OK;
    }

    // scalar
    q.variant = GATED_ACT_VARIANT_SCALAR;
    q.cluster = 1;
    q.threads = kScalarThreads;
    q.vec_per_thread = 0;
    q.rows_per_cta = 1;
    q.grid = std::min<int64_t>(T, 0x7FFFFFFF);
    return GATED_ACT_OK;
}

// Unique id of the calling thread's current CUDA context (cuCtxGetId, reached
// through the runtime's driver entry-point query, so the library links no
// driver library of its own); 0 when no context is current or the driver
// cannot tell.  Ids are never reused within a process, so a context made
// after cudaDeviceReset has a new one.
unsigned long long current_context_id() {
    using GetCurrent = CUresult (*)(CUcontext *);
    using GetId = CUresult (*)(CUcontext, unsigned long long *);
    struct Fns {
        GetCurrent cur = nullptr;
        GetId id = nullptr;
    };
    static const Fns fns = [] {
        Fns f;
        void *a = nullptr, *b = nullptr;
        cudaDriverEntryPointQueryResult qa = cudaDriverEntryPointSymbolNotFound, qb = qa;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &a, 12000, cudaEnableDefault,
                                             &qa) == cudaSuccess &&
            qa == cudaDriverEntryPointSuccess &&
            cudaGetDriverEntryPointByVersion("cuCtxGetId", &b, 12000, cudaEnableDefault, &qb) ==
                cudaSuccess &&
            qb == cudaDriverEntryPointSuccess) {
            f.cur = reinterpret_cast<GetCurrent>(a);
            f.id = reinterpret_cast<GetId>(b);
        }
        cudaGetLastError();   // a failed query is not sticky; leave no error behind
        return f;
    }();
    if (!fns.cur || !fns.id)
        return 0;
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (fns.cur(&ctx) != CUDA_SUCCESS || !ctx || fns.id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// Shared memory above 48 KB needs a per-kernel opt-in; the carveout hint asks
// for the largest shared-memory split of L1.  Both are attributes of the
// kernel in one context, so they are set once per (device, context): a new
// context (after cudaDeviceReset, or one the caller made current) sets them
// again, and where the context id is unavailable they are set on every call.
// key: a bit index in [0, 32) that names the kernel.
template <class Fn>
int ensure_smem_attr(Fn fn, int key) {
    constexpr int kMaxDevices = 64;
    struct Entry {
        unsigned long long ctx;
        unsigned bits;
    };
    static Entry done[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        dev = -1;
    const bool slot = dev >= 0 && dev < kMaxDevices;
    const unsigned bit = 1u << key;
    const unsigned long long ctx = slot ? current_context_id() : 0;
    if (ctx != 0) {
        std::lock_guard<std::mutex> lock(mu);
        if (done[dev].ctx == ctx && (done[dev].bits & bit))
            return GATED_ACT_OK;
    }
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, fn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kTmaSmemPerCta - static_cast<int>(fa.sharedSizeBytes));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess)
        return cuda_status(e);
    if (ctx != 0) {
        std::lock_guard<std::mutex> lock(mu);
        if (done[dev].ctx != ctx)
            done[dev] = Entry{ctx, 0u};
        done[dev].bits |= bit;
    }
    return GATED_ACT_OK;
}

// Pipe rows with dynamic rows: how many of the last rows run as two half
// jobs (rows of an even number of 16-byte vectors only).
int64_t pipe_split_rows(int64_t T, int64_t nvec, int64_t grid) {
    if (nvec % 2 != 0 || nvec < kPipeSplitMinVec || T < kPipeSplitMinRowsPerCta * grid)
        return 0;
    return std::min<int64_t>(T, grid / kPipeSplitDiv);
}

// workspace: zeroed counters for dynamic rows (bulk-copy geometry with
// dynamic_rows set), else ignored.
int launch(const Plan &p, void *out, const void *in, int64_t T, int64_t d, int64_t rs,
           double z, cudaStream_t stream, void *workspace = nullptr, int64_t withhold = -1,
           unsigned long long wait_ns = kWaitLimitNs) {
    uint16_t *o = static_cast<uint16_t *>(out);
    const uint16_t *x = static_cast<const uint16_t *>(in);
    const float zf = static_cast<float>(z);
    const int di = static_cast<int>(d);
    const gated_act_plan &q = p.pub;
    const dim3 grid(static_cast<unsigned>(q.grid)), block(q.threads);
    cudaError_t e = cudaSuccess;
    switch (q.variant) {
    case GATED_ACT_VARIANT_TMA_ROWS: {
        TmaFn fn = tma_fn(q.threads);
        if (!fn)
            return GATED_ACT_ERR_VARIANT;
        const int rc = ensure_smem_attr(fn, 31 - __builtin_clz(static_cast<unsigned>(q.threads)));
        if (rc != GATED_ACT_OK)
            return rc;
        unsigned long long *sched =
            q.dynamic_rows ? static_cast<unsigned long long *>(workspace) : nullptr;
        e = launch_kernel(fn, grid, block, static_cast<size_t>(q.smem_bytes), stream, 1, o, x, T,
                          di, rs, zf, static_cast<int>(q.stages), sched, withhold, wait_ns);
        break;
    }
    case GATED_ACT_VARIANT_PIPE_ROWS: {
        const int ncw = q.threads / 32 - 1;
        PipeFn fn = pipe_fn(ncw, q.vec_per_thread);
        if (!fn)
            return GATED_ACT_ERR_VARIANT;
        const int rc = ensure_smem_attr(fn, 16 + ncw / 4 + q.vec_per_thread);
        if (rc != GATED_ACT_OK)
            return rc;
        unsigned long long *sched =
            q.dynamic_rows ? static_cast<unsigned long long *>(workspace) : nullptr;
        const int64_t split = sched ? pipe_split_rows(T, d / 8, q.grid) : 0;
        e = launch_kernel(fn, grid, block, static_cast<size_t>(q.smem_bytes), stream, 1, o, x, T,
                          di, rs, zf, static_cast<int>(q.stages), sched, split, withhold,
                          wait_ns);
        break;
    }
    case GATED_ACT_VARIANT_WARP_ROWS:
        e = launch_kernel(warp_fn(q.vec_per_thread), grid, block, 0, stream, 1, o, x, T, di, rs, zf);
        break;
    case GATED_ACT_VARIANT_SPLIT_ROWS: {
        CtaFn fn = split_fn(q.threads, p.su, p.dtype, p.native);
        if (!fn)
            return GATED_ACT_ERR_VARIANT;
        e = launch_kernel(fn, grid, block, 0, stream, 1, out, in, T, di, rs, zf,
                          static_cast<int>(q.cluster), p.sv);
        break;
    }
    case GATED_ACT_VARIANT_CTA_ROW: {
        CtaFn fn = cta_fn(q.threads, q.vec_per_thread, q.cluster, p.dtype, p.native);
        if (!fn)
            return GATED_ACT_ERR_VARIANT;
        e = launch_kernel(fn, grid, block, 0, stream, q.cluster, out, in, T, di, rs, zf,
                          static_cast<int>(q.cluster), p.sv);
        break;
    }
    default:
        e = launch_kernel(scalar_fn(p.dtype, p.native), grid, block, 0, stream, 1, out, in, T, d,
                          rs, zf);
        break;
    }
    if (e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace gact

extern "C" int gelu_and_mul_sparse_plan_ex(const void *out, const void *in, int64_t T,
                                           int64_t d, int64_t row_stride, int dtype, int variant,
                                           int cluster, int sm_count, int with_workspace,
                                           gated_act_plan *plan) {
    if (!plan)
        return GATED_ACT_ERR_NULL;
    // A buffer in page-locked host memory rules out the bulk-copy geometry, as
    // at launch; a pointer the runtime cannot classify (no device, or not yet
    // allocated) plans as device memory.
    bool host = false;
    for (const void *q : {out, in}) {
        const void *dq;
        bool h = false;
        if (q && gact::resolve_ptr(q, &dq, &h) == GATED_ACT_OK)
            host = host || h;
    }
    gact::Plan p;
    const int rc = gact::make_plan(out, in, T, d, row_stride, dtype, variant, cluster, sm_count,
                                   false, &p, false, host, with_workspace != 0);
    if (rc != GATED_ACT_OK)
        return rc;
    *plan = p.pub;
    return GATED_ACT_OK;
}

extern "C" int gelu_and_mul_sparse_native_plan(const void *out, const void *in, int64_t T,
                                               int64_t d, int64_t row_stride, int dtype,
                                               int sm_count, gated_act_plan *plan) {
    if (!plan)
        return GATED_ACT_ERR_NULL;
    bool host = false;
    for (const void *q : {out, in}) {
        const void *dq;
        bool h = false;
        if (q && gact::resolve_ptr(q, &dq, &h) == GATED_ACT_OK)
            host = host || h;
    }
    gact::Plan p;
    const int rc = gact::make_plan(out, in, T, d, row_stride, dtype, GATED_ACT_VARIANT_AUTO, 0,
                                   sm_count, false, &p, true, host, false);
    if (rc != GATED_ACT_OK)
        return rc;
    *plan = p.pub;
    return GATED_ACT_OK;
}

extern "C" int gelu_and_mul_sparse_plan(const void *out, const void *in, int64_t T, int64_t d,
                                        int64_t row_stride, int dtype, int variant, int cluster,
                                        int sm_count, gated_act_plan *plan) {
    return gelu_and_mul_sparse_plan_ex(out, in, T, d, row_stride, dtype, variant, cluster,
                                       sm_count, 0, plan);
}

namespace gact {
namespace {
// Validate, resolve host buffers, plan and launch one gelu_and_mul_sparse
// call.  ws: the caller's workspace (gelu_and_mul_sparse_ws) or nullptr.
// plan_ws: plan as a call with a workspace even though ws is null (a
// no-allocation call whose plan takes no rows from a counter).
int run_gelu(void *out, const void *in, int64_t T, int64_t d, int64_t rs, double z, int dtype,
             int variant, int cluster, bool native, cudaStream_t stream,
             void *ws = nullptr, bool plan_ws = false) {
    const bool has_ws = ws != nullptr || plan_ws;
    Plan p;
    int rc = make_plan(out, in, T, d, rs, dtype, variant, cluster, 0, true, &p, native, false,
                       has_ws);
    if (rc != GATED_ACT_OK)
        return rc;
    if (plan_ws && !ws && p.pub.dynamic_rows)
        return GATED_ACT_ERR_NULL;   // such a plan needs the counters
    if (ws) {
        if (!aligned(ws, 8))
            return GATED_ACT_ERR_ALIGN;
        const int elem = elem_bytes(dtype);
        const uint64_t in_bytes = T > 0 ? elem * static_cast<uint64_t>((T - 1) * rs + 2 * d) : 0;
        const uint64_t out_bytes = elem * static_cast<uint64_t>(T * d);
        if (ranges_overlap(ws, kWorkspaceBytes, in, in_bytes) ||
            ranges_overlap(ws, kWorkspaceBytes, out, out_bytes))
            return GATED_ACT_ERR_OVERLAP;
    }
    if (T == 0)
        return GATED_ACT_OK;
    if (ws) {   // the counters are updated with atomics: device memory only
        const void *dws;
        bool hws;
        if ((rc = resolve_ptr(ws, &dws, &hws)) != GATED_ACT_OK)
            return rc;
        if (hws)
            return GATED_ACT_ERR_HOST;
    }
    const void *dout, *din;
    bool hout, hin;
    if ((rc = resolve_ptr(out, &dout, &hout)) != GATED_ACT_OK ||
        (rc = resolve_ptr(in, &din, &hin)) != GATED_ACT_OK)
        return rc;
    if (hout || hin) {
        rc = make_plan(dout, din, T, d, rs, dtype, variant, cluster, 0, true, &p, native, true,
                       has_ws);
        if (rc != GATED_ACT_OK)
            return rc;
    }
    return launch(p, const_cast<void *>(dout), din, T, d, rs, z, stream, ws);
}
}  // namespace
}  // namespace gact

extern "C" int gelu_and_mul_sparse_typed(void *out, const void *in, int64_t T, int64_t d,
                                         int64_t row_stride, double z, int dtype, int variant,
                                         int cluster, cudaStream_t stream) {
    return gact::run_gelu(out, in, T, d, row_stride, z, dtype, variant, cluster, false, stream);
}

extern "C" int gelu_and_mul_sparse_native(void *out, const void *in, int64_t T, int64_t d,
                                          int64_t row_stride, double z, int dtype,
                                          cudaStream_t stream) {
    return gact::run_gelu(out, in, T, d, row_stride, z, dtype, GATED_ACT_VARIANT_AUTO, 0, true,
                          stream);
}

extern "C" int gelu_and_mul_sparse_ex(void *out, const void *in, int64_t T, int64_t d,
                                      int64_t row_stride, double z, int variant, int cluster,
                                      cudaStream_t stream) {
    return gelu_and_mul_sparse_typed(out, in, T, d, row_stride, z, GATED_ACT_BF16, variant,
                                     cluster, stream);
}

extern "C" int gelu_and_mul_sparse(void *out, const void *in, int64_t T, int64_t d,
                                   int64_t row_stride, double z, cudaStream_t stream) {
    return gelu_and_mul_sparse_typed(out, in, T, d, row_stride, z, GATED_ACT_BF16,
                                     GATED_ACT_VARIANT_AUTO, 0, stream);
}

extern "C" size_t gelu_and_mul_sparse_workspace_bytes(void) { return gact::kWorkspaceBytes; }

extern "C" int gelu_and_mul_sparse_ws(void *out, const void *in, int64_t T, int64_t d,
                                      int64_t row_stride, double z, int dtype, int variant,
                                      int cluster, void *workspace, cudaStream_t stream) {
    if (!workspace)
        return GATED_ACT_ERR_NULL;
    return gact::run_gelu(out, in, T, d, row_stride, z, dtype, variant, cluster, false, stream,
                          workspace);
}

// ------------------------------------------------------------ no-allocation variant
// gelu_and_mul_sparse_ws_static serves callers that cannot allocate device
// memory at all: an engine that reserved every free byte for its own pool at
// start-up, or a plugin host that hands a kernel nothing but its inputs and
// outputs.  For them even 16 bytes from cudaMalloc may fail, and cudaMalloc
// and cudaFree may synchronize the device.  So the row counters live in this
// library's own scratch array below.
namespace gact {
// 256 bytes on every GPU that loads the library, kept until the process
// exits; a call needs the first kWorkspaceBytes of it.  In host code this name
// is only a stand-in for the device array, never its address: host code gets
// the address from cudaGetSymbolAddress.
constexpr size_t kStaticScratchBytes = 256;
static __device__ __align__(256) unsigned long long g_static_scratch[kStaticScratchBytes / 8];

namespace {
// Device address of g_static_scratch in the current device's current context.
// A symbol's device address belongs to one context, so the address is looked
// up once per (device, context): the first call in a context does it, and a
// new context (after cudaDeviceReset, or a context the caller made current)
// gets a fresh lookup.  Where the context id is unavailable the address is
// looked up on every call.
int static_scratch(void **addr) {
    constexpr int kMaxDevices = 64;
    struct Entry {
        unsigned long long ctx;
        void *ptr;
    };
    static Entry cache[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_status(e);
    const bool slot = dev >= 0 && dev < kMaxDevices;
    unsigned long long ctx = current_context_id();
    if (slot && ctx != 0) {
        std::lock_guard<std::mutex> lock(mu);
        if (cache[dev].ctx == ctx && cache[dev].ptr) {
            *addr = cache[dev].ptr;
            return GATED_ACT_OK;
        }
    }
    void *p = nullptr;
    // makes the device's primary context current if no context is
    e = cudaGetSymbolAddress(&p, g_static_scratch);
    if (e != cudaSuccess)
        return cuda_status(e);
    if (ctx == 0)
        ctx = current_context_id();
    if (slot && ctx != 0) {
        std::lock_guard<std::mutex> lock(mu);
        cache[dev] = Entry{ctx, p};
    }
    *addr = p;
    return GATED_ACT_OK;
}
}  // namespace
}  // namespace gact

extern "C" int gelu_and_mul_sparse_ws_static(void *out, const void *in, int64_t T, int64_t d,
                                             int64_t row_stride, double z, int dtype,
                                             int variant, int cluster, cudaStream_t stream) {
    gact::Plan p;
    int rc = gact::make_plan(out, in, T, d, row_stride, dtype, variant, cluster, 0, true, &p,
                             false, false, true);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    // scratch this call needs: the row counters, when rows are taken dynamically
    const size_t need = p.pub.dynamic_rows ? gact::kWorkspaceBytes : 0;
    if (need > gact::kStaticScratchBytes)
        return GATED_ACT_ERR_SCRATCH;
    if (need == 0)   // the array is neither read nor cleared
        return gact::run_gelu(out, in, T, d, row_stride, z, dtype, variant, cluster, false,
                              stream, nullptr, true);
    void *scratch = nullptr;
    if ((rc = gact::static_scratch(&scratch)) != GATED_ACT_OK)
        return rc;
    // every call shares the array: start from zeroed counters whatever the
    // last call left
    const cudaError_t e = cudaMemsetAsync(scratch, 0, gact::kWorkspaceBytes, stream);
    if (e != cudaSuccess)
        return gact::cuda_status(e);
    return gact::run_gelu(out, in, T, d, row_stride, z, dtype, variant, cluster, false, stream,
                          scratch);
}

extern "C" int gated_act_selftest_wait_timeout(void *out, const void *in, int64_t T, int64_t d,
                                              unsigned long long wait_ns, cudaStream_t stream) {
    if (wait_ns == 0 || wait_ns > gact::kWaitLimitNs)
        return GATED_ACT_ERR_SIZE;
    gact::Plan p;
    const int rc = gact::make_plan(out, in, T, d, 2 * d, GATED_ACT_BF16,
                                   GATED_ACT_VARIANT_TMA_ROWS, 0, 0, true, &p);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    // chunk 1 is the up half of each CTA's first row
    return gact::launch(p, out, in, T, d, 2 * d, 1.0, stream, nullptr, 1, wait_ns);
}

extern "C" int gated_act_selftest_wait_timeout_ws(void *out, const void *in, int64_t T,
                                                 int64_t d, unsigned long long wait_ns,
                                                 void *workspace, cudaStream_t stream) {
    if (wait_ns == 0 || wait_ns > gact::kWaitLimitNs)
        return GATED_ACT_ERR_SIZE;
    if (!workspace)
        return GATED_ACT_ERR_NULL;
    if (!gact::aligned(workspace, 8))
        return GATED_ACT_ERR_ALIGN;
    gact::Plan p;
    const int rc = gact::make_plan(out, in, T, d, 2 * d, GATED_ACT_BF16,
                                   GATED_ACT_VARIANT_TMA_ROWS, 0, 0, true, &p);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    // forced geometry: rows are taken dynamically; chunk 1 is the up half of
    // each CTA's first row
    return gact::launch(p, out, in, T, d, 2 * d, 1.0, stream, workspace, 1, wait_ns);
}

extern "C" int gated_act_selftest_wait_timeout_ex(void *out, const void *in, int64_t T,
                                                 int64_t d, unsigned long long wait_ns,
                                                 int variant, void *workspace,
                                                 cudaStream_t stream) {
    if (wait_ns == 0 || wait_ns > gact::kWaitLimitNs)
        return GATED_ACT_ERR_SIZE;
    if (variant != GATED_ACT_VARIANT_TMA_ROWS && variant != GATED_ACT_VARIANT_PIPE_ROWS)
        return GATED_ACT_ERR_VARIANT;
    if (workspace && !gact::aligned(workspace, 8))
        return GATED_ACT_ERR_ALIGN;
    gact::Plan p;
    const int rc = gact::make_plan(out, in, T, d, 2 * d, GATED_ACT_BF16, variant, 0, 0, true, &p);
    if (rc != GATED_ACT_OK || T == 0)
        return rc;
    // forced geometry: with a workspace rows are taken dynamically; chunk 1
    // is the up half of each CTA's first row
    return gact::launch(p, out, in, T, d, 2 * d, 1.0, stream, workspace, 1, wait_ns);
}

extern "C" int gated_act_device_status(unsigned int *flags) {
    if (!flags)
        return GATED_ACT_ERR_NULL;
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, gact::g_device_status, sizeof v);
    if (e != cudaSuccess)
        return gact::cuda_status(e);
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(gact::g_device_status, &zero, sizeof zero);
    if (e == cudaSuccess)
        e = gact::take_linear_act_status(&v);
    if (e == cudaSuccess)
        e = gact::take_cross_entropy_status(&v);
    if (e != cudaSuccess)
        return gact::cuda_status(e);
    *flags = v;
    return GATED_ACT_OK;
}
