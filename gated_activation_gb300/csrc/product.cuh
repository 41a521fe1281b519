// Matrix products on the tensor cores (tcgen05) with an epilogue of the caller's:
// the main loop of the linear_* operators.
//
// One persistent kernel, one cluster of two CTAs per pair of SMs.  A pair computes
// tiles of 256 x 256 elements of A B' (fp32 sums), 128 rows per CTA:
//   warp 0     loads 64 columns of both operands per step into a ring of shared
//              memory slots (TMA, 128-byte swizzle), in both CTAs;
//   warp 1     of the pair's first CTA issues the products (tcgen05.mma of the two
//              CTAs together, 256 x 256 x 16), whose sums lie in tensor memory;
//   warps 4-11 read finished sums back (of some jobs in parts, which they add up), a row
//              per thread and every second 32 columns, and run the epilogue while the
//              next tile is summed into the other half of the tensor memory.
// An operand is stored with its rows along the summed dimension (as the activations
// and weights of a linear layer are in its forward product) or across it (as they are
// in the products of its gradients); the TMA box and the descriptors differ, no data
// is transposed.  What lies outside a tensor is read as zeros.
//
// Why these sizes: a pair's step of 64 (256 x 256 x 64) takes 512 cycles of its tensor cores and 64 KB of
// copies, 64 bytes per cycle and SM from L2; a step of 128 columns takes 48 KB for half the products, and
// measured 0.59 to 0.68 of the time.  The ring's six slots are 3000 cycles, twice a copy's latency under load.
// Measured on GB300 (cuBLAS: 1.88 PFLOP/s in short runs, 1.72 under the power limit): 2048 x 32768 x 4096 in
// 285 us alone (1.93 PFLOP/s), 314 us in a stream of such calls; tensor cores active 89% of the cycles.
// Small products are bound by what is not overlapped: launch and allocation (2.5 us), the first copies, the
// last tile's epilogue (1 to 5 us).
//
// Every wait on an mbarrier gives up after a second (that for a sum's end later, by the sum's length); the kernel then
// sets its status bit, lets its copies land, frees its tensor memory and returns.  The allocation of tensor memory, which
// waits for earlier kernels on the SM, and the barriers of the pair have no form with a limit: what keeps the pair
// together there is that each CTA reaches all of them, since its other waits end.
#pragma once

#include <cuda.h>

#include "training.cuh"

namespace gact {

constexpr int kTile = 256;            // rows of a pair's tile, and most columns
constexpr int kHalf = kTile / 2;      // rows of one CTA's part
constexpr int kStep = 64;             // summed elements per ring slot: 128 bytes
constexpr int kRowBytes = kHalf * kStep * 2;   // of the first operand in a slot
constexpr int kRingBytes = 6 * 2 * kRowBytes;
constexpr int kMostSlots = 10;
constexpr int kMaxBatches = 1024;
constexpr int kProductThreads = 384;

// A slot of a job with N columns per tile: each CTA brings half of the second operand's rows.
template <int N> constexpr int kSlotBytes = kRowBytes + N / 2 * kStep * 2;
template <int N> constexpr int kSlots =
    kRingBytes / kSlotBytes<N> < kMostSlots ? kRingBytes / kSlotBytes<N> : kMostSlots;
constexpr unsigned long long kProductWaitNs = 1000000000ull;

static __device__ unsigned int g_product_status;   // of this translation unit

// ------------------------------------------------------------- barriers, copies

__device__ __forceinline__ uint32_t smem_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// The address of the same variable in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t a) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}
// True in one lane of a converged warp.  (Of this form the compiler knows that one lane is left, and
// keeps the operands of the copies and products in uniform registers; under `lane == 0` each took a loop
// over the lanes, and a step's instructions 500 cycles, as long as its products.)
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for the phase `parity` of `bar`; false once a wait of this CTA gave up, after a second and 20 us
// for each of `steps` ring steps that it may have to wait for (0.3 us is what one takes).
static __device__ __noinline__ bool barrier_wait_slow(uint32_t bar, uint32_t parity,
                                                      volatile uint32_t *gave_up, int steps) {
    const unsigned long long t0 = now_ns();
    for (uint32_t i = 1;; ++i) {
        if (barrier_try(bar, parity))
            return true;
        if ((i & 63u) == 0) {
            if (*gave_up)
                return false;
            if (now_ns() - t0 > kProductWaitNs + 20000ull * static_cast<uint32_t>(steps)) {
                *gave_up = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity,
                                             volatile uint32_t *gave_up, int steps = 0) {
    return barrier_try(bar, parity) || barrier_wait_slow(bar, parity, gave_up, steps);
}

// One box of a 4-D tensor into this CTA's shared memory; its bytes count on `bar` of
// the pair's first CTA.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                         int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// ------------------------------------------------------------- tensor cores

// Shared memory descriptor of an operand's slot (PTX ISA, "Shared memory descriptor"), 128-byte
// swizzle.  Rows along the sum: 8 rows of 128 bytes every 1024 bytes.  Rows across it: 8 summed
// elements every 1024 bytes, 64 rows every 64 summed elements x 128 bytes.
template <bool ACROSS> __device__ __forceinline__ uint64_t slot_descriptor(uint32_t address) {
    constexpr uint64_t lead = ACROSS ? (kStep * 128) >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t((address & 0x3FFFF) >> 4)) | lead << 16 | stride << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// What 16 summed elements add to it.
template <bool ACROSS> constexpr uint64_t kDescriptorStep = (ACROSS ? 16 * 128 : 16 * 2) >> 4;

// Instruction descriptor (PTX ISA, "Instruction descriptor", kind::f16): fp32 sums of 256 x N.
template <class T, int N, bool A_ACROSS, bool B_ACROSS>
__host__ __device__ constexpr uint32_t product_descriptor() {
    constexpr uint32_t type = std::is_same_v<T, bf16> ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | uint32_t(A_ACROSS) << 15 | uint32_t(B_ACROSS) << 16 |
           uint32_t(N / 8) << 17 | uint32_t(kTile / 16) << 24;
}
__device__ __forceinline__ void product_step(uint32_t sums, uint64_t a, uint64_t b, uint32_t desc,
                                             bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(sums), "l"(a), "l"(b), "r"(desc), "r"(uint32_t(add))
        : "memory");
}
// Arrives on `bar` of both CTAs once the products issued so far are done.
__device__ __forceinline__ void product_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar), "h"(uint16_t(3))
        : "memory");
}
__device__ __forceinline__ void sums_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void sums_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of the warp's 32 rows: v[i] is column i of the lane's row.
__device__ __forceinline__ void sums_load32(uint32_t address, float (&v)[32]) {
    uint32_t r[32];
    __syncwarp();   // the instruction is the whole warp's
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(address));
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}
// Waits for the loads; `v`, what one of them gave, is not used before.
__device__ __forceinline__ void sums_ready(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                   "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                   "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}
// G times 32 columns, 64 apart, added to v: 16 columns are on their way while the 16 before are added.
__device__ __forceinline__ void sums_load16(uint32_t address, float (&v)[16]) {
    uint32_t r[16];
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(address));
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void sums_ready(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                   "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
template <int G> __device__ __forceinline__ void sums_add(uint32_t address, float (&v)[G][32]) {
    float x[2][16];
    sums_load16(address, x[0]);
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
        sums_ready(x[i & 1]);
        if (i + 1 < 2 * G)
            sums_load16(address + (i + 1) / 2 * 64 + (i + 1) % 2 * 16, x[(i + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float *to = v[i / 2] + i % 2 * 16 + j;
            const float2 y = add2({to[0], to[1]}, {x[i & 1][j], x[i & 1][j + 1]});
            to[0] = y.x;
            to[1] = y.y;
        }
    }
}

// ------------------------------------------------------------- the kernel

// One tile of a pair: batch, first row, number of the column tile, rows of the batch, ring steps,
// live count of the batch (not read again for each step: that stalled the copies), batches.
struct Tile {
    int b, m0, n0, rows, steps, live, batches;
    bool second;   // of the job's second product
};

// A second product of a job: its first operand's rows lie across the sum, over the live counts.
struct Second {
    int batches = 0, m_tiles = 0, n_tiles = 0, rows = 0;
};

// A job J describes a product and what happens to it:
//   J::Elem                      bf16 or f16
//   J::kBAcross                  the second operand's rows lie across the sum (the first product's first ones along it)
//   J::kN                        columns of a tile
//   J::kRows                     rows that a tile counts for
//   J::Args                      what its functions read
//   J::kLive                     what the live counts bound
//   J::kSecond                   whether there is a second product (Second), whose tiles follow the
//                                first's: in one launch the SM pairs share both out more evenly
//   J::batch_of(g, b, second)    index of the live count of a batch
//   J::batches(g)                how many there are, of at most g.batches
//   J::steps_of(g, tile)         ring steps of a tile of the first product
//   J::second_steps(g, live)     with kSecond: those of a second tile
//   J::load(g, tile, step, rank, a, b, bar)   issues the step's copies of one CTA
//   J::finish(g, tile, row, sums, stage)      the epilogue of a warp's 32 rows: `row` is the
//                                lane's (of the tile, in [0, 256)), `sums` the tensor memory
//                                address of its columns, `stage` the warp's shared memory
//   J::kClosed                   ring steps after which a sum is closed: the tensor cores begin the next one at 0,
//                                and the epilogue's threads add them up, with rounding; `sums` are then the results,
//                                [i][...] those of 32 columns from 32 part + 64 i on.  0: sums are never closed
enum class Live { Rows, Columns };

template <class J> struct Product {
    CUtensorMap a, b;
    const int32_t *live;   // null: `capacity` everywhere
    int batches, capacity, rows, n_tiles, steps;
    Second second;
    typename J::Args j;

    __device__ int live_of(int b) const {
        return live ? min(max(live[b], 0), capacity) : capacity;
    }
};

// Where a warp turns 32 columns of its 32 rows, a row per thread, into row segments; rows are 80
// bytes apart, so that neither side has bank conflicts.
constexpr int kStageRow = 32 * 2 + 16;
struct ProductShared;
struct Stage {
    uint8_t *p;
    ProductShared &s;
    int part;         // which of the tile's 32 columns the warp takes: every second, from this one on
    uint32_t &uses;   // of the part's hand-over buffer
    // Writes n columns (of 32), two to a word of the lane's row, of the first `rows` of the 32 rows to
    // `to`, `stride` elements apart.  `vec`: addresses, strides and n are multiples of 16 bytes; a warp then
    // writes eight rows' 64 bytes at a time.  Else a row's at a time, element by element.
    __device__ __forceinline__ void flush(const uint32_t (&w)[16], void *to, int64_t stride, int rows, int n,
                                          bool vec) const {
        const int lane = threadIdx.x & 31;
        uint16_t *out = static_cast<uint16_t *>(to);
        uint4 *mine = reinterpret_cast<uint4 *>(p + lane * kStageRow);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
        if (vec) {
            const int c = (lane & 3) * 8;
            out += (lane >> 2) * stride + c;
#pragma unroll
            for (int i = 0; i < 4; ++i, out += 8 * stride) {
                const int row = 8 * i + (lane >> 2);
                if (row < rows && c < n)
                    st_vec_out(out, *reinterpret_cast<const uint4 *>(p + row * kStageRow + 2 * c));
            }
        } else {
            // sixteen reads on their way before the first write, which they cannot pass
            out += lane;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 16) {
                uint16_t v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = *reinterpret_cast<const uint16_t *>(p + (r0 + i) * kStageRow + 2 * lane);
#pragma unroll
                for (int i = 0; i < 16; ++i, out += stride)
                    if (r0 + i < rows && lane < n)
                        out[0] = v[i];
            }
        }
        __syncwarp();
    }
};

struct alignas(16) ProductShared {
    uint8_t stage[8][32 * kStageRow];
    uint64_t full[kMostSlots], empty[kMostSlots], sums_full[2], sums_empty[2], swap_full[2], swap_empty[2];
    uint32_t sums;             // tensor memory address
    volatile uint32_t gave_up;
    int first[kMaxBatches + 1];   // first tile row of each batch
};
constexpr size_t kProductShared = kRingBytes + sizeof(ProductShared) + 1024;

constexpr int kTallest = 8;   // tile rows that are walked together, so that the tiles of a wave
                              // share rows and columns in L2

// The tiles of one pair, in order.
template <class J> struct Walk {
    const Product<J> &g;
    const ProductShared &s;
    int at, step, b = 0, batches, total, turn = 0;
    __device__ Walk(const Product<J> &g_, const ProductShared &s_)
        : g(g_), s(s_), at(blockIdx.x >> 1), step(gridDim.x >> 1), batches(J::batches(g_)),
          total(s_.first[batches]) {}
    // The r-th tile of a batch `tall` tiles high.
    __device__ void place(Tile *t, int r, int tall, int n_tiles) const {
        const int group = r / (kTallest * n_tiles), top = group * kTallest;
        const int high = min(kTallest, tall - top), rest = r - top * n_tiles;
        t->m0 = (top + rest % high) * J::kRows;
        t->n0 = rest / high;
    }
    __device__ bool next(Tile *t) {
        t->batches = batches;
        t->second = false;
        if (at < total * g.n_tiles) {
            while (s.first[b + 1] * g.n_tiles <= at)
                ++b;
            t->b = b;
            place(t, at - s.first[b] * g.n_tiles, s.first[b + 1] - s.first[b], g.n_tiles);
            t->live = g.live_of(J::batch_of(g, b, false));
            t->rows = J::kLive == Live::Rows ? t->live : g.rows;
            t->steps = J::steps_of(g, *t);
            at += step;
            return true;
        }
        if constexpr (J::kSecond) {
            // Where some pairs have a first tile more than others, the others take second tiles for it
            // before all go on in turns.
            const int left = total * g.n_tiles % step, mine = blockIdx.x >> 1;
            const int others = left ? step - left : 0, each = g.second.m_tiles * g.second.n_tiles;
            const int live = J::kLive == Live::Rows ? total * J::kRows / max(batches, 1) : 0;
            int ahead = 0;   // second tiles for a first one
            if (others) {
                Tile f = *t;
                f.b = 0;
                f.live = live;
                ahead = J::steps_of(g, f) / max(J::second_steps(g, min(live, g.capacity)), 1);
                ahead = min(ahead, g.second.batches * each / others + 1);
            }
            const bool other = mine >= left && others;
            int r;
            if (other && turn < ahead)
                r = mine - left + turn * others;
            else
                r = ahead * others + (mine >= left ? mine - left : mine + step - left) +
                    (turn - (other ? ahead : 0)) * step;
            ++turn;
            if (r >= g.second.batches * each)
                return false;
            t->second = true;
            t->b = r / each;
            place(t, r % each, g.second.m_tiles, g.second.n_tiles);
            t->live = g.live_of(J::batch_of(g, t->b, true));
            t->rows = g.second.rows;
            t->steps = J::second_steps(g, t->live);
            return true;
        }
        return false;
    }
};

template <class J>
__global__ void __launch_bounds__(kProductThreads, 1) product_kernel(const __grid_constant__ Product<J> g) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_address(raw) + 1023u) & ~1023u;   // the swizzle's period
    constexpr int SLOTS = kSlots<J::kN>, SLOT = kSlotBytes<J::kN>;
    ProductShared &s =
        *reinterpret_cast<ProductShared *>(raw + (base - smem_address(raw)) + kRingBytes);
    const uint32_t full = smem_address(s.full), empty = smem_address(s.empty),
                   sums_full = smem_address(s.sums_full), sums_empty = smem_address(s.sums_empty);
    const uint32_t rank = cluster_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            barrier_init(full + 8 * i, 1);
            barrier_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            barrier_init(sums_full + 8 * i, 1);
            barrier_init(sums_empty + 8 * i, 16);   // eight epilogue warps of each CTA
            barrier_init(smem_address(&s.swap_full[i]), 2);
            barrier_init(smem_address(&s.swap_empty[i]), 2);
        }
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Both CTAs run before either allocates: an allocation for the pair while the other CTA had
    // not started left that one's own allocation waiting for ever.
    __syncthreads();
    cluster_barrier();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                     ::"r"(smem_address(&s.sums))
                     : "memory");
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 3) {
        int sum = 0;
        const int batches = J::batches(g);
        for (int b0 = 0; b0 < batches; b0 += 32) {
            const int b = b0 + lane;
            int n = 0;
            if (b < batches)
                n = ((J::kLive == Live::Rows ? g.live_of(J::batch_of(g, b, false))
                      : J::kLive == Live::Columns && g.live_of(J::batch_of(g, b, false)) == 0 ? 0 : g.rows) +
                     J::kRows - 1) / J::kRows;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, n, o);
                if (lane >= o)
                    n += up;
            }
            if (b < batches)
                s.first[b + 1] = sum + n;
            sum += __shfl_sync(0xFFFFFFFFu, n, 31);
        }
        if (lane == 0)
            s.first[0] = 0;
    }
    // The first CTA's products write the other's tensor memory, but they wait for its copies,
    // which it issues after this.
    sums_fence_before();
    __syncthreads();
    sums_fence_after();
    const uint32_t sums = s.sums;

    Walk<J> walk(g, s);
    Tile t;
    if (warp == 0 && elected()) {
        // the first CTA's barrier counts both CTAs' bytes
        const uint32_t first_full = in_first_cta(full);
        // what the kernels before wrote, to the copies of this one
        asm volatile("fence.proxy.async.global;" ::: "memory");
        uint32_t slot = 0, phase = 0;
        bool ok = true;
        while (ok && walk.next(&t))
            for (int k = 0; k < t.steps; ++k) {
                if (!(ok = barrier_wait(empty + 8 * slot, phase ^ 1, &s.gave_up)))
                    break;
                const uint32_t to = base + slot * SLOT;
                if (rank == 0)
                    barrier_expect(full + 8 * slot, 2 * SLOT);
                J::load(g, t, k, rank, to, to + kRowBytes, first_full + 8 * slot);
                if (++slot == SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        // every use of a slot is over (at once for one never used): nothing arrives at this CTA's
        // barriers after its end
        for (int i = 0; ok && i < SLOTS; ++i) {
            ok = barrier_wait(empty + 8 * slot, phase ^ 1, &s.gave_up);
            if (++slot == SLOTS) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1 && rank == 0 && elected()) {
        constexpr uint32_t first = product_descriptor<typename J::Elem, J::kN, false, J::kBAcross>();
        constexpr uint32_t second = product_descriptor<typename J::Elem, J::kN, true, J::kBAcross>();
        uint32_t slot = 0, phase = 0, turn = 0;
        bool ok = true;
        while (ok && walk.next(&t)) {
            const bool across = J::kSecond && t.second;
            const uint64_t a0 = across ? slot_descriptor<true>(base) : slot_descriptor<false>(base),
                           b0 = slot_descriptor<J::kBAcross>(base + kRowBytes),
                           turn16 = across ? kDescriptorStep<true> : kDescriptorStep<false>;
            const uint32_t desc = across ? second : first;
            int k = 0;
            do {
                const uint32_t half = turn++ & 1, to = sums + half * kTile;
                if (!(ok = barrier_wait(sums_empty + 8 * half, ((turn - 1) >> 1 & 1) ^ 1, &s.gave_up)))
                    break;
                sums_fence_after();
                const int begin = k, end = J::kClosed ? min(k + J::kClosed, t.steps) : t.steps;
                for (; k < end; ++k) {
                    if (!(ok = barrier_wait(full + 8 * slot, phase, &s.gave_up)))
                        break;
                    sums_fence_after();
                    const uint64_t at = slot * (SLOT >> 4);
#pragma unroll
                    for (int i = 0; i < kStep / 16; ++i)
                        product_step(to, a0 + at + i * turn16, b0 + at + i * kDescriptorStep<J::kBAcross>,
                                     desc, k > begin || i > 0);
                    product_commit(empty + 8 * slot);
                    if (++slot == SLOTS) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (ok)
                    product_commit(sums_full + 8 * half);
            } while (ok && k < t.steps);
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3;   // the tensor memory lanes that the warp may read
        uint32_t turn = 0, uses = 0;
        const int row = static_cast<int>(rank) * kHalf + quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const Stage stage{s.stage[warp - 4], s, (warp >> 2) - 1, uses};
        const auto taken = [&](uint32_t half) {   // the sums are read
            sums_fence_before();
            __syncwarp();
            if (lane == 0)
                barrier_arrive_cluster(in_first_cta(sums_empty + 8 * half));
            ++turn;
        };
        while (walk.next(&t)) {
            if constexpr (J::kClosed > 0) {
                constexpr int groups = (J::kN + 63) / 64;
                float v[groups][32] = {};
                bool ok = true;
                for (int k = 0; k < t.steps; k += J::kClosed) {
                    const uint32_t half = turn & 1;
                    if (!(ok = barrier_wait(sums_full + 8 * half, (turn >> 1) & 1, &s.gave_up, J::kClosed)))
                        break;
                    sums_fence_after();
                    if (32 * stage.part < J::kN)
                        sums_add<groups>(sums + half * kTile + lanes + 32 * stage.part, v);
                    taken(half);
                }
                if (!ok)
                    break;
                J::finish(g, t, row, v, stage);
            } else {
                const uint32_t half = turn & 1;
                if (!barrier_wait(sums_full + 8 * half, (turn >> 1) & 1, &s.gave_up, t.steps))
                    break;
                sums_fence_after();
                J::finish(g, t, row, sums + half * kTile + lanes, stage);
                taken(half);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (s.gave_up) {
        // copies in flight land well within this time
        if (threadIdx.x == 0)
            atomicOr(&g_product_status, 1u);
        const unsigned long long t0 = now_ns();
        for (int i = 0; i < 1000000 && now_ns() - t0 < 5000000ull; ++i)
            ;
    }
    __syncthreads();
    cluster_barrier();
    if (warp == 2) {
        sums_fence_after();
        // not earlier: the right to allocate is the pair's
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(sums) : "memory");
    }
    __syncthreads();
    cluster_barrier();
}

// What an epilogue is given: its sums' address, or closed sums.
template <int CLOSED, int N>
using Sums = std::conditional_t<CLOSED == 0, const uint32_t, float[(N + 63) / 64][32]>;

// f(c, v) for the warp's groups of 32 columns c that begin below n (at most N).
template <int CLOSED, int N, class F>
__device__ __forceinline__ void for_columns(Sums<CLOSED, N> &sums, int part, int n, F f) {
    if constexpr (CLOSED == 0) {
        for (int c = 32 * part; c < N && c < n; c += 64) {
            float v[32];
            sums_load32(sums + c, v);
            sums_ready(v);
            f(c, v);
        }
    } else if constexpr (N <= kHalf) {
        // not unrolled, the groups move up instead: a short call waits for its instructions (64 x 32000 x 1024
        // 12.9 us, unrolled 14.8)
#pragma unroll 1
        for (int c = 32 * part; c < N && c < n; c += 64) {
            f(c, sums[0]);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                for (int group = 1; group < (N + 63) / 64; ++group)
                    sums[group - 1][i] = sums[group][i];
        }
    } else {
#pragma unroll
        for (int group = 0; group < N / 64; ++group) {
            const int c = 32 * part + 64 * group;
            if (c < n)
                f(c, sums[group]);
        }
    }
}

// ------------------------------------------------------------- loads, stores

// The box's operand rows from `row` on, summed elements from `x` on.
__device__ __forceinline__ void load_along(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                           int x, int row, int z, int w) {
    box_load(dst, map, bar, x, row, z, w);
}
// The same of `ROWS` (64 or 128) rows of an operand whose rows lie across the sum.
template <int ROWS = kHalf>
__device__ __forceinline__ void load_across(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int row, int z, int w) {
    static_assert(ROWS == 64 || ROWS == 128);
    box_load(dst, map, bar, row, x, z, w);
    if (ROWS == 128)
        box_load(dst + kStep * 128, map, bar, row + 64, x, z, w);
}

// Eight elements at any address of theirs (with `vec` one of 16 bytes), zeros from the n-th on.
template <class T> __device__ __forceinline__ uint4 eight(const T *p, int n, bool vec) {
    if (vec && n >= 8)
        return ld_stream(p);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < n ? ld_stream_u16(reinterpret_cast<const uint16_t *>(p) + i) : 0;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

// The same of columns [c, c + 8) of a row of n, where `row + c` is a multiple of 16 bytes: zeros outside of the row.
template <class T> __device__ __forceinline__ uint4 eight_around(const T *row, int c, int n) {
    if (c >= 0 && c + 8 <= n)
        return ld_stream(row + c);
    const int first = max(c, 0), last = min(c + 8, n);
    return first < last ? eight(row + first, last - first, false) : make_uint4(0, 0, 0, 0);
}
// The elements of a row's first such vector that lie in front of the row.
template <class T> __device__ __forceinline__ int before_row(const T *row) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
}
// The largest finite magnitude of eight fp16 elements.  Magnitudes of one type order as their bits.
__device__ __forceinline__ float top_of_eight(uint4 v) {
    uint32_t most = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t lo = (&v.x)[q] & 0x7FFFu, hi = (&v.x)[q] >> 16 & 0x7FFFu;
        most = max(most, max(lo < 0x7C00u ? lo : 0u, hi < 0x7C00u ? hi : 0u));
    }
    return __half2float(__ushort_as_half(static_cast<unsigned short>(most)));
}

template <class T> __device__ __forceinline__ uint32_t pack2(float2 v);
template <> __device__ __forceinline__ uint32_t pack2<bf16>(float2 v) { return pack_bf16x2(v.x, v.y); }
template <> __device__ __forceinline__ uint32_t pack2<f16>(float2 v) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 32 values, each rounded once, as words for a Stage.
template <class T> __device__ __forceinline__ void pack32(uint32_t (&w)[16], const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i] = pack2<T>({v[2 * i], v[2 * i + 1]});
}

// The epilogue of a plain product: every column of the tile below `columns`, times `scale`, rounded
// to T, into the warp's first `rows` rows at `to`, `stride` apart.  A sum without terms is 0 whatever
// tensor memory holds.
template <int N, class T>
__device__ __forceinline__ void store_tile(uint32_t sums, const Stage &stage, T *to, int64_t stride, int rows,
                                           int columns, bool vec, float scale, bool zero) {
    for (int c = 32 * stage.part; c < N && c < columns; c += 64) {
        float v[32];
        uint32_t w[16];
        sums_load32(sums + c, v);
        sums_ready(v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = zero ? 0.f : v[i] * scale;
        pack32<T>(w, v);
        stage.flush(w, to + c, stride, rows, columns - c, vec);
    }
}

// ------------------------------------------------------------- host side

// A tensor of up to four dimensions, innermost first; strides in elements of two bytes.
struct Layout {
    const void *data;
    int64_t size[4], stride[4];   // stride[0] = 1
};

// Whether a TMA copy can address it: 16-byte rows, planes and base.
bool tma_addressable(const Layout &t);

// The tensor map of boxes of 64 x `rows` elements.
int encode_map(CUtensorMap *map, const Layout &t, int rows, bool is_bf16);

// The layout of a copy of `t` at `data` whose rows are padded to 16 bytes.
Layout packed_layout(const Layout &t, void *data);
inline uint64_t packed_bytes(const Layout &t) {
    return static_cast<uint64_t>(ceil_div64(t.size[0], 8)) * 16 * t.size[1] * t.size[2] * t.size[3];
}
// Copies `from` into `to`, a packed_layout of it (and a second pair in the same launch); the padding is zeros.
int launch_pack(const Layout &to, const Layout &from, cudaStream_t stream);
int launch_pack(const Layout &to0, const Layout &from0, const Layout &to1, const Layout &from1,
                cudaStream_t stream);

// check_regions, and no buffer in host memory.
int check_device_regions(Region *r, int n);

// Parts of a workspace, each 128-byte aligned from its start; with a null start it
// only counts.
struct Carve {
    uint8_t *start;
    uint64_t used = 0;
    explicit Carve(void *p) : start(static_cast<uint8_t *>(p)) {}
    template <class T> T *take(uint64_t bytes) {
        T *p = start ? reinterpret_cast<T *>(start + used) : nullptr;
        used += (bytes + 127) / 128 * 128;
        return p;
    }
};

inline int sm_pairs() { return device_sm_count() > 1 ? device_sm_count() / 2 : 1; }

template <class J> int launch_product(const Product<J> &g, int64_t tiles, cudaStream_t stream) {
    auto kernel = product_kernel<J>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), kProductShared);
    if (e != cudaSuccess)
        return cuda_status(e);
    const int pairs = sm_pairs();
    const unsigned grid = 2u * static_cast<unsigned>(tiles < pairs ? (tiles < 1 ? 1 : tiles) : pairs);
    return cuda_status(launch_kernel(kernel, dim3(grid), dim3(kProductThreads), kProductShared, stream, 2, g));
}

// Reads and clears this translation unit's status.
static inline cudaError_t take_product_status(unsigned int *flags) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_product_status, sizeof v);
    if (e != cudaSuccess)
        return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_product_status, &zero, sizeof zero);
    *flags |= v;
    return e;
}

}  // namespace gact
