// Tensor maps for the products' operands, and copies of those that TMA cannot address.
#include "product.cuh"

namespace gact {

bool tma_addressable(const Layout &t) {
    if (!aligned(t.data, 16))
        return false;
    for (int i = 1; i < 4; ++i)   // whole 16 bytes, below 2^40 bytes
        if (t.size[i] > 1 && (t.stride[i] % 8 || t.stride[i] >= int64_t(1) << 39))
            return false;
    return true;
}

namespace {

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                            const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                            const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
    static const Encode f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        cudaGetLastError();   // a failed query is not sticky; leave no error behind
        return reinterpret_cast<Encode>(p);
    }();
    return f;
}

}  // namespace

int encode_map(CUtensorMap *map, const Layout &t, int rows, bool is_bf16) {
    const Encode encode = encoder();
    if (!encode)
        return cuda_status(cudaErrorNotSupported);
    cuuint64_t size[4], stride[3];
    const cuuint32_t box[4] = {kStep, static_cast<cuuint32_t>(rows), 1, 1}, one[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i)
        size[i] = static_cast<cuuint64_t>(t.size[i] < 1 ? 1 : t.size[i]);
    for (int i = 1; i < 4; ++i)   // the stride of a dimension of one has no meaning, but a rule
        stride[i - 1] = t.size[i] > 1 ? static_cast<cuuint64_t>(t.stride[i]) * 2 : 16;
    const CUresult r = encode(
        map, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
        const_cast<void *>(t.data), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GATED_ACT_OK : cuda_status(cudaErrorInvalidValue);
}

int check_device_regions(Region *r, int n) {
    const int rc = check_regions(r, n);
    if (rc != GATED_ACT_OK)
        return rc;
    for (int i = 0; i < n; ++i)
        if (r[i].host)
            return GATED_ACT_ERR_HOST;
    return GATED_ACT_OK;
}

Layout packed_layout(const Layout &t, void *data) {
    Layout p = t;
    p.data = data;
    p.stride[0] = 1;
    p.stride[1] = ceil_div64(t.size[0], 8) * 8;
    p.stride[2] = p.stride[1] * t.size[1];
    p.stride[3] = p.stride[2] * t.size[2];
    return p;
}

// The eight elements that start `off` bytes (even, below 16; the same in a warp) into two vectors.
__device__ __forceinline__ uint4 shifted8(uint4 lo, uint4 hi, uint32_t off) {
    const uint32_t pick = off & 2 ? 0x5432u : 0x3210u;
    switch (off >> 2) {
    case 0:
        return make_uint4(__byte_perm(lo.x, lo.y, pick), __byte_perm(lo.y, lo.z, pick),
                          __byte_perm(lo.z, lo.w, pick), __byte_perm(lo.w, hi.x, pick));
    case 1:
        return make_uint4(__byte_perm(lo.y, lo.z, pick), __byte_perm(lo.z, lo.w, pick),
                          __byte_perm(lo.w, hi.x, pick), __byte_perm(hi.x, hi.y, pick));
    case 2:
        return make_uint4(__byte_perm(lo.z, lo.w, pick), __byte_perm(lo.w, hi.x, pick),
                          __byte_perm(hi.x, hi.y, pick), __byte_perm(hi.y, hi.z, pick));
    default:
        return make_uint4(__byte_perm(lo.w, hi.x, pick), __byte_perm(hi.x, hi.y, pick),
                          __byte_perm(hi.y, hi.z, pick), __byte_perm(hi.z, hi.w, pick));
    }
}

// Eight elements and a 16-byte store per thread and row, a row's 256 elements per warp.  Rows off
// 16-byte boundaries are read as the aligned vectors that hold them (consecutive lanes share these
// through L1); where one of the two would reach past the tensor's own bytes, and at a row's end, element
// by element.  Bound by its instructions before the shift was made the warp's (50001 x 1001: 56 us).
// Two tensors share a launch: planes of the grid from `split` on are the second's.
__global__ void __launch_bounds__(256) pack_rows(Layout to0, Layout from0, Layout to1, Layout from1,
                                                 int split) {
    pdl_wait();
    pdl_trigger();
    const bool second = static_cast<int>(blockIdx.z) >= split;
    const Layout &to = second ? to1 : to0, &from = second ? from1 : from0;
    const int64_t plane = blockIdx.z - (second ? split : 0);
    const int64_t x = (int64_t(blockIdx.x) * 32 + threadIdx.x) * 8;
    if (x >= to.size[0])
        return;
    const int64_t z = plane % to.size[2], w = plane / to.size[2];
    const uintptr_t first = reinterpret_cast<uintptr_t>(from.data);
    const uintptr_t last = first + 2 * static_cast<uintptr_t>(
        (from.size[1] - 1) * from.stride[1] + (from.size[2] - 1) * from.stride[2] +
        (from.size[3] - 1) * from.stride[3] + from.size[0]) - 32;
    const bool whole = x + 8 <= to.size[0];
    int64_t r = int64_t(blockIdx.y) * 8 + threadIdx.y;
    const int64_t step = int64_t(gridDim.y) * 8;
    const uint16_t *p = static_cast<const uint16_t *>(from.data) + z * from.stride[2] +
                        w * from.stride[3] + r * from.stride[1] + x;
    uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(to.data)) +
                    (plane * to.size[1] + r) * to.stride[1] + x;
#pragma unroll 2
    for (; r < to.size[1]; r += step, p += step * from.stride[1], out += step * to.stride[1]) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
        uint4 v;
        if (whole && at >= first && at <= last) {
            const uint4 *vec = reinterpret_cast<const uint4 *>(at);
            v = shifted8(__ldg(vec), __ldg(vec + 1), static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15));
        } else {
            uint32_t e[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                e[c] = x + c < to.size[0] ? ld_stream_u16(p + c) : 0;
            v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        }
        st_vec_out(out, v);
    }
}

int launch_pack(const Layout &to0, const Layout &from0, const Layout &to1, const Layout &from1,
                cudaStream_t stream) {
    const auto planes = [](const Layout &t) { return t.size[1] ? t.size[2] * t.size[3] : 0; };
    const int64_t n0 = planes(to0), n1 = planes(to1);
    const int64_t wide = to0.size[0] > to1.size[0] ? to0.size[0] : to1.size[0];
    const int64_t high = ceil_div64(to0.size[1] > to1.size[1] ? to0.size[1] : to1.size[1], 16);
    if (n0 + n1 == 0)
        return GATED_ACT_OK;
    const dim3 grid(static_cast<unsigned>(ceil_div64(wide, 256)),
                    static_cast<unsigned>(high < 32768 ? high : 32768), static_cast<unsigned>(n0 + n1));
    return cuda_status(launch_kernel(pack_rows, grid, dim3(32, 8), 0, stream, 1, to0, from0, to1, from1,
                                     static_cast<int>(n0)));
}

int launch_pack(const Layout &to, const Layout &from, cudaStream_t stream) {
    const Layout none = {};
    return launch_pack(to, from, none, none, stream);
}

}  // namespace gact
