// Tensor maps for the products' operands, and copies of those that TMA cannot address.
#include "product.cuh"

namespace gact {

bool tma_addressable(const Layout &t) {
    if (!aligned(t.data, 16))
        return false;
    for (int i = 1; i < 4; ++i)
        if (t.size[i] > 1 && t.stride[i] % 8)
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
    for (int i = 0; i < n; ++i) {
        const void *dev = nullptr;
        bool host = false;
        if (r[i].bytes && (resolve_ptr(r[i].p, &dev, &host) != GATED_ACT_OK || host))
            return GATED_ACT_ERR_HOST;
    }
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

// Eight elements per thread, loaded one by one (consecutive lanes read consecutive
// addresses, through L1) and stored as a vector.
__global__ void __launch_bounds__(256) pack_rows(Layout to, Layout from) {
    pdl_wait();
    pdl_trigger();
    const int64_t x = (int64_t(blockIdx.x) * 32 + threadIdx.x) * 8;
    if (x >= to.size[0])
        return;
    const int64_t rows = to.size[1] * to.size[2] * to.size[3];
    for (int64_t r = int64_t(blockIdx.y) * 8 + threadIdx.y; r < rows; r += int64_t(gridDim.y) * 8) {
        const int64_t y = r % to.size[1], zw = r / to.size[1], z = zw % to.size[2], w = zw / to.size[2];
        const uint16_t *p = static_cast<const uint16_t *>(from.data) + y * from.stride[1] +
                            z * from.stride[2] + w * from.stride[3] + x;
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = x + i < to.size[0] ? ld_stream_u16(p + i) : 0;
        st_vec(static_cast<uint16_t *>(const_cast<void *>(to.data)) + r * to.stride[1] + x,
               make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                          v[6] | v[7] << 16));
    }
}

int launch_pack(const Layout &to, const Layout &from, cudaStream_t stream) {
    const int64_t rows = to.size[1] * to.size[2] * to.size[3], blocks = ceil_div64(rows, 8);
    if (rows == 0)
        return GATED_ACT_OK;
    const dim3 grid(static_cast<unsigned>(ceil_div64(to.size[0], 256)),
                    static_cast<unsigned>(blocks < 16384 ? blocks : 16384));
    return cuda_status(launch_kernel(pack_rows, grid, dim3(32, 8), 0, stream, 1, to, from));
}

}  // namespace gact
