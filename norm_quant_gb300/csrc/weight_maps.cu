// weight_maps.cu -- the tensor maps through which the few-token products copy
// their weights to shared memory, and those of the products of grouped rows.
#include <cstdint>
#include <mutex>
#include <cuda.h>
#include <cuda_runtime.h>

#include "skinny.cuh"
#include "tensor_map.h"

namespace nqg {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's entry-point query, so that the library links no libcuda.
EncodeTiled encoder()
{
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(f);
        cudaGetLastError();
    });
    return fn;
}

bool encode(CUtensorMap &map, const void *at, int dims, const cuuint64_t *size, const cuuint64_t *stride,
            const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    const cuuint32_t step[3] = {1, 1, 1};
    return encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(dims), const_cast<void *>(at), size, stride,
                     box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace

moe_status make_maps(WeightMaps &m, const SlotPlan &plan, const WeightView &W, int row_bytes, int64_t rows, int scale_row,
                     int zero_row)
{
    m.whole = row_bytes / kStripBytes;
    if ((m.tensor || m.scale_tensor) && !encoder())
        return MOE_ERR_CUDA;
    const cuuint64_t n = static_cast<cuuint64_t>(rows), pitch = static_cast<cuuint64_t>(row_bytes);
    if (m.tensor && m.whole > 0) {
        const cuuint64_t size[3] = {kStripBytes, n, static_cast<cuuint64_t>(m.whole)}, stride[2] = {pitch, kStripBytes};
        const cuuint32_t box[3] = {kStripBytes, static_cast<cuuint32_t>(plan.block), static_cast<cuuint32_t>(plan.strips)};
        if (!encode(m.panels, W.w, 3, size, stride, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return MOE_ERR_CUDA;
    }
    if (m.tensor && row_bytes % kStripBytes != 0) {
        const cuuint64_t size[2] = {pitch, n}, stride[1] = {pitch};
        const cuuint32_t box[2] = {kStripBytes, static_cast<cuuint32_t>(plan.block)};
        if (!encode(m.strips, W.w, 2, size, stride, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return MOE_ERR_CUDA;
    }
    const auto scales = [&](CUtensorMap &map, const void *at, int row, int panel) {
        const cuuint64_t size[2] = {static_cast<cuuint64_t>(row), n}, stride[1] = {static_cast<cuuint64_t>(row)};
        const cuuint32_t box[2] = {static_cast<cuuint32_t>(panel), static_cast<cuuint32_t>(plan.block)};
        return encode(map, at, 2, size, stride, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    if (m.scale_tensor && !scales(m.scales, W.scales, scale_row, plan.scale.pitch))
        return MOE_ERR_CUDA;
    if (m.scale_tensor && zero_row && !scales(m.zeros, W.zeros, zero_row, plan.scale.zero_pitch))
        return MOE_ERR_CUDA;
    return MOE_OK;
}

moe_status make_column_map(CUtensorMap &map, const void *at, int row_bytes, int rows, int64_t pitch, int box, int chunks)
{
    if (!encoder())
        return MOE_ERR_CUDA;
    const cuuint64_t n = static_cast<cuuint64_t>(rows), bytes = static_cast<cuuint64_t>(row_bytes);
    // the pitch of a single row is its caller's business, and may pass what a map takes
    const cuuint64_t p = rows > 1 ? static_cast<cuuint64_t>(pitch) : (bytes + 15) / 16 * 16;
    const cuuint64_t size3[3] = {kStripBytes, n, bytes / kStripBytes}, stride3[2] = {p, kStripBytes};
    const cuuint64_t size2[2] = {bytes, n};
    const cuuint32_t boxes[3] = {kStripBytes, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(chunks)};
    const bool ok = row_bytes % kStripBytes == 0 ? encode(map, at, 3, size3, stride3, boxes, CU_TENSOR_MAP_SWIZZLE_128B)
                                                 : encode(map, at, 2, size2, stride3, boxes, CU_TENSOR_MAP_SWIZZLE_128B);
    return ok ? MOE_OK : MOE_ERR_CUDA;
}

bool encode_tensor(CUtensorMap &map, const void *at, const TensorShape &shape)
{
    if (!encoder())
        return false;
    cuuint64_t size[4], stride[3];
    cuuint32_t box[4], step[4];
    for (int i = 0; i < shape.dims; ++i) {
        size[i] = static_cast<cuuint64_t>(shape.size[i]);
        box[i] = static_cast<cuuint32_t>(shape.box[i]);
        step[i] = 1;
        if (i > 0)
            stride[i - 1] = 2 * static_cast<cuuint64_t>(shape.stride[i - 1]);
    }
    return encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, static_cast<cuuint32_t>(shape.dims), const_cast<void *>(at), size, stride, box,
                     step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace nqg
