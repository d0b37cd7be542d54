// tensor_map.h -- tensor maps of the block's products.
#pragma once

#include <cstdint>
#include <cuda.h>  // CUtensorMap only; no libcuda symbol is linked

namespace nqg {

// [groups, rows, width] of 16-bit elements, `stride` of them from row to row and rows * stride from group to group, in
// boxes of box_rows rows x box_width elements with the 128-byte swizzle.  What lies outside reads as zeros.
bool encode_rows(CUtensorMap &map, const void *at, int32_t width, int64_t rows, int32_t groups, int64_t stride, int32_t box_width,
                 int32_t box_rows);

} // namespace nqg
