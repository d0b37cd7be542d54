// tensor_map.h -- tensor maps of the block's products.
#pragma once

#include <cstdint>
#include <cuda.h>  // CUtensorMap only; no libcuda symbol is linked

namespace nqg {

// A tensor of 16-bit elements, the innermost dimension first, in boxes with the 128-byte swizzle.  What lies outside reads
// as zeros.
struct TensorShape {
    int32_t dims;
    int64_t size[4];
    int64_t stride[3];  // elements from one to the next of dimensions 1 to 3
    int32_t box[4];
};

bool encode_tensor(CUtensorMap &map, const void *at, const TensorShape &shape);

} // namespace nqg
