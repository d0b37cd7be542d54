// block.h -- what the feed-forward block's entry points and kernels share: the
// products of grouped rows as one problem, and host-side checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_block.h"
#include "common.h"

namespace nqg {

enum ProductKind {
    kForward = 0,  // D[r, f] = sum_k X[r, k] W[e][f, k]                 (rows X, features of W)
    kGated = 1,    // the same for W1 and W3, D = act(first) * second
    kInput = 2,    // D[r, c] = sum_n Y[r, n] W[e][n, c]                 (gradient of the rows)
    kWeight = 3    // D[e][n, c] = sum over e's rows of Y[r, n] X[r, c]  (gradient of the weights)
};

// One product of grouped rows.  `rows` is the matrix of rows (X, or Y where there are two), `other` W or, for the
// weights' gradient, X.
struct Product {
    int64_t n_rows;
    int32_t E;
    int32_t width;        // columns of `rows`
    int32_t out_width;    // columns of the result; for kGated I (W has 2 I rows)
    const void *rows;
    int64_t rows_stride;
    int32_t fold;         // kInput, kWeight: 0, or `rows` is held as a sum: its columns, up to `fold` (a multiple of 64) zeros, what
                          // they are rounded by, and zeros again
    const void *other;
    int64_t other_stride; // kWeight: elements from row to row of X
    const int32_t *offsets;
    void *out;
    int64_t out_stride;
    void *gate_up;        // kGated: both sums, or nullptr
    int64_t gate_up_stride;
    int32_t *status;
    int32_t activation;
    bool bf16, fp32_out;
    int64_t stall;        // moe_debug_stall's setting
};

moe_status run_product(ProductKind kind, const Product &p, moe_stream_t stream);

inline bool valid_io(int32_t io) { return io == MOE_IO_BF16 || io == MOE_IO_FP16; }

// A matrix of rows of `width` 16-bit elements: 16-byte aligned, with a stride that keeps every row so and that a tensor map
// takes (below 2^40 bytes).
inline bool valid_rows(const void *p, int64_t stride, int32_t width)
{
    return p && aligned16(p) && stride >= width && stride <= MOE_BLOCK_MAX_STRIDE && stride % 8 == 0;
}

} // namespace nqg
