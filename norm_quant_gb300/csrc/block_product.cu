// block_product.cu -- products of rows that are grouped by expert.
//
// A simple form: a block makes 64 x 64 values of the result from tiles of 16
// of the contraction in shared memory, with fp32 multiply-adds.
#include <cstdint>
#include <cuda_runtime.h>

#include "block.h"
#include "block_math.cuh"
#include "few_token.h"

namespace nqg {
namespace {

constexpr int kTile = 64, kStep = 16;

struct Params {
    Product p;
};

template <bool BF16>
__device__ __forceinline__ float value(const void *base, int64_t at)
{
    float lo, hi;
    unpack2<BF16>(static_cast<const uint16_t *>(base)[at], lo, hi);
    return lo;
}

template <bool BF16>
__device__ __forceinline__ void put(void *base, int64_t at, float v)
{
    static_cast<uint16_t *>(base)[at] = static_cast<uint16_t>(pack2<BF16>(v, 0.0f));
}

// offsets[e] as the kernels take it: within [0, rows], not below an earlier one.
__device__ bool bounds_of(const Product &p, int e, int64_t &first, int64_t &last)
{
    if (!p.offsets) {
        first = 0;
        last = p.n_rows;
        return true;
    }
    int64_t at = 0;
    bool good = true;
    for (int i = 0; i <= e + 1; ++i) {
        int64_t v = p.offsets[i];
        good = good && v >= at && v <= p.n_rows;
        v = v < 0 ? 0 : (v > p.n_rows ? p.n_rows : v);
        at = v > at ? v : at;
        if (i == e)
            first = at;
    }
    last = at;
    return good;
}

// grid: (column tiles of the result, row tiles, experts)
template <int KIND, bool BF16, int ACT>
__global__ void __launch_bounds__(256) product_kernel(const Params q)
{
    const Product &p = q.p;
    __shared__ float a[kStep][kTile + 4], b[2][kStep][kTile + 4];
    __shared__ int64_t range[2];
    grid_dependency_wait();
    const int tid = threadIdx.x, e = blockIdx.z;
    if (tid == 0) {
        if (!bounds_of(p, e, range[0], range[1]) && p.status)
            atomicCAS(p.status, 0, MOE_ERR_ROW_OUT_OF_RANGE);
    }
    __syncthreads();
    const int64_t first = range[0], last = range[1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t M = KIND == kWeight ? p.width : last - first;     // rows of the result
    const int64_t K = KIND == kWeight ? last - first : p.width;     // the contraction
    const int64_t N = p.out_width;
    if (m0 >= M)
        return;
    const int F = KIND == kGated ? 2 : 1;
    float acc[2][4][4] = {};
    const int ty = tid / 16, tx = tid % 16;
    for (int64_t k0 = 0; k0 < K; k0 += kStep) {
        for (int i = tid; i < kStep * kTile; i += 256) {
            const int64_t k = k0 + i % kStep, m = m0 + i / kStep;
            float v = 0.0f;
            if (k < K && m < M)
                v = KIND == kWeight ? value<BF16>(p.rows, (first + k) * p.rows_stride + m)
                                    : value<BF16>(p.rows, (first + m) * p.rows_stride + k);
            a[i % kStep][i / kStep] = v;
        }
        for (int f = 0; f < F; ++f)
            for (int i = tid; i < kStep * kTile; i += 256) {
                const int64_t k = k0 + i % kStep, n = n0 + i / kStep;
                float v = 0.0f;
                if (k < K && n < N) {
                    if (KIND == kForward || KIND == kGated)
                        v = value<BF16>(p.other, ((static_cast<int64_t>(e) * F + f) * N + n) * K + k);
                    else if (KIND == kInput)
                        v = value<BF16>(p.other, (static_cast<int64_t>(e) * K + k) * N + n);
                    else
                        v = value<BF16>(p.other, (first + k) * p.other_stride + n);
                }
                b[f][i % kStep][i / kStep] = v;
            }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[f][i][j] += a[k][ty + 16 * i] * b[f][k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= M || n >= N)
                continue;
            const float v = acc[0][i][j];
            if constexpr (KIND == kWeight) {
                const int64_t at = (static_cast<int64_t>(e) * M + m) * N + n;
                if (p.fp32_out)
                    static_cast<float *>(p.out)[at] = v;
                else
                    put<BF16>(p.out, at, v);
            } else if constexpr (KIND == kGated) {
                const float u = acc[1][i][j];
                put<BF16>(p.out, (first + m) * p.out_stride + n, act<ACT>(v) * u);
                if (p.gate_up) {
                    put<BF16>(p.gate_up, (first + m) * p.gate_up_stride + n, v);
                    put<BF16>(p.gate_up, (first + m) * p.gate_up_stride + N + n, u);
                }
            } else {
                put<BF16>(p.out, (first + m) * p.out_stride + n, v);
            }
        }
}

template <int KIND, bool BF16, int ACT>
moe_status launch(const Product &p, moe_stream_t stream)
{
    const int64_t M = KIND == kWeight ? p.width : p.n_rows;
    const dim3 grid(static_cast<unsigned>((p.out_width + kTile - 1) / kTile), static_cast<unsigned>((M + kTile - 1) / kTile),
                    static_cast<unsigned>(p.E));
    if (grid.y > 65535)
        return MOE_ERR_UNSUPPORTED;
    PdlLaunch l(1, 256, 0, stream);
    l.cfg.gridDim = grid;
    return l.run(product_kernel<KIND, BF16, ACT>, Params{p});
}

template <bool BF16>
moe_status dispatch(ProductKind kind, const Product &p, moe_stream_t stream)
{
    switch (kind) {
    case kForward: return launch<kForward, BF16, 0>(p, stream);
    case kGated: return p.activation == MOE_ACT_SILU ? launch<kGated, BF16, MOE_ACT_SILU>(p, stream) : launch<kGated, BF16, MOE_ACT_GELU_TANH>(p, stream);
    case kInput: return launch<kInput, BF16, 0>(p, stream);
    default: return launch<kWeight, BF16, 0>(p, stream);
    }
}

} // namespace

moe_status run_product(ProductKind kind, const Product &p, moe_stream_t stream)
{
    return p.bf16 ? dispatch<true>(kind, p, stream) : dispatch<false>(kind, p, stream);
}

} // namespace nqg
