// linear_w4.cu -- out[m, n] = sum_k x[m, k] W[n, k] for a few rows x and a
// matrix W in 4 bits (NVFP4, or integers with group scales).
//
// One CTA computes 16 rows of W for all M columns: its warps split k, and
// their fp32 sums are added in shared memory in the order of the warps.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_layer.h"
#include "common.h"
#include "ptx.cuh"
#include "skinny.cuh"

namespace nqg {
namespace {

constexpr int kWarps = 8;

struct LinearParams {
    WeightView W;
    const uint16_t *x;
    uint16_t *out;
    int64_t x_stride, out_stride;
    int32_t M, N;
    float divisor;
};

template <int FMT, bool BF16, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 8 ? 1 : 2) linear_w4_kernel(LinearParams p)
{
    using F = Format<FMT, BF16>;
    constexpr int kStep = 4 * F::kLane;
    constexpr int U = NT == 1 ? 4 : (NT == 2 ? 2 : 1);
    __shared__ float red[kWarps][16][8 * NT];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16;
    grid_dependency_wait();
    allow_dependent_launch();
    const auto row = [&](int r) { return F::row(p.W, n0 + r < p.N ? n0 + r : p.N - 1); };
    const uint16_t *col[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = 8 * nt + g;
        col[nt] = p.x + (c < p.M ? c : p.M - 1) * p.x_stride;
    }
    float acc[NT][4] = {};
    const int steps = (p.W.K + kStep - 1) / kStep;
    const int k0 = warp * steps / kWarps * kStep, k1 = (warp + 1) * steps / kWarps * kStep;
    skinny_product<F, BF16, NT, U>(acc, p.W, row(g), row(g + 8), col, NT, k0, k1 < p.W.K ? k1 : p.W.K, lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        red[warp][g][8 * nt + 2 * t] = acc[nt][0];
        red[warp][g][8 * nt + 2 * t + 1] = acc[nt][1];
        red[warp][g + 8][8 * nt + 2 * t] = acc[nt][2];
        red[warp][g + 8][8 * nt + 2 * t + 1] = acc[nt][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kWarps) {
        const int r = i & 15, c = i >> 4;
        if (n0 + r >= p.N || c >= p.M)
            continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            s += red[w][r][c];
        p.out[c * p.out_stride + n0 + r] = narrow16<BF16>(descale<F>(s, p.divisor));
    }
}

using LinearFn = void (*)(LinearParams);

template <int FMT, bool BF16>
LinearFn linear_fn(int64_t M)
{
    return M <= 8    ? linear_w4_kernel<FMT, BF16, 1>
           : M <= 16 ? linear_w4_kernel<FMT, BF16, 2>
           : M <= 32 ? linear_w4_kernel<FMT, BF16, 4>
                     : linear_w4_kernel<FMT, BF16, 8>;
}

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" size_t moe_linear_w4_args_size(void) { return sizeof(moe_linear_w4_args); }

extern "C" moe_status moe_linear_w4(const moe_linear_w4_args *a, moe_stream_t stream)
{
    if (!a || a->M < 0 || a->N < 1 || a->K < 1)
        return MOE_ERR_INVALID_ARG;
    const bool int4 = a->w_format == MOE_W_INT4;
    if ((!int4 && a->w_format != MOE_W_NVFP4) || (a->io_dtype != MOE_IO_BF16 && a->io_dtype != MOE_IO_FP16))
        return MOE_ERR_INVALID_ARG;
    const int shift = int4 ? group_shift(a->group_size) : 4;
    if (shift < 0 || a->K % (1 << shift) != 0 || (!int4 && (a->w_zeros || !(a->global_scale > 0.0f) || std::isinf(a->global_scale))))
        return MOE_ERR_INVALID_ARG;
    if (a->M > MOE_FEW_TOKENS || a->N > MOE_FEW_MAX_DIM || a->K > MOE_FEW_MAX_DIM)
        return MOE_ERR_UNSUPPORTED;
    if (a->M == 0)
        return MOE_OK;
    if (!a->x || !a->w || !a->w_scales || !a->out || !aligned16(a->x) || !aligned16(a->w) ||
        (reinterpret_cast<uintptr_t>(a->out) & 1u) || (int4 && (reinterpret_cast<uintptr_t>(a->w_scales) & 1u)))
        return MOE_ERR_INVALID_ARG;
    if (a->x_stride < a->K || a->x_stride % 8 != 0 || a->out_stride < a->N)
        return MOE_ERR_INVALID_ARG;
    LinearParams p{{static_cast<const uint8_t *>(a->w), static_cast<const uint8_t *>(a->w_scales),
                    static_cast<const uint8_t *>(a->w_zeros), a->K, shift},
                   static_cast<const uint16_t *>(a->x), static_cast<uint16_t *>(a->out), a->x_stride, a->out_stride,
                   static_cast<int32_t>(a->M), a->N, int4 ? 1.0f : a->global_scale};
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    const LinearFn fn = int4 ? (bf16 ? linear_fn<kWInt4, true>(a->M) : linear_fn<kWInt4, false>(a->M))
                             : (bf16 ? linear_fn<kWNvfp4, true>(a->M) : linear_fn<kWNvfp4, false>(a->M));
    const PdlLaunch launch(static_cast<unsigned>((a->N + 15) / 16), 32 * kWarps, 0, stream);
    return launch.run(fn, p);
}
