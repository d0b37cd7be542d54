// block_linear.cu -- the entry points of the block's products: checks of
// arguments, and the pass over gate_up between the gated product's gradients.
#include <cstdint>
#include <cuda_runtime.h>

#include "block.h"
#include "block_math.cuh"
#include "few_token.h"
#include "ptx.cuh"

namespace nqg {
namespace {

struct GateGradParams {
    const uint8_t *d_out, *gate_up;
    uint8_t *d_gate_up;  // [rows, 2 I], one row after the other, or (fold) [rows, 2 fold]
    int64_t d_out_stride, gate_up_stride;  // bytes
    int64_t vectors;     // rows * I / 8
    int32_t per_row;     // I / 8
    int32_t fold;        // Product::fold
};

// Eight values rounded, and (part > 0) what they are rounded by `part` bytes on; nothing for an infinity.
template <bool BF16>
__device__ __forceinline__ void store_held(uint8_t *to, const float (&v)[8], int64_t part)
{
    const uint4 held = pack8<BF16>(v);
    *reinterpret_cast<uint4 *>(to) = held;
    if (part > 0) {
        float rest[8];
        unpack8<BF16>(held, rest);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rest[i] = isinf(rest[i]) ? 0.0f : v[i] - rest[i];
        *reinterpret_cast<uint4 *>(to + part) = pack8<BF16>(rest);
    }
}

// dg = d_out * u * act'(g), du = d_out * act(g), eight elements a thread: ten bytes an element of d_out pass through, and HBM
// bounds it (4096 x 8192: 336 MB in 51.7 us, 6.5 TB/s).  A kernel of its own, as two products read what it writes, one with it
// as its contraction's rows and one as its columns.
template <bool BF16, int ACT>
__global__ void __launch_bounds__(256) gate_grad_kernel(const GateGradParams p)
{
    grid_dependency_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < p.vectors; i += step) {
        const int64_t r = i / p.per_row;
        const int64_t at = 16 * (i - r * p.per_row);
        const uint8_t *gate = p.gate_up + r * p.gate_up_stride + at;
        const int64_t half = 16 * static_cast<int64_t>(p.per_row);
        float d[8], g[8], u[8], dg[8], du[8];
        unpack8<BF16>(ldg16(p.d_out + r * p.d_out_stride + at), d);
        unpack8<BF16>(ldg16(gate), g);
        unpack8<BF16>(ldg16(gate + half), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a, slope;
            act_and_slope<ACT>(g[j], a, slope);
            dg[j] = d[j] * u[j] * slope;
            du[j] = d[j] * a;
        }
        const int64_t part = 2 * static_cast<int64_t>(p.fold);
        uint8_t *out = p.d_gate_up + r * 2 * (p.fold ? part : half) + at;
        store_held<BF16>(out, dg, part);
        store_held<BF16>(out + half, du, part);
        // zeros behind both parts
        for (int64_t zero = 2 * half + at; zero < part; zero += half) {
            *reinterpret_cast<uint4 *>(out - at + zero) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(out - at + part + zero) = make_uint4(0, 0, 0, 0);
        }
    }
}

template <bool BF16, int ACT>
moe_status launch_gate_grad(const GateGradParams &p, int sms, moe_stream_t stream)
{
    const int64_t blocks = (p.vectors + 255) / 256, most = static_cast<int64_t>(sms) * 8;
    return PdlLaunch(static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream).run(gate_grad_kernel<BF16, ACT>, p);
}

// dg and du of small calls are held as sums of two 16-bit values, and the products take every step twice.  That leaves a gradient
// no more error than its own rounding has, at any number of rows (relative, bf16: 1.65e-3 for 2.35e-3, and 2.5e-3 where sums are
// shortest; fp16: 2.1e-4 for 2.95e-4), so the limits are of cost alone: up to the rows of the narrowest tile, and up to 8192
// values a part with the columns that it is padded by.  bf16, us held / rounded once, in a graph: 32 rows, H = 256, I = 72: 13.0 /
// 12.1; 16, 2048, 200: 14.3 / 12.7; 8, 2048, 456, E = 8: 25.3 / 21.6; 2, 4096, 1984: 33.2 / 25.4; 1, 4096, 4040: 51.1 / 40.9;
// beyond: 32, 2048, 512: 17.4 / 14.5; 128, 2048, 1408, E = 8: 54.3 / 46.4; 1, 4096, 8192: 88.6 / 66.9; 2048, 2048, 4096: 173 / 100.
constexpr int64_t kHeldRows = 32, kHeldValues = 4096;  // rows, and rows * (I + 56)

int32_t part_columns(int32_t I) { return (2 * I + 63) / 64 * 64; }

// The columns of each part, or 0.
int32_t fold_of(int64_t rows, int32_t I)
{
    return rows <= kHeldRows && rows * (I + 56) <= kHeldValues ? part_columns(I) : 0;
}

// What a call of so many rows writes, and the most that one of as many or fewer rows does.
int64_t workspace_of(int64_t rows, int32_t I)
{
    const int32_t fold = fold_of(rows, I);
    return rows * (fold ? fold : I) * 4;
}

int64_t workspace_up_to(int64_t rows, int32_t I)
{
    int64_t held = kHeldValues / (I + 56);
    held = held < kHeldRows ? held : kHeldRows;
    held = held < rows ? held : rows;
    const int64_t a = workspace_of(rows, I), b = held * part_columns(I) * 4;
    return a > b ? a : b;
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - (1 << 16);

// Checks that the products share: 0 where the call can go on (rows > 0), else what to return.
int check_sizes(int64_t rows, int32_t a, int32_t b, int32_t E, int32_t io)
{
    if (rows < 0 || a < 8 || b < 8 || a % 8 != 0 || b % 8 != 0 || E < 1 || !valid_io(io))
        return MOE_ERR_INVALID_ARG;
    if (rows >= kMaxRows || a > MOE_BLOCK_MAX_DIM || b > MOE_BLOCK_MAX_DIM || E > MOE_LAYER_MAX_EXPERTS)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool valid_shared(const int32_t *offsets, int32_t E, const int32_t *status)
{
    return (offsets || E == 1) && (reinterpret_cast<uintptr_t>(offsets) & 3u) == 0 && (reinterpret_cast<uintptr_t>(status) & 3u) == 0;
}

bool valid_grad_type(int32_t grad, int32_t io)
{
    return grad == MOE_WEIGHTS_FP32 || grad == (io == MOE_IO_BF16 ? MOE_WEIGHTS_BF16 : MOE_WEIGHTS_FP16);
}

moe_status set_zero(void *at, int64_t elements, int32_t grad, moe_stream_t stream)
{
    const size_t bytes = static_cast<size_t>(elements) * (grad == MOE_WEIGHTS_FP32 ? 4 : 2);
    return cudaMemsetAsync(at, 0, bytes, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : (cudaGetLastError(), MOE_ERR_CUDA);
}

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" size_t moe_gated_linear_args_size(void) { return sizeof(moe_gated_linear_args); }
extern "C" size_t moe_gated_linear_backward_args_size(void) { return sizeof(moe_gated_linear_backward_args); }
extern "C" size_t moe_grouped_linear_args_size(void) { return sizeof(moe_grouped_linear_args); }
extern "C" size_t moe_grouped_linear_backward_args_size(void) { return sizeof(moe_grouped_linear_backward_args); }

extern "C" moe_status moe_gated_linear(const moe_gated_linear_args *a, moe_stream_t stream)
{
    if (!a || (a->activation != MOE_ACT_SILU && a->activation != MOE_ACT_GELU_TANH))
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_sizes(a->rows, a->H, a->I, a->E, a->io_dtype))
        return static_cast<moe_status>(st);
    if (a->rows == 0)
        return MOE_OK;
    if (!valid_rows(a->x, a->x_stride, a->H) || !a->w13 || !aligned16(a->w13) || !valid_rows(a->out, a->out_stride, a->I) ||
        (a->gate_up && !valid_rows(a->gate_up, a->gate_up_stride, 2 * a->I)) || !valid_shared(a->offsets, a->E, a->status))
        return MOE_ERR_INVALID_ARG;
    Product p{};
    p.n_rows = a->rows;
    p.E = a->E;
    p.width = a->H;
    p.out_width = a->I;
    p.rows = a->x;
    p.rows_stride = a->x_stride;
    p.other = a->w13;
    p.offsets = a->offsets;
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.gate_up = a->gate_up;
    p.gate_up_stride = a->gate_up_stride;
    p.status = a->status;
    p.activation = a->activation;
    p.bf16 = a->io_dtype == MOE_IO_BF16;
    p.stall = debug_stall_slots();
    return run_product(kGated, p, stream);
}

extern "C" moe_status moe_gated_linear_backward_workspace_size(int64_t rows, int32_t I, size_t *bytes)
{
    if (!bytes || rows < 0 || I < 8 || I % 8 != 0)
        return MOE_ERR_INVALID_ARG;
    if (rows >= kMaxRows || I > MOE_BLOCK_MAX_DIM)
        return MOE_ERR_UNSUPPORTED;
    *bytes = static_cast<size_t>(workspace_up_to(rows, I));
    return MOE_OK;
}

extern "C" moe_status moe_gated_linear_backward(const moe_gated_linear_backward_args *a, moe_stream_t stream)
{
    if (!a || (a->activation != MOE_ACT_SILU && a->activation != MOE_ACT_GELU_TANH))
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_sizes(a->rows, a->H, a->I, a->E, a->io_dtype))
        return static_cast<moe_status>(st);
    if (!valid_grad_type(a->grad_dtype, a->io_dtype))
        return MOE_ERR_INVALID_ARG;
    if (a->rows == 0 && !a->d_w13)
        return MOE_OK;
    if (a->d_w13 && !aligned16(a->d_w13))
        return MOE_ERR_INVALID_ARG;
    if (a->rows == 0)
        return set_zero(a->d_w13, static_cast<int64_t>(a->E) * 2 * a->I * a->H, a->grad_dtype, stream);
    if (!a->d_x && !a->d_w13)
        return MOE_ERR_INVALID_ARG;
    if (!valid_rows(a->d_out, a->d_out_stride, a->I) || !valid_rows(a->gate_up, a->gate_up_stride, 2 * a->I) ||
        !valid_shared(a->offsets, a->E, a->status))
        return MOE_ERR_INVALID_ARG;
    if (a->d_x && (!valid_rows(a->d_x, a->d_x_stride, a->H) || !a->w13 || !aligned16(a->w13)))
        return MOE_ERR_INVALID_ARG;
    if (a->d_w13 && !valid_rows(a->x, a->x_stride, a->H))
        return MOE_ERR_INVALID_ARG;
    if (!a->workspace || a->workspace_bytes < static_cast<size_t>(workspace_of(a->rows, a->I)))
        return MOE_ERR_WORKSPACE;
    if (!aligned16(a->workspace))
        return MOE_ERR_INVALID_ARG;
    const bool bf16 = a->io_dtype == MOE_IO_BF16, silu = a->activation == MOE_ACT_SILU;
    GateGradParams g{};
    g.d_out = static_cast<const uint8_t *>(a->d_out);
    g.gate_up = static_cast<const uint8_t *>(a->gate_up);
    g.d_gate_up = static_cast<uint8_t *>(a->workspace);
    g.d_out_stride = 2 * a->d_out_stride;
    g.gate_up_stride = 2 * a->gate_up_stride;
    g.per_row = a->I / 8;
    g.vectors = a->rows * g.per_row;
    g.fold = fold_of(a->rows, a->I);
    const int sms = sm_count();
    if (sms <= 0)
        return MOE_ERR_CUDA;
    moe_status st = bf16 ? (silu ? launch_gate_grad<true, MOE_ACT_SILU>(g, sms, stream) : launch_gate_grad<true, MOE_ACT_GELU_TANH>(g, sms, stream))
                         : (silu ? launch_gate_grad<false, MOE_ACT_SILU>(g, sms, stream) : launch_gate_grad<false, MOE_ACT_GELU_TANH>(g, sms, stream));
    Product p{};
    p.n_rows = a->rows;
    p.E = a->E;
    p.width = 2 * a->I;
    p.out_width = a->H;
    p.rows = a->workspace;
    p.fold = g.fold;
    p.rows_stride = g.fold ? 2 * g.fold : 2 * static_cast<int64_t>(a->I);
    p.offsets = a->offsets;
    p.status = a->status;
    p.bf16 = bf16;
    p.stall = debug_stall_slots();
    if (st == MOE_OK && a->d_x) {
        p.other = a->w13;
        p.out = a->d_x;
        p.out_stride = a->d_x_stride;
        st = run_product(kInput, p, stream);
    }
    if (st == MOE_OK && a->d_w13) {
        p.other = a->x;
        p.other_stride = a->x_stride;
        p.out = a->d_w13;
        p.out_stride = a->H;
        p.fp32_out = a->grad_dtype == MOE_WEIGHTS_FP32;
        st = run_product(kWeight, p, stream);
    }
    return st;
}

extern "C" moe_status moe_grouped_linear(const moe_grouped_linear_args *a, moe_stream_t stream)
{
    if (!a)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_sizes(a->rows, a->K, a->N, a->E, a->io_dtype))
        return static_cast<moe_status>(st);
    if (a->rows == 0)
        return MOE_OK;
    if (!valid_rows(a->x, a->x_stride, a->K) || !a->w || !aligned16(a->w) || !valid_rows(a->out, a->out_stride, a->N) ||
        !valid_shared(a->offsets, a->E, a->status))
        return MOE_ERR_INVALID_ARG;
    Product p{};
    p.n_rows = a->rows;
    p.E = a->E;
    p.width = a->K;
    p.out_width = a->N;
    p.rows = a->x;
    p.rows_stride = a->x_stride;
    p.other = a->w;
    p.offsets = a->offsets;
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.status = a->status;
    p.bf16 = a->io_dtype == MOE_IO_BF16;
    p.stall = debug_stall_slots();
    return run_product(kForward, p, stream);
}

extern "C" moe_status moe_grouped_linear_backward(const moe_grouped_linear_backward_args *a, moe_stream_t stream)
{
    if (!a)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_sizes(a->rows, a->K, a->N, a->E, a->io_dtype))
        return static_cast<moe_status>(st);
    if (!valid_grad_type(a->grad_dtype, a->io_dtype))
        return MOE_ERR_INVALID_ARG;
    if (a->rows == 0 && !a->d_w)
        return MOE_OK;
    if (a->d_w && !aligned16(a->d_w))
        return MOE_ERR_INVALID_ARG;
    if (a->rows == 0)
        return set_zero(a->d_w, static_cast<int64_t>(a->E) * a->N * a->K, a->grad_dtype, stream);
    if (!a->d_x && !a->d_w)
        return MOE_ERR_INVALID_ARG;
    if (!valid_rows(a->d_out, a->d_out_stride, a->N) || !valid_shared(a->offsets, a->E, a->status))
        return MOE_ERR_INVALID_ARG;
    if (a->d_x && (!valid_rows(a->d_x, a->d_x_stride, a->K) || !a->w || !aligned16(a->w)))
        return MOE_ERR_INVALID_ARG;
    if (a->d_w && !valid_rows(a->x, a->x_stride, a->K))
        return MOE_ERR_INVALID_ARG;
    Product p{};
    p.n_rows = a->rows;
    p.E = a->E;
    p.width = a->N;
    p.out_width = a->K;
    p.rows = a->d_out;
    p.rows_stride = a->d_out_stride;
    p.offsets = a->offsets;
    p.status = a->status;
    p.bf16 = a->io_dtype == MOE_IO_BF16;
    p.stall = debug_stall_slots();
    moe_status st = MOE_OK;
    if (a->d_x) {
        p.other = a->w;
        p.out = a->d_x;
        p.out_stride = a->d_x_stride;
        st = run_product(kInput, p, stream);
    }
    if (st == MOE_OK && a->d_w) {
        p.other = a->x;
        p.other_stride = a->x_stride;
        p.out = a->d_w;
        p.out_stride = a->K;
        p.fp32_out = a->grad_dtype == MOE_WEIGHTS_FP32;
        st = run_product(kWeight, p, stream);
    }
    return st;
}
