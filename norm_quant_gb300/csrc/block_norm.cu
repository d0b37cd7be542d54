// block_norm.cu -- the norms after a block and before the next one, with the
// block's gate and the residual's scale, forward and backward.
//
// A CTA takes a row at a time and every thread VPT vectors of 8 of its columns,
// which stay in registers between the sums over the row.  The backward pass adds
// up the columns' sums (gammas, channel gate) over the rows of a CTA, leaves
// them in the workspace, and a second kernel adds the CTAs' up in their order.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "block.h"
#include "block_math.cuh"
#include "few_token.h"

namespace nqg {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kSums = 3;  // columns' sums: post_gamma's gradient, pre_gamma's, the channel gate's

struct NormParams {
    int64_t T;
    int32_t H;
    const uint8_t *y, *residual, *post, *pre, *gate;
    int32_t gate_kind;
    float block_scale, residual_scale, eps, bias, inv_h;
    uint8_t *residual_out, *norm_out;
    const uint8_t *d_residual_out, *d_norm_out;
    uint8_t *d_y, *d_residual;
    float *d_post, *d_pre, *d_gate;
    float *partial;  // backward: [CTAs, kSums, H]
    int32_t ctas;
};

// Sums over a CTA, with one barrier each: two buffers in turn, and a thread that writes one again has passed the
// barrier behind every thread's reads of it.
struct BlockSum {
    float (*buffers)[32];
    int turn = 0;
};

// Sums of N <= 2 values over the CTA, in every thread.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], BlockSum &b)
{
    float *red = b.buffers[b.turn];
    b.turn ^= 1;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lane == 0)
            red[i * 16 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < warps ? red[i * 16 + lane] : 0.0f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
}

template <bool BF16>
__device__ __forceinline__ void load8(float (&v)[8], const uint8_t *p, int64_t bytes)
{
    unpack8<BF16>(*reinterpret_cast<const uint4 *>(p + bytes), v);
}

template <bool BF16>
__device__ __forceinline__ void gates8(float (&v)[8], const NormParams &p, float token, int bytes)
{
    if (p.gate_kind == MOE_GATE_CHANNEL) {
        unpack8<BF16>(ldg16(p.gate + bytes), v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= p.block_scale;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = token;
    }
}

// gamma + weight_bias of 8 columns, or 1.
template <bool BF16>
__device__ __forceinline__ void gammas8(float (&v)[8], const uint8_t *gamma, float bias, int bytes)
{
    if (gamma) {
        unpack8<BF16>(ldg16(gamma + bytes), v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += bias;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 1.0f;
    }
}

// block_scale times the token's gate (1 where tokens have none).
__device__ __forceinline__ float token_factor(const NormParams &p, int64_t t)
{
    return p.gate_kind == MOE_GATE_TOKEN ? p.block_scale * __ldg(reinterpret_cast<const float *>(p.gate) + t) : p.block_scale;
}

template <bool BF16, int VPT>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p)
{
    __shared__ float buffers[2][32];
    BlockSum red{buffers};
    grid_dependency_wait();
    const int vectors = p.H / 8;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t row = 2 * t * p.H;
        uint4 y[VPT], r[VPT];
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            y[j] = r[j] = make_uint4(0, 0, 0, 0);
            if (i < vectors) {
                y[j] = *reinterpret_cast<const uint4 *>(p.y + row + 16 * i);
                if (p.residual)
                    r[j] = *reinterpret_cast<const uint4 *>(p.residual + row + 16 * i);
            }
        }
        float ry = 1.0f;
        if (p.post) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float v[8];
                unpack8<BF16>(y[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[0] = fmaf(v[i], v[i], sum[0]);
            }
            block_sum(sum, red);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const float token = token_factor(p, t);
        float s[VPT][8];
        sum[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            if (i >= vectors) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[j][k] = 0.0f;
                continue;
            }
            float a[8], v[8], c[8];
            unpack8<BF16>(y[j], a);
            gammas8<BF16>(c, p.post, p.bias, 16 * i);
            gates8<BF16>(v, p, token, 16 * i);
            unpack8<BF16>(r[j], s[j]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[j][k] = fmaf(v[k], a[k] * ry * c[k], p.residual ? p.residual_scale * s[j][k] : 0.0f);
                sum[0] = fmaf(s[j][k], s[j][k], sum[0]);
            }
            if (p.residual_out)
                *reinterpret_cast<uint4 *>(p.residual_out + row + 16 * i) = pack8<BF16>(s[j]);
        }
        if (!p.norm_out)
            continue;
        block_sum(sum, red);
        const float rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            if (i >= vectors)
                continue;
            float c[8];
            gammas8<BF16>(c, p.pre, p.bias, 16 * i);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                c[k] *= s[j][k] * rs;
            *reinterpret_cast<uint4 *>(p.norm_out + row + 16 * i) = pack8<BF16>(c);
        }
    }
    allow_dependent_launch();
}

// The row's part of the backward pass, and the columns' sums over the rows of this CTA.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_kernel(const NormParams p)
{
    __shared__ float buffers[2][32];
    BlockSum red{buffers};
    extern __shared__ float sums[];  // [kSums, H]
    grid_dependency_wait();
    const int vectors = p.H / 8;
    const bool columns = p.partial != nullptr;
    if (columns) {
        for (int i = threadIdx.x; i < vectors; i += blockDim.x)
            for (int k = 0; k < 8 * kSums; ++k)
                sums[(k / 8) * p.H + 8 * i + k % 8] = 0.0f;
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t row = 2 * t * p.H;
        uint4 y[VPT], r[VPT], dx[VPT], dr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            y[j] = r[j] = dx[j] = dr[j] = make_uint4(0, 0, 0, 0);
            if (i < vectors) {
                y[j] = *reinterpret_cast<const uint4 *>(p.y + row + 16 * i);
                if (p.residual)
                    r[j] = *reinterpret_cast<const uint4 *>(p.residual + row + 16 * i);
                if (p.d_norm_out)
                    dx[j] = *reinterpret_cast<const uint4 *>(p.d_norm_out + row + 16 * i);
                if (p.d_residual_out)
                    dr[j] = *reinterpret_cast<const uint4 *>(p.d_residual_out + row + 16 * i);
            }
        }
        float ry = 1.0f;
        if (p.post) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float v[8];
                unpack8<BF16>(y[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[0] = fmaf(v[i], v[i], sum[0]);
            }
            block_sum(sum, red);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const float token = token_factor(p, t);
        // s of a vector, from the packed row
        const auto new_residual = [&](int j, int i, float (&a)[8], float (&g)[8], float (&s)[8]) {
            float c[8];
            unpack8<BF16>(y[j], a);
            gammas8<BF16>(c, p.post, p.bias, 16 * i);
            gates8<BF16>(g, p, token, 16 * i);
            unpack8<BF16>(r[j], s);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] *= ry * c[k];
                s[k] = fmaf(g[k], a[k], p.residual ? p.residual_scale * s[k] : 0.0f);
            }
        };
        float rs = 0.0f, mv = 0.0f;
        if (p.d_norm_out) {
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = threadIdx.x + j * blockDim.x;
                if (i >= vectors)
                    continue;
                float a[8], g[8], s[8], d[8], c[8];
                new_residual(j, i, a, g, s);
                unpack8<BF16>(dx[j], d);
                gammas8<BF16>(c, p.pre, p.bias, 16 * i);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    sum[0] = fmaf(s[k], s[k], sum[0]);
                    sum[1] = fmaf(s[k], d[k] * c[k], sum[1]);
                }
            }
            block_sum(sum, red);
            rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            mv = sum[1] * p.inv_h * rs;  // the mean of m v
        }
        // ds of a vector: what comes directly and what comes back through the second norm
        const auto gradient = [&](int j, int i, const float (&s)[8], float (&d)[8], float (&ds)[8]) {
            float c[8];
            unpack8<BF16>(dr[j], ds);
            unpack8<BF16>(dx[j], d);
            if (p.d_norm_out) {
                gammas8<BF16>(c, p.pre, p.bias, 16 * i);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    ds[k] = fmaf(rs, fmaf(d[k], c[k], -s[k] * rs * mv), ds[k]);
            }
        };
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            if (i >= vectors)
                continue;
            float a[8], g[8], s[8], d[8], ds[8];
            new_residual(j, i, a, g, s);
            gradient(j, i, s, d, ds);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[0] = fmaf(g[k] * ds[k], a[k], sum[0]);  // p n = da a, as a = n (gamma + bias)
                sum[1] = fmaf(ds[k], a[k], sum[1]);
            }
        }
        if (p.post || p.d_gate)
            block_sum(sum, red);
        const float pn = sum[0] * p.inv_h;
        if (p.d_gate && p.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
            p.d_gate[t] = p.block_scale * sum[1];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            if (i >= vectors)
                continue;
            float a[8], g[8], s[8], d[8], ds[8], c[8], out[8];
            new_residual(j, i, a, g, s);
            gradient(j, i, s, d, ds);
            gammas8<BF16>(c, p.post, p.bias, 16 * i);
            float n[8];
            unpack8<BF16>(y[j], n);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                n[k] *= ry;
                const float da = g[k] * ds[k];
                out[k] = p.post ? ry * fmaf(da, c[k], -n[k] * pn) : da;
                if (columns) {
                    float *at = sums + 8 * i + k;
                    if (p.d_post)
                        at[0] = fmaf(da, n[k], at[0]);
                    if (p.d_pre)
                        at[p.H] = fmaf(d[k], s[k] * rs, at[p.H]);
                    if (p.d_gate)
                        at[2 * p.H] = fmaf(ds[k], a[k], at[2 * p.H]);
                }
            }
            if (p.d_y)
                *reinterpret_cast<uint4 *>(p.d_y + row + 16 * i) = pack8<BF16>(out);
            if (p.d_residual) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    ds[k] *= p.residual_scale;
                *reinterpret_cast<uint4 *>(p.d_residual + row + 16 * i) = pack8<BF16>(ds);
            }
        }
    }
    if (columns) {
        float *out = p.partial + static_cast<int64_t>(blockIdx.x) * kSums * p.H;
        for (int i = threadIdx.x; i < vectors; i += blockDim.x)
            for (int k = 0; k < 8 * kSums; ++k)
                out[(k / 8) * p.H + 8 * i + k % 8] = sums[(k / 8) * p.H + 8 * i + k % 8];
    }
    allow_dependent_launch();
}

__global__ void __launch_bounds__(128) column_sums_kernel(const NormParams p)
{
    grid_dependency_wait();
    const int h = blockIdx.x * 128 + threadIdx.x, which = blockIdx.y;
    float *out = which == 0 ? p.d_post : (which == 1 ? p.d_pre : p.d_gate);
    if (h >= p.H || !out || (which == 2 && p.gate_kind != MOE_GATE_CHANNEL))
        return;
    float s = 0.0f;
    for (int i = 0; i < p.ctas; ++i)
        s += p.partial[(static_cast<int64_t>(i) * kSums + which) * p.H + h];
    out[h] = which == 2 ? p.block_scale * s : s;
}

// CTAs of the backward pass whose columns' sums the workspace has room for.
int64_t most_ctas(int64_t T) { return T < 1024 ? T : 1024; }

// Checks that both directions share.
template <typename Args>
bool valid_norm(const Args *a)
{
    if (!a->y || !aligned16(a->y) || !aligned16(a->residual) || !aligned16(a->post_gamma) || !aligned16(a->pre_gamma))
        return false;
    if (a->gate_kind < MOE_GATE_NONE || a->gate_kind > MOE_GATE_TOKEN || (a->gate_kind != MOE_GATE_NONE) != (a->gate != nullptr))
        return false;
    if (reinterpret_cast<uintptr_t>(a->gate) & (a->gate_kind == MOE_GATE_CHANNEL ? 15u : 3u))
        return false;
    return std::isfinite(a->block_scale) && std::isfinite(a->residual_scale) && std::isfinite(a->weight_bias) && a->eps >= 0.0f &&
           std::isfinite(a->eps);
}

template <typename Args>
NormParams norm_params(const Args *a)
{
    NormParams p{};
    p.T = a->T;
    p.H = a->H;
    p.y = static_cast<const uint8_t *>(a->y);
    p.residual = static_cast<const uint8_t *>(a->residual);
    p.post = static_cast<const uint8_t *>(a->post_gamma);
    p.pre = static_cast<const uint8_t *>(a->pre_gamma);
    p.gate = static_cast<const uint8_t *>(a->gate);
    p.gate_kind = a->gate_kind;
    p.block_scale = a->block_scale;
    p.residual_scale = a->residual_scale;
    p.eps = a->eps;
    p.bias = a->weight_bias;
    p.inv_h = static_cast<float>(1.0 / a->H);
    return p;
}

int check_norm_sizes(int64_t T, int32_t H, int32_t io)
{
    if (T < 0 || H < 8 || H % 8 != 0 || !valid_io(io))
        return MOE_ERR_INVALID_ARG;
    return H > MOE_MAX_HIDDEN || T >= (int64_t{1} << 31) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Vectors a thread, and threads a CTA.
int vectors_per_thread(int H) { return H <= 4096 ? 1 : (H <= 8192 ? 2 : 4); }
unsigned threads_of(int H, int vpt) { return static_cast<unsigned>((H / 8 + vpt * 32 - 1) / (vpt * 32) * 32); }

template <bool BF16, int VPT>
moe_status launch_norm(const NormParams &p, moe_stream_t stream)
{
    const int sms = sm_count();
    if (sms <= 0)
        return MOE_ERR_CUDA;
    const unsigned threads = threads_of(p.H, VPT);
    const int64_t most = static_cast<int64_t>(sms) * (2048 / threads < 8 ? 2048 / threads : 8);
    return PdlLaunch(static_cast<unsigned>(p.T < most ? p.T : most), threads, 0, stream).run(norm_kernel<BF16, VPT>, p);
}

template <bool BF16, int VPT>
moe_status launch_backward(NormParams &p, moe_stream_t stream)
{
    static SmemLimit limit;
    int dev = 0;
    const int sms = sm_count();
    const size_t smem = p.partial ? static_cast<size_t>(kSums) * p.H * 4 : 0;
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess ||
        ensure_dynamic_smem(norm_backward_kernel<BF16, VPT>, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int64_t most = p.partial && sms > 1024 ? 1024 : sms;
    p.ctas = static_cast<int32_t>(p.T < most ? p.T : most);
    const moe_status st = PdlLaunch(static_cast<unsigned>(p.ctas), threads_of(p.H, VPT), smem, stream).run(norm_backward_kernel<BF16, VPT>, p);
    if (st != MOE_OK || !p.partial)
        return st;
    PdlLaunch l(1, 128, 0, stream);
    l.cfg.gridDim = dim3(static_cast<unsigned>((p.H + 127) / 128), kSums);
    return l.run(column_sums_kernel, p);
}

moe_status zero_floats(float *at, int64_t n, moe_stream_t stream)
{
    if (at && cudaMemsetAsync(at, 0, static_cast<size_t>(n) * 4, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" size_t moe_block_norm_args_size(void) { return sizeof(moe_block_norm_args); }
extern "C" size_t moe_block_norm_backward_args_size(void) { return sizeof(moe_block_norm_backward_args); }

extern "C" moe_status moe_block_norm(const moe_block_norm_args *a, moe_stream_t stream)
{
    if (!a)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_norm_sizes(a->T, a->H, a->io_dtype))
        return static_cast<moe_status>(st);
    if (a->T == 0)
        return MOE_OK;
    if (!valid_norm(a) || !aligned16(a->residual_out) || !aligned16(a->norm_out) || (!a->residual_out && !a->norm_out) ||
        (a->norm_out && (!a->pre_gamma || a->norm_out == a->residual_out)))
        return MOE_ERR_INVALID_ARG;
    NormParams p = norm_params(a);
    p.residual_out = static_cast<uint8_t *>(a->residual_out);
    p.norm_out = static_cast<uint8_t *>(a->norm_out);
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    switch (vectors_per_thread(a->H)) {
    case 1: return bf16 ? launch_norm<true, 1>(p, stream) : launch_norm<false, 1>(p, stream);
    case 2: return bf16 ? launch_norm<true, 2>(p, stream) : launch_norm<false, 2>(p, stream);
    default: return bf16 ? launch_norm<true, 4>(p, stream) : launch_norm<false, 4>(p, stream);
    }
}

extern "C" moe_status moe_block_norm_backward_workspace_size(int64_t T, int32_t H, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_norm_sizes(T, H, MOE_IO_BF16))
        return static_cast<moe_status>(st);
    *bytes = static_cast<size_t>(most_ctas(T)) * kSums * H * 4;
    return MOE_OK;
}

extern "C" moe_status moe_block_norm_backward(const moe_block_norm_backward_args *a, moe_stream_t stream)
{
    if (!a)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_norm_sizes(a->T, a->H, a->io_dtype))
        return static_cast<moe_status>(st);
    if (!aligned16(a->d_post_gamma) || !aligned16(a->d_pre_gamma) || (reinterpret_cast<uintptr_t>(a->d_gate) & (a->gate_kind == MOE_GATE_CHANNEL ? 15u : 3u)) ||
        (a->d_gate && a->gate_kind != MOE_GATE_CHANNEL && a->gate_kind != MOE_GATE_TOKEN))
        return MOE_ERR_INVALID_ARG;
    const bool channel = a->d_gate && a->gate_kind == MOE_GATE_CHANNEL, columns = a->d_post_gamma || a->d_pre_gamma || channel;
    if (a->T == 0) {
        moe_status st = zero_floats(a->d_post_gamma, a->H, stream);
        st = st == MOE_OK ? zero_floats(a->d_pre_gamma, a->H, stream) : st;
        return st == MOE_OK && channel ? zero_floats(a->d_gate, a->H, stream) : st;
    }
    if (!valid_norm(a) || !aligned16(a->d_residual_out) || !aligned16(a->d_norm_out) || !aligned16(a->d_y) || !aligned16(a->d_residual) ||
        (!a->d_residual_out && !a->d_norm_out) || (a->d_norm_out && !a->pre_gamma) || (a->d_residual && !a->residual) ||
        (a->d_post_gamma && !a->post_gamma) || (a->d_pre_gamma && !a->d_norm_out) || (a->d_y && a->d_y == a->d_residual) ||
        (!a->d_y && !a->d_residual && !a->d_gate && !columns))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_block_norm_backward_workspace_size(a->T, a->H, &need);
    if (columns && (!a->workspace || a->workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (columns && !aligned16(a->workspace))
        return MOE_ERR_INVALID_ARG;
    NormParams p = norm_params(a);
    p.d_residual_out = static_cast<const uint8_t *>(a->d_residual_out);
    p.d_norm_out = static_cast<const uint8_t *>(a->d_norm_out);
    p.d_y = static_cast<uint8_t *>(a->d_y);
    p.d_residual = static_cast<uint8_t *>(a->d_residual);
    p.d_post = a->d_post_gamma;
    p.d_pre = a->d_pre_gamma;
    p.d_gate = a->d_gate;
    p.partial = columns ? static_cast<float *>(a->workspace) : nullptr;
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    switch (vectors_per_thread(a->H)) {
    case 1: return bf16 ? launch_backward<true, 1>(p, stream) : launch_backward<false, 1>(p, stream);
    case 2: return bf16 ? launch_backward<true, 2>(p, stream) : launch_backward<false, 2>(p, stream);
    default: return bf16 ? launch_backward<true, 4>(p, stream) : launch_backward<false, 4>(p, stream);
    }
}
