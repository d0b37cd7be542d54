// block_norm.cu -- the norms after a block and before the next one, with the
// block's gate and the residual's scale, forward and backward.
//
// Few operations a byte, so both passes are bound by HBM: what counts is bytes in flight.  One CTA an SM holds rows in
// slots of shared memory, which bulk copies (TMA) fill as far ahead as there is room.  Groups of warps (as many as
// a row of VPT vectors of 8 a thread takes, several groups a CTA for narrow rows) take the CTA's rows in turn, each
// with slots of its own; a row's values stay in shared memory and registers between the sums over it.  One thread of a
// group issues the copies (a producer warp of its own would make 17 warps, and leave 96 registers a thread).
//
// Backward.  With n = y / rms(y), m = s / rms(s) and c = block_scale * gate * (post_gamma + bias):
//   ds = d_residual_out + (v - m mean(v m)) / rms(s),   v = d_norm_out * (pre_gamma + bias)
//   d_y = (c ds - n mean(c ds n)) / rms(y)
// The sums over tokens of all three vectors are made of two: A = sum of ds n and B = sum of d_norm_out m, as
// d_post_gamma = block_scale gate A, d_gate = block_scale (post_gamma + bias) A and d_pre_gamma = B (a gate for each token
// goes into A).  A thread has its columns' A and B in registers over all rows of its CTA; groups are added up in shared memory,
// CTAs by a second kernel, each in its order.  Rows wider than 8192 leave no room for that: their kernel has A and B in
// shared memory and rows in registers.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "block.h"
#include "block_math.cuh"
#include "few_token.h"

namespace nqg {
namespace {

constexpr int kWarps = 16;
constexpr int kMaxThreads = 32 * kWarps;
constexpr int kMaxSlots = 64;
constexpr int kRingBytes = 220 * 1024;
constexpr int kMaxRingWidth = 8192;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

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
    float *partial;  // backward: [CTAs, 2, H], or nullptr where no sum over tokens is asked for
    int32_t ctas;
    int32_t slots, group_warps, groups, stage;  // slots of a group, of `stage` bytes each
    int32_t at_residual, at_d_norm, at_d_residual;  // where in a slot
    int64_t stall;
};

struct RingSmem {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    float red[kWarps][2][2][kWarps];  // of each group: two buffers in turn, two sums, a value a warp
};

template <bool BF16>
__device__ __forceinline__ void load8(float (&v)[8], const uint8_t *p)
{
    unpack8<BF16>(*reinterpret_cast<const uint4 *>(p), v);
}

// gamma + weight_bias of 8 columns (1 without gamma).
template <bool BF16>
__device__ __forceinline__ void gammas8(float (&v)[8], bool given, const uint4 &gamma, float bias)
{
    unpack8<BF16>(gamma, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = given ? v[i] + bias : 1.0f;
}

// block_scale * gate * (post_gamma + bias) of 8 columns; a token's gate is left out.
template <bool BF16>
__device__ __forceinline__ void factors8(float (&v)[8], const NormParams &p, const uint4 &post, const uint4 &gate)
{
    gammas8<BF16>(v, p.post != nullptr, post, p.bias);
    float g[8];
    unpack8<BF16>(gate, g);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] *= p.gate_kind == MOE_GATE_CHANNEL ? p.block_scale * g[i] : p.block_scale;
}

__device__ __forceinline__ float token_gate(const NormParams &p, int64_t t)
{
    return p.gate_kind == MOE_GATE_TOKEN ? __ldg(reinterpret_cast<const float *>(p.gate) + t) : 1.0f;
}

__device__ __forceinline__ uint4 vector_of(const uint8_t *p, int i, bool take)
{
    return take ? ldg16(p + 16 * i) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void store8(uint8_t *p, const uint4 &v) { *reinterpret_cast<uint4 *>(p) = v; }

// A group of warps that share a row.
struct Group {
    int warps, warp, lane, index;
    float (*red)[2][kWarps];
    int turn;

    // Sums of N <= 2 values over the group, in every thread.  One barrier: two buffers in turn, and a thread that
    // writes one again has passed the barrier behind every thread's reads of it.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N])
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int o = 16; o; o >>= 1)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (warps == 1)
            return;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane == 0)
                red[turn][i][warp] = v[i];
        named_barrier_sync(1 + index, 32 * warps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = lane < warps ? red[turn][i][lane] : 0.0f;
#pragma unroll
            for (int o = 8; o; o >>= 1)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            v[i] = __shfl_sync(0xffffffffu, v[i], 0);
        }
        turn ^= 1;
    }
};

__device__ __forceinline__ void ring_init(const NormParams &p, RingSmem &r)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.slots * p.groups; ++i) {
            mbar_init(smem_u32(&r.full[i]), 1);
            mbar_init(smem_u32(&r.empty[i]), static_cast<uint32_t>(p.group_warps));
        }
        fence_mbar_init();
    }
    __syncthreads();
}

// A group's rows: t, t + step, and so on, each in the next of its slots.
struct Rows {
    const NormParams &p;
    uint8_t *at;  // the slot of the row that is being worked on
    uint32_t full, empty;
    uint32_t t, step, fills;  // rows are below 2^31; fills: copies that may still be issued
    int slot;
    uint32_t phase, bytes;
    bool issues, backward, lost;

    __device__ __forceinline__ Rows(const NormParams &q, RingSmem &r, uint8_t *ring, const Group &g, bool back)
        : p(q), at(ring + static_cast<uint32_t>(g.index * q.slots) * q.stage), full(smem_u32(&r.full[g.index * q.slots])),
          empty(smem_u32(&r.empty[g.index * q.slots])), t(blockIdx.x + g.index * gridDim.x), step(q.groups * gridDim.x),
          slot(0), phase(0), issues(g.warp == 0 && g.lane == 0), backward(back),
          lost(false)
    {
        bytes = 2u * static_cast<uint32_t>(q.H) * (1u + (q.residual != nullptr) + (back && q.d_norm_out) + (back && q.d_residual_out));
        fills = blockIdx.x == 0 && g.index == 0 && q.stall >= 0 && q.stall < 0xFFFFFFFF ? static_cast<uint32_t>(q.stall) : 0xFFFFFFFFu;  // test hook (moe_debug_stall)
        for (int i = 0; issues && i < q.slots; ++i)
            fill(t + i * step, i, at + static_cast<uint32_t>(i) * q.stage);
    }

    __device__ __forceinline__ void fill(uint32_t row, int to, const uint8_t *place)
    {
        if (row >= p.T || fills == 0)
            return;
        --fills;
        const uint32_t row_bytes = 2u * static_cast<uint32_t>(p.H), dst = smem_u32(place), bar = full + 8u * to;
        const int64_t from = static_cast<int64_t>(row) * row_bytes;
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(dst, p.y + from, row_bytes, bar);
        if (p.residual)
            bulk_g2s(dst + p.at_residual, p.residual + from, row_bytes, bar);
        if (backward && p.d_norm_out)
            bulk_g2s(dst + p.at_d_norm, p.d_norm_out + from, row_bytes, bar);
        if (backward && p.d_residual_out)
            bulk_g2s(dst + p.at_d_residual, p.d_residual_out + from, row_bytes, bar);
    }

    // Waits for the row; 0, or NaN once a wait has run out: it makes the row's sums and values NaN, and no further wait is made.
    __device__ __forceinline__ float wait()
    {
        lost = lost || !mbar_wait_bounded(full + 8u * slot, phase, kWaitLimitNs);
        return lost ? __int_as_float(0x7FC00000) : 0.0f;
    }

    // The row's slot has been read: the row that comes next into it.
    __device__ __forceinline__ void release(int lane)
    {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(empty + 8u * slot);
        if (issues && !lost && t + p.slots * step < p.T) {
            if (mbar_wait_bounded(empty + 8u * slot, phase, kWaitLimitNs))
                fill(t + p.slots * step, slot, at);
            else
                fills = 0;
        }
        t += step;
        at += p.stage;
        if (++slot == p.slots) {
            slot = 0;
            phase ^= 1;
            at -= static_cast<uint32_t>(p.slots) * p.stage;
        }
    }

    // Copies that were never waited for land before the CTA leaves.
    __device__ __forceinline__ void finish()
    {
        if (!issues || !lost)
            return;
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < p.slots; ++i)
            while (!mbar_try_wait(full + 8u * i, i >= slot ? phase : phase ^ 1) && globaltimer_ns() - t0 < kWaitLimitNs / 4) {
            }
    }
};

template <bool BF16, int VPT>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const NormParams p)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingSmem r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ring_init(p, r);
    grid_dependency_wait();
    {
        Group g{p.group_warps, warp % p.group_warps, lane, warp / p.group_warps, r.red[warp / p.group_warps], 0};
        Rows rows(p, r, ring, g, false);
        const int vectors = p.H / 8, threads = 32 * g.warps, first = 32 * g.warp + lane;
        // both factors of a column stay in registers where there is room, and come from L1 at each use where not
        constexpr bool kKeep = VPT <= 2;
        const auto factors = [&](float (&c)[8], int i) {
            factors8<BF16>(c, p, vector_of(p.post, i, i < vectors && p.post), vector_of(p.gate, i, i < vectors && p.gate_kind == MOE_GATE_CHANNEL));
        };
        const auto pre_gammas = [&](float (&c)[8], int i) { gammas8<BF16>(c, p.pre != nullptr, vector_of(p.pre, i, i < vectors && p.pre), p.bias); };
        float kept[kKeep ? VPT : 1][8], kept2[kKeep ? VPT : 1][8];
        if constexpr (kKeep)
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                factors(kept[j], first + j * threads);
                pre_gammas(kept2[j], first + j * threads);
            }
        while (rows.t < p.T) {
            const float lost = rows.wait();
            const uint8_t *at = rows.at;
            const int64_t t = rows.t, row = 2 * t * p.H;
            float s[VPT][8], sum[1] = {lost};
            float ry = 1.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[j][k] = 0.0f;
                if (i < vectors)
                    load8<BF16>(s[j], at + 16 * i);
            }
            if (p.post) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sum[0] = fmaf(s[j][k], s[j][k], sum[0]);
                g.sum(sum);
                ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            }
            ry *= token_gate(p, t);
            sum[0] = lost;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
                float res[8] = {}, c[8];
                if (p.residual && i < vectors)
                    load8<BF16>(res, at + p.at_residual + 16 * i);
                if constexpr (!kKeep)
                    factors(c, i);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[j][k] = fmaf(s[j][k], ry * (kKeep ? kept[kKeep ? j : 0][k] : c[k]), p.residual ? p.residual_scale * res[k] : 0.0f) + lost;
                    sum[0] = fmaf(s[j][k], s[j][k], sum[0]);
                }
            }
            rows.release(lane);
            if (p.residual_out)
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (first + j * threads < vectors)
                        store8(p.residual_out + row + 16 * (first + j * threads), pack8<BF16>(s[j]));
            if (!p.norm_out)
                continue;
            g.sum(sum);
            const float rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float c[8];
                if constexpr (!kKeep)
                    pre_gammas(c, first + j * threads);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[j][k] *= rs * (kKeep ? kept2[kKeep ? j : 0][k] : c[k]);
                if (first + j * threads < vectors)
                    store8(p.norm_out + row + 16 * (first + j * threads), pack8<BF16>(s[j]));
            }
        }
        rows.finish();
    }
    allow_dependent_launch();
}

template <bool BF16>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_kernel(const NormParams p)
{
    constexpr int VPT = 2;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingSmem r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ring_init(p, r);
    grid_dependency_wait();
    Group g{p.group_warps, warp % p.group_warps, lane, warp / p.group_warps, r.red[warp / p.group_warps], 0};
    const int vectors = p.H / 8, threads = 32 * g.warps, first = 32 * g.warp + lane;
    float A[VPT][8] = {}, B[VPT][8] = {};
    {
        Rows rows(p, r, ring, g, true);
        // the three vectors come from L1 at each use: registers are for A and B
        const auto factors = [&](float (&c)[8], int i) {
            factors8<BF16>(c, p, vector_of(p.post, i, i < vectors && p.post), vector_of(p.gate, i, i < vectors && p.gate_kind == MOE_GATE_CHANNEL));
        };
        const auto pre_gammas = [&](float (&c)[8], int i) { gammas8<BF16>(c, true, vector_of(p.pre, i, i < vectors && p.pre), p.bias); };
        while (rows.t < p.T) {
            const float lost = rows.wait();
            const uint8_t *at = rows.at;
            const int64_t t = rows.t, row = 2 * t * p.H;
            float ry = 1.0f;
            if (p.post) {
                float sum[1] = {lost};
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = first + j * threads;
                    float y[8] = {};
                    if (i < vectors)
                        load8<BF16>(y, at + 16 * i);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sum[0] = fmaf(y[k], y[k], sum[0]);
                }
                g.sum(sum);
                ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            }
            const float token = token_gate(p, t);
            float s[VPT][8];  // s, and then ds
            float sum[2] = {lost, lost};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
                float y[8] = {}, res[8] = {}, d[8] = {}, c[8];
                if (i < vectors) {
                    load8<BF16>(y, at + 16 * i);
                    if (p.residual)
                        load8<BF16>(res, at + p.at_residual + 16 * i);
                    if (p.d_norm_out)
                        load8<BF16>(d, at + p.at_d_norm + 16 * i);
                }
                factors(c, i);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[j][k] = fmaf(y[k], token * ry * c[k], p.residual ? p.residual_scale * res[k] : 0.0f);
                    sum[0] = fmaf(s[j][k], s[j][k], sum[0]);
                }
                pre_gammas(c, i);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum[1] = fmaf(s[j][k], d[k] * c[k], sum[1]);
            }
            float rs = 0.0f, back = lost;  // back: mean(v m) / rms(s)^2
            if (p.d_norm_out) {
                g.sum(sum);
                rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
                back = sum[1] * p.inv_h * rs * rs * rs;
            }
            float dot[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
                float y[8] = {}, d[8] = {}, dr[8] = {}, c[8];
                if (i < vectors) {
                    load8<BF16>(y, at + 16 * i);
                    if (p.d_norm_out)
                        load8<BF16>(d, at + p.at_d_norm + 16 * i);
                    if (p.d_residual_out)
                        load8<BF16>(dr, at + p.at_d_residual + 16 * i);
                }
                pre_gammas(c, i);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    B[j][k] = fmaf(d[k], s[j][k] * rs, B[j][k]);
                    s[j][k] = fmaf(rs, d[k] * c[k], fmaf(-back, s[j][k], dr[k]));
                }
                factors(c, i);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    dot[0] = fmaf(s[j][k], c[k] * y[k], dot[0]);
                    A[j][k] = fmaf(s[j][k], y[k] * (ry * token), A[j][k]);
                }
            }
            if (p.post || p.gate_kind == MOE_GATE_TOKEN)
                g.sum(dot);
            if (p.d_gate && p.gate_kind == MOE_GATE_TOKEN && g.warp == 0 && lane == 0)
                p.d_gate[t] = dot[0] * ry;
            const float pull = p.post ? dot[0] * p.inv_h * token * ry * ry * ry : 0.0f;  // mean(c ds n) / rms(y)^2
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
                if (i >= vectors)
                    continue;
                if (p.d_y) {
                    float y[8], c[8];
                    load8<BF16>(y, at + 16 * i);
                    factors(c, i);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        c[k] = fmaf(ry * token, c[k] * s[j][k], -pull * y[k]);
                    store8(p.d_y + row + 16 * i, pack8<BF16>(c));
                }
                if (p.d_residual) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        s[j][k] *= p.residual_scale;
                    store8(p.d_residual + row + 16 * i, pack8<BF16>(s[j]));
                }
            }
            rows.release(lane);
        }
        rows.finish();
    }
    if (p.partial) {
        // the groups' sums, added up in their order in the ring's memory
        float *sums = reinterpret_cast<float *>(ring);  // [2, H]
        for (int turn = 0; turn < p.groups; ++turn) {
            __syncthreads();
            if (g.index != turn)
                continue;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = first + j * threads;
                if (i >= vectors)
                    continue;
                float4 *a = reinterpret_cast<float4 *>(sums + 8 * i), *b = reinterpret_cast<float4 *>(sums + p.H + 8 * i);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 x = turn ? a[k] : make_float4(0, 0, 0, 0), y = turn ? b[k] : make_float4(0, 0, 0, 0);
                    x.x += A[j][4 * k], x.y += A[j][4 * k + 1], x.z += A[j][4 * k + 2], x.w += A[j][4 * k + 3];
                    y.x += B[j][4 * k], y.y += B[j][4 * k + 1], y.z += B[j][4 * k + 2], y.w += B[j][4 * k + 3];
                    a[k] = x;
                    b[k] = y;
                }
            }
        }
        __syncthreads();
        float4 *out = reinterpret_cast<float4 *>(p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.H);
        for (int i = threadIdx.x; i < p.H / 2; i += blockDim.x)
            out[i] = reinterpret_cast<float4 *>(ring)[i];
    }
    allow_dependent_launch();
}

// The backward pass of wider rows: a row at a time in registers, A and B in shared memory.
template <bool BF16>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_wide_kernel(const NormParams p)
{
    constexpr int VPT = MOE_MAX_HIDDEN / 8 / kMaxThreads;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][2][kWarps];
    float *A = reinterpret_cast<float *>(ring), *B = A + p.H;
    grid_dependency_wait();
    const int vectors = p.H / 8;
    Group g{kMaxThreads / 32, static_cast<int>(threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31), 0, red, 0};
    for (int i = threadIdx.x; p.partial && i < vectors; i += kMaxThreads)
        for (int k = 0; k < 8; ++k)
            A[8 * i + k] = B[8 * i + k] = 0.0f;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t row = 2 * t * p.H;
        uint4 y[VPT], r[VPT], d[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * kMaxThreads;
            y[j] = r[j] = d[j] = make_uint4(0, 0, 0, 0);
            if (i < vectors) {
                y[j] = *reinterpret_cast<const uint4 *>(p.y + row + 16 * i);
                if (p.residual)
                    r[j] = *reinterpret_cast<const uint4 *>(p.residual + row + 16 * i);
                if (p.d_norm_out)
                    d[j] = *reinterpret_cast<const uint4 *>(p.d_norm_out + row + 16 * i);
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
                for (int k = 0; k < 8; ++k)
                    sum[0] = fmaf(v[k], v[k], sum[0]);
            }
            g.sum(sum);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const float token = token_gate(p, t);
        const auto new_residual = [&](int j, int i, float (&a)[8], float (&c)[8], float (&s)[8]) {
            unpack8<BF16>(y[j], a);
            unpack8<BF16>(r[j], s);
            factors8<BF16>(c, p, vector_of(p.post, i, p.post), vector_of(p.gate, i, p.gate_kind == MOE_GATE_CHANNEL));
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[k] = fmaf(a[k], token * ry * c[k], p.residual ? p.residual_scale * s[k] : 0.0f);
        };
        float sum[2] = {0.0f, 0.0f}, rs = 0.0f, back = 0.0f;
        if (p.d_norm_out) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = threadIdx.x + j * kMaxThreads;
                if (i >= vectors)
                    continue;
                float a[8], c[8], s[8], v[8];
                new_residual(j, i, a, c, s);
                unpack8<BF16>(d[j], v);
                gammas8<BF16>(c, true, ldg16(p.pre + 16 * i), p.bias);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    sum[0] = fmaf(s[k], s[k], sum[0]);
                    sum[1] = fmaf(s[k], v[k] * c[k], sum[1]);
                }
            }
            g.sum(sum);
            rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            back = sum[1] * p.inv_h * rs * rs * rs;
        }
        // ds of a vector, and what of it adds to A and B
        const auto gradient = [&](int j, int i, float (&a)[8], float (&c)[8], float (&ds)[8], bool add) {
            float s[8], v[8], c2[8];
            new_residual(j, i, a, c, s);
            unpack8<BF16>(d[j], v);
            const uint4 direct = p.d_residual_out ? *reinterpret_cast<const uint4 *>(p.d_residual_out + row + 16 * i) : make_uint4(0, 0, 0, 0);
            unpack8<BF16>(direct, ds);
            gammas8<BF16>(c2, true, vector_of(p.pre, i, p.pre), p.bias);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ds[k] = fmaf(rs, v[k] * c2[k], fmaf(-back, s[k], ds[k]));
                if (add) {
                    A[8 * i + k] = fmaf(ds[k], a[k] * (ry * token), A[8 * i + k]);
                    B[8 * i + k] = fmaf(v[k], s[k] * rs, B[8 * i + k]);
                }
            }
        };
        float dot[1] = {0.0f};
        if (p.post || p.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = threadIdx.x + j * kMaxThreads;
                if (i >= vectors)
                    continue;
                float a[8], c[8], ds[8];
                gradient(j, i, a, c, ds, false);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dot[0] = fmaf(ds[k], c[k] * a[k], dot[0]);
            }
            g.sum(dot);
        }
        if (p.d_gate && p.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
            p.d_gate[t] = dot[0] * ry;
        const float pull = p.post ? dot[0] * p.inv_h * token * ry * ry * ry : 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * kMaxThreads;
            if (i >= vectors)
                continue;
            float a[8], c[8], ds[8];
            gradient(j, i, a, c, ds, p.partial != nullptr);
            if (p.d_y) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    c[k] = fmaf(ry * token, c[k] * ds[k], -pull * a[k]);
                store8(p.d_y + row + 16 * i, pack8<BF16>(c));
            }
            if (p.d_residual) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    ds[k] *= p.residual_scale;
                store8(p.d_residual + row + 16 * i, pack8<BF16>(ds));
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; p.partial && i < 2 * p.H; i += kMaxThreads)
        p.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.H + i] = A[i];
    allow_dependent_launch();
}

// A and B over the CTAs, and the gradients that they make: 32 columns a block, 8 threads for each.
template <bool BF16>
__global__ void __launch_bounds__(256) column_sums_kernel(const NormParams p)
{
    __shared__ float part[2][8][32];
    grid_dependency_wait();
    const int column = threadIdx.x & 31, share = threadIdx.x >> 5, h = blockIdx.x * 32 + column;
    float a = 0.0f, b = 0.0f;
    if (h < p.H) {
#pragma unroll 4
        for (int i = share; i < p.ctas; i += 8) {
            const float *at = p.partial + static_cast<int64_t>(i) * 2 * p.H + h;
            a += at[0];
            b += at[p.H];
        }
    }
    part[0][share][column] = a;
    part[1][share][column] = b;
    __syncthreads();
    if (share == 0 && h < p.H) {
        for (int i = 1; i < 8; ++i) {
            a += part[0][i][column];
            b += part[1][i][column];
        }
        float gate = p.block_scale, post = p.block_scale, lo, hi;
        if (p.gate_kind == MOE_GATE_CHANNEL) {
            unpack2<BF16>(reinterpret_cast<const uint16_t *>(p.gate)[h], lo, hi);
            gate = p.block_scale * lo;
        }
        if (p.post) {
            unpack2<BF16>(reinterpret_cast<const uint16_t *>(p.post)[h], lo, hi);
            post = p.block_scale * (lo + p.bias);
        }
        if (p.d_post)
            p.d_post[h] = gate * a;
        if (p.d_pre)
            p.d_pre[h] = b;
        if (p.d_gate && p.gate_kind == MOE_GATE_CHANNEL)
            p.d_gate[h] = post * a;
    }
    allow_dependent_launch();
}

// CTAs of the backward pass whose sums the workspace has room for.
constexpr int64_t kMaxCtas = 512;
int64_t most_ctas(int64_t T) { return T < kMaxCtas ? T : kMaxCtas; }

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

// As many groups of warps as a CTA has room for, and as many slots for each.
unsigned plan_ring(NormParams &p, int vpt, int tensors)
{
    p.group_warps = (p.H / 8 + 32 * vpt - 1) / (32 * vpt);
    p.stage = (tensors * 2 * p.H + 127) / 128 * 128;
    const int room = kRingBytes / p.stage < kMaxSlots ? kRingBytes / p.stage : kMaxSlots;
    p.groups = kWarps / p.group_warps;
    p.groups = p.groups > room ? room : p.groups;
    p.slots = room / p.groups;
    return static_cast<unsigned>(32 * p.groups * p.group_warps);
}

template <bool BF16, int VPT>
moe_status launch_norm(NormParams &p, moe_stream_t stream)
{
    static SmemLimit limit;
    int dev = 0;
    const int sms = sm_count();
    p.at_residual = 2 * p.H;
    const unsigned threads = plan_ring(p, VPT, p.residual ? 2 : 1);
    const size_t smem = static_cast<size_t>(p.slots) * p.groups * p.stage;
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess ||
        ensure_dynamic_smem(norm_kernel<BF16, VPT>, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return PdlLaunch(static_cast<unsigned>(p.T < sms ? p.T : sms), threads, smem, stream).run(norm_kernel<BF16, VPT>, p);
}

template <bool BF16>
moe_status launch_backward(NormParams &p, moe_stream_t stream)
{
    static SmemLimit limits[2];
    int dev = 0;
    const int sms = sm_count();
    const bool wide = p.H > kMaxRingWidth;
    int at = 2 * p.H;
    p.at_residual = at;
    at += p.residual ? 2 * p.H : 0;
    p.at_d_norm = at;
    at += p.d_norm_out ? 2 * p.H : 0;
    p.at_d_residual = at;
    at += p.d_residual_out ? 2 * p.H : 0;
    unsigned threads = kMaxThreads;
    size_t smem = p.partial ? static_cast<size_t>(8) * p.H : 0;
    if (!wide) {
        threads = plan_ring(p, 2, at / (2 * p.H));
        // the ring's memory holds the sums at the end
        const size_t ring = static_cast<size_t>(p.slots) * p.groups * p.stage;
        smem = smem > ring ? smem : ring;
    }
    const auto kern = wide ? norm_backward_wide_kernel<BF16> : norm_backward_kernel<BF16>;
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess || ensure_dynamic_smem(kern, dev, static_cast<int>(smem), limits[wide]) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int64_t most = sms < kMaxCtas ? sms : kMaxCtas;
    p.ctas = static_cast<int32_t>(p.T < most ? p.T : most);
    const moe_status st = PdlLaunch(static_cast<unsigned>(p.ctas), threads, smem, stream).run(kern, p);
    if (st != MOE_OK || !p.partial)
        return st;
    return PdlLaunch(static_cast<unsigned>((p.H + 31) / 32), 256, 0, stream).run(column_sums_kernel<BF16>, p);
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
    p.stall = debug_stall_slots();
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    if (a->H <= kMaxRingWidth)
        return bf16 ? launch_norm<true, 2>(p, stream) : launch_norm<false, 2>(p, stream);
    return bf16 ? launch_norm<true, 4>(p, stream) : launch_norm<false, 4>(p, stream);
}

extern "C" moe_status moe_block_norm_backward_workspace_size(int64_t T, int32_t H, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    if (const int st = check_norm_sizes(T, H, MOE_IO_BF16))
        return static_cast<moe_status>(st);
    *bytes = static_cast<size_t>(most_ctas(T)) * 2 * H * 4;
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
    p.stall = debug_stall_slots();
    return a->io_dtype == MOE_IO_BF16 ? launch_backward<true>(p, stream) : launch_backward<false>(p, stream);
}
