// layer.cu -- a whole expert layer for a few tokens, in two kernels.
//
//   gate_up  a[t, e] = w[t, e] act(W1[e] x[t]) (W3[e] x[t])   for every expert e that a token takes
//   down     out[t]  = sum_e W2[e] a[t, e] + shared[t] + residual[t]
//
// Both are bound by the weights of the experts taken, 3 H I elements each,
// which are read once.  The router's weight w[t, e] is multiplied into a, so
// the second product sums over experts without a further step.
//
// Every CTA makes the list of experts taken and of the tokens of each for
// itself, from the ids: at most 64 tokens, one bit each.  Tokens of an expert
// are ordered by their index and experts by theirs, so the sums have the same
// order in every call.
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
constexpr int kThreads = 32 * kWarps;
constexpr int kTileRows = 16;

struct LayerParams {
    WeightView W13, W2;
    const float *w13_global, *w2_global;
    const uint16_t *x, *shared, *residual;
    uint16_t *out, *act;  // act: workspace, [pairs, I], pairs in the order of the list
    const int32_t *ids;
    const void *weights;
    int32_t *status;
    int64_t x_stride;
    int32_t T, H, I, E, k, weight_dtype, gelu;
};

// The experts taken, in ascending order, and the tokens of each.  A pair is
// an expert and one of its tokens.
struct Lists {
    uint32_t *mask;    // [E][2]: a bit for each token
    int32_t *expert;   // [experts taken]
    int32_t *first;    // [experts taken + 1]: the first pair of each
    float *weight;     // [pairs]
    uint8_t *token;    // [pairs]
    int32_t *scratch;  // [kWarps]
    int32_t taken;
};

__host__ __device__ inline int most_taken(int E, int slots) { return E < slots ? E : slots; }

__host__ __device__ inline size_t lists_bytes(int E, int slots)
{
    return 8 * static_cast<size_t>(E) + 4 * (2 * static_cast<size_t>(most_taken(E, slots)) + 1) +
           5 * static_cast<size_t>(slots) + 4 * kWarps + 16;
}

__device__ __forceinline__ float load_weight(const LayerParams &p, int64_t i)
{
    if (p.weight_dtype == MOE_WEIGHTS_FP32)
        return static_cast<const float *>(p.weights)[i];
    const uint16_t v = static_cast<const uint16_t *>(p.weights)[i];
    return p.weight_dtype == MOE_WEIGHTS_BF16 ? widen16<true>(v) : widen16<false>(v);
}

// All threads of the CTA.
__device__ void build_lists(Lists &L, const LayerParams &p, uint8_t *smem, bool want_weights)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slots = p.T * p.k, most = most_taken(p.E, slots);
    L.mask = reinterpret_cast<uint32_t *>(smem);
    L.expert = reinterpret_cast<int32_t *>(L.mask + 2 * p.E);
    L.first = L.expert + most;
    L.scratch = L.first + most + 1;
    L.weight = reinterpret_cast<float *>(L.scratch + kWarps);
    L.token = reinterpret_cast<uint8_t *>(L.weight + slots);
    for (int i = tid; i < 2 * p.E; i += kThreads)
        L.mask[i] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += kThreads) {
        const int e = p.ids[i], t = i / p.k;
        if (e >= 0 && e < p.E)
            atomicOr(&L.mask[2 * e + (t >> 5)], 1u << (t & 31));
        else if (e != -1 && p.status)
            atomicCAS(p.status, 0, MOE_ERR_INVALID_EXPERT);
    }
    __syncthreads();
    // number the experts taken and their pairs: a scan of (1, tokens) over the experts, packed in one word
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += kThreads) {
        const int e = e0 + tid;
        const int tokens = e < p.E ? __popc(L.mask[2 * e]) + __popc(L.mask[2 * e + 1]) : 0;
        const int own = tokens ? (1 << 16) + tokens : 0;
        int scan = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
            if (lane >= d)
                scan += v;
        }
        if (lane == 31)
            L.scratch[warp] = scan;
        __syncthreads();
        int before = base;
        for (int w = 0; w < kWarps; ++w) {
            const int v = L.scratch[w];
            before += w < warp ? v : 0;
            base += v;
        }
        before += scan - own;
        if (tokens) {
            L.expert[before >> 16] = e;
            L.first[before >> 16] = before & 0xFFFF;
        }
        __syncthreads();
    }
    L.taken = base >> 16;
    if (tid == 0)
        L.first[L.taken] = base & 0xFFFF;
    __syncthreads();
    // a warp an expert: its tokens in order, with their weights
    for (int a = warp; a < L.taken; a += kWarps) {
        const int e = L.expert[a];
        int at = L.first[a];
        for (int h = 0; h < 2; ++h) {
            const uint32_t m = L.mask[2 * e + h];
            if (m >> lane & 1) {
                const int t = 32 * h + lane, q = at + __popc(m & ((1u << lane) - 1));
                L.token[q] = static_cast<uint8_t>(t);
                if (want_weights) {
                    float w = 0.0f;
                    for (int j = 0; j < p.k; ++j)
                        if (p.ids[t * p.k + j] == e)
                            w += load_weight(p, t * p.k + j);
                    L.weight[q] = w;
                }
            }
            at += __popc(m);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float activate(float g, bool gelu)
{
    if (gelu)
        return 0.5f * g * (1.0f + tanhf(0.7978845608f * (g + 0.044715f * g * g * g)));
    return g / (1.0f + expf(-g));
}

// Units are (expert taken, 8 values of its inner dimension): the rows of W1
// and of W3 for these 8 fill one 16-row tile, so that a lane ends up with both
// factors of the same value.  CTAs take equal, consecutive shares of the units.
template <int FMT, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT == 8 ? 1 : 2) gate_up_kernel(LayerParams p)
{
    using F = Format<FMT, BF16>;
    constexpr int kStep = 4 * F::kLane;
    constexpr int U = NT == 1 ? 4 : (NT == 2 ? 2 : 1);
    __shared__ float red[kWarps][kTileRows][8 * NT];
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    grid_dependency_wait();
    allow_dependent_launch();
    Lists L;
    build_lists(L, p, smem, true);

    const int slabs = (p.I + 7) / 8;
    const int64_t units = static_cast<int64_t>(L.taken) * slabs;
    const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
    const int steps = (p.H + kStep - 1) / kStep;
    const int k0 = warp * steps / kWarps * kStep, k1 = min((warp + 1) * steps / kWarps * kStep, p.H);
    for (int64_t u = units * blockIdx.x / gridDim.x; u < u1; ++u) {
        const int a = static_cast<int>(u / slabs), i0 = static_cast<int>(u % slabs) * 8;
        const int e = L.expert[a], first = L.first[a], tokens = L.first[a + 1] - first;
        const int64_t base = static_cast<int64_t>(e) * 2 * p.I + min(i0 + g, p.I - 1);
        const uint16_t *col[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            col[nt] = p.x + L.token[first + min(8 * nt + g, tokens - 1)] * p.x_stride;
        float acc[NT][4] = {};
        skinny_product<F, BF16, NT, U>(acc, p.W13, F::row(p.W13, base), F::row(p.W13, base + p.I), col,
                                       (tokens + 7) >> 3, k0, k1, lane);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            red[warp][g][8 * nt + 2 * t] = acc[nt][0];
            red[warp][g][8 * nt + 2 * t + 1] = acc[nt][1];
            red[warp][g + 8][8 * nt + 2 * t] = acc[nt][2];
            red[warp][g + 8][8 * nt + 2 * t + 1] = acc[nt][3];
        }
        __syncthreads();
        const float div = FMT == kWNvfp4 && p.w13_global ? p.w13_global[e] : 1.0f;
        for (int i = tid; i < 8 * tokens; i += kThreads) {
            const int r = i & 7, c = i >> 3;
            if (i0 + r >= p.I)
                continue;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                gate += red[w][r][c];
                up += red[w][r + 8][c];
            }
            const float v = activate(descale<F>(gate, div), p.gelu) * descale<F>(up, div) * L.weight[first + c];
            p.act[static_cast<int64_t>(first + c) * p.I + i0 + r] = narrow16<BF16>(v);
        }
        __syncthreads();
    }
}

// A CTA computes 16 values of every token's row.  Its warps share the steps
// of all experts taken equally; each adds an expert's sums to its own
// [T, 16] part in shared memory, and the parts are added in warp order.
template <int FMT, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT == 8 ? 1 : 2) down_kernel(LayerParams p)
{
    using F = Format<FMT, BF16>;
    constexpr int kStep = 4 * F::kLane;
    constexpr int U = NT == 1 ? 4 : (NT == 2 ? 2 : 1);
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * kTileRows;
    // the ids were complete before the first kernel of this call started
    float *parts = reinterpret_cast<float *>(smem);  // [kWarps][T][16]
    Lists L;
    build_lists(L, p, smem + sizeof(float) * kWarps * p.T * kTileRows, false);
    for (int i = tid; i < kWarps * p.T * kTileRows; i += kThreads)
        parts[i] = 0.0f;
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();

    float *mine = parts + warp * p.T * kTileRows;
    const int steps = (p.I + kStep - 1) / kStep;
    const int total = L.taken * steps;
    int s = static_cast<int>(static_cast<int64_t>(total) * warp / kWarps);
    const int s1 = static_cast<int>(static_cast<int64_t>(total) * (warp + 1) / kWarps);
    while (s < s1) {
        const int a = s / steps, from = s - a * steps, to = min(steps, from + s1 - s);
        const int e = L.expert[a], first = L.first[a], tokens = L.first[a + 1] - first;
        const int64_t base = static_cast<int64_t>(e) * p.H;
        const uint16_t *col[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            col[nt] = p.act + static_cast<int64_t>(first + min(8 * nt + g, tokens - 1)) * p.I;
        float acc[NT][4] = {};
        skinny_product<F, BF16, NT, U>(acc, p.W2, F::row(p.W2, base + min(n0 + g, p.H - 1)),
                                       F::row(p.W2, base + min(n0 + g + 8, p.H - 1)), col, (tokens + 7) >> 3,
                                       from * kStep, min(to * kStep, p.I), lane);
        const float div = FMT == kWNvfp4 && p.w2_global ? p.w2_global[e] : 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 8 * nt + 2 * t + (i & 1);
                if (c < tokens)
                    mine[L.token[first + c] * kTileRows + g + (i & 2) * 4] += descale<F>(acc[nt][i], div);
            }
        s += to - from;
    }
    __syncthreads();
    for (int i = tid; i < p.T * kTileRows; i += kThreads) {
        const int n = n0 + (i & (kTileRows - 1));
        if (n >= p.H)
            continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += parts[w * p.T * kTileRows + i];
        const int64_t o = static_cast<int64_t>(i / kTileRows) * p.H + n;
        if (p.shared)
            v += widen16<BF16>(p.shared[o]);
        if (p.residual)
            v += widen16<BF16>(p.residual[o]);
        p.out[o] = narrow16<BF16>(v);
    }
}

template <int FMT, bool BF16, int NT>
moe_status launch_layer(const LayerParams &p, moe_stream_t stream)
{
    static SmemLimit gate_limit, down_limit;
    int dev = 0;
    const int sms = sm_count();
    if (cudaGetDevice(&dev) != cudaSuccess || sms <= 0)
        return MOE_ERR_CUDA;
    const size_t lists = lists_bytes(p.E, p.T * p.k);
    const size_t down = lists + sizeof(float) * kWarps * p.T * kTileRows;
    const auto gate_up = gate_up_kernel<FMT, BF16, NT>;
    const auto down_k = down_kernel<FMT, BF16, NT>;
    if (ensure_dynamic_smem(gate_up, dev, static_cast<int>(lists), gate_limit) != cudaSuccess ||
        ensure_dynamic_smem(down_k, dev, static_cast<int>(down), down_limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int64_t most_units = static_cast<int64_t>(most_taken(p.E, p.T * p.k)) * ((p.I + 7) / 8);
    const int64_t grid = most_units < 2 * sms ? most_units : 2 * sms;
    const moe_status st =
        PdlLaunch(static_cast<unsigned>(grid), kThreads, lists, stream).run(gate_up, p);
    if (st != MOE_OK)
        return st;
    return PdlLaunch(static_cast<unsigned>((p.H + kTileRows - 1) / kTileRows), kThreads, down, stream).run(down_k, p);
}

template <int FMT, bool BF16>
moe_status launch_layer(const LayerParams &p, moe_stream_t stream)
{
    return p.T <= 8    ? launch_layer<FMT, BF16, 1>(p, stream)
           : p.T <= 16 ? launch_layer<FMT, BF16, 2>(p, stream)
           : p.T <= 32 ? launch_layer<FMT, BF16, 4>(p, stream)
                       : launch_layer<FMT, BF16, 8>(p, stream);
}

bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" size_t moe_layer_args_size(void) { return sizeof(moe_layer_args); }

extern "C" moe_status moe_layer_workspace_size(int64_t T, int32_t top_k, int32_t I, size_t *bytes)
{
    if (!bytes || T < 0 || top_k < 1 || I < 1)
        return MOE_ERR_INVALID_ARG;
    if (T > MOE_FEW_TOKENS || top_k > MOE_MAX_TOP_K || I > MOE_FEW_MAX_DIM)
        return MOE_ERR_UNSUPPORTED;
    // a row of I 16-bit values for every slot
    *bytes = (static_cast<size_t>(T) * top_k * I * 2 + 255) / 256 * 256;
    return MOE_OK;
}

extern "C" moe_status moe_layer(const moe_layer_args *a, moe_stream_t stream)
{
    if (!a || a->T < 0 || a->H < 1 || a->I < 1 || a->E < 1 || a->top_k < 1)
        return MOE_ERR_INVALID_ARG;
    if (a->w_format < MOE_W_16 || a->w_format > MOE_W_INT4 || (a->io_dtype != MOE_IO_BF16 && a->io_dtype != MOE_IO_FP16) ||
        a->weight_dtype < MOE_WEIGHTS_FP32 || a->weight_dtype > MOE_WEIGHTS_FP16 ||
        (a->activation != MOE_ACT_SILU && a->activation != MOE_ACT_GELU_TANH))
        return MOE_ERR_INVALID_ARG;
    const bool int4 = a->w_format == MOE_W_INT4, nvfp4 = a->w_format == MOE_W_NVFP4;
    const int shift = int4 ? group_shift(a->group_size) : nvfp4 ? 4 : 3;
    if (shift < 0 || a->H % (1 << shift) != 0 || a->I % (1 << shift) != 0)
        return MOE_ERR_INVALID_ARG;
    if (a->T > MOE_FEW_TOKENS || a->E > MOE_LAYER_MAX_EXPERTS || a->top_k > MOE_MAX_TOP_K || a->H > MOE_FEW_MAX_DIM ||
        a->I > MOE_FEW_MAX_DIM)
        return MOE_ERR_UNSUPPORTED;
    if (a->T == 0)
        return MOE_OK;
    if (!a->x || !a->topk_ids || !a->router_weights || !a->w13 || !a->w2 || !a->out || !aligned16(a->x) ||
        !aligned16(a->w13) || !aligned16(a->w2) || misaligned(a->topk_ids, 3) ||
        misaligned(a->router_weights, a->weight_dtype == MOE_WEIGHTS_FP32 ? 3 : 1) || misaligned(a->shared_out, 1) ||
        misaligned(a->residual, 1) || misaligned(a->out, 1) || misaligned(a->status, 3) ||
        misaligned(a->w13_global, 3) || misaligned(a->w2_global, 3))
        return MOE_ERR_INVALID_ARG;
    if ((int4 || nvfp4) && (!a->w13_scales || !a->w2_scales))
        return MOE_ERR_INVALID_ARG;
    if (int4 && (misaligned(a->w13_scales, 1) || misaligned(a->w2_scales, 1)))
        return MOE_ERR_INVALID_ARG;
    if ((!int4 && (a->w13_zeros || a->w2_zeros)) || (!nvfp4 && (a->w13_global || a->w2_global)))
        return MOE_ERR_INVALID_ARG;
    if (a->x_stride < a->H || a->x_stride % 8 != 0)
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    const moe_status st = moe_layer_workspace_size(a->T, a->top_k, a->I, &need);
    if (st != MOE_OK)
        return st;
    if (!a->workspace || a->workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    if (!aligned16(a->workspace))
        return MOE_ERR_INVALID_ARG;
    const auto u8 = [](const void *q) { return static_cast<const uint8_t *>(q); };
    const auto u16 = [](const void *q) { return static_cast<const uint16_t *>(q); };
    const LayerParams p{{u8(a->w13), u8(a->w13_scales), u8(a->w13_zeros), a->H, shift},
                        {u8(a->w2), u8(a->w2_scales), u8(a->w2_zeros), a->I, shift},
                        a->w13_global,
                        a->w2_global,
                        u16(a->x),
                        u16(a->shared_out),
                        u16(a->residual),
                        static_cast<uint16_t *>(a->out),
                        static_cast<uint16_t *>(a->workspace),
                        a->topk_ids,
                        a->router_weights,
                        a->status,
                        a->x_stride,
                        static_cast<int32_t>(a->T),
                        a->H,
                        a->I,
                        a->E,
                        a->top_k,
                        a->weight_dtype,
                        a->activation == MOE_ACT_GELU_TANH};
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    if (int4)
        return bf16 ? launch_layer<kWInt4, true>(p, stream) : launch_layer<kWInt4, false>(p, stream);
    if (nvfp4)
        return bf16 ? launch_layer<kWNvfp4, true>(p, stream) : launch_layer<kWNvfp4, false>(p, stream);
    return bf16 ? launch_layer<kW16, true>(p, stream) : launch_layer<kW16, false>(p, stream);
}
