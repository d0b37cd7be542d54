// select.cu -- expert selection: the top_k largest router logits of every
// token, in order, and their weights.
//
// One warp a token; lane l holds the logits of experts l, l + 32, ... in
// registers as order-preserving integers.  Each of the top_k rounds takes the
// largest value of the warp and the lowest expert index that has it, with two
// warp reductions, and closes that expert.  The work is a chain of top_k
// dependent rounds for a few hundred bytes a token: many warps in flight hide
// the chain, and a small batch is bound by it.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_layer.h"
#include "common.h"
#include "ptx.cuh"
#include "skinny.cuh"

namespace nqg {
namespace {

constexpr int kWarps = 4;

// A float's bits as an unsigned integer in the order of the floats, with -0
// equal to 0.  0 stands for a closed expert (-inf or NaN): no float that can
// be selected maps to it.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x > -INFINITY))
        return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

template <int DT>
__device__ __forceinline__ float load_logit(const void *row, int e)
{
    if constexpr (DT == MOE_WEIGHTS_FP32)
        return static_cast<const float *>(row)[e];
    return widen16<DT == MOE_WEIGHTS_BF16>(static_cast<const uint16_t *>(row)[e]);
}

struct SelectParams {
    const void *logits;
    int64_t T, stride;
    int32_t E, k, sigmoid, renorm;
    float scale;
    int32_t *ids;
    void *weights;
    int32_t weight_dtype;
};

constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ float finite_value(uint32_t key)
{
    return fminf(fmaxf(key_value(key), -kLargest), kLargest);
}

// The k largest of a warp's keys, key[i] of lane l at position l + 32 i:
// lane j < k gets the j-th largest and its position (equal keys by position),
// or 0 where fewer than k are open.  Closes what it takes.
template <int VPT>
__device__ __forceinline__ void take(uint32_t (&key)[VPT], int k, int lane, uint32_t &my_key, uint32_t &my_at)
{
    my_key = my_at = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0, at = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32u * i;
            }
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
        if (top == 0)
            break;
        at = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0xFFFFFFFFu);
        if (lane == j) {
            my_key = top;
            my_at = at;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (at == lane + 32u * i)
                key[i] = 0;
    }
}

template <int DT, int VPT>
__device__ __forceinline__ void load_keys(const SelectParams &p, int64_t t, int e0, int lane, uint32_t (&key)[VPT])
{
    const char *row = static_cast<const char *>(p.logits) + t * p.stride * (DT == MOE_WEIGHTS_FP32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = e0 + lane + 32 * i;
        key[i] = e < p.E ? order_key(load_logit<DT>(row, e)) : 0u;
    }
}

// Sum over the open keys of a warp of exp(value - most).
template <int VPT>
__device__ __forceinline__ float exp_sum(const uint32_t (&key)[VPT], float most)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        s += key[i] ? expf(finite_value(key[i]) - most) : 0.0f;
    return warp_sum(s);
}

// Lane j writes slot j of token t.  all: the softmax's sum over every open
// expert, relative to `most`, the largest value; unused otherwise.
__device__ __forceinline__ void write_slots(const SelectParams &p, int64_t t, int lane, uint32_t my_key, int my_id,
                                            float most, float all)
{
    // far below zero 1 + exp(l) is 1 in fp32: the sigmoids' ratios are those of
    // the exponentials, which relative to the largest do not all underflow
    const bool sigmoid = p.sigmoid && !(p.renorm && most < -60.0f);
    float w = 0.0f;
    if (my_key)
        w = sigmoid ? 1.0f / (1.0f + expf(-key_value(my_key))) : expf(finite_value(my_key) - most);
    const float taken = warp_sum(w);
    if (p.renorm || !p.sigmoid)
        w = my_key ? w / (p.renorm ? taken : all) : 0.0f;
    w *= p.scale;
    if (lane >= p.k)
        return;
    const int64_t o = t * p.k + lane;
    p.ids[o] = my_key ? my_id : -1;
    if (p.weight_dtype == MOE_WEIGHTS_FP32)
        static_cast<float *>(p.weights)[o] = w;
    else
        static_cast<uint16_t *>(p.weights)[o] =
            p.weight_dtype == MOE_WEIGHTS_BF16 ? narrow16<true>(w) : narrow16<false>(w);
}

// VPT: experts a lane holds, at least E / 32.
template <int DT, int VPT>
__global__ void __launch_bounds__(32 * kWarps) select_kernel(SelectParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    allow_dependent_launch();
    if (t >= p.T)
        return;
    uint32_t key[VPT], my_key, my_at;
    load_keys<DT>(p, t, 0, lane, key);
    const bool over_all = !p.sigmoid && !p.renorm;
    float most = 0.0f, all = 0.0f;
    if (over_all) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            best = max(best, key[i]);
        most = finite_value(__reduce_max_sync(0xFFFFFFFFu, best));
        all = exp_sum(key, most);
    }
    take(key, p.k, lane, my_key, my_at);
    if (!over_all)
        most = finite_value(__shfl_sync(0xFFFFFFFFu, my_key, 0));
    write_slots(p, t, lane, my_key, static_cast<int>(my_at), most, all);
}

// More than 1024 experts: a CTA a token.  Each warp takes the k largest of
// its own 1024 experts; they stay in order, so the position among all
// candidates orders equal values by their expert, and warp 0 takes the k
// largest of them.
template <int DT>
__global__ void __launch_bounds__(256) select_wide_kernel(SelectParams p)
{
    constexpr int kParts = MOE_MAX_EXPERTS / 1024;
    __shared__ uint32_t keys[kParts * MOE_MAX_TOP_K], at[kParts * MOE_MAX_TOP_K];
    __shared__ float sums[kParts];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    {
        uint32_t key[32], my_key, my_at;
        load_keys<DT>(p, t, 1024 * warp, lane, key);
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            best = max(best, key[i]);
        const float sum = exp_sum(key, finite_value(__reduce_max_sync(0xFFFFFFFFu, best)));
        take(key, p.k, lane, my_key, my_at);
        keys[warp * MOE_MAX_TOP_K + lane] = my_key;
        at[warp * MOE_MAX_TOP_K + lane] = 1024u * warp + my_at;
        if (lane == 0)
            sums[warp] = sum;
    }
    __syncthreads();
    if (warp != 0)
        return;
    uint32_t key[kParts], my_key, my_at;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        key[i] = keys[32 * i + lane];
    const uint32_t part = lane < kParts ? keys[32 * lane] : 0u;  // the largest of each warp's experts
    const float own_most = finite_value(part);
    const float most = finite_value(__reduce_max_sync(0xFFFFFFFFu, part));
    const float all = warp_sum(part ? sums[lane] * expf(own_most - most) : 0.0f);
    take(key, p.k, lane, my_key, my_at);
    write_slots(p, t, lane, my_key, static_cast<int>(at[my_at]), most, all);
}

using SelectFn = void (*)(SelectParams);

template <int DT>
SelectFn select_fn(int E)
{
    if (E <= 32)
        return select_kernel<DT, 1>;
    if (E <= 128)
        return select_kernel<DT, 4>;
    if (E <= 256)
        return select_kernel<DT, 8>;
    if (E <= 512)
        return select_kernel<DT, 16>;
    if (E <= 1024)
        return select_kernel<DT, 32>;
    return select_wide_kernel<DT>;
}

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" moe_status moe_select_experts(const void *logits, int64_t T, int32_t E, int64_t logits_stride,
                                         int32_t logits_dtype, int32_t top_k, int32_t scoring, int32_t renormalize,
                                         float scale, int32_t *topk_ids, void *router_weights, int32_t weight_dtype,
                                         moe_stream_t stream)
{
    if (T < 0 || E < 1 || top_k < 1 || top_k > E || logits_stride < E)
        return MOE_ERR_INVALID_ARG;
    if (logits_dtype < MOE_WEIGHTS_FP32 || logits_dtype > MOE_WEIGHTS_FP16 || weight_dtype < MOE_WEIGHTS_FP32 ||
        weight_dtype > MOE_WEIGHTS_FP16 || (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) ||
        !(scale > -INFINITY && scale < INFINITY))
        return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || top_k > MOE_MAX_TOP_K || T > (int64_t{1} << 31) / MOE_MAX_TOP_K)
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    const uintptr_t lmask = logits_dtype == MOE_WEIGHTS_FP32 ? 3u : 1u, wmask = weight_dtype == MOE_WEIGHTS_FP32 ? 3u : 1u;
    if (!logits || !topk_ids || !router_weights || (reinterpret_cast<uintptr_t>(logits) & lmask) ||
        (reinterpret_cast<uintptr_t>(topk_ids) & 3u) || (reinterpret_cast<uintptr_t>(router_weights) & wmask))
        return MOE_ERR_INVALID_ARG;
    const SelectFn fn = logits_dtype == MOE_WEIGHTS_FP32   ? select_fn<MOE_WEIGHTS_FP32>(E)
                        : logits_dtype == MOE_WEIGHTS_BF16 ? select_fn<MOE_WEIGHTS_BF16>(E)
                                                           : select_fn<MOE_WEIGHTS_FP16>(E);
    SelectParams p{logits, T, logits_stride, E, top_k, scoring == MOE_SCORE_SIGMOID, renormalize != 0, scale,
                   topk_ids, router_weights, weight_dtype};
    if (E > 1024)
        return PdlLaunch(static_cast<unsigned>(T), 256, 0, stream).run(fn, p);
    return PdlLaunch(static_cast<unsigned>((T + kWarps - 1) / kWarps), 32 * kWarps, 0, stream).run(fn, p);
}
