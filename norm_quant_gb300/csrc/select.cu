// select.cu -- expert selection: the top_k largest router logits of every
// token, in order, and their weights.
//
// One warp a token; lane l holds the logits of experts l, l + 32, ... in
// registers as order-preserving integers.  Each of the top_k rounds takes the
// largest value of the warp and the lowest expert index that has it, and closes
// that expert.  With up to 8 experts a lane, a lane first sorts its own, so that
// a round looks at one value a lane and the taking lane moves up by one; otherwise
// it looks through them in every round.  The work is a chain of top_k dependent
// rounds for a few hundred bytes a token: a large batch is bound by the
// instructions, a small one by the chain.
// A 16-bit logit and its expert's index make one word whose order is that of
// the selection, ties included: a round is one warp reduction.  A 32-bit logit
// takes a reduction for the value and, among equals, one for the index, and
// sorting it exchanges two words: it pays for large batches with 8 experts a lane
// only (T = 16384, E = 256, k = 8: 12.7 us against 14.9; T = 1: 3.5 against 3.0;
// T = 16384, E = 128, k = 4: 7.0 against 6.6).  16-bit logits: 7.6 us against 9.9,
// 1.5 against 1.6, 5.0 against 5.2.
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

__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -kLargest), kLargest); }
__device__ __forceinline__ float finite_value(uint32_t key) { return finite(key_value(key)); }

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

// Sorts descending with a network of 19 exchanges for 8 values, 5 for 4.
template <int VPT, class Exchange>
__device__ __forceinline__ void sort_network(Exchange x)
{
    if constexpr (VPT == 2) {
        x(0, 1);
    } else if constexpr (VPT == 4) {
        x(0, 1), x(2, 3), x(0, 2), x(1, 3), x(1, 2);
    } else if constexpr (VPT == 8) {
        x(0, 1), x(2, 3), x(4, 5), x(6, 7), x(0, 2), x(1, 3), x(4, 6), x(5, 7), x(1, 2), x(5, 6);
        x(0, 4), x(3, 7), x(1, 5), x(2, 6), x(1, 4), x(3, 6), x(2, 4), x(3, 5), x(3, 4);
    }
}

// As take(), by sorting each lane's keys first.
template <int VPT>
__device__ __forceinline__ void take_sorted(uint32_t (&key)[VPT], int k, int lane, uint32_t &my_key, uint32_t &my_at)
{
    uint32_t places = 0, at[VPT];  // places: of the sorted keys, 4 bits each
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        at[i] = i;
    const auto exchange = [&](int a, int b, bool swap) {
        const uint32_t ka = key[a], ia = at[a];
        key[a] = swap ? key[b] : ka;
        at[a] = swap ? at[b] : ia;
        key[b] = swap ? ka : key[b];
        at[b] = swap ? ia : at[b];
    };
    sort_network<VPT>([&](int a, int b) { exchange(a, b, key[b] > key[a]); });
    bool equal = false;
#pragma unroll
    for (int i = 0; i + 1 < VPT; ++i)
        equal |= key[i] == key[i + 1] && key[i];
    if (__any_sync(0xFFFFFFFFu, equal))  // the network does not keep equal keys in order
#pragma unroll 1
        for (int pass = 0; pass + 1 < VPT; ++pass)
#pragma unroll
            for (int i = 0; i + 1 < VPT; ++i)
                exchange(i, i + 1, key[i] == key[i + 1] && at[i] > at[i + 1]);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        places |= at[i] << (4 * i);
    my_key = my_at = 0;
    for (int j = 0; j < k; ++j) {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key[0]);
        if (top == 0)
            break;
        uint32_t e = lane + 32u * (places & 15u);
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, key[0] == top);
        if (who & (who - 1))
            e = __reduce_min_sync(0xFFFFFFFFu, key[0] == top ? e : 0xFFFFFFFFu);
        else
            e = __shfl_sync(0xFFFFFFFFu, e, __ffs(who) - 1);
        if (lane == j) {
            my_key = top;
            my_at = e;
        }
        if ((e & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
            for (int i = 0; i + 1 < VPT; ++i)
                key[i] = key[i + 1];
            key[VPT - 1] = 0;
            places >>= 4;
        }
    }
}

// A 16-bit logit's order key in the upper half, its expert's index, larger for
// lower ones, in the lower; 0 for a closed expert.
template <bool BF16>
__device__ __forceinline__ uint32_t order_word(uint32_t bits, uint32_t e)
{
    constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
    if (bits == 0x8000u)
        bits = 0;  // -0
    const uint32_t key = bits & 0x8000u ? bits ^ 0xFFFFu : bits | 0x8000u;
    // open: from next to -inf's key, which is kInf's complement, to +inf's, both included; NaNs lie
    // below (and wrap around) or above
    const bool open = key - (0x8000u - kInf) <= 2 * kInf;
    return open ? key << 16 | (0xFFFFu - e) : 0u;
}

template <bool BF16>
__device__ __forceinline__ float word_value(uint32_t word)
{
    const uint32_t key = word >> 16;
    return widen16<BF16>(static_cast<uint16_t>(key & 0x8000u ? key & 0x7FFFu : key ^ 0xFFFFu));
}

// Lane j gets the word of slot j, or 0.
template <int VPT>
__device__ __forceinline__ uint32_t take_words(uint32_t (&word)[VPT], int k, int lane)
{
    uint32_t mine = 0;
    if constexpr (VPT <= 8)
        sort_network<VPT>([&](int a, int b) {
            const uint32_t hi = max(word[a], word[b]);
            word[b] = min(word[a], word[b]);
            word[a] = hi;
        });
    for (int j = 0; j < k; ++j) {
        uint32_t head = word[0];
        if constexpr (VPT > 8)
#pragma unroll
            for (int i = 1; i < VPT; ++i)
                head = max(head, word[i]);
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, head);
        if (lane == j)
            mine = top;
        if constexpr (VPT > 8) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                word[i] = word[i] == top ? 0u : word[i];
        } else if (head == top) {  // lanes that are out of experts shift zeros
#pragma unroll
            for (int i = 0; i + 1 < VPT; ++i)
                word[i] = word[i + 1];
            word[VPT - 1] = 0;
        }
    }
    return mine;
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

// Lane j writes slot j of token t: expert my_id with logit `value`, if open.
// most: the largest logit, finite; all: the softmax's sum over every open
// expert, relative to it (unused otherwise).
__device__ __forceinline__ void write_slots(const SelectParams &p, int64_t t, int lane, bool open, float value, int my_id,
                                            float most, float all)
{
    float w = 0.0f;
    if (open && p.sigmoid) {
        // Below zero exp(l) / (1 + exp(l)), whose ratios hold over the whole range when renormalised: relative to
        // the largest (or to 0) the exponentials do not underflow before their ratio does.
        const float from = p.renorm ? fminf(most, 0.0f) : 0.0f;
        w = value > 0.0f ? 1.0f / (1.0f + expf(-value)) : expf(finite(value) - from) / (1.0f + expf(value));
    } else if (open) {
        w = expf(finite(value) - most);
    }
    const float taken = p.renorm ? warp_sum(w) : 0.0f;
    if (lane >= p.k)
        return;
    if (p.renorm || !p.sigmoid)
        w /= p.renorm ? taken : all;
    w = open ? w * p.scale : 0.0f;
    const int64_t o = t * p.k + lane;
    p.ids[o] = open ? my_id : -1;
    if (p.weight_dtype == MOE_WEIGHTS_FP32)
        static_cast<float *>(p.weights)[o] = w;
    else
        static_cast<uint16_t *>(p.weights)[o] =
            p.weight_dtype == MOE_WEIGHTS_BF16 ? narrow16<true>(w) : narrow16<false>(w);
}

// VPT: experts a lane holds, at least E / 32.  SORT: of 32-bit logits.
template <int DT, int VPT, bool SORT = false>
__global__ void __launch_bounds__(32 * kWarps) select_kernel(SelectParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    allow_dependent_launch();
    if (t >= p.T)
        return;
    const bool over_all = !p.sigmoid && !p.renorm;
    float all = 0.0f;
    if constexpr (DT == MOE_WEIGHTS_FP32) {
        uint32_t key[VPT], my_key, my_at;
        load_keys<DT>(p, t, 0, lane, key);
        if (over_all) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                best = max(best, key[i]);
            all = exp_sum(key, finite_value(__reduce_max_sync(0xFFFFFFFFu, best)));
        }
        if constexpr (SORT)
            take_sorted(key, p.k, lane, my_key, my_at);
        else
            take(key, p.k, lane, my_key, my_at);
        const float most = finite_value(__shfl_sync(0xFFFFFFFFu, my_key, 0));
        write_slots(p, t, lane, my_key != 0, key_value(my_key), static_cast<int>(my_at), most, all);
    } else {
        constexpr bool kBf16 = DT == MOE_WEIGHTS_BF16;
        const uint16_t *row = static_cast<const uint16_t *>(p.logits) + t * p.stride;
        uint32_t word[VPT], best = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = lane + 32 * i;
            word[i] = e < p.E ? order_word<kBf16>(row[e], e) : 0u;
        }
        if (over_all) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                best = max(best, word[i]);
            const float most = finite(word_value<kBf16>(__reduce_max_sync(0xFFFFFFFFu, best)));
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                all += word[i] ? expf(finite(word_value<kBf16>(word[i])) - most) : 0.0f;
            all = warp_sum(all);
        }
        const uint32_t mine = take_words(word, p.k, lane);
        const float value = word_value<kBf16>(mine), most = finite(__shfl_sync(0xFFFFFFFFu, value, 0));
        write_slots(p, t, lane, mine != 0, value, static_cast<int>(0xFFFFu - (mine & 0xFFFFu)), most, all);
    }
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
    write_slots(p, t, lane, my_key != 0, key_value(my_key), static_cast<int>(at[my_at]), most, all);
}

using SelectFn = void (*)(SelectParams);

template <int DT>
SelectFn select_fn(int E, int64_t T)
{
    if (E <= 32)
        return select_kernel<DT, 1>;
    if (E <= 64)
        return select_kernel<DT, 2>;
    if (E <= 128)
        return select_kernel<DT, 4>;
    if (E <= 256)
        return DT == MOE_WEIGHTS_FP32 && T >= 4096 ? select_kernel<DT, 8, DT == MOE_WEIGHTS_FP32> : select_kernel<DT, 8>;
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
    const SelectFn fn = logits_dtype == MOE_WEIGHTS_FP32   ? select_fn<MOE_WEIGHTS_FP32>(E, T)
                        : logits_dtype == MOE_WEIGHTS_BF16 ? select_fn<MOE_WEIGHTS_BF16>(E, T)
                                                           : select_fn<MOE_WEIGHTS_FP16>(E, T);
    SelectParams p{logits, T, logits_stride, E, top_k, scoring == MOE_SCORE_SIGMOID, renormalize != 0, scale,
                   topk_ids, router_weights, weight_dtype};
    if (E > 1024)
        return PdlLaunch(static_cast<unsigned>(T), 256, 0, stream).run(fn, p);
    return PdlLaunch(static_cast<unsigned>((T + kWarps - 1) / kWarps), 32 * kWarps, 0, stream).run(fn, p);
}
