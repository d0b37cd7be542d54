// block_math.cuh -- element arithmetic of the feed-forward block: 16-bit
// vectors to fp32 and back, and the activations with their derivatives.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_layer.h"
#include "ptx.cuh"

namespace nqg {

__device__ __forceinline__ uint4 ldg16(const void *p) { return __ldg(static_cast<const uint4 *>(p)); }

template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi)
{
    if constexpr (BF16)
        bf16x2_to_f32(w, lo, hi);
    else
        f16x2_to_f32(w, lo, hi);
}

// Two fp32 to the 16-bit type, round to nearest even; a result beyond fp16's range is an infinity.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return BF16 ? f32x2_to_bf16x2(lo, hi) : f32x2_to_f16x2(lo, hi);
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    unpack2<BF16>(w.x, v[0], v[1]);
    unpack2<BF16>(w.y, v[2], v[3]);
    unpack2<BF16>(w.z, v[4], v[5]);
    unpack2<BF16>(w.w, v[6], v[7]);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
}

// p = 1 / (1 + exp(-z)).  exp overflows to infinity below z = -88, where p is 0.  The intrinsics' errors (2 ulp of
// the quotient, |z| 2^-24 + 2 ulp of the exponential) are far below the rounding to 16 bits that follows.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kSqrt8OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act(g) and act'(g).  gelu: 0.5 g (1 + tanh(z)) = g p(2 z), which does not cancel for negative g;
// z = sqrt(2 / pi) (g + 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ float act(float g)
{
    if constexpr (ACT == MOE_ACT_SILU)
        return g * sigmoid(g);
    return g * sigmoid(kSqrt8OverPi * (g + 0.044715f * g * g * g));
}

template <int ACT>
__device__ __forceinline__ void act_and_slope(float g, float &a, float &slope)
{
    if constexpr (ACT == MOE_ACT_SILU) {
        const float p = sigmoid(g);
        a = g * p;
        slope = p + a * (1.0f - p);
    } else {
        const float p = sigmoid(kSqrt8OverPi * (g + 0.044715f * g * g * g));
        // beyond |g| = 100 the factor in front of the square is 0, and an infinite square would make it NaN
        const float m = fminf(fabsf(g), 100.0f);
        a = g * p;
        slope = p + a * (1.0f - p) * kSqrt8OverPi * (1.0f + 0.134145f * m * m);
    }
}

} // namespace nqg
