// skinny.cuh -- products of a weight matrix with a few columns, the inner
// loop of the 4-bit linear and of the few-token expert layer.
//
//   D[n, c] = sum_k W[n, k] X[c, k],   c < 8 NT columns (tokens)
//
// One warp computes 16 rows of W by 8 NT columns over a range of k with
// mma.sync m16n8k16: W is the 16-row operand, the tokens are the 8-column one,
// and the sums stay in fp32.  The products are bound by the stream of W (a
// weight is used for a handful of tokens), so the weights go from global
// memory straight into the registers that the matrix instruction reads; no
// shared memory and no barrier stands in between.
//
// The order of k inside a step is free as long as both operands agree on it.
// A lane (g = lane / 4, t = lane % 4) therefore loads consecutive elements of
// the rows g and g + 8 with one wide load each, and the same elements of
// column g, and feeds them to the instruction's k slots in that order:
//   16-bit weights   8 elements a lane (16 bytes), a step of 32 k, 2 instructions
//   4-bit weights   16 elements a lane (8 bytes), a step of 64 k, 4 instructions
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace nqg {

enum WeightFormat { kW16 = 0, kWNvfp4 = 1, kWInt4 = 2 };

// One matrix of weights [rows, K] with its scales, as a kernel sees it.
struct WeightView {
    const uint8_t *w;       // rows of K elements (16-bit) or K / 2 bytes (4-bit)
    const uint8_t *scales;  // rows of K / group scales: e4m3 bytes (nvfp4) or 16-bit (int4)
    const uint8_t *zeros;   // rows of K / group zero points (int4), or nullptr: 8
    int32_t K;
    int32_t group_shift;    // log2(group) (int4)
};

// ------------------------------------------------------------ instructions

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Loads of weights: read once, so they do not displace the tokens in L1.
__device__ __forceinline__ uint4 ldg_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 ldg_stream8(const void *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Loads of columns: written by the kernel before, so they take the coherent path.
__device__ __forceinline__ uint4 load_column(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

template <bool BF16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (BF16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t v)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(v));
    return f;
}

template <bool BF16>
__device__ __forceinline__ uint16_t narrow16(float f)
{
    uint16_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    else
        asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
}

// An e4m3 byte's value in fp16 (exact: 4 significant bits, exponents -9 to 8).
__device__ __forceinline__ uint16_t e4m3_to_f16(uint32_t code)
{
    uint32_t r;
    const uint16_t c = static_cast<uint16_t>(code);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return static_cast<uint16_t>(r);
}

// ---------------------------------------------------------- weight formats
//
// A format loads one lane's slice of a row and turns it into the row's
// operand registers, pairs[2 m] and pairs[2 m + 1] for instruction m, after
// which scale_after (int4) multiplies the instruction's sums.

template <int FMT, bool BF16>
struct Format;

template <bool BF16>
struct Format<kW16, BF16> {
    static constexpr int kLane = 8;       // elements of a row that a lane holds in a step
    static constexpr int kMma = 2;        // instructions in a step
    static constexpr bool kSplit = false; // pairs are elements (j, j + 4) of 8, not (2 j, 2 j + 1)
    static constexpr bool kAfter = false;
    static constexpr float kPost = 1.0f;  // the sums are to be multiplied by this
    struct Slice {
        uint4 v;
    };
    struct Row {
        const uint8_t *w;
    };
    __device__ static Row row(const WeightView &W, int64_t r)
    {
        return {W.w + r * W.K * 2};
    }
    __device__ static void load(Slice &s, const WeightView &, const Row &row, int k)
    {
        s.v = ldg_stream16(row.w + static_cast<int64_t>(k) * 2);
    }
    __device__ static void none(Slice &s) { s.v = make_uint4(0, 0, 0, 0); }
    __device__ static void pairs(const Slice &s, uint32_t (&p)[4])
    {
        p[0] = s.v.x;
        p[1] = s.v.y;
        p[2] = s.v.z;
        p[3] = s.v.w;
    }
};

// NVFP4: a weight is e2m1 x e4m3.  The product has at most 2 + 4 significant
// bits, so it is exact in bf16 and fp16 and the scale is multiplied into the
// operand: one instruction for two weights.
template <bool BF16>
struct Format<kWNvfp4, BF16> {
    static constexpr int kLane = 16;
    static constexpr int kMma = 4;
    static constexpr bool kSplit = BF16;
    static constexpr bool kAfter = false;
    // bf16: an e2m1 code's bits s, eem moved to bits 15 and 8..6 are the bf16
    // number value x 2^-126 (the subnormals included); the scale carries 2^100
    // of it back, which keeps it finite, and the sums the other 2^26.
    static constexpr float kPost = BF16 ? 0x1p26f : 1.0f;
    struct Slice {
        uint2 v;
        uint32_t scale;
    };
    struct Row {
        const uint8_t *w, *s;
    };
    __device__ static Row row(const WeightView &W, int64_t r)
    {
        return {W.w + r * (W.K / 2), W.scales + r * (W.K / 16)};
    }
    __device__ static void load(Slice &s, const WeightView &, const Row &row, int k)
    {
        s.v = ldg_stream8(row.w + (k >> 1));
        s.scale = __ldg(row.s + (k >> 4));
    }
    __device__ static void none(Slice &s)
    {
        s.v = make_uint2(0, 0);
        s.scale = 0;
    }
    __device__ static void eight(uint32_t w, uint32_t scale, uint32_t *p)
    {
        if constexpr (BF16) {
            constexpr uint32_t kSign = 0x80008000u, kMag = 0x01C001C0u;
            p[0] = mul2<true>(((w << 12) & kSign) | ((w << 6) & kMag), scale);
            p[1] = mul2<true>(((w << 8) & kSign) | ((w << 2) & kMag), scale);
            p[2] = mul2<true>(((w << 4) & kSign) | ((w >> 2) & kMag), scale);
            p[3] = mul2<true>((w & kSign) | ((w >> 6) & kMag), scale);
        } else {
            uint32_t h[4];
            asm("{ .reg .b8 b0, b1, b2, b3;\n"
                "  mov.b32 {b0, b1, b2, b3}, %4;\n"
                "  cvt.rn.f16x2.e2m1x2 %0, b0;\n"
                "  cvt.rn.f16x2.e2m1x2 %1, b1;\n"
                "  cvt.rn.f16x2.e2m1x2 %2, b2;\n"
                "  cvt.rn.f16x2.e2m1x2 %3, b3; }"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                : "r"(w));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = mul2<false>(h[j], scale);
        }
    }
    __device__ static void pairs(const Slice &s, uint32_t (&p)[8])
    {
        uint32_t scale = e4m3_to_f16(s.scale);
        if constexpr (BF16)
            scale = narrow16<true>(widen16<false>(static_cast<uint16_t>(scale)) * 0x1p100f);
        scale |= scale << 16;
        eight(s.v.x, scale, p);
        eight(s.v.y, scale, p + 4);
    }
};

// 4-bit integers: (code - zero) has at most 5 bits and is exact in bf16 and
// fp16.  Times a 16-bit scale it would not be, so the scale multiplies the
// fp32 sums of a step, all of whose k lie in one group (group % 64 == 0).
// A nibble or-ed into the mantissa of 128 (bf16) or 1024 (fp16) is that
// number plus the code.
template <bool BF16>
struct Format<kWInt4, BF16> {
    static constexpr int kLane = 16;
    static constexpr int kMma = 4;
    static constexpr bool kSplit = true;
    static constexpr bool kAfter = true;
    static constexpr float kPost = 1.0f;
    static constexpr uint32_t kMagic = BF16 ? 0x43004300u : 0x64006400u;
    struct Slice {
        uint2 v;
        uint32_t zero;
        uint16_t scale;
    };
    struct Row {
        const uint8_t *w, *s, *z;
    };
    __device__ static Row row(const WeightView &W, int64_t r)
    {
        const int64_t groups = W.K >> W.group_shift;
        return {W.w + r * (W.K / 2), W.scales + r * groups * 2, W.zeros ? W.zeros + r * groups : nullptr};
    }
    __device__ static void load(Slice &s, const WeightView &W, const Row &row, int k)
    {
        s.v = ldg_stream8(row.w + (k >> 1));
        const int grp = k >> W.group_shift;
        s.scale = __ldg(reinterpret_cast<const uint16_t *>(row.s) + grp);
        s.zero = row.z ? __ldg(row.z + grp) : 8u;
    }
    __device__ static void none(Slice &s)
    {
        s.v = make_uint2(0, 0);
        s.zero = 0;
        s.scale = 0;
    }
    __device__ static void pairs(const Slice &s, uint32_t (&p)[8])
    {
        const uint32_t zero = kMagic | (s.zero & 15u) * 0x00010001u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = sub2<BF16>(((s.v.x >> (4 * j)) & 0x000F000Fu) | kMagic, zero);
            p[4 + j] = sub2<BF16>(((s.v.y >> (4 * j)) & 0x000F000Fu) | kMagic, zero);
        }
    }
    __device__ static float scale_after(const Slice &s) { return widen16<BF16>(s.scale); }
};

// ------------------------------------------------------------- the product

// A lane's slice of a column: kLane consecutive 16-bit elements.
template <int N>
struct ColumnSlice {
    uint4 v[N / 8];
};

template <class F>
__device__ __forceinline__ void column_pairs(const ColumnSlice<F::kLane> &c, uint32_t (&b)[F::kLane / 2])
{
#pragma unroll
    for (int h = 0; h < F::kLane / 8; ++h) {
        const uint4 v = c.v[h];
        if constexpr (F::kSplit) {
            b[4 * h + 0] = __byte_perm(v.x, v.z, 0x5410);
            b[4 * h + 1] = __byte_perm(v.x, v.z, 0x7632);
            b[4 * h + 2] = __byte_perm(v.y, v.w, 0x5410);
            b[4 * h + 3] = __byte_perm(v.y, v.w, 0x7632);
        } else {
            b[4 * h + 0] = v.x;
            b[4 * h + 1] = v.y;
            b[4 * h + 2] = v.z;
            b[4 * h + 3] = v.w;
        }
    }
}

// acc[nt] += W[rows of this lane, k0..k1) x columns, for the tiles of columns
// nt < tiles (the same for every lane).  `lo` and `hi` are rows g and g + 8,
// col[nt] the lane's column g of tile nt; a row or column past the end points
// at any valid one and its sums are ignored.  k0 is a multiple of the step and
// k1 of a lane's slice; past k1 the slices are zero.
template <class F, bool BF16, int NT, int U>
__device__ __forceinline__ void skinny_product(float (&acc)[NT][4], const WeightView &W, const typename F::Row &lo,
                                               const typename F::Row &hi, const uint16_t *const (&col)[NT], int tiles,
                                               int k0, int k1, int lane)
{
    constexpr int kStep = 4 * F::kLane;
    const int own = (lane & 3) * F::kLane;
    for (int k = k0 + own; k < k1 + own; k += U * kStep) {
        typename F::Slice a[U][2];
        ColumnSlice<F::kLane> b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ku = k + u * kStep;
            if (ku < k1) {
                F::load(a[u][0], W, lo, ku);
                F::load(a[u][1], W, hi, ku);
            } else {
                F::none(a[u][0]);
                F::none(a[u][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < F::kLane / 8; ++i)
                    b[u][nt].v[i] = nt < tiles && ku < k1 ? load_column(col[nt] + ku + 8 * i)
                                                          : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t p[2][F::kLane / 2];
            F::pairs(a[u][0], p[0]);
            F::pairs(a[u][1], p[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt >= tiles)
                    continue;
                uint32_t q[F::kLane / 2];
                column_pairs<F>(b[u][nt], q);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                float(&d)[4] = F::kAfter ? part : acc[nt];
#pragma unroll
                for (int m = 0; m < F::kMma; ++m) {
                    const uint32_t frag[4] = {p[0][2 * m], p[1][2 * m], p[0][2 * m + 1], p[1][2 * m + 1]};
                    mma16816<BF16>(d, frag, q[2 * m], q[2 * m + 1]);
                }
                if constexpr (F::kAfter) {
                    const float slo = F::scale_after(a[u][0]), shi = F::scale_after(a[u][1]);
                    acc[nt][0] = fmaf(slo, part[0], acc[nt][0]);
                    acc[nt][1] = fmaf(slo, part[1], acc[nt][1]);
                    acc[nt][2] = fmaf(shi, part[2], acc[nt][2]);
                    acc[nt][3] = fmaf(shi, part[3], acc[nt][3]);
                }
            }
        }
    }
}

// A product's sum times kPost and divided by the global scale g.  For g >= 1
// the quotient is taken first: a sum near the largest float may not survive
// kPost alone.  For g < 1 that would mean that the result overflows too.
template <class F>
__device__ __forceinline__ float descale(float sum, float g)
{
    return g >= 1.0f ? sum * (F::kPost / g) : sum * F::kPost / g;
}

} // namespace nqg
