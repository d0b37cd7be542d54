// skinny.cuh -- products of a weight matrix with a few columns, the inner
// loop of the 4-bit linear and of the few-token expert layer.
//
//   D[n, c] = sum_k W[n, k] X[c, k],   c < 8 columns (tokens), or up to 64 of the linear's
//
// One warp computes 16 rows of W by 8 columns, or by up to 8 times 8 with an
// operand of W, over a range of k with mma.sync m16n8k16: W is the 16-row operand, the tokens are the 8-column one,
// and the sums stay in fp32.  The products are bound by the stream of W (a
// weight is used for a handful of tokens), so what counts is the bytes that
// are in flight and the instructions spent on each weight.
//
// In flight: a CTA has a ring of slots in shared memory.  A slot holds one
// panel, 128 bytes of each of 16 rows for every warp of a group or two, and a
// producer warp fills slots with tensor copies (TMA), as far ahead as the ring goes,
// across the ends of row blocks.  The warps of a group share out the k of a
// panel; several groups take different row blocks, so that enough warps are
// there to hide each other's latencies.  (Tensor copies of 8 rows x 128 bytes x
// strips reach 6.3 TB/s whatever the panel's width; a bulk copy for each row
// costs about 80 cycles, 3.7 TB/s with rows of 1 KB.)
//
// Instructions: the columns are laid out in the order in which the matrix
// instruction takes them, once for many rows (those that are streamed with the
// weights are permuted for each use, or spared that by widening neighbours).
// Integers are widened to the type of the columns with one and-or, one subtraction
// or fma, and a quarter (fp16) to three quarters (bf16) of a shift for two;
// neighbours with a permutation and, in bf16, a quarter of a shift.  e2m1 codes take
// one conversion for two of them to fp16, and three operations and a quarter to
// bf16 (neighbours one more), and both one multiplication by the scale.  For bf16 columns that are used for many rows, the columns
// are therefore held as fp16 times a power of two, chosen for each column and
// each strip of k (256 elements) so that the largest magnitude lies in
// [2^14, 2^15): every element down to 2^-29 of the largest keeps all its bits,
// and a smaller one is off by at most 2^-39 of the largest (half of fp16's last
// place, 2^-25, against 2^14), far below the rounding of the fp32 sum that it goes
// into.  For a strip whose largest is below about 2^-111 max(g, 1), with g the
// global scale, the power is smaller, so that the factor 2^-e / g stays a normal
// float; an element is then off by up to 2^-150 max(g, 1).
#pragma once

#include <cstdint>
#include <cuda.h>  // CUtensorMap only; no libcuda symbol is linked
#include <cuda_runtime.h>

#include "common.h"
#include "few_token.h"
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

// d = a b + (FIRST ? 0 : d)
template <bool BF16, bool FIRST = false>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (FIRST) {
        if constexpr (BF16)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        return;
    }
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A constant that the compiler does not see.
__device__ __forceinline__ uint32_t opaque(uint32_t v)
{
    uint32_t r;
    asm("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "n"(MASK), "r"(c));
    return r;
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

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
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

// ---------------------------------------------------------- weight formats
//
// A strip is 128 bytes of each of 16 rows, what one warp takes of a panel; it
// goes through it in kSteps steps of kMma instructions.  The order of k inside
// a strip is free as long as both operands agree on it: in step u, lane
// (g = lane / 4, t = lane % 4) takes kLane consecutive elements of the rows g
// and g + 8 and of column g, from element 16 t + 8 u of the strip on with
// 16-bit weights, 64 t + 16 u with NVFP4, and 64 u + 16 t with integers and STEPS.
//
// Rows of a strip lie 128 bytes apart with their 16-byte chunks exchanged as
// the 128-byte swizzle of the tensor copies does it: chunk i of row g is at
// position i ^ g.  A lane's slices are chosen so that 8 lanes of two rows meet
// all banks (16 lanes of 4 rows meet half of them with int4's 8-byte slices).
//
//   Slice    one lane's bytes of a row for all steps of the strip
//   Scales   what it needs of the row's scales
//   operand  p[2 i], p[2 i + 1]: the row's operand registers of instruction i

constexpr int kStripBytes = 128;

// Consumer warps of a CTA: with the producer's 24, for 80 registers a thread, or
// 17 with integers, whose steps would spill.
template <int FMT>
constexpr int kMaxConsumers = FMT == kWInt4 ? 16 : 23;

constexpr int kColumns = 8;

// NATIVE: operands of the columns' type; otherwise nvfp4's are fp16.  STEPS:
// for columns that are read as they lie in memory.  nvfp4's lanes take 64
// elements a step between them, as int4's do; and what widens two codes at a time
// takes neighbours (kPairs), or codes 16 bits apart (kApart), which leaves it to the
// columns to be paired the same way.  Neighbours take 2 to 4 operations more for 8 codes, and spare
// each 8 columns 8 permutations for 32 codes.
enum : int { kLaidOut, kApart, kPairs };

template <int FMT, bool BF16, bool NATIVE = false, int STEPS = kLaidOut>
struct Format;

__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

__device__ __forceinline__ uint32_t lds4(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

__device__ __forceinline__ uint16_t lds2(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}

__device__ __forceinline__ uint32_t lds1(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

// Where a slot's scales lie, from the start of the slot, and how.
struct ScalePlace {
    uint32_t at, pitch;            // scales of a row
    uint32_t zero_at, zero_pitch;  // zero points, pitch 0: none
    int32_t down, zero_down;       // int4: a row's scales start at a group that is a multiple of down + 1
};

// How the slots of a ring are laid out.  A slot: for every strip of the panel
// 128 bytes of each row, in blocks of `block` consecutive rows of the matrix;
// then the scales of all rows; and then columns, if any.  Either the slot's
// 16-row tiles are one block, or there are two blocks of 8 rows for one tile.
struct SlotPlan {
    int32_t warps;      // of a group for each tile
    int32_t strips;     // of a panel: warp j takes strips j, j + warps, ...
    int32_t tiles;      // of 16 rows in a slot
    int32_t block;      // rows: 16 tiles, or 8
    int32_t strip;      // bytes from strip to strip of a block
    int32_t half;       // bytes from rows 0 to 7 of a tile to rows 8 to 15
    ScalePlace scale;   // from the start of a slot
    int32_t columns_at;
    int32_t bytes;      // of a slot, a multiple of 1024
    int32_t depth;      // slots of a group's ring
};

template <bool BF16, bool NATIVE>
struct Format<kW16, BF16, NATIVE, kLaidOut> {
    static constexpr float kPost = 1.0f;  // the sums are to be multiplied by this
    static constexpr bool kHalf = !BF16;  // the operands are fp16
    static constexpr int kStripK = 64, kSteps = 2, kLane = 8, kMma = 2;
    static constexpr bool kSplit = false;  // columns: pairs are elements (j, j + 4) of 8, not (2 j, 2 j + 1)
    static constexpr bool kAfter = false;  // scales multiply the sums of a step, not the operands
    struct Scales {};
    struct Slice {
        uint4 v[2];
    };
    __host__ __device__ static int row_bytes(int K) { return K * 2; }
    __device__ static uint32_t scale_at(const ScalePlace &, int, int) { return 0; }
    __device__ static void load_scales(Scales (&)[2], uint32_t, const SlotPlan &, const WeightView &, int, int, int) {}
    __device__ static void load(Slice &s, uint32_t tile)  // tile: of the lane's row, at lane_at()
    {
        s.v[0] = lds16(tile);
        s.v[1] = lds16(tile ^ 16);
    }
    __device__ static uint32_t lane_at(int g, int t) { return g * kStripBytes + ((2 * t) ^ g) * 16; }
    // Clears the elements from `left` of the strip on.
    __device__ static void clear(Slice &s, Scales &, int left, int t)
    {
        if (16 * t >= left)
            s.v[0] = make_uint4(0, 0, 0, 0);
        if (16 * t + 8 >= left)
            s.v[1] = make_uint4(0, 0, 0, 0);
    }
    __device__ static void operand(const Slice &s, const Scales &, int u, uint32_t (&p)[4])
    {
        p[0] = s.v[u].x;
        p[1] = s.v[u].y;
        p[2] = s.v[u].z;
        p[3] = s.v[u].w;
    }
};

// NVFP4: a weight is e2m1 x e4m3.  The product has at most 2 + 4 significant
// bits and lies between 2^-10 and 2688, so it is exact in fp16 and the scale is
// multiplied into the operand: one instruction for two weights.  Lane t takes
// the elements 64 t to 64 t + 63 of a strip, so that the four scales that it
// needs of a row are one word.
template <bool BF16, bool NATIVE>
struct Format<kWNvfp4, BF16, NATIVE, kLaidOut> {
    static constexpr bool kHalf = !(BF16 && NATIVE);
    // bf16: a code's bits s, eem moved to bits 15 and 8..6 are the bf16 number
    // value x 2^-126 (the subnormals included); the scale carries 2^100 of it
    // back, which keeps it finite, and the sums the other 2^26.
    static constexpr float kPost = kHalf ? 1.0f : 0x1p26f;
    static constexpr int kStripK = 256, kSteps = 4, kLane = 16, kMma = 4;
    static constexpr bool kSplit = !kHalf;
    static constexpr bool kAfter = false;
    struct Scales {
        uint32_t codes;
    };
    struct Slice {
        uint4 v[2];
    };
    __host__ __device__ static int row_bytes(int K) { return K / 2; }
    // Of row r of the slot, from its start on; row r + 8 lies 8 rows further.
    __device__ static uint32_t scale_at(const ScalePlace &pl, int r, int t) { return pl.at + r * pl.pitch + 4 * t; }
    __device__ static void load_scales(Scales (&s)[2], uint32_t at, const SlotPlan &plan, const WeightView &, int, int i, int)
    {
        s[0].codes = lds4(at + 16 * i);
        s[1].codes = lds4(at + 16 * i + 8 * plan.scale.pitch);
    }
    __device__ static void load(Slice &s, uint32_t tile)  // tile: of the lane's row, at lane_at()
    {
        s.v[0] = lds16(tile);
        s.v[1] = lds16(tile ^ 16);
    }
    __device__ static uint32_t lane_at(int g, int t) { return g * kStripBytes + ((2 * t) ^ g) * 16; }
    __device__ static void clear(Slice &s, Scales &sc, int left, int t)
    {
        const int groups = min(max((left - 64 * t) / 16, 0), 4);  // of this lane's four
        sc.codes &= groups == 4 ? 0xFFFFFFFFu : (1u << (8 * groups)) - 1;
        if (groups < 1)
            s.v[0].x = s.v[0].y = 0;
        if (groups < 2)
            s.v[0].z = s.v[0].w = 0;
        if (groups < 3)
            s.v[1].x = s.v[1].y = 0;
        if (groups < 4)
            s.v[1].z = s.v[1].w = 0;
    }
    // The factor of the operands, from the scale twice in fp16.
    __device__ static uint32_t operand_scale(uint32_t twice)
    {
        if constexpr (kHalf)
            return twice;
        const float f = widen16<false>(static_cast<uint16_t>(twice)) * 0x1p100f;
        return f32x2_to_bf16x2(f, f);
    }
    template <bool PAIRS = false>
    __device__ static void eight(uint32_t w, uint32_t scale, uint32_t *p)
    {
        uint32_t h[4];
        if constexpr (kHalf) {
            asm("{ .reg .b8 b0, b1, b2, b3;\n"
                "  mov.b32 {b0, b1, b2, b3}, %4;\n"
                "  cvt.rn.f16x2.e2m1x2 %0, b0;\n"
                "  cvt.rn.f16x2.e2m1x2 %1, b1;\n"
                "  cvt.rn.f16x2.e2m1x2 %2, b2;\n"
                "  cvt.rn.f16x2.e2m1x2 %3, b3; }"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                : "r"(w));
        } else if constexpr (PAIRS) {
            const uint32_t v = w >> 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = ((__byte_perm(w, v, 0x0400 + 0x0101 * j) & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
        } else {  // the sum of two shifted copies is one multiplication, on the other pipe
            const uint32_t v = w >> 8;
            h[0] = ((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            h[1] = ((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
            h[2] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            h[3] = ((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[j] = mul2<!kHalf>(h[j], scale);
    }
    __device__ static void operand(const Slice &s, const Scales &sc, int u, uint32_t (&p)[8])
    {
        uint32_t two;  // the scales of steps 2 (u / 2) and the next
        const uint16_t c = static_cast<uint16_t>(sc.codes >> (16 * (u >> 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(c));
        const uint32_t scale = operand_scale(__byte_perm(two, two, u & 1 ? 0x3232 : 0x1010));
        eight(u & 1 ? s.v[u >> 1].z : s.v[u >> 1].x, scale, p);
        eight(u & 1 ? s.v[u >> 1].w : s.v[u >> 1].y, scale, p + 4);
    }
};

template <bool BF16, int STEPS>
struct Nvfp4Steps : Format<kWNvfp4, BF16, true, kLaidOut> {
    using Base = Format<kWNvfp4, BF16, true, kLaidOut>;
    static constexpr bool kSplit = Base::kSplit && STEPS == kApart;
    struct Scales {
        uint32_t codes[4];  // of the four groups of each step; lane t's is byte t
    };
    struct Slice {  // read step by step
        uint32_t at;
    };
    __device__ static uint32_t scale_at(const ScalePlace &pl, int r, int) { return pl.at + r * pl.pitch; }
    __device__ static void load_scales(Scales (&s)[2], uint32_t at, const SlotPlan &plan, const WeightView &, int, int i, int)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 v = lds16(at + 16 * i + 8 * h * plan.scale.pitch);
            s[h].codes[0] = v.x;
            s[h].codes[1] = v.y;
            s[h].codes[2] = v.z;
            s[h].codes[3] = v.w;
        }
    }
    __device__ static void load(Slice &s, uint32_t tile) { s.at = tile; }
    __device__ static uint32_t lane_at(int g, int t) { return g * kStripBytes + ((t >> 1) ^ g) * 16 + (t & 1) * 8; }
    // Past the end the columns are zero, and codes are finite whatever they are.
    __device__ static void clear(Slice &, Scales &sc, int left, int t)
    {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (64 * u + 16 * t >= left)
                sc.codes[u] = 0;
    }
    __device__ static void operand(const Slice &s, const Scales &sc, int u, uint32_t (&p)[8])
    {
        uint32_t two;
        const uint32_t word = u & 2 ? (u & 1 ? sc.codes[3] : sc.codes[2]) : (u & 1 ? sc.codes[1] : sc.codes[0]);
        const uint16_t c = static_cast<uint16_t>((word >> (8 * (threadIdx.x & 3))) & 0xFFu);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(c));
        const uint32_t scale = Base::operand_scale(__byte_perm(two, two, 0x1010));
        const uint2 w = lds8(s.at ^ (32 * u));
        Base::template eight<STEPS == kPairs>(w.x, scale, p);
        Base::template eight<STEPS == kPairs>(w.y, scale, p + 4);
    }
};

template <bool BF16>
struct Format<kWNvfp4, BF16, true, kApart> : Nvfp4Steps<BF16, kApart> {};
template <bool BF16>
struct Format<kWNvfp4, BF16, true, kPairs> : Nvfp4Steps<BF16, kPairs> {};

// 4-bit integers: code - zero has at most 5 bits and is exact in bf16 and fp16.
// Times a 16-bit scale it would not be, so the scale multiplies the fp32 sums of
// a step, all of whose k lie in one group (group % 64 == 0): lane t takes the
// elements 16 t to 16 t + 15 of the step's 64.
// A code in bits 3..0 of the mantissa of 128 (bf16) or 1024 (fp16) makes that
// number plus the code, and in fp16 one in bits 7..4 makes 1024 + 16 code; either
// less the zero point is one exact instruction.
template <bool BF16, bool NATIVE, int STEPS>
struct Format<kWInt4, BF16, NATIVE, STEPS> {
    static constexpr bool kHalf = !BF16;
    static constexpr float kPost = 1.0f;
    static constexpr int kStripK = 256, kSteps = 4, kLane = 16, kMma = 4;
    static constexpr bool kSplit = STEPS != kPairs;
    static constexpr bool kAfter = true;
    struct Scales {
        uint32_t scale[2];  // two steps' in a word
        uint32_t zero;      // a byte for each step
    };
    struct Slice {  // read step by step
        uint32_t at;
    };
    __host__ __device__ static int row_bytes(int K) { return K / 2; }
    // the row alone: scales and zero points have pitches of their own
    __device__ static uint32_t scale_at(const ScalePlace &, int r, int) { return r; }
    // strip: of the row, i of the panel; from: the panel's first element.  A strip starts with a
    // group, or inside one of 512 and more.  What is read for steps past the end
    // is cleared later.
    __device__ static void load_scales(Scales (&s)[2], uint32_t at, const SlotPlan &plan, const WeightView &W, int strip, int, int from)
    {
        const int shift = W.group_shift, group = (strip * kStripK) >> shift;
        const int first = group - ((from >> shift) & ~plan.scale.down), zero = group - ((from >> shift) & ~plan.scale.zero_down);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = (at & 127) + 8 * h;  // slots are 1024-byte aligned
            const uint32_t a = (at & ~127u) + plan.scale.at + 2 * first + r * plan.scale.pitch;
            const uint32_t z = (at & ~127u) + plan.scale.zero_at + zero + r * plan.scale.zero_pitch;
            s[h].zero = 0x08080808u;
            if (shift == 6) {  // four groups
                const uint2 v = lds8(a);
                s[h].scale[0] = v.x;
                s[h].scale[1] = v.y;
                if (plan.scale.zero_pitch)
                    s[h].zero = lds4(z);
            } else if (shift == 7) {
                const uint32_t v = lds4(a);
                s[h].scale[0] = __byte_perm(v, v, 0x1010);
                s[h].scale[1] = __byte_perm(v, v, 0x3232);
                if (plan.scale.zero_pitch)
                    s[h].zero = __byte_perm(lds2(z), 0, 0x1100);
            } else {
                const uint32_t v = lds2(a);
                s[h].scale[0] = s[h].scale[1] = __byte_perm(v, v, 0x1010);
                if (plan.scale.zero_pitch)
                    s[h].zero = __byte_perm(lds1(z), 0, 0x0000);
            }
            s[h].zero &= 0x0F0F0F0Fu;
        }
    }
    __device__ static void load(Slice &s, uint32_t tile) { s.at = tile; }
    __device__ static uint32_t lane_at(int g, int t) { return g * kStripBytes + ((t >> 1) ^ g) * 16 + (t & 1) * 8; }
    // Past the end the columns are zero, and codes are finite whatever they are.
    __device__ static void clear(Slice &, Scales &sc, int left, int)
    {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (64 * u >= left)
                sc.scale[u >> 1] &= u & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
    __device__ static void operand(const Slice &s, const Scales &sc, int u, uint32_t (&p)[8])
    {
        if constexpr (!kSplit) {
            pairs(s, sc, u, p);
            return;
        }
        // in a register, so that and and or are one instruction
        const uint32_t base = opaque(BF16 ? 0x43004300u : 0x64006400u);
        const uint32_t less = __byte_perm(sc.zero, 0, 0x4040 + 0x0101 * u) | base;  // 128 or 1024, + zero
        const uint2 w8 = lds8(s.at ^ (32 * u));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? w8.y : w8.x;
            if constexpr (BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[4 * h + i] = sub2<true>(and_or<0x000F000Fu>(w >> (4 * i), base), less);
            } else {
                constexpr uint32_t kSixteenth = 0x2C002C00u;
                const uint32_t less16 = sub2<false>(0x63806380u, less);  // 960 - 1024 - zero
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t v = b ? w >> 8 : w;
                    p[4 * h + 2 * b] = sub2<false>(and_or<0x000F000Fu>(v, base), less);
                    p[4 * h + 2 * b + 1] = fma_f16x2(and_or<0x00F000F0u>(v, base), kSixteenth, less16);
                }
            }
        }
    }
    // Of a byte's two codes the lower one is taken as above.  The upper one is in
    // fp16 bits 7..4 as above, and in bf16, moved down by one, bits 6..3 of the
    // mantissa of 16, which makes 16 plus the code.
    __device__ static void pairs(const Slice &s, const Scales &sc, int u, uint32_t (&p)[8])
    {
        const uint32_t base = opaque(BF16 ? 0x41804300u : 0x64006400u);
        const uint32_t zero = __byte_perm(sc.zero, 0, 0x4040 + 0x0101 * u);
        // bf16: 128 + zero and 16 + zero; fp16: -1024 - zero and -64 - zero
        const uint32_t less = BF16 ? (zero & 0x0000FFFFu | (zero & 0xFFFF0000u) << 3) + 0x41804300u
                                   : (zero & 0x0000FFFFu | (zero & 0xFFFF0000u) << 4) + 0xD400E400u;
        const uint2 w8 = lds8(s.at ^ (32 * u));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? w8.y : w8.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16)
                    p[4 * h + i] = sub2<true>(and_or<0x0078000Fu>(__byte_perm(w, w >> 1, 0x0400 + 0x0101 * i), base), less);
                else
                    p[4 * h + i] = fma_f16x2(and_or<0x00F0000Fu>(__byte_perm(w, w, 0x0400 + 0x0101 * i), base), 0x2C003C00u, less);
            }
        }
    }
    __device__ static float scale_after(const Scales &s, int u) { return widen16<BF16>(static_cast<uint16_t>((u & 2 ? s.scale[1] : s.scale[0]) >> (16 * (u & 1)))); }
};

template <class F>
__host__ __device__ inline int strips_of(int K)
{
    return (K + F::kStripK - 1) / F::kStripK;
}

// sums = (FRESH) or += 16 rows of a strip x n columns.  tile: the lane's
// row g of the strip, at lane_at(); row g + 8 lies `half` bytes further.
// column: the lane's, at column_at(); scales: of the two rows; left: elements of
// the strip that the matrix has.  A row or column past the end is any valid one
// or zero, and its sums are ignored.
template <class F, bool BF16, bool FRESH>
__device__ __forceinline__ void strip_product(float (&sums)[4], uint32_t tile, uint32_t half, uint32_t column, uint32_t swap,
                                              typename F::Scales (&sc)[2], int left, int t)
{
    typename F::Slice a, b;
    F::load(a, tile);
    F::load(b, tile + half);
    if (left < F::kStripK) {
        F::clear(a, sc[0], left, t);
        F::clear(b, sc[1], left, t);
    }
    const uint32_t even = column + swap, odd = column - swap;
#pragma unroll
    for (int u = 0; u < F::kSteps; ++u) {
        uint32_t p[F::kLane / 2], q[F::kLane / 2], c[F::kLane / 2];
#pragma unroll
        for (int h = 0; h < F::kLane / 8; ++h) {
            const int i = u * (F::kLane / 8) + h;
            const uint4 v = lds16((i & 1 ? odd : even) + i * 64);
            c[4 * h] = v.x;
            c[4 * h + 1] = v.y;
            c[4 * h + 2] = v.z;
            c[4 * h + 3] = v.w;
        }
        F::operand(a, sc[0], u, p);
        F::operand(b, sc[1], u, q);
        float part[4];
        float(&d)[4] = F::kAfter ? part : sums;
#pragma unroll
        for (int m = 0; m < F::kMma; ++m) {
            const uint32_t frag[4] = {p[2 * m], q[2 * m], p[2 * m + 1], q[2 * m + 1]};
            if (m == 0 && (F::kAfter || (FRESH && u == 0)))
                mma16816<!F::kHalf, true>(d, frag, c[2 * m], c[2 * m + 1]);
            else
                mma16816<!F::kHalf>(d, frag, c[2 * m], c[2 * m + 1]);
        }
        if constexpr (F::kAfter) {
            const float slo = F::scale_after(sc[0], u), shi = F::scale_after(sc[1], u);
            const bool first = FRESH && u == 0;
            sums[0] = first ? slo * part[0] : fmaf(slo, part[0], sums[0]);
            sums[1] = first ? slo * part[1] : fmaf(slo, part[1], sums[1]);
            sums[2] = first ? shi * part[2] : fmaf(shi, part[2], sums[2]);
            sums[3] = first ? shi * part[3] : fmaf(shi, part[3], sums[3]);
        }
    }
}

// sums[nt] += 16 rows of a strip x the columns 8 nt to 8 nt + 7 for nt < NT, for
// columns that lie as tensor copies bring them: 128 bytes of each of `rows`
// rows, swizzled, for every 64 elements.  columns: the lane's, at wide_column_at().
// The warp takes the share-th of SHARES equal shares of the strip's steps.
template <class F, bool BF16, int NT, int SHARES>
__device__ __forceinline__ void wide_product(float (&sums)[NT][4], uint32_t tile, uint32_t half, uint32_t columns, uint32_t rows,
                                             typename F::Scales (&sc)[2], int left, int share, int t)
{
    typename F::Slice a, b;
    F::load(a, tile);
    F::load(b, tile + half);
    if (left < F::kStripK) {
        F::clear(a, sc[0], left, t);
        F::clear(b, sc[1], left, t);
    }
    constexpr int kAtOnce = F::kAfter && NT == 8 ? 1 : F::kSteps / SHARES;  // more would spill
#pragma unroll kAtOnce
    for (int i = 0; i < F::kSteps / SHARES; ++i) {
        const int u = SHARES == 1 ? i : share * (F::kSteps / SHARES) + i;
        uint32_t p[8], q[8];
        F::operand(a, sc[0], u, p);
        F::operand(b, sc[1], u, q);
        const uint32_t at = columns + u * rows * kStripBytes;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t c[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v = lds16((at ^ (16 * h)) + nt * 8 * kStripBytes);
                if constexpr (F::kSplit) {
                    c[4 * h] = __byte_perm(v.x, v.z, 0x5410);
                    c[4 * h + 1] = __byte_perm(v.x, v.z, 0x7632);
                    c[4 * h + 2] = __byte_perm(v.y, v.w, 0x5410);
                    c[4 * h + 3] = __byte_perm(v.y, v.w, 0x7632);
                } else {
                    c[4 * h] = v.x;
                    c[4 * h + 1] = v.y;
                    c[4 * h + 2] = v.z;
                    c[4 * h + 3] = v.w;
                }
            }
            float part[4];
            float(&d)[4] = F::kAfter ? part : sums[nt];
#pragma unroll
            for (int m = 0; m < F::kMma; ++m) {
                const uint32_t frag[4] = {p[2 * m], q[2 * m], p[2 * m + 1], q[2 * m + 1]};
                if (m == 0 && F::kAfter)
                    mma16816<!F::kHalf, true>(d, frag, c[2 * m], c[2 * m + 1]);
                else
                    mma16816<!F::kHalf>(d, frag, c[2 * m], c[2 * m + 1]);
            }
            if constexpr (F::kAfter) {
                const float slo = F::scale_after(sc[0], u), shi = F::scale_after(sc[1], u);
                sums[nt][0] = fmaf(slo, part[0], sums[nt][0]);
                sums[nt][1] = fmaf(slo, part[1], sums[nt][1]);
                sums[nt][2] = fmaf(shi, part[2], sums[nt][2]);
                sums[nt][3] = fmaf(shi, part[3], sums[nt][3]);
            }
        }
    }
}

__device__ __forceinline__ uint32_t wide_column_at(int lane)
{
    const int g = lane >> 2, t = lane & 3;
    return g * kStripBytes + ((2 * t) ^ g) * 16;
}

// ------------------------------------------------------------- the columns

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Eight bf16 values times `by` as fp16.
__device__ __forceinline__ uint4 scale_to_f16(uint4 v, float by)
{
    const auto two = [by](uint32_t w) {
        float lo, hi;
        bf16x2_to_f32(w, lo, hi);
        return f32x2_to_f16x2(lo * by, hi * by);
    };
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

// The largest finite magnitude of two bf16 values, as its bits, and `most`.
__device__ __forceinline__ uint32_t largest_bf16(uint32_t w, uint32_t most)
{
    const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    most = lo < 0x7F80u ? max(most, lo) : most;
    return hi < 0x7F80u ? max(most, hi) : most;
}

__device__ __forceinline__ uint32_t largest_bf16(uint4 v, uint32_t most)
{
    return largest_bf16(v.x, largest_bf16(v.y, largest_bf16(v.z, largest_bf16(v.w, most))));
}

// The exponent s for which a largest magnitude with bits `most` times 2^s lies
// in [2^14, 2^15), as far as 2^-s / divisor is a normal float; divisor >= 1.
__device__ __forceinline__ int column_exponent(uint32_t most, float divisor)
{
    const int top = 125 + 127 - static_cast<int>(__float_as_uint(divisor) >> 23);
    return most ? min(14 + 127 - static_cast<int>(most >> 7), top) : 0;
}

// Shared memory of `n` columns of `strips` strips.
template <class F>
__host__ __device__ constexpr int column_bytes(int n, int strips)
{
    return n * strips * F::kStripK * 2;
}

// Where a lane's column lies in a strip: in pieces of 64 bytes for the four
// lanes of a column, odd columns' pieces exchanged in pairs, so that two columns
// meet all banks.  `swap`: what is added for even pieces and taken off for odd.
// odd: column 0 counts as odd; size: bytes from column to column.
template <class F>
__device__ __forceinline__ uint32_t column_at(int n, int lane, uint32_t &swap, int odd = 0, uint32_t size = F::kStripK * 2)
{
    const int c = min(lane >> 2, n - 1);
    swap = ((c + odd) & 1) * 64;
    return c * size + (lane & 3) * 16;
}

// Where the i-th eight consecutive elements of a strip lie in its column, in
// bytes; odd: of an odd column.
template <class F>
__host__ __device__ __forceinline__ int piece_at(int i, int odd)
{
    // element k of a strip is lane tt's in step u
    const int k = 8 * i;
    int u, tt, half;
    if constexpr (F::kLane == 8) {
        u = (k >> 3) & 1;
        tt = k >> 4;
        half = 0;
    } else {
        half = (k >> 3) & 1;
        u = F::kAfter ? k >> 6 : (k >> 4) & 3;
        tt = F::kAfter ? (k >> 4) & 3 : k >> 6;
    }
    return ((u * (F::kLane / 8) + half) ^ odd) * 64 + tt * 16;
}

// Where element r of such eight lies, in elements.
template <class F>
__device__ __forceinline__ int element_at(int r)
{
    return F::kSplit ? 2 * (r & 3) + (r >> 2) : r;
}

// Whether columns are held times a power of two.
template <class F, bool BF16>
constexpr bool kScaled = BF16 && F::kHalf;

// Lays out the strips first, first + step, ... of columns [0, n) of K elements,
// zero past K; strip s comes to columns + s * column_bytes(n, 1).  column(c):
// where column c lies in global memory.  factors[8 s + c]: what the sums of the
// strip's column c have to be multiplied by, a power of two over `divisor`,
// which is at least 1 (kScaled).  One warp: it copies all its strips as they are, at once, and then
// rearranges each in place.
template <class F, bool BF16, class Column>
__device__ __forceinline__ void lay_out_strips(uint32_t columns, float *factors, Column column, int n, int first, int step,
                                               int K, float divisor, int lane)
{
    constexpr int kPieces = F::kStripK / 8;  // of a strip's column, 8 elements each
    constexpr int kAtOnce = 32 / kPieces;    // columns
    const int strips = strips_of<F>(K), i = lane % kPieces;
    for (int s = first; s < strips; s += step) {
        const int k = s * F::kStripK + 8 * i;
        const uint32_t to = columns + s * column_bytes<F>(n, 1) + 16 * lane;
        for (int c = lane / kPieces; c < n; c += kAtOnce)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (c - lane / kPieces) * (F::kStripK * 2)),
                         "l"(column(c) + (k < K ? k : 0)), "r"(k < K ? 16 : 0)
                         : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    for (int s = first; s < strips; s += step) {
        const uint32_t strip = columns + s * column_bytes<F>(n, 1);
        for (int c0 = 0; c0 < n; c0 += kAtOnce) {
            const int c = c0 + lane / kPieces;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (c < n)
                v = lds16(strip + c0 * (F::kStripK * 2) + 16 * lane);
            if constexpr (kScaled<F, BF16>) {  // a column is 32 lanes' pieces
                const int e = column_exponent(__reduce_max_sync(0xFFFFFFFFu, largest_bf16(v, 0)), divisor);
                v = scale_to_f16(v, pow2(e));
                if (lane == 0)
                    factors[s * kColumns + c] = pow2(-e) / divisor;
            }
            __syncwarp();
            if constexpr (F::kSplit)
                v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                               __byte_perm(v.y, v.w, 0x7632));
            if (c < n)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(strip + c * (F::kStripK * 2) + piece_at<F>(i, c & 1)),
                             "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
        }
    }
    __syncwarp();
}

// A global scale g divides the sums in two places.  g >= 1 comes with the
// columns' factors, which are far from overflow there although the sums times
// a factor alone may not be; g < 1 comes last, where an overflow is the result's.
__device__ __forceinline__ float early(float g) { return g >= 1.0f ? g : 1.0f; }
__device__ __forceinline__ float late(float g) { return g >= 1.0f ? 1.0f : g; }

// A warp's sums to shared memory, [8 columns][16 rows].
__device__ __forceinline__ void store_sums(float *to, const float (&acc)[4], int lane)
{
    const int g = lane >> 2, t = lane & 3;
    to[2 * t * 16 + g] = acc[0];
    to[(2 * t + 1) * 16 + g] = acc[1];
    to[2 * t * 16 + g + 8] = acc[2];
    to[(2 * t + 1) * 16 + g + 8] = acc[3];
}

// ----------------------------------------------------------------- the ring

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// The tensor copies of a matrix.
struct WeightMaps {
    CUtensorMap panels;  // [row][strip of the whole strips][128 bytes]: a block's rows x a panel's strips
    CUtensorMap strips;  // [row][byte]: a block's rows x 128 bytes, zero past the end of a row
    CUtensorMap scales;  // [row][byte of scales]: a block's rows x a panel's
    CUtensorMap zeros;   // int4: likewise
    int32_t tensor;        // rows are multiples of 16 bytes: the copies above; 0: 8-byte copies
    int32_t whole;         // whole strips of a row
    int32_t scale_tensor;  // the scales (and zero points, if any) of a panel are multiples of 16 bytes
    int32_t by_hand;       // lanes' own copies come with every slot
    uint32_t scale_bytes;  // of a panel's tensor copies of scales and zero points
    int32_t plain;         // tensor copies alone, and a row is whole strips
    uint32_t bytes;        // of a slot's tensor copies then
};

// A position in a ring.  Every group of consumers has a ring of its own: a slot
// that went from one group to another would let a group mistake the phase
// before the other's for the one that it waits for.
struct RingAt {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int depth)
    {
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
    }
};

constexpr int kMaxGroups = 8;

// Barriers of a slot: full, then empty, 8 bytes each.
constexpr int kBarrierBytes = 16;

__device__ __forceinline__ void tensor_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                     "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tensor_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
                     "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

// Copies `bytes` from src(r) for r < rows (a multiple of 16) to dst + r * pitch,
// by one warp, two lanes a row: in asynchronous pieces of 16, 8 or 4 bytes, as
// the alignment of every row allows (`align`: all addresses and `bytes` or-ed
// together), or else byte by byte at once.
template <class Source>
__device__ __forceinline__ void copy_rows(uint32_t dst, int pitch, int rows, Source src, int bytes, uintptr_t align, int lane)
{
    const int odd = lane & 1;
    for (int r = lane >> 1; r < rows; r += 16) {
        const uint8_t *from = src(r);
        const uint32_t to = dst + r * pitch;
        if (align % 16 == 0) {
            for (int b = 16 * odd; b < bytes; b += 32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + b), "l"(from + b) : "memory");
        } else if (align % 8 == 0) {
            for (int b = 8 * odd; b < bytes; b += 16)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + b), "l"(from + b) : "memory");
        } else if (align % 4 == 0) {
            for (int b = 4 * odd; b < bytes; b += 8)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + b), "l"(from + b) : "memory");
        } else {
#pragma unroll 4
            for (int b = odd; b < bytes; b += 2) {
                const uint32_t v = __ldg(from + b);
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + b), "r"(v) : "memory");
            }
        }
    }
}

// Arrivals that make a slot full: one with the tensor copies' bytes, and every
// lane's when its own copies have landed, if the producer's lanes make any.
__host__ __device__ inline int fill_arrivals(const WeightMaps &maps) { return maps.by_hand ? 33 : 1; }

// Where the tensor copies of scales and zero points of a panel that starts with
// strip `strip` begin in a row, in bytes: a multiple of 16.
template <class F, int FMT>
__device__ __forceinline__ int scale_x(const SlotPlan &plan, const WeightView &W, int strip)
{
    return FMT == kWNvfp4 ? 16 * strip : 2 * (((strip * F::kStripK) >> W.group_shift) & ~plan.scale.down);
}

template <class F>
__device__ __forceinline__ int zero_x(const SlotPlan &plan, const WeightView &W, int strip)
{
    return ((strip * F::kStripK) >> W.group_shift) & ~plan.scale.zero_down;
}

// The tensor copies into one slot of panel `panel` of the rows from lo on and,
// where a tile is two blocks, from hi on; `more` bytes come by other copies.
// One thread.
template <class F, int FMT>
__device__ __forceinline__ void fill_by_tensor(uint32_t slot, uint32_t full, const SlotPlan &plan, const WeightView &W,
                                               const WeightMaps &maps, int panel, int lo, int hi, uint32_t more)
{
    const int strip = panel * plan.strips;
    if (maps.plain) {  // the usual case, in as few instructions as it takes: the producer is one warp
        const bool pair = plan.half > 8 * kStripBytes;
        mbar_arrive_expect_tx(full, maps.bytes + more);
        tensor_3d(slot, &maps.panels, 0, lo, strip, full);
        if (pair)
            tensor_3d(slot + plan.half, &maps.panels, 0, hi, strip, full);
        if constexpr (FMT != kW16) {
            const uint32_t to = slot + plan.scale.at;
            const int x = scale_x<F, FMT>(plan, W, strip);
            tensor_2d(to, &maps.scales, x, lo, full);
            if (pair)
                tensor_2d(to + 8 * plan.scale.pitch, &maps.scales, x, hi, full);
            if (FMT == kWInt4 && plan.scale.zero_pitch) {
                const uint32_t z = slot + plan.scale.zero_at;
                const int zx = zero_x<F>(plan, W, strip);
                tensor_2d(z, &maps.zeros, zx, lo, full);
                if (pair)
                    tensor_2d(z + 8 * plan.scale.zero_pitch, &maps.zeros, zx, hi, full);
            }
        }
        return;
    }
    const int blocks = 16 * plan.tiles / plan.block;
    const bool by_panel = strip + plan.strips <= maps.whole || maps.whole * kStripBytes == F::row_bytes(W.K);
    const int here = by_panel ? plan.strips : min(plan.strips, (F::row_bytes(W.K) + kStripBytes - 1) / kStripBytes - strip);
    mbar_arrive_expect_tx(full, (maps.tensor ? 16 * plan.tiles * kStripBytes * here : 0) + maps.scale_bytes + more);
    for (int b = 0; b < blocks; ++b) {
        const int row = b ? hi : lo;
        const uint32_t to = slot + b * plan.half;
        if (maps.tensor) {
            if (by_panel)
                tensor_3d(to, &maps.panels, 0, row, strip, full);
            else
                for (int i = 0; i < here; ++i)
                    tensor_2d(to + i * plan.strip, &maps.strips, (strip + i) * kStripBytes, row, full);
        }
        if (FMT != kW16 && maps.scale_tensor) {
            tensor_2d(slot + plan.scale.at + b * 8 * plan.scale.pitch, &maps.scales, scale_x<F, FMT>(plan, W, strip), row, full);
            if (FMT == kWInt4 && plan.scale.zero_pitch)
                tensor_2d(slot + plan.scale.zero_at + b * 8 * plan.scale.zero_pitch, &maps.zeros, zero_x<F>(plan, W, strip), row,
                          full);
        }
    }
}

// What tensor copies cannot bring, by the lanes of one warp; rows from `rows`
// on are past the end of the matrix, and the last row stands in for them.
template <class F, int FMT>
__device__ __forceinline__ void fill_by_hand(uint32_t slot, uint32_t full, const SlotPlan &plan, const WeightView &W,
                                             const WeightMaps &maps, int panel, int lo, int hi, int rows, int lane)
{
    const int strip = panel * plan.strips, all = 16 * plan.tiles;
    const bool pair = plan.block < all;
    const auto row = [&](int r) { return static_cast<int64_t>(min(pair ? (r & 8 ? hi : lo) + (r & 7) : lo + r, rows - 1)); };
    if (!maps.tensor) {
        const int row_bytes = F::row_bytes(W.K), bytes = min(plan.strips * kStripBytes, row_bytes - strip * kStripBytes);
        for (int r = lane >> 1; r < all; r += 16) {
            const uint8_t *from = W.w + row(r) * row_bytes + strip * kStripBytes;
            const uint32_t to = slot + (pair ? (r >> 3) * plan.half + (r & 7) * kStripBytes : r * kStripBytes);
            for (int b = 8 * (lane & 1); b < bytes; b += 16)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + b / kStripBytes * plan.strip +
                                                                              (((b % kStripBytes) >> 4 ^ (r & 7)) << 4) + (b & 8)),
                             "l"(from + b)
                             : "memory");
        }
    }
    if (FMT != kW16 && !maps.scale_tensor) {
        const int shift = FMT == kWNvfp4 ? 4 : W.group_shift, size = FMT == kWNvfp4 ? 1 : 2;
        const int groups = W.K >> shift, k0 = strip * F::kStripK, k1 = min(k0 + plan.strips * F::kStripK, W.K);
        const int g0 = k0 >> shift, n = ((k1 - 1) >> shift) + 1 - g0;
        copy_rows(slot + plan.scale.at, plan.scale.pitch, all, [&](int r) { return W.scales + (row(r) * groups + g0) * size; },
                  size * n, reinterpret_cast<uintptr_t>(W.scales) | size * groups | size * g0 | size * n, lane);
        if (FMT == kWInt4 && plan.scale.zero_pitch)
            copy_rows(slot + plan.scale.zero_at, plan.scale.zero_pitch, all,
                      [&](int r) { return W.zeros + row(r) * groups + g0; }, n,
                      reinterpret_cast<uintptr_t>(W.zeros) | groups | g0 | n, lane);
    }
    // what was copied at once is visible to whoever sees the arrival; the asynchronous copies arrive by themselves
    __threadfence_block();
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p;\n"
                 "  mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 "  selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// The producer warp's work.  Lane g keeps group g's ring filled from items,
// which are the lane's own:
//   bool next(panel, lo, hi)     the panel and the rows of the next slot, or false at the end
//   uint32_t column_bytes()      what the slot also holds, by bulk copies of columns(slot, bar)
// The lanes go side by side, so that the producer's instructions are shared by
// the groups' slots, but none waits for another: groups meet at barriers, and a
// group may need more slots before it gets there while another's ring is full.
// Copies by hand take the whole warp and go group by group.  EARLY: weights may
// be read before the kernel before has ended, which is then waited for here;
// otherwise the caller has waited.
// `limit`: slots that lane 0 fills at most.
template <class F, int FMT, bool COLUMNS, bool EARLY, class Items>
__device__ __forceinline__ void produce(Items items, int groups, uint32_t slots, uint32_t bars, const SlotPlan &plan,
                                        const WeightView &W, const WeightMaps &maps, int rows, int64_t limit, int lane)
{
    RingAt at;
    const uint32_t ring = slots + lane * plan.depth * plan.bytes, ring_bars = bars + lane * plan.depth * kBarrierBytes;
    int panel = 0, lo = 0, hi = 0;
    bool more = lane < groups && !(lane == 0 && limit <= 0);
    if constexpr (EARLY) {
        if (maps.by_hand) {
            grid_dependency_wait();
            more = more && items.next(panel, lo, hi);
        } else {
            // the weights of the rings' slots first, and their columns when these are there
            Items columns = items;
            int primed = 0;
            while (more && (more = items.next(panel, lo, hi)) && primed < plan.depth) {
                fill_by_tensor<F, FMT>(ring + primed * plan.bytes, ring_bars + primed * kBarrierBytes, plan, W, maps, panel, lo, hi,
                                       items.column_bytes());
                ++primed;
            }
            __syncwarp();
            grid_dependency_wait();
            for (int i = 0; i < primed; ++i) {
                int x, y, z;
                columns.next(x, y, z);
                columns.columns(ring + i * plan.bytes, ring_bars + i * kBarrierBytes);
                at.next(plan.depth);
            }
        }
    } else {
        more = more && items.next(panel, lo, hi);
    }
    uint64_t since = 0;  // when the last slot was filled, or 0: just now
    while (__any_sync(0xFFFFFFFFu, more)) {
        const uint32_t bar = ring_bars + at.slot * kBarrierBytes, slot = ring + at.slot * plan.bytes;
        const bool ready = more && mbar_test(bar + 8, at.phase ^ 1);
        uint32_t filled = __ballot_sync(0xFFFFFFFFu, ready);
        if (!filled) {
            const uint64_t now = globaltimer_ns();
            if (since == 0)
                since = now;
            else if (now - since > kWaitLimitNs)
                break;
            __nanosleep(32);
            continue;
        }
        since = 0;
        if (ready) {
            uint32_t bytes = 0;
            if constexpr (COLUMNS)
                bytes = items.column_bytes();
            fill_by_tensor<F, FMT>(slot, bar, plan, W, maps, panel, lo, hi, bytes);
            if constexpr (COLUMNS)
                items.columns(slot, bar);
        }
        if (maps.by_hand)
            for (; filled; filled &= filled - 1) {
                const int g = __ffs(filled) - 1;
                fill_by_hand<F, FMT>(__shfl_sync(0xFFFFFFFFu, slot, g), __shfl_sync(0xFFFFFFFFu, bar, g), plan, W, maps,
                                     __shfl_sync(0xFFFFFFFFu, panel, g), __shfl_sync(0xFFFFFFFFu, lo, g),
                                     __shfl_sync(0xFFFFFFFFu, hi, g), rows, lane);
            }
        if (ready) {
            at.next(plan.depth);
            more = !(lane == 0 && --limit <= 0) && items.next(panel, lo, hi);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // No copy is left in flight when the CTA ends, even if the consumers have given up: every slot's last fill,
    // of this lap up to the next slot and of the lap before from it on.  (A parity that was never filled passes.)
    for (int s = 0; lane < groups && s < plan.depth; ++s)
        if (!mbar_wait_bounded(ring_bars + s * kBarrierBytes, at.phase ^ (s >= at.slot ? 1u : 0u), kWaitLimitNs))
            break;
}

// Waits of the consumers.  Once one has run out (after two seconds, which no
// healthy launch comes near) the warp goes through the rest of its work
// without waiting, so that barriers still match, and the results are marked.
// It gives no slot back any more, since a copy may still be on its way into it:
// the producer fills no slot a second time, and its own wait runs out.
struct Patience {
    volatile int32_t *failed;  // shared memory
    bool gone = false;
    __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity)
    {
        if (!gone && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
            gone = true;
            *failed = 1;
        }
    }
};

// A consumer warp at its group's ring: it takes strips j, j + warps, ... of
// every panel for one of the slot's tiles.
template <class F, int FMT, bool BF16>
struct Consumer {
    const SlotPlan &plan;
    const WeightView &W;
    Patience patience;
    uint32_t slot, bar;           // addresses of the next slot and its barriers
    int at = 0;                   // its place in the ring
    uint32_t phase = 0;
    uint32_t tile_at, scale_at;   // the lane's in the panel's first strip, from a slot on
    int j, t;

    __device__ Consumer(const SlotPlan &p, const WeightView &w, volatile int32_t *failed, uint32_t ring, uint32_t ring_bars, int tile,
                        int j_, int lane)
        : plan(p), W(w), patience{failed}, slot(ring), bar(ring_bars), j(j_), t(lane & 3)
    {
        tile_at = tile * 16 * kStripBytes + F::lane_at(lane >> 2, t);
        scale_at = F::scale_at(p.scale, tile * 16 + (lane >> 2), t);
    }

    __device__ __forceinline__ void wait() { patience.wait(bar, phase); }

    __device__ __forceinline__ void give_back()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0 && !patience.gone)
            mbar_arrive(bar + 8);
        slot += plan.bytes;
        bar += kBarrierBytes;
        if (++at == plan.depth) {
            slot -= at * plan.bytes;
            bar -= at * kBarrierBytes;
            at = 0;
            phase ^= 1;
        }
    }

    // The next slot, which holds panel `panel` and has been waited for: sums +=
    // its strips of this warp x columns.  column, swap: from column_at, in the
    // panel's first strip, strip_size bytes from strip to strip; factors: of the
    // panel's first strip's columns (SCALED), by which a strip's sums are
    // multiplied.  Gives the slot back.
    template <bool SCALED>
    __device__ __forceinline__ void take(float (&sums)[4], int panel, uint32_t column, uint32_t strip_size, uint32_t swap,
                                         uint32_t factors)
    {
        const int first = panel * plan.strips, from = first * F::kStripK;
#pragma unroll 1
        for (int i = j; i < plan.strips; i += plan.warps) {
            const int left = W.K - (first + i) * F::kStripK;
            if (left <= 0)
                break;
            typename F::Scales sc[2];
            F::load_scales(sc, slot + scale_at, plan, W, first + i, i, from);
            const uint32_t tile = slot + tile_at + i * plan.strip, col = column + i * strip_size;
            if constexpr (SCALED) {
                float part[4];
                strip_product<F, BF16, true>(part, tile, plan.half, col, swap, sc, left, t);
                const uint2 f = lds8(factors + i * (kColumns * 4) + 8 * t);
                sums[0] = fmaf(part[0], __uint_as_float(f.x), sums[0]);
                sums[1] = fmaf(part[1], __uint_as_float(f.y), sums[1]);
                sums[2] = fmaf(part[2], __uint_as_float(f.x), sums[2]);
                sums[3] = fmaf(part[3], __uint_as_float(f.y), sums[3]);
            } else {
                strip_product<F, BF16, false>(sums, tile, plan.half, col, swap, sc, left, t);
            }
        }
        give_back();
    }
};

// -------------------------------------------------------------- host side

constexpr size_t kSmemPerCta = 227 * 1024;

// Warps that split `strips` strips: at most `most`, and as few as leave the
// busiest warp no more strips than that.
inline int split_warps(int strips, int most)
{
    const int each = (strips + most - 1) / most;
    return (strips + each - 1) / each;
}

// Bytes of the box that brings one row's scales or zero points (`size` bytes a
// group) of a panel, from a multiple of 16 bytes on, by tensor copies; or 0 where
// rows do not allow them.
inline int tensor_scale_bytes(int strip_k, int strips, int K, int shift, int size, const void *at)
{
    if (!aligned16(at) || ((K >> shift) * size) % 16 != 0)
        return 0;
    const int bytes = ((strips * strip_k + (1 << shift) - 1) >> shift) * size;
    // what the panels start with is a multiple of the panel's bytes, or anything where groups are cut
    const bool whole = (strips * strip_k) % (1 << shift) == 0 && bytes % 16 == 0;
    const int box = whole ? bytes : (bytes + size + 15 + 15) / 16 * 16;
    return box <= 256 ? box : 0;
}

// A slot with `strips` strips of `tiles` tiles of 16 rows, for `warps` warps
// each, and `more` bytes of columns, and the kind of copies that fill it.  pair:
// the tile's halves are apart in the matrix.
template <class F, int FMT>
SlotPlan slot_plan(int warps, int strips, int tiles, bool pair, int more, const WeightView &W, WeightMaps &maps)
{
    SlotPlan s{};
    const int rows = 16 * tiles;
    s.warps = warps;
    s.strips = strips;
    s.tiles = tiles;
    s.block = pair ? 8 : rows;
    s.strip = s.block * kStripBytes;
    s.half = pair ? (strips * s.strip > 8 * kStripBytes ? strips * s.strip : 2 * s.strip) : 8 * kStripBytes;
    maps.tensor = F::row_bytes(W.K) % 16 == 0;
    int at = pair ? 2 * s.half : rows * strips * kStripBytes;
    if (FMT != kW16) {
        const int shift = FMT == kWNvfp4 ? 4 : W.group_shift, size = FMT == kWNvfp4 ? 1 : 2;
        const int bytes = tensor_scale_bytes(F::kStripK, strips, W.K, shift, size, W.scales);
        const int zeros = W.zeros ? tensor_scale_bytes(F::kStripK, strips, W.K, shift, 1, W.zeros) : 0;
        maps.scale_tensor = bytes > 0 && (!W.zeros || zeros > 0);
        maps.scale_bytes = maps.scale_tensor ? rows * (bytes + zeros) : 0;
        // by hand: a panel may start inside a group; an odd multiple of 16 spreads 8 rows over all banks
        const int groups = ((strips * F::kStripK) >> shift) + 2;
        s.scale.at = at;
        s.scale.pitch = maps.scale_tensor ? bytes : (size * groups + 15) / 16 * 16 | 16;
        s.scale.down = maps.scale_tensor ? 7 : 0;
        s.scale.zero_down = maps.scale_tensor ? 15 : 0;
        at = (at + rows * s.scale.pitch + 127) / 128 * 128;
        if (W.zeros) {
            s.scale.zero_at = at;
            s.scale.zero_pitch = maps.scale_tensor ? zeros : (groups + 15) / 16 * 16 | 16;
            at += rows * s.scale.zero_pitch;
        }
    }
    maps.by_hand = !maps.tensor || (FMT != kW16 && !maps.scale_tensor);
    maps.plain = !maps.by_hand && F::row_bytes(W.K) % kStripBytes == 0;
    maps.bytes = rows * strips * kStripBytes + maps.scale_bytes;
    s.columns_at = (at + 1023) / 1024 * 1024;
    s.bytes = (s.columns_at + more + 1023) / 1024 * 1024;
    return s;
}

// The tensor copies of 128 bytes of each of `box` rows of a matrix [rows, row_bytes], rows `pitch` bytes apart, for
// `chunks` runs of 128 bytes at once where a row is a whole number of them (a 3-dimensional map), or else one.
moe_status make_column_map(CUtensorMap &map, const void *at, int row_bytes, int rows, int64_t pitch, int box, int chunks);

// Encodes the tensor copies that slot_plan chose for W's `rows` rows (weight_maps.cu).
moe_status make_maps(WeightMaps &m, const SlotPlan &plan, const WeightView &W, int row_bytes, int64_t rows, int scale_row,
                     int zero_row);

// The same for a format; scale_row, zero_row: bytes of a row's scales and zero points.
template <class F, int FMT>
moe_status make_maps(WeightMaps &m, const SlotPlan &plan, const WeightView &W, int64_t rows)
{
    const int groups = FMT == kWNvfp4 ? W.K / 16 : FMT == kWInt4 ? W.K >> W.group_shift : 0;
    return make_maps(m, plan, W, F::row_bytes(W.K), rows, FMT == kWInt4 ? 2 * groups : groups, W.zeros ? groups : 0);
}

} // namespace nqg
