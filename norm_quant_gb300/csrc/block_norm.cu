// block_norm.cu -- the norms after a block and before the next one, with the
// block's gate and the residual's scale, forward and backward.
//
// Few operations a byte, so both passes are bound by HBM: what counts is bytes in flight.  One CTA an SM holds rows in
// slots of shared memory, which bulk copies (TMA) fill as far ahead as there is room.  Groups of warps (as many as
// a row of VPT vectors of 8 a thread takes, several groups a CTA for narrow rows) take the CTA's rows in turn, each
// with slots of its own; a row's values stay in shared memory and registers between the sums over it.  One thread of a
// group issues the copies (a producer warp of its own would make 17 warps, and leave 96 registers a thread).
// T = 8192, H = 4096: 48.5 us, 5.5 TB/s (6 us are launch, first rows and last; a register form without slots took 68).
//
// Backward.  With n = y / rms(y), m = s / rms(s) and c = block_scale * gate * (post_gamma + bias):
//   ds = d_residual_out + (v - m mean(v m)) / rms(s),   v = d_norm_out * (pre_gamma + bias)
//   d_y = (c ds - n mean(c ds n)) / rms(y)
// The sums over tokens of all three vectors are made of two: A = sum of ds n and B = sum of d_norm_out m, as
// d_post_gamma = block_scale gate A, d_gate = block_scale (post_gamma + bias) A and d_pre_gamma = B (a gate for each token
// goes into A).  A thread has its columns' A and B in registers over all rows of its CTA; groups are added up in shared memory,
// CTAs by a second kernel, each in its order.  T = 4096, H = 7168: 74 us, 4.8 TB/s.  That many registers leave room for 7 or 8
// warps of 32 columns a thread (16 of 16 columns: 76 us), and their chains of instructions, 33 an element, are what bounds it:
// issue slots are 35 % taken, DRAM 55 % busy.  Rows wider than 8192 leave no room for that: their kernel has A and B in
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
constexpr int kSums = 5;  // values that are added up over a row together
constexpr int kRingBytes = 226 * 1024;  // with a kilobyte of barriers, what a CTA may have
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
};

// Of each group, in shared memory: two buffers in turn, a value a warp.  Four of them are read at once.
struct alignas(16) GroupSums {
    float turns[2][kSums][kWarps];
};
static_assert(kWarps % 4 == 0 && sizeof(GroupSums) == 2 * kSums * kWarps * sizeof(float), "rows of whole vectors, one after the other");

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

__device__ __forceinline__ uint4 vector_of(const uint8_t *p, int i, bool take)
{
    return take ? ldg16(p + 16 * i) : make_uint4(0, 0, 0, 0);
}

// Two fp32 in a register pair: the packed instructions do both at once, each rounded like the scalar one.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void split(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t both(float v) { return pair_of(v, v); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ float total(uint64_t v)
{
    float lo, hi;
    split(v, lo, hi);
    return lo + hi;
}

// 8 elements as four pairs, and back.
template <bool BF16>
__device__ __forceinline__ void pairs8(uint64_t (&v)[4], const uint4 &w)
{
    float f[8];
    unpack8<BF16>(w, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pair_of(f[2 * i], f[2 * i + 1]);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&v)[4])
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        split(v[i], f[2 * i], f[2 * i + 1]);
    return pack8<BF16>(f);
}

// The columns' two factors, block_scale * gate * (post_gamma + bias) and pre_gamma + bias, as fp32 in shared memory: the
// first four of each vector of 8, and then the others, so that neighbouring lanes read neighbouring 16 bytes.
struct Factors {
    const float *c, *c2;
    int half;  // H / 2

    __device__ __forceinline__ static void read(uint64_t (&v)[4], const float *at, int i, int half)
    {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(at + 4 * i), b = *reinterpret_cast<const ulonglong2 *>(at + half + 4 * i);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
};

template <bool BF16>
__device__ __forceinline__ void fill_factors(const NormParams &p, float *c)
{
    constexpr int kAtOnce = 4;  // vectors whose loads are in flight together
    const int half = p.H / 2, vectors = p.H / 8;
    for (int base = threadIdx.x; base < vectors; base += kAtOnce * blockDim.x) {
        uint4 post[kAtOnce], gate[kAtOnce], pre[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = base + j * blockDim.x;
            const bool in = i < vectors;
            post[j] = vector_of(p.post, i, in && p.post);
            gate[j] = vector_of(p.gate, i, in && p.gate_kind == MOE_GATE_CHANNEL);
            pre[j] = vector_of(p.pre, i, in && p.pre);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = base + j * blockDim.x;
            if (i >= vectors)
                break;
            float v[8];
            factors8<BF16>(v, p, post[j], gate[j]);
            *reinterpret_cast<float4 *>(c + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(c + half + 4 * i) = make_float4(v[4], v[5], v[6], v[7]);
            gammas8<BF16>(v, p.pre != nullptr, pre[j], p.bias);
            *reinterpret_cast<float4 *>(c + p.H + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(c + p.H + half + 4 * i) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

__device__ __forceinline__ float token_gate(const NormParams &p, int64_t t)
{
    return p.gate_kind == MOE_GATE_TOKEN ? __ldg(reinterpret_cast<const float *>(p.gate) + t) : 1.0f;
}

__device__ __forceinline__ void store8(uint8_t *p, const uint4 &v) { *reinterpret_cast<uint4 *>(p) = v; }

// A group of warps that share a row.
struct Group {
    int warps, warp, lane, index;
    GroupSums &red;
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
                red.turns[turn][i][warp] = v[i];
        named_barrier_sync(1 + index, 32 * warps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = lane < warps ? red.turns[turn][i][lane] : 0.0f;
#pragma unroll
            for (int o = 8; o; o >>= 1)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            v[i] = __shfl_sync(0xffffffffu, v[i], 0);
        }
        turn ^= 1;
    }

    // Sums of kSums values over the group; the others are zeros.  Lanes share them out while they add up: 9 exchanges
    // instead of 40, and lane 4 i has the i-th.  Values of warps that the group does not have are 0 in `red`.
    __device__ __forceinline__ void sum8(float (&v)[8])
    {
#pragma unroll
        for (int n = 4, o = 16; n; n /= 2, o /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool upper = lane & o;
                const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        float mine = v[0];
        mine += __shfl_xor_sync(0xffffffffu, mine, 2);
        mine += __shfl_xor_sync(0xffffffffu, mine, 1);
        if (warps > 1) {
            const int which = lane / 4 < kSums ? lane / 4 : kSums - 1;
            if (lane % 4 == 0 && lane / 4 < kSums)
                red.turns[turn][which][warp] = mine;
            named_barrier_sync(1 + index, 32 * warps);
            const float4 w = *reinterpret_cast<const float4 *>(&red.turns[turn][which][4 * (lane % 4)]);
            mine = (w.x + w.y) + (w.z + w.w);
            mine += __shfl_xor_sync(0xffffffffu, mine, 2);
            mine += __shfl_xor_sync(0xffffffffu, mine, 1);
            turn ^= 1;
        }
#pragma unroll
        for (int i = 0; i < kSums; ++i)
            v[i] = __shfl_sync(0xffffffffu, mine, 4 * i);
    }
};

// The barriers, and the groups' sums in front of the slots.
__device__ __forceinline__ void ring_init(const NormParams &p, RingSmem &r, GroupSums *red)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.slots * p.groups; ++i) {
            mbar_init(smem_u32(&r.full[i]), 1);
            mbar_init(smem_u32(&r.empty[i]), static_cast<uint32_t>(p.group_warps));
        }
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < p.groups * 2 * kSums * kWarps; i += blockDim.x)
        (&red[0].turns[0][0][0])[i] = 0.0f;
    __syncthreads();
}

// A group's rows: t, t + step, and so on, each in the next of its slots.
template <bool BACKWARD>
struct Rows {
    const NormParams &p;
    const uint8_t *ring;  // the group's slots in shared memory
    uint32_t full;        // and their barriers
    uint32_t t;           // the row that is being worked on (rows are below 2^31), its slot and the phase of that one's barriers
    int slot;
    uint32_t flags;       // that phase, and kLost once a wait has run out
    uint32_t fills;       // copies that this thread may still issue: 0 in all threads but one
    static constexpr uint32_t kLost = 2;

    __device__ __forceinline__ Rows(const NormParams &q, RingSmem &r, const uint8_t *slots, const Group &g)
        : p(q), ring(slots + g.index * q.slots * q.stage), full(smem_u32(&r.full[g.index * q.slots])),
          t(blockIdx.x + g.index * gridDim.x), slot(0), flags(0), fills(0)
    {
        if (g.warp == 0 && g.lane == 0) {
            // test hook (moe_debug_stall)
            fills = blockIdx.x == 0 && g.index == 0 && q.stall >= 0 && q.stall < 0xFFFFFFFF ? static_cast<uint32_t>(q.stall) : 0xFFFFFFFFu;
            for (int i = 0; i < q.slots; ++i)
                fill(t + i * step(), i);
        }
    }

    __device__ __forceinline__ uint32_t step() const { return p.groups * gridDim.x; }
    __device__ __forceinline__ uint32_t empty(int i) const { return full + static_cast<uint32_t>(sizeof(RingSmem::full)) + 8u * i; }

    __device__ __forceinline__ void fill(uint32_t row, int to)
    {
        if (row >= p.T || fills == 0)
            return;
        --fills;
        const uint32_t row_bytes = 2u * static_cast<uint32_t>(p.H), dst = smem_u32(ring + to * p.stage), bar = full + 8u * to;
        const int64_t from = static_cast<int64_t>(row) * row_bytes;
        const bool dn = BACKWARD && p.d_norm_out, dr = BACKWARD && p.d_residual_out;
        mbar_arrive_expect_tx(bar, row_bytes * (1u + (p.residual != nullptr) + dn + dr));
        bulk_g2s(dst, p.y + from, row_bytes, bar);
        if (p.residual)
            bulk_g2s(dst + p.at_residual, p.residual + from, row_bytes, bar);
        if (dn)
            bulk_g2s(dst + p.at_d_norm, p.d_norm_out + from, row_bytes, bar);
        if (dr)
            bulk_g2s(dst + p.at_d_residual, p.d_residual_out + from, row_bytes, bar);
    }

    // Waits for the row; 0, or NaN once a wait has run out: it makes the row's sums and values NaN, and no further wait is made.
    __device__ __forceinline__ float wait()
    {
        if (!(flags & kLost) && !mbar_wait_bounded(full + 8u * slot, flags & 1, kWaitLimitNs))
            flags |= kLost;
        return flags & kLost ? __int_as_float(0x7FC00000) : 0.0f;
    }

    // 16 bytes of the row.
    __device__ __forceinline__ uint4 read(int at) const { return *reinterpret_cast<const uint4 *>(ring + slot * p.stage + at); }

    // The row's slot has been read: the row that comes next into it.
    __device__ __forceinline__ void release(const Group &g)
    {
        __syncwarp();
        if (g.lane == 0)
            mbar_arrive(empty(slot));
        if (fills && !(flags & kLost) && t + p.slots * step() < p.T) {
            if (mbar_wait_bounded(empty(slot), flags & 1, kWaitLimitNs))
                fill(t + p.slots * step(), slot);
            else
                fills = 0;
        }
        t += step();
        if (++slot == p.slots) {
            slot = 0;
            flags ^= 1;
        }
    }

    // Copies that were never waited for land before the CTA leaves.
    __device__ __forceinline__ void finish(const Group &g)
    {
        if (g.warp != 0 || g.lane != 0 || !(flags & kLost))
            return;
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < p.slots; ++i)
            while (!mbar_try_wait(full + 8u * i, (i >= slot ? flags : flags ^ 1) & 1) && globaltimer_ns() - t0 < kWaitLimitNs / 4) {
            }
    }
};

// FACTORS: the columns' factors are in shared memory behind the slots; else (rows that leave no room) they come from L1 at
// each use.
template <bool BF16, int VPT, bool FACTORS>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const NormParams p)
{
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ RingSmem r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    GroupSums *red = reinterpret_cast<GroupSums *>(dynamic);
    uint8_t *ring = dynamic + p.groups * sizeof(GroupSums);
    float *factors = reinterpret_cast<float *>(ring + p.slots * p.groups * p.stage);
    ring_init(p, r, red);
    grid_dependency_wait();
    Group g{p.group_warps, warp % p.group_warps, lane, warp / p.group_warps, red[warp / p.group_warps], 0};
    Rows<false> rows(p, r, ring, g);
    const int vectors = p.H / 8, threads = 32 * g.warps, first = 32 * g.warp + lane;
    if constexpr (FACTORS) {
        fill_factors<BF16>(p, factors);
        __syncthreads();
    }
    const auto factor = [&](uint64_t (&c)[4], int i, bool pre) {
        if constexpr (FACTORS) {
            Factors::read(c, factors + (pre ? p.H : 0), i, p.H / 2);
        } else {
            float v[8];
            if (pre)
                gammas8<BF16>(v, p.pre != nullptr, vector_of(p.pre, i, p.pre), p.bias);
            else
                factors8<BF16>(v, p, vector_of(p.post, i, p.post), vector_of(p.gate, i, p.gate_kind == MOE_GATE_CHANNEL));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c[k] = pair_of(v[2 * k], v[2 * k + 1]);
        }
    };
    while (rows.t < p.T) {
        const float lost = rows.wait();
        const int64_t t = rows.t, row = 2 * t * p.H;
        uint64_t s[VPT][4], acc = both(0.0f);
        float ry = 1.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            pairs8<BF16>(s[j], i < vectors ? rows.read(16 * i) : make_uint4(0, 0, 0, 0));
        }
        if (p.post) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc = fma2(s[j][k], s[j][k], acc);
            float sum[1] = {total(acc) + lost};
            g.sum(sum);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const uint64_t scale = both(ry * token_gate(p, t) + lost), from_residual = both(p.residual_scale);
        acc = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            if (i >= vectors)
                continue;  // zeros from here on, as they were
            uint64_t c[4], res[4];
            factor(c, i, false);
            if (p.residual) {
                pairs8<BF16>(res, rows.read(p.at_residual + 16 * i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[j][k] = fma2(s[j][k], mul2(scale, c[k]), mul2(from_residual, res[k]));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[j][k] = mul2(s[j][k], mul2(scale, c[k]));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc = fma2(s[j][k], s[j][k], acc);
        }
        rows.release(g);
        if (p.residual_out) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (first + j * threads < vectors)
                    store8(p.residual_out + row + 16 * (first + j * threads), pack_pairs<BF16>(s[j]));
        }
        if (!p.norm_out)
            continue;
        float sum[1] = {total(acc)};
        g.sum(sum);
        const uint64_t rs = both(rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps)));
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            if (i >= vectors)
                continue;
            uint64_t c[4];
            factor(c, i, true);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s[j][k] = mul2(s[j][k], mul2(rs, c[k]));
            store8(p.norm_out + row + 16 * i, pack_pairs<BF16>(s[j]));
        }
    }
    rows.finish(g);
}

// ALL: both norms, the residual and both gradients are there, as in training, and nothing has to be asked for them.
template <bool BF16, int VPT, bool ALL>
__global__ void __launch_bounds__(2 * kMaxThreads / VPT, 1) norm_backward_kernel(const NormParams p)
{
    const bool with_post = ALL || p.post, with_residual = ALL || p.residual, with_norm = ALL || p.d_norm_out, with_direct = ALL || p.d_residual_out;
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ RingSmem r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    GroupSums *red = reinterpret_cast<GroupSums *>(dynamic);
    uint8_t *ring = dynamic + p.groups * sizeof(GroupSums);
    float *factors = reinterpret_cast<float *>(ring + p.slots * p.groups * p.stage);
    ring_init(p, r, red);
    grid_dependency_wait();
    Group g{p.group_warps, warp % p.group_warps, lane, warp / p.group_warps, red[warp / p.group_warps], 0};
    Rows<true> rows(p, r, ring, g);
    const int vectors = p.H / 8, threads = 32 * g.warps, first = 32 * g.warp + lane, half = p.H / 2;
    fill_factors<BF16>(p, factors);
    __syncthreads();
    uint64_t A[VPT][4], B[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            A[j][k] = B[j][k] = both(0.0f);
    while (rows.t < p.T) {
        const float lost = rows.wait();
        const uint32_t t = rows.t;
        uint64_t y[VPT][4], s[VPT][4], acc = both(0.0f);
        // what the second pass over the row takes of it again; with two vectors a thread there are no registers for d_residual_out,
        // which stays in its slot
        constexpr bool kHold = VPT == 4;
        uint4 d[VPT], dr[VPT];
        float ry = 1.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            pairs8<BF16>(y[j], i < vectors ? rows.read(16 * i) : make_uint4(0, 0, 0, 0));
        }
        if (with_post) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc = fma2(y[j][k], y[j][k], acc);
            float sum[1] = {total(acc) + lost};
            g.sum(sum);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const float token = ry * token_gate(p, t) + lost;  // the token's gate over rms(y)
        const uint64_t scale = both(token);
        // with e = c y and v = d (pre_gamma + bias): the sums of s s, s v, and of dr e, v e and s e, of which that of ds e is made
        uint64_t ss = both(0.0f), sv = ss, re = ss, ve = ss, se = ss;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            d[j] = dr[j] = make_uint4(0, 0, 0, 0);
            if (i >= vectors)
                continue;
            uint64_t c[4], e[4], v[4];
            Factors::read(c, factors, i, half);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[k] = mul2(c[k], y[j][k]);
                s[j][k] = mul2(e[k], scale);
            }
            if (with_residual) {
                pairs8<BF16>(v, rows.read(p.at_residual + 16 * i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[j][k] = fma2(v[k], both(p.residual_scale), s[j][k]);
            }
            if (with_direct) {
                dr[j] = rows.read(p.at_d_residual + 16 * i);
                pairs8<BF16>(v, dr[j]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    re = fma2(v[k], e[k], re);
            }
            if (with_norm) {
                d[j] = rows.read(p.at_d_norm + 16 * i);
                pairs8<BF16>(v, d[j]);
                Factors::read(c, factors + p.H, i, half);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = mul2(v[k], c[k]);
                    ss = fma2(s[j][k], s[j][k], ss);
                    sv = fma2(s[j][k], v[k], sv);
                    ve = fma2(v[k], e[k], ve);
                    se = fma2(s[j][k], e[k], se);
                }
            }
        }
        if constexpr (kHold)
            rows.release(g);
        float rs = 0.0f, back = 0.0f, dot = 0.0f;  // 1 / rms(s), mean(v m) / rms(s)^2, the sum of c ds y
        if (with_norm) {
            float sum[8] = {total(ss), total(sv), total(re), total(ve), total(se), 0.0f, 0.0f, 0.0f};
            g.sum8(sum);
            rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            back = sum[1] * p.inv_h * rs * rs * rs;
            dot = sum[2] + rs * sum[3] - back * sum[4];
        } else if (with_post || p.gate_kind == MOE_GATE_TOKEN) {
            // `lost` too: without a norm after the block nothing else in a token's d_gate is NaN where its row never came
            float sum[1] = {total(re) + lost};
            g.sum(sum);
            dot = sum[0];
        }
        if (p.d_gate && p.gate_kind == MOE_GATE_TOKEN && g.warp == 0 && lane == 0)
            p.d_gate[t] = dot * ry;
        const uint64_t pull = both(with_post ? -dot * p.inv_h * token * ry * ry : 0.0f);  // - mean(c ds n) / rms(y)^2
        const uint64_t rs2 = both(rs), back2 = both(lost - back);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * threads;
            if (i >= vectors)
                continue;
            uint64_t c[4], ds[4];
            if constexpr (!kHold)
                dr[j] = with_direct ? rows.read(p.at_d_residual + 16 * i) : make_uint4(0, 0, 0, 0);
            pairs8<BF16>(ds, dr[j]);
            if (with_norm) {
                uint64_t v[4];
                pairs8<BF16>(v, d[j]);
                Factors::read(c, factors + p.H, i, half);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = mul2(v[k], rs2);
                    B[j][k] = fma2(v[k], s[j][k], B[j][k]);
                    ds[k] = fma2(v[k], c[k], fma2(back2, s[j][k], ds[k]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ds[k] = fma2(back2, s[j][k], ds[k]);  // back is 0, or NaN for a lost row
            }
            Factors::read(c, factors, i, half);
            uint64_t out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t f = mul2(ds[k], scale);
                A[j][k] = fma2(f, y[j][k], A[j][k]);
                out[k] = fma2(f, c[k], mul2(pull, y[j][k]));
                ds[k] = mul2(both(p.residual_scale), ds[k]);
            }
            const int64_t to = 2 * static_cast<int64_t>(t) * p.H + 16 * i;
            if (ALL || p.d_y)
                store8(p.d_y + to, pack_pairs<BF16>(out));
            if (ALL || p.d_residual)
                store8(p.d_residual + to, pack_pairs<BF16>(ds));
        }
        if constexpr (!kHold)
            rows.release(g);
    }
    rows.finish(g);
    if (p.partial) {
        // the groups' sums, added up in their order in dynamic shared memory
        float *sums = reinterpret_cast<float *>(dynamic);  // [2, H]
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
                    float4 x, y;
                    split(A[j][2 * k], x.x, x.y);
                    split(A[j][2 * k + 1], x.z, x.w);
                    split(B[j][2 * k], y.x, y.y);
                    split(B[j][2 * k + 1], y.z, y.w);
                    if (turn > 0) {
                        const float4 u = a[k], v = b[k];
                        x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
                        y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                    }
                    a[k] = x;
                    b[k] = y;
                }
            }
        }
        __syncthreads();
        float4 *out = reinterpret_cast<float4 *>(p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.H);
        for (int i = threadIdx.x; i < p.H / 2; i += blockDim.x)
            out[i] = reinterpret_cast<float4 *>(dynamic)[i];
    }
}

// The backward pass of wider rows: a row at a time in registers as it is in memory, A and B in shared memory in the order of
// Factors.
template <bool BF16>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_wide_kernel(const NormParams p)
{
    constexpr int VPT = MOE_MAX_HIDDEN / 8 / kMaxThreads;
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ GroupSums red;
    float *A = reinterpret_cast<float *>(dynamic), *B = A + p.H;
    grid_dependency_wait();
    const int vectors = p.H / 8, half = p.H / 2;
    Group g{kWarps, static_cast<int>(threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31), 0, red, 0};
    for (int i = threadIdx.x; p.partial && i < 2 * p.H; i += kMaxThreads)
        A[i] = 0.0f;
    __syncthreads();
    const auto factors = [&](uint64_t (&c)[4], int i, bool pre) {
        float v[8];
        if (pre)
            gammas8<BF16>(v, true, ldg16(p.pre + 16 * i), p.bias);
        else
            factors8<BF16>(v, p, vector_of(p.post, i, p.post), vector_of(p.gate, i, p.gate_kind == MOE_GATE_CHANNEL));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            c[k] = pair_of(v[2 * k], v[2 * k + 1]);
    };
    const auto add = [&](float *to, int i, const uint64_t (&v)[4]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float4 *at = reinterpret_cast<float4 *>(to + k * half + 4 * i);
            float4 a = *at, b;
            split(v[2 * k], b.x, b.y);
            split(v[2 * k + 1], b.z, b.w);
            *at = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
    };
    for (uint32_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t row = 2 * static_cast<int64_t>(t) * p.H;
        uint4 y[VPT], r[VPT], d[VPT], dr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * kMaxThreads;
            const int64_t at = row + 16 * i;
            y[j] = r[j] = d[j] = dr[j] = make_uint4(0, 0, 0, 0);
            if (i < vectors) {
                y[j] = *reinterpret_cast<const uint4 *>(p.y + at);
                if (p.residual)
                    r[j] = *reinterpret_cast<const uint4 *>(p.residual + at);
                if (p.d_norm_out)
                    d[j] = *reinterpret_cast<const uint4 *>(p.d_norm_out + at);
                if (p.d_residual_out)
                    dr[j] = *reinterpret_cast<const uint4 *>(p.d_residual_out + at);
            }
        }
        float ry = 1.0f;
        if (p.post) {
            uint64_t acc = both(0.0f);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                uint64_t v[4];
                pairs8<BF16>(v, y[j]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc = fma2(v[k], v[k], acc);
            }
            float sum[1] = {total(acc)};
            g.sum(sum);
            ry = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
        }
        const float token = ry * token_gate(p, t);
        const uint64_t scale = both(token), from_residual = both(p.residual_scale);
        // e = c y and s of a vector
        const auto parts = [&](int j, int i, uint64_t (&e)[4], uint64_t (&s)[4]) {
            uint64_t v[4];
            factors(e, i, false);
            pairs8<BF16>(v, y[j]);
            pairs8<BF16>(s, r[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[k] = mul2(e[k], v[k]);
                s[k] = fma2(e[k], scale, mul2(from_residual, s[k]));
            }
        };
        uint64_t ss = both(0.0f), sv = ss, re = ss, ve = ss, se = ss;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * kMaxThreads;
            if (i >= vectors)
                continue;
            uint64_t e[4], s[4], v[4], c[4];
            parts(j, i, e, s);
            pairs8<BF16>(v, dr[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                re = fma2(v[k], e[k], re);
            if (!p.d_norm_out)
                continue;
            pairs8<BF16>(v, d[j]);
            factors(c, i, true);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = mul2(v[k], c[k]);
                ss = fma2(s[k], s[k], ss);
                sv = fma2(s[k], v[k], sv);
                ve = fma2(v[k], e[k], ve);
                se = fma2(s[k], e[k], se);
            }
        }
        float sum[8] = {total(ss), total(sv), total(re), total(ve), total(se), 0.0f, 0.0f, 0.0f};
        g.sum8(sum);
        float rs = 0.0f, back = 0.0f;
        if (p.d_norm_out) {
            rs = rsqrt_newton(fmaf(sum[0], p.inv_h, p.eps));
            back = sum[1] * p.inv_h * rs * rs * rs;
        }
        const float dot = p.d_norm_out ? sum[2] + rs * sum[3] - back * sum[4] : sum[2];
        if (p.d_gate && p.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
            p.d_gate[t] = dot * ry;
        const uint64_t pull = both(p.post ? -dot * p.inv_h * token * ry * ry : 0.0f), rs2 = both(rs), back2 = both(-back);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = threadIdx.x + j * kMaxThreads;
            if (i >= vectors)
                continue;
            uint64_t e[4], s[4], v[4], c[4], ds[4];
            parts(j, i, e, s);
            pairs8<BF16>(ds, dr[j]);
            if (p.d_norm_out) {
                pairs8<BF16>(v, d[j]);
                factors(c, i, true);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = mul2(v[k], rs2);
                    ds[k] = fma2(v[k], c[k], fma2(back2, s[k], ds[k]));
                    v[k] = mul2(v[k], s[k]);
                }
                if (p.partial)
                    add(B, i, v);
            }
            factors(c, i, false);
            pairs8<BF16>(v, y[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[k] = mul2(ds[k], scale);
                c[k] = fma2(e[k], c[k], mul2(pull, v[k]));
                v[k] = mul2(e[k], v[k]);
                ds[k] = mul2(from_residual, ds[k]);
            }
            if (p.partial)
                add(A, i, v);
            if (p.d_y)
                store8(p.d_y + row + 16 * i, pack_pairs<BF16>(c));
            if (p.d_residual)
                store8(p.d_residual + row + 16 * i, pack_pairs<BF16>(ds));
        }
    }
    __syncthreads();
    float *out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.H;
    for (int i = threadIdx.x; p.partial && i < 2 * p.H; i += kMaxThreads) {
        const int h = i < p.H ? i : i - p.H;
        out[i] = A[i - h + (h / 4 % 2) * half + h / 8 * 4 + h % 4];
    }
}

// A and B over the CTAs, and the gradients that they make: 32 columns a block.  A warp adds up every 32nd CTA's, so that a
// thread has a handful of loads in flight at once, and then the 32 sums of one column.
template <bool BF16>
__global__ void __launch_bounds__(1024) column_sums_kernel(const NormParams p)
{
    __shared__ float part[2][32][33];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    grid_dependency_wait();
    int h = blockIdx.x * 32 + lane;
    float a = 0.0f, b = 0.0f;
    if (h < p.H) {
#pragma unroll 8
        for (int i = share; i < p.ctas; i += 32) {
            const float *at = p.partial + static_cast<int64_t>(i) * 2 * p.H + h;
            a += __ldg(at);
            b += __ldg(at + p.H);
        }
    }
    part[0][share][lane] = a;
    part[1][share][lane] = b;
    __syncthreads();
    a = part[0][lane][share];
    b = part[1][lane][share];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    h = blockIdx.x * 32 + share;
    if (lane == 0 && h < p.H) {
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
unsigned plan_ring(NormParams &p, int vpt, int tensors, bool factors, int warps)
{
    p.group_warps = (p.H / 8 + 32 * vpt - 1) / (32 * vpt);
    p.stage = (tensors * 2 * p.H + 127) / 128 * 128;
    p.groups = warps / p.group_warps;
    const int bytes = kRingBytes - p.groups * static_cast<int>(sizeof(GroupSums)) - (factors ? 8 * p.H : 0);
    const int room = bytes / p.stage < kMaxSlots ? bytes / p.stage : kMaxSlots;
    p.groups = p.groups > room ? room : p.groups;
    p.slots = room / p.groups;
    return static_cast<unsigned>(32 * p.groups * p.group_warps);
}

template <bool BF16, int VPT, bool FACTORS>
moe_status launch_norm(NormParams &p, moe_stream_t stream)
{
    static SmemLimit limit;
    int dev = 0;
    const int sms = sm_count();
    p.at_residual = 2 * p.H;
    const unsigned threads = plan_ring(p, VPT, p.residual ? 2 : 1, FACTORS, kWarps);
    const size_t smem = p.groups * sizeof(GroupSums) + static_cast<size_t>(p.slots) * p.groups * p.stage + (FACTORS ? 8 * p.H : 0);
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess ||
        ensure_dynamic_smem(norm_kernel<BF16, VPT, FACTORS>, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return PdlLaunch(static_cast<unsigned>(p.T < sms ? p.T : sms), threads, smem, stream).run(norm_kernel<BF16, VPT, FACTORS>, p);
}

// One for all forms that launch the kernel of wide rows: it is the kernel whose limit it keeps.
template <bool BF16>
SmemLimit &wide_limit()
{
    static SmemLimit limit;
    return limit;
}

template <bool BF16, int VPT, bool ALL>
moe_status launch_backward(NormParams &p, moe_stream_t stream)
{
    static SmemLimit limit;
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
        threads = plan_ring(p, VPT, at / (2 * p.H), true, 2 * kWarps / VPT);
        // the slots' memory holds the sums at the end
        const size_t ring = p.groups * sizeof(GroupSums) + static_cast<size_t>(p.slots) * p.groups * p.stage + 8 * p.H;
        smem = smem > ring ? smem : ring;
    }
    const auto kern = wide ? norm_backward_wide_kernel<BF16> : norm_backward_kernel<BF16, VPT, ALL>;
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess ||
        ensure_dynamic_smem(kern, dev, static_cast<int>(smem), wide ? wide_limit<BF16>() : limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int64_t most = sms < kMaxCtas ? sms : kMaxCtas;
    p.ctas = static_cast<int32_t>(p.T < most ? p.T : most);
    const moe_status st = PdlLaunch(static_cast<unsigned>(p.ctas), threads, smem, stream).run(kern, p);
    if (st != MOE_OK || !p.partial)
        return st;
    return PdlLaunch(static_cast<unsigned>((p.H + 31) / 32), 1024, 0, stream).run(column_sums_kernel<BF16>, p);
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
    if (a->H <= 2048)
        return bf16 ? launch_norm<true, 2, true>(p, stream) : launch_norm<false, 2, true>(p, stream);
    if (a->H <= kMaxRingWidth)
        return bf16 ? launch_norm<true, 4, true>(p, stream) : launch_norm<false, 4, true>(p, stream);
    return bf16 ? launch_norm<true, 4, false>(p, stream) : launch_norm<false, 4, false>(p, stream);
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
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    const bool all = p.post && p.residual && p.d_norm_out && p.d_residual_out && p.d_y && p.d_residual;
    // Four vectors a thread and half the warps amortise what a row costs beside its elements, where they leave no warp idle.
    // Two / four, us: T = 4096, H = 8192: 77.6 / 73.2, 7168: 76.0 / 71.8; T = 8192, H = 4096: 73.7 / 71.6; T = 16384, H =
    // 1024: 44.2 / 42.9; with warps idle, T = 4096, H = 6144: 67.3 / 70.6; T = 1021, H = 2056: 13.5 / 14.7.
    const int row_warps = (a->H / 8 + 127) / 128, used = 8 / row_warps * row_warps;
    if (all && a->H > 512 && used >= 7)
        return bf16 ? launch_backward<true, 4, true>(p, stream) : launch_backward<false, 4, true>(p, stream);
    if (all)
        return bf16 ? launch_backward<true, 2, true>(p, stream) : launch_backward<false, 2, true>(p, stream);
    return bf16 ? launch_backward<true, 2, false>(p, stream) : launch_backward<false, 2, false>(p, stream);
}
