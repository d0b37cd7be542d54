// linear_w4.cu -- out[m, n] = sum_k x[m, k] W[n, k] for a few rows x and a
// matrix W in 4 bits (NVFP4, or integers with group scales).
//
// Two kernels.  In both a CTA, one an SM, takes an equal, consecutive share of
// the blocks of 16 rows of W, and warps that split k add their fp32 sums in the
// order of the warps, so that a result does not depend on timing.
//
// The wide one streams columns (rows of x) with the weights, and takes the
// blocks of a CTA together, so that the columns are read once for up to 4.
// The resident one holds the columns in shared memory for the whole of k, as
// fp16 times a power of two.  It is there for bf16 columns and NVFP4 alone: e2m1
// codes widen to fp16 in one conversion for two but to bf16 in three or four operations, and
// with a column or two the widening is what a CTA's time goes into.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_layer.h"
#include "common.h"
#include "ptx.cuh"
#include "skinny.cuh"

namespace nqg {
namespace {

struct LinearParams {
    WeightMaps maps;
    WeightView W;
    SlotPlan plan;
    const uint16_t *x;
    uint16_t *out;
    int64_t x_stride, out_stride;
    int32_t M, N, panels, groups;
    float divisor;
    int64_t stall;  // test hook: CTA 0 fills no more than this many slots (-1: off)
};

// Shared memory: slots, barriers and a flag, the columns' factors, two sets of sums a group, columns.
__host__ __device__ inline uint32_t bars_at(const SlotPlan &s, int groups) { return groups * s.depth * s.bytes; }
__host__ __device__ inline uint32_t factors_at(const SlotPlan &s, int groups)
{
    return bars_at(s, groups) + (groups * s.depth * kBarrierBytes + 4 + 15) / 16 * 16;
}
__host__ __device__ inline uint32_t sums_at(const SlotPlan &s, int groups, int panels)
{
    return factors_at(s, groups) + panels * s.strips * kColumns * 4;
}
__host__ __device__ inline uint32_t columns_at(const SlotPlan &s, int groups, int panels)
{
    return sums_at(s, groups, panels) + groups * s.warps * 1024;
}

// The resident kernel.  The consumer warps form groups, each with a ring of its
// own: the warps of a group split k, and the groups take different blocks of 16
// rows.  Bound by the instructions that widen codes, about 300 a warp for 4096
// weights.  K = 7168, M = 1: N = 16384, 17.3 us, 3.8 TB/s of weights; N = 2048, 5.5 us, and
// 4.7 with the weights in L2, of which 2.5 are the launch.
__global__ void __launch_bounds__(32 * (kMaxConsumers<kWNvfp4> + 1), 1)
    linear_w4_resident_kernel(const __grid_constant__ LinearParams p)
{
    using F = Format<kWNvfp4, true>;
    static_assert(kScaled<F, true>);
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = p.plan.warps, depth = p.plan.depth;
    const int consumers = warps * p.groups;
    const uint32_t slots = smem_u32(smem), bars = slots + bars_at(p.plan, p.groups);
    volatile int32_t *failed =
        reinterpret_cast<volatile int32_t *>(smem + bars_at(p.plan, p.groups) + p.groups * depth * kBarrierBytes);
    float *factors = reinterpret_cast<float *>(smem + factors_at(p.plan, p.groups));  // [panels * warps][8]
    const int all = (p.N + 15) / 16;
    const int first = static_cast<int>(static_cast<int64_t>(all) * blockIdx.x / gridDim.x);
    const int last = static_cast<int>(static_cast<int64_t>(all) * (blockIdx.x + 1) / gridDim.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.groups * depth; ++i) {
            mbar_init(bars + i * kBarrierBytes, fill_arrivals(p.maps));
            mbar_init(bars + i * kBarrierBytes + 8, warps);
        }
        *failed = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == consumers) {  // the producer
        struct Items {  // the slots of one group
            int b, panel, last, step, panels;
            __device__ bool next(int &at, int &lo, int &hi)
            {
                if (panel == panels) {
                    panel = 0;
                    b += step;
                }
                if (b >= last)
                    return false;
                at = panel++;
                lo = 16 * b;
                hi = 16 * b + 8;
                return true;
            }
        };
        produce<F, kWNvfp4, false, false>(Items{first + lane, 0, last, p.groups, p.panels}, p.groups, slots, bars, p.plan, p.W,
                                          p.maps, p.N, blockIdx.x == 0 && p.stall >= 0 ? p.stall : INT64_MAX, lane);
        return;
    }
    const int group = warp / warps, j = warp - group * warps;
    Consumer<F, kWNvfp4, true> consumer(p.plan, p.W, failed, slots + group * depth * p.plan.bytes,
                                        bars + group * depth * kBarrierBytes, 0, j, lane);
    const uint32_t columns = slots + columns_at(p.plan, p.groups, p.panels);
    float *red = reinterpret_cast<float *>(smem + sums_at(p.plan, p.groups, p.panels)) + group * warps * 256;  // [2][warps][8 columns][16 rows]
    lay_out_strips<F, true>(columns, factors, [&](int c) { return p.x + c * p.x_stride; }, p.M, warp, consumers, p.W.K,
                            early(p.divisor), lane);
    named_barrier_sync(1, 32 * consumers);
    uint32_t swap;
    const uint32_t column = columns + column_at<F>(p.M, lane, swap), size = column_bytes<F>(p.M, 1);
    int turn = 0;
    for (int b = first + group; b < last; b += p.groups, ++turn) {
        float acc[4] = {};
        for (int panel = 0; panel < p.panels; ++panel) {
            consumer.wait();
            consumer.template take<true>(acc, panel, column + panel * p.plan.strips * size, size, swap,
                                         smem_u32(factors + panel * p.plan.strips * kColumns));
        }
        float *set = red + (turn & 1) * warps * 128;
        store_sums(set + j * 128, acc, lane);
        named_barrier_sync(2 + group, 32 * warps);
        // the other set is written next, and this one only after another barrier
        if (j == turn % warps) {
            const int n0 = 16 * b;
            for (int i = lane; i < 16 * p.M; i += 32) {
                float s = 0.0f;
                for (int w = 0; w < warps; ++w)
                    s += set[w * 128 + i];
                if (*failed)
                    s = __int_as_float(0x7FC00000);
                s /= late(p.divisor);  // the columns' factors hold the early part
                if (n0 + (i & 15) < p.N)
                    p.out[(i >> 4) * p.out_stride + n0 + (i & 15)] = narrow16<true>(s);
            }
        }
    }
}

// What a launch of that kernel takes, or false where the columns do not fit
// beside three slots (two for each of several groups).
bool plan_resident(LinearParams &p, int sms, size_t &smem)
{
    using F = Format<kWNvfp4, true>;
    const int strips = strips_of<F>(p.W.K), blocks = (p.N + 15) / 16, each = (blocks + sms - 1) / sms;
    // Few blocks: one group of as many warps as split k.  More: groups of up to 8, as many as there are warps.
    const int warps = split_warps(strips, each < 2 ? 16 : 8);
    const auto bytes = [&](int depth) {
        SlotPlan s = p.plan;
        s.depth = depth;
        return static_cast<size_t>(columns_at(s, p.groups, p.panels)) + column_bytes<F>(p.M, s.strips * p.panels);
    };
    const auto least = [&] { return p.groups < 2 ? 3 : 2; };
    int most = kMaxConsumers<kWNvfp4> / warps;
    most = most < each ? most : each;
    most = most < kMaxGroups ? most : kMaxGroups;
    // Two strips a warp in a slot where that fits for all groups, else one, and as
    // many groups as fit; what is left holds more slots.
    for (int m = strips >= 2 * warps ? 2 : 1; m > 0; --m) {
        p.panels = (strips + m * warps - 1) / (m * warps);
        p.plan = slot_plan<F, kWNvfp4>(warps, m * warps, 1, false, 0, p.W, p.maps);
        for (p.groups = most; p.groups > 0; --p.groups) {
            if (bytes(least()) > kSmemPerCta) {
                if (m > 1)
                    break;
                continue;
            }
            p.plan.depth = least();
            while (p.plan.depth * p.groups < 16 && bytes(p.plan.depth + 1) <= kSmemPerCta)
                ++p.plan.depth;
            smem = bytes(p.plan.depth);
            return true;
        }
    }
    return false;
}

moe_status launch_resident(LinearParams &p, int sms, size_t smem, moe_stream_t stream)
{
    static SmemLimit limit;
    const int blocks = (p.N + 15) / 16;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        ensure_dynamic_smem(linear_w4_resident_kernel, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const moe_status st = make_maps<Format<kWNvfp4, true>, kWNvfp4>(p.maps, p.plan, p.W, p.N);
    if (st != MOE_OK)
        return st;
    return PdlLaunch(static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * (p.plan.warps * p.groups + 1), smem, stream)
        .run(linear_w4_resident_kernel, p);
}

// The wide kernel.  A CTA takes its blocks of 16 rows as the tiles of a slot,
// in passes of up to 4.  The columns come with the weights, as they lie in
// memory, and are read once for all tiles of a pass.  A consumer warp takes strip j
// of every panel, or half of its steps, for one tile and all columns (1, 2, 4 or 8 times
// 8), so that a weight is widened once.  With 32 columns and more the matrix
// instruction is the bound: 47 cycles of an SM a strip (4096 weights) and 8
// columns, against 100 that the strip's bytes take; below that it is the issue
// of the instructions that widen and lay out, 270 a strip.
// N = 16384, K = 7168: fp16 columns and NVFP4, M = 1 to 8, 17.3 us, 3.8 TB/s of
// weights; integers, group 128, 22 us.  N = K = 7168, weights from HBM (in L2): NVFP4, M = 32, 16.6
// (15.9) us; integers, M = 64, 24.9 (23.8) us, 264 Tflop/s.
// Scales that tensor copies cannot take (rows that are no multiple of 16 bytes) are copied by the
// producer's lanes: bf16, group 128 with zero points, N = 7168, M = 1: K = 8192 by tensor copies
// 12.5 us, K = 7168 by lanes 17.5; NVFP4, N = 16384, M = 8: K = 2816 12.9, K = 2880 15.8.
//
// Consumers: with the producer 24 warps, for 80 registers each, or 16, for 128.
// With 23 instead of 15 consumers and 8 columns N = 16384 takes 17.4 instead of
// 18.6 us, N = 7168 8.0 instead of 7.8.
template <int NT>
constexpr int kWideWarps = NT == 1 ? 23 : 15;

// With 16 columns and fewer their permutations cost less than neighbours.
template <int NT>
constexpr int kWideSteps = NT > 2 ? kPairs : kApart;

// Warps that share a strip's steps: with more columns, shared memory holds fewer strips.
template <int NT>
constexpr int kShares = NT <= 2 ? 1 : 2;

struct WideParams {
    WeightMaps maps;
    CUtensorMap x;
    WeightView W;
    SlotPlan plan;
    uint16_t *out;
    int64_t out_stride;
    int32_t M, N, panels;
    float divisor;
    int64_t stall;
};

__host__ __device__ inline uint32_t wide_sums_at(const SlotPlan &s)
{
    return (s.depth * (s.bytes + kBarrierBytes) + 4 + 15) / 16 * 16;
}

template <int FMT, bool BF16, int NT>
__global__ void __launch_bounds__(32 * (kWideWarps<NT> + 1), 1) linear_w4_wide_kernel(const __grid_constant__ WideParams p)
{
    using F = Format<FMT, BF16, true, kWideSteps<NT>>;
    constexpr int kRows = 8 * NT;  // of the columns' boxes
    extern __shared__ __align__(1024) uint8_t smem[];
    const SlotPlan &plan = p.plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = plan.strips * kShares<NT>,
              consumers = warps * plan.tiles;
    const uint32_t slots = smem_u32(smem), bars = slots + plan.depth * plan.bytes;
    volatile int32_t *failed = reinterpret_cast<volatile int32_t *>(smem + plan.depth * (plan.bytes + kBarrierBytes));
    float *red = reinterpret_cast<float *>(smem + wide_sums_at(plan));  // [tiles][warps][columns][16]
    const int all = (p.N + 15) / 16;
    const int first = static_cast<int>(static_cast<int64_t>(all) * blockIdx.x / gridDim.x);
    const int last = static_cast<int>(static_cast<int64_t>(all) * (blockIdx.x + 1) / gridDim.x);
    if (tid == 0) {
        for (int i = 0; i < plan.depth; ++i) {
            mbar_init(bars + i * kBarrierBytes, fill_arrivals(p.maps));
            mbar_init(bars + i * kBarrierBytes + 8, consumers);
        }
        *failed = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == consumers) {  // the producer
        struct Items {
            const WideParams &p;
            int b, panel, last, now;
            __device__ bool next(int &at, int &lo, int &hi)
            {
                if (panel == p.panels) {
                    panel = 0;
                    b += p.plan.tiles;
                }
                if (b >= last)
                    return false;
                at = now = panel++;
                lo = 16 * b;
                hi = lo + 8;
                return true;
            }
            // runs of 64 elements; what lies past the end of a row is zero
            __device__ uint32_t column_bytes() const { return 4 * p.plan.strips * kRows * kStripBytes; }
            __device__ void columns(uint32_t slot, uint32_t bar) const
            {
                const int chunk = 4 * now * p.plan.strips;
                if (p.W.K % 64 == 0)
                    tensor_3d(slot + p.plan.columns_at, &p.x, 0, 0, chunk, bar);
                else
                    for (int i = 0; i < 4 * p.plan.strips; ++i)
                        tensor_2d(slot + p.plan.columns_at + i * kRows * kStripBytes, &p.x, (chunk + i) * kStripBytes, 0, bar);
            }
        };
        produce<F, FMT, true, false>(Items{p, first, 0, last, 0}, 1, slots, bars, plan, p.W, p.maps, p.N,
                                     blockIdx.x == 0 && p.stall >= 0 ? p.stall : INT64_MAX, lane);
        return;
    }
    const int tile = warp / warps, j = (warp - tile * warps) / kShares<NT>, share = warp % kShares<NT>, t = lane & 3;
    Consumer<F, FMT, BF16> consumer(plan, p.W, failed, slots, bars, tile, j, lane);
    const uint32_t column = plan.columns_at + j * 4 * kRows * kStripBytes + wide_column_at(lane);
    for (int b0 = first; b0 < last; b0 += plan.tiles) {
        float acc[NT][4] = {};
        for (int panel = 0; panel < p.panels; ++panel) {
            const int strip = panel * plan.strips + j, left = p.W.K - strip * F::kStripK;
            consumer.wait();
            if (left > 0) {
                typename F::Scales sc[2];
                F::load_scales(sc, consumer.slot + consumer.scale_at, plan, p.W, strip, j, panel * plan.strips * F::kStripK);
                wide_product<F, BF16, NT, kShares<NT>>(acc, consumer.slot + consumer.tile_at + j * plan.strip, plan.half, consumer.slot + column, kRows,
                                          sc, left, share, t);
            }
            consumer.give_back();
        }
        float *mine = red + warp * kRows * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            store_sums(mine + nt * 128, acc[nt], lane);
        named_barrier_sync(1, 32 * consumers);
        for (int i = tid; i < 16 * p.M * plan.tiles; i += 32 * consumers) {
            const int r = i & 15, c = (i >> 4) % p.M, q = (i >> 4) / p.M, n = 16 * (b0 + q) + r;
            if (b0 + q >= last || n >= p.N)
                continue;
            float s = 0.0f;
            for (int w = 0; w < warps; ++w)
                s += red[(q * warps + w) * kRows * 16 + c * 16 + r];
            if (*failed)
                s = __int_as_float(0x7FC00000);
            if (FMT == kWNvfp4)
                s = s * (F::kPost / early(p.divisor)) / late(p.divisor);
            p.out[c * p.out_stride + n] = narrow16<BF16>(s);
        }
        named_barrier_sync(1, 32 * consumers);  // the sums have been read
    }
}

template <int FMT, bool BF16, int NT>
moe_status launch_wide(const LinearParams &a, moe_stream_t stream)
{
    using F = Format<FMT, BF16, true, kWideSteps<NT>>;
    constexpr int kRows = 8 * NT;
    static SmemLimit limit;
    const int sms = sm_count(), strips = strips_of<F>(a.W.K), blocks = (a.N + 15) / 16;
    if (sms <= 0)
        return MOE_ERR_CUDA;
    WideParams p{};
    p.W = a.W;
    p.out = a.out;
    p.out_stride = a.out_stride;
    p.M = a.M;
    p.N = a.N;
    p.divisor = a.divisor;
    p.stall = a.stall;
    const auto bytes = [&](int depth) {
        SlotPlan s = p.plan;
        s.depth = depth;
        return static_cast<size_t>(wide_sums_at(s)) + static_cast<size_t>(s.tiles) * s.strips * kShares<NT> * kRows * 64;
    };
    const int per_cta = (blocks + sms - 1) / sms;
    // equal passes of at most 4 tiles
    const int passes = (per_cta + 3) / 4, tiles = (per_cta + passes - 1) / passes;
    for (int w = split_warps(strips, kWideWarps<NT> / (tiles * kShares<NT>));; --w) {
        p.plan = slot_plan<F, FMT>(w, w, tiles, false, w * 4 * kRows * kStripBytes, p.W, p.maps);
        if (bytes(2) <= kSmemPerCta)
            break;
        if (w == 1)
            return MOE_ERR_UNSUPPORTED;
    }
    p.panels = (strips + p.plan.strips - 1) / p.plan.strips;
    p.plan.depth = 2;
    while (p.plan.depth < 8 && bytes(p.plan.depth + 1) <= kSmemPerCta)
        ++p.plan.depth;
    const size_t smem = bytes(p.plan.depth);
    int dev = 0;
    const auto kern = linear_w4_wide_kernel<FMT, BF16, NT>;
    if (cudaGetDevice(&dev) != cudaSuccess || ensure_dynamic_smem(kern, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    moe_status st = make_maps<F, FMT>(p.maps, p.plan, p.W, p.N);
    if (st == MOE_OK)
        st = make_column_map(p.x, a.x, 2 * p.W.K, p.M, 2 * a.x_stride, kRows, 4 * p.plan.strips);
    if (st != MOE_OK)
        return st;
    return PdlLaunch(static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * (p.plan.strips * kShares<NT> * tiles + 1), smem, stream).run(kern, p);
}

template <int FMT, bool BF16>
moe_status launch(LinearParams &p, moe_stream_t stream)
{
    if constexpr (FMT == kWNvfp4 && BF16) {
        const int sms = sm_count();
        size_t smem;
        if (sms <= 0)
            return MOE_ERR_CUDA;
        // Both kernels timed with K = 7168 (weights that fit in L2 are there), us, resident against wide: N = 16384,
        // M = 1: 18.3 / 23.9, 4: 21.1 / 23.9, 6: 23.6 / 24.0, 8: 27.7 / 24.0; N = 7168, M = 1:
        // 8.6 / 10.8, 2: 9.4 / 10.5, 3: 10.5 / 10.6, 6: 15.2 / 10.4; N = 2048, M = 1: 4.8 / 5.9,
        // 3: 6.9 / 5.6.  With little k there is not enough to do to lay columns out:
        // N = 7000, K = 2048, M = 1: 5.1 / 4.8; N = K = 4096, M = 1: 5.8 / 6.1.
        if (p.M <= 6 && p.M <= 1 + p.N / 4096 && p.W.K >= 4096 && plan_resident(p, sms, smem))
            return launch_resident(p, sms, smem, stream);
    }
    return p.M <= 8    ? launch_wide<FMT, BF16, 1>(p, stream)
           : p.M <= 16 ? launch_wide<FMT, BF16, 2>(p, stream)
           : p.M <= 32 ? launch_wide<FMT, BF16, 4>(p, stream)
                       : launch_wide<FMT, BF16, 8>(p, stream);
}

} // namespace
} // namespace nqg

using namespace nqg;

extern "C" size_t moe_linear_w4_args_size(void) { return sizeof(moe_linear_w4_args); }

extern "C" moe_status moe_linear_w4(const moe_linear_w4_args *a, moe_stream_t stream)
{
    if (!a || a->M < 0 || a->N < 1 || a->K < 1)
        return MOE_ERR_INVALID_ARG;
    const bool int4 = a->w_format == MOE_W_INT4;
    if ((!int4 && a->w_format != MOE_W_NVFP4) || (a->io_dtype != MOE_IO_BF16 && a->io_dtype != MOE_IO_FP16))
        return MOE_ERR_INVALID_ARG;
    const int shift = int4 ? group_shift(a->group_size) : 4;
    if (shift < 0 || a->K % (1 << shift) != 0 || (!int4 && (a->w_zeros || !(a->global_scale > 0.0f) || std::isinf(a->global_scale))))
        return MOE_ERR_INVALID_ARG;
    if (a->M > MOE_FEW_TOKENS || a->N > MOE_FEW_MAX_DIM || a->K > MOE_FEW_MAX_K)
        return MOE_ERR_UNSUPPORTED;
    if (a->M == 0)
        return MOE_OK;
    if (!a->x || !a->w || !a->w_scales || !a->out || !aligned16(a->x) || !aligned16(a->w) ||
        (reinterpret_cast<uintptr_t>(a->out) & 1u) || (int4 && (reinterpret_cast<uintptr_t>(a->w_scales) & 1u)))
        return MOE_ERR_INVALID_ARG;
    if (a->x_stride < a->K || a->x_stride % 8 != 0 || a->out_stride < a->N)
        return MOE_ERR_INVALID_ARG;
    LinearParams p{};
    p.W = {static_cast<const uint8_t *>(a->w), static_cast<const uint8_t *>(a->w_scales),
           static_cast<const uint8_t *>(a->w_zeros), a->K, shift};
    p.x = static_cast<const uint16_t *>(a->x);
    p.out = static_cast<uint16_t *>(a->out);
    p.x_stride = a->x_stride;
    p.out_stride = a->out_stride;
    p.M = static_cast<int32_t>(a->M);
    p.N = a->N;
    p.divisor = int4 ? 1.0f : a->global_scale;
    p.stall = debug_stall_slots();
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    if (int4)
        return bf16 ? launch<kWInt4, true>(p, stream) : launch<kWInt4, false>(p, stream);
    return bf16 ? launch<kWNvfp4, true>(p, stream) : launch<kWNvfp4, false>(p, stream);
}
