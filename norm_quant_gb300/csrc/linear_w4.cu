// linear_w4.cu -- out[m, n] = sum_k x[m, k] W[n, k] for a few rows x and a
// matrix W in 4 bits (NVFP4, or integers with group scales).
//
// One CTA an SM; CTAs take equal, consecutive shares of the blocks of 16 rows.
// The consumer warps form groups: the warps of a group split k and add their
// fp32 sums in the order of the warps, and the groups take different blocks.
// The columns are laid out once for all of them.  Columns that do not fit at
// once are taken in rounds, for which the weights come from L2.
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
    int32_t round;  // columns at a time
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

template <int FMT, bool BF16>
__global__ void __launch_bounds__(32 * (kMaxConsumers<FMT> + 1), 1) linear_w4_kernel(const __grid_constant__ LinearParams p)
{
    using F = Format<FMT, BF16>;
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
            int b, panel, round, start, last, step, panels, rounds;
            __device__ bool next(int &at, int &lo, int &hi)
            {
                if (panel == panels) {
                    panel = 0;
                    b += step;
                    if (b >= last) {
                        b = start;
                        ++round;
                    }
                }
                if (round >= rounds || b >= last)
                    return false;
                at = panel++;
                lo = 16 * b;
                hi = 16 * b + 8;
                return true;
            }
        };
        produce<F, FMT, false>(Items{first + lane, 0, 0, first + lane, last, p.groups, p.panels, (p.M + p.round - 1) / p.round}, p.groups,
                        slots, bars, p.plan, p.W, p.maps, p.N,
                        blockIdx.x == 0 && p.stall >= 0 ? p.stall : INT64_MAX, lane);
        return;
    }
    const int group = warp / warps, j = warp - group * warps;
    Consumer<F, FMT, BF16> consumer(p.plan, p.W, failed, slots + group * depth * p.plan.bytes,
                                    bars + group * depth * kBarrierBytes, 0, j, lane);
    const uint32_t columns = slots + columns_at(p.plan, p.groups, p.panels);
    float *red = reinterpret_cast<float *>(smem + sums_at(p.plan, p.groups, p.panels)) + group * warps * 256;  // [2][warps][8 columns][16 rows]
    int turn = 0;
    for (int m0 = 0; m0 < p.M; m0 += p.round) {
        const int n = min(p.round, p.M - m0);
        if (m0 > 0)
            named_barrier_sync(1, 32 * consumers);  // the columns before have been read
        lay_out_strips<F, BF16>(columns, factors, [&](int c) { return p.x + (m0 + c) * p.x_stride; }, n, warp, consumers, p.W.K,
                                early(p.divisor), lane);
        named_barrier_sync(1, 32 * consumers);
        uint32_t swap;
        const uint32_t column = columns + column_at<F>(n, lane, swap), size = column_bytes<F>(n, 1);
        for (int b = first + group; b < last; b += p.groups) {
            float acc[4] = {};
            for (int panel = 0; panel < p.panels; ++panel) {
                consumer.wait();
                consumer.template take<kScaled<F, BF16>>(acc, panel, column + panel * p.plan.strips * size, size, swap,
                                                         smem_u32(factors + panel * p.plan.strips * kColumns));
            }
            float *set = red + (turn & 1) * warps * 128;
            store_sums(set + j * 128, acc, lane);
            named_barrier_sync(2 + group, 32 * warps);
            // the other set is written next, and this one only after another barrier
            if (j == turn % warps) {
                const int n0 = 16 * b;
                for (int i = lane; i < 16 * n; i += 32) {
                    float s = 0.0f;
                    for (int w = 0; w < warps; ++w)
                        s += set[w * 128 + i];
                    if (*failed)
                        s = __int_as_float(0x7FC00000);
                    if (FMT == kWNvfp4)  // scaled columns' factors hold the early part
                        s = s / (kScaled<F, BF16> ? 1.0f : early(p.divisor)) / late(p.divisor);
                    if (n0 + (i & 15) < p.N)
                        p.out[(m0 + (i >> 4)) * p.out_stride + n0 + (i & 15)] = narrow16<BF16>(s);
                }
            }
            ++turn;
        }
    }
}

template <int FMT, bool BF16>
moe_status launch_linear(LinearParams &p, moe_stream_t stream)
{
    using F = Format<FMT, BF16>;
    static SmemLimit limit;
    const int sms = sm_count(), strips = strips_of<F>(p.W.K), blocks = (p.N + 15) / 16;
    if (sms <= 0)
        return MOE_ERR_CUDA;
    // Few blocks: one group of as many warps as split k.  More: groups of up to 8, as many as there are warps.
    const int each = (blocks + sms - 1) / sms;
    const int warps = split_warps(strips, each < 2 ? 16 : 8);
    const auto bytes = [&](int round, int depth) {
        SlotPlan s = p.plan;
        s.depth = depth;
        return static_cast<size_t>(columns_at(s, p.groups, p.panels)) + column_bytes<F>(round, s.strips * p.panels);
    };
    // As many groups as let all columns (up to 8) fit beside two slots a group,
    // three of a single one, since a second round would read the weights again;
    // with one group, as many columns as fit.  Two strips a warp in a slot where
    // that fits too.  What is left holds more slots.
    const int most_groups = kMaxConsumers<FMT> / warps < each ? kMaxConsumers<FMT> / warps : each;
    p.round = p.M < kColumns ? p.M : kColumns;
    int least = 3;
    for (int m = strips >= 2 * warps ? 2 : 1; m > 0; --m) {
        p.panels = (strips + m * warps - 1) / (m * warps);
        p.plan = slot_plan<F, FMT>(warps, m * warps, 1, 0, p.W, p.maps);
        p.groups = most_groups < kMaxGroups ? most_groups : kMaxGroups;
        if (m > 1 && bytes(p.round, p.groups < 2 ? 3 : 2) > kSmemPerCta)
            continue;
        while (p.groups > 1 && bytes(p.round, 2) > kSmemPerCta)
            --p.groups;
        least = p.groups < 2 ? 3 : 2;
        break;
    }
    while (p.round > 0 && bytes(p.round, least) > kSmemPerCta)
        --p.round;
    if (p.round < 1)
        return MOE_ERR_UNSUPPORTED;
    p.plan.depth = least;
    while (p.plan.depth * p.groups < 16 && bytes(p.round, p.plan.depth + 1) <= kSmemPerCta)
        ++p.plan.depth;
    const size_t smem = bytes(p.round, p.plan.depth);
    int dev = 0;
    const auto kern = linear_w4_kernel<FMT, BF16>;
    if (cudaGetDevice(&dev) != cudaSuccess || ensure_dynamic_smem(kern, dev, static_cast<int>(smem), limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const moe_status st = make_maps<F, FMT>(p.maps, p.plan, p.W, p.N);
    if (st != MOE_OK)
        return st;
    return PdlLaunch(static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * (warps * p.groups + 1), smem, stream).run(kern, p);
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
        return bf16 ? launch_linear<kWInt4, true>(p, stream) : launch_linear<kWInt4, false>(p, stream);
    return bf16 ? launch_linear<kWNvfp4, true>(p, stream) : launch_linear<kWNvfp4, false>(p, stream);
}
