// layer.cu -- a whole expert layer for a few tokens, in two kernels.
//
//   gate_up  a[t, e] = w[t, e] act(W1[e] x[t]) (W3[e] x[t])   for every expert e that a token takes
//   down     out[t]  = sum_e W2[e] a[t, e] + shared[t] + residual[t]
//
// Both are bound by the weights of the experts taken, 3 H I elements each,
// which are read once for every part of up to 8 of an expert's tokens.  The
// router's weight w[t, e] is multiplied into a, so the second product sums over
// experts without a further step.
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


// Consumer warps of the first kernel.  With integers 16 warps, for 128 registers a thread:
// with 20 the steps of a strip do not fit unrolled, and an expert layer of H = 4096, I =
// 2048, E = 8, k = 2 takes 66 instead of 61 us for 32 tokens.
template <int FMT>
constexpr int kGateUpConsumers = FMT == kWInt4 ? 15 : kMaxConsumers<FMT>;

struct LayerParams {
    WeightMaps maps13, maps2;
    WeightView W13, W2;
    const float *w13_global, *w2_global;
    const uint16_t *x, *shared, *residual;
    uint16_t *out, *act;  // act: workspace, a row of whole strips for each pair, in the order of the list
    const int32_t *ids;
    const void *weights;
    int32_t *status;
    int64_t x_stride;
    int32_t T, H, I, E, k, weight_dtype, gelu;
    // launch plans of the two kernels; most: tokens of a part
    SlotPlan gate_up, down;
    int32_t gate_up_panels, gate_up_groups, gate_up_most;
    int32_t down_panels, down_groups, down_most;
    int64_t stall;  // test hook: CTA 0 of the first kernel fills no more than this many slots (-1: off)
};

// The experts taken, in ascending order, and the tokens of each.  A pair is
// an expert and one of its tokens.  An expert with more tokens than `most`
// fit at once is listed in parts of nearly equal size, one after the other.
struct Lists {
    uint32_t *mask;    // [E][2]: a bit for each token
    int32_t *expert;   // [parts]
    int32_t *first;    // [parts + 1]: the first pair of each
    float *weight;     // [pairs]: the router's; in the second kernel [parts]: w2's global scale
    uint8_t *token;    // [pairs]
    int32_t *scratch;  // [32]
    int32_t parts;
};

// Most parts of up to `most` tokens that `slots` slots on E experts make: one
// for each expert taken, and another for every `most` pairs at most.
__host__ __device__ inline int most_parts(int E, int slots, int most)
{
    const int parts = (E < slots ? E : slots) + slots / most;
    return parts < slots ? parts : slots;
}

__host__ __device__ inline size_t lists_bytes(int E, int slots, int most)
{
    return (8 * static_cast<size_t>(E) + 4 * (2 * static_cast<size_t>(most_parts(E, slots, most)) + 1) +
            5 * static_cast<size_t>(slots) + 4 * 32 + 15) / 16 * 16;
}

__device__ __forceinline__ float load_weight(const LayerParams &p, int64_t i)
{
    if (p.weight_dtype == MOE_WEIGHTS_FP32)
        return static_cast<const float *>(p.weights)[i];
    const uint16_t v = static_cast<const uint16_t *>(p.weights)[i];
    return p.weight_dtype == MOE_WEIGHTS_BF16 ? widen16<true>(v) : widen16<false>(v);
}

// All threads of the CTA; `warps` is at most 32.  Every loop is short or starts with a
// load: unrolled they only make the kernels' start longer (0.5 us of 10 with a small layer).
__device__ void build_lists(Lists &L, const LayerParams &p, uint8_t *smem, int most, bool want_weights)
{
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
    const int slots = p.T * p.k, room = most_parts(p.E, slots, most);
    L.mask = reinterpret_cast<uint32_t *>(smem);
    L.expert = reinterpret_cast<int32_t *>(L.mask + 2 * p.E);
    L.first = L.expert + room;
    L.scratch = L.first + room + 1;
    L.weight = reinterpret_cast<float *>(L.scratch + 32);
    L.token = reinterpret_cast<uint8_t *>(L.weight + slots);
#pragma unroll 1
    for (int i = tid; i < 2 * p.E; i += threads)
        L.mask[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < slots; i += threads) {
        const int e = p.ids[i], t = i / p.k;
        if (e >= 0 && e < p.E)
            atomicOr(&L.mask[2 * e + (t >> 5)], 1u << (t & 31));
        else if (e != -1 && p.status)
            atomicCAS(p.status, 0, MOE_ERR_INVALID_EXPERT);
    }
    __syncthreads();
    // number the parts and their pairs: a scan of (parts, tokens) over the experts, packed in one word
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += threads) {
        const int e = e0 + tid;
        const uint32_t m0 = e < p.E ? L.mask[2 * e] : 0u, m1 = e < p.E ? L.mask[2 * e + 1] : 0u;
        const int tokens = __popc(m0) + __popc(m1), parts = (tokens + most - 1) / most;
        const int own = (parts << 16) + tokens;
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
#pragma unroll 1
        for (int w = 0; w < warps; ++w) {
            const int v = L.scratch[w];
            before += w < warp ? v : 0;
            base += v;
        }
        before += scan - own;
#pragma unroll 1
        for (int i = 0; i < parts; ++i) {
            L.expert[(before >> 16) + i] = e;
            L.first[(before >> 16) + i] = (before & 0xFFFF) + tokens * i / parts;
        }
        int at = before & 0xFFFF;
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
            for (uint32_t m = h ? m1 : m0; m; m &= m - 1)
                L.token[at++] = static_cast<uint8_t>(32 * h + __ffs(m) - 1);
        __syncthreads();
    }
    L.parts = base >> 16;
    const int pairs = base & 0xFFFF;
    if (tid == 0)
        L.first[L.parts] = pairs;
    __syncthreads();
    if (!want_weights) {
#pragma unroll 1
        for (int a = tid; a < L.parts; a += threads)
            L.weight[a] = p.w2_global ? p.w2_global[L.expert[a]] : 1.0f;
    } else {
        for (int a = warp; a < L.parts; a += warps) {
            const int e = L.expert[a];
            for (int q = L.first[a] + lane; q < L.first[a + 1]; q += 32) {
                const int t = L.token[q];
                float w = 0.0f;
#pragma unroll 1
                for (int j = 0; j < p.k; ++j)
                    if (p.ids[t * p.k + j] == e)
                        w += load_weight(p, t * p.k + j);
                L.weight[q] = w;
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float activate(float g, bool gelu)
{
    if (gelu)
        return 0.5f * g * (1.0f + tanhf(0.7978845608f * (g + 0.044715f * g * g * g)));
    // Two units in the last place at most, far below the 16-bit rounding that follows; the quotient of a huge
    // divisor, 0 here, is below 2^-119.
    return __fdividef(g, 1.0f + expf(-g));
}

__device__ __forceinline__ float not_a_number() { return __int_as_float(0x7FC00000); }

__host__ __device__ inline uint32_t round16(uint32_t n) { return (n + 15) / 16 * 16; }

// Shared memory of the first kernel: slots, barriers and a flag, the columns'
// factors, two sets of sums a group, lists, columns.
__host__ __device__ inline uint32_t bars_at(const SlotPlan &s, int groups) { return groups * s.depth * s.bytes; }
__host__ __device__ inline uint32_t factors_at(const SlotPlan &s, int groups)
{
    return round16(bars_at(s, groups) + groups * s.depth * kBarrierBytes + 4);
}
__host__ __device__ inline uint32_t sums_at(const SlotPlan &s, int groups, int panels)
{
    return factors_at(s, groups) + panels * s.strips * kColumns * 4;
}
__host__ __device__ inline uint32_t gate_up_lists_at(const SlotPlan &s, int groups, int panels)
{
    return sums_at(s, groups, panels) + groups * s.warps * 1024;
}

// The eight values from 8 piece on of a pair's row of the workspace, whose
// strips lie in the order in which the second kernel takes them.  Neighbouring
// pairs' pieces are exchanged as those of neighbouring columns are.
template <int FMT, bool BF16>
__device__ __forceinline__ uint16_t *act_piece(const LayerParams &p, int pair, int piece)
{
    using F = Format<FMT, BF16, true>;
    constexpr int kPieces = F::kStripK / 8;
    return p.act + (static_cast<int64_t>(pair) * strips_of<F>(p.I) + piece / kPieces) * F::kStripK +
           piece_at<F>(piece % kPieces, pair & 1) / 2;
}

// The first kernel.  A unit is (part of an expert's tokens, 8 values of its
// inner dimension): the rows of W1 and of W3 for these 8 fill one 16-row tile,
// so that a lane ends up with both factors of the same value.  One CTA an SM;
// CTAs take equal, consecutive shares of the units.  The consumer warps form
// groups: the warps of a group split k, and the groups take different units of
// one part, whose columns are laid out once for all of them.
// 16-bit weights are bound by HBM: H = 7168, I = 2048, E = 256, k = 8, both kernels,
// 1 token 108 us, 8 tokens 725 us, 0.96 and more of the copy rate.  4-bit weights are
// bound by the instructions that widen them, about 370 a warp for 4096 weights
// with what belongs to a unit: 16 tokens, NVFP4, 212 us of 374 for both kernels; 8
// tokens, H = 4096, I = 8192, E = 8, integers, 61 of 103.  Groups of 3 to 6 instead of 8 warps
// are 2 % faster to 10 % slower with NVFP4, and with integers those of 4 or 5 are the fastest.
template <int FMT, bool BF16>
__global__ void __launch_bounds__(32 * (kGateUpConsumers<FMT> + 1), 1) gate_up_kernel(const __grid_constant__ LayerParams p)
{
    using F = Format<FMT, BF16>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const SlotPlan &plan = p.gate_up;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = plan.warps, depth = plan.depth;
    const int groups = p.gate_up_groups, consumers = warps * groups, panels = p.gate_up_panels;
    const uint32_t slots = smem_u32(smem), bars = slots + bars_at(plan, groups);
    volatile int32_t *failed = reinterpret_cast<volatile int32_t *>(smem + bars_at(plan, groups) + groups * depth * kBarrierBytes);
    float *factors = reinterpret_cast<float *>(smem + factors_at(plan, groups));  // [panels * warps][8]
    const uint32_t lists_at = gate_up_lists_at(plan, groups, panels);
    if (threadIdx.x == 0) {
        for (int i = 0; i < groups * depth; ++i) {
            mbar_init(bars + i * kBarrierBytes, fill_arrivals(p.maps13));
            mbar_init(bars + i * kBarrierBytes + 8, warps);
        }
        *failed = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    Lists L;
    build_lists(L, p, smem + lists_at, p.gate_up_most, true);

    const int slabs = p.I / 8;
    const int64_t all = static_cast<int64_t>(L.parts) * slabs;
    const int64_t from = all * blockIdx.x / gridDim.x;
    int left = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x - from);
    int a = static_cast<int>(from / slabs), slab0 = static_cast<int>(from % slabs);
    if (warp == consumers) {  // the producer
        struct Items {  // the slots of one group
            const int32_t *expert;
            int a, slab, end, panel, left, group, groups, panels, slabs, I;
            __device__ bool next(int &at, int &lo, int &hi)
            {
                if (panel == panels) {
                    panel = 0;
                    slab += groups;
                }
                while (slab >= end) {  // to the next part
                    if (left <= 0)
                        return false;
                    ++a;
                    slab = group;
                    end = min(slabs, left);
                    left -= end;
                }
                at = panel++;
                lo = expert[a] * 2 * I + 8 * slab;
                hi = lo + I;
                return true;
            }
        };
        const int end = min(slabs, slab0 + left);
        produce<F, FMT, false, false>(Items{L.expert, a, slab0 + lane, end, 0, left - (end - slab0), lane, groups, panels, slabs, p.I},
                        groups, slots, bars, plan, p.W13, p.maps13, p.E * 2 * p.I,
                        blockIdx.x == 0 && p.stall >= 0 ? p.stall : INT64_MAX, lane);
        return;
    }
    const int group = warp / warps, j = warp - group * warps;
    Consumer<F, FMT, BF16> consumer(plan, p.W13, failed, slots + group * depth * plan.bytes,
                                    bars + group * depth * kBarrierBytes, 0, j, lane);
    const uint32_t columns = slots + lists_at + static_cast<uint32_t>(lists_bytes(p.E, p.T * p.k, p.gate_up_most));
    float *red = reinterpret_cast<float *>(smem + sums_at(plan, groups, panels)) + group * warps * 256;  // [2][warps][8 columns][16 rows]
    int turn = 0;
    for (bool later = false; left > 0; ++a, slab0 = 0, later = true) {
        const int end = min(slabs, slab0 + left), first = L.first[a], n = L.first[a + 1] - first;
        left -= end - slab0;
        const float div = FMT == kWNvfp4 && p.w13_global ? p.w13_global[L.expert[a]] : 1.0f;
        const float back = 1.0f / (kScaled<F, BF16> ? 1.0f : early(div));  // otherwise the columns' factors hold it
        if (later)
            named_barrier_sync(1, 32 * consumers);  // the columns before have been read
        lay_out_strips<F, BF16>(columns, factors, [&](int c) { return p.x + L.token[first + c] * p.x_stride; }, n, warp, consumers,
                                p.H, early(div), lane);
        named_barrier_sync(1, 32 * consumers);
        uint32_t swap;
        const uint32_t column = columns + column_at<F>(n, lane, swap), size = column_bytes<F>(n, 1);
        for (int slab = slab0 + group; slab < end; slab += groups) {
            float acc[4] = {};
            for (int panel = 0; panel < panels; ++panel) {
                consumer.wait();
                consumer.template take<kScaled<F, BF16>>(acc, panel, column + panel * plan.strips * size, size, swap,
                                                         smem_u32(factors + panel * plan.strips * kColumns));
            }
            float *set = red + (turn & 1) * warps * 128;
            store_sums(set + j * 128, acc, lane);
            named_barrier_sync(2 + group, 32 * warps);
            // the other set of sums is written next, and this one only after another barrier
            if (j == turn % warps) {
                if (*failed && lane == 0 && p.status)
                    atomicCAS(p.status, 0, MOE_ERR_DEVICE_TIMEOUT);
                for (int i = lane; i < 8 * n; i += 32) {
                    const int r = i & 7, c = i >> 3;
                    const float *sum = set + c * 16 + r;
                    float gate = 0.0f, up = 0.0f;
                    for (int w = 0; w < warps; ++w) {
                        gate += sum[w * 128];
                        up += sum[w * 128 + 8];
                    }
                    if constexpr (FMT == kWNvfp4) {
                        gate *= back;
                        up *= back;
                        if (div < 1.0f) {
                            gate /= div;
                            up /= div;
                        }
                    }
                    if (*failed)
                        gate = not_a_number();
                    // Rounded to the I/O type, as the second product's operand: 32 bits would double its instructions.
                    // Against 64 bits the layer is then off by 1.8e-3 to 2.4e-3 in bf16, where the rounding of out
                    // alone makes 1.7e-3 (fp16: 2.1e-4 to 3.0e-4 and 2.1e-4).
                    act_piece<FMT, BF16>(p, first + c, slab)[element_at<Format<FMT, BF16, true>>(r)] = narrow16<BF16>(
                        activate(gate, p.gelu) * up * L.weight[first + c]);
                }
                if (slab == slabs - 1) {  // zeros from I to the end of the last strip
                    const int more = strips_of<Format<FMT, BF16, true>>(p.I) * (Format<FMT, BF16, true>::kStripK / 8) - slabs;
                    for (int i = lane; i < 8 * more * n; i += 32)
                        act_piece<FMT, BF16>(p, first + i / (8 * more), slabs + i / 8 % more)[i & 7] = 0;
                }
            }
            ++turn;
        }
    }
}

// The second kernel.  One CTA an SM; CTAs take equal, consecutive shares of
// the blocks of 16 rows, as many of them in a pass as a slot has tiles.  The
// panels of all parts go by, and the groups of consumers take turns at them.  A
// group has `warps` warps for every tile, which split the panel's k.  A slot
// brings the panel's columns with it, which the first kernel has left in the
// order of the matrix instruction.  Each warp adds its sums to its own [T, 16]
// part of the result in shared memory, and the parts of a tile are added in the
// order of the warps.
// Its columns are of the I/O type, since the largest value of a strip is known
// to no single CTA of the first kernel: NVFP4's codes are widened to bf16, which
// takes 540 instructions a warp for 4096 weights with all that belongs to a part.  16
// tokens, NVFP4: 160 us of 374 for both kernels; with fp16 I/O 16-bit weights reach 0.95 of
// the copy rate (64 tokens, H = 4096, I = 1024, E = 128, k = 8: 493 us for both).
__host__ __device__ inline uint32_t results_at(const SlotPlan &s, int groups)
{
    return round16(bars_at(s, groups) + groups * s.depth * kBarrierBytes + 4);
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(32 * (kMaxConsumers<FMT> + 1), 1) down_kernel(const __grid_constant__ LayerParams p)
{
    using F = Format<FMT, BF16, true>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const SlotPlan &plan = p.down;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int warps = plan.warps, depth = plan.depth, groups = p.down_groups, each = warps * plan.tiles, consumers = each * groups;
    const int panels = p.down_panels, per_warp = p.T * 16;
    const uint32_t slots = smem_u32(smem), bars = slots + bars_at(plan, groups);
    volatile int32_t *failed = reinterpret_cast<volatile int32_t *>(smem + bars_at(plan, groups) + groups * depth * kBarrierBytes);
    float *results = reinterpret_cast<float *>(smem + results_at(plan, groups));  // [consumers][T][16]
    const int blocks = (p.H + 15) / 16, strips = strips_of<F>(p.I);
    const int first_block = static_cast<int>(static_cast<int64_t>(blocks) * blockIdx.x / gridDim.x);
    const int last_block = static_cast<int>(static_cast<int64_t>(blocks) * (blockIdx.x + 1) / gridDim.x);
    if (tid == 0) {
        for (int i = 0; i < groups * depth; ++i) {
            mbar_init(bars + i * kBarrierBytes, fill_arrivals(p.maps2));
            mbar_init(bars + i * kBarrierBytes + 8, each);
        }
        *failed = 0;
        fence_mbar_init();
    }
    // the ids were complete before the first kernel of this call started, and so were the weights
    Lists L;
    build_lists(L, p, smem + results_at(plan, groups) + consumers * per_warp * sizeof(float), p.down_most, false);

    // The slots of one group: every groups-th of the panels of the parts of the passes.
    struct Items {
        const LayerParams &p;
        const Lists &L;
        int a, panel, b0, last, strips;
        __device__ bool settle()  // false at the end
        {
            while (panel >= p.down_panels) {
                panel -= p.down_panels;
                if (++a == L.parts) {
                    a = 0;
                    b0 += p.down.tiles;
                }
            }
            return b0 < last;
        }
        int of_a, of_panel;  // the item that next gave
        __device__ bool next(int &at, int &lo, int &hi)
        {
            if (!settle())
                return false;
            at = of_panel = panel;
            of_a = a;
            lo = L.expert[a] * p.H + 16 * b0;
            hi = lo + 8;
            panel += p.down_groups;
            return true;
        }
        __device__ int here() const { return min(p.down.strips, strips - of_panel * p.down.strips); }
        __device__ uint32_t column_bytes() const { return nqg::column_bytes<F>(L.first[of_a + 1] - L.first[of_a], here()); }
        __device__ void columns(uint32_t slot, uint32_t bar) const
        {
            const int first = L.first[of_a], n = L.first[of_a + 1] - first;
            for (int c = 0; c < n; ++c)
                bulk_g2s(slot + p.down.columns_at + c * nqg::column_bytes<F>(1, p.down.strips),
                         p.act + (static_cast<int64_t>(first + c) * strips + of_panel * p.down.strips) * F::kStripK,
                         nqg::column_bytes<F>(1, here()), bar);
        }
    };
    if (warp == consumers) {  // the producer
        if (L.parts > 0)
            produce<F, FMT, true, true>(Items{p, L, 0, lane, first_block, last_block, strips, 0, 0}, groups, slots, bars, plan,
                                  p.W2, p.maps2, p.E * p.H, INT64_MAX, lane);
        return;
    }
    const int group = warp / each, tile = (warp - group * each) / warps, j = warp % warps;
    float *mine = results + warp * per_warp;
    grid_dependency_wait();
    allow_dependent_launch();
    Consumer<F, FMT, BF16> consumer(plan, p.W2, failed, slots + group * depth * plan.bytes,
                                    bars + group * depth * kBarrierBytes, tile, j, lane);
    int panel = group;  // the group's next one, from the part in turn on
    for (int b0 = first_block; b0 < last_block; b0 += plan.tiles) {
        for (int i = lane; i < per_warp; i += 32)
            mine[i] = 0.0f;
        __syncwarp();
        for (int a = 0; a < L.parts; ++a, panel -= panels) {
            if (panel >= panels)
                continue;
            const int first = L.first[a], n = L.first[a + 1] - first;
            uint32_t swap;
            const uint32_t column = plan.columns_at + column_at<F>(n, lane, swap, first & 1, column_bytes<F>(1, plan.strips));
            float acc[4] = {};
            for (; panel < panels; panel += groups) {
                consumer.wait();
                consumer.template take<false>(acc, panel, consumer.slot + column, column_bytes<F>(1, 1), swap, 0);
            }
            if constexpr (FMT == kWNvfp4) {
                const float div = L.weight[a], factor = F::kPost / early(div);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] *= factor;
                if (div < 1.0f)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[i] /= div;
            }
            // the lane's sums are of columns 2 t and 2 t + 1
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (2 * t + i < n) {
                    float *const to = mine + L.token[first + 2 * t + i] * 16 + g;
                    to[0] += acc[i];
                    to[8] += acc[2 + i];
                }
        }
        named_barrier_sync(1, 32 * consumers);
        if (*failed && tid == 0 && p.status)
            atomicCAS(p.status, 0, MOE_ERR_DEVICE_TIMEOUT);
        const int width = 16 * plan.tiles;
        for (int i = tid; i < p.T * width; i += 32 * consumers) {
            const int token = i / width, r = i - token * width, n = 16 * b0 + r;
            if (n >= min(16 * last_block, p.H))
                continue;
            float v = 0.0f;
            for (int q = 0; q < groups; ++q)
                for (int w = 0; w < warps; ++w)
                    v += results[(q * each + (r >> 4) * warps + w) * per_warp + token * 16 + (r & 15)];
            const int64_t o = static_cast<int64_t>(token) * p.H + n;
            if (p.shared)
                v += widen16<BF16>(p.shared[o]);
            if (p.residual)
                v += widen16<BF16>(p.residual[o]);
            p.out[o] = narrow16<BF16>(*failed ? not_a_number() : v);
        }
        named_barrier_sync(1, 32 * consumers);  // the parts have been read
    }
}

template <int FMT, bool BF16>
moe_status launch_layer(LayerParams &p, moe_stream_t stream)
{
    using F = Format<FMT, BF16>;
    static SmemLimit gate_limit, down_limit;
    int dev = 0;
    const int sms = sm_count();
    if (cudaGetDevice(&dev) != cudaSuccess || sms <= 0)
        return MOE_ERR_CUDA;
    const int slots = p.T * p.k;
    // Tokens of a part: twice what an expert that is taken has on average if ids
    // are uniform, at least 2.  Room for columns is taken from the slots in
    // flight, and the few experts with more tokens are read again, from L2, and
    // widened again.  Ids that are not uniform at all pay for it: 64 tokens on one
    // of E = 256 experts (k = 1, H = 4096, I = 2048) make 22 parts and take 120 us,
    // 8 tokens 29; with NVFP4 99 and 24.
    const double taken = p.E * (1.0 - std::pow(1.0 - static_cast<double>(p.k < p.E ? p.k : p.E) / p.E, p.T));
    int most = static_cast<int>(std::ceil(2.0 * slots / (taken < 1.0 ? 1.0 : taken)));
    most = most < 2 ? 2 : most > kColumns ? kColumns : most;
    most = most < p.T ? most : p.T;

    // First kernel.  Few units: one group of as many warps as split k.  More: groups of up to 8 (5 of
    // 15 with integers), as many as there are warps.
    const int strips = strips_of<F>(p.H);
    const int64_t units = static_cast<int64_t>(p.E < slots ? p.E : slots) * (p.I / 8);
    const int64_t each = (units + sms - 1) / sms;
    constexpr int kConsumers = kGateUpConsumers<FMT>;
    const int warps = split_warps(strips, each >= 2 ? (kConsumers < 16 ? 5 : 8) : kConsumers < 16 ? kConsumers : 16);
    const auto gate_bytes = [&](int columns, int depth) {
        SlotPlan s = p.gate_up;
        s.depth = depth;
        return gate_up_lists_at(s, p.gate_up_groups, p.gate_up_panels) + lists_bytes(p.E, slots, columns) +
               column_bytes<F>(columns, s.strips * p.gate_up_panels);
    };
    // As many groups as let the columns of a part fit beside two slots a group,
    // three of a single one.  Two strips a warp in a slot where that fits too.
    // What is left holds more slots.
    const int64_t most_groups = kConsumers / warps < each ? kConsumers / warps : each;
    p.gate_up_most = most;
    int least = 3;
    for (int m = strips >= 2 * warps ? 2 : 1; m > 0; --m) {
        p.gate_up_panels = (strips + m * warps - 1) / (m * warps);
        p.gate_up = slot_plan<F, FMT>(warps, m * warps, 1, true, 0, p.W13, p.maps13);
        p.gate_up_groups = most_groups < kMaxGroups ? static_cast<int>(most_groups) : kMaxGroups;
        if (m > 1 && gate_bytes(most, p.gate_up_groups < 2 ? 3 : 2) > kSmemPerCta)
            continue;
        while (p.gate_up_groups > 1 && gate_bytes(most, 2) > kSmemPerCta)
            --p.gate_up_groups;
        least = p.gate_up_groups < 2 ? 3 : 2;
        break;
    }
    while (p.gate_up_most > 0 && gate_bytes(p.gate_up_most, least) > kSmemPerCta)
        --p.gate_up_most;
    if (p.gate_up_most < 1)
        return MOE_ERR_UNSUPPORTED;
    p.gate_up.depth = least;
    while (p.gate_up.depth * p.gate_up_groups < 16 && gate_bytes(p.gate_up_most, p.gate_up.depth + 1) <= kSmemPerCta)
        ++p.gate_up.depth;
    const size_t gate = gate_bytes(p.gate_up_most, p.gate_up.depth);

    // Second kernel: the blocks of a CTA are the tiles of a slot, up to 3; panels
    // of up to 8 strips, two for a warp where that leaves enough warps; as many
    // groups as fit with two slots each, or fewer tiles.
    using F2 = Format<FMT, BF16, true>;
    const int inner = strips_of<F2>(p.I), blocks = (p.H + 15) / 16, per_cta = (blocks + sms - 1) / sms;
    const int panel_strips = split_warps(inner, 8);
    p.down_panels = (inner + panel_strips - 1) / panel_strips;
    p.down_most = most;
    const auto down_bytes = [&](int depth) {
        SlotPlan s = p.down;
        s.depth = depth;
        return results_at(s, p.down_groups) + static_cast<size_t>(p.down_groups) * s.warps * s.tiles * p.T * 64 +
               lists_bytes(p.E, slots, p.down_most);
    };
    for (int tiles = per_cta < 3 ? per_cta : 3;; --tiles) {
        const int down_warps = panel_strips * tiles > 12 ? (panel_strips + 1) / 2 : panel_strips;
        p.down = slot_plan<F2, FMT>(down_warps, panel_strips, tiles, false, column_bytes<F2>(p.down_most, panel_strips), p.W2, p.maps2);
        p.down_groups = kMaxConsumers<FMT> / (down_warps * tiles) < kMaxGroups ? kMaxConsumers<FMT> / (down_warps * tiles) : kMaxGroups;
        while (p.down_groups > 1 && down_bytes(2) > kSmemPerCta)
            --p.down_groups;
        if (down_bytes(2) <= kSmemPerCta)
            break;
        if (tiles == 1)
            return MOE_ERR_UNSUPPORTED;
    }
    p.down.depth = 2;
    while (p.down.depth * p.down_groups < 16 && down_bytes(p.down.depth + 1) <= kSmemPerCta)
        ++p.down.depth;
    const size_t down = down_bytes(p.down.depth);

    const auto gate_up = gate_up_kernel<FMT, BF16>;
    const auto down_k = down_kernel<FMT, BF16>;
    if (ensure_dynamic_smem(gate_up, dev, static_cast<int>(gate), gate_limit) != cudaSuccess ||
        ensure_dynamic_smem(down_k, dev, static_cast<int>(down), down_limit) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    moe_status st = make_maps<F, FMT>(p.maps13, p.gate_up, p.W13, static_cast<int64_t>(p.E) * 2 * p.I);
    if (st == MOE_OK)
        st = make_maps<F2, FMT>(p.maps2, p.down, p.W2, static_cast<int64_t>(p.E) * p.H);
    if (st == MOE_OK)
        st = PdlLaunch(static_cast<unsigned>(units < sms ? units : sms), 32 * (warps * p.gate_up_groups + 1), gate, stream)
                 .run(gate_up, p);
    if (st == MOE_OK)
        st = PdlLaunch(static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * (p.down.warps * p.down.tiles * p.down_groups + 1),
                       down, stream)
                 .run(down_k, p);
    return st;
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
    // a row of I 16-bit values for every slot, in whole strips of 256
    *bytes = static_cast<size_t>(T) * top_k * ((I + 255) / 256) * 512;
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
    if (a->T > MOE_FEW_TOKENS || a->E > MOE_LAYER_MAX_EXPERTS || a->top_k > MOE_MAX_TOP_K || a->H > MOE_FEW_MAX_K ||
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
    if (!a->workspace)
        return MOE_ERR_WORKSPACE;
    if (!aligned16(a->workspace))
        return MOE_ERR_INVALID_ARG;
    if (a->workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    const auto u8 = [](const void *q) { return static_cast<const uint8_t *>(q); };
    const auto u16 = [](const void *q) { return static_cast<const uint16_t *>(q); };
    LayerParams p{};
    p.W13 = {u8(a->w13), u8(a->w13_scales), u8(a->w13_zeros), a->H, shift};
    p.W2 = {u8(a->w2), u8(a->w2_scales), u8(a->w2_zeros), a->I, shift};
    p.w13_global = a->w13_global;
    p.w2_global = a->w2_global;
    p.x = u16(a->x);
    p.shared = u16(a->shared_out);
    p.residual = u16(a->residual);
    p.out = static_cast<uint16_t *>(a->out);
    p.act = static_cast<uint16_t *>(a->workspace);
    p.ids = a->topk_ids;
    p.weights = a->router_weights;
    p.status = a->status;
    p.x_stride = a->x_stride;
    p.T = static_cast<int32_t>(a->T);
    p.H = a->H;
    p.I = a->I;
    p.E = a->E;
    p.k = a->top_k;
    p.weight_dtype = a->weight_dtype;
    p.gelu = a->activation == MOE_ACT_GELU_TANH;
    p.stall = debug_stall_slots();
    const bool bf16 = a->io_dtype == MOE_IO_BF16;
    if (int4)
        return bf16 ? launch_layer<kWInt4, true>(p, stream) : launch_layer<kWInt4, false>(p, stream);
    if (nvfp4)
        return bf16 ? launch_layer<kWNvfp4, true>(p, stream) : launch_layer<kWNvfp4, false>(p, stream);
    return bf16 ? launch_layer<kW16, true>(p, stream) : launch_layer<kW16, false>(p, stream);
}
