// block_product.cu -- products of rows that are grouped by expert, on the
// tensor cores of pairs of CTAs (tcgen05, cta_group::2).
//
// The four products (block.h) are one kernel over tiles of 256 x N values:
//
//   product   the 256 of a tile         its N                    contraction
//   forward   features of W[e]          up to 256 rows of e      K, in lines of both operands
//   gated     128 of W1[e] and of W3[e] up to 256 rows of e      K, the same
//   input     columns of W[e]           up to 256 rows of e      rows of W[e] (an operand across)
//   weight    columns of Y              columns of X             e's rows (both across)
//
// Rows are the N side because N comes in steps of 32: a group's rows are spread over as few tiles as hold them,
// all of the same N, so that 128 rows an expert cost 128 to 160 columns and not 256.
//
// Each CTA of a pair holds 128 of the 256 and half of the N in shared memory (32 KB for 64 of the contraction at N =
// 256, six such stages), which is what the matrix instruction of a pair wants: 64 bytes a cycle and SM instead of the 96 that a
// 128 x 256 tile alone would take from L2.  Sums are in tensor memory, in two buffers of 256 columns, so that one
// tile is written out while the next is multiplied.  Warps: 0 copies (TMA), 1 issues matrix instructions (in the
// pair's first CTA, for both), 4 to 11 write results.
//
// What bounds it: with many rows an expert the matrix instruction (R = 8192, K = 4096, N = 8192, bf16: forward 287 us, 1918
// TFLOP/s, gated 283, rows' gradient 290, weights' gradient 287, where the power limit holds cuBLAS at 271; the tensor pipe is active
// 93 % of the time at K = N = 4096), with few the weights' bytes (gated, R = 32768, H = 7168, I = 2048, E = 256: 14.2 GB in 2.12 ms,
// 6.7 TB/s), between the two the operands' way from L2 (R = 32768, K = 1024, N = 4096, E = 128: 255 us, some 13 TB/s out of L2).
//
// CTAs stay (one pair for two SMs) and take every P-th tile.  Within an expert, blocks of 8 tiles of one side pass along
// the other, so that the pairs at work share their operands in L2.
//
// Few tiles with a long contraction leave most SMs idle.  There, 2 to 4 pairs form a cluster and share a tile's contraction:
// each makes sums of its part, sends them to the pair that writes their columns (chunks of columns in turns), through
// distributed shared memory, and that one adds them up in the shares' order.
#include <cstdint>
#include <cuda_runtime.h>

#include "block.h"
#include "block_math.cuh"
#include "ring_place.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace nqg {
namespace {

constexpr int kWriters = 8;                 // writing warps: two for each 32 lanes of tensor memory, which take chunks of 32 columns in turns
constexpr int kThreads = 128 + 32 * kWriters;
constexpr int kStages = 6;
constexpr int kStep = 64;                   // elements of the contraction a stage holds: a line of 128 bytes
constexpr int kLine = 2 * kStep;
constexpr int kSide = 128;                  // rows of an operand a CTA holds at most
constexpr int kOperand = kSide * kLine;
constexpr int kStage = 2 * kOperand;
constexpr int kChunk = 64 * kLine;          // 64 rows of an operand across
constexpr int kMaxN = 256;
constexpr int kRowBoxes = 4;
constexpr int kEndBoxes = 9;                // 1, 2, 3, 4, 8, 12, 16, 32 and 48 rows: the digits of fewer than 64 to the base of 4
constexpr int kPitch = 144;                 // bytes from row to row of a staging: 16 more than a line, so that eight rows meet no bank twice
constexpr int kBlock = 8;                   // tiles of one side that pass along the other together
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kStepLimitNs = 4000;     // a step takes 0.15 to 0.31 us

// How long a wait may last that ends only when so many steps have been made.
__device__ __forceinline__ uint64_t wait_limit(int64_t steps) { return kWaitLimitNs + static_cast<uint64_t>(steps) * kStepLimitNs; }

// b: of rows in boxes of 16, 32, 64 and 128.
template <int KIND>
struct Maps {
    CUtensorMap a, b[kRowBoxes];
};

// a, b: of both operands' rows in boxes of 64; end_*: of 64 columns of fewer rows, those at an expert's end.
template <>
struct Maps<kWeight> {
    CUtensorMap a, b[1], end_a[kEndBoxes], end_b[kEndBoxes];
};

struct Params {
    int64_t n_rows;
    int32_t E, width, out_width;
    int32_t fold;                              // Product::fold; each step of the contraction is then made twice, once for each part
    int32_t m_tiles, n_tiles, n_columns;       // n_*: the weights' gradient's N side
    int32_t cap;                               // columns of a tile at most
    int32_t shares;                            // pairs that share a tile's contraction
    int32_t wide_a, wide_b;                    // an operand across comes in boxes of 128 columns (two chunks), not 64
    const int32_t *offsets;
    uint8_t *out, *gate_up;
    int64_t out_stride, gate_up_stride;        // elements
    int32_t *status;
    int32_t fp32_out;
    int64_t stall;
};

// Shared memory.
struct Layout {
    static constexpr int staging = kStages * kStage;  // 32 lines for two writing warps, or 16 where sums are exchanged
    static constexpr int exchange = staging + kWriters / 2 * 16 * kPitch;  // gated: 2 KB a writing warp
    static constexpr int bars = exchange + kWriters * 2048;
    static constexpr int full = bars, empty = full + 8 * kStages, sums_full = empty + 8 * kStages, sums_empty = sums_full + 16,
                         done = sums_empty + 16, tmem = done + 8, first = tmem + 8;
    static int bytes(int E) { return first + 2 * 4 * (E + 1); }
};
static_assert(kWriters * 2048 >= kWriters / 2 * 16 * kPitch, "stagings of 32 lines reach into the room of the exchange");
static_assert(Layout::first + 2 * 4 * (MOE_LAYER_MAX_EXPERTS + 1) <= 232448, "shared memory of a CTA");

struct Tile {
    int e;
    int64_t row;     // first row
    int32_t rows;    // rows of the tile (N side), or of the expert (weights' gradient)
    int32_t n;       // columns of the matrix instruction
    int32_t m0, n0;  // first of the 256, first column (weights' gradient)
    int32_t steps;
    int32_t begin, end;  // this pair's

    // The first step of share i of n.
    __device__ int32_t first_of(int i, int n) const { return static_cast<int32_t>(static_cast<int64_t>(steps) * i / n); }

    // Whether a step of the weights' gradient takes the last of the expert's rows and there are not 64 of them.
    __device__ bool ends(int k, int32_t fold) const { return rows % kStep != 0 && k >= steps - (fold ? 2 : 1); }
};

template <int KIND>
struct Schedule {
    const Params &p;
    const int32_t *first, *tile0;  // rows and (not for the weights' gradient) tiles of rows before each expert
    int share, shares;             // this pair's part of the contraction
    uint32_t total;  // below 2^31

    __device__ Schedule(const Params &q, const int32_t *f, const int32_t *t, int i, int n) : p(q), first(f), tile0(t), share(i), shares(n)
    {
        total = static_cast<uint32_t>(KIND == kWeight ? p.E * p.n_tiles : tile0[p.E]) * p.m_tiles;
    }

    __device__ Tile at(uint32_t q) const
    {
        Tile t;
        const uint32_t m_tiles = static_cast<uint32_t>(p.m_tiles);
        uint32_t within, along;  // along: tiles of the side that passes in blocks
        if constexpr (KIND == kWeight) {
            const uint32_t each = m_tiles * p.n_tiles;
            t.e = static_cast<int>(q / each);
            within = q - t.e * each;
            along = static_cast<uint32_t>(p.n_tiles);
        } else {
            const int32_t x = static_cast<int32_t>(q / m_tiles);
            int lo = 0, hi = p.E;  // the last expert whose first tile is not behind x
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tile0[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            t.e = lo;
            within = q - static_cast<uint32_t>(tile0[lo]) * m_tiles;
            along = static_cast<uint32_t>(tile0[lo + 1] - tile0[lo]);
        }
        const uint32_t block = within / (kBlock * m_tiles), left = along - block * kBlock, g = left < kBlock ? left : kBlock;
        const uint32_t r = within - block * kBlock * m_tiles, m = r / g, i = block * kBlock + (r - m * g);
        t.m0 = static_cast<int32_t>(m) * (KIND == kGated ? 128 : 256);
        const int32_t begin = first[t.e], n = first[t.e + 1] - begin;
        if constexpr (KIND == kWeight) {
            t.row = begin;
            t.rows = n;
            t.n = p.n_columns;
            t.n0 = static_cast<int32_t>(i) * p.n_columns;
            t.steps = (n + kStep - 1) / kStep * (p.fold ? 2 : 1);
        } else {
            t.n = static_cast<int32_t>((static_cast<uint32_t>(n) + along - 1) / along + 31) / 32 * 32;
            t.row = begin + static_cast<int64_t>(i) * t.n;
            const int64_t rest = begin + n - t.row;
            t.rows = static_cast<int32_t>(rest < t.n ? rest : t.n);
            t.n0 = 0;
            t.steps = (p.width + kStep - 1) / kStep * (p.fold ? 2 : 1);
        }
        t.begin = t.first_of(share, shares);
        t.end = t.first_of(share + 1, shares);
        return t;
    }
};

// The offsets as the kernels take them (none below its predecessor, all within [0, rows]) and, with TILES, the tiles of
// rows before each expert.  One warp, EACH neighbours a lane at a time, whose loads are in flight together (196 experts, a few
// rows: 6.0 us, 8.1 with one a lane).  Returns whether all were as they should be.
template <bool TILES, int EACH>
__device__ bool read_offsets(const Params &p, int32_t *first, int32_t *tile0, int lane)
{
    bool good = true;
    int32_t low = 0, tiles = 0;  // the offset and the tiles before these
    for (int base = 0; base <= p.E; base += 32 * EACH) {
        int32_t v[EACH], most = 0;
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int i = base + EACH * lane + k;
            v[k] = i > p.E ? 0 : (p.offsets ? p.offsets[i] : (i == 0 ? 0 : static_cast<int32_t>(p.n_rows)));
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int32_t c = v[k] < 0 ? 0 : (v[k] > p.n_rows ? static_cast<int32_t>(p.n_rows) : v[k]);
            most = c > most ? c : most;
            good = good && (base + EACH * lane + k > p.E || most == v[k]);
            v[k] = most;  // of this lane's up to here
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int32_t u = __shfl_up_sync(0xffffffffu, most, o);
            if (lane >= o)
                most = u > most ? u : most;
        }
        int32_t before = __shfl_up_sync(0xffffffffu, most, 1);
        before = lane == 0 || before < low ? low : before;
        good = good && (base + EACH * lane > p.E || v[0] >= before);
        int32_t sum = 0, prev = before, n[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int i = base + EACH * lane + k;
            const int32_t at = v[k] > before ? v[k] : before;
            if (i <= p.E)
                first[i] = at;
            if constexpr (TILES) {
                // tiles of expert i - 1
                sum += i == 0 || i > p.E ? 0 : (at - prev + p.cap - 1) / p.cap;
                n[k] = sum;
                prev = at;
            }
        }
        if constexpr (TILES) {
            int32_t all = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int32_t u = __shfl_up_sync(0xffffffffu, all, o);
                all += lane >= o ? u : 0;
            }
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                if (base + EACH * lane + k <= p.E)
                    tile0[base + EACH * lane + k] = tiles + all - sum + n[k];
            tiles += __shfl_sync(0xffffffffu, all, 31);
        }
        most = __shfl_sync(0xffffffffu, most, 31);
        low = most > low ? most : low;
    }
    return __all_sync(0xffffffffu, good);
}

// A bounded wait by a whole warp, which stays together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimitNs));
}

// ROWS rows of 128 bytes in shared memory to global memory: row r to out + r * stride (bytes) for r < rows, and of each the first
// `left` bytes (a multiple of 16).  Whole lines: lines written half by half, by whichever warps, took twice the time (a weights' gradient of 1.07 GB 311
// us, 3.5 TB/s; whole lines 164 us).
template <int ROWS>
__device__ __forceinline__ void store_lines(const uint8_t *staging, uint8_t *out, int64_t stride, int rows, int left, int lane)
{
#pragma unroll
    for (int i = 0; i < ROWS; i += 4) {
        const int r = i + lane / 8, part = lane % 8;
        if (r < rows && 16 * part < left)
            *reinterpret_cast<uint4 *>(out + r * stride + 16 * part) = *reinterpret_cast<const uint4 *>(staging + r * kPitch + 16 * part);
    }
}

// Sums that other pairs made of parts of a tile's contraction.  A unit is 32 values a thread: 32 columns of a warp's 32 lanes,
// or 64 of 16 lanes.  `inbox` holds, for every share, quarter and unit that this CTA writes, 32 values of 32 threads.
struct Shares {
    float *inbox;
    int count, mine, rank;  // pairs, this one, this CTA's place in it
    int units;              // most of a quarter's units that one pair writes

    __device__ int at(int share, int quarter, int unit) const { return ((share * 4 + quarter) * units + unit) * 1024; }

    // This CTA's part of a unit to the CTA that writes it.
    __device__ void send(int owner, int quarter, int unit, int lane, const uint32_t *v) const
    {
        const uint32_t to = cluster_map(smem_u32(inbox + at(mine, quarter, unit) + lane), 2 * owner + rank);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            store_cluster(to + 128 * i, v[i]);
    }

    // Adds what the others sent, in their order.
    __device__ void add(const Tile &t, int quarter, int unit, int lane, uint32_t *v) const
    {
        for (int s = 0; s < count; ++s) {
            if (s == mine || t.first_of(s, count) == t.first_of(s + 1, count))
                continue;
            const float *from = inbox + at(s, quarter, unit) + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = __float_as_uint(__uint_as_float(v[i]) + from[32 * i]);
        }
    }
};

// A tile of the weights' gradient: lanes are rows of the result, so a warp has whole lines of it, 64 columns (32 of fp32) of
// 16 rows at a time.
// 64 columns from c on of 16 of the warp's lanes; zeros where there are no steps, NaN where they were lost.
__device__ __forceinline__ void load_unit64(uint32_t (&raw)[32], const Tile &t, uint32_t sums, int quarter, int h, int c, bool lost)
{
    if (t.begin < t.end && !lost) {
        tmem_load_fragments(sums + (static_cast<uint32_t>(32 * quarter + 16 * h) << 16) + c, raw);
        tmem_load_wait();
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            raw[j] = lost ? 0x7FC00000u : 0u;
    }
}

// 32 columns from c on of the warp's lanes, 16 and then 16, the same way.
__device__ __forceinline__ void load_unit32(uint32_t (&raw)[2][16], const Tile &t, uint32_t sums, int quarter, int c, bool lost)
{
    if (t.begin < t.end && !lost) {
        const uint32_t from = sums + (static_cast<uint32_t>(quarter) << 21) + c;
        tmem_load_fragments(from, raw[0]);
        tmem_load_fragments(from + (16u << 16), raw[1]);
        tmem_load_wait();
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            raw[0][j] = raw[1][j] = lost ? 0x7FC00000u : 0u;
    }
}

// What this pair made of a shared tile and others write.
template <int KIND>
__device__ __forceinline__ void send_sums(const Tile &t, uint32_t sums, int quarter, int part, int lane, const Shares &shares, bool lost)
{
    if (t.begin == t.end)
        return;
    if constexpr (KIND == kWeight) {
        for (int q = 0; 64 * q < t.n; ++q) {  // the two warps of a quarter take 16 lanes each
            uint32_t raw[32];
            if (q % shares.count == shares.mine)
                continue;
            __syncwarp();
            load_unit64(raw, t, sums, quarter, part, 64 * q, lost);
            shares.send(q % shares.count, quarter, 2 * (q / shares.count) + part, lane, raw);
        }
    } else {
        for (int q = part; 32 * q < t.n; q += 2) {
            uint32_t raw[2][16];
            if (q % shares.count == shares.mine)
                continue;
            __syncwarp();
            load_unit32(raw, t, sums, quarter, 32 * q, lost);
            shares.send(q % shares.count, quarter, q / shares.count, lane, &raw[0][0]);
        }
    }
}

template <bool BF16, bool SPLIT>
__device__ __forceinline__ void write_gradient(const Params &p, const Tile &t, uint32_t sums, int quarter, int part, int lane, int rank,
                                               uint8_t *staging, const Shares &shares, bool lost)
{
    // The two warps of a quarter take every other chunk of 64 columns, or half of the lanes each where there is an odd number of
    // chunks (59 rows, K = 576, N = 2528, E = 125, three chunks a tile: 67 us, 77 with a warp taking two of them; 57
    // with the addresses' products made once a tile).
    const int columns = p.out_width - t.n0 < t.n ? p.out_width - t.n0 : t.n;
    const int step = SPLIT ? shares.count : 1, mine = SPLIT ? shares.mine : 0, chunks = ((columns + 63) / 64 - mine + step - 1) / step;
    const int size = p.fp32_out ? 4 : 2, row = t.m0 + rank * kSide + 32 * quarter;
    const int64_t stride = size * static_cast<int64_t>(p.out_width);
    uint8_t *const out = p.out + (static_cast<int64_t>(t.e) * p.width + row) * stride + size * t.n0;
#pragma unroll 1
    for (int u = 0; u < chunks; ++u) {
        const int h = chunks % 2 ? part : u % 2, q = mine + step * (chunks % 2 ? u : u - h + part), c = 64 * q;
        uint32_t raw[32];
        load_unit64(raw, t, sums, quarter, h, c, lost);
        if constexpr (SPLIT)
            shares.add(t, quarter, 2 * (q / shares.count) + h, lane, raw);
        const auto sum = [&](int s, int b, int j) { return __uint_as_float(raw[4 * b + 2 * s + j]); };
        uint8_t *const to = out + 16 * h * stride + size * c;
        const int rows = p.width - row - 16 * h, left = size * (columns - c);
        if (p.fp32_out) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        *reinterpret_cast<float2 *>(staging + (8 * s + lane / 4) * kPitch + 32 * b + 8 * (lane % 4)) =
                            make_float2(sum(s, 4 * x + b, 0), sum(s, 4 * x + b, 1));
                __syncwarp();
                store_lines<16>(staging, to + kLine * x, stride, rows, left - kLine * x, lane);
                __syncwarp();
            }
        } else {
            const uint32_t at_lane = smem_u32(staging) + (lane % 8) * kPitch + (lane / 8) * 16;
            const auto pair = [&](int s, int b) { return pack2<BF16>(sum(s, b, 0), sum(s, b, 1)); };
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < 8; b += 4)
                    store_fragments<false>(at_lane + 8 * s * kPitch + 16 * b, pair(s, b), pair(s, b + 1), pair(s, b + 2), pair(s, b + 3));
            __syncwarp();
            store_lines<16>(staging, to, stride, rows, left, lane);
            __syncwarp();
        }
    }
}

// A tile of rows to its place: warps `quarter` (0 to 3) of the CTA of rank `rank` have lanes 32 quarter on, and take turns.
// Lanes are columns of the result here.  Sums come as fragments of 8 x 8, and two warps put the 64 columns of theirs together
// in a staging, so that whole lines are written.
template <int KIND, bool BF16, int ACT, bool SPLIT>
__device__ __forceinline__ void write_tile(const Params &p, const Tile &t, uint32_t sums, int quarter, int part, int lane, int rank,
                                           uint8_t *staging, float *exchange, const Shares &shares, bool lost)
{
    const int second = quarter & 1;  // of the two warps
    const uint32_t at_lane = smem_u32(staging) + (lane % 8) * kPitch + (lane / 8) * 16 + 64 * second;
    for (int q = SPLIT ? shares.mine + shares.count * part : part; 32 * q < t.n; q += SPLIT ? 2 * shares.count : 2) {
        const int c = 32 * q;
        __syncwarp();
        uint32_t raw[2][16];
        load_unit32(raw, t, sums, quarter, c, lost);
        if constexpr (SPLIT)
            shares.add(t, quarter, q / shares.count, lane, &raw[0][0]);
        // the sum of lane 8 i + (lane / 4), column 8 b + 2 (lane % 4) + j of the chunk
        const auto sum = [&](int i, int b, int j) { return __uint_as_float(raw[i / 2][4 * b + 2 * (i % 2) + j]); };
        const auto pair = [&](int i, int b) { return pack2<BF16>(sum(i, b, 0), sum(i, b, 1)); };
        if constexpr (KIND == kGated) {
            // quarters 0 and 1 hold W1's sums, 2 and 3 W3's of the same features; the gate's warps take the chunk's first 16
            // columns and the others the last, and each gives the other what it needs
            const int f = t.m0 + rank * 64;
            const bool up = quarter >= 2;
            const uint32_t all = 1 + part;  // the barrier of the four warps
            float *give = exchange + (4 * part + quarter) * 512 + lane, *take = exchange + (4 * part + (quarter ^ 2)) * 512 + lane;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = j / 4, b = j / 2 % 2;
                give[32 * j] = up ? sum(i, b, j % 2) : sum(i, 2 + b, j % 2);
            }
            if (p.gate_up) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        store_fragments<true>(at_lane + 8 * b * kPitch, pair(0, 2 * h + b), pair(1, 2 * h + b), pair(2, 2 * h + b), pair(3, 2 * h + b));
                    named_barrier_sync(all, 128);
                    const int column = c + 16 * h + 8 * second;
                    store_lines<8>(staging + 8 * second * kPitch, p.gate_up + 2 * ((t.row + column) * p.gate_up_stride + (up ? p.out_width : 0) + f),
                                   2 * p.gate_up_stride, t.rows - column, 2 * (p.out_width - f), lane);
                    named_barrier_sync(all, 128);
                }
            } else {
                named_barrier_sync(all, 128);
            }
            float h[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = j / 4, b = j / 2 % 2;
                const float other = take[32 * j];
                const float g = up ? other : sum(i, b, j % 2), u = up ? sum(i, 2 + b, j % 2) : other;
                h[j] = act<ACT>(g) * u;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
                store_fragments<true>(at_lane + 8 * b * kPitch, pack2<BF16>(h[2 * b], h[2 * b + 1]), pack2<BF16>(h[4 + 2 * b], h[5 + 2 * b]),
                                      pack2<BF16>(h[8 + 2 * b], h[9 + 2 * b]), pack2<BF16>(h[12 + 2 * b], h[13 + 2 * b]));
            named_barrier_sync(all, 128);
            const int column = c + (up ? 16 : 0) + 8 * second;
            store_lines<8>(staging + 8 * second * kPitch, p.out + 2 * ((t.row + column) * p.out_stride + f), 2 * p.out_stride, t.rows - column,
                           2 * (p.out_width - f), lane);
            named_barrier_sync(all, 128);
        } else {
            const int f = t.m0 + rank * kSide + 64 * (quarter / 2);
            const uint32_t both = 1 + 2 * part + quarter / 2;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                store_fragments<true>(at_lane + 8 * b * kPitch, pair(0, b), pair(1, b), pair(2, b), pair(3, b));
            named_barrier_sync(both, 64);
            const int column = c + 16 * second;
            store_lines<16>(staging + 16 * second * kPitch, p.out + 2 * ((t.row + column) * p.out_stride + f), 2 * p.out_stride, t.rows - column,
                            2 * (p.out_width - f), lane);
            named_barrier_sync(both, 64);
        }
    }
}

// 64 columns of `rows` rows, fewer than 64, to shared memory, in a box for each digit of their number.  step 0: `row` is behind the
// tensor's last, and zeros are copied.
__device__ __forceinline__ void load_rows(uint32_t to, const CUtensorMap *boxes, int32_t column, int32_t row, int rows, int step, uint32_t bar)
{
#pragma unroll
    for (int place = 2; place >= 0; --place) {
        const int digit = (rows >> (2 * place)) & 3, n = digit << (2 * place);
        if (digit == 0)
            continue;
        tensor_load_pair(to, &boxes[3 * place + digit - 1], column, row, 0, 0, bar);
        to += n * kLine;
        row += n * step;
    }
}

// SPLIT: clusters of several pairs, a tile each; otherwise clusters of a pair, which take many.
template <int KIND, bool BF16, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps<KIND> maps)
{
    constexpr bool kAcrossA = KIND == kInput || KIND == kWeight, kAcrossB = KIND == kWeight;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int cta = static_cast<int>(cluster_rank()), rank = cta & 1, leader = SPLIT ? cta & ~1 : 0;
    const uint32_t both = 3u << leader;
    int32_t *first = reinterpret_cast<int32_t *>(smem + Layout::first), *tile0 = first + p.E + 1;
    const uint32_t full = base + Layout::full, empty = base + Layout::empty, sums_full = base + Layout::sums_full,
                   sums_empty = base + Layout::sums_empty, done = base + Layout::done;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + 8 * s, 2);   // both CTAs' copies
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sums_full + 8 * i, 1);
            mbar_init(sums_empty + 8 * i, 2 * kWriters);  // the writing warps of both CTAs
        }
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_map(&maps.a);
        for (int i = 0; i < (kAcrossB ? 1 : kRowBoxes); ++i)
            prefetch_map(&maps.b[i]);
    }
    if (warp == 2)
        tmem_alloc_pair(base + Layout::tmem, 512);
    if (warp == 0) {
        const bool good = p.E < 32 ? read_offsets<KIND != kWeight, 1>(p, first, tile0, lane) : read_offsets<KIND != kWeight, 9>(p, first, tile0, lane);
        if (!good && lane == 0 && p.status && blockIdx.x == 0)
            atomicCAS(p.status, 0, MOE_ERR_ROW_OUT_OF_RANGE);
    }
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_rel();
    cluster_wait_acq();
    tcgen05_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + Layout::tmem);
    const Schedule<KIND> plan(p, first, tile0, SPLIT ? cta / 2 : 0, SPLIT ? p.shares : 1);
    const uint32_t pair = cluster_id_x(), pairs = cluster_count_x();
    bool lost = false;  // writing warps: a wait has run out

    if (warp == 0) {
        // copies: this CTA's 128 of the tile's 256 and half of its N
        const uint32_t full_of_pair = cluster_map(full, leader);
        int64_t left = pair == 0 && cta == 0 && p.stall >= 0 ? p.stall : INT64_MAX;  // test hook (moe_debug_stall)
        RingPlace<kStages> place;
        bool good = true;
        for (uint32_t q = pair; q < plan.total && good; q += pairs) {
            const Tile t = plan.at(q);
            const int half = t.n / 2;
            const int chunks = (half + 63) / 64;
            const uint32_t bytes = kOperand + static_cast<uint32_t>(kAcrossB ? (p.wide_b ? 2 * kChunk : chunks * kChunk) : half * kLine);
            // the first step whose rows have boxes of their own
            const bool within = KIND == kWeight && t.rows % kStep != 0 && t.row + t.rows < p.n_rows;
            const int apart = within ? t.steps - (p.fold ? 2 : 1) : INT32_MAX;
            for (int k = t.begin; k < t.end; ++k) {
                if (left-- <= 0 || !warp_wait(empty + 8 * place.slot, place.phase)) {
                    good = false;
                    break;
                }
                const uint32_t a = base + place.slot * kStage, b = a + kOperand;
                const uint32_t bar = full_of_pair + 8 * place.slot;
                place.next();
                if (!elect_lane())
                    continue;
                const int x = (p.fold ? k / 2 : k) * kStep, part = p.fold && k % 2 ? p.fold : 0;
                const int32_t row = static_cast<int32_t>(t.row) + (KIND == kWeight ? x : rank * half);
                if constexpr (KIND == kWeight) {
                    // The last rows of an expert, and zeros up to a multiple of 16, all that the matrix instructions take (a
                    // neighbour's values times zero would not do, as they may be infinities).  The zeros are copies too, of
                    // rows that the tensor does not have, so that one barrier announces all of it to the pair: zeros stored by a
                    // warp of either CTA had to be released to the pair, which waits for the writing warps' stores as well (R =
                    // 8191, K = 2048, N = 2816, E = 64: 177 us; 137 this way; 136 with zeros that nothing orders for the other CTA).
                    // An expert whose rows end with the tensor has them without this.
                    if (k >= apart) {
                        const int rest = t.rows % kStep, zeros = -rest & 15;
                        mbar_arrive_expect_tx_cluster(bar, static_cast<uint32_t>((2 + chunks) * (rest + zeros) * kLine));
#pragma unroll 1
                        for (int c = 0; c < 2 + chunks; ++c) {
                            const CUtensorMap *boxes = c < 2 ? maps.end_a : maps.end_b;
                            const int32_t column = c < 2 ? t.m0 + rank * kSide + part + 64 * c : t.n0 + rank * half + 64 * (c - 2);
                            load_rows(a + c * kChunk, boxes, column, row, rest, 1, bar);
                            load_rows(a + c * kChunk + rest * kLine, maps.end_a, 0, static_cast<int32_t>(p.n_rows), zeros, 0, bar);
                        }
                        continue;
                    }
                }
                mbar_arrive_expect_tx_cluster(bar, bytes);
                if constexpr (KIND == kForward) {
                    tensor_load_pair(a, &maps.a, x, t.m0 + rank * kSide, t.e, bar);
                } else if constexpr (KIND == kGated) {
                    tensor_load_pair(a, &maps.a, x, t.m0 + rank * 64, 0, t.e, bar);  // 64 rows of W1 and the same of W3
                } else {
                    const int y = KIND == kInput ? x : row, e = KIND == kInput ? t.e : 0, column = t.m0 + rank * kSide + (KIND == kWeight ? part : 0);
                    if (p.wide_a) {
                        tensor_load_pair(a, &maps.a, 0, y, column / 64, e, bar);
                    } else {
                        tensor_load_pair(a, &maps.a, column, y, 0, e, bar);
                        tensor_load_pair(a + kChunk, &maps.a, column + 64, y, 0, e, bar);
                    }
                }
                if constexpr (kAcrossB) {
                    const int column = t.n0 + rank * half;
                    if (p.wide_b) {
                        tensor_load_pair(b, &maps.b[0], 0, row, column / 64, 0, bar);
                    } else {
                        for (int c = 0; c < chunks; ++c)
                            tensor_load_pair(b + c * kChunk, &maps.b[0], column + 64 * c, row, 0, 0, bar);
                    }
                } else {
                    // half is a multiple of 16: one box for each of its bits
                    int at = 0;
#pragma unroll
                    for (int i = kRowBoxes - 1; i >= 0; --i)
                        if (half & (16 << i)) {
                            tensor_load_pair(b + at * kLine, &maps.b[i], x + part, row + at, 0, bar);
                            at += 16 << i;
                        }
                }
            }
        }
        // the last arrivals at this CTA's barriers land before it leaves
        if (good)
            place.drain([&](uint32_t slot, uint32_t phase) { return warp_wait(empty + 8 * slot, phase); });
    } else if (warp == 1 && rank == 0) {
        uint32_t slot = 0, phase = 0, turn = 0;
        bool good = true;
        for (uint32_t q = pair; q < plan.total && good; q += pairs) {
            const Tile t = plan.at(q);
            if (t.begin == t.end)
                continue;
            const uint32_t idesc = mma_f16_descriptor(BF16, kAcrossA, kAcrossB, 256, static_cast<uint32_t>(t.n));
            const uint32_t sums = tmem + (turn & 1) * kMaxN;
            good = warp_wait(sums_empty + 8 * (turn & 1), ((turn >> 1) & 1) ^ 1);
            tcgen05_fence_after();
            for (int k = t.begin; k < t.end && good; ++k) {
                good = warp_wait(full + 8 * slot, phase);
                if (!good)
                    break;
                tcgen05_fence_after();
                const uint32_t at = base + slot * kStage;
                const uint64_t a = kAcrossA ? operand_across(at, kChunk) : operand_along(at);
                const uint64_t b = kAcrossB ? operand_across(at + kOperand, kChunk) : operand_along(at + kOperand);
                // 16 of the contraction each: 32 bytes of a line, or 16 lines; of the rows that end in this step, what there is of them
                const int sixteens = KIND == kWeight && t.ends(k, p.fold) ? (t.rows % kStep + 15) / 16 : kStep / 16;
                if (elect_lane()) {
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j)
                        if (KIND != kWeight || j < sixteens)
                            mma_pair_f16(sums, a + j * (kAcrossA ? 16 * kLine / 16 : 2), b + j * (kAcrossB ? 16 * kLine / 16 : 2), idesc, k > t.begin || j > 0);
                    mma_pair_commit(empty + 8 * slot, both);
                }
                __syncwarp();
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (good && elect_lane())
                mma_pair_commit(sums_full + 8 * (turn & 1), both);
            __syncwarp();
            ++turn;
        }
        if (!good) {
            // what is in flight ends before the pair leaves: matrix instructions, and copies (those of a slot that only one CTA
            // filled never complete its barrier, and have long landed after the wait)
            if (elect_lane())
                mma_pair_commit(done, 1u << leader);  // the other CTA does not wait for it
            __syncwarp();
            warp_wait(done, 0);
            const uint64_t t0 = globaltimer_ns();
            for (int s = 0; s < kStages; ++s) {
                while (!mbar_try_wait(full + 8 * slot, phase) && globaltimer_ns() - t0 < kWaitLimitNs / 4) {
                }
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, part = warp / 4 - 1;
        const uint32_t empty_of_pair = cluster_map(sums_empty, leader);
        uint8_t *staging = smem + Layout::staging + (KIND == kWeight ? warp - 4 : (KIND == kGated ? 1 : 2) * (warp / 2 - 2)) * 16 * kPitch;
        float *exchange = reinterpret_cast<float *>(smem + Layout::exchange);
        uint32_t turn = 0;
        for (uint32_t q = pair; q < plan.total; q += pairs) {
            const Tile t = plan.at(q);
            const uint32_t i = turn & 1;
            if (t.begin < t.end && !lost) {
                // a long contraction takes longer than the limit alone
                lost = !mbar_wait_bounded(sums_full + 8 * i, (turn >> 1) & 1, wait_limit(t.steps));
                lost = __any_sync(0xffffffffu, lost);
                tcgen05_fence_after();
            }
            if constexpr (SPLIT)
                break;  // the tile is written below
            if constexpr (KIND == kWeight)
                write_gradient<BF16, false>(p, t, tmem + i * kMaxN, quarter, part, lane, rank, staging, {}, lost);
            else
                write_tile<KIND, BF16, ACT, false>(p, t, tmem + i * kMaxN, quarter, part, lane, rank, staging, exchange, {}, lost);
            if (t.begin < t.end) {
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0 && !lost)
                    mbar_arrive_cluster(empty_of_pair + 8 * i);
                ++turn;
            }
        }
        if (lost && lane == 0 && p.status)
            atomicCAS(p.status, 0, MOE_ERR_DEVICE_TIMEOUT);
    }
    if constexpr (SPLIT) {
        __syncwarp();
        // every pair's matrix instructions are complete, and the slots' memory is free for sums
        cluster_arrive_rel();
        cluster_wait_acq();
        const int quarter = warp & 3, part = warp / 4 - 1;
        const bool writes = warp >= 4 && pair < plan.total;
        const Tile t = writes ? plan.at(pair) : Tile{};
        const Shares shares{reinterpret_cast<float *>(smem), p.shares, cta / 2, rank,
                            KIND == kWeight ? 2 * (((t.n + 63) / 64 + p.shares - 1) / p.shares) : (t.n / 32 + p.shares - 1) / p.shares};
        if (writes)
            send_sums<KIND>(t, tmem, quarter, part, lane, shares, lost);
        __syncwarp();
        cluster_arrive_rel();
        cluster_wait_acq();
        if (writes) {
            uint8_t *staging = smem + Layout::staging + (KIND == kWeight ? warp - 4 : (KIND == kGated ? 1 : 2) * (warp / 2 - 2)) * 16 * kPitch;
            if constexpr (KIND == kWeight)
                write_gradient<BF16, true>(p, t, tmem, quarter, part, lane, rank, staging, shares, lost);
            else
                write_tile<KIND, BF16, ACT, true>(p, t, tmem, quarter, part, lane, rank, staging, reinterpret_cast<float *>(smem + Layout::exchange),
                                                  shares, lost);
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    cluster_arrive_rel();
    cluster_wait_acq();
    tcgen05_fence_after();
    if (warp == 2)
        tmem_free_pair(tmem, 512);
}

// -------------------------------------------------------------------------------------------------- launch

// Tiles at most, and exactly with one expert.
int64_t tiles_of(int64_t rows, int64_t E, int cap, int64_t m_tiles)
{
    return (E == 1 ? (rows + cap - 1) / cap : rows / cap + (rows < E ? rows : E)) * m_tiles;
}

template <int KIND, bool BF16, int ACT>
moe_status launch(const Product &a, moe_stream_t stream)
{
    static SmemLimit limits[2];
    const int sms = sm_count();
    int dev = 0;
    Params p{};
    Maps<KIND> maps{};
    p.n_rows = a.n_rows;
    p.E = a.E;
    p.width = a.width;
    p.out_width = a.out_width;
    p.fold = a.fold;
    p.offsets = a.offsets;
    p.out = static_cast<uint8_t *>(a.out);
    p.out_stride = a.out_stride;
    p.gate_up = static_cast<uint8_t *>(a.gate_up);
    p.gate_up_stride = a.gate_up_stride;
    p.status = a.status;
    p.fp32_out = a.fp32_out;
    p.stall = a.stall;
    const int64_t steps = KIND == kWeight ? a.n_rows / a.E / kStep : (a.width + kStep - 1) / kStep * (a.fold ? 2 : 1);
    // Pairs that share a tile, 1 / 2 / 3 / 4, us in a graph: 16 rows, N = 2048 (8 tiles), K = 2048: 9.1 / 10.0 / 9.4 / 9.2, 2560:
    // 10.3 / 10.8 / 10.0 / 9.7, 4096: 14.0 / 13.4 / 11.6 / 11.0, 8192: 23.6 / 20.1 / 16.0 / 14.4; weights' gradient of 1024 x 1024,
    // 2048 rows: 13.6 / 13.2 / - / 14.0, 4096: - / 17.8 / 18.8 / -, 8192: 38.8 / 27.0 / 25.2 / 20.3.  Tiles of many rows have too many
    // sums to send for three (256 rows, K = N = 4096: 14.9 with two and 128 columns, 17.2 with three and 256).  No more than 15 clusters
    // of 8 CTAs run at once (16 tiles: 21 us instead of 11), 23 of 6 and 36 of 4.
    const auto shares_of = [&](int64_t count, int columns) {
        if (count <= sms / 10 && steps >= 40)
            return 4;
        if (count <= sms / 6 - 2 && (KIND == kWeight ? steps >= 80 : columns <= kMaxN / 2 && steps >= 48))
            return 3;
        return count <= sms / 4 - 2 && steps >= 64 ? 2 : 1;
    };
    // Narrower tiles where they make fewer or emptier rounds.  A step of a tile of n columns takes about as long as its way through
    // an SM's shared memory, in lines of 128 bytes: 128 + n / 2 written and 128 + n read (153 ns at n = 32, 230 at 128, 308 at
    // 256).  R = 4096, N = 4096, K = 16384 is 4 rounds of 256 tiles or 4 of 304 with 224 columns (319 and 298 us); the weights'
    // gradient of R = N = K = 4096 took 82 and 77 us.  Tiles of rows of several experts are known here only where they make one
    // round.
    int64_t tiles, least = INT64_MAX;
    const int64_t pairs = sms / 2;
    const auto better = [&](int64_t count, int columns, bool known) {
        const int64_t rounds = (count + pairs - 1) / (pairs > 0 ? pairs : 1), cost = rounds * (2 * kMaxN + 3 * columns) * 12 / shares_of(count, columns);
        if (cost >= least || !(known || rounds == 1))
            return false;
        least = cost;
        return true;
    };
    if (KIND == kWeight) {
        p.m_tiles = (a.width + 255) / 256;
        const auto count = [&](int columns) { return static_cast<int64_t>(a.E) * p.m_tiles * ((a.out_width + columns - 1) / columns); };
        p.n_columns = a.out_width > 64 ? 128 : 64;
        for (int columns = kMaxN; columns >= kMaxN / 2 && a.out_width > 128; columns -= 32)
            if (better(count(columns), columns, true))
                p.n_columns = columns;
        p.n_tiles = (a.out_width + p.n_columns - 1) / p.n_columns;
        tiles = count(p.n_columns);
    } else {
        p.m_tiles = KIND == kGated ? (a.out_width + 127) / 128 : (a.out_width + 255) / 256;
        p.cap = kMaxN;
        for (int cap = kMaxN; cap >= kMaxN / 2; cap -= 32)
            if (better(tiles_of(a.n_rows, a.E, cap, p.m_tiles), cap, a.E == 1))
                p.cap = cap;
        tiles = tiles_of(a.n_rows, a.E, p.cap, p.m_tiles);
    }
    p.shares = shares_of(tiles, KIND == kWeight ? p.n_columns : p.cap);
    const auto kern = p.shares > 1 ? product_kernel<KIND, BF16, ACT, true> : product_kernel<KIND, BF16, ACT, false>;
    const int64_t W = a.width, F = a.out_width, held = a.fold ? 2 * a.fold : W;  // held: columns of `rows` in memory
    // [rows, columns] across, of `groups` matrices: chunks of 64 columns, two in a box where the columns are whole chunks
    const auto across = [](CUtensorMap &map, const void *at, int64_t columns, int64_t rows, int64_t groups, int64_t stride, bool wide,
                           int box = kStep) {
        if (wide)
            return encode_tensor(map, at, {4, {64, rows, columns / 64, groups}, {stride, 64, groups > 1 ? rows * stride : stride}, {64, box, 2, 1}});
        return encode_tensor(map, at, {4, {columns, rows, 1, groups}, {stride, stride, groups > 1 ? rows * stride : stride}, {64, box, 1, 1}});
    };
    if (tiles >= int64_t{1} << 31)
        return MOE_ERR_UNSUPPORTED;
    bool ok = true;
    if constexpr (KIND == kForward) {
        ok = encode_tensor(maps.a, a.other, {3, {W, F, a.E}, {W, F * W}, {kStep, kSide, 1}});
    } else if constexpr (KIND == kGated) {
        ok = encode_tensor(maps.a, a.other, {4, {W, F, 2, a.E}, {W, F * W, 2 * F * W}, {kStep, 64, 2, 1}});
    } else if constexpr (KIND == kInput) {
        p.wide_a = F % 64 == 0;
        ok = across(maps.a, a.other, F, W, a.E, F, p.wide_a);
    }
    if constexpr (KIND == kWeight) {
        p.wide_a = held % 64 == 0;
        p.wide_b = F % 64 == 0 && p.n_columns == 256;
        ok = across(maps.a, a.rows, held, a.n_rows, 1, a.rows_stride, p.wide_a) && across(maps.b[0], a.other, F, a.n_rows, 1, a.other_stride, p.wide_b);
        for (int i = 0; a.offsets && i < kEndBoxes; ++i)  // without offsets the only expert's rows end with the tensor
            ok = ok && across(maps.end_a[i], a.rows, held, a.n_rows, 1, a.rows_stride, false, (i % 3 + 1) << (i / 3 * 2)) &&
                 across(maps.end_b[i], a.other, F, a.n_rows, 1, a.other_stride, false, (i % 3 + 1) << (i / 3 * 2));
    } else {
        for (int i = 0; i < kRowBoxes; ++i)
            ok = ok && encode_tensor(maps.b[i], a.rows, {3, {held, a.n_rows, 1}, {a.rows_stride, a.rows_stride}, {kStep, 16 << i, 1}});
    }
    const size_t smem = static_cast<size_t>(Layout::bytes(a.E));
    if (!ok || sms < 2 || cudaGetDevice(&dev) != cudaSuccess || ensure_dynamic_smem(kern, dev, static_cast<int>(smem), limits[p.shares > 1]) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const int64_t clusters = p.shares > 1 || tiles < sms / 2 ? tiles : sms / 2;
    // an ordinary launch: pairs that were resident before the kernel in front of them had ended were not worth their risk (a
    // CTA holds all tensor memory of its SM)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * p.shares);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * p.shares * (clusters < 1 ? 1 : clusters)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p, maps) == cudaSuccess)
        return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

template <bool BF16>
moe_status dispatch(ProductKind kind, const Product &p, moe_stream_t stream)
{
    switch (kind) {
    case kForward: return launch<kForward, BF16, 0>(p, stream);
    case kGated: return p.activation == MOE_ACT_SILU ? launch<kGated, BF16, MOE_ACT_SILU>(p, stream) : launch<kGated, BF16, MOE_ACT_GELU_TANH>(p, stream);
    case kInput: return launch<kInput, BF16, 0>(p, stream);
    default: return launch<kWeight, BF16, 0>(p, stream);
    }
}

} // namespace

moe_status run_product(ProductKind kind, const Product &p, moe_stream_t stream)
{
    return p.bf16 ? dispatch<true>(kind, p, stream) : dispatch<false>(kind, p, stream);
}

} // namespace nqg
