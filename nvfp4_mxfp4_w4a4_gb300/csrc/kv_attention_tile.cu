// kv_attention_tile.cu -- attention of many rows (trees of drafted tokens)
// over the MX-quantized paged cache, on the 5th-generation tensor cores.
//
// The same operation as kv_attention.cu, whose warps would each convert the
// cache's codes again for every few rows.  Here a CTA owns up to NR = 128 rows
// (drafted token x query head of one key/value head) and walks the context in
// tiles of 128 tokens; each tile is converted once, to bf16 in shared memory,
// and multiplied by tcgen05.mma with the tokens on the M side, so that the MMA
// work follows the number of rows:
//   S^T [128 tokens x NR]  = K [tokens x dims] Q^T       (both K-major)
//   O^T [dims x NR]       += V^T [dims x tokens] P^T     (both MN-major: V and
//                            P lie token by token, as they are produced)
// A softmax thread is one token, its registers hold that token's scores of all
// rows, so a row's maximum and sum run across threads.  The maximum is
// therefore lazy: scores are taken relative to the row's reference in shared
// memory, and only when one passes it by 2^8 (one vote per tile) are the
// references, the sums and O^T rescaled; a thread keeps its own share of every
// row's sum until the end.
//
// Numbers: as in kv_attention.cu (exact bf16 elements with a multiplier that
// carries 2^-64, probabilities rounded to bf16, everything else fp32), keys
// included.  Elements of a group of 4 (E4M3) or 8 (E2M1) are stored in the
// order in which their bits come out of a word; Q is stored in that order too,
// and the output's rows are put back at the end.
//
// The work is cut on the device: the tiles of all (sequence, key/value head,
// row tile) units in one line, with a few places for each unit's start and end,
// an equal run of the line per CTA, one CTA per SM.
// A unit whose tiles fall to several CTAs leaves partial results (a CTA has at
// most two: of the unit that began before its run and of the one that goes on
// after it), which the join kernel adds.  With a grid of equal chunks instead,
// the last round of CTAs and every CTA's start and end cost as much as the
// tiles (8 trees of 31 tokens over up to 16001 tokens: 139 us).
//
// Warps: 0-7 softmax (quadrant of tokens x half of the rows; they also load Q
// and write the results), 8-11 convert keys, 12-15 values, 16 issues the first
// product's MMAs and 17 the second's (18, 19 fill the register group).  A wait
// costs an issuing thread a few hundred cycles even when its phase is complete,
// so each product of a tile has one: its barrier counts the converters and the
// softmax warps.  K, V, S and P are double-buffered, and the converters run
// ahead into the CTA's next unit.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "kv_attention.cuh"
#include "ptx.cuh"

namespace fp4lin {
namespace {

constexpr int kTile = 128;  // tokens
constexpr int kSlab = kTile * 128;  // bytes of 64 bf16 elements of a tile's tokens
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 8 + 4) * 32;
// The work line: a unit is kUnitTiles places (its start and end cost about as
// much as five tiles: 9 us against 1.8 us with 128 rows) and then its tiles.
constexpr int kUnitTiles = 5;
constexpr int kLeastRun = kUnitTiles + 4;
constexpr float kUnset = -1e30f;  // a row's reference before its first visible token
constexpr uint32_t kSlackBits = 0x4380u;  // bf16 bits of 2^8: weights above it move the references
constexpr float kCeiling = 100.0f;        // of a weight's exponent, until they have moved

// d[0..1] = a[0..1] * m + c[0..1] in one instruction.
__device__ __forceinline__ void fma_pair(float* d, float a0, float a1, float2 m, float c0, float c1)
{
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a0), "f"(a1), "f"(m.x), "f"(m.y), "f"(c0), "f"(c1));
}

// The smaller, or NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int kFmt, int kDim, int NR>
struct TileCfg {
    static constexpr int SLABS = kDim / 64;
    static constexpr int P_SLABS = NR > 64 ? 2 : 1;
    static constexpr int OFF_K = NR * 128 * SLABS;  // Q first
    static constexpr int OFF_V = OFF_K + 2 * SLABS * kSlab;
    static constexpr int OFF_P = OFF_V + 2 * SLABS * kSlab;
    static constexpr int OFF_REF = OFF_P + 2 * P_SLABS * kSlab;  // float [NR]: the rows' references, negated
    static constexpr int OFF_POISON = OFF_REF + NR * 4;          // uint32 [NR]: blocks of a row that are NaN
    static constexpr int OFF_BAR = OFF_POISON + NR * 4;
    static constexpr int OFF_SLOT = OFF_BAR + 8 * 8;  // TMEM address, flags, the run's tiles
    static constexpr int OFF_WALK = OFF_SLOT + 32;  // the run's first unit; the softmax's current one
    static constexpr int OFF_SCRATCH = OFF_WALK + 2 * 64;  // two halves' [5][COLS] floats (below 128 rows)
    static constexpr int SMEM = OFF_SCRATCH + (NR < 128 ? 5 * NR * 4 : 0) + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = NR == 32 ? 128 : NR == 64 ? 256 : 512;
    static constexpr int COLS = NR / 2;  // rows per softmax thread
    // conversion: 16-byte chunks of a token's codes, one per lane
    static constexpr int ROW = kFmt == kKvMxfp8 ? kDim : kDim / 2;
    static constexpr int CH = ROW / 16;
    static constexpr int SB = kDim / 32;
    // With few rows a tile takes less time than its codes from memory, so two
    // tiles are on their way: 64 KB (E4M3) per SM.
    static constexpr int AHEAD = NR == 128 ? 1 : 2;
    // registers per thread of the three groups, out of 96 x 640 at launch (a
    // softmax thread keeps COLS sums, a converter AHEAD tiles' codes)
    static constexpr int REGS_SOFTMAX = NR == 128 ? 136 : NR == 64 ? 104 : 88,
                         REGS_CONVERT = NR == 128 ? 88 : NR == 64 ? 120 : 136, REGS_MMA = NR == 128 ? 24 : 32;
    static constexpr int REGS = 256 * REGS_SOFTMAX + 256 * REGS_CONVERT + 128 * REGS_MMA;
    static_assert(REGS <= 96 * kThreads, "register split");
    static_assert(SMEM <= 232448, "shared memory budget");
};

// The calling warpgroup's registers per thread, from 96 at launch.
template <int kRegs>
__device__ __forceinline__ void set_registers()
{
    if constexpr (kRegs > 96)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else if constexpr (kRegs < 96)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Element that is stored at position `pos` of a head.
template <int kFmt>
__device__ __forceinline__ int element_at(int pos)
{
    return kFmt == kKvMxfp8 ? (pos & ~3) | ((pos & 1) << 1) | ((pos >> 1) & 1) : (pos & ~7) | ((pos & 1) << 2) | ((pos >> 1) & 3);
}

// One unit after the other: its sequence, head, first row and tiles.
template <int NR>
struct Walk {
    int b, unit, units, row_tiles, tiles;  // units of the sequence, tiles of a unit
    int ctx, len, n, q_start;
    int lo;    // first tile of the CTA's run in this unit
    int lead;  // places of the unit's start that lie in the run
    int head;

    __device__ __forceinline__ void sequence(const AttnParams& p)
    {
        group_rows(p.q_offsets, b, p.T, &q_start, &n);
        ctx = max(min(__ldg(p.context_lens + b), p.max_len - n), 0);
        len = min(ctx + n, p.max_len);
        tiles = (len + kTile - 1) / kTile;
        row_tiles = min((n * p.group + NR - 1) / NR, p.row_tiles);
        units = row_tiles * p.cache.heads;
    }
    __device__ __forceinline__ void next(const AttnParams& p)
    {
        lo = 0;
        lead = kUnitTiles;
        ++unit;
        while (unit >= units && b + 1 < p.batch) {
            ++b;
            unit = 0;
            sequence(p);
        }
        head = row_tiles > 0 ? unit / row_tiles : 0;
    }
    // Tiles of this unit in a run with `left` places to go, which it takes away.
    __device__ __forceinline__ int run(const AttnParams& p, int64_t& left) const
    {
        if (p.whole) {
            --left;
            return tiles;
        }
        const int64_t here = min(left - lead, static_cast<int64_t>(tiles - lo));
        left -= lead + max(here, int64_t(0));
        return static_cast<int>(max(here, int64_t(0)));
    }
    __device__ __forceinline__ int row0() const { return (unit - head * row_tiles) * NR; }
};

// A tile for the converters.
struct TileRef {
    int t0, len, head, page[2];
    bool edge;  // (values) not all its tokens are context
};

template <int kFmt, int kDim, int NR>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tile_kernel(const AttnParams p)
{
    using C = TileCfg<kFmt, kDim, NR>;
    extern __shared__ uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    // ------------------------------------------------ this CTA's run of tiles
    // (p.whole: units instead of tiles are dealt out, and none is cut)
    static_assert(sizeof(Walk<NR>) <= 64, "its place in shared memory");
    int64_t count;  // tiles (units) of the run
    {
        struct Scan {
            int64_t warp_sum[kThreads / 32];
            int64_t offset;
            int b;
        };
        Scan* scan = reinterpret_cast<Scan*>(smem);
        auto weight = [&](int i) -> int64_t {
            if (i >= p.batch)
                return 0;
            Walk<NR> w;
            w.b = i;
            w.sequence(p);
            return p.whole ? w.units : static_cast<int64_t>(w.units) * (w.tiles + kUnitTiles);
        };
        // sum over the block of v, and of the threads before this one
        auto block_scan = [&](int64_t v, int64_t* before) -> int64_t {
            int64_t x = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                x += lane >= d ? y : 0;
            }
            __syncthreads();
            if (lane == 31)
                scan->warp_sum[warp] = x;
            __syncthreads();
            int64_t total = 0, base = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                base += w < warp ? scan->warp_sum[w] : 0;
                total += scan->warp_sum[w];
            }
            *before = base + x - v;
            return total;
        };
        int64_t total = 0, before, mine = 0;
        for (int i = 0; i < p.batch; i += kThreads) {
            mine = weight(i + threadIdx.x);
            total += block_scan(mine, &before);
        }
        const int64_t per = max((total + gridDim.x - 1) / gridDim.x, int64_t(p.whole ? 1 : kLeastRun));
        const int64_t start = blockIdx.x * per;
        count = min(per, total - start);
        int64_t base = 0;
        for (int i = 0; i < p.batch; i += kThreads) {
            const int me = i + threadIdx.x;
            if (p.batch > kThreads) {
                mine = weight(me);
                const int64_t sum = block_scan(mine, &before);
                before += base;
                base += sum;
            }
            if (start >= before && start < before + mine) {
                scan->b = me;
                scan->offset = start - before;
            }
            if (blockIdx.x == 0 && me < p.batch)
                p.prefix[me] = before;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0)
            p.prefix[p.batch] = per;
        __syncthreads();
        if (count <= 0)
            return;
        if (threadIdx.x == 0) {
            Walk<NR> w;
            w.b = scan->b;
            w.sequence(p);
            const int64_t off = scan->offset;
            const int length = p.whole ? 1 : w.tiles + kUnitTiles;
            w.unit = static_cast<int>(off / length);
            w.head = w.unit / w.row_tiles;
            const int in_unit = static_cast<int>(off - static_cast<int64_t>(w.unit) * length);
            w.lead = max(kUnitTiles - in_unit, 0);
            w.lo = p.whole ? 0 : max(in_unit - kUnitTiles, 0);
            *reinterpret_cast<Walk<NR>*>(smem + C::OFF_WALK) = w;
            *reinterpret_cast<Walk<NR>*>(smem + C::OFF_WALK + 64) = w;
            uint32_t total = 0;
            for (int64_t left = count; left > 0; w.next(p))
                total += w.run(p, left);
            reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT)[7] = total;
        }
        __syncthreads();
    }
    float* ref = reinterpret_cast<float*>(smem + C::OFF_REF);
    uint32_t* poison = reinterpret_cast<uint32_t*>(smem + C::OFF_POISON);
    // the tile's keys (and its unit's Q) are in shared memory, and the S^T before the last has been read
    uint64_t* s_ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* s_done = s_ready + 2;    // S^T is complete (and the keys' buffer free)
    uint64_t* pv_ready = s_done + 2;   // values and P^T are in shared memory
    uint64_t* pv_done = pv_ready + 2;  // the tile is in O^T (the values' and P^T's buffers free)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* unit_start = tmem_slot + 1;  // by tile parity: the tile is its unit's first
    volatile uint32_t* gave_up = tmem_slot + 3;     // by half and tile parity: a softmax wait of the tile ran out
    const uint32_t* total_tiles = tmem_slot + 7;    // of the run

    if (threadIdx.x == 0) {
        gave_up[0] = gave_up[1] = gave_up[2] = gave_up[3] = 0u;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_ready[i], 4 + kSoftmaxWarps);
            mbar_init(&s_done[i], 1);
            mbar_init(&pv_ready[i], 4 + kSoftmaxWarps);
            mbar_init(&pv_done[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_o = tmem + 2 * NR;
    const uint64_t limit = p.wait_ns;
    bool ok = true;

    if (warp >= 16) {
        // ----------------------------------------------------- MMA issuers
        set_registers<C::REGS_MMA>();
        // (the whole warp walks the loop and one elected lane issues: the operands
        // of the MMAs then stay in uniform registers)
        if (warp == 16) {
            constexpr uint32_t idesc = idesc_bf16(128, NR, 0, 0);
            const uint64_t kd = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2);
            for (uint32_t g = 0, end = *total_tiles; g < end; ++g) {
                const uint32_t f = g & 1u;
                ok = mbar_wait_bounded(&s_ready[f], (g >> 1) & 1u, p.status, kStatusTimeout, limit);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after_sync();
                const uint64_t kf = kd + ((f * C::SLABS * kSlab) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kDim / 16; ++k)
                        tc_mma_f16(tmem + f * NR, kf + (((k >> 2) * kSlab + 32 * (k & 3)) >> 4),
                                   qd + (((k >> 2) * (NR * 128) + 32 * (k & 3)) >> 4), idesc, k != 0);
                    tc_commit(&s_done[f]);
                }
                __syncwarp();
            }
        } else if (warp == 17) {
            constexpr uint32_t idesc = idesc_bf16(128, NR, 1, 1);
            const uint64_t vd = smem_desc(smem_u32(smem + C::OFF_V), kSlab, 1024, 2);
            const uint64_t pd = smem_desc(smem_u32(smem + C::OFF_P), kSlab, 1024, 2);
            for (uint32_t g = 0, end = *total_tiles; g < end; ++g) {
                const uint32_t f = g & 1u;
                ok = mbar_wait_bounded(&pv_ready[f], (g >> 1) & 1u, p.status, kStatusTimeout, limit);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after_sync();
                const uint64_t vf = vd + ((f * C::SLABS * kSlab) >> 4), pf = pd + ((f * C::P_SLABS * kSlab) >> 4);
                const uint32_t add = unit_start[f] ? 0u : 1u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_f16(tmem_o, vf + ((2048 * k) >> 4), pf + ((2048 * k) >> 4), idesc, k ? 1u : add);
                    tc_commit(&pv_done[f]);
                }
                __syncwarp();
            }
        }
    } else if (warp >= kSoftmaxWarps) {
        // --------------------------------------------- codes -> bf16 tiles
        set_registers<C::REGS_CONVERT>();
        // 16-byte chunks of the codes, one per lane.  Eight lanes in a row store to
        // one slab, for tokens whose swizzles differ, so that their 16-byte pieces
        // fall in different banks.
        const bool value = warp >= kSoftmaxWarps + 4;
        const int w32 = (warp & 3) * 32;              // this warp's tokens of the tile
        constexpr int TPI = 32 / C::CH;               // tokens per load
        constexpr int HC = C::CH / C::SLABS;          // chunks of a token per slab
        const int chunk = ((lane >> 3) % C::SLABS) * HC + lane % HC;
        const int sub = (lane >> 3) / C::SLABS * (8 / HC) + lane / HC % (8 / HC);
        const uint8_t* codes = (value ? p.cache.v_codes : p.cache.k_codes) + sub * C::ROW + chunk * 16;
        const uint8_t* scales =
            (value ? p.cache.v_scales : p.cache.k_scales) + sub * C::SB + (kFmt == kKvMxfp8 ? chunk / 2 : chunk);
        // where the lane's 16-byte pieces of its first token go
        constexpr int PIECES = kFmt == kKvMxfp8 ? 2 : 4;
        uint32_t at_piece[PIECES];
#pragma unroll
        for (int h = 0; h < PIECES; ++h) {
            const int piece = PIECES * chunk + h;
            at_piece[h] = smem_u32(smem + (value ? C::OFF_V : C::OFF_K)) + (piece >> 3) * kSlab + (w32 + sub) * 128 +
                          (((piece & 7) ^ (sub & 7)) << 4);
        }
        uint64_t* full = value ? pv_ready : s_ready;
        uint64_t* freed = value ? pv_done : s_done;
        // The run's tiles in order: a tile's pages are looked up three tiles ahead, its
        // tokens' places found two ahead, its codes loaded one ahead.
        Walk<NR> w = *reinterpret_cast<const Walk<NR>*>(smem + C::OFF_WALK);
        int64_t left = count;
        int tiles = w.run(p, left), at = 0;  // of the unit that the look-up is in
        auto look_up = [&](TileRef& r) -> bool {
            while (at == tiles) {  // (a run may hold no tile of its first and last unit)
                if (left <= 0)
                    return false;
                w.next(p);
                tiles = w.run(p, left);
                at = 0;
            }
            r.t0 = (w.lo + at) * kTile;
            r.len = w.len;
            r.head = w.head;
            r.edge = value && r.t0 + kTile > w.ctx;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r.page[h] = __ldg(p.block_table + w.b * p.table_stride +
                                  div_by_magic(min(r.t0 + w32 + 16 * h, (w.len - 1) & ~15), p.page_div));
            ++at;
            return true;
        };
        // a group of 16 tokens lies in one page; groups past the end read the last one
        auto find_groups = [&](const TileRef& r, int64_t* group) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = min(r.t0 + w32 + 16 * h, (r.len - 1) & ~15);
                const int off = t - static_cast<int>(div_by_magic(t, p.page_div)) * p.cache.page_size;
                const int pg = min(max(r.page[h], 0), static_cast<int>(p.cache.pages - 1));
                group[h] = (static_cast<int64_t>(pg) * p.cache.heads + r.head) * p.cache.page_size + off;
            }
        };
        constexpr int AHEAD = C::AHEAD;  // tiles whose codes are in registers or on their way
        uint4 raw[AHEAD][C::CH];
        uint32_t sc[AHEAD][C::CH];
        bool have[AHEAD], edge[AHEAD];
        int64_t group[2];  // of the tile to load next
        TileRef r = {};
        bool look = look_up(r);  // the tile looked up
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            have[k] = look;
            edge[k] = r.edge;
            if (look) {
                find_groups(r, group);
#pragma unroll
                for (int i = 0; i < C::CH; ++i) {
                    const int64_t from = group[(i * TPI) >> 4] + ((i * TPI) & 15);
                    sc[k][i] = __ldg(scales + from * C::SB);
                    raw[k][i] = __ldg(reinterpret_cast<const uint4*>(codes + from * C::ROW));
                }
                look = look_up(r);
            }
        }
        bool loads = look, edge_next = r.edge;
        if (look) {
            find_groups(r, group);
            look = look_up(r);
        }
        // converts the tile in raw[k] into the buffers f and starts the loads of the
        // tile AHEAD after it
        auto convert = [&](auto slot, uint32_t f, uint32_t ph) -> bool {
            constexpr int k = decltype(slot)::value;
            ok = mbar_wait_bounded(&freed[f], ph, p.status, kStatusTimeout, limit);
            if (!__all_sync(0xFFFFFFFFu, ok))
                return false;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < C::CH; ++i)
                top = max(top, sc[k][i]);
            // multipliers: in range for all but blocks of very large values and NaN; NaN
            // values of an edge tile are kept out of the product (see the softmax)
            constexpr uint32_t PLUS = (kFmt == kKvMxfp8 ? 120u : 126u) - kScaleShift;
            if (__any_sync(0xFFFFFFFFu, top > 254u - PLUS)) {
#pragma unroll
                for (int i = 0; i < C::CH; ++i)
                    sc[k][i] = edge[k] && sc[k][i] == 0xFFu ? 0u : block_multiplier<kFmt>(sc[k][i]) * 0x10001u;
            } else {
#pragma unroll
                for (int i = 0; i < C::CH; ++i)
                    sc[k][i] = sc[k][i] * 0x00800080u + PLUS * 0x00800080u;
            }
            const uint32_t buf = f * C::SLABS * kSlab;
#pragma unroll
            for (int i = 0; i < C::CH; ++i) {
                const uint32_t c4[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
                const uint32_t mul = sc[k][i];
                // the token's place in its group of 8 turns the pieces: of it, i decides
                // the bits from TPI up
                const uint32_t turn = ((i * TPI) & 7) << 4, down = i * TPI * 128;
#pragma unroll
                for (int h = 0; h < PIECES; ++h) {
                    uint32_t o[4];
                    if constexpr (kFmt == kKvMxfp8) {
                        place_codes<kFmt>(c4[2 * h], o);
                        place_codes<kFmt>(c4[2 * h + 1], o + 2);
                    } else {
                        place_codes<kFmt>(c4[h], o);
                    }
                    st_shared_v4(((at_piece[h] + buf) ^ turn) + down, mul_bf16x2(o[0], mul), mul_bf16x2(o[1], mul),
                                 mul_bf16x2(o[2], mul), mul_bf16x2(o[3], mul));
                }
                if (loads) {
                    const int64_t from = group[(i * TPI) >> 4] + ((i * TPI) & 15);
                    raw[k][i] = __ldg(reinterpret_cast<const uint4*>(codes + from * C::ROW));
                    sc[k][i] = __ldg(scales + from * C::SB);
                }
            }
            find_groups(r, group);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[f]);
            have[k] = loads;
            edge[k] = edge_next;
            loads = look;
            edge_next = r.edge;
            look = look && look_up(r);
            return true;
        };
        for (uint32_t g = 0;; g += 2) {
            const uint32_t ph = ((g >> 1) & 1u) ^ 1u;
            if (!have[0] || !convert(std::integral_constant<int, 0>(), 0, ph))
                break;
            constexpr int second = AHEAD > 1 ? 1 : 0;
            if (!have[second] || !convert(std::integral_constant<int, second>(), 1, ph))
                break;
        }
    } else {
        // --------------------------------------------------------- softmax
        set_registers<C::REGS_SOFTMAX>();
        // the two halves of the rows go their own ways within a unit
        const int quad = warp & 3, half = warp >> 2, col0 = half * C::COLS;
        const int token = quad * 32 + lane;  // of the tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        constexpr int CW = C::COLS == 32 ? 32 : 16;  // columns at a time
        const float2 xs = make_float2(p.xscale, p.xscale);
        auto load_cols = [&](uint32_t addr, uint32_t* r) {
            if constexpr (CW == 32)
                tmem_ld_32x32b_x32(addr, r);
            else
                tmem_ld_32x32b_x16(addr, r);
        };
        // a half's memory for moving its references: with 128 rows its own part of
        // P^T's buffer
        auto scratch = [&](uint8_t* pbuf) {
            return reinterpret_cast<float*>(NR == 128 ? pbuf + half * kSlab : smem + C::OFF_SCRATCH + half * 5 * C::COLS * 4);
        };
        // the current unit stays in shared memory: one thread moves it on
        Walk<NR>& wk = *reinterpret_cast<Walk<NR>*>(smem + C::OFF_WALK + 64);
        uint32_t g = 0;
        bool leave = false;
        for (int64_t left = count; left > 0 && !leave;) {
            const int tiles = wk.run(p, left);
            if (tiles == 0) {
                named_barrier_sync(5, kSoftmaxWarps * 32);  // everyone has read the unit
                if (threadIdx.x == 0 && left > 0)
                    wk.next(p);
                named_barrier_sync(5, kSoftmaxWarps * 32);
                continue;
            }
            const int head = wk.head, row0 = wk.row0(), n = wk.n, ctx = wk.ctx, len = wk.len, b = wk.b;
            const int q_start = wk.q_start, lo = wk.lo;
            const int rows = min(NR, n * p.group - row0);

            // Q, in the stored order of a head's elements; fresh references
            for (int i = threadIdx.x; i < NR * (kDim / 8); i += kSoftmaxWarps * 32) {
                const int r = i / (kDim / 8), c = i - r * (kDim / 8);
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) {
                    const int node = static_cast<int>(div_by_magic(row0 + r, p.group_div));
                    q = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(q_start + node) * p.qt +
                                                        static_cast<int64_t>(head * p.group + row0 + r - node * p.group) * p.qh +
                                                        c * 8);
                }
                const uint4 o = kFmt == kKvMxfp8
                                    ? make_uint4(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.x, q.y, 0x7632),
                                                 __byte_perm(q.z, q.w, 0x5410), __byte_perm(q.z, q.w, 0x7632))
                                    : make_uint4(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632),
                                                 __byte_perm(q.y, q.w, 0x5410), __byte_perm(q.y, q.w, 0x7632));
                *reinterpret_cast<uint4*>(smem + (c >> 3) * (NR * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = o;
            }
            for (int i = threadIdx.x; i < NR; i += kSoftmaxWarps * 32) {
                ref[i] = -kUnset;
                poison[i] = 0u;
            }
            fence_proxy_async_smem();
            named_barrier_sync(5, kSoftmaxWarps * 32);
            if (lane == 0) {
                mbar_arrive(&s_ready[g & 1u]);
                if (tiles > 1)
                    mbar_arrive(&s_ready[(g + 1u) & 1u]);
            }
            float l[C::COLS];
#pragma unroll
            for (int c = 0; c < C::COLS; ++c)
                l[c] = 0.0f;

            for (int it = 0; it < tiles; ++it, ++g) {
                const uint32_t f = g & 1u, ph = (g >> 1) & 1u;
                const int t = (lo + it) * kTile + token;
                const bool edge = (lo + it + 1) * kTile > ctx;
                const uint32_t s_addr = tmem + lanes + f * NR + col0;
                uint8_t* pbuf = smem + C::OFF_P + f * C::P_SLABS * kSlab;
                const int j = t - ctx;
                // edge tiles: which of the thread's rows see its token, a node (drafted
                // token, `group` rows) at a time
                uint64_t vis = 0;
                if (edge) {
                    const int from = row0 + col0;  // of the head's rows
                    if (j < 0) {
                        vis = ~uint64_t(0);
                    } else if (j < n && p.mask == nullptr) {
                        const int c = max(j * p.group - from, 0);  // nodes from j on
                        vis = c < C::COLS ? ~uint64_t(0) << c : 0;
                    } else if (j < n && (j >> 5) < p.mask_words) {
                        int node = static_cast<int>(div_by_magic(from, p.group_div));
                        const uint32_t* word = p.mask + static_cast<int64_t>(q_start + node) * p.mask_words + (j >> 5);
#pragma unroll 4
                        for (int c = node * p.group - from; c < C::COLS && node < n; c += p.group, ++node) {
                            const uint64_t bit = (__ldg(word) >> (j & 31)) & 1u;
                            const int end = min(c + p.group, 64), begin = max(c, 0);
                            const uint64_t run = (end == 64 ? ~uint64_t(0) : (uint64_t(1) << end) - 1) >> begin << begin;
                            vis |= bit ? run : 0;
                            word += p.mask_words;
                        }
                    }
                }
                const uint32_t vis_lo = static_cast<uint32_t>(vis), vis_hi = static_cast<uint32_t>(vis >> 32);
                // the scores' weights into P^T's buffer and the rows' sums; returns whether
                // one is above 2^kSlack.  Edge tiles have code of their own (a branch per
                // score would keep the compiler from overlapping them).
                auto weigh = [&](auto masked, float2 sign) {
                    uint32_t top = 0u;
                    uint32_t sb[2][CW];
                    load_cols(s_addr, sb[0]);
#pragma unroll
                    for (int c = 0; c < C::COLS; c += CW) {
                        uint32_t* s = sb[c / CW & 1];
                        tmem_ld_wait();
                        if (c + CW < C::COLS)
                            load_cols(s_addr + c + CW, sb[(c / CW + 1) & 1]);
                        uint32_t w[CW / 2];
#pragma unroll
                        for (int k = 0; k < CW; k += 4) {
                            const float4 r = *reinterpret_cast<const float4*>(ref + col0 + c + k);
                            float x[4], e[4];
                            fma_pair(x, __uint_as_float(s[k]), __uint_as_float(s[k + 1]), xs, r.x, r.y);
                            fma_pair(x + 2, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]), xs, r.z, r.w);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                // finite however far the score lies above its reference
                                e[h] = exp2_approx(min_nan(x[h], kCeiling));
                                if constexpr (decltype(masked)::value)
                                    e[h] = ((c + k + h < 32 ? vis_lo : vis_hi) >> ((c + k + h) & 31)) & 1u ? e[h] : 0.0f;
                            }
                            fma_pair(l + c + k, e[0], e[1], sign, l[c + k], l[c + k + 1]);
                            fma_pair(l + c + k + 2, e[2], e[3], sign, l[c + k + 2], l[c + k + 3]);
                            w[k / 2] = pack2(e[0], e[1]);
                            w[k / 2 + 1] = pack2(e[2], e[3]);
                            top = __vmaxu2(top, __vmaxu2(w[k / 2], w[k / 2 + 1]));
                        }
#pragma unroll
                        for (int h = 0; h < CW / 8; ++h) {
                            const int piece = (col0 + c) / 8 + h;
                            *reinterpret_cast<uint4*>(pbuf + (piece >> 3) * kSlab + token * 128 +
                                                      (((piece & 7) ^ (token & 7)) << 4)) =
                                make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
                        }
                    }
                    return max(top & 0xFFFFu, top >> 16) > kSlackBits;
                };
                ok = mbar_wait_bounded(&s_done[f], ph, p.status, kStatusTimeout, limit) && ok;
                // P^T's buffer is free when the tile before the last is in O^T
                ok = mbar_wait_bounded(&pv_done[f], ph ^ 1, p.status, kStatusTimeout, limit) && ok;
                __syncwarp();
                tc_fence_after_sync();
                auto tops = [&](auto masked, float* top) {
#pragma unroll
                    for (int c = 0; c < C::COLS; c += 16) {
                        uint32_t s[16];
                        tmem_ld_32x32b_x16(s_addr + c, s);
                        tmem_ld_wait();
                        float mine = 0.0f;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float x = __uint_as_float(s[k]) * p.xscale;
                            if constexpr (decltype(masked)::value)
                                x = ((c + k < 32 ? vis_lo : vis_hi) >> ((c + k) & 31)) & 1u ? x : -INFINITY;
                            x = warp_max(x);
                            mine = lane == k ? x : mine;
                        }
                        if (lane < 16)
                            top[quad * C::COLS + c + lane] = mine;
                    }
                };
                // Weigh the tile; if a weight is too large, take its weights back, move the
                // references to the rows' largest scores (per quadrant of tokens, by way of
                // P^T's buffer) and weigh it again.  The first tile starts with that.  (What
                // a sum loses by the subtraction is 2^-24 of the weight that made the
                // reference move, which stays in the sum.)
                enum { kFirst, kBack, kAgain };
#pragma unroll 1
                for (int step = it > 0 ? kFirst : kAgain;; ++step) {
                    if (step == kAgain) {
                        float* top = scratch(pbuf);  // [4][COLS]
                        float* factor = top + 4 * C::COLS;
                        named_barrier_sync(3 + half, 128);
                        if (edge)
                            tops(std::true_type(), top);
                        else
                            tops(std::false_type(), top);
                        named_barrier_sync(3 + half, 128);
                        const int r = threadIdx.x & 127;
                        if (r < C::COLS) {
                            const float old = -ref[col0 + r];
                            float now = fmaxf(fmaxf(top[r], top[C::COLS + r]), fmaxf(top[2 * C::COLS + r], top[3 * C::COLS + r]));
                            now = fmaxf(now, old);
                            factor[r] = exp2_approx(old - now);
                            ref[col0 + r] = -now;
                        }
                        named_barrier_sync(3 + half, 128);
                        if (it > 0) {
#pragma unroll
                            for (int c = 0; c < C::COLS; ++c)
                                l[c] *= factor[c];
                            ok = mbar_wait_bounded(&pv_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u, p.status, kStatusTimeout, limit) && ok;
                            __syncwarp();
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < C::COLS; c += 16) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(tmem_o + lanes + col0 + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[c + k]);
                                tmem_st_32x32b_x16(tmem_o + lanes + col0 + c, o);
                            }
                            tmem_st_wait();
                            named_barrier_sync(3 + half, 128);  // the factors have been read
                        }
                    }
                    const float2 sign = step == kBack ? make_float2(-1.0f, -1.0f) : make_float2(1.0f, 1.0f);
                    const bool grow = edge ? weigh(std::true_type(), sign) : weigh(std::false_type(), sign);
                    if (step == kAgain)
                        break;
                    if (step == kFirst) {
                        if (!ok)
                            gave_up[2 * half + f] = 1u;
                        __syncwarp();
                        const bool rescale = named_barrier_or(1 + half, 128, grow);
                        leave = gave_up[2 * half + f] != 0u;
                        if (leave || !rescale)
                            break;
                    }
                }
                if (leave)
                    break;  // all threads of the half at the same tile
                if (edge && t < len) {
                    // a NaN value reaches exactly the rows that see its token
                    const int pi = static_cast<int>(div_by_magic(t, p.page_div));
                    const int64_t pg = min(max(static_cast<int64_t>(__ldg(p.block_table + b * p.table_stride + pi)), int64_t(0)),
                                           p.cache.pages - 1);
                    const uint8_t* vs = p.cache.v_scales + ((pg * p.cache.heads + head) * p.cache.page_size +
                                                            (t - pi * p.cache.page_size)) * C::SB;
                    uint32_t bad = 0;
#pragma unroll
                    for (int k = 0; k < C::SB; ++k)
                        bad |= __ldg(vs + k) == 0xFFu ? 1u << k : 0u;
                    if (bad)
                        for (int c = 0; c < C::COLS; ++c)
                            if ((vis >> c) & 1u)
                                atomicOr(&poison[col0 + c], bad);
                }
                tc_fence_before_sync();
                fence_proxy_async_smem();
                __syncwarp();
                if (threadIdx.x == 0)
                    unit_start[f] = it == 0;
                if (lane == 0) {
                    mbar_arrive(&pv_ready[f]);
                    if (it + 2 < tiles)
                        mbar_arrive(&s_ready[f]);
                }
            }

            // --------------------------------------------------- results
            mbar_wait_bounded(&pv_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u, p.status, kStatusTimeout, limit);
            __syncwarp();
            tc_fence_after_sync();
            // the unit's MMAs have read their operands: [4][NR] sums go to Q's place,
            // the rows of each half to one of P^T's buffers
            float* sums = reinterpret_cast<float*>(smem);
            float* tile = reinterpret_cast<float*>(smem + C::OFF_P + (warp >> 2) * C::P_SLABS * kSlab);
            static_assert(C::COLS * kDim * 4 <= C::P_SLABS * kSlab, "a half's outputs in one buffer");
            // sums of the rows over the warp's tokens: each step sends half of the rows
            // away and adds the other half's, until a lane holds COLS / 32 rows (or two
            // lanes the same one)
#pragma unroll
            for (int d = 16, w = C::COLS / 2; d > 0; d >>= 1, w >>= 1) {
                if (w > 0) {
                    const bool up = lane & d;
#pragma unroll
                    for (int c = 0; c < w; ++c) {
                        const float send = up ? l[c] : l[c + w];
                        const float keep = up ? l[c + w] : l[c];
                        l[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, d);
                    }
                } else {
                    l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], d);
                }
            }
            {
                // the rows that the steps left: bit 4 of the lane chose the half, bit 3 the quarter, ...
                constexpr int PER = C::COLS >= 32 ? C::COLS / 32 : 1;
                const int r = C::COLS >= 32 ? lane * PER : lane >> 1;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    sums[quad * NR + col0 + r + c] = l[c];
            }
            {
                const int d = element_at<kFmt>(token);  // TMEM lane = position in the head
#pragma unroll 1
                for (int c = 0; c < C::COLS && col0 + c < rows; c += 16) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(tmem_o + lanes + col0 + c, o);
                    tmem_ld_wait();
                    if (token < kDim)
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            tile[(c + k) * kDim + d] = __uint_as_float(o[k]);
                }
            }
            tc_fence_before_sync();
            named_barrier_sync(5, kSoftmaxWarps * 32);
            // complete, or a part: of the unit that began before this run (slot 0), or of
            // the one that goes on after it (slot 1)
            const bool part = lo > 0 || tiles < wk.tiles;
            const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (lo > 0 ? 0 : 1)) * NR;
            for (int i = threadIdx.x; i < rows * (kDim / 8); i += kSoftmaxWarps * 32) {
                const int r = i / (kDim / 8), d = (i - r * (kDim / 8)) * 8;
                const float ls = sums[r] + sums[NR + r] + sums[2 * NR + r] + sums[3 * NR + r];
                const float m = ref[r] == -kUnset ? -INFINITY : -ref[r];
                const float* src = reinterpret_cast<const float*>(smem + C::OFF_P + (r >= C::COLS ? C::P_SLABS * kSlab : 0)) +
                                   (r >= C::COLS ? r - C::COLS : r) * kDim + d;
                const float4 u = *reinterpret_cast<const float4*>(src);
                const float4 v = *reinterpret_cast<const float4*>(src + 4);
                float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                const bool nan = (poison[r] >> (d >> 5)) & 1u;
                const float scale = nan    ? __uint_as_float(0x7FC00000u)
                                    : part ? kUnscale
                                           : (ls == 0.0f ? 0.0f : kUnscale * (1.0f / ls));
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] *= scale;
                if (!part) {
                    const int node = static_cast<int>(div_by_magic(row0 + r, p.group_div));
                    const int64_t tok = q_start + node;
                    const int hq = head * p.group + row0 + r - node * p.group;
                    *reinterpret_cast<uint4*>(p.out + tok * p.ot + hq * p.oh + d) =
                        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
                    if (d == 0 && p.lse != nullptr)
                        p.lse[tok * p.q_heads + hq] = (m + log2f(ls)) * 0.69314718055994531f;
                } else {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (slot + r) * kDim + d);
                    dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                    dst[1] = make_float4(x[4], x[5], x[6], x[7]);
                    if (d == 0)
                        *reinterpret_cast<float2*>(p.part_ml + (slot + r) * 2) = make_float2(m, ls);
                }
            }
            // Q's and P^T's places and the unit may be written again
            named_barrier_sync(5, kSoftmaxWarps * 32);
            if (left > 0) {
                if (threadIdx.x == 0)
                    wk.next(p);
                named_barrier_sync(5, kSoftmaxWarps * 32);
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the parts of the rows whose unit fell to several CTAs.
template <int kDim, int NR, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_attention_tile_join_kernel(const AttnParams p)
{
    __shared__ JoinScratch<kDim, kJoinWarps> scratch;
    grid_dependency_wait();
    launch_dependents();
    const int64_t row = blockIdx.x;
    const int tok = static_cast<int>(row / p.q_heads);
    const int hq = static_cast<int>(row - static_cast<int64_t>(tok) * p.q_heads);
    Walk<NR> w;
    w.b = sequence_of(p, tok);
    w.sequence(p);
    const int head = hq / p.group;
    const int r = (tok - w.q_start) * p.group + hq - head * p.group;  // of the head's rows
    if (tok < w.q_start || tok >= w.q_start + w.n || r >= w.row_tiles * NR)
        return;
    const int64_t per = p.prefix[p.batch];
    const int64_t from = p.prefix[w.b] + static_cast<int64_t>(head * w.row_tiles + r / NR) * (w.tiles + kUnitTiles) +
                         kUnitTiles;
    const int c0 = static_cast<int>(from / per), c1 = static_cast<int>((from + w.tiles - 1) / per);
    if (c0 == c1)
        return;  // written by its CTA
    join_row<kDim, kJoinWarps>(p, &scratch, tok, hq, c1 - c0 + 1, [&](int s) -> int64_t {
        return (2 * static_cast<int64_t>(c0) + (s == 0 ? 1 : 2 * s)) * NR + r % NR;
    });
}

template <int kFmt, int kDim, int NR>
cudaError_t launch_tile(const AttnParams& p, cudaStream_t stream)
{
    using C = TileCfg<kFmt, kDim, NR>;
    auto kern = kv_attention_tile_kernel<kFmt, kDim, NR>;
    // per device and context, once: the shared-memory opt-in and the register split
    static std::mutex mu;
    static unsigned long long configured[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= 64)
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (err != cudaSuccess)
                return err;
            // setmaxnreg.inc waits until the registers it asks for are free: never
            // launch a split that the launch's allocation cannot cover
            cudaFuncAttributes fa;
            err = cudaFuncGetAttributes(&fa, kern);
            if (err != cudaSuccess)
                return err;
            if (fa.numRegs * kThreads < C::REGS)
                return cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
        }
    }
    err = launch_pdl(kern, dim3(static_cast<unsigned>(sm_count())), dim3(kThreads), C::SMEM, stream, p);
    if (err != cudaSuccess || p.whole)
        return err;
    // parts per unit: about the runs over the units
    const bool few = 4 * static_cast<int64_t>(p.batch) * p.cache.heads * p.row_tiles >= sm_count();
    return launch_pdl(few ? kv_attention_tile_join_kernel<kDim, NR, 1> : kv_attention_tile_join_kernel<kDim, NR, 4>,
                      dim3(static_cast<unsigned>(p.T) * p.q_heads), dim3(few ? 32 : 128), 0, stream, p);
}

template <int kFmt, int kDim>
cudaError_t launch_rows(const AttnParams& p, int rows, cudaStream_t stream)
{
    return rows == 32   ? launch_tile<kFmt, kDim, 32>(p, stream)
           : rows == 64 ? launch_tile<kFmt, kDim, 64>(p, stream)
                        : launch_tile<kFmt, kDim, 128>(p, stream);
}

}  // namespace

// Two partial results per CTA, and the sequences' first tiles.
size_t kv_attention_tile_workspace(int rows, int dim, int batch)
{
    return static_cast<size_t>(2 * sm_count()) * rows * (dim + 2) * sizeof(float) + (static_cast<size_t>(batch) + 2) / 2 * 16;
}

cudaError_t launch_kv_attention_tile(const AttnParams& params, int rows, void* workspace, cudaStream_t stream)
{
    AttnParams p = params;
    p.xscale *= kUnscale;  // scores come out of the MMA times 2^-64
    const size_t part_rows = static_cast<size_t>(2 * sm_count()) * rows;
    p.prefix = static_cast<int64_t*>(workspace);
    p.part_o = reinterpret_cast<float*>(p.prefix + (params.batch + 2) / 2 * 2);
    p.part_ml = p.part_o + part_rows * p.cache.dim;
    if (p.cache.format == kKvMxfp8)
        return p.cache.dim == 128 ? launch_rows<kKvMxfp8, 128>(p, rows, stream)
                                  : launch_rows<kKvMxfp8, 64>(p, rows, stream);
    return p.cache.dim == 128 ? launch_rows<kKvMxfp4, 128>(p, rows, stream) : launch_rows<kKvMxfp4, 64>(p, rows, stream);
}

}  // namespace fp4lin
