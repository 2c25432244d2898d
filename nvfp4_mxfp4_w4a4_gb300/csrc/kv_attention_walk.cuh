// kv_attention_walk.cuh -- what the two tensor-core attention kernels share
// (kv_attention_tile.cu and kv_attention_rows.cu): the cut of the work into
// runs of 128-token tiles, the warps that convert a run's codes to bf16 tiles
// in shared memory, and the kernel that joins the parts of a row.
//
// The work is cut on the device: the tiles of all (sequence, key/value head,
// row tile) units in one line, with a few places for each unit's start and end,
// an equal run of the line per CTA, one CTA per SM.
// A unit whose tiles fall to several CTAs leaves partial results (a CTA has at
// most two: of the unit that began before its run and of the one that goes on
// after it), which the join kernel adds.  With a grid of equal chunks instead,
// the last round of CTAs and every CTA's start and end cost as much as the
// tiles (8 trees of 31 tokens over up to 16001 tokens of MXFP4, tiles of 1.8 us:
// 139 us against 113).
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "kv_attention.cuh"
#include "ptx.cuh"

namespace fp4lin {

constexpr int kTile = 128;  // tokens
constexpr int kSlab = kTile * 128;  // bytes of 64 bf16 elements of 128 tokens (or rows)
constexpr int kSoftmaxWarps = 8;    // then 4 converting keys, 4 values, 4 (of which 2 issue MMAs)
constexpr int kThreads = (kSoftmaxWarps + 8 + 4) * 32;
constexpr int kLaunchRegs = 96;  // per thread, which setmaxnreg deals out anew
// The work line: a unit is kUnitTiles places (its start and end cost about as
// much as five to nine tiles: 8 trees of 31 tokens over up to 16001, MXFP4, 98 /
// 79 / 79 / 79 us with 3 / 5 / 7 / 9 places; 64 sequences of 8 tokens over 4000,
// MXFP8, 158 / 158 / 161 / 161 us) and then its tiles.
constexpr int kUnitTiles = 5;
constexpr int kLeastRun = kUnitTiles + 4;
// a row's reference before its first visible token: the lowest float32, which no score lies under
constexpr float kUnset = -3.402823466e38f;

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

// The calling warpgroup's registers per thread, from kLaunchRegs.
template <int kRegs>
__device__ __forceinline__ void set_registers()
{
    if constexpr (kRegs > kLaunchRegs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else if constexpr (kRegs < kLaunchRegs)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Element that is stored at position `pos` of a head.
template <int kFmt>
__device__ __forceinline__ int element_at(int pos)
{
    return kFmt == kKvMxfp8 ? (pos & ~3) | ((pos & 1) << 1) | ((pos >> 1) & 1) : (pos & ~7) | ((pos & 1) << 2) | ((pos >> 1) & 3);
}

// One unit after the other: its sequence, head, first row and tiles.
template <int kRows>
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
        row_tiles = (rows(p) + kRows - 1) / kRows;
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
    // of a key head: those of the drafted tokens within the bound
    __device__ __forceinline__ int rows(const AttnParams& p) const { return min(n, p.max_draft) * p.group; }
    __device__ __forceinline__ int row0() const { return (unit - head * row_tiles) * kRows; }
};

// Copies of a CTA's place in its run: the softmax's and each converting warp's.
constexpr int kWalks = 1 + 8;
template <int kRows>
struct alignas(64) Place {
    Walk<kRows> walk;
};

// This CTA's run: its places on the line (units, with p.whole: units instead of
// tiles are dealt out then, and none is cut), where it starts and its tiles.
// All threads call it; `scratch` is free afterwards.
template <int kRows>
__device__ __forceinline__ int64_t find_run(const AttnParams& p, uint8_t* scratch, Place<kRows>* places, uint32_t* tiles)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    struct Scan {
        int64_t warp_sum[kThreads / 32];
        int64_t offset;
        int b;
    };
    Scan* scan = reinterpret_cast<Scan*>(scratch);
    auto weight = [&](int i) -> int64_t {
        if (i >= p.batch)
            return 0;
        Walk<kRows> w;
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
    const int64_t count = min(per, total - start);
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
        return 0;
    if (threadIdx.x == 0) {
        Walk<kRows> w;
        w.b = scan->b;
        w.sequence(p);
        const int64_t off = scan->offset;
        const int length = p.whole ? 1 : w.tiles + kUnitTiles;
        w.unit = static_cast<int>(off / length);
        w.head = w.unit / w.row_tiles;
        const int in_unit = static_cast<int>(off - static_cast<int64_t>(w.unit) * length);
        w.lead = max(kUnitTiles - in_unit, 0);
        w.lo = p.whole ? 0 : max(in_unit - kUnitTiles, 0);
        for (int i = 0; i < kWalks; ++i)
            places[i].walk = w;
        uint32_t total = 0;
        for (int64_t left = count; left > 0; w.next(p))
            total += w.run(p, left);
        *tiles = total;
    }
    __syncthreads();
    return count;
}

// A tile for the converters.
struct TileRef {
    int t0, len, head, page[2];
    bool edge;  // (values) not all its tokens are context
};

// Warps 8-15: the run's codes -> double-buffered bf16 tiles, K and V token by
// token (slabs of 64 elements, 16-byte pieces turned by the token: the 128-byte
// swizzle).  AHEAD: tiles whose codes are in registers or on their way.
// The walk is in shared memory: registers are short.
template <int kFmt, int kDim, int kRows, int AHEAD>
__device__ __forceinline__ void convert_run(const AttnParams& p, Walk<kRows>& w, int64_t count, uint8_t* k_tiles,
                                            uint8_t* v_tiles, uint64_t* full, uint64_t* freed)
{
    constexpr int SLABS = kDim / 64;
    constexpr int ROW = kFmt == kKvMxfp8 ? kDim : kDim / 2;
    constexpr int CH = ROW / 16;  // 16-byte chunks of a token's codes, one per lane
    constexpr int SB = kDim / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // 16-byte chunks of the codes, one per lane.  Eight lanes in a row store to
    // one slab, for tokens whose swizzles differ, so that their 16-byte pieces
    // fall in different banks.
    const bool value = warp >= kSoftmaxWarps + 4;
    const int w32 = (warp & 3) * 32;              // this warp's tokens of the tile
    constexpr int TPI = 32 / CH;               // tokens per load
    constexpr int HC = CH / SLABS;          // chunks of a token per slab
    const int chunk = ((lane >> 3) % SLABS) * HC + lane % HC;
    const int sub = (lane >> 3) / SLABS * (8 / HC) + lane / HC % (8 / HC);
    const uint8_t* codes = (value ? p.cache.v_codes : p.cache.k_codes) + sub * ROW + chunk * 16;
    const uint8_t* scales =
        (value ? p.cache.v_scales : p.cache.k_scales) + sub * SB + (kFmt == kKvMxfp8 ? chunk / 2 : chunk);
    // where the lane's 16-byte pieces of its first token go
    constexpr int PIECES = kFmt == kKvMxfp8 ? 2 : 4;
    uint32_t at_piece[PIECES];
#pragma unroll
    for (int h = 0; h < PIECES; ++h) {
        const int piece = PIECES * chunk + h;
        at_piece[h] = smem_u32(value ? v_tiles : k_tiles) + (piece >> 3) * kSlab + (w32 + sub) * 128 +
                      (((piece & 7) ^ (sub & 7)) << 4);
    }
    // The run's tiles in order: a tile's pages are looked up three tiles ahead, its
    // tokens' places found two ahead, its codes loaded one ahead.
    int64_t left = count;
    int tiles = w.run(p, left), at = 0;  // of the unit that the look-up is in
    auto look_up = [&](TileRef& r) -> bool {
        while (at == tiles) {  // (a run may hold no tile of its first and last unit)
            if (left <= 0)
                return false;
            __syncwarp();
            if (lane == 0)
                w.next(p);
            __syncwarp();
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
    // raw, sc: tiles whose codes are in registers or on their way
    uint4 raw[AHEAD][CH];
    uint32_t sc[AHEAD][CH];
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
            for (int i = 0; i < CH; ++i) {
                const int64_t from = group[(i * TPI) >> 4] + ((i * TPI) & 15);
                sc[k][i] = __ldg(scales + from * SB);
                raw[k][i] = __ldg(reinterpret_cast<const uint4*>(codes + from * ROW));
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
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&freed[f], ph, p.status, kStatusTimeout, p.wait_ns)))
            return false;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            top = max(top, sc[k][i]);
        // multipliers: in range for all but blocks of very large values and NaN; NaN
        // values of an edge tile are kept out of the product (see the softmax)
        constexpr uint32_t PLUS = (kFmt == kKvMxfp8 ? 120u : 126u) - kScaleShift;
        if (__any_sync(0xFFFFFFFFu, top > 254u - PLUS)) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                sc[k][i] = edge[k] && sc[k][i] == 0xFFu ? 0u : block_multiplier<kFmt>(sc[k][i]) * 0x10001u;
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                sc[k][i] = sc[k][i] * 0x00800080u + PLUS * 0x00800080u;
        }
        const uint32_t buf = f * SLABS * kSlab;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
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
                raw[k][i] = __ldg(reinterpret_cast<const uint4*>(codes + from * ROW));
                sc[k][i] = __ldg(scales + from * SB);
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
}

// Joins the parts of the rows whose unit fell to several CTAs: four warps for a
// row with many parts, one where most rows have a few.  Those rows' look-ups set
// the time, not the bytes, so all of them should be resident at once: 8 rows a
// CTA and 32 registers, 64 rows per SM (32 trees of 31 tokens x 4 heads over up
// to 2000 tokens of MXFP4: 70 us with the join; a CTA per row, 32 rows per SM, 84).
constexpr int kJoinRows = 8;

template <int kDim, int kRows, bool kFew>
__global__ void __launch_bounds__(kFew ? kJoinRows * 32 : 128, 8) kv_attention_run_join_kernel(const AttnParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t row = kFew ? static_cast<int64_t>(blockIdx.x) * kJoinRows + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= static_cast<int64_t>(p.T) * p.q_heads)
        return;
    const int tok = static_cast<int>(row / p.q_heads);
    const int hq = static_cast<int>(row - static_cast<int64_t>(tok) * p.q_heads);
    Walk<kRows> w;
    w.b = sequence_of(p, tok);
    w.sequence(p);
    if (tok < w.q_start || tok - w.q_start >= min(w.n, p.max_draft))
        return;
    const int head = hq / p.group;
    const int r = (tok - w.q_start) * p.group + hq - head * p.group;  // of the head's rows
    const int64_t per = p.prefix[p.batch];
    const int64_t from = p.prefix[w.b] + static_cast<int64_t>(head * w.row_tiles + r / kRows) * (w.tiles + kUnitTiles) +
                         kUnitTiles;
    const int c0 = static_cast<int>(from / per), c1 = static_cast<int>((from + w.tiles - 1) / per);
    if (c0 == c1)
        return;  // written by its CTA
    auto index = [&](int s) -> int64_t {
        return (2 * static_cast<int64_t>(c0) + (s == 0 ? 1 : 2 * s)) * p.part_rows + r % kRows;
    };
    if constexpr (kFew) {
        join_row_warp<kDim>(p, tok, hq, c1 - c0 + 1, index);
    } else {
        __shared__ JoinScratch<kDim, 4> scratch;
        join_row<kDim, 4>(p, &scratch, tok, hq, c1 - c0 + 1, index);
    }
}

// Launches a kernel of runs, whose registers after setmaxnreg are `regs` in all,
// and the join.
template <typename Kernel, Kernel kern, int kDim, int kRows>
cudaError_t launch_runs(const AttnParams& p, int smem, int regs, cudaStream_t stream)
{
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
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (err != cudaSuccess)
                return err;
            // setmaxnreg.inc waits until the registers it asks for are free: never
            // launch a split that the launch's allocation cannot cover
            cudaFuncAttributes fa;
            err = cudaFuncGetAttributes(&fa, kern);
            if (err != cudaSuccess)
                return err;
            if (fa.numRegs * kThreads < regs)
                return cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
        }
    }
    err = launch_pdl(kern, dim3(static_cast<unsigned>(sm_count())), dim3(kThreads), smem, stream, p);
    if (err != cudaSuccess || p.whole)
        return err;
    // parts per unit: about the runs over the units
    const bool few = 4 * static_cast<int64_t>(p.batch) * p.cache.heads * p.row_tiles >= sm_count();
    const unsigned rows = static_cast<unsigned>(p.T) * p.q_heads;
    return few ? launch_pdl(kv_attention_run_join_kernel<kDim, kRows, true>, dim3((rows + kJoinRows - 1) / kJoinRows),
                            dim3(kJoinRows * 32), 0, stream, p)
               : launch_pdl(kv_attention_run_join_kernel<kDim, kRows, false>, dim3(rows), dim3(128), 0, stream, p);
}

}  // namespace fp4lin
