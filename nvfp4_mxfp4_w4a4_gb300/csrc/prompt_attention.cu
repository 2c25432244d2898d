// prompt_attention.cu -- softmax attention over whole prompts: packed sequences of
// different lengths, grouped heads, causal or not, all in bf16, on the
// 5th-generation tensor cores.
//
//   S [rows x keys] = Q K^T,  P = exp2(S scale log2(e) - m),  O += P V
//
// A unit is two halves of up to 128 rows of a key/value head: a few tokens with
// the query heads that read it, side by side.  The halves' tiles of 128 keys take
// turns: while the MMAs of one half run, the other half's scores are weighed.  A
// softmax thread is one row: the tile's 128 scores are in its registers at once,
// maximum (a by-product of their load from tensor memory) and sum stay there, and
// the probabilities (bf16) go back to tensor memory over the scores.  The row's
// reference m moves only when a score passes it by 2^8, so most tiles leave O as
// it is.
//
// Only tiles in which some row sees not all keys are masked.  There the values
// get a look too: a weight of zero times NaN or Inf is NaN, so elements that are
// not finite leave the tile in shared memory and are added at the end to the rows
// that see them (rows past the last key of a sequence, which belong to other
// sequences or to nobody, go the same way).
//
// The work is cut on the device: the tiles of all units in one line, with a few
// places for each unit's start and end, an equal run of the line per CTA, one CTA
// per SM.  A unit whose tiles fall to several CTAs leaves partial results, which a
// second kernel joins.  Where all units are short, they are dealt out whole.
//
// 16381 tokens, 8 x 4 heads of 128, causal: 1265 to 1365 us (from GPU to GPU), 0.84 to
// 0.91 of the rate of a large bf16 product; the tensor pipe is busy 77 % of a run's
// cycles, the exponentials' 39 %.  Heads of 64: 1013 us, 0.57 of that rate (a tile's
// exponentials take as long as its products, so that neither hides the hand-over).  A
// chunk of 2048 tokens behind 14333 keys, heads of 128: 312 us (0.86), one of 512: 101
// (0.70).  16 sequences of up to 509 tokens, heads of 64: 38 us, 5 of them before the
// first unit's products; a unit of two tiles is load, S, weights, P V and results one
// behind the other, and a seventh of the time its warps wait for instructions.
//
// The weights go to the second product as bf16 (off by 2^-8 of each at most, their sum is
// of the unrounded ones): its operands have one type, the values are bf16, and f16
// values would lose their range.  A second product with what the rounding leaves would
// be half as many operations again in a kernel that the tensor pipe bounds.
//
// Warps: 0-3 and 4-7 the softmax of the halves (they also write the results), 8
// loads queries, keys and values (TMA), 9 issues the MMAs, 10 looks through values
// and sees to their loads, 11 goes over the run's units, a few ahead.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kHalf = 128;           // rows of a half, at most
constexpr int kRows = 2 * kHalf;     // of a unit
constexpr int kTile = 128;           // keys of a tile
constexpr int kSlab = 128 * 128;     // bytes of 64 bf16 elements of 128 rows or keys
constexpr int kThreads = 384;
// places of a unit's start and end on the line (2 to 5: 38.2 / 37.4 / 37.4 / 39.6 us for the short
// prompts above, 1305 to 1313 for the long one)
constexpr int kUnitPlaces = 3;
constexpr int kLeastRun = kUnitPlaces + 4;
// units of at most so many tiles are never cut (the long prompt uncut: 1379 us against 1311; the
// short ones cut: 39.0 us against 37.4, 36.5 without the join's launch; one prompt of 1000 tokens
// with fewer units than there are SMs, 1 / 2 / 8 key heads x 4 of 128, 17.9 / 18.1 / 20.2 us
// whole, 21.7 / 22.0 / 23.9 cut, with 4 of 64 17.1 and 21.2 for 8 key heads)
constexpr int kWholeTiles = 8;
constexpr int kParts = 4;            // of the run whose descriptions are in shared memory
constexpr int kWarpSequences = 96;   // up to so many sequences, a warp adds one up
constexpr float kSlack = 8.0f;       // a score this far above its reference moves it
// a row's reference before its first seen key: the lowest float32, which no score lies under
constexpr float kUnset = -3.402823466e38f;
// registers per thread: at launch, and dealt out anew to the softmax and the others
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 184, kOtherRegs = 128;
constexpr int kAllRegs = 256 * kSoftmaxRegs + 128 * kOtherRegs;
static_assert(kAllRegs <= kLaunchRegs * kThreads, "register split");

// What a CTA leaves to the join: whether its run begins within a unit that goes on
// behind it, and the unit that begins in it and goes on.
struct Cut {
    int through;
    int open;
    int b, head, block;
    int pad[3];
};

struct PromptParams {
    PromptArgs a;
    int heads;      // query heads of a half's token: all of a key head's, or 128 of them
    int chunks;     // such groups of a key head
    int tokens;     // of a half
    DivMagic heads_div;
    float xscale;   // scale * log2(e)
    float* part_o;  // [CTA][2][half][dim / 4][kHalf][4]
    float2* part_ml;  // [CTA][2][half][kHalf]
    Cut* cuts;      // [CTA]
    bool may_cut;
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// d[0..1] = a[0..1] * m + c[0..1] in one instruction.
__device__ __forceinline__ void fma_pair(float* d, float a0, float a1, float2 m, float c)
{
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %6};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a0), "f"(a1), "f"(m.x), "f"(m.y), "f"(c));
}

__device__ __forceinline__ float2 add_pair(float2 a, float b0, float b1)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b0), "f"(b1));
    return r;
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

template <int kRegs>
__device__ __forceinline__ void set_registers()
{
    if constexpr (kRegs > kLaunchRegs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The rest of a bounded wait whose first look found the phase incomplete.
__device__ __forceinline__ bool wait_longer(uint32_t bar, uint32_t parity, unsigned int* status, uint64_t limit_ns)
{
    const uint64_t t0 = global_timer_ns();
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity))
                return true;
    } while (global_timer_ns() - t0 <= limit_ns);
    atomicOr(status, kStatusTimeout);
    return false;
}

// ---------------------------------------------------------------- the line

// A place on the line: one unit after the other, by sequence, key head and block
// of rows.
struct Walk {
    int b, head, block, blocks;  // head: key head and chunk; blocks of the sequence
    int q0, n, k0, m;

    __device__ __forceinline__ void sequence(const PromptParams& p)
    {
        group_rows(p.a.q_offsets, b, static_cast<int>(p.a.T), &q0, &n);
        group_rows(p.a.k_offsets, b, static_cast<int>(p.a.keys), &k0, &m);
        blocks = (n + 2 * p.tokens - 1) / (2 * p.tokens);
    }
    // Keys that query i of the sequence sees.  (n before m: n + m may pass 2^31)
    __device__ __forceinline__ int limit(const PromptParams& p, int i) const
    {
        return p.a.causal ? max(min(i + 1 - n + m, m), 0) : m;
    }
    __device__ __forceinline__ int tiles(const PromptParams& p, int half) const
    {
        const int i = (2 * block + half) * p.tokens;
        return i >= n ? 0 : (limit(p, min(i + p.tokens, n) - 1) + kTile - 1) / kTile;
    }
    __device__ __forceinline__ int tiles(const PromptParams& p) const { return max(tiles(p, 0), tiles(p, 1)); }
    __device__ __forceinline__ void next(const PromptParams& p)
    {
        if (++block < blocks)
            return;
        block = 0;
        if (++head < p.a.kv_heads * p.chunks)
            return;
        head = 0;
        blocks = 0;
        while (blocks == 0 && b + 1 < p.a.batch) {
            ++b;
            sequence(p);
        }
    }
};

// The units of a CTA's run, one part after the other: tiles [lo, hi) of the unit.
struct Run {
    Walk w;
    int64_t left;  // places to go (whole units: to the end of the units that begin in the run)
    int skip;      // places of the first unit that lie before the run
    int whole;
    int lo, hi, tiles;

    // The next part, or false at the end.  (w is the part's unit.)
    __device__ __forceinline__ bool part(const PromptParams& p, bool& started)
    {
        while (true) {
            if (started)
                w.next(p);
            started = true;
            if (left <= 0)
                return false;
            tiles = w.tiles(p);
            const int places = kUnitPlaces + tiles - skip;
            if (whole) {
                left -= places;
                const bool mine = skip == 0;
                skip = 0;
                lo = 0, hi = tiles;
                if (mine)
                    return true;
                continue;
            }
            lo = max(skip - kUnitPlaces, 0);
            const int lead = max(kUnitPlaces - skip, 0);
            const bool begins = skip == 0;
            hi = lo + static_cast<int>(max(min(left - lead, static_cast<int64_t>(tiles - lo)), int64_t(0)));
            left -= places;
            skip = 0;
            // (a unit without tiles belongs to the run that it begins in)
            if (hi > lo || (tiles == 0 && begins))
                return true;
        }
    }
};

// What find_run's threads tell one another.
struct Scan {
    int64_t weight[kWarpSequences];  // places of a sequence's key head
    int64_t warp_sum[kThreads / 32];
    int64_t offset, per_head;
    int longest[kThreads / 32];
    int b;
};

// This CTA's run; false if it has none.  All threads call it; `scan` is free
// afterwards.
__device__ bool find_run(const PromptParams& p, Scan* scan, Run* shared)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int batch = p.a.batch;
    const bool by_warp = batch <= kWarpSequences;
    auto places = [&](Walk& w, int first, int step) {
        int64_t sum = 0;
        for (w.block = first; w.block < w.blocks; w.block += step)
            sum += kUnitPlaces + w.tiles(p);
        return sum;
    };
    int longest = 0;
    if (by_warp) {
        for (int b = warp; b < batch; b += kWarps) {
            Walk w;
            w.b = b;
            w.sequence(p);
            int64_t sum = places(w, lane, 32);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            longest = max(longest, w.n > 0 ? (w.m + kTile - 1) / kTile : 0);
            if (lane == 0)
                scan->weight[b] = sum;
        }
        __syncthreads();
    }
    auto weight = [&](int i) -> int64_t {
        if (i >= batch)
            return 0;
        if (by_warp)
            return scan->weight[i];
        Walk w;
        w.b = i;
        w.sequence(p);
        longest = max(longest, w.n > 0 ? (w.m + kTile - 1) / kTile : 0);
        return places(w, 0, 1);
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
        for (int w = 0; w < kWarps; ++w) {
            base += w < warp ? scan->warp_sum[w] : 0;
            total += scan->warp_sum[w];
        }
        *before = base + x - v;
        return total;
    };
    const int heads = p.a.kv_heads * p.chunks;
    int64_t total = 0, before = 0, mine = 0;
    for (int i = 0; i < batch; i += kThreads) {
        mine = weight(i + threadIdx.x);
        total += block_scan(mine * heads, &before);
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if (lane == 0)
        scan->longest[warp] = longest;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
        longest = max(longest, scan->longest[w]);
    const int whole = !p.may_cut || longest <= kWholeTiles;
    // (a division of 32 bits where that is enough: those of 64 take some 100 instructions)
    const int64_t up = total + gridDim.x - 1;
    const int64_t share = up < (int64_t(1) << 32) ? static_cast<uint32_t>(up) / gridDim.x : up / gridDim.x;
    const int64_t per = max(share, int64_t(whole ? 1 : kLeastRun));
    const int64_t start = blockIdx.x * per;
    const int64_t count = min(per, total - start);
    int64_t base = 0;
    for (int i = 0; i < batch; i += kThreads) {
        if (batch > kThreads) {
            mine = weight(i + threadIdx.x);
            const int64_t sum = block_scan(mine * heads, &before);
            before += base;
            base += sum;
        }
        if (start >= before && start < before + mine * heads) {
            scan->b = i + threadIdx.x;
            scan->offset = start - before;
            scan->per_head = mine;
        }
    }
    __syncthreads();
    if (count <= 0)
        return false;
    if (warp == 0) {
        Run r;
        r.w.b = scan->b;
        r.w.sequence(p);
        const int64_t offset = scan->offset, per_head = scan->per_head;
        r.w.head = offset < (int64_t(1) << 32) ? static_cast<int>(static_cast<uint32_t>(offset) / static_cast<uint32_t>(min(per_head, offset + 1)))
                                               : static_cast<int>(offset / per_head);
        int64_t in_head = scan->offset - r.w.head * scan->per_head;
        // the block that the start falls into, 32 at a time
        int first = 0;
        while (true) {
            Walk w = r.w;
            w.block = first + lane;
            const int mine32 = w.block < w.blocks ? kUnitPlaces + w.tiles(p) : 0;
            int x = mine32;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                x += lane >= d ? y : 0;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, in_head < x);
            if (past != 0 || first + 32 >= w.blocks) {
                const int at = past != 0 ? __ffs(past) - 1 : 31;
                r.w.block = first + at;
                r.skip = static_cast<int>(in_head) - __shfl_sync(0xFFFFFFFFu, x - mine32, at);
                break;
            }
            in_head -= __shfl_sync(0xFFFFFFFFu, x, 31);
            first += 32;
        }
        r.left = count;
        r.whole = whole;
        r.lo = r.hi = r.tiles = 0;
        if (lane == 0)
            *shared = r;
    }
    __syncthreads();
    return true;
}

// ------------------------------------------------------------------ kernel

// A part of the run, as the warps see it.
struct alignas(16) Part {
    int lo, hi;      // tiles; lo < 0: the run has ended
    int end[2];      // the halves' own tiles end here
    int token;       // first query of the unit
    int tokens;      // of the sequence from there on
    int first_seen;  // keys seen by that query, before they are clamped to [0, m]
    int k0, m;       // the sequence's keys
    int key_head, q_head, q_heads;  // the chunk's first query head, and how many
    int slot;        // of the partial results, -1: the part is the whole unit
    int masked;      // first tile in which some row sees not all keys
};

template <int kDim>
struct Cfg {
    static constexpr int SLABS = kDim / 64;
    static constexpr int TILE = SLABS * kSlab;  // bytes of a tile of K or V, or of a half's Q
    static constexpr int STAGES = kDim == 128 ? 2 : 4;
    static constexpr int QBUFS = kDim == 128 ? 1 : 2;  // of a half's Q
    static constexpr int OFF_K = 2 * QBUFS * TILE;  // Q first
    static constexpr int OFF_V = OFF_K + STAGES * TILE;
    static constexpr int OFF_BAD = OFF_V + STAGES * TILE;  // int [2][3][kDim]: first keys whose value is inf, -inf, NaN
    static constexpr int OFF_OUT = OFF_BAD + 2 * 3 * kDim * 4;  // [8 warps] 32 elements of 32 rows
    static constexpr int OFF_BAR = OFF_OUT + 8 * 2048;
    static constexpr int BARS = 4 * STAGES + 4 * QBUFS + 2 * 6 + 2 * kParts + 1;
    static constexpr int OFF_SLOT = OFF_BAR + BARS * 8;  // TMEM address, flags
    static constexpr int OFF_RUN = (OFF_SLOT + 32 + 15) / 16 * 16;
    static constexpr int OFF_PARTS = OFF_RUN + 128;
    static constexpr int SMEM = OFF_PARTS + kParts * static_cast<int>(sizeof(Part)) + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = 512;  // S of the halves, then O
    static constexpr int TMEM_O = 2 * kTile;
    static_assert(sizeof(Run) <= 128 && sizeof(Scan) <= OFF_BAR - OFF_OUT, "");
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const PromptParams p, const __grid_constant__ CUtensorMap q_map,
                            const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map)
{
    using C = Cfg<kDim>;
    constexpr int STAGES = C::STAGES, QBUFS = C::QBUFS;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (by an offset, not a cast of the address: the compiler has to see shared memory)
    uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_full = bars;               // [STAGES] a tile has landed
    uint64_t* k_free = k_full + STAGES;    // [STAGES] both halves' products with it have ended
    uint64_t* v_full = k_free + STAGES;    // [STAGES]
    uint64_t* v_free = v_full + STAGES;    // [STAGES]
    uint64_t* q_full = v_free + STAGES;       // [QBUFS][2] by half
    uint64_t* q_free = q_full + 2 * QBUFS; // [QBUFS][2]
    uint64_t* s_full = q_free + 2 * QBUFS; // [2] scores are complete (and the tile before is in O)
    uint64_t* p_half = s_full + 2;         // [2] half the probabilities are in tensor memory, the values and the next keys have landed
    uint64_t* p_full = p_half + 2;         // [2] and the other half
    uint64_t* o_full = p_full + 2;         // [2] the part's last tile is in O
    uint64_t* bad_full = o_full + 2;       // [2] by part: its masked tiles are looked through
    uint64_t* bad_free = bad_full + 2;     // [2] and what was found is read
    uint64_t* part_full = bad_free + 2;    // [kParts] a part is described
    uint64_t* part_free = part_full + kParts;  // [kParts] and done with
    uint64_t* drained = part_free + kParts;    // every MMA has ended
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* any_bad = tmem_slot + 1;  // [2] by part
    Run* run = reinterpret_cast<Run*>(smem + C::OFF_RUN);
    volatile Part* parts = reinterpret_cast<Part*>(smem + C::OFF_PARTS);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_free[i], 1);
        }
        for (int i = 0; i < 2 * QBUFS; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_half[i], 4 + 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&bad_full[i], 1);
            mbar_init(&bad_free[i], 8);
            any_bad[i] = 0u;
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&part_full[i], 1);
            mbar_init(&part_free[i], 8 + 3);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    launch_dependents();
    // (in a place that no copy writes: nothing would order these writes before the copies')
    const bool have = find_run(p, reinterpret_cast<Scan*>(smem + C::OFF_OUT), run);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint64_t limit_ns = p.a.wait_ns;
    bool ok = true;
    // a wait of one thread, and one of a whole warp (quick where the phase is complete: a
    // few hundred cycles of serial code at every wait of the MMA warp would be time that
    // its products wait for); once one has run out, the role ends
    auto wait_one = [&](uint64_t* bar, uint32_t parity) {
        const uint32_t at = smem_u32(bar);
        if (!mbar_try_wait(at, parity & 1u))
            ok = ok && wait_longer(at, parity & 1u, p.a.status, limit_ns);
        return ok;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const uint32_t at = smem_u32(bar);
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(at, parity & 1u)))
            ok = __all_sync(0xFFFFFFFFu, ok && wait_longer(at, parity & 1u, p.a.status, limit_ns));
        return ok;
    };
    // the next part's description, or nullptr at the end of the run
    uint32_t part_count = 0;
    auto next_part = [&]() -> volatile Part* {
        const uint32_t i = part_count % kParts;
        if (!wait(&part_full[i], part_count / kParts) || parts[i].lo < 0)
            return nullptr;
        return &parts[i];
    };
    auto part_done = [&]() {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&part_free[part_count % kParts]);
        ++part_count;
    };

    if (warp >= 8) {
        set_registers<kOtherRegs>();
        if (!have) {
            if (p.may_cut && warp == 11 && lane == 0)
                p.cuts[blockIdx.x] = Cut{};
        } else if (warp == 11) {
            // -------------------------------------------------------- the run
            if (lane == 0) {
                Run r = *run;
                bool started = false;
                Cut cut = {};
                const int group = p.a.q_heads / p.a.kv_heads;
                while (true) {
                    const uint32_t i = part_count % kParts;
                    const bool more = r.part(p, started);
                    if (!wait_one(&part_free[i], (part_count / kParts) ^ 1u))
                        break;
                    volatile Part& d = parts[i];
                    if (!more) {
                        d.lo = -1;
                        mbar_arrive(&part_full[i]);
                        break;
                    }
                    const Walk& w = r.w;
                    const int key_head = p.chunks == 1 ? w.head : w.head / p.chunks, chunk = w.head - key_head * p.chunks;
                    const int first = 2 * w.block * p.tokens;
                    d.lo = r.lo, d.hi = r.hi;
                    d.end[0] = max(r.lo, min(r.hi, w.tiles(p, 0)));
                    d.end[1] = max(r.lo, min(r.hi, w.tiles(p, 1)));
                    d.token = w.q0 + first;
                    d.tokens = w.n - first;
                    d.first_seen = p.a.causal ? first + 1 - w.n + w.m : w.m;
                    d.k0 = w.k0, d.m = w.m;
                    d.key_head = key_head, d.q_head = key_head * group + chunk * kHalf;
                    d.q_heads = min(p.heads, group - chunk * kHalf);
                    d.slot = r.lo == 0 && r.hi == r.tiles ? -1 : r.lo > 0 ? 0 : 1;
                    d.masked = w.limit(p, first) / kTile;
                    mbar_arrive(&part_full[i]);
                    ++part_count;
                    if (r.hi < r.tiles) {
                        if (r.lo > 0)
                            cut.through = 1;
                        else
                            cut.open = 1, cut.b = w.b, cut.head = w.head, cut.block = w.block;
                    }
                }
                if (p.may_cut)
                    p.cuts[blockIdx.x] = cut;
            }
        } else if (warp == 8) {
            // ------------------------------------------ queries, keys and values
            uint32_t g = 0, queries[2] = {0, 0};  // tiles, and a half's Q, so far
            auto landed = [&](uint64_t* bar, uint32_t parity) { wait_longer(smem_u32(bar), parity, p.a.status, limit_ns); };
            while (volatile Part* d = next_part()) {
                const int lo = d->lo, hi = d->hi, key_head = d->key_head, q_head = d->q_head, token = d->token, k0 = d->k0;
                const int end[2] = {d->end[0], d->end[1]};
                for (int j = lo; ok && j < hi; ++j, ++g) {
                    const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1u;
                    if (!wait(&k_free[slot], phase ^ 1u))
                        break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&k_full[slot], C::TILE);
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
                            tma_load_3d(smem + C::OFF_K + slot * C::TILE + s * kSlab, &k_map, &k_full[slot], s * 64,
                                        k0 + j * kTile, key_head);
                    }
                    __syncwarp();
                    if (j == lo) {  // (the queries behind the first keys, whose place is free earlier)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (end[h] == lo)
                                continue;
                            const uint32_t buf = (queries[h] % QBUFS) * 2 + h;
                            if (!wait(&q_free[buf], (queries[h] / QBUFS) ^ 1u))
                                break;
                            ++queries[h];
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&q_full[buf], p.tokens * p.heads * kDim * 2);
#pragma unroll
                                for (int s = 0; s < C::SLABS; ++s)
                                    tma_load_3d(smem + buf * C::TILE + s * kSlab, &q_map, &q_full[buf], s * 64, q_head,
                                                token + h * p.tokens);
                            }
                            __syncwarp();
                        }
                    }
                    if (!ok || !wait(&v_free[slot], phase ^ 1u)) {
                        landed(&k_full[slot], phase);
                        break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&v_full[slot], C::TILE);
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
                            tma_load_3d(smem + C::OFF_V + slot * C::TILE + s * kSlab, &v_map, &v_full[slot], s * 64,
                                        k0 + j * kTile, key_head);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
                part_done();
            }
            // nothing of this CTA may be in flight when it ends
            for (uint32_t i = 1; i <= STAGES && i <= g; ++i) {
                const uint32_t slot = (g - i) % STAGES, phase = ((g - i) / STAGES) & 1u;
                landed(&k_full[slot], phase);
                landed(&v_full[slot], phase);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                for (uint32_t i = 1; i <= QBUFS && i <= queries[h]; ++i) {
                    const uint32_t use = queries[h] - i;
                    landed(&q_full[(use % QBUFS) * 2 + h], (use / QBUFS) & 1u);
                }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMAs
            // (the whole warp walks the loop and one elected lane issues: the operands
            // of the MMAs then stay in uniform registers.  One warp for both halves: their
            // products come one after the other, not both at half the rate, so that a half's
            // scores are weighed while the other's products run)
            constexpr uint32_t idesc_s = idesc_bf16(kHalf, kTile, 0, 0);
            constexpr uint32_t idesc_o = idesc_bf16(kHalf, kDim, 0, 1);
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t kd = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
            const uint64_t vd = smem_desc(smem_u32(smem + C::OFF_V), kSlab, 1024, 2);
            const bool withhold = p.a.withhold && blockIdx.x == 0;
            uint32_t g = 0, turns[2] = {0, 0}, queries[2] = {0, 0};
            while (volatile Part* d = next_part()) {
                // (by shuffles: what the MMAs' operands depend on has to be uniform for the compiler too)
                const int lo = uniform(d->lo), hi = uniform(d->hi);
                const int end[2] = {uniform(d->end[0]), uniform(d->end[1])};
                uint32_t buf[2] = {};
                // S of a half with the tile in a slot of K
                auto scores = [&](int h, uint32_t slot, bool last) {
                    const uint64_t q = qd + ((buf[h] * C::TILE) >> 4), k = kd + ((slot * C::TILE) >> 4);
#pragma unroll
                    for (int i = 0; i < kDim / 16; ++i) {
                        const uint64_t at = ((i >> 2) * kSlab + 32 * (i & 3)) >> 4;
                        tc_mma_f16(tmem + h * kTile, q + at, k + at, idesc_s, i != 0);
                    }
                    tc_commit(&s_full[h]);
                    if (last)
                        tc_commit(&q_free[buf[h]]);
                };
                // (the second half has the unit's last tile, unless it has no rows)
                const int closing = end[1] > lo ? 1 : 0;
                if (hi > lo && !wait(&k_full[g % STAGES], g / STAGES))
                    break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    buf[h] = (queries[h] % QBUFS) * 2 + h;
                    if (end[h] > lo) {
                        if (!wait(&q_full[buf[h]], queries[h]++ / QBUFS))
                            break;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            scores(h, g % STAGES, lo == end[h] - 1);
                            if (h == closing)
                                tc_commit(&k_free[g % STAGES]);
                        }
                        __syncwarp();
                    }
                }
                for (int j = lo; ok && j < hi; ++j, ++g) {
                    const uint32_t slot = g % STAGES, next = (g + 1) % STAGES;
                    const uint64_t v = vd + ((slot * C::TILE) >> 4);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (j >= end[h])
                            continue;
                        // half of the keys after the other, as their probabilities come
                        if (!wait(&p_half[h], turns[h]))
                            break;
                        tc_fence_after_sync();
                        if (elect_one() && !withhold) {
#pragma unroll
                            for (int i = 0; i < kTile / 32; ++i)
                                tc_mma_f16_ts(tmem + C::TMEM_O + h * kDim, tmem + h * kTile + 8 * i, v + ((2048 * i) >> 4),
                                              idesc_o, i != 0 || j != lo);
                        }
                        __syncwarp();
                        if (!wait(&p_full[h], turns[h]++))
                            break;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            if (!withhold) {
#pragma unroll
                                for (int i = kTile / 32; i < kTile / 16; ++i)
                                    tc_mma_f16_ts(tmem + C::TMEM_O + h * kDim, tmem + h * kTile + 8 * i, v + ((2048 * i) >> 4),
                                                  idesc_o, 1);
                                if (j == end[h] - 1)
                                    tc_commit(&o_full[h]);
                            }
                            if (j + 1 < end[h])
                                scores(h, next, j + 1 == end[h] - 1);
                            if (h == closing) {
                                tc_commit(&v_free[slot]);
                                if (j + 1 < hi)
                                    tc_commit(&k_free[next]);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (!ok)
                    break;
                part_done();
            }
            // whatever was issued has ended before tensor and shared memory go
            if (elect_one())
                tc_commit(drained);
            __syncwarp();
            wait_longer(smem_u32(drained), 0, p.a.status, limit_ns);
        } else if (warp == 10) {
            // -------------- what the second product of a tile needs beside P
            // its values, looked through where the tile is masked, and the next tile's keys:
            // one more arrival on its barrier, so that the MMA warp has fewer waits
            uint32_t g = 0, turns[2] = {0, 0};
            while (volatile Part* d = next_part()) {
                const int lo = d->lo, hi = d->hi, masked = d->masked;
                const int end[2] = {d->end[0], d->end[1]};
                const uint32_t par = part_count & 1u;
                if (!wait(&bad_free[par], (part_count >> 1) ^ 1u))
                    break;
                int* bad = reinterpret_cast<int*>(smem + C::OFF_BAD) + par * 3 * kDim;
                if (lane == 0)
                    any_bad[par] = 0u;
                bool cleared = false;
                for (int j = lo; j < hi; ++j, ++g) {
                    if (!wait(&v_full[g % STAGES], g / STAGES))
                        break;
                    if (j >= masked) {
                        uint8_t* v = smem + C::OFF_V + (g % STAGES) * C::TILE;
                        constexpr int PIECES = C::TILE / 16 / 32;
                        __nv_bfloat162 top = __float2bfloat162_rn(0.0f);
#pragma unroll 8
                        for (int i = 0; i < PIECES; ++i) {
                            const uint4 x = *reinterpret_cast<const uint4*>(v + (i * 32 + lane) * 16);
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])));
                        }
                        const bool found = !(__bfloat162float(top.x) < INFINITY && __bfloat162float(top.y) < INFINITY);
                        if (__any_sync(0xFFFFFFFFu, found)) {
                            if (!cleared) {
                                for (int i = lane; i < 3 * kDim; i += 32)
                                    bad[i] = 0x7FFFFFFF;
                                if (lane == 0)
                                    any_bad[par] = 1u;
                                cleared = true;
                            }
                            __syncwarp();
                            for (int i = 0; i < PIECES; ++i) {
                                const int piece = i * 32 + lane, in_slab = piece % (kSlab / 16), key = in_slab / 8;
                                const int d0 = piece / (kSlab / 16) * 64 + ((in_slab & 7) ^ (key & 7)) * 8;
                                uint16_t* e = reinterpret_cast<uint16_t*>(v + piece * 16);
                                for (int k = 0; k < 8; ++k) {
                                    if ((e[k] & 0x7F80u) != 0x7F80u)
                                        continue;
                                    const int kind = (e[k] & 0x7Fu) != 0u ? 2 : e[k] >> 15;
                                    atomicMin(&bad[kind * kDim + d0 + k], j * kTile + key);
                                    e[k] = 0;
                                }
                            }
                            fence_proxy_async_smem();
                            __syncwarp();  // (a vote orders no memory)
                        }
                    }
                    if (j + 1 < hi && !wait(&k_full[(g + 1) % STAGES], (g + 1) / STAGES))
                        break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (j >= end[h])
                            continue;
                        // (the half's tile before has to have all its arrivals)
                        if (!wait(&p_half[h], turns[h]++ ^ 1u))
                            break;
                        if (lane == 0)
                            mbar_arrive(&p_half[h]);
                    }
                    if (!ok)
                        break;
                }
                if (!ok)
                    break;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bad_full[par]);
                part_done();
            }
        }
    } else {
        // --------------------------------------------------------- softmax
        set_registers<kSoftmaxRegs>();
        const int h = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;  // of the half
        const int of_half = static_cast<int>(div_by_magic(row, p.heads_div));  // its token
        const int head = row - of_half * p.heads;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_addr = tmem + lanes + h * kTile, o_addr = tmem + lanes + C::TMEM_O + h * kDim;
        const float2 xs = make_float2(p.xscale, p.xscale);
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            tc_fence_after_sync();
            return ok;
        };
        uint32_t turns = 0, uses = 0;
        while (have) {
            volatile Part* d = next_part();
            if (d == nullptr)
                break;
            const int lo = d->lo, end = d->end[h];
            const int tok = h * p.tokens + of_half;  // of the unit
            // (rows without a query have no say in when their warp's references move, so that
            // nothing of them reaches the results)
            const bool live = of_half < p.tokens && tok < d->tokens && head < d->q_heads;
            int limit, free_keys;  // keys that this row sees, and the half's first one
            {
                const int m = d->m, seen = d->first_seen;
                limit = p.a.causal ? max(min(seen + tok, m), 0) : m;
                free_keys = p.a.causal ? max(min(seen + h * p.tokens, m), 0) : m;
            }
            float m = kUnset;
            float2 l = make_float2(0.0f, 0.0f);
            for (int j = lo; j < end; ++j) {
                if (!wait_all(&s_full[h], turns))
                    break;
                ++turns;
                // the tile's maximum: a by-product of reading it, but for what is masked.  Half
                // of the scores stay in registers, the others are read again (all 128 would
                // take code of 128 columns for everything, which the instruction cache has to
                // bring in for every few tiles of a short prompt)
                float s[64], top;
                const int seen = limit - j * kTile;
                const bool masked = (j + 1) * kTile > free_keys;
                // the warp's rows see all keys below `least` and none from `most` on
                int least = kTile, most = kTile;
                if (masked) {
                    most = __reduce_max_sync(0xFFFFFFFFu, live ? seen : 0);
                    least = __reduce_min_sync(0xFFFFFFFFu, live ? seen : kTile);
                    top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < min(most, kTile); c += 32) {
                        float t = tmem_ld_max_32x32b_x32(s_addr + c, reinterpret_cast<uint32_t*>(s));
                        tmem_ld_wait();
                        if (c + 32 > least) {
                            t = -INFINITY;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                t = k < seen - c ? fmaxf(t, s[k]) : t;
                        }
                        top = fmaxf(top, t);
                    }
                } else {
                    float mx[4];
                    mx[2] = tmem_ld_max_32x32b_x32(s_addr + 64, reinterpret_cast<uint32_t*>(s));
                    mx[3] = tmem_ld_max_32x32b_x32(s_addr + 96, reinterpret_cast<uint32_t*>(s + 32));
                    mx[0] = tmem_ld_max_32x32b_x32(s_addr, reinterpret_cast<uint32_t*>(s));
                    mx[1] = tmem_ld_max_32x32b_x32(s_addr + 32, reinterpret_cast<uint32_t*>(s + 32));
                    tmem_ld_wait();
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                }
                top *= p.xscale;
                const bool moves = top > m + kSlack;
                if (__any_sync(0xFFFFFFFFu, live && moves)) {
                    // (a row whose own score does not ask for it keeps its reference, a factor of one: what
                    // the warp's other rows see has no part in its bits)
                    const float next = moves ? top : m;
                    const float factor = exp2_approx(m - next);
                    m = next;
                    l.x *= factor;
                    l.y *= factor;
                    if (j > lo) {  // (the part's tiles so far are in O: this one's S came after them)
#pragma unroll 1
                        for (int c = 0; c < kDim; c += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_addr + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
                            tmem_st_32x32b_x16(o_addr + c, o);
                        }
                    }
                }
                const float minus = -m;
                // half of the keys after the other: the MMAs begin with the first
                float2 more = make_float2(0.0f, 0.0f);
                auto weigh = [&](float x0, float x1, int k) {
                    float x[2];
                    fma_pair(x, x0, x1, xs, minus);
                    x[0] = exp2_approx(x[0]);
                    x[1] = exp2_approx(x[1]);
                    if (k & 2)
                        more = add_pair(more, x[0], x[1]);
                    else
                        l = add_pair(l, x[0], x[1]);
                    return pack2(x[0], x[1]);
                };
                auto written = [&](uint64_t* bar) {
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar);
                };
                // (masked tiles have code of their own, since a branch in the others' costs them a
                // tenth, and short code, 32 keys at a time: short prompts take 37.3 us with it, 40.3
                // with the others' 64; those in 32 as well: a long prompt 1383 us against 1324)
                if (masked) {
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 32) {
                        uint32_t w[16] = {};
                        if (c < most) {
                            tmem_ld_32x32b_x32(s_addr + c, reinterpret_cast<uint32_t*>(s));
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                w[k / 2] = weigh(k < seen - c ? s[k] : -INFINITY, k + 1 < seen - c ? s[k + 1] : -INFINITY, k);
                        }
                        tmem_st_32x32b_x16(s_addr + c / 2, w);
                        if (c & 32)
                            written(c == 32 ? &p_half[h] : &p_full[h]);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 64) {
                        uint32_t w[32];
#pragma unroll
                        for (int q = 0; q < 64; q += 32) {
#pragma unroll
                            for (int k = q; k < q + 32; k += 2)
                                w[k / 2] = weigh(s[k], s[k + 1], k);
                            if (c == 0)
                                tmem_ld_32x32b_x32(s_addr + 64 + q, reinterpret_cast<uint32_t*>(s + q));
                        }
                        tmem_st_32x32b_x32(s_addr + c / 2, w);
                        written(c == 0 ? &p_half[h] : &p_full[h]);
                        tmem_ld_wait();
                    }
                }
                l = add_pair(l, more.x, more.y);
            }
            // ------------------------------------------------------- results
            const bool some = end > lo;
            if (ok && some) {
                wait_all(&o_full[h], uses);
                ++uses;
            }
            if (!ok || !wait(&bad_full[part_count & 1u], part_count >> 1))
                break;
            const int* bad = any_bad[part_count & 1u] ? reinterpret_cast<const int*>(smem + C::OFF_BAD) + (part_count & 1u) * 3 * kDim : nullptr;
            const int slot = d->slot;
            const float sum = l.x + l.y;
            const float scale = slot >= 0 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t token = d->token + static_cast<int64_t>(tok);
            const int hq = d->q_head + head;
            const int64_t out_row = live ? token * p.a.ot + hq * p.a.oh : -1;
            const int64_t part_half = (2 * static_cast<int64_t>(blockIdx.x) + slot) * 2 + h;
            uint8_t* mine = smem + C::OFF_OUT + warp * 2048;
#pragma unroll 1
            for (int c = 0; c < kDim; c += 32) {
                float x[32];
                if (some) {
                    tmem_ld_32x32b_x32(o_addr + c, reinterpret_cast<uint32_t*>(x));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        x[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    x[k] *= scale;
                if (bad != nullptr) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float add = 0.0f;
                        if (bad[c + k] < limit)
                            add += INFINITY;
                        if (bad[kDim + c + k] < limit)
                            add -= INFINITY;
                        if (bad[2 * kDim + c + k] < limit)
                            add = __uint_as_float(0x7FC00000u);
                        x[k] += add;
                    }
                }
                if (slot < 0) {
                    // by way of shared memory, so that four lanes write 64 bytes of a row
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(mine + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = pack8(x + 8 * k);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int from = k * 8 + (lane >> 2);  // lane of the row
                        const int64_t dst = __shfl_sync(0xFFFFFFFFu, out_row, from);
                        const uint4 v = *reinterpret_cast<const uint4*>(mine + from * 64 + (((lane & 3) ^ ((from >> 1) & 3)) << 4));
                        if (dst >= 0)
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + dst + c + (lane & 3) * 8) = v;
                    }
                    __syncwarp();
                } else if (live) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o) + (part_half * (kDim / 4) + c / 4) * kHalf + row;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k * kHalf] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
            }
            if (live) {
                if (slot >= 0)
                    p.part_ml[part_half * kHalf + row] = make_float2(m, sum);
                else if (p.a.lse != nullptr)
                    p.a.lse[token * p.a.q_heads + hq] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
            }
            // O, and what was found in the values, may be written again
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bad_free[part_count & 1u]);
            part_done();
        }
        // a wait ran out: these rows' partial results may be missing, which a reference that is
        // NaN (as none ever is) tells the join
        if (__builtin_expect(!ok, 0) && p.may_cut) {
            float2* at = p.part_ml + (4 * static_cast<int64_t>(blockIdx.x) + h) * kHalf + row;
            at[0].x = at[2 * kHalf].x = __uint_as_float(0x7FC00000u);  // (both places of the CTA)
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the parts of the unit that begins in a CTA's run and goes on behind it: a
// block has 32 rows, a lane each, and a warp 4 elements of every 32.
constexpr int kJoinWarps = 8;

template <int kDim>
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(const PromptParams p)
{
    constexpr int W = kDim / (4 * kJoinWarps);  // groups of 4 elements of a thread
    __shared__ uint2 rows[32][kDim / 4 + 1];
    grid_dependency_wait();
    launch_dependents();
    const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut cut = p.cuts[c0];
    if (!cut.open)
        return;
    // the unit's parts: this one, those that it runs through, and the one behind
    int parts = 2;
    for (int c = c0 + 1;; c += 32) {
        const bool through = c + lane < static_cast<int>(gridDim.x) && p.cuts[c + lane].through;
        const uint32_t ends = ~__ballot_sync(0xFFFFFFFFu, through);
        if (ends != 0u) {
            parts += c - (c0 + 1) + __ffs(ends) - 1;
            break;
        }
    }
    parts = min(parts, static_cast<int>(gridDim.x) - c0);
    Walk w;
    w.b = cut.b;
    w.sequence(p);
    const int half = blockIdx.y >> 2, group = p.a.q_heads / p.a.kv_heads, key_head = cut.head / p.chunks;
    auto row_of = [&](int row, int64_t* token, int* hq) {  // of the half
        const int of_half = static_cast<int>(div_by_magic(row, p.heads_div)), head = row - of_half * p.heads;
        const int tok = (2 * cut.block + half) * p.tokens + of_half, of_group = (cut.head - key_head * p.chunks) * kHalf + head;
        *token = static_cast<int64_t>(w.q0) + tok;
        *hq = key_head * group + of_group;
        return of_half < p.tokens && tok < w.n && of_group < group;
    };
    const int row0 = (blockIdx.y & 3) * 32, row = row0 + lane;
    int64_t token;
    int hq;
    const bool live = row_of(row, &token, &hq);
    auto index = [&](int i) -> int64_t { return (2 * static_cast<int64_t>(c0) + (i == 0 ? 1 : 2 * i)) * 2 + half; };
    float mx = kUnset;
    bool missing = false;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float m = live ? p.part_ml[index(i) * kHalf + row].x : kUnset;
        mx = fmaxf(mx, m);
        missing |= m != m;
    }
    if (__any_sync(0xFFFFFFFFu, missing))  // (a part whose waits ran out: the block's rows, one warp's there, stay as they are)
        return;
    float4 o[W] = {};
    float sum = 0.0f;
#pragma unroll 2
    for (int i = 0; i < (live ? parts : 0); ++i) {
        const int64_t at = index(i);
        const float2 ml = p.part_ml[at * kHalf + row];
        const float f = exp2_approx(ml.x - mx);
        sum += f * ml.y;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float4 x = reinterpret_cast<const float4*>(p.part_o)[(at * (kDim / 4) + k * kJoinWarps + warp) * kHalf + row];
            o[k].x += f * x.x, o[k].y += f * x.y, o[k].z += f * x.z, o[k].w += f * x.w;
        }
    }
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < W; ++k)
        rows[lane][k * kJoinWarps + warp] = make_uint2(pack2(o[k].x * scale, o[k].y * scale), pack2(o[k].z * scale, o[k].w * scale));
    if (warp == 0 && live && p.a.lse != nullptr)
        p.a.lse[token * p.a.q_heads + hq] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (kDim / 4); i += kJoinWarps * 32) {
        const int r = i / (kDim / 4), c = i % (kDim / 4);
        if (row_of(row0 + r, &token, &hq))
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + token * p.a.ot + hq * p.a.oh + c * 4) = rows[r][c];
    }
}

template <int kDim>
cudaError_t launch(const PromptParams& p, cudaStream_t stream)
{
    using C = Cfg<kDim>;
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
            err = cudaFuncSetAttribute(prompt_attention_kernel<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (err != cudaSuccess)
                return err;
            // setmaxnreg.inc waits until the registers it asks for are free: never
            // launch a split that the launch's allocation cannot cover
            cudaFuncAttributes fa;
            err = cudaFuncGetAttributes(&fa, prompt_attention_kernel<kDim>);
            if (err != cudaSuccess)
                return err;
            if (fa.numRegs * kThreads < kAllRegs)
                return cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
        }
    }
    // (without keys nothing is loaded: the maps only have to be valid)
    const bool keys = p.a.keys > 0;
    CUtensorMap q_map, k_map, v_map;
    if (!make_heads_map(&q_map, p.a.q, p.a.T, p.a.q_heads, kDim, p.a.qt, p.a.qh, p.tokens, p.heads, true) ||
        !make_heads_map(&k_map, keys ? p.a.k : p.a.q, std::max<int64_t>(p.a.keys, 1), keys ? p.a.kv_heads : 1, kDim, p.a.kt, p.a.kh, kTile, 1, false) ||
        !make_heads_map(&v_map, keys ? p.a.v : p.a.q, std::max<int64_t>(p.a.keys, 1), keys ? p.a.kv_heads : 1, kDim, p.a.vt, p.a.vh, kTile, 1, false))
        return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(sm_count());
    err = launch_pdl(prompt_attention_kernel<kDim>, dim3(ctas), dim3(kThreads), C::SMEM, stream, p, q_map, k_map, v_map);
    if (err != cudaSuccess || !p.may_cut)
        return err;
    return launch_pdl(prompt_join_kernel<kDim>, dim3(ctas, kRows / 32), dim3(kJoinWarps * 32), 0, stream, p);
}

// Places of the partial results in the workspace, of all the CTAs.
struct Layout {
    size_t ml, cuts, bytes;
};

Layout layout_of(int dim)
{
    const size_t ctas = static_cast<size_t>(sm_count());
    Layout l;
    l.ml = ctas * 2 * kRows * dim * sizeof(float);
    l.cuts = l.ml + ctas * 2 * kRows * sizeof(float2);
    l.bytes = l.cuts + (ctas * sizeof(Cut) + 255) / 256 * 256;
    return l;
}

}  // namespace

size_t prompt_attention_workspace_bytes(int, int64_t, int64_t keys, int, int, int dim)
{
    // units of few tiles are never cut
    return keys <= kWholeTiles * kTile ? 0 : layout_of(dim).bytes;
}

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream)
{
    PromptParams p = {};
    p.a = a;
    const int group = a.q_heads / a.kv_heads;
    p.heads = std::min(group, kHalf);
    p.chunks = (group + kHalf - 1) / kHalf;
    p.tokens = kHalf / p.heads;
    p.heads_div = div_magic(p.heads);
    p.xscale = a.scale * 1.44269504088896341f;
    p.may_cut = a.keys > kWholeTiles * kTile;
    if (p.may_cut) {
        const Layout l = layout_of(a.dim);
        uint8_t* ws = static_cast<uint8_t*>(a.workspace);
        p.part_o = reinterpret_cast<float*>(ws);
        p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
        p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
    }
    return a.dim == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace fp4lin
