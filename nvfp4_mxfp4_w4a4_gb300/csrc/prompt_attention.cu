// prompt_attention.cu -- softmax attention over whole prompts: packed sequences of
// different lengths, grouped heads, causal or not, all in bf16, on the
// 5th-generation tensor cores.
//
//   S [rows x keys] = Q K^T,  P = exp2(S scale log2(e) - m),  O += P V
//
// A unit is 256 rows of a key/value head: the queries' heads that read it side by
// side, (token, head) pairs in the tokens' order, as two halves of 128 rows.  The
// halves' tiles of 128 keys take turns: while the MMAs of one half run, the other
// half's scores are weighed.  A softmax thread is one row: the tile's 128 scores
// are in its registers at once, maximum and sum stay there, and the
// probabilities (bf16) go back to tensor memory over the scores.  The row's
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
// Warps: 0-3 and 4-7 the softmax of the halves (they also write the results), 8
// loads keys and values (TMA), 9 issues the MMAs, 10 and 11 load the queries and
// look through the values.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kHalf = 128;           // rows of a half
constexpr int kRows = 2 * kHalf;     // of a unit
constexpr int kTile = 128;           // keys of a tile
constexpr int kSlab = 128 * 128;     // bytes of 64 bf16 elements of 128 rows or keys
constexpr int kThreads = 384;
constexpr int kUnitPlaces = 3;       // of a unit's start and end on the line
constexpr int kLeastRun = kUnitPlaces + 4;
constexpr int kWholeTiles = 8;       // units of at most so many tiles are never cut
constexpr int kWarpSequences = 96;   // up to so many sequences, a warp adds one up
constexpr float kSlack = 8.0f;       // a score this far above its reference moves it
// a row's reference before its first seen key: the lowest float32, which no score lies under
constexpr float kUnset = -3.402823466e38f;
// registers per thread: at launch, and dealt out anew to the softmax and the others
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kLaunchRegs * kThreads, "register split");

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
    DivMagic group_div;
    int group;
    float xscale;   // scale * log2(e)
    float* part_o;  // [CTA][2][kRows][dim]
    float2* part_ml;
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

template <int kRegs>
__device__ __forceinline__ void set_registers()
{
    if constexpr (kRegs > kLaunchRegs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---------------------------------------------------------------- the line

// A place on the line: one unit after the other, by sequence, key head and block
// of rows.
struct Walk {
    int b, head, block, blocks;  // blocks of the sequence
    int q0, n, k0, m;

    __device__ __forceinline__ void sequence(const PromptParams& p)
    {
        group_rows(p.a.q_offsets, b, static_cast<int>(p.a.T), &q0, &n);
        group_rows(p.a.k_offsets, b, static_cast<int>(p.a.keys), &k0, &m);
        blocks = static_cast<int>((static_cast<uint32_t>(n) * p.group + kRows - 1) / kRows);
    }
    // Keys that row r (of the sequence's rows) sees.
    __device__ __forceinline__ int limit(const PromptParams& p, int r) const
    {
        if (!p.a.causal)
            return m;
        const int i = min(static_cast<int>(div_by_magic(r, p.group_div)), n - 1);
        return max(min(i + 1 + m - n, m), 0);
    }
    __device__ __forceinline__ int first_row(int half) const { return block * kRows + half * kHalf; }
    __device__ __forceinline__ int tiles(const PromptParams& p, int half) const
    {
        const int r0 = first_row(half), rows = n * p.group;
        return r0 >= rows ? 0 : (limit(p, min(r0 + kHalf, rows) - 1) + kTile - 1) / kTile;
    }
    __device__ __forceinline__ int tiles(const PromptParams& p) const { return max(tiles(p, 0), tiles(p, 1)); }
    __device__ __forceinline__ void next(const PromptParams& p)
    {
        if (++block < blocks)
            return;
        block = 0;
        if (++head < p.a.kv_heads)
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

// This CTA's run; false if it has none.  All threads call it; `scratch` is free
// afterwards.
__device__ bool find_run(const PromptParams& p, uint8_t* scratch, Run* shared)
{
    constexpr int kWarps = kThreads / 32;
    struct Scan {
        int64_t weight[kWarpSequences];  // places of a sequence's key head
        int64_t warp_sum[kWarps];
        int64_t offset, per_head;
        int longest[kWarps];
        int b;
    };
    Scan* scan = reinterpret_cast<Scan*>(scratch);
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
    const int heads = p.a.kv_heads;
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
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, int64_t(whole ? 1 : kLeastRun));
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
        r.w.head = static_cast<int>(scan->offset / scan->per_head);
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

template <int kDim>
struct Cfg {
    static constexpr int SLABS = kDim / 64;
    static constexpr int TILE = SLABS * kSlab;  // bytes of a tile of K or V, or of a half's Q
    static constexpr int STAGES = kDim == 128 ? 2 : 4;
    static constexpr int OFF_K = 2 * TILE;  // Q first
    static constexpr int OFF_V = OFF_K + STAGES * TILE;
    static constexpr int OFF_BAD = OFF_V + STAGES * TILE;  // int [2][3][kDim]: first keys whose value is inf, -inf, NaN
    static constexpr int OFF_BAR = OFF_BAD + 2 * 3 * kDim * 4;
    static constexpr int BARS = 4 * STAGES + 4 + 2 * 7 + 1;
    static constexpr int OFF_SLOT = OFF_BAR + BARS * 8;  // TMEM address, flags
    static constexpr int OFF_RUN = (OFF_SLOT + 32 + 15) / 16 * 16;
    static constexpr int SMEM = OFF_RUN + 128 + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = 512;  // S of the halves, then O
    static constexpr int TMEM_O = 2 * kTile;
    static_assert(sizeof(Run) <= 128, "");
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const PromptParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map)
{
    using C = Cfg<kDim>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_full = bars;              // [STAGES] a tile has landed
    uint64_t* k_free = k_full + STAGES;   // [STAGES] and is multiplied
    uint64_t* v_full = k_free + STAGES;   // [STAGES]
    uint64_t* v_free = v_full + STAGES;   // [STAGES]
    uint64_t* v_seen = v_free + STAGES;   // [4] a masked tile's values are looked through
    uint64_t* q_full = v_seen + 4;        // [2] by half
    uint64_t* q_free = q_full + 2;        // [2]
    uint64_t* s_full = q_free + 2;        // [2] scores are complete (and the tile before is in O)
    uint64_t* p_full = s_full + 2;        // [2] probabilities are in tensor memory
    uint64_t* o_full = p_full + 2;        // [2] the part's last tile is in O
    uint64_t* bad_full = o_full + 2;      // [2] by part: its masked tiles are looked through
    uint64_t* bad_free = bad_full + 2;    // [2] and what was found is read
    uint64_t* drained = bad_free + 2;     // every MMA has ended
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* any_bad = tmem_slot + 1;  // [2] by part
    Run* run = reinterpret_cast<Run*>(smem + C::OFF_RUN);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_free[i], 1);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&v_seen[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 2);
            mbar_init(&q_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&bad_full[i], 2);
            mbar_init(&bad_free[i], 8);
            any_bad[i] = 0u;
        }
        mbar_init(drained, 1);
        fence_mbar_init();
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    launch_dependents();
    const bool have = find_run(p, smem, run);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint64_t limit_ns = p.a.wait_ns;
    bool ok = true;
    // a wait of one thread, and one of a whole warp; once one has run out, the role ends
    auto wait_one = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait_bounded(bar, parity & 1u, p.a.status, kStatusTimeout, limit_ns);
        return ok;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xFFFFFFFFu, wait_one(bar, parity));
        return ok;
    };
    Cut cut = {};
    cut.open = 0;

    if (warp >= 8) {
        set_registers<kOtherRegs>();
        if (!have) {
        } else if (warp == 8) {
            // ------------------------------------------------ keys and values
            if (lane == 0) {
                Run r = *run;
                bool started = false;
                uint32_t g = 0;  // tiles so far
                auto landed = [&](uint64_t* full, uint32_t slot, uint32_t phase) {
                    mbar_wait_bounded(&full[slot], phase, p.a.status, kStatusTimeout, limit_ns);
                };
                while (ok && r.part(p, started)) {
                    for (int j = r.lo; ok && j < r.hi; ++j, ++g) {
                        const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1u;
                        const int at = r.w.k0 + j * kTile;
                        if (!wait_one(&k_free[slot], phase ^ 1u))
                            break;
                        mbar_arrive_expect_tx(&k_full[slot], C::TILE);
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
                            tma_load_3d(smem + C::OFF_K + slot * C::TILE + s * kSlab, &k_map, &k_full[slot], s * 64, at, r.w.head);
                        if (!wait_one(&v_free[slot], phase ^ 1u)) {
                            landed(k_full, slot, phase);
                            break;
                        }
                        mbar_arrive_expect_tx(&v_full[slot], C::TILE);
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
                            tma_load_3d(smem + C::OFF_V + slot * C::TILE + s * kSlab, &v_map, &v_full[slot], s * 64, at, r.w.head);
                    }
                }
                // nothing of this CTA may be in flight when it ends
                for (uint32_t i = 0; i < STAGES && i < g; ++i) {
                    const uint32_t last = g - 1 - i;
                    landed(k_full, last % STAGES, (last / STAGES) & 1u);
                    landed(v_full, last % STAGES, (last / STAGES) & 1u);
                }
            }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMAs
            constexpr uint32_t idesc_s = idesc_bf16(kHalf, kTile, 0, 0);
            constexpr uint32_t idesc_o = idesc_bf16(kHalf, kDim, 0, 1);
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t kd = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
            const uint64_t vd = smem_desc(smem_u32(smem + C::OFF_V), kSlab, 1024, 2);
            // a step is a tile of the run: the tiles of each half in its part
            struct Step {
                bool live, masked;
                bool has[2], first[2], last[2];
            };
            Run r = *run;
            bool started = false, more = true;
            int j = 0, end[2] = {0, 0}, free_keys = 0;
            r.hi = 0;
            auto next_step = [&]() {
                Step s = {};
                if (++j >= r.hi) {
                    do
                        more = more && r.part(p, started);
                    while (more && r.hi == r.lo);
                    if (!more)
                        return s;
                    j = r.lo;
                    end[0] = min(r.hi, r.w.tiles(p, 0));
                    end[1] = min(r.hi, r.w.tiles(p, 1));
                    free_keys = r.w.limit(p, r.w.first_row(0));
                }
                s.live = true;
                s.masked = (j + 1) * kTile > free_keys;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s.has[h] = j < end[h];
                    s.first[h] = j == r.lo;
                    s.last[h] = j == end[h] - 1;
                }
                return s;
            };
            uint32_t uses[2] = {0, 0};   // of a half's Q
            uint32_t turns[2] = {0, 0};  // of a half's probabilities
            uint32_t seen = 0;           // masked tiles
            auto scores = [&](const Step& s, int h, uint32_t g) {
                // S of the half; Q's place is free after the part's last tile
                if (!s.has[h])
                    return;
                if (s.first[h] && !wait(&q_full[h], uses[h]++))
                    return;
                tc_fence_after_sync();
                const uint64_t q = qd + ((h * C::TILE) >> 4), k = kd + (((g % STAGES) * C::TILE) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kDim / 16; ++i) {
                        const uint64_t at = ((i >> 2) * kSlab + 32 * (i & 3)) >> 4;
                        tc_mma_f16(tmem + h * kTile, q + at, k + at, idesc_s, i != 0);
                    }
                    tc_commit(&s_full[h]);
                    if (s.last[h])
                        tc_commit(&q_free[h]);
                }
                __syncwarp();
            };
            auto free_slot = [&](uint64_t* bar) {
                if (elect_one())
                    tc_commit(bar);
                __syncwarp();
            };
            Step now = next_step();
            if (now.live && wait(&k_full[0], 0)) {
                scores(now, 0, 0);
                scores(now, 1, 0);
                if (ok)
                    free_slot(&k_free[0]);
            }
            for (uint32_t g = 0; now.live && ok; ++g) {
                const Step then = next_step();
                const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1u;
                if (!wait(&v_full[slot], phase))
                    break;
                if (now.masked) {
                    if (!wait(&v_seen[seen & 3u], seen >> 2))
                        break;
                    ++seen;
                }
                if (then.live && !wait(&k_full[(g + 1) % STAGES], (g + 1) / STAGES))
                    break;
                const uint64_t v = vd + ((slot * C::TILE) >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (now.has[h]) {
                        if (!wait(&p_full[h], turns[h]++))
                            break;
                        tc_fence_after_sync();
                        if (elect_one() && !(p.a.withhold && blockIdx.x == 0)) {
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i)
                                tc_mma_f16_ts(tmem + C::TMEM_O + h * kDim, tmem + h * kTile + 8 * i, v + ((2048 * i) >> 4),
                                              idesc_o, i != 0 || !now.first[h]);
                            if (now.last[h])
                                tc_commit(&o_full[h]);
                        }
                        __syncwarp();
                    }
                    if (then.live)
                        scores(then, h, g + 1);
                    if (!ok)
                        break;
                }
                if (!ok)
                    break;
                free_slot(&v_free[slot]);
                if (then.live)
                    free_slot(&k_free[(g + 1) % STAGES]);
                now = then;
            }
            // whatever was issued has ended before tensor and shared memory go
            if (elect_one())
                tc_commit(drained);
            __syncwarp();
            mbar_wait_bounded(drained, 0, p.a.status, kStatusTimeout, limit_ns);
        } else {
            // ----------------------------------- queries; looks through values
            const int t = threadIdx.x - 320;
            // a wait of both warps, which go on or end together
            auto wait_both = [&](uint64_t* bar, uint32_t parity) {
                ok = !named_barrier_or(1, 64, !wait_one(bar, parity));
                return ok;
            };
            Run r = *run;
            bool started = false;
            uint32_t uses[2] = {0, 0}, g = 0, seen = 0, parts = 0;
            while (ok && r.part(p, started)) {
                const int rows = r.w.n * p.group;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (r.lo >= min(r.hi, r.w.tiles(p, h)))
                        continue;
                    if (!wait_both(&q_free[h], (uses[h] & 1u) ^ 1u))
                        break;
                    ++uses[h];
                    constexpr int VECS = kDim / 8, PER = 64 / VECS;  // vectors of a row, rows of a round
                    const int c = t % VECS;
                    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q) + c * 8;
#pragma unroll 4
                    for (int i = 0; i < kHalf / PER; ++i) {
                        const int row = i * PER + t / VECS, at = r.w.first_row(h) + row;
                        const int tok = static_cast<int>(div_by_magic(at, p.group_div));
                        const bool live = at < rows;
                        const __nv_bfloat16* src = q + static_cast<int64_t>(r.w.q0 + tok) * p.a.qt +
                                                   static_cast<int64_t>(r.w.head * p.group + at - tok * p.group) * p.a.qh;
                        cp_async_16(smem + h * C::TILE + (c >> 3) * kSlab + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                                    live ? src : p.a.q, live);
                    }
                    cp_async_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&q_full[h]);
                }
                if (!ok)
                    break;
                // the part's masked tiles
                const uint32_t par = parts & 1u;
                if (!wait_both(&bad_free[par], ((parts >> 1) & 1u) ^ 1u))
                    break;
                int* bad = reinterpret_cast<int*>(smem + C::OFF_BAD) + par * 3 * kDim;
                const int free_keys = r.w.limit(p, r.w.first_row(0));
                if (t == 0)
                    any_bad[par] = 0u;
                bool cleared = false;
                for (int j = r.lo; ok && j < r.hi; ++j) {
                    if ((j + 1) * kTile <= free_keys)
                        continue;
                    const uint32_t tile = g + (j - r.lo), slot = tile % STAGES;
                    if (!wait_both(&v_full[slot], tile / STAGES))
                        break;
                    uint8_t* v = smem + C::OFF_V + slot * C::TILE;
                    bool found = false;
                    constexpr int PIECES = C::TILE / 16 / 64;
#pragma unroll 8
                    for (int i = 0; i < PIECES; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(v + (i * 64 + t) * 16);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            found |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
                    }
                    // (both warps decide together: they write the same list)
                    if (named_barrier_or(1, 64, found)) {
                        if (!cleared) {
                            for (int i = t; i < 3 * kDim; i += 64)
                                bad[i] = 0x7FFFFFFF;
                            if (t == 0)
                                any_bad[par] = 1u;
                            cleared = true;
                        }
                        named_barrier_sync(1, 64);
                        for (int i = 0; i < PIECES; ++i) {
                            const int piece = i * 64 + t, in_slab = piece % (kSlab / 16), key = in_slab / 8;
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
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&v_seen[seen & 3u]);
                    ++seen;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bad_full[par]);
                g += r.hi - r.lo;
                ++parts;
            }
        }
    } else {
        // --------------------------------------------------------- softmax
        set_registers<kSoftmaxRegs>();
        const int h = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;  // of the half
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_addr = tmem + lanes + h * kTile, o_addr = tmem + lanes + C::TMEM_O + h * kDim;
        const float2 xs = make_float2(p.xscale, p.xscale);
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            tc_fence_after_sync();
            return ok;
        };
        uint32_t turns = 0, uses = 0, parts = 0;
        Run r = *run;
        bool started = false;
        while (have && ok && r.part(p, started)) {
            const int at = r.w.first_row(h) + row;  // row of the sequence's key head
            const int rows = r.w.n * p.group;
            const int mine = min(r.hi, r.w.tiles(p, h));  // this half's tiles end here
            const int limit = r.w.limit(p, at);
            const int free_keys = r.w.limit(p, r.w.first_row(h));
            float m = kUnset;
            float2 l = make_float2(0.0f, 0.0f);
            for (int j = r.lo; j < mine; ++j) {
                if (!wait_all(&s_full[h], turns))
                    break;
                ++turns;
                float s[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32)
                    tmem_ld_32x32b_x32(s_addr + c, reinterpret_cast<uint32_t*>(s + c));
                tmem_ld_wait();
                if ((j + 1) * kTile > free_keys) {
                    const int seen = limit - j * kTile;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        s[c] = c < seen ? s[c] : -INFINITY;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTile; c += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = fmaxf(mx[k], fmaxf(s[c + k], s[c + k + 4]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.xscale;
                if (__any_sync(0xFFFFFFFFu, top > m + kSlack)) {
                    const float next = fmaxf(m, top);
                    const float factor = exp2_approx(m - next);
                    m = next;
                    l.x *= factor;
                    l.y *= factor;
                    if (j > r.lo) {  // (the part's tiles so far are in O: this one's S came after them)
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
#pragma unroll
                for (int c = 0; c < kTile; c += 64) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        float x[2];
                        fma_pair(x, s[c + k], s[c + k + 1], xs, minus);
                        x[0] = exp2_approx(x[0]);
                        x[1] = exp2_approx(x[1]);
                        l = add_pair(l, x[0], x[1]);
                        w[k / 2] = pack2(x[0], x[1]);
                    }
                    tmem_st_32x32b_x32(s_addr + c / 2, w);
                }
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[h]);
            }
            // ------------------------------------------------------- results
            const bool some = mine > r.lo;
            if (ok && some) {
                wait_all(&o_full[h], uses);
                ++uses;
            }
            if (ok)
                wait_all(&bad_full[parts & 1u], parts >> 1);
            if (!ok)
                break;
            const bool whole = r.lo == 0 && r.hi == r.tiles;
            const int* bad = any_bad[parts & 1u] ? reinterpret_cast<const int*>(smem + C::OFF_BAD) + (parts & 1u) * 3 * kDim : nullptr;
            const float sum = l.x + l.y;
            const float scale = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            const int tok = static_cast<int>(div_by_magic(at, p.group_div));
            const int64_t token = r.w.q0 + tok;
            const int hq = r.w.head * p.group + at - tok * p.group;
            const int64_t part_row = (2 * static_cast<int64_t>(blockIdx.x) + (r.lo > 0 ? 0 : 1)) * kRows + h * kHalf + row;
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
#pragma unroll 4
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
                if (at < rows) {
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + token * p.a.ot + hq * p.a.oh + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dst[k] = pack8(x + 8 * k);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + part_row * kDim + c);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                    }
                }
            }
            if (at < rows) {
                if (!whole)
                    p.part_ml[part_row] = make_float2(m, sum);
                else if (p.a.lse != nullptr)
                    p.a.lse[token * p.a.q_heads + hq] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
            }
            if (r.hi < r.tiles) {
                if (r.lo > 0) {
                    cut.through = 1;
                } else {
                    cut.open = 1;
                    cut.b = r.w.b, cut.head = r.w.head, cut.block = r.w.block;
                }
            }
            // O, and what was found in the values, may be written again
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bad_free[parts & 1u]);
            ++parts;
        }
        if (threadIdx.x == 0 && p.may_cut) {
            if (!ok)
                cut.open = cut.through = 0;
            p.cuts[blockIdx.x] = cut;
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
// warp per row.
constexpr int kJoinWarps = 8;

template <int kDim>
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(const PromptParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int c0 = blockIdx.x, lane = threadIdx.x & 31;
    const Cut cut = p.cuts[c0];
    if (!cut.open)
        return;
    const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    Walk w;
    w.b = cut.b;
    w.sequence(p);
    const int at = cut.block * kRows + row;
    if (at >= w.n * p.group)
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
    auto index = [&](int i) -> int64_t { return (2 * static_cast<int64_t>(c0) + (i == 0 ? 1 : 2 * i)) * kRows + row; };
    float mx = kUnset;
    for (int i = lane; i < parts; i += 32)
        mx = fmaxf(mx, p.part_ml[index(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    constexpr int W = kDim / 32;  // elements of a lane
    float o[W] = {}, sum = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += 32) {
        float mine = 0.0f, add = 0.0f;
        if (i0 + lane < parts) {
            const float2 ml = p.part_ml[index(i0 + lane)];
            mine = exp2_approx(ml.x - mx);
            add = mine * ml.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
        sum += add;
        const int here = min(32, parts - i0);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float f = __shfl_sync(0xFFFFFFFFu, mine, i);
            const float* src = p.part_o + index(i0 + i) * kDim + lane * W;
#pragma unroll
            for (int k = 0; k < W; k += 2) {
                const float2 x = *reinterpret_cast<const float2*>(src + k);
                o[k] += f * x.x;
                o[k + 1] += f * x.y;
            }
        }
    }
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int tok = static_cast<int>(div_by_magic(at, p.group_div));
    const int64_t token = w.q0 + tok;
    const int hq = cut.head * p.group + at - tok * p.group;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.out) + token * p.a.ot + hq * p.a.oh + lane * W);
#pragma unroll
    for (int k = 0; k < W / 2; ++k)
        dst[k] = pack2(o[2 * k] * scale, o[2 * k + 1] * scale);
    if (lane == 0 && p.a.lse != nullptr)
        p.a.lse[token * p.a.q_heads + hq] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
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
            if (fa.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs)
                return cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
        }
    }
    // (without keys nothing is loaded: the maps only have to be valid)
    const bool keys = p.a.keys > 0;
    CUtensorMap k_map, v_map;
    if (!make_heads_map(&k_map, keys ? p.a.k : p.a.q, std::max<int64_t>(p.a.keys, 1), keys ? p.a.kv_heads : 1, kDim, p.a.kt, p.a.kh, kTile) ||
        !make_heads_map(&v_map, keys ? p.a.v : p.a.q, std::max<int64_t>(p.a.keys, 1), keys ? p.a.kv_heads : 1, kDim, p.a.vt, p.a.vh, kTile))
        return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(sm_count());
    err = launch_pdl(prompt_attention_kernel<kDim>, dim3(ctas), dim3(kThreads), C::SMEM, stream, p, k_map, v_map);
    if (err != cudaSuccess || !p.may_cut)
        return err;
    return launch_pdl(prompt_join_kernel<kDim>, dim3(ctas, kRows / kJoinWarps), dim3(kJoinWarps * 32), 0, stream, p);
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
    p.group = a.q_heads / a.kv_heads;
    p.group_div = div_magic(p.group);
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
