// kv_attention_rows.cu -- attention of more than 32 rows (trees of drafted tokens)
// over the MX-quantized paged cache, on the 5th-generation tensor cores.
//
// The same operation as kv_attention.cu, whose warps would each convert the
// cache's codes again for every few rows.  Here a CTA owns up to 128 rows
// (drafted token x query head of one key/value head) and walks the context in
// tiles of 128 tokens; each tile is converted once, to bf16 in shared memory,
// and multiplied by tcgen05.mma with the rows on the M side:
//   S [rows x tokens] = Q [rows x dims] K^T      (both K-major)
//   O [rows x dims]  += P [rows x tokens] V      (P from tensor memory, V token
//                                                 by token as it is converted)
// A softmax thread is one row of a tile: the maximum, the sum and the reference
// of its row are registers, and its probabilities go back to tensor memory, over
// the scores that they come from.  The reference moves only when a score passes
// it by 2^8, so most tiles leave O as it is.  Even and odd tiles belong to two
// groups of four softmax warps, each with sums and an O of its own, joined at
// the end of a unit: the groups never wait for one another, so that one's
// products run while the other weighs its scores.
//
// Numbers: as in kv_attention.cu (exact bf16 elements with a multiplier that
// carries 2^-64, probabilities rounded to bf16, everything else fp32), keys
// included.  (The rounding is relative 2^-8 at most, the size of the output's own;
// what a product with its rest too would cost here was not measured.)  Elements of a group of 4 (E4M3) or 8 (E2M1) are stored in the
// order in which their bits come out of a word; Q is stored in that order too,
// and the output's elements are put back at the end.
//
// Warps: 0-3 and 4-7 the softmax of even and odd tiles (they also load Q and
// write the results), 8-11 convert keys, 12-15 values, 16 issues the first
// product's MMAs and 17 the second's (18, 19 fill the register group).  A wait
// costs an issuing thread a few hundred cycles even when its phase is complete,
// so each product of a tile has one: its barrier counts all it needs.  K, V and
// S are double-buffered, and the converters run ahead into the CTA's next unit.
//
// Measured: 8 trees of 31 tokens x 4 heads over up to 16001 tokens, 8 key heads
// of 128: 78 us with MXFP4, 84 with MXFP8 (464 and 432 TFLOPS of the two
// products; with the tokens on the M side and P in shared memory as in
// kv_attention_tile.cu 113 and 140).  A tile takes about 1.05 us, of which the
// MMAs are 0.5 and the issue slots 0.6: what bounds it is the way of a group's
// tile from S through the weights and P V to the S after the next, 2.1 us for
// two tiles.  Shared memory is the reason for P in tensor memory: an MMA with
// both operands there reads 128 bytes a cycle, all there is, and the converters
// and softmax stores wait (126 us).  Not kept: weights in one pass with the
// probabilities in registers until their vote (106 us, spills), Q loaded a
// unit ahead (83 us), codes prefetched into L2 (82 to 84 us).
#include "kv_attention_walk.cuh"

namespace fp4lin {
namespace {

constexpr int kRows = 128;      // rows of a unit
constexpr float kSlack = 8.0f;  // a score this far above its reference moves it

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

template <int kFmt, int kDim>
struct RowsCfg {
    static constexpr int SLABS = kDim / 64;
    static constexpr int OFF_K = SLABS * kSlab;  // Q first
    static constexpr int OFF_V = OFF_K + 2 * SLABS * kSlab;
    static constexpr int OFF_STATS = OFF_V + 2 * SLABS * kSlab;  // float [2][kRows][2]: the groups' references and sums
    static constexpr int OFF_POISON = OFF_STATS + 2 * kRows * 8;  // uint8 [2][kTile]: NaN blocks of an edge tile's values
    static constexpr int OFF_BAR = OFF_POISON + 2 * kTile;
    static constexpr int OFF_SLOT = OFF_BAR + 8 * 8;  // TMEM address, flags, the run's tiles
    static constexpr int OFF_WALK = (OFF_SLOT + 32 + 63) / 64 * 64;  // Place [kWalks]
    static constexpr int SMEM = OFF_WALK + kWalks * 64 + 1024;  // + alignment slack
    // TMEM columns: S of even and odd tiles, then O of both
    static constexpr int TMEM_O = 2 * kTile;
    static constexpr int TMEM_COLS = 512;
    static constexpr int SB = kDim / 32;
    // tiles whose codes are on their way, as far as registers hold them
    static constexpr int AHEAD = kFmt == kKvMxfp8 && kDim == 128 ? 1 : 2;
    // registers per thread of the three groups, out of 96 x 640 at launch
    static constexpr int REGS_SOFTMAX = 112, REGS_CONVERT = 104, REGS_MMA = 48;
    static constexpr int REGS = 256 * REGS_SOFTMAX + 256 * REGS_CONVERT + 128 * REGS_MMA;
    static_assert(REGS <= kLaunchRegs * kThreads, "register split");
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int kFmt, int kDim>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_rows_kernel(const AttnParams p)
{
    using C = RowsCfg<kFmt, kDim>;
    extern __shared__ uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    Place<kRows>* places = reinterpret_cast<Place<kRows>*>(smem + C::OFF_WALK);
    const int64_t count = find_run(p, smem, places, reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT) + 7);
    if (count <= 0)
        return;
    // the tile's keys and its unit's Q are in shared memory, and the tile before the last is in O
    uint64_t* s_ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* s_done = s_ready + 2;    // S is complete (and the keys' buffer free)
    uint64_t* pv_ready = s_done + 2;   // values are in shared memory and P in tensor memory
    uint64_t* pv_done = pv_ready + 2;  // the tile is in O (and the values' buffer free)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* group_start = tmem_slot + 1;  // by tile parity: the tile is its group's first of the unit
    volatile uint32_t* gave_up = tmem_slot + 3;      // a wait of the softmax ran out
    const uint32_t* total_tiles = tmem_slot + 7;     // of the run

    if (threadIdx.x == 0) {
        *gave_up = 0u;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_ready[i], 4 + 4 + 1);  // converters, softmax group, the second product
            mbar_init(&s_done[i], 1);
            mbar_init(&pv_ready[i], 4 + 4);
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
    const uint64_t limit = p.wait_ns;
    bool ok = true;

    if (warp >= 16) {
        // ----------------------------------------------------- MMA issuers
        set_registers<C::REGS_MMA>();
        // (the whole warp walks the loop and one elected lane issues: the operands
        // of the MMAs then stay in uniform registers)
        if (warp == 16) {
            constexpr uint32_t idesc = idesc_bf16(kRows, kTile, 0, 0);
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
                    for (int k = 0; k < kDim / 16; ++k) {
                        const uint64_t at = ((k >> 2) * kSlab + 32 * (k & 3)) >> 4;
                        tc_mma_f16(tmem + f * kTile, qd + at, kf + at, idesc, k != 0);
                    }
                    tc_commit(&s_done[f]);
                }
                __syncwarp();
            }
        } else if (warp == 17) {
            constexpr uint32_t idesc = idesc_bf16(kRows, kDim, 0, 1);
            const uint64_t vd = smem_desc(smem_u32(smem + C::OFF_V), kSlab, 1024, 2);
            // nothing comes before the first two tiles
            if (lane == 0) {
                mbar_arrive(&s_ready[0]);
                mbar_arrive(&s_ready[1]);
            }
            __syncwarp();
            for (uint32_t g = 0, end = p.withhold && blockIdx.x == 0 ? 0u : *total_tiles; g < end; ++g) {
                const uint32_t f = g & 1u;
                ok = mbar_wait_bounded(&pv_ready[f], (g >> 1) & 1u, p.status, kStatusTimeout, limit);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after_sync();
                const uint64_t vf = vd + ((f * C::SLABS * kSlab) >> 4);
                const uint32_t add = group_start[f] ? 0u : 1u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_f16_ts(tmem + C::TMEM_O + f * kDim, tmem + f * kTile + 8 * k, vf + ((2048 * k) >> 4), idesc,
                                      k ? 1u : add);
                    if (g + 2 < end)
                        tc_commit(&s_ready[f]);
                    tc_commit(&pv_done[f]);
                }
                __syncwarp();
            }
        }
    } else if (warp >= kSoftmaxWarps) {
        set_registers<C::REGS_CONVERT>();
        const bool value = warp >= kSoftmaxWarps + 4;
        convert_run<kFmt, kDim, kRows, C::AHEAD>(p, places[1 + warp - kSoftmaxWarps].walk, count, smem + C::OFF_K,
                                                 smem + C::OFF_V, value ? pv_ready : s_ready, value ? pv_done : s_done);
    } else {
        // --------------------------------------------------------- softmax
        set_registers<C::REGS_SOFTMAX>();
        const int quad = warp & 3, grp = warp >> 2;
        const int r = quad * 32 + lane;  // row of the unit
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_addr = tmem + lanes + grp * kTile, o_addr = tmem + lanes + C::TMEM_O;
        const float2 xs = make_float2(p.xscale, p.xscale);
        float2* stats = reinterpret_cast<float2*>(smem + C::OFF_STATS);
        uint8_t* poison = smem + C::OFF_POISON + grp * kTile;
        auto wait = [&](uint64_t* bar, uint32_t g) {
            // (once one has run out, the rest of the unit goes by without waiting)
            if (ok)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, (g >> 1) & 1u, p.status, kStatusTimeout, limit));
            tc_fence_after_sync();
        };
        // the current unit stays in shared memory: one thread moves it on
        Walk<kRows>& wk = places[0].walk;
        uint32_t g0 = 0;  // the unit's first tile, counted over the run
        for (int64_t left = count; left > 0;) {
            const int tiles = wk.run(p, left);
            if (tiles == 0) {
                named_barrier_sync(1, kSoftmaxWarps * 32);  // everyone has read the unit
                if (threadIdx.x == 0 && left > 0)
                    wk.next(p);
                named_barrier_sync(1, kSoftmaxWarps * 32);
                continue;
            }
            const int head = wk.head, row0 = wk.row0(), ctx = wk.ctx, len = wk.len, b = wk.b;
            const int q_start = wk.q_start, lo = wk.lo;
            const int rows = min(p.part_rows, wk.rows(p) - row0);
            const int node = static_cast<int>(div_by_magic(row0 + r, p.group_div));  // of this thread's row

            // Q, in the stored order of a head's elements (rows past the last keep what is
            // there; they have no say in when their warp's references move, so that nothing
            // of it reaches the results)
            for (int i = threadIdx.x; i < rows * (kDim / 8); i += kSoftmaxWarps * 32) {
                const int qr = i / (kDim / 8), c = i - qr * (kDim / 8);
                const int qn = static_cast<int>(div_by_magic(row0 + qr, p.group_div));
                const uint4 q = *reinterpret_cast<const uint4*>(
                    p.q + static_cast<int64_t>(q_start + qn) * p.qt +
                    static_cast<int64_t>(head * p.group + row0 + qr - qn * p.group) * p.qh + c * 8);
                const uint4 o = kFmt == kKvMxfp8
                                    ? make_uint4(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.x, q.y, 0x7632),
                                                 __byte_perm(q.z, q.w, 0x5410), __byte_perm(q.z, q.w, 0x7632))
                                    : make_uint4(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632),
                                                 __byte_perm(q.y, q.w, 0x5410), __byte_perm(q.y, q.w, 0x7632));
                *reinterpret_cast<uint4*>(smem + (c >> 3) * kSlab + qr * 128 + (((c & 7) ^ (qr & 7)) << 4)) = o;
            }
            fence_proxy_async_smem();
            named_barrier_sync(1, kSoftmaxWarps * 32);
            const int first = (grp ^ g0) & 1;  // this group's first tile of the unit
            if (first < tiles && ok && lane == 0)
                mbar_arrive(&s_ready[grp]);

            float m = kUnset;
            float2 l = make_float2(0.0f, 0.0f);
            uint32_t bad = 0;  // blocks of the row's output that a NaN value reaches
            for (int it = first; it < tiles; it += 2) {
                const int t0 = (lo + it) * kTile;
                const bool edge = t0 + kTile > ctx;
                uint32_t vis[4];  // edge tiles: the tokens that the row sees
                if (edge) {
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        vis[w] = r < rows ? visible32(p, q_start + node, node, len - ctx, t0 + 32 * w - ctx) : 0u;
                    // and the values of the tile that are NaN, by token
                    const int t = t0 + r;
                    uint32_t nan = 0;
                    if (t < len) {
                        const int pi = static_cast<int>(div_by_magic(t, p.page_div));
                        const int64_t pg = min(max(static_cast<int64_t>(__ldg(p.block_table + b * p.table_stride + pi)), int64_t(0)),
                                               p.cache.pages - 1);
                        const uint8_t* vs = p.cache.v_scales + ((pg * p.cache.heads + head) * p.cache.page_size +
                                                                (t - pi * p.cache.page_size)) * C::SB;
#pragma unroll
                        for (int k = 0; k < C::SB; ++k)
                            nan |= __ldg(vs + k) == 0xFFu ? 1u << k : 0u;
                    }
                    poison[r] = static_cast<uint8_t>(nan);
                    if (named_barrier_or(2 + grp, 128, nan != 0u)) {
                        for (int c = 0; c < kTile; ++c)
                            bad |= (vis[c >> 5] >> (c & 31)) & 1u ? poison[c] : 0u;
                    }
                    named_barrier_sync(2 + grp, 128);  // (the flags may be written again)
                }
                wait(&s_done[grp], g0 + it);
                if (quad * 32 < rows) {
                    // scores -> the row's largest; then weights, their sum, and P over the scores.
                    // Edge tiles have code of their own (a branch per score would keep the
                    // compiler from overlapping them).
                    auto top = [&](auto masked) {
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        uint32_t sb[2][16];
                        tmem_ld_32x32b_x16(s_addr, sb[0]);
#pragma unroll
                        for (int c = 0; c < kTile; c += 16) {
                            const uint32_t* s = sb[c / 16 & 1];
                            tmem_ld_wait();
                            if (c + 16 < kTile)
                                tmem_ld_32x32b_x16(s_addr + c + 16, sb[(c / 16 + 1) & 1]);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                float x = __uint_as_float(s[k]);
                                if constexpr (decltype(masked)::value)
                                    x = (vis[c / 32] >> ((c + k) & 31)) & 1u ? x : -INFINITY;
                                mx[k & 3] = fmaxf(mx[k & 3], x);
                            }
                        }
                        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.xscale;
                    };
                    const float now = edge ? top(std::true_type()) : top(std::false_type());
                    if (__any_sync(0xFFFFFFFFu, r < rows && now > m + kSlack)) {
                        const float next = fmaxf(m, now);
                        const float factor = exp2_approx(m - next);
                        m = next;
                        l.x *= factor;
                        l.y *= factor;
                        if (it > first) {  // (the group's tiles so far are in O: this one's S came after them)
#pragma unroll 1
                            for (int c = 0; c < kDim; c += 16) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(o_addr + grp * kDim + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
                                tmem_st_32x32b_x16(o_addr + grp * kDim + c, o);
                            }
                        }
                    }
                    auto weigh = [&](auto masked) {
                        const float minus = -m;
                        uint32_t sb[2][16], w[16];
                        tmem_ld_32x32b_x16(s_addr, sb[0]);
#pragma unroll
                        for (int c = 0; c < kTile; c += 16) {
                            const uint32_t* s = sb[c / 16 & 1];
                            tmem_ld_wait();
                            if (c + 16 < kTile)
                                tmem_ld_32x32b_x16(s_addr + c + 16, sb[(c / 16 + 1) & 1]);
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                float x[2];
                                fma_pair(x, __uint_as_float(s[k]), __uint_as_float(s[k + 1]), xs, minus, minus);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    x[h] = exp2_approx(x[h]);
                                    if constexpr (decltype(masked)::value)
                                        x[h] = (vis[c / 32] >> ((c + k + h) & 31)) & 1u ? x[h] : 0.0f;
                                }
                                l = add_pair(l, x[0], x[1]);
                                w[(c + k) / 2 & 15] = pack2(x[0], x[1]);
                            }
                            if (c & 16)
                                tmem_st_32x32b_x16(s_addr + (c - 16) / 2, w);
                        }
                    };
                    if (edge)
                        weigh(std::true_type());
                    else
                        weigh(std::false_type());
                    tmem_st_wait();
                }
                tc_fence_before_sync();
                if (threadIdx.x % 128 == 0)
                    group_start[grp] = it == first;
                __syncwarp();
                if (ok && lane == 0) {
                    mbar_arrive(&pv_ready[grp]);
                    if (it + 2 < tiles)
                        mbar_arrive(&s_ready[grp]);
                }
            }

            // --------------------------------------------------- results
            stats[grp * kRows + r] = make_float2(m, l.x + l.y);
            poison[r] = static_cast<uint8_t>(bad);
            for (int k = max(tiles - 2, 0); k < tiles; ++k)
                wait(&pv_done[(g0 + k) & 1u], g0 + k);
            if (!ok)
                *gave_up = 1u;
            named_barrier_sync(1, kSoftmaxWarps * 32);
            if (*gave_up)
                break;
            // complete, or a part: of the unit that began before this run (slot 0), or of
            // the one that goes on after it (slot 1)
            const bool part = lo > 0 || tiles < wk.tiles;
            if (quad * 32 < rows) {
                // the row's two sums; the group's half of its elements
                const float2 s0 = stats[r], s1 = stats[kRows + r];
                const bool has[2] = {((g0 & 1u) == 0u || tiles > 1), ((g0 & 1u) == 1u || tiles > 1)};
                const float top = fmaxf(s0.x, s1.x);
                const float f0 = exp2_approx(s0.x - top), f1 = exp2_approx(s1.x - top);
                const float sum = (has[0] ? f0 * s0.y : 0.0f) + (has[1] ? f1 * s1.y : 0.0f);
                const uint32_t nan = smem[C::OFF_POISON + r] | smem[C::OFF_POISON + kTile + r];
                const float unit_scale = part ? kUnscale : (sum == 0.0f ? 0.0f : kUnscale * (1.0f / sum));
                const float ml = top == kUnset ? -INFINITY : top;
                const int64_t tok = q_start + node;
                const int hq = head * p.group + row0 + r - node * p.group;
                const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + (lo > 0 ? 0 : 1)) * p.part_rows + r;
#pragma unroll 1
                for (int c = grp * (kDim / 2); c < (grp + 1) * (kDim / 2); c += 16) {
                    uint32_t o0[16], o1[16];
                    if (has[0])
                        tmem_ld_32x32b_x16(o_addr + c, o0);
                    if (has[1])
                        tmem_ld_32x32b_x16(o_addr + kDim + c, o1);
                    tmem_ld_wait();
                    float x[16];
                    const float scale = (nan >> (c >> 5)) & 1u ? __uint_as_float(0x7FC00000u) : unit_scale;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        x[element_at<kFmt>(k)] = ((has[0] ? __uint_as_float(o0[k]) * f0 : 0.0f) +
                                                  (has[1] ? __uint_as_float(o1[k]) * f1 : 0.0f)) * scale;
                    if (r < rows) {
                        if (!part) {
                            uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.ot + hq * p.oh + c);
                            dst[0] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
                            dst[1] = make_uint4(pack2(x[8], x[9]), pack2(x[10], x[11]), pack2(x[12], x[13]), pack2(x[14], x[15]));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(p.part_o + at * kDim + c);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                        }
                    }
                }
                if (grp == 0 && r < rows) {
                    if (part)
                        *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(ml, sum);
                    else if (p.lse != nullptr)
                        p.lse[tok * p.q_heads + hq] = (ml + log2f(sum)) * 0.69314718055994531f;
                }
            }
            if (wk.n > p.max_draft && wk.lo == 0 && wk.row0() == 0)
                void_rows(p, wk.head, wk.q_start, wk.n, threadIdx.x, kSoftmaxWarps * 32);
            g0 += tiles;
            // Q's place, O and the unit may be written again
            tc_fence_before_sync();
            named_barrier_sync(1, kSoftmaxWarps * 32);
            if (left > 0) {
                if (threadIdx.x == 0)
                    wk.next(p);
                named_barrier_sync(1, kSoftmaxWarps * 32);
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

template <int kFmt, int kDim>
cudaError_t launch(const AttnParams& p, cudaStream_t stream)
{
    using C = RowsCfg<kFmt, kDim>;
    return launch_runs<void (*)(AttnParams), kv_attention_rows_kernel<kFmt, kDim>, kDim, kRows>(p, C::SMEM, C::REGS, stream);
}

}  // namespace

cudaError_t launch_kv_attention_rows(const AttnParams& p, cudaStream_t stream)
{
    if (p.cache.format == kKvMxfp8)
        return p.cache.dim == 128 ? launch<kKvMxfp8, 128>(p, stream) : launch<kKvMxfp8, 64>(p, stream);
    return p.cache.dim == 128 ? launch<kKvMxfp4, 128>(p, stream) : launch<kKvMxfp4, 64>(p, stream);
}

}  // namespace fp4lin
