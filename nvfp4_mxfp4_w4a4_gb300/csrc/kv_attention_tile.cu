// kv_attention_tile.cu -- attention of 17 to 32 rows (a few drafted tokens) over
// the MX-quantized paged cache, on the 5th-generation tensor cores.
//
// The same operation as kv_attention.cu, whose warps would each convert the
// cache's codes again for every few rows.  Here a CTA owns up to NR = 32 rows
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
// included.  (The rounding is relative 2^-8 at most, the size of the output's own;
// what a product with its rest too would cost here was not measured.)  Elements of a group of 4 (E4M3) or 8 (E2M1) are stored in the
// order in which their bits come out of a word; Q is stored in that order too,
// and the output's rows are put back at the end.
//
// Warps: 0-7 softmax (quadrant of tokens x half of the rows; they also load Q
// and write the results), 8-11 convert keys, 12-15 values, 16 issues the first
// product's MMAs and 17 the second's (18, 19 fill the register group).  A wait
// costs an issuing thread a few hundred cycles even when its phase is complete,
// so each product of a tile has one: its barrier counts the converters and the
// softmax warps.  K, V, S and P are double-buffered, and the converters run
// ahead into the CTA's next unit.
//
// Measured: 4 tokens x 8 heads over 262139 of MXFP8, 8 key heads of 128: 172 us
// (3.2 TB/s); 64 sequences of 8 tokens x 4 heads over 4000: 141 us with MXFP4,
// 156 with MXFP8.  The converters' instructions bound it (92 of the 172 us of
// every issue slot), then the latency between a tile's steps.
#include "kv_attention_walk.cuh"

namespace fp4lin {
namespace {

constexpr int NR = 32;  // rows of a unit
constexpr uint32_t kSlackBits = 0x4380u;  // bf16 bits of 2^8: weights above it move the references
constexpr float kCeiling = 100.0f;        // of a weight's exponent, until they have moved

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

template <int kFmt, int kDim>
struct TileCfg {
    static constexpr int SLABS = kDim / 64;
    static constexpr int COLS = NR / 2;  // rows per softmax thread, one tensor memory load
    static constexpr int OFF_K = NR * 128 * SLABS;  // Q first
    static constexpr int OFF_V = OFF_K + 2 * SLABS * kSlab;
    static constexpr int OFF_P = OFF_V + 2 * SLABS * kSlab;
    static constexpr int OFF_REF = OFF_P + 2 * kSlab;         // float [NR]: the rows' references, negated
    static constexpr int OFF_POISON = OFF_REF + NR * 4;       // uint32 [NR]: blocks of a row that are NaN
    static constexpr int OFF_BAR = OFF_POISON + NR * 4;
    static constexpr int OFF_SLOT = OFF_BAR + 8 * 8;          // TMEM address, flags, the run's tiles
    static constexpr int OFF_WALK = (OFF_SLOT + 32 + 63) / 64 * 64;  // Place [kWalks]
    static constexpr int OFF_SCRATCH = OFF_WALK + kWalks * 64;  // two halves' [5][COLS] floats
    static constexpr int SMEM = OFF_SCRATCH + 5 * NR * 4 + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = 128;
    static constexpr int SB = kDim / 32;
    // A tile takes less time than its codes from memory, so two tiles are on their
    // way: 64 KB (E4M3) per SM.
    static constexpr int AHEAD = 2;
    // registers per thread of the three groups
    static constexpr int REGS_SOFTMAX = 80, REGS_CONVERT = 136, REGS_MMA = 48;
    static constexpr int REGS = 256 * REGS_SOFTMAX + 256 * REGS_CONVERT + 128 * REGS_MMA;
    static_assert(REGS <= kLaunchRegs * kThreads, "register split");
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int kFmt, int kDim>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tile_kernel(const AttnParams p)
{
    using C = TileCfg<kFmt, kDim>;
    extern __shared__ uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    Place<NR>* places = reinterpret_cast<Place<NR>*>(smem + C::OFF_WALK);
    const int64_t count = find_run(p, smem, places, reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT) + 7);
    if (count <= 0)
        return;
    float* ref = reinterpret_cast<float*>(smem + C::OFF_REF);
    uint32_t* poison = reinterpret_cast<uint32_t*>(smem + C::OFF_POISON);
    // the tile's keys (and its unit's Q) are in shared memory, and the S^T before the last has been read
    uint64_t* s_ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* s_done = s_ready + 2;    // S^T is complete (and the keys' buffer free)
    uint64_t* pv_ready = s_done + 2;   // values and P^T are in shared memory
    uint64_t* pv_done = pv_ready + 2;  // the tile is in O^T (the values' and P^T's buffers free)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* unit_start = tmem_slot + 1;  // by tile parity: the tile is its unit's first
    volatile uint32_t* gave_up = tmem_slot + 3;     // a wait of the softmax ran out
    const uint32_t* total_tiles = tmem_slot + 7;    // of the run

    if (threadIdx.x == 0) {
        *gave_up = 0u;
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
            for (uint32_t g = 0, end = p.withhold && blockIdx.x == 0 ? 0u : *total_tiles; g < end; ++g) {
                const uint32_t f = g & 1u;
                ok = mbar_wait_bounded(&pv_ready[f], (g >> 1) & 1u, p.status, kStatusTimeout, limit);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after_sync();
                const uint64_t vf = vd + ((f * C::SLABS * kSlab) >> 4), pf = pd + ((f * kSlab) >> 4);
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
        set_registers<C::REGS_CONVERT>();
        const bool value = warp >= kSoftmaxWarps + 4;
        convert_run<kFmt, kDim, NR, C::AHEAD>(p, places[1 + warp - kSoftmaxWarps].walk, count, smem + C::OFF_K,
                                              smem + C::OFF_V, value ? pv_ready : s_ready, value ? pv_done : s_done);
    } else {
        // --------------------------------------------------------- softmax
        set_registers<C::REGS_SOFTMAX>();
        // the two halves of the rows go their own ways within a unit
        const int quad = warp & 3, half = warp >> 2, col0 = half * C::COLS;
        const int token = quad * 32 + lane;  // of the tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const float2 xs = make_float2(p.xscale, p.xscale);
        // a half's memory for moving its references
        float* scratch = reinterpret_cast<float*>(smem + C::OFF_SCRATCH) + half * 5 * C::COLS;
        // the current unit stays in shared memory: one thread moves it on
        Walk<NR>& wk = places[0].walk;
        // (once a wait has run out, the rest of the unit goes by without waiting; both halves
        // leave together at its end)
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok)
                ok = mbar_wait_bounded(bar, parity, p.status, kStatusTimeout, limit);
        };
        uint32_t g = 0;
        for (int64_t left = count; left > 0;) {
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
            const int rows = min(NR, wk.rows(p) - row0);

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
            if (ok && lane == 0) {
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
                uint8_t* pbuf = smem + C::OFF_P + f * kSlab;
                const int j = t - ctx;
                // edge tiles: which of the thread's rows see its token, a node (drafted
                // token, `group` rows) at a time
                uint32_t vis = 0;
                if (edge) {
                    const int from = row0 + col0;  // of the head's rows
                    if (j < 0) {
                        vis = 0xFFFFu;
                    } else if (j < len - ctx && p.mask == nullptr) {
                        const int c = max(j * p.group - from, 0);  // nodes from j on
                        vis = c < C::COLS ? 0xFFFFu << c : 0u;
                    } else if (j < len - ctx && (j >> 5) < p.mask_words) {
                        int node = static_cast<int>(div_by_magic(from, p.group_div));
                        const uint32_t* word = p.mask + static_cast<int64_t>(q_start + node) * p.mask_words + (j >> 5);
#pragma unroll 2
                        for (int c = node * p.group - from; c < C::COLS && node < n; c += p.group, ++node) {
                            const uint32_t bit = (__ldg(word) >> (j & 31)) & 1u;
                            const int end = min(c + p.group, C::COLS), begin = max(c, 0);
                            vis |= bit ? ((1u << end) - 1u) >> begin << begin : 0u;
                            word += p.mask_words;
                        }
                    }
                }
                // the scores' weights into P^T's buffer and the rows' sums; returns whether
                // one is above 2^kSlack.  Edge tiles have code of their own (a branch per
                // score would keep the compiler from overlapping them).
                auto weigh = [&](auto masked, float2 sign) {
                    uint32_t top = 0u;
                    uint32_t s[C::COLS], w[C::COLS / 2];
                    tmem_ld_32x32b_x16(s_addr, s);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < C::COLS; k += 4) {
                        const float4 r = *reinterpret_cast<const float4*>(ref + col0 + k);
                        float x[4], e[4];
                        fma_pair(x, __uint_as_float(s[k]), __uint_as_float(s[k + 1]), xs, r.x, r.y);
                        fma_pair(x + 2, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]), xs, r.z, r.w);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            // finite however far the score lies above its reference
                            e[h] = exp2_approx(min_nan(x[h], kCeiling));
                            if constexpr (decltype(masked)::value)
                                e[h] = (vis >> (k + h)) & 1u ? e[h] : 0.0f;
                        }
                        fma_pair(l + k, e[0], e[1], sign, l[k], l[k + 1]);
                        fma_pair(l + k + 2, e[2], e[3], sign, l[k + 2], l[k + 3]);
                        w[k / 2] = pack2(e[0], e[1]);
                        w[k / 2 + 1] = pack2(e[2], e[3]);
                        top = __vmaxu2(top, __vmaxu2(w[k / 2], w[k / 2 + 1]));
                    }
#pragma unroll
                    for (int h = 0; h < C::COLS / 8; ++h) {
                        const int piece = col0 / 8 + h;
                        *reinterpret_cast<uint4*>(pbuf + token * 128 + ((piece ^ (token & 7)) << 4)) =
                            make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
                    }
                    return max(top & 0xFFFFu, top >> 16) > kSlackBits;
                };
                wait(&s_done[f], ph);
                // P^T's buffer is free when the tile before the last is in O^T
                wait(&pv_done[f], ph ^ 1);
                __syncwarp();
                tc_fence_after_sync();
                auto tops = [&](auto masked, float* top) {
                    uint32_t s[C::COLS];
                    tmem_ld_32x32b_x16(s_addr, s);
                    tmem_ld_wait();
                    float mine = 0.0f;
#pragma unroll
                    for (int k = 0; k < C::COLS; ++k) {
                        float x = __uint_as_float(s[k]) * p.xscale;
                        if constexpr (decltype(masked)::value)
                            x = (vis >> k) & 1u ? x : -INFINITY;
                        x = warp_max(x);
                        mine = lane == k ? x : mine;
                    }
                    if (lane < C::COLS)
                        top[quad * C::COLS + lane] = mine;
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
                        float* top = scratch;  // [4][COLS]
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
                            wait(&pv_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u);
                            __syncwarp();
                            tc_fence_after_sync();
                            uint32_t o[C::COLS];
                            tmem_ld_32x32b_x16(tmem_o + lanes + col0, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < C::COLS; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[k]);
                            tmem_st_32x32b_x16(tmem_o + lanes + col0, o);
                            tmem_st_wait();
                            named_barrier_sync(3 + half, 128);  // the factors have been read
                        }
                    }
                    const float2 sign = step == kBack ? make_float2(-1.0f, -1.0f) : make_float2(1.0f, 1.0f);
                    const bool grow = edge ? weigh(std::true_type(), sign) : weigh(std::false_type(), sign);
                    if (step == kAgain || (step == kFirst && !named_barrier_or(1 + half, 128, grow)))
                        break;
                }
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
#pragma unroll 1
                        for (int c = 0; c < C::COLS; ++c)
                            if ((vis >> c) & 1u)
                                atomicOr(&poison[col0 + c], bad);
                }
                tc_fence_before_sync();
                fence_proxy_async_smem();
                __syncwarp();
                if (threadIdx.x == 0)
                    unit_start[f] = it == 0;
                if (ok && lane == 0) {
                    mbar_arrive(&pv_ready[f]);
                    if (it + 2 < tiles)
                        mbar_arrive(&s_ready[f]);
                }
            }

            // --------------------------------------------------- results
            wait(&pv_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u);
            if (!ok)
                *gave_up = 1u;
            __syncwarp();
            tc_fence_after_sync();
            // the unit's MMAs have read their operands: [4][NR] sums go to Q's place,
            // the rows of each half to one of P^T's buffers
            float* sums = reinterpret_cast<float*>(smem);
            float* tile = reinterpret_cast<float*>(smem + C::OFF_P + (warp >> 2) * kSlab);
            static_assert(C::COLS * kDim * 4 <= kSlab, "a half's outputs in one buffer");
            // sums of the rows over the warp's tokens: each step sends half of the rows
            // away and adds the other half's, until two lanes hold the same row
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
            // (bit 4 of the lane chose the half of the rows, bit 3 the quarter, ...)
            sums[quad * NR + col0 + (lane >> 1)] = l[0];
            if (col0 < rows) {
                const int d = element_at<kFmt>(token);  // TMEM lane = position in the head
                uint32_t o[C::COLS];
                tmem_ld_32x32b_x16(tmem_o + lanes + col0, o);
                tmem_ld_wait();
                if (token < kDim)
#pragma unroll
                    for (int k = 0; k < C::COLS; ++k)
                        tile[k * kDim + d] = __uint_as_float(o[k]);
            }
            tc_fence_before_sync();
            named_barrier_sync(5, kSoftmaxWarps * 32);
            if (*gave_up)
                break;
            // complete, or a part: of the unit that began before this run (slot 0), or of
            // the one that goes on after it (slot 1)
            const bool part = lo > 0 || tiles < wk.tiles;
            const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (lo > 0 ? 0 : 1)) * NR;
            for (int i = threadIdx.x; i < rows * (kDim / 8); i += kSoftmaxWarps * 32) {
                const int r = i / (kDim / 8), d = (i - r * (kDim / 8)) * 8;
                const float ls = sums[r] + sums[NR + r] + sums[2 * NR + r] + sums[3 * NR + r];
                const float m = ref[r] == -kUnset ? -INFINITY : -ref[r];
                const float* src = reinterpret_cast<const float*>(smem + C::OFF_P + (r >= C::COLS ? kSlab : 0)) +
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
            if (wk.n > p.max_draft && wk.lo == 0 && wk.row0() == 0)
                void_rows(p, wk.head, wk.q_start, wk.n, threadIdx.x, kSoftmaxWarps * 32);
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

template <int kFmt, int kDim>
cudaError_t launch(const AttnParams& p, cudaStream_t stream)
{
    using C = TileCfg<kFmt, kDim>;
    return launch_runs<void (*)(AttnParams), kv_attention_tile_kernel<kFmt, kDim>, kDim, NR>(p, C::SMEM, C::REGS, stream);
}

}  // namespace

cudaError_t launch_kv_attention_tile(const AttnParams& p, cudaStream_t stream)
{
    if (p.cache.format == kKvMxfp8)
        return p.cache.dim == 128 ? launch<kKvMxfp8, 128>(p, stream) : launch<kKvMxfp8, 64>(p, stream);
    return p.cache.dim == 128 ? launch<kKvMxfp4, 128>(p, stream) : launch<kKvMxfp4, 64>(p, stream);
}

}  // namespace fp4lin
