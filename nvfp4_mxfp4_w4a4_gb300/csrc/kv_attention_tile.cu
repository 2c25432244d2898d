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
// Warps: 0-7 softmax (quadrant of tokens x half of the rows), 8-11 convert
// keys, 12-15 values, 16 issues the first product's MMAs and 17 the second's
// (18, 19 fill the register group).  A wait costs an issuing thread a few
// hundred cycles even when its phase is complete, so each product of a tile has
// one: its barrier counts the converters and the softmax warps.  K, V, S and P
// are double-buffered.
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
// registers per thread of the three groups, out of 96 x 640 at launch
constexpr int kRegsSoftmax = 136, kRegsConvert = 88, kRegsMma = 24;
constexpr int kRegsNeeded = 256 * kRegsSoftmax + 256 * kRegsConvert + 128 * kRegsMma;
static_assert(kRegsNeeded <= 96 * kThreads, "register split");
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
    static constexpr int OFF_SLOT = OFF_BAR + 8 * 8;  // TMEM address, two abort flags
    static constexpr int SMEM = OFF_SLOT + 16 + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = NR == 32 ? 128 : NR == 64 ? 256 : 512;
    static constexpr int COLS = NR / 2;  // rows per softmax thread
    // conversion: 16-byte chunks of a token's codes, one per lane
    static constexpr int ROW = kFmt == kKvMxfp8 ? kDim : kDim / 2;
    static constexpr int CH = ROW / 16;
    static constexpr int SB = kDim / 32;
    static_assert(SMEM <= 232448, "shared memory budget");
};

// Element that is stored at position `pos` of a head.
template <int kFmt>
__device__ __forceinline__ int element_at(int pos)
{
    return kFmt == kKvMxfp8 ? (pos & ~3) | ((pos & 1) << 1) | ((pos >> 1) & 1) : (pos & ~7) | ((pos & 1) << 2) | ((pos >> 1) & 3);
}

template <int kFmt, int kDim, int NR>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tile_kernel(const AttnParams p)
{
    using C = TileCfg<kFmt, kDim, NR>;
    extern __shared__ uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z;
    const int head = blockIdx.y / p.row_tiles;
    const int row0 = (blockIdx.y - head * p.row_tiles) * NR;
    int q_start, n;
    group_rows(p.q_offsets, b, p.T, &q_start, &n);
    if (row0 >= n * p.group)
        return;
    const int ctx = max(min(__ldg(p.context_lens + b), p.max_len - n), 0);
    const int len = min(ctx + n, p.max_len);
    const int t_begin = blockIdx.x * p.chunk;
    if (t_begin >= len)
        return;
    const int tiles = (min(len, t_begin + p.chunk) - t_begin + kTile - 1) / kTile;
    const int rows = min(NR, n * p.group - row0);
    const int splits = (len + p.chunk - 1) / p.chunk;

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* ref = reinterpret_cast<float*>(smem + C::OFF_REF);
    uint32_t* poison = reinterpret_cast<uint32_t*>(smem + C::OFF_POISON);
    // the tile's keys are in shared memory, and the S^T before the last has been read
    uint64_t* s_ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* s_done = s_ready + 2;    // S^T is complete (and the keys' buffer free)
    uint64_t* pv_ready = s_done + 2;   // values and P^T are in shared memory
    uint64_t* pv_done = pv_ready + 2;  // the tile is in O^T (the values' and P^T's buffers free)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    volatile uint32_t* gave_up = tmem_slot + 1;  // by tile parity: a softmax wait of the tile ran out

    // The converters' share of a tile: 16-byte chunks of the codes, one per lane.
    // Eight lanes in a row store to one slab, for tokens whose swizzles differ, so
    // that their 16-byte pieces fall in different banks.
    const bool value = warp >= kSoftmaxWarps + 4;
    const int w32 = (warp & 3) * 32;              // this warp's tokens of the tile
    constexpr int TPI = 32 / C::CH;               // tokens per load
    constexpr int HC = C::CH / C::SLABS;          // chunks of a token per slab
    const int chunk = ((lane >> 3) % C::SLABS) * HC + lane % HC;
    const int sub = (lane >> 3) / C::SLABS * (8 / HC) + lane / HC % (8 / HC);
    const uint8_t* codes_at[2];   // this lane's part of the first token of two groups of 16
    const uint8_t* scales_at[2];
    int page[2] = {0, 0};         // pages of the next tile's groups, looked up a tile ahead
    uint4 raw[C::CH];
    uint32_t sc[C::CH];
    // a group of 16 tokens lies in one page; groups past the end read the last one
    auto page_of = [&](int t) {
        return __ldg(p.block_table + b * p.table_stride + div_by_magic(min(t, (len - 1) & ~15), p.page_div));
    };
    auto find_group = [&](int t, int page, int which) {
        t = min(t, (len - 1) & ~15);
        const int off = t - static_cast<int>(div_by_magic(t, p.page_div)) * p.cache.page_size;
        const int64_t pg = min(max(static_cast<int64_t>(page), int64_t(0)), p.cache.pages - 1);
        const int64_t at = (pg * p.cache.heads + head) * p.cache.page_size + off + sub;
        codes_at[which] = (value ? p.cache.v_codes : p.cache.k_codes) + at * C::ROW + chunk * 16;
        scales_at[which] = (value ? p.cache.v_scales : p.cache.k_scales) + at * C::SB + (kFmt == kKvMxfp8 ? chunk / 2 : chunk);
    };
    auto load = [&](int i) {
        const int which = (i * TPI) >> 4, off = (i * TPI) & 15;
        raw[i] = __ldg(reinterpret_cast<const uint4*>(codes_at[which] + off * C::ROW));
        sc[i] = __ldg(scales_at[which] + off * C::SB);
    };
    if (warp >= kSoftmaxWarps && warp < kSoftmaxWarps + 8) {
        // the first tile's loads run under the set-up
        find_group(t_begin + w32, page_of(t_begin + w32), 0);
        find_group(t_begin + w32 + 16, page_of(t_begin + w32 + 16), 1);
        page[0] = page_of(t_begin + kTile + w32);
        page[1] = page_of(t_begin + kTile + w32 + 16);
#pragma unroll
        for (int i = 0; i < C::CH; ++i)
            load(i);
    }

    if (threadIdx.x == 0) {
        gave_up[0] = gave_up[1] = 0u;
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
    for (int i = threadIdx.x; i < NR; i += kThreads) {
        ref[i] = -kUnset;
        poison[i] = 0u;
    }
    // Q, in the stored order of a head's elements
    for (int i = threadIdx.x; i < NR * (kDim / 8); i += kThreads) {
        const int r = i / (kDim / 8), c = i - r * (kDim / 8);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const int node = (row0 + r) / p.group;
            w = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(q_start + node) * p.qt +
                                                static_cast<int64_t>(head * p.group + row0 + r - node * p.group) * p.qh +
                                                c * 8);
        }
        const uint4 o = kFmt == kKvMxfp8
                            ? make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632),
                                         __byte_perm(w.z, w.w, 0x5410), __byte_perm(w.z, w.w, 0x7632))
                            : make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                                         __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
        *reinterpret_cast<uint4*>(smem + (c >> 3) * (NR * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = o;
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_o = tmem + 2 * NR;
    const uint64_t limit = p.wait_ns;
    bool ok = true;

    if (warp >= 16) {
        // ----------------------------------------------------- MMA issuers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
        if (warp == 16 && lane == 0) {
            constexpr uint32_t idesc = idesc_bf16(128, NR, 0, 0);
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t kd = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
            for (int i = 0; i < tiles; ++i) {
                const int f = i & 1;
                if (!mbar_wait_bounded(&s_ready[f], (i >> 1) & 1, p.status, kStatusTimeout, limit))
                    break;
                tc_fence_after_sync();
                const uint64_t kf = kd + ((f * C::SLABS * kSlab) >> 4);
#pragma unroll
                for (int k = 0; k < kDim / 16; ++k)
                    tc_mma_f16(tmem + f * NR, kf + (((k >> 2) * kSlab + 32 * (k & 3)) >> 4),
                               qd + (((k >> 2) * (NR * 128) + 32 * (k & 3)) >> 4), idesc, k != 0);
                tc_commit(&s_done[f]);
            }
        } else if (warp == 17 && lane == 0) {
            constexpr uint32_t idesc = idesc_bf16(128, NR, 1, 1);
            const uint64_t vd = smem_desc(smem_u32(smem + C::OFF_V), kSlab, 1024, 2);
            const uint64_t pd = smem_desc(smem_u32(smem + C::OFF_P), kSlab, 1024, 2);
            for (int i = 0; i < tiles; ++i) {
                const int f = i & 1;
                if (!mbar_wait_bounded(&pv_ready[f], (i >> 1) & 1, p.status, kStatusTimeout, limit))
                    break;
                tc_fence_after_sync();
                const uint64_t vf = vd + ((f * C::SLABS * kSlab) >> 4), pf = pd + ((f * C::P_SLABS * kSlab) >> 4);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc_mma_f16(tmem_o, vf + ((2048 * k) >> 4), pf + ((2048 * k) >> 4), idesc, i | k ? 1u : 0u);
                tc_commit(&pv_done[f]);
            }
        }
    } else if (warp >= kSoftmaxWarps) {
        // --------------------------------------------- codes -> bf16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
        uint8_t* dst = smem + (value ? C::OFF_V : C::OFF_K);
        uint64_t* full = value ? pv_ready : s_ready;
        uint64_t* freed = value ? pv_done : s_done;
        for (int it = 0; it < tiles; ++it) {
            const int tile0 = t_begin + it * kTile, f = it & 1;
            const bool more = it + 1 < tiles;
            if (more) {
                find_group(tile0 + kTile + w32, page[0], 0);
                find_group(tile0 + kTile + w32 + 16, page[1], 1);
                page[0] = page_of(tile0 + 2 * kTile + w32);
                page[1] = page_of(tile0 + 2 * kTile + w32 + 16);
            }
            ok = mbar_wait_bounded(&freed[f], ((it >> 1) & 1) ^ 1, p.status, kStatusTimeout, limit);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            const bool edge = value && tile0 + kTile > ctx;
#pragma unroll
            for (int i = 0; i < C::CH; ++i) {
                const int tok = w32 + i * TPI + sub;
                // NaN values of an edge tile are kept out of the product (see the softmax)
                const uint32_t mul = edge && sc[i] == 0xFFu ? 0u : block_multiplier<kFmt>(sc[i]) * 0x10001u;
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint8_t* row = dst + f * C::SLABS * kSlab + tok * 128;
                if constexpr (kFmt == kKvMxfp8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[2], c[2];
                        place_codes<kFmt>(w[2 * h], a);
                        place_codes<kFmt>(w[2 * h + 1], c);
                        const int piece = 2 * chunk + h;
                        *reinterpret_cast<uint4*>(row + (piece >> 3) * kSlab + (((piece & 7) ^ (tok & 7)) << 4)) =
                            make_uint4(mul_bf16x2(a[0], mul), mul_bf16x2(a[1], mul), mul_bf16x2(c[0], mul),
                                       mul_bf16x2(c[1], mul));
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t a[4];
                        place_codes<kFmt>(w[h], a);
                        const int piece = 4 * chunk + h;
                        *reinterpret_cast<uint4*>(row + (piece >> 3) * kSlab + (((piece & 7) ^ (tok & 7)) << 4)) =
                            make_uint4(mul_bf16x2(a[0], mul), mul_bf16x2(a[1], mul), mul_bf16x2(a[2], mul),
                                       mul_bf16x2(a[3], mul));
                    }
                }
                if (more)
                    load(i);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[f]);
        }
    } else {
        // --------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int quad = warp & 3, col0 = (warp >> 2) * C::COLS;
        const int token = quad * 32 + lane;  // of the tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        constexpr int CW = C::COLS == 32 ? 32 : 16;  // columns at a time
        if (lane == 0) {  // both S^T buffers start free
            mbar_arrive(&s_ready[0]);
            mbar_arrive(&s_ready[1]);
        }
        float l[C::COLS];
#pragma unroll
        for (int c = 0; c < C::COLS; ++c)
            l[c] = 0.0f;
        const float2 xs = make_float2(p.xscale, p.xscale);
        auto load_cols = [&](uint32_t addr, uint32_t* r) {
            if constexpr (CW == 32)
                tmem_ld_32x32b_x32(addr, r);
            else
                tmem_ld_32x32b_x16(addr, r);
        };
        for (int it = 0; it < tiles; ++it) {
            const int f = it & 1, ph = (it >> 1) & 1;
            const int t = t_begin + it * kTile + token;
            const bool edge = t_begin + (it + 1) * kTile > ctx;
            const uint32_t s_addr = tmem + lanes + f * NR + col0;
            uint8_t* pbuf = smem + C::OFF_P + f * C::P_SLABS * kSlab;
            const int j = t - ctx;
            auto seen = [&](int row) -> bool {
                if (j < 0)
                    return true;
                if (j >= n || row >= rows)
                    return false;
                const int node = static_cast<int>(div_by_magic(row0 + row, p.group_div));
                if (p.mask == nullptr)
                    return j <= node;
                return (j >> 5) < p.mask_words &&
                       ((__ldg(p.mask + static_cast<int64_t>(q_start + node) * p.mask_words + (j >> 5)) >> (j & 31)) & 1u);
            };
            uint32_t vis[(C::COLS + 31) / 32];  // edge tiles: whether a row sees the token
            if (edge) {
#pragma unroll
                for (int w = 0; w < (C::COLS + 31) / 32; ++w) {
                    vis[w] = 0u;
#pragma unroll 1
                    for (int c = 0; c < 32 && 32 * w + c < C::COLS; ++c)
                        vis[w] |= seen(col0 + 32 * w + c) ? 1u << c : 0u;
                }
            }
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
                                e[h] = (vis[(c + k + h) / 32] >> ((c + k + h) & 31)) & 1u ? e[h] : 0.0f;
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
                            x = (vis[(c + k) / 32] >> ((c + k) & 31)) & 1u ? x : -INFINITY;
                        x = warp_max(x);
                        mine = lane == k ? x : mine;
                    }
                    if (lane < 16)
                        top[quad * NR + col0 + c + lane] = mine;
                }
            };
            // Weigh the tile; if a weight is too large, take its weights back, move the
            // references to the rows' largest scores (per quadrant of tokens, by way of
            // P^T's buffer) and weigh it again.  The first tile starts with that.  (What
            // a sum loses by the subtraction is 2^-24 of the weight that made the
            // reference move, which stays in the sum.)
            enum { kFirst, kBack, kAgain };
            bool leave = false;
#pragma unroll 1
            for (int step = it > 0 ? kFirst : kAgain;; ++step) {
                if (step == kAgain) {
                    float* top = reinterpret_cast<float*>(pbuf);  // [4][NR]
                    float* factor = top + 4 * NR;
                    named_barrier_sync(2, kSoftmaxWarps * 32);
                    if (edge)
                        tops(std::true_type(), top);
                    else
                        tops(std::false_type(), top);
                    named_barrier_sync(2, kSoftmaxWarps * 32);
                    if (threadIdx.x < NR) {
                        const int r = threadIdx.x;
                        const float old = -ref[r];
                        float now = fmaxf(fmaxf(top[r], top[NR + r]), fmaxf(top[2 * NR + r], top[3 * NR + r]));
                        now = fmaxf(now, old);
                        factor[r] = exp2_approx(old - now);
                        ref[r] = -now;
                    }
                    named_barrier_sync(2, kSoftmaxWarps * 32);
                    if (it > 0) {
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c)
                            l[c] *= factor[col0 + c];
                        ok = mbar_wait_bounded(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, p.status, kStatusTimeout, limit) && ok;
                        __syncwarp();
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < C::COLS; c += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(tmem_o + lanes + col0 + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[col0 + c + k]);
                            tmem_st_32x32b_x16(tmem_o + lanes + col0 + c, o);
                        }
                        tmem_st_wait();
                        named_barrier_sync(2, kSoftmaxWarps * 32);  // the factors have been read
                    }
                }
                const float2 sign = step == kBack ? make_float2(-1.0f, -1.0f) : make_float2(1.0f, 1.0f);
                const bool grow = edge ? weigh(std::true_type(), sign) : weigh(std::false_type(), sign);
                if (step == kAgain)
                    break;
                if (step == kFirst) {
                    if (!ok)
                        gave_up[f] = 1u;
                    __syncwarp();
                    const bool rescale = named_barrier_or(1, kSoftmaxWarps * 32, grow);
                    leave = gave_up[f] != 0u;
                    if (leave || !rescale)
                        break;
                }
            }
            if (leave)
                break;  // all softmax threads at the same tile
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
#pragma unroll
                    for (int w = 0; w < (C::COLS + 31) / 32; ++w)
                        for (uint32_t m = vis[w]; m != 0u; m &= m - 1u)
                            atomicOr(&poison[col0 + 32 * w + __ffs(m) - 1], bad);
            }
            tc_fence_before_sync();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s_ready[f]);
                mbar_arrive(&pv_ready[f]);
            }
        }

        // ------------------------------------------------------- results
        const int last = tiles - 1;
        if (!gave_up[0] && !gave_up[1])
            mbar_wait_bounded(&pv_done[last & 1], (last >> 1) & 1, p.status, kStatusTimeout, limit);
        __syncwarp();
        tc_fence_after_sync();
        // every MMA has read its operands: [4][NR] sums in P^T's buffers, [NR][kDim + 4]
        // outputs in the keys' and values'
        float* sums = reinterpret_cast<float*>(smem + C::OFF_P);
        float* tile = reinterpret_cast<float*>(smem + C::OFF_K);
        constexpr int LD = kDim + 4;
        static_assert(NR * LD * 4 <= 4 * C::SLABS * kSlab, "outputs reuse the tiles");
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
                        tile[(col0 + c + k) * LD + d] = __uint_as_float(o[k]);
            }
        }
        named_barrier_sync(2, kSoftmaxWarps * 32);
        for (int i = threadIdx.x; i < rows * (kDim / 8); i += kSoftmaxWarps * 32) {
            const int r = i / (kDim / 8), d = (i - r * (kDim / 8)) * 8;
            const float ls = sums[r] + sums[NR + r] + sums[2 * NR + r] + sums[3 * NR + r];
            const float m = ref[r] == -kUnset ? -INFINITY : -ref[r];
            const float4 u = *reinterpret_cast<const float4*>(tile + r * LD + d);
            const float4 v = *reinterpret_cast<const float4*>(tile + r * LD + d + 4);
            float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            const bool nan = (poison[r] >> (d >> 5)) & 1u;
            const float scale = nan ? __uint_as_float(0x7FC00000u)
                                : splits > 1 ? kUnscale : ls == 0.0f ? 0.0f : kUnscale * (1.0f / ls);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] *= scale;
            const int node = static_cast<int>(div_by_magic(row0 + r, p.group_div));
            const int64_t tok = q_start + node;
            const int hq = head * p.group + row0 + r - node * p.group;
            if (splits == 1) {
                *reinterpret_cast<uint4*>(p.out + tok * p.ot + hq * p.oh + d) =
                    make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
                if (d == 0 && p.lse != nullptr)
                    p.lse[tok * p.q_heads + hq] = (m + log2f(ls)) * 0.69314718055994531f;
            } else {
                const int64_t at = (static_cast<int64_t>(blockIdx.x) * p.T + tok) * p.q_heads + hq;
                float4* dst = reinterpret_cast<float4*>(p.part_o + at * kDim + d);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
                if (d == 0)
                    *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, ls);
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

template <int kFmt, int kDim, int NR>
cudaError_t launch_tile(const AttnParams& p, dim3 grid, cudaStream_t stream)
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
            if (fa.numRegs * kThreads < kRegsNeeded)
                return cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
        }
    }
    return launch_pdl(kern, grid, dim3(kThreads), C::SMEM, stream, p);
}

template <int kFmt, int kDim>
cudaError_t launch_rows(const AttnParams& p, int rows, dim3 grid, cudaStream_t stream)
{
    return rows == 32   ? launch_tile<kFmt, kDim, 32>(p, grid, stream)
           : rows == 64 ? launch_tile<kFmt, kDim, 64>(p, grid, stream)
                        : launch_tile<kFmt, kDim, 128>(p, grid, stream);
}

}  // namespace

cudaError_t launch_kv_attention_tile(const AttnParams& params, int rows, int splits, cudaStream_t stream)
{
    AttnParams p = params;
    p.xscale *= kUnscale;  // scores come out of the MMA times 2^-64
    const dim3 grid(splits, p.cache.heads * p.row_tiles, p.batch);
    if (p.cache.format == kKvMxfp8)
        return p.cache.dim == 128 ? launch_rows<kKvMxfp8, 128>(p, rows, grid, stream)
                                  : launch_rows<kKvMxfp8, 64>(p, rows, grid, stream);
    return p.cache.dim == 128 ? launch_rows<kKvMxfp4, 128>(p, rows, grid, stream)
                              : launch_rows<kKvMxfp4, 64>(p, rows, grid, stream);
}

}  // namespace fp4lin
