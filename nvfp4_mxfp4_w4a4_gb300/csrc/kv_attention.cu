// kv_attention.cu -- softmax attention of drafted tokens over the MX-quantized
// paged cache, by streaming the cache once through registers.
//
//   x[i, t] = scale q[i] . k[t],   out[i] = sum_t softmax(x[i])[t] v[t]
//
// over the tokens t that row i sees: the whole context of its sequence and,
// of the sequence's drafted tokens (their keys and values follow the context
// in the cache), those its tree mask names.  A single token per sequence is
// the ordinary decode step.
//
// A warp owns 8 * NT rows (drafted token x query head of one key/value head)
// and 16 tokens at a time, and computes the transposed products with
// mma.m16n8k16: S^T = K Q^T (tokens on the MMA's 16 rows, attention rows on
// its 8 columns), O^T += V^T P^T.  With few rows (a decode step has as many
// as query heads share a key head) this wastes least of the MMA, halves the
// accumulators against rows on the 16 side, and lets one conversion of K and
// V serve every column tile.  The order of the tokens inside a step is free,
// and so is that of an MMA's elements, so each lane takes contiguous bytes: of
// a key 8 elements of every block (4 lanes a block), of a value 1/8 head of
// four tokens.  Codes are copied asynchronously to a ring of steps in shared
// memory that belongs to the warp (no barriers in the loop; 16-byte chunks
// swizzled so that no read has a bank conflict at a head of 128 bytes) and go
// from there to registers to MMA fragments.
//
// Keys become f16 by the hardware's pair conversion, exactly, and enter
// without their scale: each MMA step lies in one block of 32, and the block's
// scale is applied in fp32 to the block's partial score.  (f16 holds every
// code; a query row is scaled by a power of two to a largest magnitude in
// [2^14, 2^15), which keeps 2^-38 of it.)  Placing the bits of a code in a
// bf16 with integer operations instead costs 6 times the issue slots.
//
// Values and probabilities need the exponents of bf16 (a probability of 2^-30
// counts where the winning token's element is zero), so values are placed:
// the code's bits in the bf16's exponent and mantissa fields (subnormals
// included) are 2^-120 (E4M3) or 2^-126 (E2M1) times the code's value, and one
// bf16 multiply by a power of two applies the block's scale.  That multiplier
// carries 2^-64 (put back in fp32 at the end), so that it stays a finite bf16
// up to values of 2^66.  Scores, softmax statistics and sums are fp32, and the
// sum of the probabilities is taken before they are rounded to bf16 for the
// second product.  Up to 4 rows what that rounding leaves is multiplied too, at
// no cost: the MMA's columns 4 ... 7 repeat the rows and take it (64 sequences
// up to 8190 tokens of MXFP8, 8 key heads: 144 us both ways).  More rows keep
// one rounding, relative 2^-8 at most, the size of the output's own: a second
// product costs 149 us instead of 143 at 8 rows and 212 instead of 189 at 16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "formats.cuh"
#include "internal.h"
#include "kv_attention.cuh"
#include "kv_cache.h"
#include "ptx.cuh"

namespace fp4lin {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;         // tokens a warp takes at a time
constexpr int kStages = 3;        // steps in a warp's ring

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 2^e as a float, e in [-126, 127]; below that zero.
__device__ __forceinline__ float exp2_int(int e)
{
    return __uint_as_float(static_cast<uint32_t>(max(e + 127, 0)) << 23);
}

// The codes of a word, in their order, as f16 pairs.
template <int kFmt>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t* out)
{
    if constexpr (kFmt == kKvMxfp8) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(out[0]), "=r"(out[1])
            : "r"(w));
    } else {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
            : "r"(w));
    }
}

// Whether a byte of four is 0xFF (the high bits of those that are).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;
}

// Dimensions: a lane holds 8 elements of each block of a key and dim / 8
// consecutive elements of a value.
template <int kFmt, int kDim>
struct Shape {
    static constexpr int BITS = kFmt == kKvMxfp8 ? 8 : 4;
    static constexpr int ROW = kDim * BITS / 8;  // code bytes of a token
    static constexpr int SB = kDim / 32;         // blocks (scale bytes) of a token
    static constexpr int KW = BITS / 4;          // 32-bit words per lane and block of a key
    static constexpr int VW = ROW / 32;          // 32-bit words of a value per lane
    static constexpr int PAIRS = 32 / (2 * BITS);  // element pairs per word
    static constexpr int MT = kDim / 16;         // 16-element tiles of the output
    // one step in shared memory: key codes, value codes, key scales, value scales
    static constexpr int CODES = kStep * ROW;
    static constexpr int SCALES = kStep * SB;
    static constexpr int STEP_BYTES = 2 * CODES + 2 * SCALES;
    // place of byte `at` (a multiple of the read's size) of token t: the 16-byte
    // chunks of a row are permuted by the 128-byte line that it lies in
    static __device__ __forceinline__ int place(int t, int at)
    {
        return t * ROW + (((at >> 4) ^ ((t * ROW >> 7) & (ROW / 16 - 1))) << 4) + (at & 15);
    }
};

template <int W>
__device__ __forceinline__ void read_words(const uint8_t* p, uint32_t* r)
{
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ROWS attention rows in COLS MMA columns; column c holds row c mod ROWS.
template <int kFmt, int kDim, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, ROWS <= 8 ? 4 : 3) kv_attention_kernel(const AttnParams p)
{
    using S = Shape<kFmt, kDim>;
    constexpr int NT = ROWS <= 8 ? 1 : ROWS / 8;
    constexpr int COLS = 8 * NT;
    constexpr bool TWICE = ROWS < COLS;
    extern __shared__ __align__(128) float smem[];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, qd = lane & 3;
    const int b = blockIdx.z;
    const int head = blockIdx.y;
    int q_start, n;
    group_rows(p.q_offsets, b, p.T, &q_start, &n);
    if (n == 0)
        return;
    const int ctx = max(min(__ldg(p.context_lens + b), p.max_len - n), 0);
    const int len = min(ctx + n, p.max_len);
    const int t_begin = blockIdx.x * p.chunk;
    if (t_begin >= len)
        return;
    const int t_end = min(len, t_begin + p.chunk);
    const int rows = min(n, p.max_draft) * p.group;  // of the head, at most ROWS
    const int splits = (len + p.chunk - 1) / p.chunk;
    if (n > p.max_draft && blockIdx.x == 0)
        void_rows(p, head, q_start, n, threadIdx.x, kWarps * 32);

    // this lane's share of Q: row g of each column tile, 8 elements of every
    // block, as f16 times a power of two of the row
    uint32_t qf[NT][4 * S::SB];
    float qs[NT][2];  // the inverse power times xscale, of rows 2 qd and 2 qd + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rr = (8 * nt + g) % ROWS;
        const bool live = rr < rows;
        const int i = rr / p.group;
        const __nv_bfloat16* src = p.q + static_cast<int64_t>(q_start + i) * p.qt +
                                   static_cast<int64_t>(head * p.group + rr - i * p.group) * p.qh + qd * 8;
        uint32_t w[4 * S::SB];
        uint32_t am = 0;
#pragma unroll
        for (int k = 0; k < S::SB; ++k) {
            const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 32 * k) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 4 * S::SB; ++k)
            am = __vmaxu2(am, w[k] & 0x7FFF7FFFu);
        am = max(am & 0xFFFFu, am >> 16);
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        // 2^(14 - floor(log2 amax)), within float range; NaN and Inf rows stay what they are
        const int shift = am == 0u || am >= 0x7F80u ? 0 : min(14 + 127 - static_cast<int>(am >> 7), 126);
        const float up = exp2_int(shift);
#pragma unroll
        for (int k = 0; k < 4 * S::SB; ++k)
            qf[nt][k] = pack2_f16(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
        const float down = exp2_int(-shift) * p.xscale;
        qs[nt][0] = __shfl_sync(0xFFFFFFFFu, down, 8 * qd);
        qs[nt][1] = __shfl_sync(0xFFFFFFFFu, down, 8 * qd + 4);
    }

    float o[S::MT][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt)
            o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.0f;
    }

    // The steps' copies.  A step's 16 tokens lie in one page (page sizes are
    // multiples of 16) and are contiguous there; tokens past the end come along
    // (the page holds them) and are masked.
    uint8_t* ring = reinterpret_cast<uint8_t*>(smem) + warp * (kStages * S::STEP_BYTES);
    const int32_t* table = p.block_table + b * p.table_stride;
    auto page_at = [&](int t) { return __ldg(table + div_by_magic(t, p.page_div)); };
    auto copy_step = [&](uint8_t* dst, int t, int page) {
        const int pg = static_cast<int>(min(max(static_cast<int64_t>(page), int64_t(0)), p.cache.pages - 1));
        const int off = t - static_cast<int>(div_by_magic(t, p.page_div)) * p.cache.page_size;
        const int64_t base = (static_cast<int64_t>(pg) * p.cache.heads + head) * p.cache.page_size + off;
        const uint8_t* kc = p.cache.k_codes + base * S::ROW + lane * 16;
        const uint8_t* vc = p.cache.v_codes + base * S::ROW + lane * 16;
        constexpr int PER_ROW = S::ROW / 16;
#pragma unroll
        for (int i = 0; i < S::CODES / 512; ++i) {
            const int at = S::place((32 * i + lane) / PER_ROW, (lane % PER_ROW) * 16);
            cp_async_16(dst + at, kc + 512 * i, true);
            cp_async_16(dst + S::CODES + at, vc + 512 * i, true);
        }
        constexpr int SCALE_CHUNKS = S::SCALES / 16;
        if (lane < 2 * SCALE_CHUNKS) {
            const int c = lane % SCALE_CHUNKS;
            const uint8_t* src = (lane < SCALE_CHUNKS ? p.cache.k_scales : p.cache.v_scales) + base * S::SB + 16 * c;
            cp_async_16(dst + 2 * S::CODES + lane * 16, src, true);
        }
    };

    int t0 = t_begin + warp * kStep;
    int t_copy = t0;      // next step to copy, its page, and the ring slot it goes to
    int page = t0 < t_end ? page_at(t0) : 0;
    auto copy_next = [&](int slot) {
        if (t_copy < t_end) {
            copy_step(ring + slot * S::STEP_BYTES, t_copy, page);
            t_copy += kWarps * kStep;
            if (t_copy < t_end)
                page = page_at(t_copy);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        copy_next(i);
    int slot = 0;
    for (; t0 < t_end; t0 += kWarps * kStep, slot = slot + 1 == kStages ? 0 : slot + 1) {
        // this step has landed and every lane is done with the one before it
        cp_async_wait<kStages - 2>();
        __syncwarp();
        copy_next(slot == 0 ? kStages - 1 : slot - 1);
        const uint8_t* step = ring + slot * S::STEP_BYTES;
        uint32_t ks[2], vs[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t* sc = step + 2 * S::CODES + (g + 8 * j) * S::SB;
            if constexpr (S::SB == 4)
                ks[j] = *reinterpret_cast<const uint32_t*>(sc);
            else
                ks[j] = *reinterpret_cast<const uint16_t*>(sc);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            vs[j] = step[2 * S::CODES + S::SCALES + (2 * qd + (j & 1) + 8 * (j >> 1)) * S::SB + g * S::SB / 8];

        // ---------------------------------------------------- S^T = K Q^T
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < S::SB; ++k) {
            uint32_t kw[S::KW];
            uint32_t a0[4], a1[4];  // the lane's 8 elements of tokens g and g + 8
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                read_words<S::KW>(step + S::place(g + 8 * j, k * (S::ROW / S::SB) + qd * (4 * S::KW)), kw);
                uint32_t* a = j ? a1 : a0;
#pragma unroll
                for (int w = 0; w < S::KW; ++w)
                    codes_to_f16<kFmt>(kw[w], a + w * S::PAIRS);
            }
            const uint32_t first[4] = {a0[0], a1[0], a0[1], a1[1]}, second[4] = {a0[2], a1[2], a0[3], a1[3]};
            // 2^(s - 127) of both tokens' block
            const float s0 = __uint_as_float(((ks[0] >> (8 * k)) & 0xFFu) << 23);
            const float s1 = __uint_as_float(((ks[1] >> (8 * k)) & 0xFFu) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(part, first, qf[nt][4 * k], qf[nt][4 * k + 1]);
                mma_f16(part, second, qf[nt][4 * k + 2], qf[nt][4 * k + 3]);
                x[nt][0] = fmaf(part[0], s0, x[nt][0]);
                x[nt][1] = fmaf(part[1], s0, x[nt][1]);
                x[nt][2] = fmaf(part[2], s1, x[nt][2]);
                x[nt][3] = fmaf(part[3], s1, x[nt][3]);
            }
        }
        const uint32_t knan0 = nan_bytes(ks[0]), knan1 = nan_bytes(ks[1]);
        if (__any_sync(0xFFFFFFFFu, (knan0 | knan1) != 0u)) {
            const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                x[nt][0] = knan0 ? nan : x[nt][0];
                x[nt][1] = knan0 ? nan : x[nt][1];
                x[nt][2] = knan1 ? nan : x[nt][2];
                x[nt][3] = knan1 ? nan : x[nt][3];
            }
        }
        // ------------------------------------------- mask, online softmax
        // a lane holds tokens g and g + 8 of rows 2 qd and 2 qd + 1
        const bool edge = t0 + kStep > ctx || t0 + kStep > t_end;
        uint32_t vis[NT][2];
        if (edge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = (8 * nt + 2 * qd + e) % ROWS;
                    const int i = rr / p.group;
                    vis[nt][e] = rr < rows ? visible32(p, q_start + i, i, n, t0 - ctx) : 0u;
                    if (t_end - t0 < kStep)
                        vis[nt][e] &= (1u << (t_end - t0)) - 1u;
                }
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float& x0 = x[nt][e];
                float& x1 = x[nt][2 + e];
                x0 *= qs[nt][e];
                x1 *= qs[nt][e];
                if (edge) {
                    x0 = (vis[nt][e] >> g) & 1u ? x0 : -INFINITY;
                    x1 = (vis[nt][e] >> (g + 8)) & 1u ? x1 : -INFINITY;
                }
                // the running maximum moves only when a score passes it by 2^8: the
                // sums stay far from overflow and most steps skip the rescaling
                grow = grow || fmaxf(x0, x1) > m[nt][e] + 8.0f;
            }
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(x[nt][e], x[nt][2 + e]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
                    const float now = fmaxf(m[nt][e], mx);
                    const float f = now == -INFINITY ? 1.0f : exp2_approx(m[nt][e] - now);
                    m[nt][e] = now;
                    l[nt][e] *= f;
#pragma unroll
                    for (int mt = 0; mt < S::MT; ++mt) {
                        o[mt][nt][e] *= f;
                        o[mt][nt][2 + e] *= f;
                    }
                }
        }
        // P^T fragments: tokens 2 qd, 2 qd + 1 (and + 8) of column g; columns that repeat a
        // row take what the rounding of its probabilities left
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ref = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
                pr[e] = exp2_approx(x[nt][e] - ref);
                pr[2 + e] = exp2_approx(x[nt][2 + e] - ref);
                l[nt][e] += pr[e] + pr[2 + e];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t v = pack2(pr[2 * j], pr[2 * j + 1]);
                if (TWICE) {
                    const uint32_t rest = pack2(pr[2 * j] - __uint_as_float(v << 16),
                                                pr[2 * j + 1] - __uint_as_float(v & 0xFFFF0000u));
                    v = qd >= 2 ? rest : v;
                }
                pf[nt][j] = movmatrix_trans(v);
            }
        }

        // -------------------------------------------------- O^T += V^T P^T
        uint32_t bad = 0;  // edge steps: tokens whose block is NaN, kept out of the product
        if (edge) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool nan = vs[j] == 0xFFu;
                bad |= nan ? 1u << (2 * qd + (j & 1) + 8 * (j >> 1)) : 0u;
                vs[j] = nan ? 0u : vs[j];
            }
        }
        const uint32_t vm0 = block_multiplier<kFmt>(vs[0]) | (block_multiplier<kFmt>(vs[1]) << 16);
        const uint32_t vm1 = block_multiplier<kFmt>(vs[2]) | (block_multiplier<kFmt>(vs[3]) << 16);
        uint32_t vw[4][S::VW];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            read_words<S::VW>(step + S::CODES + S::place(2 * qd + (j & 1) + 8 * (j >> 1), g * (4 * S::VW)), vw[j]);
        // two bytes of token 2 qd beside the same two of token 2 qd + 1
#pragma unroll
        for (int h = 0; h < 2 * S::VW; ++h) {
            const uint32_t pick = h & 1 ? 0x7632u : 0x5410u;
            uint32_t p0[S::PAIRS], p1[S::PAIRS];
            place_codes<kFmt>(__byte_perm(vw[0][h >> 1], vw[1][h >> 1], pick), p0);
            place_codes<kFmt>(__byte_perm(vw[2][h >> 1], vw[3][h >> 1], pick), p1);
#pragma unroll
            for (int s = 0; s < S::PAIRS; s += 2) {
                // elements 2 mt and 2 mt + 1 of the lane's run: rows g and g + 8 of A
                const uint32_t a[4] = {mul_bf16x2(p0[s], vm0), mul_bf16x2(p0[s + 1], vm0), mul_bf16x2(p1[s], vm1),
                                       mul_bf16x2(p1[s + 1], vm1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(o[(h * S::PAIRS + s) / 2][nt], a, pf[nt][0], pf[nt][1]);
            }
        }
        if (edge && __any_sync(0xFFFFFFFFu, bad != 0u)) {
            // a NaN value reaches exactly the rows that see its token
            bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 1);
            bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (vis[nt][e] & bad) {
#pragma unroll
                        for (int mt = 0; mt < S::MT; ++mt)
                            o[mt][nt][e] = o[mt][nt][2 + e] = __uint_as_float(0x7FC00000u);
                    }
        }
    }
    cp_async_wait<0>();
    __syncthreads();  // the ring's memory takes the results

    // ------------------------------------------------- join the warps
    float* sm_ml = smem;                         // [kWarps][COLS][2]
    float* sm_o = smem + kWarps * COLS * 2;      // [kWarps][COLS][kDim]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float s = l[nt][e];
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
            const int r = 8 * nt + 2 * qd + e;
            if (g == 0) {
                sm_ml[(warp * COLS + r) * 2] = m[nt][e];
                sm_ml[(warp * COLS + r) * 2 + 1] = s;
            }
            float* dst = sm_o + (warp * COLS + r) * kDim + g * (kDim / 8);
#pragma unroll
            for (int mt = 0; mt < S::MT; ++mt) {
                // accumulator rows g and g + 8 are elements 2 mt and 2 mt + 1 of the lane's run
                dst[2 * mt] = o[mt][nt][e];
                dst[2 * mt + 1] = o[mt][nt][2 + e];
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (kDim / 2); i += kWarps * 32) {
        const int r = i / (kDim / 2), d = (i - r * (kDim / 2)) * 2;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            mx = fmaxf(mx, sm_ml[(w * COLS + r) * 2]);
        float a0 = 0.0f, a1 = 0.0f, ls = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_ml[(w * COLS + r) * 2];
            const float lw = sm_ml[(w * COLS + r) * 2 + 1];
            // a warp without a visible token has m = -inf and zero sums (or NaN sums, which count)
            const float f = mw == -INFINITY ? 1.0f : exp2_approx(mw - mx);
            const float* po = sm_o + (w * COLS + r) * kDim + d;
            a0 += f * (TWICE ? po[0] + po[ROWS * kDim] : po[0]);
            a1 += f * (TWICE ? po[1] + po[ROWS * kDim + 1] : po[1]);
            ls += f * lw;
        }
        a0 *= kUnscale;
        a1 *= kUnscale;
        const int ri = r / p.group;
        const int64_t tok = q_start + ri;
        const int hq = head * p.group + r - ri * p.group;
        if (splits == 1) {
            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
            *reinterpret_cast<uint32_t*>(p.out + tok * p.ot + hq * p.oh + d) = pack2(a0 * inv, a1 * inv);
            if (d == 0 && p.lse != nullptr)
                p.lse[tok * p.q_heads + hq] = (mx + log2f(ls)) * 0.69314718055994531f;
        } else {
            const int64_t at = (static_cast<int64_t>(blockIdx.x) * p.T + tok) * p.q_heads + hq;
            *reinterpret_cast<float2*>(p.part_o + at * kDim + d) = make_float2(a0, a1);
            if (d == 0)
                *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mx, ls);
        }
    }
}

// Joins the splits of a row.
constexpr int kJoinWarps = 4;

template <int kDim>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_attention_join_kernel(const AttnParams p)
{
    __shared__ JoinScratch<kDim, kJoinWarps> scratch;
    grid_dependency_wait();
    launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t total = static_cast<int64_t>(p.T) * p.q_heads;
    const int tok = static_cast<int>(row / p.q_heads);
    const int hq = static_cast<int>(row - static_cast<int64_t>(tok) * p.q_heads);
    int q_start, n;
    const int b = sequence_of(p, tok);
    group_rows(p.q_offsets, b, p.T, &q_start, &n);
    if (tok < q_start || tok >= q_start + min(n, p.max_draft))
        return;
    const int ctx = max(min(__ldg(p.context_lens + b), p.max_len - n), 0);
    const int splits = min((min(ctx + n, p.max_len) + p.chunk - 1) / p.chunk, kMaxSplits);
    if (splits <= 1)
        return;  // written by the split itself
    join_row<kDim, kJoinWarps>(p, &scratch, tok, hq, splits, [&](int s) { return s * total + row; });
}

// How the work is cut: rows per tile (4, 8 or 16: the kernel above; 32 and 128:
// the tile and row kernels, which cut the contexts themselves), row tiles per key/value head,
// and for the kernel above the tokens per split.
struct Plan {
    int rows;
    int row_tiles;
    int chunk;
    int splits;  // at max_seq
    bool tile;
    int part_rows;  // of a partial result of the tile and row kernels
};

Plan make_plan(int batch, int kv_heads, int group, int64_t max_seq, int max_draft)
{
    Plan pl;
    const int rows = group * max_draft;
    // Up to 32 rows the tile kernel: 8 tokens x 4 heads over 4000 tokens, 64
    // sequences, 141 us with MXFP4 and 156 with MXFP8 (the row kernel 164 and 168).
    // Above that the row kernel: 31 tokens over 16001, 8 sequences, 78 and 84 us
    // (a tile kernel with units of 128 rows 113 and 140); 15 tokens 72 and 77
    // (with units of 64 rows 78 and 125).
    pl.rows = rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
    pl.row_tiles = (rows + pl.rows - 1) / pl.rows;
    pl.tile = pl.rows > 16;
    pl.part_rows = std::min(pl.rows, (rows + 31) / 32 * 32);
    const int64_t units = static_cast<int64_t>(batch) * kv_heads * pl.row_tiles;
    // Eight steps a warp at least, so that a context of up to 512 tokens is done
    // without a second kernel (503 tokens, 8 heads: 9.3 us against 13 us cut in
    // two), and about 16 CTAs per SM, four of them resident (64 sequences up to
    // 8190 tokens: 152 / 145 / 149 us with 8 / 16 / 32).
    constexpr int64_t least = 8 * kWarps * kStep, unit = kWarps * kStep;
    const int64_t ctas = static_cast<int64_t>(sm_count()) * 16;
    const int64_t want = std::min<int64_t>(std::max<int64_t>(1, (ctas + units - 1) / units), kMaxSplits);
    const int64_t chunk = std::max(least, ((max_seq + want - 1) / want + unit - 1) / unit * unit);
    pl.chunk = static_cast<int>(chunk);
    pl.splits = pl.tile ? 1 : static_cast<int>((max_seq + chunk - 1) / chunk);
    return pl;
}

template <int kFmt, int kDim, int ROWS>
cudaError_t launch_stream(const AttnParams& p, const Plan& pl, cudaStream_t stream)
{
    // the ring, and in the same memory the warps' results
    constexpr int cols = std::max(ROWS, 8);
    constexpr int smem = std::max(kWarps * kStages * Shape<kFmt, kDim>::STEP_BYTES, kWarps * cols * (kDim + 2) * 4);
    auto kern = kv_attention_kernel<kFmt, kDim, ROWS>;
    if constexpr (smem > 48 * 1024) {
        // per device and context, once: the shared-memory opt-in
        static std::mutex mu;
        static unsigned long long configured[64] = {};
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess || dev < 0 || dev >= 64)
            return err != cudaSuccess ? err : cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (err != cudaSuccess)
                return err;
            configured[dev] = ctx;
        }
    }
    const dim3 grid(pl.splits, p.cache.heads, p.batch);
    return launch_pdl(kern, grid, dim3(kWarps * 32), smem, stream, p);
}

template <int kFmt, int kDim>
cudaError_t launch_rows(const AttnParams& p, const Plan& pl, cudaStream_t stream)
{
    cudaError_t err = pl.rows == 4    ? launch_stream<kFmt, kDim, 4>(p, pl, stream)
                      : pl.rows == 8  ? launch_stream<kFmt, kDim, 8>(p, pl, stream)
                                      : launch_stream<kFmt, kDim, 16>(p, pl, stream);
    if (err != cudaSuccess || pl.splits <= 1)
        return err;
    const int64_t rows = static_cast<int64_t>(p.T) * p.q_heads;
    return launch_pdl(kv_attention_join_kernel<kDim>, dim3(static_cast<unsigned>(rows)), dim3(kJoinWarps * 32), 0,
                      stream, p);
}

}  // namespace

// int64 [batch + 1] before the partial results, which start on 16 bytes
static size_t prefix_words(int batch) { return (static_cast<size_t>(batch) + 2) / 2 * 2; }

size_t kv_attention_workspace_bytes(int batch, int64_t T, int q_heads, int kv_heads, int dim, int64_t max_seq,
                                    int max_draft)
{
    const Plan pl = make_plan(batch, kv_heads, q_heads / kv_heads, max_seq, max_draft);
    if (pl.tile)  // the sequences' first tiles, and two partial results per CTA
        return prefix_words(batch) * sizeof(int64_t) + static_cast<size_t>(2 * sm_count()) * pl.part_rows * (dim + 2) * sizeof(float);
    if (pl.splits <= 1)
        return 0;
    return static_cast<size_t>(pl.splits) * T * q_heads * (dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream)
{
    const Plan pl = make_plan(a.batch, a.cache.heads, a.q_heads / a.cache.heads, a.max_seq, a.max_draft);
    AttnParams p;
    p.cache = a.cache;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.qt = a.qt, p.qh = a.qh, p.ot = a.ot, p.oh = a.oh;
    p.block_table = a.block_table;
    p.table_stride = a.table_stride;
    p.context_lens = a.context_lens;
    p.q_offsets = a.q_offsets;
    p.mask = a.tree_mask;
    p.mask_words = a.mask_words;
    p.batch = a.batch;
    p.T = static_cast<int>(a.T);
    p.q_heads = a.q_heads;
    p.group = a.q_heads / a.cache.heads;
    p.row_tiles = pl.row_tiles;
    p.max_draft = a.max_draft;
    p.chunk = pl.chunk;
    p.whole = a.max_seq <= 512;
    p.prefix = nullptr;
    p.page_div = div_magic(static_cast<uint32_t>(a.cache.page_size));
    p.group_div = div_magic(static_cast<uint32_t>(p.group));
    p.max_len = static_cast<int>(std::min<int64_t>(a.max_seq, a.table_stride * a.cache.page_size));
    p.xscale = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    p.status = a.status;
    p.withhold = a.withhold;
    p.part_rows = pl.part_rows;
    if (pl.tile) {
        p.xscale *= kUnscale;  // scores come out of the MMA times 2^-64
        p.prefix = static_cast<int64_t*>(a.workspace);
        p.part_o = reinterpret_cast<float*>(p.prefix + prefix_words(a.batch));
        p.part_ml = p.part_o + static_cast<size_t>(2 * sm_count()) * pl.part_rows * a.cache.dim;
        return pl.rows == 32 ? launch_kv_attention_tile(p, stream) : launch_kv_attention_rows(p, stream);
    }
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o + static_cast<size_t>(pl.splits) * a.T * a.q_heads * a.cache.dim;
    if (a.cache.format == kKvMxfp8)
        return a.cache.dim == 128 ? launch_rows<kKvMxfp8, 128>(p, pl, stream)
                                    : launch_rows<kKvMxfp8, 64>(p, pl, stream);
    return a.cache.dim == 128 ? launch_rows<kKvMxfp4, 128>(p, pl, stream)
                              : launch_rows<kKvMxfp4, 64>(p, pl, stream);
}

}  // namespace fp4lin
