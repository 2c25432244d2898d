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
// V serve every column tile.  The order of a dot product's elements and of
// the tokens inside a step is free, so each lane simply takes contiguous
// bytes: of a key a quarter head (a lane of the quad), of a value 1/8 head of
// four tokens.  Codes go from global memory to registers to MMA fragments;
// shared memory only holds the per-warp results at the end.
//
// Elements become bf16 exactly: the code's bits are placed in the bf16's
// exponent and mantissa fields (subnormals included), which makes the value
// 2^-120 (E4M3) or 2^-126 (E2M1) of the code's, and one bf16 multiply by a
// power of two applies the block's scale.  That multiplier carries 2^-64 (put
// back in fp32 at the end), so that it stays a finite bf16 up to values of
// 2^66.  Scores, softmax statistics and sums are fp32; the probabilities are
// rounded to bf16 for the second product (relative 2^-8 at most, of the size of the
// output's own rounding), their sum is taken before that rounding.
#include <cuda_bf16.h>

#include <algorithm>

#include "formats.cuh"
#include "internal.h"
#include "kv_cache.h"
#include "ptx.cuh"

namespace fp4lin {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;         // tokens a warp takes at a time
constexpr float kUnscale = 18446744073709551616.0f;  // 2^64
constexpr int kScaleShift = 64;

struct AttnParams {
    KvCache cache;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    int64_t qt, qh, ot, oh;
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    const uint32_t* mask;
    int mask_words;
    int batch;
    int T;
    int q_heads;
    int group;
    int row_tiles;
    int chunk;      // tokens per split, a multiple of kWarps * kStep
    int max_len;    // tokens a sequence's block table row can name
    float xscale;   // scale * log2(e) * 2^64
    float* part_o;  // [splits][T * q_heads][dim]
    float* part_ml; // [splits][T * q_heads][2]
};

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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// bf16 bits of the multiplier of a block: 2^(s - 127) times the placement's
// 2^120 (E4M3) or 2^126 (E2M1) times 2^-64; NaN for the NaN scale.
template <int kFmt>
__device__ __forceinline__ uint32_t block_multiplier(uint32_t s)
{
    const uint32_t field = min(s + (kFmt == kKvMxfp8 ? 120u : 126u) - kScaleShift, 254u);
    return s == 0xFFu ? 0x7FC0u : field << 7;
}

// Two E4M3 codes in the high bytes of the halves -> bf16 pair (times 2^-120).
__device__ __forceinline__ uint32_t place_e4m3(uint32_t p)
{
    return (p & 0x80008000u) | ((p >> 4) & 0x07F007F0u);
}

// Dimensions: a lane holds dim / 4 elements of a key (KB bytes) and dim / 8
// of a value (VB bytes).
template <int kFmt, int kDim>
struct Shape {
    static constexpr int BITS = kFmt == kKvMxfp8 ? 8 : 4;
    static constexpr int ROW = kDim * BITS / 8;  // code bytes of a token
    static constexpr int KW = ROW / 16;          // 32-bit words of a key per lane
    static constexpr int VW = ROW / 32;          // 32-bit words of a value per lane
    static constexpr int KSTEPS = kDim / 16;
    static constexpr int MT = kDim / 16;         // 16-element tiles of the output
    static constexpr int SB = kDim / 32;         // scale bytes of a token
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* r, bool live)
{
    if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(p) + i / 4) : make_uint4(0u, 0u, 0u, 0u);
            r[i] = v.x, r[i + 1] = v.y, r[i + 2] = v.z, r[i + 3] = v.w;
        }
    } else if constexpr (W == 2) {
        const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0u, 0u);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = live ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    }
}

// The 16 visibility bits of row `node` for tokens base ... base + 15 relative
// to the end of the context (negative: context tokens, always seen).
__device__ __forceinline__ uint32_t visible16(const AttnParams& p, int64_t token, int node, int n, int base)
{
    uint32_t bits = 0;
    const int lo = max(base, 0);
    if (lo < n) {
        if (p.mask != nullptr) {
            const uint32_t* m = p.mask + token * p.mask_words;
            const int w = lo >> 5;
            const uint32_t w0 = w < p.mask_words ? __ldg(m + w) : 0u;
            const uint32_t w1 = w + 1 < p.mask_words ? __ldg(m + w + 1) : 0u;
            bits = __funnelshift_r(w0, w1, lo & 31);
        } else {
            const int k = node - lo;  // the row sees tokens up to itself
            bits = k < 0 ? 0u : k >= 31 ? 0xFFFFFFFFu : (2u << k) - 1u;
        }
        if (n - lo < 32)
            bits &= (1u << (n - lo)) - 1u;
    }
    if (base < 0)
        bits = base <= -16 ? 0xFFFFu : (bits << -base) | ((1u << -base) - 1u);
    return bits & 0xFFFFu;
}

template <int kFmt, int kDim, int NT>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(const AttnParams p)
{
    using S = Shape<kFmt, kDim>;
    constexpr int ROWS = 8 * NT;
    extern __shared__ float smem[];  // [kWarps][ROWS][2] then [kWarps][ROWS][kDim]
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, qd = lane & 3;
    const int b = blockIdx.z;
    const int head = blockIdx.y / p.row_tiles;
    const int row0 = (blockIdx.y - head * p.row_tiles) * ROWS;
    int q_start, n;
    group_rows(p.q_offsets, b, p.T, &q_start, &n);
    if (row0 >= n * p.group)
        return;
    const int ctx = max(min(__ldg(p.context_lens + b), p.max_len - n), 0);
    const int len = min(ctx + n, p.max_len);
    const int t_begin = blockIdx.x * p.chunk;
    if (t_begin >= len)
        return;
    const int t_end = min(len, t_begin + p.chunk);
    const int rows = min(ROWS, n * p.group - row0);
    const int splits = (len + p.chunk - 1) / p.chunk;

    // this lane's share of Q: row g of each column tile, its quarter of the head,
    // paired as the key codes come out of their words
    uint32_t qf[NT][2 * S::KSTEPS];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + 8 * nt + g;
        const bool live = 8 * nt + g < rows;
        const int i = r / p.group;
        const __nv_bfloat16* src = p.q + static_cast<int64_t>(q_start + i) * p.qt +
                                   static_cast<int64_t>(head * p.group + r - i * p.group) * p.qh + qd * (kDim / 4);
        uint32_t w[kDim / 8];
#pragma unroll
        for (int k = 0; k < kDim / 8; k += 4) {
            const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 2 * k) : make_uint4(0u, 0u, 0u, 0u);
            w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
        }
        if constexpr (kFmt == kKvMxfp8) {
#pragma unroll
            for (int k = 0; k < kDim / 8; ++k)
                qf[nt][k] = w[k];
        } else {
            // eight codes of a word pair up as (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
            for (int k = 0; k < kDim / 8; k += 4) {
                qf[nt][k] = __byte_perm(w[k], w[k + 2], 0x5410);
                qf[nt][k + 1] = __byte_perm(w[k], w[k + 2], 0x7632);
                qf[nt][k + 2] = __byte_perm(w[k + 1], w[k + 3], 0x5410);
                qf[nt][k + 3] = __byte_perm(w[k + 1], w[k + 3], 0x7632);
            }
        }
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

    uint32_t kw[2][S::KW], vw[4][S::VW], ks[2], vs[4];
    // codes and scales of the 16 tokens at t0 (all in one page: page sizes are
    // multiples of 16); tokens past the end come as zeros
    auto token_base = [&](int t0) -> int64_t {
        const int pi = t0 / p.cache.page_size;
        const int64_t page = min(max(static_cast<int64_t>(__ldg(p.block_table + b * p.table_stride + pi)), int64_t(0)),
                                 p.cache.pages - 1);
        return (page * p.cache.heads + head) * p.cache.page_size + (t0 - pi * p.cache.page_size);
    };
    auto load_k = [&](int64_t base, int left) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = g + 8 * j;
            const bool live = t < left;
            load_words<S::KW>(p.cache.k_codes + (base + t) * S::ROW + qd * (4 * S::KW), kw[j], live);
            ks[j] = live ? __ldg(p.cache.k_scales + (base + t) * S::SB + qd * S::SB / 4) : 0u;
        }
    };
    auto load_v = [&](int64_t base, int left) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 2 * qd + (j & 1) + 8 * (j >> 1);
            const bool live = t < left;
            load_words<S::VW>(p.cache.v_codes + (base + t) * S::ROW + g * (4 * S::VW), vw[j], live);
            vs[j] = live ? __ldg(p.cache.v_scales + (base + t) * S::SB + g * S::SB / 8) : 0u;
        }
    };

    int t0 = t_begin + warp * kStep;
    int64_t base = 0;
    if (t0 < t_end) {
        base = token_base(t0);
        load_k(base, t_end - t0);
        load_v(base, t_end - t0);
    }
    for (; t0 < t_end; t0 += kWarps * kStep) {
        const int next = t0 + kWarps * kStep;
        const bool more = next < t_end;
        const int64_t next_base = more ? token_base(next) : 0;

        // ---------------------------------------------------- S^T = K Q^T
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
        const uint32_t km0 = block_multiplier<kFmt>(ks[0]) * 0x10001u;
        const uint32_t km1 = block_multiplier<kFmt>(ks[1]) * 0x10001u;
        if constexpr (kFmt == kKvMxfp8) {
#pragma unroll
            for (int s = 0; s < S::KSTEPS; ++s) {
                uint32_t a[4];
                a[0] = mul_bf16x2(place_e4m3(__byte_perm(kw[0][s], 0u, 0x1404)), km0);
                a[1] = mul_bf16x2(place_e4m3(__byte_perm(kw[1][s], 0u, 0x1404)), km1);
                a[2] = mul_bf16x2(place_e4m3(__byte_perm(kw[0][s], 0u, 0x3424)), km0);
                a[3] = mul_bf16x2(place_e4m3(__byte_perm(kw[1][s], 0u, 0x3424)), km1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(x[nt], a, qf[nt][2 * s], qf[nt][2 * s + 1]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S::KSTEPS; ++s) {
                const uint32_t w0 = kw[0][s >> 1], w1 = kw[1][s >> 1];
                uint32_t a[4];
                if ((s & 1) == 0) {
                    a[0] = ((w0 << 12) & 0x80008000u) | ((w0 << 6) & 0x01C001C0u);
                    a[1] = ((w1 << 12) & 0x80008000u) | ((w1 << 6) & 0x01C001C0u);
                    a[2] = ((w0 << 8) & 0x80008000u) | ((w0 << 2) & 0x01C001C0u);
                    a[3] = ((w1 << 8) & 0x80008000u) | ((w1 << 2) & 0x01C001C0u);
                } else {
                    a[0] = ((w0 << 4) & 0x80008000u) | ((w0 >> 2) & 0x01C001C0u);
                    a[1] = ((w1 << 4) & 0x80008000u) | ((w1 >> 2) & 0x01C001C0u);
                    a[2] = (w0 & 0x80008000u) | ((w0 >> 6) & 0x01C001C0u);
                    a[3] = (w1 & 0x80008000u) | ((w1 >> 6) & 0x01C001C0u);
                }
                a[0] = mul_bf16x2(a[0], km0);
                a[1] = mul_bf16x2(a[1], km1);
                a[2] = mul_bf16x2(a[2], km0);
                a[3] = mul_bf16x2(a[3], km1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(x[nt], a, qf[nt][2 * s], qf[nt][2 * s + 1]);
            }
        }
        if (more)
            load_k(next_base, t_end - next);

        // ------------------------------------------- mask, online softmax
        // a lane holds tokens g and g + 8 of rows 2 qd and 2 qd + 1
        const bool edge = t0 + kStep > ctx || t0 + kStep > t_end;
        uint32_t vis[NT][2];
        if (edge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = 8 * nt + 2 * qd + e;
                    const int i = (row0 + rr) / p.group;
                    vis[nt][e] = rr < rows ? visible16(p, q_start + i, i, n, t0 - ctx) : 0u;
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
                x0 *= p.xscale;
                x1 *= p.xscale;
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
        uint32_t pf[NT][2];  // P^T fragments: tokens 2 qd, 2 qd + 1 (and + 8) of row g
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
            pf[nt][0] = movmatrix_trans(pack2(pr[0], pr[1]));
            pf[nt][1] = movmatrix_trans(pack2(pr[2], pr[3]));
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
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt) {
            uint32_t a[4];
            if constexpr (kFmt == kKvMxfp8) {
                // elements 2 mt and 2 mt + 1 of the lane's run
                constexpr uint32_t pick[4] = {0x4400u, 0x5511u, 0x6622u, 0x7733u};
                const int w = mt >> 1, e0 = (mt & 1) * 2;
                a[0] = mul_bf16x2(place_e4m3(__byte_perm(vw[0][w], vw[1][w], pick[e0])), vm0);
                a[1] = mul_bf16x2(place_e4m3(__byte_perm(vw[0][w], vw[1][w], pick[e0 + 1])), vm0);
                a[2] = mul_bf16x2(place_e4m3(__byte_perm(vw[2][w], vw[3][w], pick[e0])), vm1);
                a[3] = mul_bf16x2(place_e4m3(__byte_perm(vw[2][w], vw[3][w], pick[e0 + 1])), vm1);
            } else {
                constexpr uint32_t pick[4] = {0x4400u, 0x5511u, 0x6622u, 0x7733u};
                const int w = mt >> 2, by = mt & 3;
                const uint32_t p0 = __byte_perm(vw[0][w], vw[1][w], pick[by]);
                const uint32_t p1 = __byte_perm(vw[2][w], vw[3][w], pick[by]);
                a[0] = mul_bf16x2(((p0 << 4) & 0x80008000u) | ((p0 >> 2) & 0x01C001C0u), vm0);
                a[1] = mul_bf16x2((p0 & 0x80008000u) | ((p0 >> 6) & 0x01C001C0u), vm0);
                a[2] = mul_bf16x2(((p1 << 4) & 0x80008000u) | ((p1 >> 2) & 0x01C001C0u), vm1);
                a[3] = mul_bf16x2((p1 & 0x80008000u) | ((p1 >> 6) & 0x01C001C0u), vm1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_bf16(o[mt][nt], a, pf[nt][0], pf[nt][1]);
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
        if (more)
            load_v(next_base, t_end - next);
    }

    // ------------------------------------------------- join the warps
    float* sm_ml = smem;                         // [kWarps][ROWS][2]
    float* sm_o = smem + kWarps * ROWS * 2;      // [kWarps][ROWS][kDim]
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
                sm_ml[(warp * ROWS + r) * 2] = m[nt][e];
                sm_ml[(warp * ROWS + r) * 2 + 1] = s;
            }
            float* dst = sm_o + (warp * ROWS + r) * kDim + g * (kDim / 8);
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
            mx = fmaxf(mx, sm_ml[(w * ROWS + r) * 2]);
        float a0 = 0.0f, a1 = 0.0f, ls = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_ml[(w * ROWS + r) * 2];
            const float lw = sm_ml[(w * ROWS + r) * 2 + 1];
            // a warp without a visible token has m = -inf and zero sums (or NaN sums, which count)
            const float f = mw == -INFINITY ? 1.0f : exp2_approx(mw - mx);
            a0 += f * sm_o[(w * ROWS + r) * kDim + d];
            a1 += f * sm_o[(w * ROWS + r) * kDim + d + 1];
            ls += f * lw;
        }
        a0 *= kUnscale;
        a1 *= kUnscale;
        const int ri = (row0 + r) / p.group;
        const int64_t tok = q_start + ri;
        const int hq = head * p.group + row0 + r - ri * p.group;
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

// Joins the splits of a row, in their order: one warp per row.
template <int kDim>
__global__ void __launch_bounds__(128) kv_attention_join_kernel(const AttnParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int64_t total = static_cast<int64_t>(p.T) * p.q_heads;
    if (row >= total)
        return;
    const int tok = static_cast<int>(row / p.q_heads);
    const int hq = static_cast<int>(row - static_cast<int64_t>(tok) * p.q_heads);
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.q_offsets + mid) <= tok)
            lo = mid;
        else
            hi = mid;
    }
    int q_start, n;
    group_rows(p.q_offsets, lo, p.T, &q_start, &n);
    if (tok < q_start || tok >= q_start + n)
        return;
    const int ctx = max(min(__ldg(p.context_lens + lo), p.max_len - n), 0);
    const int splits = (min(ctx + n, p.max_len) + p.chunk - 1) / p.chunk;
    if (splits <= 1)
        return;
    float mx = -INFINITY;
    for (int s = lane; s < splits; s += 32)
        mx = fmaxf(mx, p.part_ml[(s * total + row) * 2]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    constexpr int W = kDim / 32;
    float acc[W] = {};
    float ls = 0.0f;
    for (int s = 0; s < splits; ++s) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (s * total + row) * 2);
        const float f = ml.x == -INFINITY ? 1.0f : exp2_approx(ml.x - mx);
        ls += f * ml.y;
        const float* src = p.part_o + (s * total + row) * kDim + lane * W;
#pragma unroll
        for (int j = 0; j < W; ++j)
            acc[j] += f * src[j];
    }
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    __nv_bfloat16* out = p.out + tok * p.ot + hq * p.oh + lane * W;
#pragma unroll
    for (int j = 0; j < W; j += 2)
        *reinterpret_cast<uint32_t*>(out + j) = pack2(acc[j] * inv, acc[j + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = (mx + log2f(ls)) * 0.69314718055994531f;
}

// How the work is cut: column tiles per warp, row tiles per key/value head,
// tokens per split.
struct Plan {
    int nt;
    int row_tiles;
    int chunk;
    int splits;  // at max_seq
};

Plan make_plan(int batch, int kv_heads, int group, int64_t max_seq, int max_draft)
{
    Plan pl;
    const int rows = group * max_draft;
    pl.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    pl.row_tiles = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
    const int64_t units = static_cast<int64_t>(batch) * kv_heads * pl.row_tiles;
    constexpr int kMin = 4 * kWarps * kStep;  // four steps a warp at least
    const int64_t want = std::max<int64_t>(1, (static_cast<int64_t>(sm_count()) * 8 + units - 1) / units);
    int64_t chunk = (max_seq + want - 1) / want;
    chunk = std::max<int64_t>(kMin, (chunk + kWarps * kStep - 1) / (kWarps * kStep) * (kWarps * kStep));
    pl.chunk = static_cast<int>(chunk);
    pl.splits = static_cast<int>((max_seq + chunk - 1) / chunk);
    return pl;
}

template <int kFmt, int kDim, int NT>
cudaError_t launch_stream(const AttnParams& p, const Plan& pl, cudaStream_t stream)
{
    constexpr int smem = kWarps * 8 * NT * (kDim + 2) * 4;
    auto kern = kv_attention_kernel<kFmt, kDim, NT>;
    if constexpr (smem > 48 * 1024) {
        // per device and context, once
        static unsigned long long configured[64] = {};
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess || dev < 0 || dev >= 64)
            return err != cudaSuccess ? err : cudaErrorInvalidDevice;
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (err != cudaSuccess)
                return err;
            configured[dev] = ctx;
        }
    }
    const dim3 grid(pl.splits, p.cache.heads * pl.row_tiles, p.batch);
    return launch_pdl(kern, grid, dim3(kWarps * 32), smem, stream, p);
}

template <int kFmt, int kDim>
cudaError_t launch_rows(const AttnParams& p, const Plan& pl, cudaStream_t stream)
{
    cudaError_t err = pl.nt == 1   ? launch_stream<kFmt, kDim, 1>(p, pl, stream)
                      : pl.nt == 2 ? launch_stream<kFmt, kDim, 2>(p, pl, stream)
                                   : launch_stream<kFmt, kDim, 4>(p, pl, stream);
    if (err != cudaSuccess || pl.splits <= 1)
        return err;
    const int64_t rows = static_cast<int64_t>(p.T) * p.q_heads;
    return launch_pdl(kv_attention_join_kernel<kDim>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream,
                      p);
}

}  // namespace

size_t kv_attention_workspace_bytes(int batch, int64_t T, int q_heads, int kv_heads, int dim, int64_t max_seq,
                                    int max_draft)
{
    const Plan pl = make_plan(batch, kv_heads, q_heads / kv_heads, max_seq, max_draft);
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
    p.chunk = pl.chunk;
    p.max_len = static_cast<int>(std::min<int64_t>(a.max_seq, a.table_stride * a.cache.page_size));
    p.xscale = a.scale * 1.4426950408889634f * kUnscale;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o + static_cast<size_t>(pl.splits) * a.T * a.q_heads * a.cache.dim;
    if (a.cache.format == kKvMxfp8)
        return a.cache.dim == 128 ? launch_rows<kKvMxfp8, 128>(p, pl, stream) : launch_rows<kKvMxfp8, 64>(p, pl, stream);
    return a.cache.dim == 128 ? launch_rows<kKvMxfp4, 128>(p, pl, stream) : launch_rows<kKvMxfp4, 64>(p, pl, stream);
}

}  // namespace fp4lin
