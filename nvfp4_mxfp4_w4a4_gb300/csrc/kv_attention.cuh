// kv_attention.cuh -- what the attention kernels over the MX-quantized cache
// share: the launch's parameters, the exact bf16 form of a code, the tokens that
// a row sees, and the joining of a row's parts.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "formats.cuh"
#include "kv_cache.h"

namespace fp4lin {

constexpr float kUnscale = 18446744073709551616.0f;  // 2^64
constexpr int kScaleShift = 64;
constexpr int kMaxSplits = 1024;  // of one context

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
    int row_tiles;  // of a key head, at most (tile and row kernels)
    int max_draft;  // drafted tokens of a sequence that are computed; those past it give NaN
    int chunk;      // tokens per split (stream kernel)
    DivMagic page_div;  // by the page size
    DivMagic group_div;  // by the query heads per key/value head
    int max_len;    // tokens a sequence's block table row can name
    float xscale;   // scale * log2(e)
    float* part_o;  // [splits][T * q_heads][dim]
    float* part_ml; // [splits][T * q_heads][2]
    unsigned long long wait_ns;  // limit of the bounded device waits, and where they report
    unsigned int* status;
    bool withhold;  // test hook of the tile and row kernels: CTA 0 leaves out its second products
    // tile and row kernels: deal out whole units (short contexts) instead of tiles, and
    // where it leaves the sequences' first tiles and, behind them, a run's length
    bool whole;
    int part_rows;  // rows of a partial result
    int64_t* prefix;
};

// The kernels of 17 to 32 rows and of more (units of 32 and 128 rows), whose
// partial results' rows p.part_rows counts.
cudaError_t launch_kv_attention_tile(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_kv_attention_rows(const AttnParams& p, cudaStream_t stream);

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

// bf16 bits of the multiplier of a value block: 2^(s - 127) times the
// placement's 2^120 (E4M3) or 2^126 (E2M1) times 2^-64; NaN for the NaN scale.
template <int kFmt>
__device__ __forceinline__ uint32_t block_multiplier(uint32_t s)
{
    const uint32_t field = min(s + (kFmt == kKvMxfp8 ? 120u : 126u) - kScaleShift, 254u);
    return s == 0xFFu ? 0x7FC0u : field << 7;
}

// The codes of a word whose halves hold one element each per position, as
// bf16 pairs (times 2^-120 / 2^-126, see above).  These integer operations run
// on the ALU pipe at half the issue rate, so right shifts are kept few and
// left shifts are written as multiplications, which the multiply-add pipe can
// take.
//   E4M3  byte 0 and 2 -> out[0], byte 1 and 3 -> out[1]
//   E2M1  nibble j of both halves -> out[j]
template <int kFmt>
__device__ __forceinline__ void place_codes(uint32_t w, uint32_t* out)
{
    if constexpr (kFmt == kKvMxfp8) {
        out[0] = ((w * 256u) & 0x80008000u) | ((w * 16u) & 0x07F007F0u);
        out[1] = (w & 0x80008000u) | ((w >> 4) & 0x07F007F0u);
    } else {
        const uint32_t w6 = w >> 6;
        out[0] = ((w * 4096u) & 0x80008000u) | ((w * 64u) & 0x01C001C0u);
        out[1] = ((w * 256u) & 0x80008000u) | ((w * 4u) & 0x01C001C0u);
        out[2] = ((w * 16u) & 0x80008000u) | ((w6 * 16u) & 0x01C001C0u);
        out[3] = (w & 0x80008000u) | (w6 & 0x01C001C0u);
    }
}

// The 32 visibility bits of row `node` for tokens base ... base + 31 relative
// to the end of the context (negative: context tokens, always seen); n drafted
// tokens are in the cache.
__device__ __forceinline__ uint32_t visible32(const AttnParams& p, int64_t token, int node, int n, int base)
{
    uint32_t bits = 0;
    const int lo = max(base, 0);
    if (base > -32 && lo < n) {
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
        bits = base <= -32 ? 0xFFFFFFFFu : (bits << -base) | ((1u << -base) - 1u);
    return bits;
}

// The sequence that holds drafted token `tok`: the last that starts at or before it.
__device__ __forceinline__ int sequence_of(const AttnParams& p, int tok)
{
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.q_offsets + mid) <= tok)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The rows of a key head of sequence tokens past the bound: NaN, so that a bound
// which the caller's offsets exceed shows in the results.
__device__ __forceinline__ void void_rows(const AttnParams& p, int head, int q_start, int n, int thread, int threads)
{
    const int vectors = p.cache.dim / 8;
    const int64_t count = static_cast<int64_t>(n - p.max_draft) * p.group * vectors;
#pragma unroll 1
    for (int64_t i = thread; i < count; i += threads) {
        const int64_t row = i / vectors;
        const int d = static_cast<int>(i - row * vectors) * 8;
        const int64_t tok = q_start + p.max_draft + row / p.group;
        const int hq = head * p.group + static_cast<int>(row % p.group);
        *reinterpret_cast<uint4*>(p.out + tok * p.ot + hq * p.oh + d) = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        if (d == 0 && p.lse != nullptr)
            p.lse[tok * p.q_heads + hq] = __uint_as_float(0x7FC00000u);
    }
}

// Joining a row's parts: one CTA per row, for rows with many parts; its warps
// take the parts in turn, and their sums are added in the warps' order.
template <int kDim, int kWarps>
struct JoinScratch {
    float weight[kMaxSplits];
    float red[kWarps];
    float part[kWarps][kDim];
};

// index(s): where part s of the row is in part_o and part_ml, in rows.
template <int kDim, int kJoinWarps, typename Index>
__device__ __forceinline__ void join_row(const AttnParams& p, JoinScratch<kDim, kJoinWarps>* sc, int tok, int hq, int parts, Index index)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float mx = -INFINITY;
    for (int s = threadIdx.x; s < parts; s += kJoinWarps * 32) {
        const float v = ml[index(s)].x;
        sc->weight[s] = v;
        mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    if (lane == 0)
        sc->red[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
        mx = fmaxf(mx, sc->red[w]);
    __syncthreads();
    float ls = 0.0f;
    for (int s = threadIdx.x; s < parts; s += kJoinWarps * 32) {
        // a part without a visible token has m = -inf and zero sums (or NaN sums, which count)
        const float f = sc->weight[s] == -INFINITY ? 1.0f : exp2_approx(sc->weight[s] - mx);
        sc->weight[s] = f;
        ls += f * ml[index(s)].y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        ls += __shfl_xor_sync(0xFFFFFFFFu, ls, d);
    if (lane == 0)
        sc->red[warp] = ls;
    __syncthreads();
    ls = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
        ls += sc->red[w];
    constexpr int W = kDim / 32;
    float acc[W] = {};
#pragma unroll 8
    for (int s = warp; s < parts; s += kJoinWarps) {
        const float f = sc->weight[s];
        const float* src = p.part_o + index(s) * kDim + lane * W;
        if constexpr (W == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            acc[0] += f * v.x, acc[1] += f * v.y;
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
        sc->part[warp][lane * W + j] = acc[j];
    __syncthreads();
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    for (int d = threadIdx.x * 2; d < kDim; d += kJoinWarps * 64) {
        float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            a0 += sc->part[w][d];
            a1 += sc->part[w][d + 1];
        }
        *reinterpret_cast<uint32_t*>(p.out + tok * p.ot + hq * p.oh + d) = pack2(a0 * inv, a1 * inv);
    }
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(tok) * p.q_heads + hq] = (mx + log2f(ls)) * 0.69314718055994531f;
}

// The same by one warp, for rows with a few parts.
template <int kDim, typename Index>
__device__ __forceinline__ void join_row_warp(const AttnParams& p, int tok, int hq, int parts, Index index)
{
    const int lane = threadIdx.x & 31;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float mx = -INFINITY;
    for (int s = lane; s < parts; s += 32)
        mx = fmaxf(mx, ml[index(s)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    constexpr int W = kDim / 32;
    float acc[W] = {}, ls = 0.0f;
#pragma unroll 3
    for (int s = 0; s < parts; ++s) {
        const float2 v = ml[index(s)];
        // a part without a visible token has m = -inf and zero sums (or NaN sums, which count)
        const float f = v.x == -INFINITY ? 1.0f : exp2_approx(v.x - mx);
        ls += f * v.y;
        const float* src = p.part_o + index(s) * kDim + lane * W;
        if constexpr (W == 4) {
            const float4 o = *reinterpret_cast<const float4*>(src);
            acc[0] += f * o.x, acc[1] += f * o.y, acc[2] += f * o.z, acc[3] += f * o.w;
        } else {
            const float2 o = *reinterpret_cast<const float2*>(src);
            acc[0] += f * o.x, acc[1] += f * o.y;
        }
    }
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + tok * p.ot + hq * p.oh + lane * W);
    if constexpr (W == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
    else
        *dst = pack2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(tok) * p.q_heads + hq] = (mx + log2f(ls)) * 0.69314718055994531f;
}

}  // namespace fp4lin
