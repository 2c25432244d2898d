// kv_attention.cuh -- what the two attention kernels over the MX-quantized
// cache share: the launch's parameters and the exact bf16 form of a code.
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
    int row_tiles;
    int chunk;      // tokens per split, a multiple of 64 (stream) or 128 (tile)
    DivMagic page_div;  // by the page size
    DivMagic group_div;  // by the query heads per key/value head
    int max_len;    // tokens a sequence's block table row can name
    float xscale;   // scale * log2(e)
    float* part_o;  // [splits][T * q_heads][dim]
    float* part_ml; // [splits][T * q_heads][2]
    unsigned long long wait_ns;  // limit of the bounded device waits, and where they report
    unsigned int* status;
};

// The kernel of many rows (kv_attention_tile.cu): row tiles of 32, 64 or 128
// rows, chunks of a multiple of 128 tokens.
cudaError_t launch_kv_attention_tile(const AttnParams& p, int rows, int splits, cudaStream_t stream);

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

}  // namespace fp4lin
