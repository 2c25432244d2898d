// kv_cache.h -- arguments shared by the rotary-position, key/value cache and
// attention kernels and the C ABI layer.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp4lin {

// Formats of the cache (the numbers of FP4_ACT_MXFP4 and FP4_ACT_MXFP8).
enum : int { kKvMxfp4 = 0, kKvMxfp8 = 1 };
// Rotary layouts and scalings (the numbers of fp4_rope_layout, fp4_rope_scaling_kind).
enum : int { kRopeHalf = 0, kRopeInterleaved = 1 };
enum : int { kRopeNone = 0, kRopeLinear = 1, kRopeByParts = 2 };

// codes [pages][heads][page_size][dim or dim / 2 bytes],
// scales [pages][heads][page_size][dim / 32]
struct KvCache {
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
    int64_t pages;
    int page_size;
    int heads;
    int dim;
    int format;
};

struct RopeArgs {
    const float* table;  // [table_positions][rot]: rot / 2 cosines, rot / 2 sines
    int64_t table_positions;
    const int32_t* positions;  // [T]
    int rot;                   // 0: no rotation
    int layout;
    int inverse;
};

struct RopeFrequencies {
    double base;
    int scaling;
    double factor;
    double low, high;  // ramp of the by-parts scaling, in frequency indexes
    double magnitude;  // factor on cosines and sines
};

cudaError_t launch_rope_table(float* table, int64_t positions, int rot, const RopeFrequencies& f, cudaStream_t stream);
cudaError_t launch_rope(const void* x, void* out, const RopeArgs& rope, int64_t T, int heads, int dim, int64_t xt,
                        int64_t xh, int64_t ot, int64_t oh, cudaStream_t stream);
cudaError_t launch_kv_append(const KvCache& cache, const void* k, const void* v, int64_t T, int64_t kt, int64_t kh,
                             int64_t vt, int64_t vh, const int64_t* slots, const RopeArgs& rope, cudaStream_t stream);
cudaError_t launch_kv_read(const KvCache& cache, const int32_t* block_table, int64_t table_stride,
                           const int32_t* cu_lens, int batch, int64_t rows, void* k, void* v, cudaStream_t stream);

struct KvAttentionArgs {
    KvCache cache;
    const void* q;
    void* out;
    float* lse;  // nullable
    int64_t qt, qh, ot, oh;
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    const uint32_t* tree_mask;  // nullable: causal
    int mask_words;
    int batch;
    int64_t T;
    int q_heads;
    int64_t max_seq;
    int max_draft;
    float scale;
    void* workspace;
    unsigned int* status;
    unsigned long long wait_ns;
    bool withhold;  // test hook
};

size_t kv_attention_workspace_bytes(int batch, int64_t T, int q_heads, int kv_heads, int dim, int64_t max_seq,
                                    int max_draft);
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream);

}  // namespace fp4lin
