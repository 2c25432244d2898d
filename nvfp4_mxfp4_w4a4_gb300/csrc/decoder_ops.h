// decoder_ops.h -- arguments shared by the kernels of head norms, prompt
// attention, matrix-vector products and expert dispatch and the C ABI layer.
// Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_cache.h"

namespace fp4lin {

// Queries (part 0) and keys (part 1); strides in elements.
struct HeadNormArgs {
    struct Part {
        const void* x;
        void* out;
        const void* weight;
        int64_t xt, xh, ot, oh;
    } part[2];
    RopeArgs rope;  // rot == 0: no rotation
    int64_t T;
    int q_heads, kv_heads, dim;
    float eps;
};

cudaError_t launch_head_norm(const HeadNormArgs& a, cudaStream_t stream);

struct PromptArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;  // nullable
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
    const int32_t* q_offsets;
    const int32_t* k_offsets;
    int64_t T, keys;
    int batch, q_heads, kv_heads, dim;
    int causal;
    float scale;
    void* workspace;
    unsigned int* status;
    unsigned long long wait_ns;
    bool withhold;  // test hook
};

size_t prompt_attention_workspace_bytes(int batch, int64_t T, int64_t keys, int q_heads, int kv_heads, int dim);
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream);

struct GemvArgs {
    const void* x;
    const uint8_t* w;
    const uint8_t* sw;
    const void* bias;  // nullable
    void* out;
    int M;
    int64_t N, K;
    bool nv;  // NVFP4 (E4M3 scales per 16) instead of MXFP4
    float w_global;
    const int32_t* expert_ids;  // nullable: one weight for all rows
    int E, rows_per_x;
    unsigned int* status;
    unsigned long long wait_ns;
    bool withhold;  // test hook
};

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t stream);

cudaError_t launch_moe_dispatch(const void* x, const int32_t* ids, int64_t tokens, int top_k, int E, int64_t width, int64_t xt,
                                void* sorted, int32_t* row_offsets, int32_t* row_of, cudaStream_t stream);
cudaError_t launch_moe_combine(const void* y, const int32_t* row_of, const float* weights, int64_t tokens, int top_k,
                               int64_t rows, int64_t width, void* out, int64_t ot, cudaStream_t stream);
cudaError_t launch_moe_combine_backward(const void* grad, const void* y, const int32_t* row_of, const float* weights,
                                        int64_t tokens, int top_k, int64_t rows, int64_t width, int64_t gt, void* grad_y,
                                        float* grad_weights, cudaStream_t stream);

}  // namespace fp4lin
