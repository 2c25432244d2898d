// gemm_fp8.h -- launchers of the FP8 linear layer with a scale per block of
// 128.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp4lin {

struct Fp8GemmArgs {
    const uint8_t* a;  // [M, K] E4M3
    const float* sa;   // [ceil(K / 128)][M rounded up to 4]
    const uint8_t* b;  // [N, K] E4M3
    const float* sb;   // [ceil(N / 128)][ceil(K / 128)]
    const void* bias;  // bf16 [N] or null
    void* out;         // bf16 [M, N]
    int64_t M, N, K;
    unsigned int* status;
    unsigned long long wait_ns;
    bool early_weights;  // the kernel ahead in the stream is this call's own quantizer
};

cudaError_t launch_quant_act_fp8(const void* x, uint8_t* codes, float* scales, int64_t M, int64_t K,
                                 cudaStream_t stream);
cudaError_t launch_quant_weight_fp8(const void* w, uint8_t* codes, float* scales, int64_t N, int64_t K,
                                    cudaStream_t stream);
cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, cudaStream_t stream);

}  // namespace fp4lin
