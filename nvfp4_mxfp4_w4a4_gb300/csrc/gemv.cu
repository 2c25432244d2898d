// gemv.cu -- products of a few rows of bf16 activations with 4-bit weights and
// group scales (MXFP4: E8M0 per 32, NVFP4: E4M3 per 16), the activations as they
// are: out[m, n] = bf16(sum_k x[m, k] W[n, k] + bias[n]).
//
// Bound by HBM: a weight is 0.53 (0.56) bytes and 2 M operations.  A warp per
// output: a lane takes 32 consecutive elements of every 1024.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kThreads = 256;

struct GemvParams {
    GemvArgs a;
    int64_t expert_codes, expert_scales;  // bytes of an expert
    int kb4;                              // groups of 4 scales of a row
};

__device__ __forceinline__ void e2m1x8(uint32_t w, float* f)
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
}

__device__ __forceinline__ float scale_value(uint32_t byte, bool nv)
{
    if (nv) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
        return __half2float(__half(h));
    }
    // 2^(s - 127): s = 0 is the subnormal 2^-127, 0xFF NaN
    return __uint_as_float(byte == 0xFFu ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

template <int kM>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const GemvArgs& a = p.a;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (n >= a.N)
        return;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    const uint8_t* w = a.w;
    const uint8_t* sw = a.sw;
    const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(a.bias);
    if (a.expert_ids != nullptr) {
        const int r = blockIdx.y, e = __ldg(a.expert_ids + r);
        out += r * a.N;
        if (e < 0 || e >= a.E) {
            if (lane == 0)
                out[n] = __float2bfloat16(0.0f);
            return;
        }
        x += static_cast<int64_t>(r / a.rows_per_x) * a.K;
        w += e * p.expert_codes;
        sw += e * p.expert_scales;
        bias = bias != nullptr ? bias + e * a.N : nullptr;
    }
    float sum[kM] = {};
    for (int64_t k = lane * 32; k < a.K; k += 1024) {
        const uint4 c = __ldg(reinterpret_cast<const uint4*>(w + (n * a.K + k) / 2));
        const uint32_t words[4] = {c.x, c.y, c.z, c.w};
        float part[kM][2] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[8];
            e2m1x8(words[q], f);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                float v[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(x + m * a.K + k + 8 * q)), v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    part[m][q >> 1] += f[i] * v[i];
            }
        }
        float s[2];
        if (a.nv) {
            s[0] = scale_value(__ldg(sw + sf_swizzled_offset(n, k / 16, p.kb4)), true);
            s[1] = scale_value(__ldg(sw + sf_swizzled_offset(n, k / 16 + 1, p.kb4)), true);
        } else {
            s[0] = s[1] = scale_value(__ldg(sw + sf_swizzled_offset(n, k / 32, p.kb4)), false);
        }
#pragma unroll
        for (int m = 0; m < kM; ++m)
            sum[m] += part[m][0] * s[0] + part[m][1] * s[1];
    }
    const float b = bias != nullptr ? __bfloat162float(bias[n]) : 0.0f;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum[m] += __shfl_xor_sync(0xFFFFFFFFu, sum[m], d);
        if (lane == 0)
            out[m * a.N + n] = __float2bfloat16(sum[m] * a.w_global + b);
    }
}

using Kernel = void (*)(GemvParams);

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t stream)
{
    static const Kernel kernels[8] = {gemv_kernel<1>, gemv_kernel<2>, gemv_kernel<3>, gemv_kernel<4>,
                                      gemv_kernel<5>, gemv_kernel<6>, gemv_kernel<7>, gemv_kernel<8>};
    GemvParams p;
    p.a = a;
    const int64_t blocks = a.K / (a.nv ? 16 : 32);
    p.kb4 = static_cast<int>((blocks + 3) / 4);
    p.expert_codes = a.N * a.K / 2;
    p.expert_scales = (a.N + 127) / 128 * 512 * p.kb4;
    const unsigned grid = static_cast<unsigned>((a.N + kThreads / 32 - 1) / (kThreads / 32));
    const bool experts = a.expert_ids != nullptr;
    return launch_pdl(kernels[experts ? 0 : a.M - 1], dim3(grid, experts ? a.M : 1), dim3(kThreads), 0, stream, p);
}

}  // namespace fp4lin
