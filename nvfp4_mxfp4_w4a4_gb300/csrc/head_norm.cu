// head_norm.cu -- norms of the queries' and keys' heads, with the rotation of
// their pairs in the same pass.
//
//   y = x / sqrt(sum(x^2) / dim + eps) * weight, pairs of y turned, one rounding
//
// A unit is 16 elements of a head, the two vectors whose elements pair up (or 16
// elements past the rotated part): a head's units lie in neighbouring lanes, and
// the sum over the head is a butterfly of shuffles.  Every element is read and
// written once; bound by HBM.
#include <cuda_bf16.h>

#include <algorithm>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kThreads = 128;
constexpr int kUnits = 2;  // of a thread, a block's threads apart

struct HeadNormParams {
    HeadNormArgs a;
    uint32_t units;  // T * (q_heads + kv_heads) * dim / 16
    DivMagic per_token;
    int token_units;
};

template <int kDim>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const HeadNormParams p)
{
    grid_dependency_wait();
    launch_dependents();
    constexpr int LANES = kDim / 16;  // units of a head
    const int rot = p.a.rope.rot;
    const bool halves = p.a.rope.layout == kRopeHalf;
    uint4 v0[kUnits], v1[kUnits];
    const float* row[kUnits];
    const __nv_bfloat16* weight[kUnits];
    __nv_bfloat16* dst[kUnits];
    int p0[kUnits], p1[kUnits];  // first elements of the unit's two vectors
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const uint32_t i = (blockIdx.x * kUnits + k) * kThreads + threadIdx.x;
        dst[k] = nullptr;
        row[k] = nullptr;
        v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
        if (i >= p.units)  // (a head's lanes together)
            continue;
        const uint32_t t = div_by_magic(i, p.per_token);
        const int in_token = static_cast<int>(i - t * p.token_units);
        int h = in_token / LANES;
        const int u = in_token % LANES;
        const HeadNormArgs::Part& part = p.a.part[h >= p.a.q_heads];
        h -= h >= p.a.q_heads ? p.a.q_heads : 0;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(part.x) + t * part.xt + h * part.xh;
        dst[k] = static_cast<__nv_bfloat16*>(part.out) + t * part.ot + h * part.oh;
        weight[k] = static_cast<const __nv_bfloat16*>(part.weight);
        p0[k] = u * 16, p1[k] = u * 16 + 8;
        if (u * 16 < rot) {
            row[k] = table_row(p.a.rope, t) + u * 8;
            if (halves)
                p0[k] = u * 8, p1[k] = u * 8 + rot / 2;
        }
        v0[k] = *reinterpret_cast<const uint4*>(x + p0[k]);
        v1[k] = *reinterpret_cast<const uint4*>(x + p1[k]);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        float f0[8], f1[8];
        unpack8(v0[k], f0);
        unpack8(v1[k], f1);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum += f0[j] * f0[j] + f1[j] * f1[j];
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (dst[k] == nullptr)
            continue;
        const float r = 1.0f / sqrtf(sum * (1.0f / kDim) + p.a.eps);
        float w0[8], w1[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight[k] + p0[k])), w0);
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight[k] + p1[k])), w1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f0[j] *= r * w0[j];
            f1[j] *= r * w1[j];
        }
        if (row[k] != nullptr) {
            float c[8], s[8], r0[8], r1[8];
            load8f(row[k], c);
            load8f(row[k] + rot / 2, s);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = p.a.rope.inverse ? -s[j] : s[j];
            if (halves) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    r0[j] = rot_first(f0[j], f1[j], c[j], s[j]);
                    r1[j] = rot_second(f0[j], f1[j], c[j], s[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r0[2 * j] = rot_first(f0[2 * j], f0[2 * j + 1], c[j], s[j]);
                    r0[2 * j + 1] = rot_second(f0[2 * j], f0[2 * j + 1], c[j], s[j]);
                    r1[2 * j] = rot_first(f1[2 * j], f1[2 * j + 1], c[j + 4], s[j + 4]);
                    r1[2 * j + 1] = rot_second(f1[2 * j], f1[2 * j + 1], c[j + 4], s[j + 4]);
                }
            }
            v0[k] = pack8(r0);
            v1[k] = pack8(r1);
        } else {
            v0[k] = pack8(f0);
            v1[k] = pack8(f1);
        }
        *reinterpret_cast<uint4*>(dst[k] + p0[k]) = v0[k];
        *reinterpret_cast<uint4*>(dst[k] + p1[k]) = v1[k];
    }
}

}  // namespace

cudaError_t launch_head_norm(const HeadNormArgs& a, cudaStream_t stream)
{
    HeadNormParams p;
    p.a = a;
    p.token_units = (a.q_heads + a.kv_heads) * (a.dim / 16);
    p.units = static_cast<uint32_t>(a.T * p.token_units);
    p.per_token = div_magic(p.token_units);
    const int64_t per_block = kUnits * kThreads;
    const dim3 grid(static_cast<unsigned>((p.units + per_block - 1) / per_block));
    auto kern = a.dim == 64 ? head_norm_kernel<64> : a.dim == 128 ? head_norm_kernel<128> : head_norm_kernel<256>;
    return launch_pdl(kern, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace fp4lin
