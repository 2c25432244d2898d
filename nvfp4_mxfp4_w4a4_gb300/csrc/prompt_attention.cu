// prompt_attention.cu -- softmax attention over whole prompts: packed sequences of
// different lengths, grouped heads, causal or not, all in bf16.
//
// A warp per query and head: 32 keys at a time, a lane each, with the running
// maximum and sum of the row; the values are then added with a lane's own
// elements of the head.
#include <cuda_bf16.h>

#include <algorithm>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kWarps = 4;

template <int kDim>
__global__ void __launch_bounds__(kWarps * 32) prompt_attention_kernel(const PromptArgs a)
{
    __shared__ float qs[kWarps][kDim];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (row >= a.T * a.q_heads)
        return;
    const int tok = static_cast<int>(row / a.q_heads), hq = static_cast<int>(row - static_cast<int64_t>(tok) * a.q_heads);
    int lo = 0, hi = a.batch;  // the first sequence that ends behind the token
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (__ldg(a.q_offsets + mid + 1) > tok)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo == a.batch)
        return;
    int q0, n, k0, m;
    group_rows(a.q_offsets, lo, static_cast<int>(a.T), &q0, &n);
    group_rows(a.k_offsets, lo, static_cast<int>(a.keys), &k0, &m);
    if (tok < q0 || tok >= q0 + n)
        return;
    const int head = hq / (a.q_heads / a.kv_heads);
    const int seen = a.causal ? max(min(tok - q0 + m - n + 1, m), 0) : m;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + tok * a.qt + hq * a.qh;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + k0 * a.kt + head * a.kh;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + k0 * a.vt + head * a.vh;
    for (int i = lane; i < kDim; i += 32)
        qs[warp][i] = __bfloat162float(q[i]);
    __syncwarp();
    float mx = -INFINITY, sum = 0.0f, o[kDim / 32] = {};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < seen) {
            s = 0.0f;
            for (int d = 0; d < kDim; d += 8) {
                float f[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(k + j * a.kt + d)), f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s += f[i] * qs[warp][d + i];
            }
            s *= a.scale;
        }
        float top = s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float next = fmaxf(mx, top);
        const float z = next == -INFINITY ? 0.0f : next;
        const float p = j < seen ? __expf(s - z) : 0.0f;
        const float keep = __expf(mx - z);
        float add = p;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
        mx = next;
        sum = sum * keep + add;
#pragma unroll
        for (int i = 0; i < kDim / 32; ++i)
            o[i] *= keep;
        for (int jj = 0; jj < min(32, seen - j0); ++jj) {
            const float pj = __shfl_sync(0xFFFFFFFFu, p, jj);
#pragma unroll
            for (int i = 0; i < kDim / 32; ++i)
                o[i] += pj * __bfloat162float(v[(j0 + jj) * a.vt + i * 32 + lane]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + tok * a.ot + hq * a.oh;
#pragma unroll
    for (int i = 0; i < kDim / 32; ++i)
        out[i * 32 + lane] = __float2bfloat16(o[i] * inv);
    if (a.lse != nullptr && lane == 0)
        a.lse[row] = sum == 0.0f ? -INFINITY : mx + logf(sum);
}

}  // namespace

size_t prompt_attention_workspace_bytes(int, int64_t, int64_t, int, int, int) { return 0; }

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream)
{
    const int64_t blocks = (a.T * a.q_heads + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    return launch_pdl(a.dim == 128 ? prompt_attention_kernel<128> : prompt_attention_kernel<64>,
                      dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace fp4lin
