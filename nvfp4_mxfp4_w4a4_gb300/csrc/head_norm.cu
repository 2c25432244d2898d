// head_norm.cu -- norms of the queries' and keys' heads, with the rotation of
// their pairs in the same pass.
//
//   y = x / sqrt(sum(x^2) / dim + eps) * weight, pairs of y turned, one rounding
//
// A unit is 16 elements of a head, the two vectors whose elements pair up (or 16
// elements past the rotated part): a head's units lie in neighbouring lanes, and
// the sum over the head is a butterfly of shuffles.  A thread has the same unit of
// several heads of one token, so that the cosines and sines, as many bytes as the
// unit, are loaded once for all of them.  Every element is read and written once;
// bound by HBM, and not far from the instructions (65 % of the issue slots): 16381
// tokens x 64 heads of 128 in 94.9 us, 0.84 of a plain copy's rate.
#include <cuda_bf16.h>

#include <algorithm>

#include "decoder_ops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kThreads = 128;  // 256: 117 us, 512: 164 us, for those heads
constexpr int kHeads = 2;      // of a thread, on their way at once (1: 101 us, 4: 103 us)

struct HeadNormParams {
    HeadNormArgs a;
    int token_log;  // threads of a token: a power of two, whole heads
};

template <int kDim>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const HeadNormParams p)
{
    constexpr int LANES = kDim / 16;  // units of a head
    const HeadNormArgs& a = p.a;
    const int rot = a.rope.rot, heads = a.q_heads + a.kv_heads;
    const bool halves = a.rope.layout == kRopeHalf;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads >> p.token_log) + (threadIdx.x >> p.token_log);
    const int in_token = threadIdx.x & ((1 << p.token_log) - 1);
    const int u = in_token % LANES, step = (1 << p.token_log) / LANES;  // heads between a thread's
    const bool turned = u * 16 < rot;
    // first elements of the unit's two vectors
    const int p0 = turned && halves ? u * 8 : u * 16, p1 = turned && halves ? u * 8 + rot / 2 : u * 16 + 8;
    grid_dependency_wait();
    launch_dependents();
    const bool live = t < a.T;
    float c[8], s[8];
    if (live && turned) {
        const float* row = table_row(a.rope, t) + u * 8;
        load8f(row, c);
        load8f(row + rot / 2, s);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = a.rope.inverse ? -s[j] : s[j];
    }
    for (int h0 = 0; h0 < heads; h0 += kHeads * step) {
        uint4 v0[kHeads], v1[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * step + in_token / LANES;
            v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
            if (live && h < heads) {  // (a head's lanes together)
                const bool key = h >= a.q_heads;
                const HeadNormArgs::Part& part = a.part[key];
                const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(part.x) + t * part.xt + (key ? h - a.q_heads : h) * part.xh;
                v0[k] = *reinterpret_cast<const uint4*>(x + p0);
                v1[k] = *reinterpret_cast<const uint4*>(x + p1);
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * step + in_token / LANES;
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
            if (!live || h >= heads)
                continue;
            const bool key = h >= a.q_heads;
            const HeadNormArgs::Part& part = a.part[key];
            const float r = 1.0f / sqrtf(sum * (1.0f / kDim) + a.eps);
            float w0[8], w1[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(part.weight) + p0)), w0);
            unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(part.weight) + p1)), w1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f0[j] *= r * w0[j];
                f1[j] *= r * w1[j];
            }
            if (turned) {
                float r0[8], r1[8];
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
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(part.out) + t * part.ot + (key ? h - a.q_heads : h) * part.oh;
            *reinterpret_cast<uint4*>(dst + p0) = v0[k];
            *reinterpret_cast<uint4*>(dst + p1) = v1[k];
        }
    }
}

}  // namespace

cudaError_t launch_head_norm(const HeadNormArgs& a, cudaStream_t stream)
{
    HeadNormParams p;
    p.a = a;
    // as many threads as a token has units, up to a block's
    p.token_log = 2;  // (a head of 64)
    while ((1 << p.token_log) < kThreads && (1 << p.token_log) < (a.q_heads + a.kv_heads) * (a.dim / 16))
        ++p.token_log;
    while ((1 << p.token_log) < a.dim / 16)
        ++p.token_log;
    const int64_t tokens = kThreads >> p.token_log;
    auto kern = a.dim == 64 ? head_norm_kernel<64> : a.dim == 128 ? head_norm_kernel<128> : head_norm_kernel<256>;
    return launch_pdl(kern, dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens)), dim3(kThreads), 0, stream, p);
}

}  // namespace fp4lin
