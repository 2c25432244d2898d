// rope.cuh -- bf16 vectors of 8 and the rotation of a pair, shared by the kernels
// that rotate heads.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "kv_cache.h"

namespace fp4lin {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(uint4 v, float* f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf_lo(w[i]);
        f[2 * i + 1] = bf_hi(w[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ void load8f(const float* p, float* f)
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + 4));
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Row of the cos/sin table of a token; positions outside the table read its
// nearest row, so no access leaves it.
__device__ __forceinline__ const float* table_row(const RopeArgs& r, int64_t token)
{
    int64_t p = __ldg(r.positions + token);
    p = min(max(p, int64_t(0)), r.table_positions - 1);
    return r.table + p * r.rot;
}

// The first element of the rotation a' = a cos - b sin and the second b' =
// b cos + a sin; the inverse turns by the negative angle.
__device__ __forceinline__ float rot_first(float a, float b, float c, float s)
{
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}

__device__ __forceinline__ float rot_second(float a, float b, float c, float s)
{
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

}  // namespace fp4lin
