// kv_cache.cu -- rotary positions and the MX-quantized paged key/value cache:
// the memory-bound operators between the q/k/v projections and attention.
//
//   rope       (a, b) -> (a cos - b sin, b cos + a sin) on pairs (i, i + rot/2)
//              or (2i, 2i + 1) of the first `rot` elements of every head
//   append     keys (optionally rotated first) and values -> MX codes + E8M0
//              scales in the pages' slots
//   read       the tokens of each sequence back to bf16, packed
//
// The block rule is the library's OCP rule on 32 elements of a head: shared
// exponent e = floor(log2 amax) - 8 (E4M3) or - 2 (E2M1), clamped to
// [-127, 127], elements rounded to nearest even, saturating; a block with a
// NaN or Inf gets scale 0xFF and zero codes.  Rotation and quantization are
// float32 with one IEEE operation at a time (no fused multiply-add), so that
// the stored codes do not depend on how the compiler contracts them.
#include <cuda_bf16.h>

#include <algorithm>

#include "formats.cuh"
#include "internal.h"
#include "kv_cache.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kThreads = 128;

// ------------------------------------------------------------------- table

// One thread per (position, frequency): the angle and its cosine and sine in
// 64 bits, rounded once (run once per model, so the rate does not matter).
__global__ void __launch_bounds__(kThreads) rope_table_kernel(float* __restrict__ table, int64_t positions, int half,
                                                              RopeFrequencies f)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= positions * half)
        return;
    const int64_t p = i / half;
    const int j = static_cast<int>(i - p * half);
    const double extrapolated = pow(f.base, -static_cast<double>(j) / half);
    double w = extrapolated;
    if (f.scaling == kRopeLinear) {
        w = extrapolated / f.factor;
    } else if (f.scaling == kRopeByParts) {
        // frequencies that turn often within the original context stay, slow
        // ones are interpolated, with a linear ramp between (a step behind `high` if it is empty)
        const double t = f.high > f.low ? (j - f.low) / (f.high - f.low) : (j > f.high ? 1.0 : 0.0);
        const double ramp = fmin(fmax(t, 0.0), 1.0);
        w = extrapolated * (1.0 - ramp) + extrapolated / f.factor * ramp;
    }
    double s, c;
    sincos(static_cast<double>(p) * w, &s, &c);
    table[p * 2 * half + j] = static_cast<float>(c * f.magnitude);
    table[p * 2 * half + half + j] = static_cast<float>(s * f.magnitude);
}

// -------------------------------------------------------------------- rope

// A unit is 16 elements of a head: 8 rotated pairs, or 16 elements past `rot`
// that are copied.  A thread takes kRopeUnits of them, a block's threads apart,
// and starts all their loads first.  Index arithmetic is 32-bit with
// multiplications for the divisions (with 64-bit divisions the kernel ran at
// 0.81 of the copy rate, 16381 tokens x 56 heads of 128).
constexpr int kRopeUnits = 2;

struct RopeKernelArgs {
    const __nv_bfloat16* x;
    __nv_bfloat16* out;
    RopeArgs rope;
    uint32_t units;  // T * heads * dim / 16
    DivMagic per_token, per_head;  // by the units of a token, of a head
    int token_units, head_units;
    int64_t xt, xh, ot, oh;  // token and head strides in elements
};

__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeKernelArgs a)
{
    grid_dependency_wait();
    launch_dependents();
    const int rot = a.rope.rot;
    const bool halves = a.rope.layout == kRopeHalf;
    uint4 v0[kRopeUnits], v1[kRopeUnits];
    const float* row[kRopeUnits];
    __nv_bfloat16* dst[kRopeUnits];
    int p0[kRopeUnits], p1[kRopeUnits];  // first elements of the unit's two vectors
#pragma unroll
    for (int k = 0; k < kRopeUnits; ++k) {
        const uint32_t i = (blockIdx.x * kRopeUnits + k) * kThreads + threadIdx.x;
        dst[k] = nullptr;
        if (i >= a.units)
            continue;
        const uint32_t t = div_by_magic(i, a.per_token);
        const uint32_t in_token = i - t * a.token_units;
        const uint32_t h = div_by_magic(in_token, a.per_head);
        const int u = static_cast<int>(in_token - h * a.head_units);
        const __nv_bfloat16* x = a.x + t * a.xt + h * a.xh;
        dst[k] = a.out + t * a.ot + h * a.oh;
        p0[k] = u * 16, p1[k] = u * 16 + 8;
        row[k] = nullptr;
        if (u * 16 < rot) {
            row[k] = table_row(a.rope, t) + u * 8;
            if (halves)
                p0[k] = u * 8, p1[k] = u * 8 + rot / 2;
        }
        v0[k] = *reinterpret_cast<const uint4*>(x + p0[k]);
        v1[k] = *reinterpret_cast<const uint4*>(x + p1[k]);
    }
#pragma unroll
    for (int k = 0; k < kRopeUnits; ++k) {
        if (dst[k] == nullptr)
            continue;
        if (row[k] != nullptr) {
            float c[8], s[8], f0[8], f1[8], r0[8], r1[8];
            load8f(row[k], c);
            load8f(row[k] + rot / 2, s);
            unpack8(v0[k], f0);
            unpack8(v1[k], f1);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = a.rope.inverse ? -s[j] : s[j];
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
        }
        *reinterpret_cast<uint4*>(dst[k] + p0[k]) = v0[k];
        *reinterpret_cast<uint4*>(dst[k] + p1[k]) = v1[k];
    }
}

// ------------------------------------------------------------------ append

struct AppendKernelArgs {
    KvCache cache;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const int64_t* slots;
    RopeArgs rope;  // rot == 0: keys are stored as they are
    uint32_t vectors;  // T * 2 * heads * dim / 8
    DivMagic per_token, page_div;  // by the vectors of a token, by the page size
    int token_vectors;
    int64_t kt, kh, vt, vh;
};

// A lane owns 8 consecutive elements, 4 lanes a block.  A thread takes
// kAppendVectors of them: a vector waits for its token's position and then for
// the table's row, and with one per thread those waits, not the bytes, set the
// time.
constexpr int kAppendVectors = 2;

template <int kFmt>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendKernelArgs a)
{
    grid_dependency_wait();
    launch_dependents();
    const int shift = a.cache.dim == 128 ? 4 : 3;  // vectors of a head
    const int half = a.rope.rot / 2;
    const bool halves = a.rope.layout == kRopeHalf;
    bool live[kAppendVectors], value[kAppendVectors], turn[kAppendVectors];
    int head[kAppendVectors], elem[kAppendVectors];
    int64_t slot[kAppendVectors];
    const float* cs[kAppendVectors];
    uint4 x[kAppendVectors], partner[kAppendVectors];
#pragma unroll
    for (int k = 0; k < kAppendVectors; ++k) {
        uint32_t i = (blockIdx.x * kAppendVectors + k) * kThreads + threadIdx.x;
        live[k] = i < a.vectors;  // whole quads: a head is a multiple of 4 vectors
        i = live[k] ? i : 0u;
        const uint32_t t = div_by_magic(i, a.per_token);
        const uint32_t in_token = i - t * a.token_vectors;
        const int hv = static_cast<int>(in_token >> shift);
        const int d = static_cast<int>(in_token - (hv << shift)) * 8;
        value[k] = hv >= a.cache.heads;
        head[k] = value[k] ? hv - a.cache.heads : hv;
        elem[k] = d;
        slot[k] = __ldg(a.slots + t);
        const __nv_bfloat16* src = value[k] ? a.v + t * a.vt + head[k] * a.vh : a.k + t * a.kt + head[k] * a.kh;
        x[k] = *reinterpret_cast<const uint4*>(src + d);
        turn[k] = !value[k] && d < a.rope.rot;
        if (turn[k]) {
            cs[k] = table_row(a.rope, t);
            if (halves)
                partner[k] = *reinterpret_cast<const uint4*>(src + (d < half ? d + half : d - half));
        }
    }
#pragma unroll
    for (int k = 0; k < kAppendVectors; ++k) {
        const int d = elem[k];
        float f[8];
        unpack8(x[k], f);
        if (turn[k]) {
            if (halves) {
                const bool first = d < half;
                const int j0 = first ? d : d - half;
                float g[8], c[8], s[8];
                unpack8(partner[k], g);
                load8f(cs[k] + j0, c);
                load8f(cs[k] + half + j0, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float sj = a.rope.inverse ? -s[j] : s[j];
                    f[j] = first ? rot_first(f[j], g[j], c[j], sj) : rot_second(g[j], f[j], c[j], sj);
                }
            } else {
                const float4 c = __ldg(reinterpret_cast<const float4*>(cs[k] + d / 2));
                const float4 s = __ldg(reinterpret_cast<const float4*>(cs[k] + half + d / 2));
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float sj = a.rope.inverse ? -ss[j] : ss[j];
                    const float p = f[2 * j], q = f[2 * j + 1];
                    f[2 * j] = rot_first(p, q, cc[j], sj);
                    f[2 * j + 1] = rot_second(p, q, cc[j], sj);
                }
            }
        }
        // |x| as bit patterns: NaN above Inf above every finite value
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            am = max(am, __float_as_uint(f[j]) & 0x7FFFFFFFu);
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        const bool finite = am < 0x7F800000u;
        // floor(log2 amax) - emax; zero and subnormal maxima fall to the clamp
        const int e = max(-127, static_cast<int>(am >> 23) - 127 - (kFmt == kKvMxfp8 ? 8 : 2));
        const float inv = exp2_neg(e);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = finite ? __fmul_rn(f[j], inv) : 0.0f;
        if (!live[k] || slot[k] < 0 || slot[k] >= a.cache.pages * a.cache.page_size)
            continue;
        const int64_t page =
            slot[k] >> 32 ? slot[k] / a.cache.page_size : div_by_magic(static_cast<uint32_t>(slot[k]), a.page_div);
        const int64_t at = (page * a.cache.heads + head[k]) * a.cache.page_size + (slot[k] - page * a.cache.page_size);
        uint8_t* codes = value[k] ? a.cache.v_codes : a.cache.k_codes;
        uint8_t* scales = value[k] ? a.cache.v_scales : a.cache.k_scales;
        if constexpr (kFmt == kKvMxfp8) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t lo =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j], f[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi =
                    __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j + 2], f[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
                w[j] = lo | (hi << 16);
            }
            *reinterpret_cast<uint2*>(codes + at * a.cache.dim + d) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint32_t*>(codes + (at * a.cache.dim + d) / 2) =
                e2m1x8_pack(f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]);
        }
        if ((d & 31) == 0)
            scales[at * (a.cache.dim >> 5) + (d >> 5)] = static_cast<uint8_t>(finite ? e + 127 : 0xFF);
    }
}

// -------------------------------------------------------------------- read

struct ReadKernelArgs {
    KvCache cache;
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* cu_lens;
    int batch;
    int64_t rows;
    int block_rows;   // tokens per block
    int row_items;    // 2 * heads * dim / 8
    DivMagic per_row;
    __nv_bfloat16* k;
    __nv_bfloat16* v;
};

constexpr int kReadRows = 32;   // tokens per block at most
constexpr int kReadItems = 8;   // of 8 elements, per thread

// Eight codes as float32 values.
template <int kFmt>
__device__ __forceinline__ void decode8(uint2 w, float* f)
{
    uint32_t h[4];  // f16 pairs
    if constexpr (kFmt == kKvMxfp8) {
        const float2 a = e4m3x2_to_float2(w.x), b = e4m3x2_to_float2(w.x >> 16), c = e4m3x2_to_float2(w.y),
                     d = e4m3x2_to_float2(w.y >> 16);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
    } else {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w.x));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        }
    }
}

// Each token's place in the cache is found once per block; then a thread turns
// 8 codes at a time into one 16-byte vector (consecutive threads write
// consecutive vectors), all its loads started first.
template <int kFmt>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadKernelArgs a)
{
    __shared__ int64_t place[kReadRows];  // (page * heads) * page_size + slot, or -1
    grid_dependency_wait();
    launch_dependents();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.block_rows;
    if (threadIdx.x < 32) {
        // the last sequence that starts at or before the block's first row, 32 probes
        // at a time (the look-up's latency is the block's start-up)
        const int lane = threadIdx.x;
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5;
            const int at = lo + lane * step;
            const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && (at == lo || __ldg(a.cu_lens + at) <= row0));
            lo += (31 - __clz(below)) * step;
            hi = min(hi, lo + step);
        }
        const int64_t r = row0 + lane;
        int64_t p = -1;
        if (lane < a.block_rows && r < a.rows) {
            while (lo + 1 < a.batch && __ldg(a.cu_lens + lo + 1) <= r)
                ++lo;
            const int64_t pos = r - __ldg(a.cu_lens + lo);
            const int64_t pi = pos / a.cache.page_size;
            if (pos >= 0 && r < __ldg(a.cu_lens + lo + 1) && pi < a.table_stride) {
                const int64_t page = __ldg(a.block_table + lo * a.table_stride + pi);
                if (page >= 0 && page < a.cache.pages)
                    p = page * a.cache.heads * a.cache.page_size + (pos - pi * a.cache.page_size);
            }
        }
        place[lane] = p;
    }
    __syncthreads();
    const int shift = a.cache.dim == 128 ? 4 : 3;  // vectors of a head
    const int items = a.block_rows * a.row_items;
    for (int i0 = threadIdx.x; i0 < items; i0 += kReadItems * kThreads) {
        uint2 w[kReadItems];
        uint32_t sb[kReadItems];
        __nv_bfloat16* out[kReadItems];
#pragma unroll
        for (int k = 0; k < kReadItems; ++k) {
            const int i = i0 + k * kThreads;
            out[k] = nullptr;
            if (i >= items)
                continue;
            const int r = static_cast<int>(div_by_magic(i, a.per_row));
            const int64_t p = place[r];
            if (p < 0)
                continue;
            const int in_row = i - r * a.row_items;
            const int hv = in_row >> shift;
            const int d = (in_row - (hv << shift)) * 8;
            const bool value = hv >= a.cache.heads;
            const int h = value ? hv - a.cache.heads : hv;
            const int64_t at = p + static_cast<int64_t>(h) * a.cache.page_size;
            const uint8_t* codes = value ? a.cache.v_codes : a.cache.k_codes;
            const uint8_t* scales = value ? a.cache.v_scales : a.cache.k_scales;
            if constexpr (kFmt == kKvMxfp8)
                w[k] = __ldg(reinterpret_cast<const uint2*>(codes + at * a.cache.dim + d));
            else
                w[k].x = __ldg(reinterpret_cast<const uint32_t*>(codes + (at * a.cache.dim + d) / 2));
            sb[k] = __ldg(scales + at * (a.cache.dim >> 5) + (d >> 5));
            out[k] = (value ? a.v : a.k) + ((row0 + r) * a.cache.heads + h) * a.cache.dim + d;
        }
#pragma unroll
        for (int k = 0; k < kReadItems; ++k) {
            if (out[k] == nullptr)
                continue;
            // 2^(s - 127): s = 0 is the subnormal 2^-127, 0xFF NaN
            const float sc = __uint_as_float(sb[k] == 0xFFu ? 0x7FC00000u : sb[k] == 0 ? 0x00400000u : sb[k] << 23);
            float f[8];
            decode8<kFmt>(w[k], f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] *= sc;
            *reinterpret_cast<uint4*>(out[k]) = pack8(f);
        }
    }
}

inline int blocks_for(int64_t threads) { return static_cast<int>((threads + kThreads - 1) / kThreads); }

}  // namespace

cudaError_t launch_rope_table(float* table, int64_t positions, int rot, const RopeFrequencies& f, cudaStream_t stream)
{
    return launch_pdl(rope_table_kernel, dim3(blocks_for(positions * (rot / 2))), dim3(kThreads), 0, stream, table,
                      positions, rot / 2, f);
}

cudaError_t launch_rope(const void* x, void* out, const RopeArgs& rope, int64_t T, int heads, int dim, int64_t xt,
                        int64_t xh, int64_t ot, int64_t oh, cudaStream_t stream)
{
    RopeKernelArgs a;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.rope = rope;
    a.head_units = dim / 16;
    a.token_units = heads * a.head_units;
    a.units = static_cast<uint32_t>(T * a.token_units);
    a.per_token = div_magic(a.token_units);
    a.per_head = div_magic(a.head_units);
    a.xt = xt, a.xh = xh, a.ot = ot, a.oh = oh;
    return launch_pdl(rope_kernel, dim3(blocks_for((static_cast<int64_t>(a.units) + kRopeUnits - 1) / kRopeUnits)),
                      dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kv_append(const KvCache& cache, const void* k, const void* v, int64_t T, int64_t kt, int64_t kh,
                             int64_t vt, int64_t vh, const int64_t* slots, const RopeArgs& rope, cudaStream_t stream)
{
    AppendKernelArgs a;
    a.cache = cache;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.slots = slots;
    a.rope = rope;
    a.token_vectors = 2 * cache.heads * (cache.dim / 8);
    a.vectors = static_cast<uint32_t>(T * a.token_vectors);
    a.per_token = div_magic(a.token_vectors);
    a.page_div = div_magic(cache.page_size);
    a.kt = kt, a.kh = kh, a.vt = vt, a.vh = vh;
    return launch_pdl(cache.format == kKvMxfp8 ? kv_append_kernel<kKvMxfp8> : kv_append_kernel<kKvMxfp4>,
                      dim3(blocks_for((static_cast<int64_t>(a.vectors) + kAppendVectors - 1) / kAppendVectors)), dim3(kThreads), 0,
                      stream, a);
}

cudaError_t launch_kv_read(const KvCache& cache, const int32_t* block_table, int64_t table_stride,
                           const int32_t* cu_lens, int batch, int64_t rows, void* k, void* v, cudaStream_t stream)
{
    ReadKernelArgs a;
    a.cache = cache;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.cu_lens = cu_lens;
    a.batch = batch;
    a.rows = rows;
    a.k = static_cast<__nv_bfloat16*>(k);
    a.v = static_cast<__nv_bfloat16*>(v);
    a.row_items = 2 * cache.heads * (cache.dim / 8);
    a.per_row = div_magic(a.row_items);
    // one round of the block's loop (more rounds per look-up measured slower, in
    // blocks of 256 threads: 28.9 us with 8 rows of 8 heads a block, 34.1 with 44)
    a.block_rows = std::max(1, std::min(kReadRows, kReadItems * kThreads / a.row_items));
    return launch_pdl(cache.format == kKvMxfp8 ? kv_read_kernel<kKvMxfp8> : kv_read_kernel<kKvMxfp4>,
                      dim3(static_cast<unsigned>((rows + a.block_rows - 1) / a.block_rows)), dim3(kThreads), 0, stream,
                      a);
}

}  // namespace fp4lin
