// gemv.cu -- products of a few rows of bf16 activations with 4-bit weights and
// group scales (MXFP4: E8M0 per 32, NVFP4: E4M3 per 16), the activations as they
// are: out[m, n] = bf16(sum_k x[m, k] W[n, k] + bias[n]).
//
// Its floor is HBM: a weight is 0.53 (0.56) bytes and 2 M operations.  So two warps
// do nothing but bring in the weights (TMA) into a ring in shared memory that holds
// as much as there is room for, while 16 warps multiply what has landed.  (Weights
// straight to registers took 11 to 14 us for 14336 x 4096.)  A CTA takes sets of 32
// rows, an equal run of them, whole rows each; a stage of the ring is 1024 elements
// of the set's rows, 128 (a chunk) for each of 8 warps, the other 8 have the next
// stage.  The warps' sums of a set are added up by one more warp, in one order.
//
// On the device, weights in L2 (and from memory, other weights each call): MXFP4, 1
// token, 4096 x 4096 4.6 us (5.8); NVFP4, 3 tokens, 14336 x 4096 10.4 (12.1); MXFP4, 8
// tokens, 18429 x 7168 20.2 (22.6); 8 experts of 2048 x 4096 10.9 (12.4).  The loads
// alone take 3.1 / 5.0 / 9.1 / 6.1 us, all but the decoding and the MMAs 3.2 / 5.6 /
// 12.6 / 6.2, so the decoding is what a call takes longer for: 190 to 250 instructions
// per 32 rows x 128 elements, 64 of them conversions of two codes that take the ALU two
// cycles each.  But they do not fill any pipe (issue slots 41 to 59 % busy, the ALU 35
// to 49 %, the tensor pipe 14 to 18 %): the rest is what does not overlap with them,
// the launch, the activations' way into shared memory before the first product (3 us
// at 8 tokens of 7168), the first stages, and four multiplying warps a scheduler that
// wait for shared memory, for one another's stages and for the last sums.
//
// Decoding goes through one conversion per two codes (E2M1 -> f16, exact), the
// products through m16n8k16 MMAs with float32 sums.  Codes of MXFP4 never meet
// their scales one by one: an MMA's sum stays within one block of 32, and takes
// the block's scale (times that of the activations) in one multiply-add.  NVFP4's
// scales are multiplied into the f16 elements, exactly (E2M1 x E4M3 has 6 bits).
//   - 1 or 2 tokens: a lane of a quad has one block of a row, 16 bytes; the quad's
//     lanes hold different k of the MMA, so each block has its own columns: column
//     (block, token) of B holds the token's activations in the k of that block's
//     lane and zeros elsewhere.  Eight MMAs per 16 rows and chunk.
//   - up to 8 tokens: a column each; the quad's lanes have four words of one block,
//     so that the MMA's sum stays in it.  Eight MMAs too, but more loads from
//     shared memory and more multiply-adds.
// Activations go into shared memory once, as f16 times a power of two per block of
// 32 (the block's largest lies in [2^14, 2^15)): exact but for elements below
// 2^-31 of it.
//
// The swizzled scales of a chunk lie 4 bytes for a row of the set, 12 for those of
// three other sets: the ring takes them whole, 512 bytes a run (bytes that the L2
// has when the next sets want them; copies of 128 bytes for rows that are 32 apart
// measured half the rate: bulk copies cost their issue, about 140 cycles each).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "decoder_ops.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

constexpr int kChunk = 128;             // elements of K of a warp's step
constexpr int kChunks = 8;              // of a stage
constexpr int kGroups = 2;              // of warps, which take the stages in turns
constexpr int kWarps = kGroups * kChunks;  // that multiply
constexpr int kStageK = kChunks * kChunk;
constexpr int kLoaders = 2;             // that load, stages in turns too
constexpr int kThreads = (kWarps + kLoaders + 1) * 32;  // and one that adds up
constexpr int kSetRows = 32;
constexpr int kMostStages = 12;
constexpr int kMaxSmem = 227 * 1024;

struct GemvParams {
    GemvArgs a;
    int64_t expert_scales;  // bytes of an expert
    int kb4;     // groups of 4 scales of a row
    int chunks;  // of K
    int sets;    // of a weight's rows
    int stages;
    int per;     // sets of a CTA (of all rows' weights with experts)
    int64_t all;
};

// A stage: slabs of 128 bytes (two chunks) of the set's rows, 16-byte pieces turned by
// the row (the 128-byte swizzle), then the chunks' scales.
constexpr int kSlab = kSetRows * 128;
constexpr int kCodeBytes = kStageK / 256 * kSlab;

template <bool kNv>
constexpr int stage_bytes()
{
    return kCodeBytes + kChunks * (kNv ? 1024 : 512);
}

// Eight codes to f16 pairs, in order.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t* h)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// d (+)= A B; the first of a sum has no addend.
template <bool kFirst>
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (kFirst)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(b - 127) of the two bytes in the low half of w (0xFF: NaN).
__device__ __forceinline__ float2 e8m0x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h, u;\n\t"
        "mov.b32 {h, u}, %1;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(w));
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
}

// The two E4M3 scales in the low half of w as f16, exact.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h, u;\n\t"
        "mov.b32 {h, u}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// acc[i] += d[i] * (f * x[i]), both at once.
__device__ __forceinline__ void add_scaled(float* acc, const float* d, float f, float2 x)
{
    asm("{\n\t.reg .b64 a, b, c, e;\n\t"
        "mov.b64 a, {%4, %4};\n\t"
        "mov.b64 b, {%5, %6};\n\t"
        "mov.b64 c, {%2, %3};\n\t"
        "mov.b64 e, {%0, %1};\n\t"
        "mul.rn.f32x2 a, a, b;\n\t"
        "fma.rn.f32x2 e, c, a, e;\n\t"
        "mov.b64 {%0, %1}, e;\n\t}"
        : "+f"(acc[0]), "+f"(acc[1])
        : "f"(d[0]), "f"(d[1]), "f"(f), "f"(x.x), "f"(x.y));
}

// A place among a CTA's sets: the output's row (with experts) and the set of the
// weight's rows.
struct Place {
    int row, set;
    int x_row;   // first row of x
    int id;      // expert, not checked

    __device__ __forceinline__ void find(const GemvParams& p, int64_t v)
    {
        const bool experts = p.a.expert_ids != nullptr;
        row = experts ? static_cast<int>(v / p.sets) : 0;
        set = static_cast<int>(v - static_cast<int64_t>(row) * p.sets);
        id = x_row = 0;
        if (experts) {
            x_row = row / p.a.rows_per_x;
            id = __ldg(p.a.expert_ids + row);
        }
    }
    // (-1: none)
    __device__ __forceinline__ int expert(const GemvParams& p) const
    {
        return p.a.expert_ids == nullptr || (id >= 0 && id < p.a.E) ? id : -1;
    }
    __device__ __forceinline__ void next(const GemvParams& p, int64_t v)
    {
        if (++set == p.sets && v < p.all)
            find(p, v);
    }
};

// Sets whose sums have a place (8 tokens' take 16 KB).
__host__ __device__ constexpr uint32_t sum_buffers(bool wide) { return wide ? 1 : 2; }

// A place in the ring and the parity of its round.
struct Turn {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t stages)
    {
        if (++slot == stages)
            slot = 0, phase ^= 1u;
    }
};

// kWide: up to 8 tokens, else up to 2.
template <bool kWide, bool kNv>
__global__ void __launch_bounds__(kThreads, 1) gemv_kernel(const GemvParams p, const __grid_constant__ CUtensorMap w_map)
{
    constexpr int TOK = kWide ? 8 : 2;
    constexpr uint32_t SUMS = sum_buffers(kWide);
    constexpr int PAD = kWide ? 32 : 0;  // elements between tokens, so that they fall in different banks
    constexpr int BYTES = stage_bytes<kNv>(), RUN = kNv ? 1024 : 512;
    extern __shared__ uint4 smem_raw[];
    const GemvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    const int padded = p.chunks * kChunk, pitch = padded + PAD;
    const int tokens = a.expert_ids != nullptr ? 1 : a.M;
    const int N = static_cast<int>(a.N), K = static_cast<int>(a.K);
    // (by an offset, not a cast of the address: the compiler has to see shared memory)
    uint8_t* ring = reinterpret_cast<uint8_t*>(smem_raw) + ((0u - smem_u32(smem_raw)) & 1023u);
    float* red = reinterpret_cast<float*>(ring + p.stages * BYTES);        // [SUMS][kWarps][TOK][kSetRows]
    float* xscale = red + SUMS * kWarps * TOK * kSetRows;                      // [padded / 32][TOK]
    uint4* zeros = reinterpret_cast<uint4*>(xscale + TOK * (padded / 32));  // [4]
    uint64_t* full = reinterpret_cast<uint64_t*>(zeros + 4);                // [kMostStages]
    uint64_t* free_ = full + kMostStages;                                   // [kMostStages]
    uint64_t* summed = free_ + kMostStages;                                 // [2] the warps' sums of a set are there
    uint64_t* taken = summed + 2;                                           // [2]
    __half* xs = reinterpret_cast<__half*>(taken + 2);                      // [tokens][pitch]
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&free_[i], kChunks);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&summed[i], kWarps);
            mbar_init(&taken[i], 1);
        }
        fence_mbar_init();
    }
    grid_dependency_wait();
    launch_dependents();
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per;
    const int64_t end = min(first + p.per, p.all);
    const int steps = (p.chunks + kChunks - 1) / kChunks;  // stages of a set
    if (first >= end)
        return;

    if (warp == kWarps + kLoaders) {
        // ------------------------------------------------------------ results
        // the warps' sums of a set, in their order, while the next set is multiplied
        Place at;
        at.find(p, first);
        uint32_t sets = 0;
        for (int64_t v = first; v < end; at.next(p, ++v), ++sets) {
            const uint32_t place = sets % SUMS;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&summed[place], sets / SUMS & 1u, a.status, kStatusTimeout, a.wait_ns)))
                return;
            const int n = at.set * kSetRows + lane;
            float bias = 0.0f;
            if (a.bias != nullptr && at.expert(p) >= 0 && n < N)
                bias = __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[at.expert(p) * a.N + n]);
            for (int t = 0; t < tokens; ++t) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum += red[((place * kWarps + w) * TOK + t) * kSetRows + lane];
                if (n < N)
                    static_cast<__nv_bfloat16*>(a.out)[static_cast<int64_t>(at.row + t) * N + n] = __float2bfloat16(sum * a.w_global + bias);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&taken[place]);
        }
        return;
    }
    if (warp >= kWarps) {
        // ------------------------------------------------------------ weights
        {  // (the whole warp walks the loop: the copies' operands are then uniform)
            Place at;
            at.find(p, first);
            Turn turn;
            uint32_t issued = 0;  // of all stages
            const uint32_t mine = warp - kWarps;
            bool ok = true;
            for (int64_t v = first; ok && v < end; at.next(p, ++v)) {
                const int expert = at.expert(p);
                if (expert < 0)
                    continue;
                // (rows past the last are zeros, or the next expert's: they are not written)
                const int row0 = static_cast<int>(expert * a.N) + at.set * kSetRows;
                const uint8_t* scales = a.sw + expert * p.expert_scales + static_cast<int64_t>(at.set >> 2) * p.kb4 * 512;
                for (int step = 0; step < steps; ++step, turn.next(p.stages), ++issued) {
                    if ((issued & (kLoaders - 1)) != mine)
                        continue;
                    if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(&free_[turn.slot]), turn.phase ^ 1u)))
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&free_[turn.slot], turn.phase ^ 1u, a.status, kStatusTimeout, a.wait_ns));
                    if (!ok)
                        break;
                    uint8_t* to = ring + turn.slot * BYTES;
                    uint64_t* bar = &full[turn.slot];
                    const uint32_t bytes = min(kChunks * RUN, p.kb4 * 512 - step * (kChunks * RUN));
                    const int slabs = min(kStageK / 256, (K - step * kStageK + 255) / 256);
                    // (test hook: the first CTA's first stage never comes)
                    if (elect_one() && !(a.withhold && blockIdx.x == 0 && issued == 0)) {
                        mbar_arrive_expect_tx(bar, slabs * kSlab + bytes);
                        for (int i = 0; i < slabs; ++i)
                            tma_load_2d(to + i * kSlab, &w_map, bar, step * (kStageK / 2) + i * 128, row0);
                        bulk_load(to + kCodeBytes, scales + static_cast<int64_t>(step) * (kChunks * RUN), bytes, bar);
                    }
                    __syncwarp();
                }
            }
            // (every copy is waited for by the warps that multiply, unless they gave up)
            for (uint32_t i = 0; i < static_cast<uint32_t>(p.stages) && i < issued; ++i) {
                if (turn.slot == 0)
                    turn.slot = p.stages, turn.phase ^= 1u;
                --turn.slot;
                if (((issued - 1 - i) & (kLoaders - 1)) == mine)
                    mbar_wait_bounded(&full[turn.slot], turn.phase, a.status, kStatusTimeout, a.wait_ns);
            }
        }
        return;
    }

    // ------------------------------------------------------------- products
    const int chunk = warp & (kChunks - 1), group = warp / kChunks;
    if (threadIdx.x < 4)
        zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);
    Place at;
    at.find(p, first);
    int x_row = -1;
    Turn turn;
    uint32_t odd = 0, sets = 0;  // parity of the stages so far; sets so far
    bool ok = true;
    const bool own_block = (g >> 1) == j;  // (1 or 2 tokens) this lane's column has its own block's activations
    const bool reads = kWide ? g < tokens : own_block && (g & 1) < tokens;
    // Lanes without activations read zeros.
    const uint32_t b_at = reads ? static_cast<uint32_t>(reinterpret_cast<uint8_t*>(xs + (kWide ? g * pitch + 8 * j : (g & 1) * pitch + 32 * j)) - ring)
                                : static_cast<uint32_t>(reinterpret_cast<uint8_t*>(zeros) - ring);
    const uint32_t b_step = reads ? kChunk * 2 : 0, b_block = reads ? 64 : 0;
    // A warp whose wait has run out multiplies no more, but goes on to the barriers: they count
    // all 16 warps and know no limit, so that the warps give up together, at the next of them.
    for (int64_t v = first; v < end; at.next(p, ++v), ++sets) {
        if (at.x_row != x_row) {
            // activations: a lane has 8 elements of every token, four lanes a block of 32 (whole
            // warps go round: their lanes exchange)
            if (x_row >= 0 && named_barrier_or(1, kWarps * 32, !ok))
                break;
            x_row = at.x_row;
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + static_cast<int64_t>(x_row) * K;
            for (int k0 = warp * 256; k0 < padded; k0 += kWarps * 256) {
                const int k = k0 + lane * 8;
                uint4 q[TOK];
#pragma unroll
                for (int t = 0; t < TOK; ++t) {
                    q[t] = make_uint4(0, 0, 0, 0);
                    if (t < tokens && k < K)
                        q[t] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * K + k));
                }
#pragma unroll
                for (int t = 0; t < TOK; ++t) {
                    if (t >= tokens)
                        break;
                    const uint32_t w[4] = {q[t].x, q[t].y, q[t].z, q[t].w};
                    // (the largest magnitude as bits: NaN and Inf come out on top)
                    const uint32_t two = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                                  __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
                    uint32_t top = max(two & 0xFFFFu, two >> 16);
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const uint32_t e = max(top >> 7, 15u);
                    const bool finite = e < 255u;
                    const float up = __uint_as_float((268u - e) << 23);  // 2^(14 - e)
                    uint32_t h[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        float lo = bf_lo(w[n]), hi = bf_hi(w[n]);
                        if (finite) {
                            lo *= up, hi *= up;
                        } else {  // (beside NaN or Inf the finite ones do not matter)
                            lo = isfinite(lo) ? 0.0f : lo, hi = isfinite(hi) ? 0.0f : hi;
                        }
                        const __half2 v2 = __floats2half2_rn(lo, hi);
                        h[n] = *reinterpret_cast<const uint32_t*>(&v2);
                    }
                    if (k < padded) {
                        *reinterpret_cast<uint4*>(xs + t * pitch + k) = make_uint4(h[0], h[1], h[2], h[3]);
                        if (j == 0)
                            xscale[(k / 32) * TOK + t] = finite ? __uint_as_float((e - 14u) << 23) : 1.0f;
                    }
                }
            }
            named_barrier_sync(1, kWarps * 32);
        }
        if (!ok)
            continue;
        const bool live_set = at.expert(p) >= 0;
        float acc[4][2] = {};  // rows g + 8 q, tokens 2 j and 2 j + 1 (of 1 or 2: both, of the lane's blocks)
        for (int step = 0; live_set && step < steps; ++step, turn.next(p.stages), odd ^= 1u) {
            if (odd != static_cast<uint32_t>(group))
                continue;
            const uint32_t slot = turn.slot;
            if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(&full[slot]), turn.phase)))
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[slot], turn.phase, a.status, kStatusTimeout, a.wait_ns));
            if (!ok)
                break;
            // the stage may be loaded again as soon as its codes and scales are in registers
            auto release = [&]() {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&free_[slot]);
            };
            const int c = step * kChunks + chunk;
            if (c < p.chunks) {
                // piece i of row g + 8 q is at codes + 1024 q + ((i ^ g) << 4)
                const uint8_t* codes = ring + slot * BYTES + (chunk >> 1) * kSlab + g * 128;
                const int piece = (chunk & 1) * 4;
                const uint8_t* scales = ring + slot * BYTES + kCodeBytes + chunk * RUN + g * 16 + (at.set & 3) * 4;
                // (codes behind K are zeros; scales of groups that are not there are not used)
                const bool whole = (c + 1) * kChunk <= K;
                if constexpr (!kWide) {
                    const bool live = whole || c * kChunk + 32 * j < K;
                    uint32_t scw[4];
                    uint4 cw[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        scw[q] = *reinterpret_cast<const uint32_t*>(scales + q * 128 + (kNv && live ? (j >> 1) * 512 : 0));
                        cw[q] = *reinterpret_cast<const uint4*>(codes + q * 1024 + (((piece + j) ^ g) << 4));
                    }
                    release();
                    const float2 xsc = *reinterpret_cast<const float2*>(xscale + (c * 4 + j) * TOK);
                    uint32_t pairs[4];  // NVFP4: both groups' scales of a row
                    if constexpr (kNv) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            pairs[q] = e4m3x2(live ? scw[q] >> ((j & 1) * 16) : 0u);
                    }
                    float d[2][2][4];  // (two sums a tile, so that the MMAs wait less for one another)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint4 b = reinterpret_cast<const uint4*>(ring + b_at + c * b_step)[n];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t h[2][4];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                e2m1x8(reinterpret_cast<const uint32_t*>(&cw[2 * t + r])[n], h[r]);
                                if constexpr (kNv) {
                                    const uint32_t f = __byte_perm(pairs[2 * t + r], 0, n < 2 ? 0x1010 : 0x3232);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        h[r][k] = mul_f16x2(h[r][k], f);
                                }
                            }
                            if (n == 0) {
                                mma_16816<true>(d[t][0], h[0][0], h[1][0], h[0][1], h[1][1], b.x, b.y);
                                mma_16816<true>(d[t][1], h[0][2], h[1][2], h[0][3], h[1][3], b.z, b.w);
                            } else {
                                mma_16816<false>(d[t][0], h[0][0], h[1][0], h[0][1], h[1][1], b.x, b.y);
                                mma_16816<false>(d[t][1], h[0][2], h[1][2], h[0][3], h[1][3], b.z, b.w);
                            }
                        }
                    }
                    if (live) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            float2 f = make_float2(1.0f, 1.0f);
                            if constexpr (!kNv)
                                f = e8m0x2(__byte_perm(scw[2 * t], scw[2 * t + 1], j * 0x11 + 0x40));
                            acc[2 * t][0] += (d[t][0][0] + d[t][1][0]) * (f.x * xsc.x);
                            acc[2 * t][1] += (d[t][0][1] + d[t][1][1]) * (f.x * xsc.y);
                            acc[2 * t + 1][0] += (d[t][0][2] + d[t][1][2]) * (f.y * xsc.x);
                            acc[2 * t + 1][1] += (d[t][0][3] + d[t][1][3]) * (f.y * xsc.y);
                        }
                    }
                } else {
                    uint32_t scw[4], scv[4], cw[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        scw[q] = *reinterpret_cast<const uint32_t*>(scales + q * 128);
                        scv[q] = kNv ? *reinterpret_cast<const uint32_t*>(scales + q * 128 + 512) : 0u;
#pragma unroll
                        for (int bl = 0; bl < 4; ++bl)
                            cw[q][bl] = *reinterpret_cast<const uint32_t*>(codes + q * 1024 + (((piece + bl) ^ g) << 4) + j * 4);
                    }
                    release();
#pragma unroll
                    for (int bl = 0; bl < 4; ++bl) {
                        if (!whole && c * kChunk + 32 * bl >= K)
                            break;
                        const uint4 b = *reinterpret_cast<const uint4*>(ring + b_at + c * b_step + bl * b_block);
                        const float2 xsc = *reinterpret_cast<const float2*>(xscale + (c * 4 + bl) * TOK + 2 * j);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t h[2][4];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int q = 2 * t + r;
                                e2m1x8(cw[q][bl], h[r]);
                                if constexpr (kNv) {
                                    const uint32_t both = e4m3x2((bl < 2 ? scw[q] : scv[q]) >> ((bl & 1) * 16));
                                    const uint32_t f = __byte_perm(both, 0, j < 2 ? 0x1010 : 0x3232);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        h[r][k] = mul_f16x2(h[r][k], f);
                                }
                            }
                            float d[4];
                            mma_16816<true>(d, h[0][0], h[1][0], h[0][1], h[1][1], b.x, b.y);
                            mma_16816<false>(d, h[0][2], h[1][2], h[0][3], h[1][3], b.z, b.w);
                            float2 f = make_float2(1.0f, 1.0f);
                            if constexpr (!kNv)
                                f = e8m0x2(__byte_perm(scw[2 * t], scw[2 * t + 1], bl * 0x11 + 0x40));
                            add_scaled(acc[2 * t], d, f.x, xsc);
                            add_scaled(acc[2 * t + 1], d + 2, f.y, xsc);
                        }
                    }
                }
            } else {
                release();
            }
        }
        // (1 or 2 tokens: the blocks of a quad, then) this warp's sums
        const uint32_t place = sets % SUMS;
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(&taken[place]), (sets / SUMS & 1u) ^ 1u)))
            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_bounded(&taken[place], (sets / SUMS & 1u) ^ 1u, a.status, kStatusTimeout, a.wait_ns));
        if (!ok)
            continue;
        float* mine = red + (place * kWarps + warp) * TOK * kSetRows;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float sum = acc[q][t];
                if constexpr (!kWide) {
                    if (t >= tokens)
                        continue;
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                    if (j == t)
                        mine[t * kSetRows + q * 8 + g] = sum;
                } else {
                    mine[(2 * j + t) * kSetRows + q * 8 + g] = sum;
                }
            }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&summed[place]);
    }
}

// Shared memory beside the ring (and what aligns it).
size_t fixed_bytes(int chunks, int tokens, bool wide)
{
    const size_t padded = static_cast<size_t>(chunks) * kChunk, tok = wide ? 8 : 2;
    return 1024 + sum_buffers(wide) * kWarps * tok * kSetRows * 4 + tok * (padded / 32) * 4 + 64 + (2 * kMostStages + 4) * 8 + tokens * (padded + (wide ? 32 : 0)) * 2;
}

template <bool kWide, bool kNv>
cudaError_t launch(const GemvParams& p, int tokens, cudaStream_t stream)
{
    static std::mutex mu;
    static unsigned long long configured[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= 64)
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    auto kern = gemv_kernel<kWide, kNv>;
    {
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
            if (err != cudaSuccess)
                return err;
            configured[dev] = ctx;
        }
    }
    const size_t fixed = fixed_bytes(p.chunks, tokens, kWide);
    constexpr size_t stage = stage_bytes<kNv>();
    GemvParams q = p;
    q.all = p.a.expert_ids != nullptr ? static_cast<int64_t>(p.sets) * p.a.M : p.sets;
    const int64_t sms = sm_count();
    q.per = static_cast<int>((q.all + sms - 1) / sms);
    const int64_t steps = static_cast<int64_t>((p.chunks + kChunks - 1) / kChunks) * q.per;
    // An even number: a place of the ring then belongs to one loading warp and one group, which
    // wait for its rounds one by one.  (With an odd one a place changes hands every round; a
    // warp that is ahead could take the parity of the round before the last for the last's.)
    static_assert(kGroups == 2 && kLoaders == 2 && kMostStages % 2 == 0, "places of the ring");
    q.stages = static_cast<int>(std::min<int64_t>({static_cast<int64_t>((kMaxSmem - fixed) / stage), kMostStages, steps + 1}) / 2 * 2);
    if (fixed + 2 * stage > kMaxSmem || q.stages < 2)
        return cudaErrorInvalidValue;
    // (make_operand_map's bytes: rows of K / 2 of all the weights.  One copy of a stage's four
    // slabs, where K allows it, measured the same as four)
    CUtensorMap w_map;
    if (!make_operand_map(&w_map, p.a.w, p.a.N * (p.a.expert_ids != nullptr ? p.a.E : 1), p.a.K / 2, kSetRows, 1, kOpBytes))
        return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>((q.all + q.per - 1) / q.per);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), fixed + q.stages * stage, stream, q, w_map);
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t stream)
{
    GemvParams p = {};
    p.a = a;
    p.kb4 = static_cast<int>((a.K / (a.nv ? 16 : 32) + 3) / 4);
    p.chunks = static_cast<int>((a.K + kChunk - 1) / kChunk);
    p.sets = static_cast<int>((a.N + kSetRows - 1) / kSetRows);
    p.expert_scales = (a.N + 127) / 128 * 512 * p.kb4;
    if (a.expert_ids != nullptr)
        return launch<false, false>(p, 1, stream);
    // the activations of a launch's rows have to fit into shared memory beside two stages:
    // long ones go a few at a time.  1 and 2 tokens, in the narrow / the wide form: MXFP4 4.5 / 4.5
    // and 5.2 / 4.9 us at 4096 x 4096, 8.6 / 8.9 and 9.6 / 9.2 at 14336 x 4096, 15.4 / 16.7 and
    // 17.0 / 17.2 at 18432 x 7168; NVFP4 4.9 / 4.9 and 5.5 / 5.2, 9.6 / 9.9 and 10.5 / 10.1, 17.4 /
    // 19.0 and 18.8 / 19.4: the narrow form gains more at the large ones than it loses for two
    // tokens at the small ones
    int step = a.M;
    while (step > 1 && fixed_bytes(p.chunks, step, step > 2) + 2 * (a.nv ? stage_bytes<true>() : stage_bytes<false>()) > kMaxSmem)
        --step;
    for (int m = 0; m < a.M; m += step) {
        const int tokens = std::min(step, a.M - m);
        p.a.x = static_cast<const __nv_bfloat16*>(a.x) + m * a.K;
        p.a.out = static_cast<__nv_bfloat16*>(a.out) + m * a.N;
        p.a.M = tokens;
        const cudaError_t err = tokens > 2 ? (a.nv ? launch<true, true>(p, tokens, stream) : launch<true, false>(p, tokens, stream))
                                           : (a.nv ? launch<false, true>(p, tokens, stream) : launch<false, false>(p, tokens, stream));
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace fp4lin
