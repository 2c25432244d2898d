// gemm_fp8.cu -- the FP8 linear layer with a scale per block of 128: the
// layers that a mixed-precision checkpoint keeps out of FP4 ("Efficiently
// Serving NVFP4 Models on AMD Instinct MI350X/MI355X ... via Online NVFP4 to
// Quark MXFP4 Requantization", pipeline description: FP8 layers are loaded
// as they are).
//
//   out[m, n] = bf16( sum_b sa[b, m] sw[n / 128, b]
//                       sum_{k in block b} A[m, k] B[n, k]  + bias[n] )
//
// A [M, K] and B [N, K] are E4M3, b runs over the blocks of 128 along K; sa
// is float32 per row and block, sw float32 per 128 x 128 block.
//
// The tensor cores multiply E4M3 without scales (tcgen05.mma kind::f8f6f4),
// so a block's products are summed in TMEM and each block's sum is scaled
// and added to a running fp32 sum in registers ("promotion"): one fused
// multiply-add per output and block, by warps that read one accumulator
// while the MMAs fill the next.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "formats.cuh"
#include "gemm_fp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace fp4lin {
namespace {

constexpr int kBlock = 128;  // elements of K per scale, and bytes of K per pipeline stage
constexpr int kThreadsQ = 256;
// blocks whose largest magnitude is below this are scaled as if it were this,
// so that neither the scale nor its inverse leaves the normal float32 range
constexpr float kAmaxFloor = 7.703719777548943e-34f;  // 2^-110
constexpr float kE4m3Max = 448.0f;

// ------------------------------------------------------------ quantizers

struct BlockScale {
    float scale, inverse;
};

// From the bit pattern of the block's largest |x|; NaN and Inf give a NaN
// scale (and the caller zero codes).
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits)
{
    BlockScale r;
    if (amax_bits >= 0x7F800000u) {
        r.scale = __uint_as_float(0x7FC00000u);
        r.inverse = 0.0f;
        return r;
    }
    const float a = fmaxf(__uint_as_float(amax_bits), kAmaxFloor);
    r.scale = __fdiv_rn(a, kE4m3Max);
    r.inverse = __fdiv_rn(kE4m3Max, a);
    return r;
}

__device__ __forceinline__ uint32_t bf16x8_amax(uint4 v)
{
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(a & 0xFFFFu, a >> 16);
}

__device__ __forceinline__ uint2 e4m3x8(uint4 v, float inv, bool zero)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(__uint_as_float(w[j] << 16), inv),
                                                    __fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return zero ? make_uint2(0u, 0u) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Activations: 16 lanes take one row's block of 128, 8 elements each, and
// kActBlocks blocks in turn with their loads started together.
constexpr int kActBlocks = 4;

__global__ void __launch_bounds__(kThreadsQ) quant_act_fp8_kernel(const __nv_bfloat16* __restrict__ x,
                                                                  uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales, uint32_t blocks, int K,
                                                                  DivMagic per_row, int kb, int ms)
{
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 15;
    const uint32_t first = blockIdx.x * (kThreadsQ / 16 * kActBlocks) + (threadIdx.x >> 4);
    uint4 v[kActBlocks];
    uint32_t row[kActBlocks];
    int b[kActBlocks];
#pragma unroll
    for (int i = 0; i < kActBlocks; ++i) {
        const uint32_t item = first + i * (kThreadsQ / 16);
        row[i] = div_by_magic(item, per_row);
        b[i] = static_cast<int>(item - row[i] * kb);
        const int col = b[i] * kBlock + lane * 8;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (item < blocks && col < K)
            v[i] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row[i]) * K + col));
    }
#pragma unroll
    for (int i = 0; i < kActBlocks; ++i) {
        const uint32_t item = first + i * (kThreadsQ / 16);
        uint32_t am = bf16x8_amax(v[i]);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
            am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, d));
        const BlockScale s = block_scale(am << 16);
        const int col = b[i] * kBlock + lane * 8;
        if (item < blocks && col < K)
            *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(row[i]) * K + col) =
                e4m3x8(v[i], s.inverse, s.inverse == 0.0f);
        if (item < blocks && lane == 0)
            scales[static_cast<int64_t>(b[i]) * ms + row[i]] = s.scale;
    }
}

// Weights: one CTA per 128 x 128 block; the block stays in registers between
// its maximum and its codes.
__global__ void __launch_bounds__(kThreadsQ) quant_weight_fp8_kernel(const __nv_bfloat16* __restrict__ w,
                                                                     uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales, int64_t N, int K, int kb)
{
    __shared__ uint32_t part[kThreadsQ / 32];
    grid_dependency_wait();
    launch_dependents();
    const int64_t nb = blockIdx.x / kb;
    const int b = static_cast<int>(blockIdx.x - nb * kb);
    const int col = b * kBlock + (threadIdx.x & 15) * 8;
    const int64_t row0 = nb * kBlock + (threadIdx.x >> 4);
    uint4 v[8];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        v[i] = (row < N && col < K) ? __ldg(reinterpret_cast<const uint4*>(w + row * K + col)) : make_uint4(0u, 0u, 0u, 0u);
        am = max(am, bf16x8_amax(v[i]));
    }
    am = __reduce_max_sync(0xFFFFFFFFu, am);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = am;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreadsQ / 32; ++i)
        am = max(am, part[i]);
    const BlockScale s = block_scale(am << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        if (row < N && col < K)
            *reinterpret_cast<uint2*>(codes + row * K + col) = e4m3x8(v[i], s.inverse, s.inverse == 0.0f);
    }
    if (threadIdx.x == 0)
        scales[nb * kb + b] = s.scale;
}

// ------------------------------------------- GEMM, weights on the M side
//
// One CTA: 128 weight rows x NT tokens, a run of the K blocks.  The CTAs of a
// cluster share one output tile and split K; at the end each writes its sums
// to the shared memory of the CTA that owns the token, which adds them in the
// CTAs' order: one cluster barrier (about 1 us), no memory traffic, no second
// kernel.
//   warp 0  TMA of the weights (which no kernel of the same call writes, so
//           they stream before the quantizer ahead of this kernel is done)
//   warp 1  TMEM, MMAs: four of K = 32 per block into one of BUFS accumulators
//   warp 2  TMA of the tokens
//   warp 3  a block's scales, to a ring in shared memory
//   warps 4..  promotion: lane = weight row, NT / WGS columns per warp
// Every wait that may last starts behind the grid dependency: its limit is for
// this kernel's own copies and products, not for the kernel ahead, beside which
// the CTA may already be resident (1 x 4096 x 4096: 7.78 us, 7.63 without).
// A block has two barriers, `ready` (its operands and scales have landed and
// its accumulator has been read) and `done` (its MMAs are complete), so that
// the MMA thread, the one serial part, waits and commits once per block.
template <int NT>
struct SwapCfg {
    static constexpr int STAGES = NT == 16 ? 5 : NT == 32 ? 4 : NT == 64 ? 3 : 4;
    static constexpr int WGS = NT >= 64 ? 2 : 1;   // promotion warpgroups
    static constexpr int COLS = NT / WGS;          // columns per promotion warp
    static constexpr int BUFS = NT >= 64 ? 2 : 4;
    static constexpr int CTAS = NT >= 128 ? 1 : 2;   // per SM
    // blocks of scales in shared memory: a slot is written when block j - STAGES is
    // done, which block j - STAGES - BUFS's accumulator had to be read for; the
    // scales of that block may still be in use then, those of the one before not
    static constexpr int RING = STAGES + BUFS + 1;
    static constexpr int SLOT = NT + 4;            // the tokens' scales, then the weight's
    static constexpr int W_BYTES = 128 * kBlock;
    static constexpr int X_BYTES = NT * kBlock;
    static constexpr int OFF_X = STAGES * W_BYTES;
    // [splits][tokens of this CTA][128] floats: up to 7 more than NT rows where the
    // cluster's size does not divide the tokens
    static constexpr int OFF_SUM = OFF_X + STAGES * X_BYTES;
    static constexpr int OFF_SA = OFF_SUM + (NT + 7) * 128 * 4;
    static constexpr int OFF_BAR = OFF_SA + RING * SLOT * 4;
    static constexpr int NUM_BARS = 2 * STAGES;
    static constexpr int OFF_SLOT = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM = OFF_SLOT + 16 + 1024;  // + alignment slack
    static constexpr int TMEM_COLS = BUFS * NT < 32 ? 32 : BUFS * NT;
    static constexpr int THREADS = 128 + 128 * WGS;
    static_assert(BUFS <= STAGES, "an accumulator's release counts on the barrier of a later block");
    static_assert(TMEM_COLS * CTAS <= 512 && SMEM * CTAS <= 226 * 1024, "CTAs per SM");
};

struct SwapParams {
    const float* sa;
    const float* sw;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    int M, N;
    int kb;       // blocks of K
    int ms;       // row stride of sa
    int splits;   // cluster size
    int early_w;  // the weights are complete before this kernel may start
    unsigned long long wait_ns;
    unsigned int* status;
};

template <int NT>
__global__ void __launch_bounds__(SwapCfg<NT>::THREADS, SwapCfg<NT>::CTAS)
    gemm_fp8_swap_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const SwapParams p)
{
    using C = SwapCfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* done = ready + C::STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x;
    const int n0 = blockIdx.y * 128, m0 = blockIdx.z * NT;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * split / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (split + 1) / p.splits);
    const int nkb = kb1 - kb0;
    const uint64_t limit = p.wait_ns;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ready[s], 2 + 32 + 4 * C::WGS);  // two producers, the scales' lanes, the promotion warps
            mbar_init(&done[s], 1);
        }
        fence_mbar_init();
        tma_prefetch_map(&tmW);
        tma_prefetch_map(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (p.splits > 1)
        cluster_arrive();  // waited for before the first access to another CTA
    const uint32_t tmem = *tmem_slot;
    launch_dependents();

    float acc[C::COLS];
    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------- TMA producers
        if (lane == 0) {
            const bool w = warp == 0;
            if (!w || !p.early_w)
                grid_dependency_wait();
            uint8_t* base = w ? smem : smem + C::OFF_X;
            const int bytes = w ? C::W_BYTES : C::X_BYTES;
            int it = 0;
            for (; it < nkb; ++it) {
                const int s = it % C::STAGES;
                if (it == C::STAGES && w && p.early_w)
                    grid_dependency_wait();  // the first round of slots is free
                // (a wait that gives up has given the copies in flight its whole limit to land)
                if (!mbar_wait_bounded(&done[s], ((it / C::STAGES) & 1) ^ 1, p.status, kStatusTimeout, limit))
                    break;
                mbar_arrive_expect_tx(&ready[s], bytes);
                tma_load_2d(base + s * bytes, w ? &tmW : &tmX, &ready[s], (kb0 + it) * kBlock, w ? n0 : m0);
            }
        }
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer
        if (lane == 0) {
            grid_dependency_wait();
            constexpr uint32_t idesc = idesc_e4m3(128, NT);
            const uint64_t wd = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t xd = smem_desc(smem_u32(smem + C::OFF_X), 16, 1024, 2);
            for (int it = 0; it < nkb; ++it) {
                const int s = it % C::STAGES;
                if (!mbar_wait_bounded(&ready[s], (it / C::STAGES) & 1, p.status, kStatusTimeout, limit))
                    break;
                tc_fence_after_sync();
                const uint32_t acc_addr = tmem + (it % C::BUFS) * NT;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_f8f6f4(acc_addr, wd + ((s * C::W_BYTES + 32 * k) >> 4), xd + ((s * C::X_BYTES + 32 * k) >> 4),
                                  idesc, k != 0);
                tc_commit(&done[s]);
            }
        }
    } else if (warp == 3) {
        // --------------------------------------------------------- scales
        grid_dependency_wait();
        float* ring = reinterpret_cast<float*>(smem + C::OFF_SA);
        const float* sw = p.sw + static_cast<int64_t>(blockIdx.y) * p.kb + kb0;
        for (int it = 0; it < nkb; ++it) {
            const int s = it % C::STAGES;
            float* slot = ring + (it % C::RING) * C::SLOT;
            const bool ok = lane != 0 || mbar_wait_bounded(&done[s], ((it / C::STAGES) & 1) ^ 1, p.status,
                                                           kStatusTimeout, limit);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            if (lane < NT / 4) {
                const int m = m0 + lane * 4;  // rows are padded to a multiple of 4
                cp_async_16(slot + lane * 4, p.sa + static_cast<int64_t>(kb0 + it) * p.ms + (m < p.ms ? m : 0), m < p.ms);
            }
            if (lane == 0)
                cp_async_4(slot + NT, sw + it);
            cp_async_arrive(&ready[s]);
        }
        cp_async_wait_all();
    } else if (warp >= 4) {
        // ------------------------------------------------------ promotion
        grid_dependency_wait();
        const int quad = warp & 3, col0 = ((warp - 4) >> 2) * C::COLS;
#pragma unroll
        for (int j = 0; j < C::COLS; ++j)
            acc[j] = 0.0f;
        const float* ring = reinterpret_cast<const float*>(smem + C::OFF_SA);
        if (lane == 0)  // the accumulators start free
            for (int i = 0; i < C::BUFS; ++i)
                mbar_arrive(&ready[i]);
        for (int it = 0; it < nkb; ++it) {
            const bool ok = mbar_wait_bounded(&done[it % C::STAGES], (it / C::STAGES) & 1, p.status, kStatusTimeout, limit);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            tc_fence_after_sync();
            const uint32_t addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (it % C::BUFS) * NT + col0;
            const float* slot = ring + (it % C::RING) * C::SLOT;
            const float w = slot[NT];
            constexpr int CH = C::COLS < 32 ? C::COLS : 32;
#pragma unroll
            for (int c = 0; c < C::COLS; c += CH) {
                uint32_t d[CH];
                if constexpr (CH == 32)
                    tmem_ld_32x32b_x32(addr + c, d);
                else
                    tmem_ld_32x32b_x16(addr, d);
                tmem_ld_wait();
                if (c + CH == C::COLS) {
                    // block it + BUFS may overwrite the accumulator
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&ready[(it + C::BUFS) % C::STAGES]);
                }
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    const float4 s = *reinterpret_cast<const float4*>(slot + col0 + c + j);
                    acc[c + j] = fmaf(__uint_as_float(d[j]), s.x * w, acc[c + j]);
                    acc[c + j + 1] = fmaf(__uint_as_float(d[j + 1]), s.y * w, acc[c + j + 1]);
                    acc[c + j + 2] = fmaf(__uint_as_float(d[j + 2]), s.z * w, acc[c + j + 2]);
                    acc[c + j + 3] = fmaf(__uint_as_float(d[j + 3]), s.w * w, acc[c + j + 3]);
                }
            }
        }
    }

    // ---------------------------------------------------- reduce and store
    // token r of the tile belongs to CTA r / per of the cluster
    __syncwarp();
    const int rows = min(NT, p.M - m0);
    const int per = (rows + p.splits - 1) / p.splits;
    float* sums = reinterpret_cast<float*>(smem + C::OFF_SUM);  // [splits][per][128]
    if (p.splits > 1)
        cluster_wait();
    if (warp >= 4) {
        const int quad = warp & 3, col0 = ((warp - 4) >> 2) * C::COLS;
        const uint32_t mine = smem_u32(sums + split * per * 128 + quad * 32 + lane);
        int owner = col0 / per, r = col0 - owner * per;
        uint32_t dst = mapa_shared(mine, min(owner, p.splits - 1));
#pragma unroll
        for (int j = 0; j < C::COLS; ++j) {
            if (col0 + j < rows)
                st_cluster_f32(dst + r * 512, acc[j]);
            if (++r == per) {
                r = 0;
                ++owner;
                dst = mapa_shared(mine, min(owner, p.splits - 1));
            }
        }
    }
    tc_fence_before_sync();
    if (p.splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // 8 outputs of a token per thread
    const int own = max(0, min(per, rows - split * per));
    for (int i = threadIdx.x; i < own * 16; i += C::THREADS) {
        const int r = i >> 4, c = (i & 15) * 8;
        if (n0 + c >= p.N)
            continue;
        float f[8] = {};
#pragma unroll 2
        for (int k = 0; k < p.splits; ++k) {
            const float4* src = reinterpret_cast<const float4*>(sums + (k * per + r) * 128 + c);
            const float4 u = src[0], v = src[1];
            f[0] += u.x, f[1] += u.y, f[2] += u.z, f[3] += u.w;
            f[4] += v.x, f[5] += v.y, f[6] += v.z, f[7] += v.w;
        }
        if (p.bias != nullptr) {
            const uint4 bb = *reinterpret_cast<const uint4*>(p.bias + n0 + c);
            const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] += __uint_as_float(bw[j] << 16);
                f[2 * j + 1] += __uint_as_float(bw[j] & 0xFFFF0000u);
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(m0 + split * per + r) * p.N + n0 + c) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int NT>
cudaError_t launch_swap(const Fp8GemmArgs& a, int splits, cudaStream_t stream)
{
    using C = SwapCfg<NT>;
    CUtensorMap tmW, tmX;
    if (!make_operand_map(&tmW, a.b, a.N, a.K, 128, 1, kOpBytes) ||
        !make_operand_map(&tmX, a.a, a.M, a.K, NT, 1, kOpBytes))
        return cudaErrorInvalidValue;
    SwapParams p;
    p.sa = a.sa;
    p.sw = a.sb;
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.M = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.kb = static_cast<int>((a.K + kBlock - 1) / kBlock);
    p.ms = static_cast<int>((a.M + 3) / 4 * 4);
    p.splits = splits;
    p.early_w = a.early_weights ? 1 : 0;
    p.wait_ns = a.wait_ns;
    p.status = a.status;
    auto kern = gemm_fp8_swap_kernel<NT>;
    static std::mutex mu;
    static unsigned long long configured[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= 64)
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    {
        // per device and context, once: the shared-memory opt-in
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (err != cudaSuccess)
                return err;
            configured[dev] = ctx;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, static_cast<unsigned>((a.N + 127) / 128), static_cast<unsigned>((a.M + NT - 1) / NT));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tmW, tmX, p);
}

// ------------------------------------------------- GEMM on CTA pairs
//
// Large problems: 256 x 256 output tiles of a cluster of two CTAs, as the FP4
// pair kernel (a 256-row MMA needs half the operand bytes per SM and cycle of
// two 128-row ones).  Each CTA holds 128 rows of A and of B per stage of 128
// K-elements, and the sums of its 128 rows x 256 columns.
//   warp 0, 2  TMA of A and of B, counted on the leader's ready barrier
//   warp 1     TMEM; in the leader, the pair's MMAs: one scale block into one
//              of two accumulators of 256 columns.  A barrier wait costs this
//              thread a few hundred cycles even when the phase is complete, and
//              a commit costs it too, against the 512 cycles of a block's MMAs;
//              so a block has one wait and one commit: `ready` of its stage
//              counts the operands and the promotion warps that have read the
//              accumulator (two blocks before), and `done` of its stage tells
//              both the producers and the promotion warps.  (2041 x 18432 x
//              7168 with the additions left out: 177 us with separate barriers,
//              150 us so.)
//   warps 4..11  promotion: warp (quad, half) owns 32 rows x 128 columns in
//              registers, a row per lane, the 128 columns one weight block: one
//              scale product per lane and block; then bias, bf16, TMA store
struct PairCfg {
    static constexpr int STAGES = 6;
    static constexpr int BYTES = 128 * kBlock;  // of A, and of B, per stage and CTA
    static constexpr int OFF_B = STAGES * BYTES;
    static constexpr int OFF_EPI = 2 * STAGES * BYTES;
    static constexpr int BOX_COLS = 64;
    static constexpr int BOX_BYTES = 32 * BOX_COLS * 2;
    static constexpr int OFF_BAR = OFF_EPI + 8 * BOX_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES;
    static constexpr int OFF_SLOT = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM = OFF_SLOT + 16 + 1024;  // + alignment slack
    static constexpr int THREADS = 384;
    static constexpr int REGS_LOW = 40, REGS_HIGH = 232;
    static_assert(REGS_LOW * 128 + REGS_HIGH * 256 <= 168 * THREADS, "register split");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct Fp8PairParams {
    const float* sa;
    const float* sw;
    const __nv_bfloat16* bias;
    int M, N;
    int kb;       // blocks of K
    int ms;       // row stride of sa
    int nb;       // 128-row blocks of B
    int m_pairs;  // 256-row tiles of A
    int tiles;
    unsigned long long wait_ns;
    unsigned int* status;
};

// a.xy + b.xy * c.xy, two fused multiply-adds in one instruction
__device__ __forceinline__ void fma2(float2& a, uint32_t b0, uint32_t b1, float2 c)
{
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%0, %1};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "r"(b0), "r"(b1), "f"(c.x), "f"(c.y));
}

__global__ void __launch_bounds__(PairCfg::THREADS, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmO, const Fp8PairParams p)
{
    using C = PairCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // leader: both CTAs' operands have landed and their promotion warps have
    // read the block's accumulator
    uint64_t* ready = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* done = ready + C::STAGES;  // the block's MMAs are complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    const uint64_t limit = p.wait_ns;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ready[s], 1 + 16);  // the bytes, 8 promotion warps x 2 CTAs
            mbar_init(&done[s], 1);
        }
        fence_mbar_init();
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        tma_prefetch_map(&tmO);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();
    grid_dependency_wait();
    launch_dependents();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOW));
        if ((warp == 0 || warp == 2) && lane == 0) {
            // ------------------------------------------------ TMA producers
            const bool is_a = warp == 0;
            const CUtensorMap* map = is_a ? &tmA : &tmB;
            uint8_t* base = smem + (is_a ? 0 : C::OFF_B);
            const uint32_t ready_leader = mapa_shared(smem_u32(ready), 0);
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < p.tiles && ok; t += pairs) {
                const int row0 = (is_a ? (t % p.m_pairs) : (t / p.m_pairs)) * 256 + 128 * rank;
                for (int kb = 0; kb < p.kb; ++kb, ++it) {
                    const int s = static_cast<int>(it % C::STAGES);
                    if (!mbar_wait_bounded(&done[s], ((it / C::STAGES) & 1u) ^ 1u, p.status, kStatusTimeout, limit)) {
                        ok = false;
                        break;
                    }
                    if (leader && is_a)
                        mbar_arrive_expect_tx(&ready[s], 4u * C::BYTES);
                    tma_load_2d_pair(base + s * C::BYTES, map, ready_leader + 8u * s, kb * kBlock, row0);
                }
            }
            // gave up: the copies in flight have had the wait's limit to land
        } else if (warp == 1 && leader && lane == 0) {
            // --------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_e4m3(256, 256);
            const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, 2);
            const uint64_t bd = smem_desc(smem_u32(smem + C::OFF_B), 16, 1024, 2);
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < p.tiles && ok; t += pairs) {
                for (int kb = 0; kb < p.kb; ++kb, ++it) {
                    const uint32_t s = it % C::STAGES, b = it & 1u;
                    if (!mbar_wait_bounded(&ready[s], (it / C::STAGES) & 1u, p.status, kStatusTimeout, limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t off = (s * C::BYTES) >> 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f8f6f4_pair(tmem + b * 256, ad + off + 2 * k, bd + off + 2 * k, idesc, k != 0);
                    tc_commit_pair_multicast(&done[s], 0x3);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_HIGH));
        // ------------------------------------------- promotion and epilogue
        const int ew = warp - 4, quad = warp & 3, half = ew >> 2;
        const uint32_t ready_leader = mapa_shared(smem_u32(ready), 0);
        if (lane == 0) {  // both accumulators start free
            mbar_arrive_cluster(ready_leader);
            mbar_arrive_cluster(ready_leader + 8u);
        }
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        uint8_t* stg = smem + C::OFF_EPI + ew * C::BOX_BYTES;
        uint32_t stage = 0, phase = 0, buf = 0;
        bool stored = false;
        for (int t = pair; t < p.tiles; t += pairs) {
            const float* sa = p.sa + min((t % p.m_pairs) * 256 + 128 * rank + 32 * quad + lane, p.ms - 1);
            const float* sw = p.sw + static_cast<int64_t>(min((t / p.m_pairs) * 2 + half, p.nb - 1)) * p.kb;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j)
                acc[j] = make_float2(0.0f, 0.0f);
            float a_next = __ldg(sa), w_next = __ldg(sw);
            bool ok = true;
            for (int left = p.kb; left > 0; --left) {
                const float s = a_next * w_next;
                if (left > 1) {
                    sa += p.ms;
                    ++sw;
                    a_next = __ldg(sa);
                    w_next = __ldg(sw);
                }
                ok = mbar_wait_bounded(&done[stage], phase, p.status, kStatusTimeout, limit);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t addr = tmem + lanes + buf * 256 + half * 128;
                const float2 ss = make_float2(s, s);
                // 32 columns at a time; the third and fourth loads run under the
                // first two's additions, so that a block shows the load's latency once
                uint32_t d[2][32];
                tmem_ld_32x32b_x32(addr, d[0]);
                tmem_ld_32x32b_x32(addr + 32, d[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c == 2) {
                        tmem_ld_wait();
                        // the block after the next may overwrite the accumulator
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(ready_leader +
                                                8u * (stage + 2 < C::STAGES ? stage + 2 : stage + 2 - C::STAGES));
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        fma2(acc[16 * c + j], d[c & 1][2 * j], d[c & 1][2 * j + 1], ss);
                    if (c < 2)
                        tmem_ld_32x32b_x32(addr + 64 + 32 * c, d[c]);
                }
                buf ^= 1u;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            // ---- bias, bf16, boxes of 32 rows x 64 columns
            const int row0 = (t % p.m_pairs) * 256 + 128 * rank + 32 * quad;
            const int n0 = (t / p.m_pairs) * 256 + 128 * half;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col0 = n0 + c * C::BOX_COLS;
                if (stored && lane == 0)
                    bulk_wait_group_read0();
                __syncwarp();
                uint8_t* my_row = stg + lane * (C::BOX_COLS * 2);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[2 * i] = acc[c * 32 + j * 4 + i].x;
                        f[2 * i + 1] = acc[c * 32 + j * 4 + i].y;
                    }
                    if (p.bias != nullptr && col0 + 8 * j < p.N) {
                        const uint4 bb = __ldg(reinterpret_cast<const uint4*>(p.bias + col0 + 8 * j));
                        const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[2 * i] += __uint_as_float(bw[i] << 16);
                            f[2 * i + 1] += __uint_as_float(bw[i] & 0xFFFF0000u);
                        }
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                        o[i] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    // 128-byte swizzle of the box
                    *reinterpret_cast<uint4*>(my_row + ((j ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                // boxes past the output's edge are clipped, whole ones skipped
                if (row0 < p.M && col0 < p.N) {
                    if (lane == 0) {
                        tma_store_2d(&tmO, stg, col0, row0);
                        bulk_commit_group();
                    }
                    stored = true;
                }
            }
        }
        if (stored && lane == 0)
            bulk_wait_group_read0();  // shared memory stays valid until the last store has read it
    }

    // both CTAs are done with the pair's barriers, shared memory and TMEM
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, 512);
    }
}

cudaError_t launch_pair(const Fp8GemmArgs& a, cudaStream_t stream)
{
    using C = PairCfg;
    CUtensorMap tmA, tmB, tmO;
    if (!make_operand_map(&tmA, a.a, a.M, a.K, 128, 1, kOpBytes) ||
        !make_operand_map(&tmB, a.b, a.N, a.K, 128, 1, kOpBytes) ||
        !make_output_map(&tmO, a.out, a.M, a.N, C::BOX_COLS, 32, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    Fp8PairParams p;
    p.sa = a.sa;
    p.sw = a.sb;
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    p.M = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.kb = static_cast<int>((a.K + kBlock - 1) / kBlock);
    p.ms = static_cast<int>((a.M + 3) / 4 * 4);
    p.nb = static_cast<int>((a.N + 127) / 128);
    p.m_pairs = static_cast<int>((a.M + 255) / 256);
    const int64_t tiles = p.m_pairs * ((a.N + 255) / 256);
    p.tiles = static_cast<int>(tiles);
    p.wait_ns = a.wait_ns;
    p.status = a.status;
    // per device and context, once: the shared-memory opt-in, the register
    // split check (setmaxnreg.inc waits until the registers it asks for are
    // free: never launch a split that the launch's allocation cannot cover) and
    // the number of pairs that fit on the GPU at once
    static std::mutex mu;
    static int resident[64] = {};
    static unsigned long long configured[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= 64)
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    {
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (resident[dev] == 0 || configured[dev] != ctx) {
            err = cudaFuncSetAttribute(gemm_fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (err != cudaSuccess)
                return err;
            cudaFuncAttributes fa;
            err = cudaFuncGetAttributes(&fa, gemm_fp8_pair_kernel);
            if (err != cudaSuccess)
                return err;
            if (fa.numRegs * C::THREADS < C::REGS_LOW * 128 + C::REGS_HIGH * 256)
                return cudaErrorInvalidConfiguration;
            cfg.gridDim = dim3(2);
            cfg.numAttrs = 1;
            int clusters = 0;
            err = cudaOccupancyMaxActiveClusters(&clusters, gemm_fp8_pair_kernel, &cfg);
            if (err != cudaSuccess || clusters <= 0)
                return err != cudaSuccess ? err : cudaErrorInvalidConfiguration;
            configured[dev] = ctx;
            resident[dev] = std::min(clusters, sm_count() / 2);
        }
    }
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(tiles, resident[dev])));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_fp8_pair_kernel, tmA, tmB, tmO, p);
}

}  // namespace

cudaError_t launch_quant_act_fp8(const void* x, uint8_t* codes, float* scales, int64_t M, int64_t K,
                                 cudaStream_t stream)
{
    const int kb = static_cast<int>((K + kBlock - 1) / kBlock);
    const int64_t blocks = M * kb;
    constexpr int per_cta = kThreadsQ / 16 * kActBlocks;
    return launch_pdl(quant_act_fp8_kernel, dim3(static_cast<unsigned>((blocks + per_cta - 1) / per_cta)), dim3(kThreadsQ),
                      0, stream, static_cast<const __nv_bfloat16*>(x), codes, scales, static_cast<uint32_t>(blocks),
                      static_cast<int>(K), div_magic(static_cast<uint32_t>(kb)), kb, static_cast<int>((M + 3) / 4 * 4));
}

cudaError_t launch_quant_weight_fp8(const void* w, uint8_t* codes, float* scales, int64_t N, int64_t K,
                                    cudaStream_t stream)
{
    const int kb = static_cast<int>((K + kBlock - 1) / kBlock);
    return launch_pdl(quant_weight_fp8_kernel, dim3(static_cast<unsigned>((N + 127) / 128 * kb)), dim3(kThreadsQ), 0,
                      stream, static_cast<const __nv_bfloat16*>(w), codes, scales, N, static_cast<int>(K), kb);
}

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, cudaStream_t stream)
{
    const int64_t kb = (a.K + kBlock - 1) / kBlock;
    const int nt = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
    const int64_t tiles = (a.N + 127) / 128 * ((a.M + nt - 1) / nt);
    const int64_t slots = nt == 128 ? sm_count() : 2 * sm_count();  // CTAs resident at once
    // Tiles of 128 x 128 while they fit the GPU at once, CTA pairs beyond:
    // 512 x 4096 x 4096 (128 tiles) 19.4 / 19.1 us, 256 x 14336 x 4096 (224)
    // 37.8 / 21.8 us, 256 x 4096 x 4096 (64, K in two) 12.8 / 18.4 us.
    if (a.M > 128 && tiles > slots)
        return launch_pair(a, stream);
    // Split K as far as one wave of CTAs goes and every part keeps two blocks:
    // 64 x 14336 x 4096 (112 tiles, 304 slots) 23.7 / 16.8 / 22.8 us in 1 / 2 / 4
    // parts, 1 x 4096 x 4096 (32 tiles) 13.4 / 8.8 / 7.2 / 6.8 us in 1 / 2 / 4 / 8.
    // Clusters of 3 and 6 leave places of a GPC empty: with the quantizer 64 x 11264
    // x 4096 (88 tiles) 18.8 / 16.6 us in 2 / 3 parts, 128 x 5120 x 13824 (40 tiles,
    // 152 slots) 31.6 / 25.1, but 64 x 12800 x 5120 (100 tiles) 21.5 / 26.8; 5 and 7
    // parts were never faster than 4 (64 x 7680 x 4096, 60 tiles: 13.3 / 19.0 in 4 / 5).
    int splits = 1;
    for (const int s : {2, 3, 4, 6, 8})
        if (tiles * s <= (s % 3 ? slots : slots * 7 / 8) && kb / s >= 2)
            splits = s;
    switch (nt) {
    case 16: return launch_swap<16>(a, splits, stream);
    case 32: return launch_swap<32>(a, splits, stream);
    case 64: return launch_swap<64>(a, splits, stream);
    default: return launch_swap<128>(a, splits, stream);
    }
}

}  // namespace fp4lin
