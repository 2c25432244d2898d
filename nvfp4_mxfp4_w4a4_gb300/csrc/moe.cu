// moe.cu -- the (token, choice) pairs of a mixture-of-experts layer as rows
// grouped by expert, and back: the steps before and behind the grouped GEMM.
//
//   dispatch   a stable counting sort of the pairs by expert (row_offsets,
//              row_of), then every token's vector to the rows of its choices;
//              in one launch where the pairs are few
//   combine    out[t] = sum_j w[t, j] y[row_of[t, j]]
//   backward   grad_y[row_of[t, j]] = w[t, j] grad[t],
//              grad_w[t, j] = <grad[t], y[row_of[t, j]]>
//
// All are bound by HBM but for the smallest calls, where the launches count: 4096
// tokens x 8 of 64 experts, 4096 wide, are 302 MB in 44.8 us (0.99 of a plain
// copy's rate) behind a sort of 8; the same tokens' sum 52 us (302 MB, 0.86), its
// gradient 89 us (571 MB, 0.95).  32 tokens: 3.3 us sorted and copied, 3.2 us summed,
// on the device; one token's sum 3.0.
// Nothing is added by atomics: every result has one order.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "decoder_ops.h"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace fp4lin {
namespace {

// ---------------------------------------------------------------- sorting

// One cluster sorts all pairs.  A warp owns a run of them and counts its experts
// (lanes of one expert find one another by ballots over the bits of its number,
// their first lane adds); sums over the warps, over the cluster's CTAs (through
// their shared memory) and over the experts then give each warp the row at which
// its pairs of an expert begin.  The ballots' instructions and the steps' latency
// are what it costs: 32768 pairs of 64 experts, sorted and their rows of 64
// elements copied, take 8.4 us, 12.0 with __match_any_sync.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Those of the warp's live lanes that have this live lane's number (below 2^bits).
__device__ __forceinline__ uint32_t lanes_of(bool live, int e, int bits)
{
    uint32_t same = __ballot_sync(0xFFFFFFFFu, live);
    for (int b = 0; b < bits; ++b) {
        const bool one = e >> b & 1;
        const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

constexpr int kAhead = 4;  // steps whose experts are loaded at once

template <int kCtas>
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                int32_t* __restrict__ row_offsets,
                                                                int32_t* __restrict__ row_of)
{
    extern __shared__ uint32_t smem[];
    uint32_t* hist = smem;                    // [kSortWarps][E]
    uint32_t* total = hist + kSortWarps * E;  // [E] of this CTA
    uint32_t* base = total + E;               // [E] first row of this CTA's pairs of an expert
    __shared__ uint32_t warp_sum[kSortWarps];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int bits = 32 - __clz(E - 1);
    // runs of whole warps' widths
    const int steps = (pairs + kCtas * kSortThreads - 1) / (kCtas * kSortThreads);
    const int first = (static_cast<int>(rank) * kSortWarps + warp) * steps * 32;
    for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads)
        hist[i] = 0;
    __syncthreads();
    uint32_t* mine = hist + warp * E;
    int ahead[kAhead];
    auto load = [&](int s) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = first + (s + k) * 32 + lane;
            ahead[k] = s + k < steps && i < pairs ? __ldg(ids + i) : -1;
        }
    };
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
        load(s0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s0 + k >= steps)
                break;
            const int e = ahead[k];
            const bool live = e >= 0 && e < E;
            const uint32_t same = lanes_of(live, e, bits);
            if (live && lane == __ffs(same) - 1)
                mine[e] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // counts -> those of the warps before, and the CTA's sums
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        uint32_t n[kSortWarps], sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w)
            n[w] = hist[w * E + e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            hist[w * E + e] = sum;
            sum += n[w];
        }
        total[e] = sum;
    }
    cluster_sync_all();
    // (E <= kSortThreads: a thread per expert)
    const int e = threadIdx.x;
    uint32_t before = 0, all = 0;
    if (e < E) {
#pragma unroll
        for (int r = 0; r < kCtas; ++r) {
            const uint32_t n = ld_cluster_u32(mapa_shared(smem_u32(total + e), r));
            before += r < static_cast<int>(rank) ? n : 0u;
            all += n;
        }
    }
    uint32_t x = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        x += lane >= d ? y : 0u;
    }
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    uint32_t offset = x - all;
    for (int w = 0; w < warp; ++w)
        offset += warp_sum[w];
    if (e < E) {
        base[e] = offset + before;
        if (rank == 0) {
            row_offsets[e] = static_cast<int32_t>(offset);
            if (e == E - 1)
                row_offsets[E] = static_cast<int32_t>(offset + all);
        }
    }
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
        if (steps > kAhead)  // (else they are still there)
            load(s0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s0 + k >= steps)
                break;
            const int i = first + (s0 + k) * 32 + lane, ex = ahead[k];
            const bool live = ex >= 0 && ex < E;
            const uint32_t same = lanes_of(live, ex, bits);
            if (i < pairs)
                row_of[i] = live ? static_cast<int32_t>(base[ex] + mine[ex] + __popc(same & ((1u << lane) - 1u))) : -1;
            __syncwarp();
            if (live && lane == __ffs(same) - 1)
                mine[ex] += __popc(same);
            __syncwarp();
        }
    }
    cluster_sync_all();  // the others may still read this CTA's sums
}

// ---------------------------------------------------------------- vectors

// Threads of a block: `across` (a power of two) vectors of 8 of a token, and as
// many tokens as fit.
constexpr int kThreads = 128;

struct Shape {
    int across_log;
    dim3 grid;
};

Shape shape_of(int64_t tokens, int64_t width)
{
    Shape s;
    s.across_log = 0;
    while ((1 << s.across_log) < kThreads && (int64_t(8) << s.across_log) < width)
        ++s.across_log;
    const int64_t down = kThreads >> s.across_log;
    s.grid = dim3(static_cast<unsigned>((tokens + down - 1) / down),
                  static_cast<unsigned>((width / 8 + (int64_t(1) << s.across_log) - 1) >> s.across_log));
    return s;
}

struct Place {
    int64_t token;
    int64_t at;  // first element of the vector
};

__device__ __forceinline__ Place place_of(int across_log)
{
    const int across = 1 << across_log;
    return {static_cast<int64_t>(blockIdx.x) * (kThreads >> across_log) + (threadIdx.x >> across_log),
            (static_cast<int64_t>(blockIdx.y) * across + (threadIdx.x & (across - 1))) * 8};
}

__global__ void __launch_bounds__(kThreads) moe_gather_kernel(const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ row_of,
                                                              int64_t tokens, int top_k, int64_t width, int64_t xt,
                                                              __nv_bfloat16* __restrict__ sorted, int across_log)
{
    const Place p = place_of(across_log);
    const bool live = p.token < tokens && p.at < width;
    uint4 v = make_uint4(0, 0, 0, 0);
    // (before the sort has ended: what came before it, and may have written x, ended before
    // the sort let this kernel start)
    if (live)
        v = *reinterpret_cast<const uint4*>(x + p.token * xt + p.at);
    grid_dependency_wait();
    launch_dependents();
    if (!live)
        return;
    for (int j = 0; j < top_k; ++j) {
        const int64_t row = row_of[p.token * top_k + j];
        if (row >= 0)
            *reinterpret_cast<uint4*>(sorted + row * width + p.at) = v;
    }
}

// Few pairs: every block finds the rows of its own tokens' choices by counting, over
// all pairs, those of lower experts and the earlier ones of the same.  Block 0 also
// writes the offsets.  At most kFewPairs pairs, kFewOwn of them a block's: one launch
// takes 3.2 us for 256 pairs, 4096 wide, and 4.0 for 1024 where the sort and the copies
// take 5.2 and 6.4; 16 choices a block 4.3 against 5.7, but 32 6.1 against 5.6.
constexpr int kFewPairs = 1024, kFewOwn = 16;

__global__ void __launch_bounds__(kThreads) moe_dispatch_few_kernel(const __nv_bfloat16* __restrict__ x,
                                                                    const int32_t* __restrict__ ids, int tokens, int top_k,
                                                                    int E, int64_t width, int64_t xt,
                                                                    __nv_bfloat16* __restrict__ sorted,
                                                                    int32_t* __restrict__ row_offsets,
                                                                    int32_t* __restrict__ row_of, int across_log)
{
    constexpr int kWarps = kThreads / 32, kMine = kFewPairs / kThreads;
    constexpr int kNone = 0x7FFFFFFF;  // of no expert: behind all
    __shared__ int own[kFewOwn], part[kWarps][kFewOwn];
    extern __shared__ int counts[];  // [E], block 0's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place p = place_of(across_log);
    const bool live = p.token < tokens && p.at < width;
    const int pairs = tokens * top_k;
    const int down = kThreads >> across_log;
    const int first = static_cast<int>(blockIdx.x) * down * top_k;  // pair of the block
    const int owned = min(down * top_k, pairs - first);
    grid_dependency_wait();
    launch_dependents();
    uint4 v = make_uint4(0, 0, 0, 0);
    if (live)
        v = *reinterpret_cast<const uint4*>(x + p.token * xt + p.at);
    int mine[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int q = k * kThreads + threadIdx.x;
        const int e = q < pairs ? __ldg(ids + q) : -1;
        mine[k] = e >= 0 && e < E ? e : kNone;
        if (q >= first && q < first + owned)
            own[q - first] = mine[k];
    }
    __syncthreads();
    for (int o = 0; o < owned; ++o) {
        const int e = own[o], at = first + o;
        int n = 0;
#pragma unroll
        for (int k = 0; k < kMine; ++k)
            n += mine[k] < e || (mine[k] == e && k * kThreads + static_cast<int>(threadIdx.x) < at);
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0)
            part[warp][o] = n;
    }
    __syncthreads();
    for (int o = threadIdx.x; o < owned; o += kThreads) {
        int row = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            row += part[w][o];
        row = own[o] != kNone ? row : -1;
        own[o] = row;
        if (blockIdx.y == 0)
            row_of[first + o] = row;
    }
    __syncthreads();
    if (live) {
        const int* rows = own + (threadIdx.x >> across_log) * top_k;
        for (int j = 0; j < top_k; ++j)
            if (rows[j] >= 0)
                *reinterpret_cast<uint4*>(sorted + rows[j] * width + p.at) = v;
    }
    if (blockIdx.x != 0 || blockIdx.y != 0)
        return;
    for (int e = threadIdx.x; e < E; e += kThreads)
        counts[e] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        if (mine[k] != kNone)
            atomicAdd(&counts[mine[k]], 1);  // (whole numbers: in any order)
    __syncthreads();
    // a thread has a run of experts
    const int run = (E + kThreads - 1) / kThreads, e0 = min(threadIdx.x * run, E), e1 = min(e0 + run, E);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        sum += counts[e];
    int before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, before, d);
        before += lane >= d ? y : 0;
    }
    if (lane == 31)
        part[0][warp] = before;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w)
        before += part[0][w];
    for (int e = e0; e < e1; ++e) {
        row_offsets[e] = before;
        before += counts[e];
    }
    if (threadIdx.x == kThreads - 1)
        row_offsets[E] = before;
}

__global__ void __launch_bounds__(kThreads) moe_combine_kernel(const __nv_bfloat16* __restrict__ y, const int32_t* __restrict__ row_of,
                                                               const float* __restrict__ weights, int64_t tokens, int top_k,
                                                               int64_t rows, int64_t width, __nv_bfloat16* __restrict__ out,
                                                               int64_t ot, int across_log)
{
    const Place p = place_of(across_log);
    grid_dependency_wait();
    launch_dependents();
    if (p.token >= tokens || p.at >= width)
        return;
    float sum[8] = {};
#pragma unroll 4
    for (int j = 0; j < top_k; ++j) {
        const int64_t pair = p.token * top_k + j;
        const int64_t row = row_of != nullptr ? __ldg(row_of + pair) : pair;
        if (row < 0 || row >= rows)
            continue;
        const float w = weights != nullptr ? __ldg(weights + pair) : 1.0f;
        float f[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(y + row * width + p.at)), f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] += w * f[i];
    }
    *reinterpret_cast<uint4*>(out + p.token * ot + p.at) = pack8(sum);
}

// A warp per choice; the choices of a token share its gradient through L1.
__global__ void __launch_bounds__(256) moe_combine_backward_kernel(const __nv_bfloat16* __restrict__ grad,
                                                                   const __nv_bfloat16* __restrict__ y,
                                                                   const int32_t* __restrict__ row_of,
                                                                   const float* __restrict__ weights, int64_t pairs, int top_k,
                                                                   int64_t rows, int64_t width, int64_t gt,
                                                                   __nv_bfloat16* __restrict__ grad_y,
                                                                   float* __restrict__ grad_w)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (pair >= pairs)
        return;
    const int64_t row = row_of != nullptr ? __ldg(row_of + pair) : pair;
    float dot = 0.0f;
    if (row >= 0 && row < rows) {
        const float w = weights != nullptr ? __ldg(weights + pair) : 1.0f;
        const __nv_bfloat16* g = grad + pair / top_k * gt;
        for (int64_t at = lane * 8; at < width; at += 256) {
            float f[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(g + at)), f);
            if (grad_w != nullptr) {
                float v[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(y + row * width + at)), v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dot += f[i] * v[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] *= w;
            *reinterpret_cast<uint4*>(grad_y + row * width + at) = pack8(f);
        }
    }
    if (grad_w != nullptr) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
        if (lane == 0)
            grad_w[pair] = dot;
    }
}

}  // namespace

cudaError_t launch_moe_dispatch(const void* x, const int32_t* ids, int64_t tokens, int top_k, int E, int64_t width, int64_t xt,
                                void* sorted, int32_t* row_offsets, int32_t* row_of, cudaStream_t stream)
{
    const int64_t pairs = tokens * top_k;
    const Shape s = shape_of(tokens, width);
    if (tokens > 0 && pairs <= kFewPairs && (kThreads >> s.across_log) * top_k <= kFewOwn)
        return launch_pdl(moe_dispatch_few_kernel, s.grid, dim3(kThreads), static_cast<size_t>(E) * 4, stream,
                          static_cast<const __nv_bfloat16*>(x), ids, static_cast<int>(tokens), top_k, E, width, xt,
                          static_cast<__nv_bfloat16*>(sorted), row_offsets, row_of, s.across_log);
    // per device and context, once: the shared-memory opt-in
    static std::mutex mu;
    static unsigned long long configured[64] = {};
    constexpr int kMaxSmem = (kSortWarps + 2) * kMaxGroupedExperts * 4;
    static_assert(kMaxSmem <= 232448 - 1024 && kMaxGroupedExperts <= kSortThreads, "a thread per expert");
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= 64)
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long ctx = current_context_id();
        if (configured[dev] == 0 || configured[dev] != ctx) {
            for (auto* kern : {moe_sort_kernel<1>, moe_sort_kernel<kSortCluster>})
                if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) != cudaSuccess)
                    return err;
            configured[dev] = ctx;
        }
    }
    // one step of a CTA, or a cluster: 2048 pairs in 6.6 / 5.9 us, 8192 in 11.6 / 6.0, 32768 in
    // 31.8 / 8.4 (11.9 with 4 CTAs); up to 1024 the same.  Beyond that the cluster's 8 CTAs are
    // all there is: a million pairs, rows of 8 elements, take 118 us, nearly all of it the sort
    const int ctas = pairs <= kSortThreads ? 1 : kSortCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(kSortWarps + 2) * E * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, ctas == 1 ? moe_sort_kernel<1> : moe_sort_kernel<kSortCluster>, ids, static_cast<int>(pairs), E, row_offsets, row_of);
    if (err != cudaSuccess || tokens == 0)
        return err;
    return launch_pdl(moe_gather_kernel, s.grid, dim3(kThreads), 0, stream, static_cast<const __nv_bfloat16*>(x), row_of, tokens,
                      top_k, width, xt, static_cast<__nv_bfloat16*>(sorted), s.across_log);
}

cudaError_t launch_moe_combine(const void* y, const int32_t* row_of, const float* weights, int64_t tokens, int top_k,
                               int64_t rows, int64_t width, void* out, int64_t ot, cudaStream_t stream)
{
    const Shape s = shape_of(tokens, width);
    return launch_pdl(moe_combine_kernel, s.grid, dim3(kThreads), 0, stream, static_cast<const __nv_bfloat16*>(y), row_of,
                      weights, tokens, top_k, rows, width, static_cast<__nv_bfloat16*>(out), ot, s.across_log);
}

cudaError_t launch_moe_combine_backward(const void* grad, const void* y, const int32_t* row_of, const float* weights,
                                        int64_t tokens, int top_k, int64_t rows, int64_t width, int64_t gt, void* grad_y,
                                        float* grad_weights, cudaStream_t stream)
{
    const int64_t pairs = tokens * top_k;
    return launch_pdl(moe_combine_backward_kernel, dim3(static_cast<unsigned>((pairs + 7) / 8)), dim3(256), 0, stream,
                      static_cast<const __nv_bfloat16*>(grad), static_cast<const __nv_bfloat16*>(y), row_of, weights, pairs,
                      top_k, rows, width, gt, static_cast<__nv_bfloat16*>(grad_y), grad_weights);
}

}  // namespace fp4lin
