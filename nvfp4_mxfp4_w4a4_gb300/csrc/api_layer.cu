// api_layer.cu -- the extern "C" entry points of the operators around the FP4
// linear layer: the FP8 linear layer, rotary positions, the MX-quantized
// key/value cache and attention over it, norms of queries and keys, attention
// over whole prompts, matrix-vector products with 4-bit weights, and the way of
// tokens to their experts and back.  Same rules as api.cu: arguments are
// checked on the host before anything is enqueued, nothing is allocated,
// nothing synchronizes.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/fp4lin.h"
#include "decoder_ops.h"
#include "gemm_fp8.h"
#include "internal.h"
#include "kv_cache.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr double kTwoPi = 6.283185307179586476925286766559;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline fp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA; }
inline size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

inline fp4_status device(unsigned int** status = nullptr)
{
    return static_cast<fp4_status>(fp4lin::api_current_device(status));
}

// ------------------------------------------------------------- FP8 linear

int64_t fp8_blocks(int64_t n) { return (n + 127) / 128; }

bool fp8_dims_ok(int64_t rows, int64_t K)
{
    return rows >= 0 && K > 0 && K % 16 == 0 && rows < kMaxDim - 256 && K < kMaxDim - 256;
}

bool fp8_shape_ok(int64_t M, int64_t N, int64_t K)
{
    // tiles of 16 rows of M and 128 of N are grid dimensions
    return fp8_dims_ok(M, K) && M * fp8_blocks(K) < kMaxDim && N > 0 && N % 8 == 0 && N <= 65535 * int64_t(128) && M <= 65535 * int64_t(128);
}

// --------------------------------------------------------- cache and rope

fp4_status check_cache(const fp4_kv_cache* c, fp4lin::KvCache* out)
{
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
        return FP4_ERR_INVALID_ARG;
    if (c->format != FP4_ACT_MXFP4 && c->format != FP4_ACT_MXFP8)
        return FP4_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->num_pages >= kMaxDim || c->page_size <= 0 || c->page_size % 16 != 0 ||
        c->page_size > 4096 || c->kv_heads <= 0 || c->kv_heads > 1024 || (c->head_dim != 64 && c->head_dim != 128))
        return FP4_ERR_SHAPE;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
        return FP4_ERR_ALIGNMENT;
    out->k_codes = c->k_codes;
    out->k_scales = c->k_scales;
    out->v_codes = c->v_codes;
    out->v_scales = c->v_scales;
    out->pages = c->num_pages;
    out->page_size = c->page_size;
    out->heads = c->kv_heads;
    out->dim = c->head_dim;
    out->format = c->format;
    return FP4_OK;
}

fp4_status check_rope(const fp4_rope_params* r, const int32_t* positions, int64_t dim, fp4lin::RopeArgs* out)
{
    if (!r || !r->table || !positions)
        return FP4_ERR_INVALID_ARG;
    if (r->layout != FP4_ROPE_HALF && r->layout != FP4_ROPE_INTERLEAVED)
        return FP4_ERR_INVALID_ARG;
    if (r->flags & ~FP4_ROPE_INVERSE)
        return FP4_ERR_INVALID_ARG;
    if (r->table_positions <= 0 || r->table_positions >= kMaxDim || r->rot_dim <= 0 || r->rot_dim % 16 != 0 ||
        r->rot_dim > dim)
        return FP4_ERR_SHAPE;
    if (!aligned(r->table, 16) || !aligned(positions, 4))
        return FP4_ERR_ALIGNMENT;
    out->table = r->table;
    out->table_positions = r->table_positions;
    out->positions = positions;
    out->rot = r->rot_dim;
    out->layout = r->layout;
    out->inverse = (r->flags & FP4_ROPE_INVERSE) ? 1 : 0;
    return FP4_OK;
}

// Strides, in elements, of a [tokens][heads][dim] bf16 tensor whose rows the
// kernels read as 16-byte vectors.
fp4_status check_strides(const void* p, int64_t token, int64_t head)
{
    if (token < 0 || head < 0)
        return FP4_ERR_SHAPE;
    return aligned(p, 16) && token % 8 == 0 && head % 8 == 0 ? FP4_OK : FP4_ERR_ALIGNMENT;
}

fp4_status check_attention_shape(int32_t batch, int64_t total, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                 int64_t max_seq_len, int32_t max_draft)
{
    if (batch <= 0 || batch > 65535 || total < 0 || total >= (int64_t(1) << 24) || q_heads <= 0 || q_heads > 4096 ||
        kv_heads <= 0 || q_heads % kv_heads != 0 || (dim != 64 && dim != 128) || max_seq_len <= 0 ||
        max_seq_len > (int64_t(1) << 30) || max_draft <= 0 || max_draft > 1024 || max_draft > max_seq_len)
        return FP4_ERR_SHAPE;
    return FP4_OK;
}

fp4_status check_prompt_shape(int32_t batch, int64_t tokens, int64_t keys, int32_t q_heads, int32_t kv_heads, int32_t dim)
{
    if (batch <= 0 || batch > 65535 || tokens < 0 || tokens >= kMaxDim - 256 || keys < 0 || keys >= kMaxDim - 256 ||
        q_heads <= 0 || q_heads > 4096 || kv_heads <= 0 || q_heads % kv_heads != 0 || (dim != 64 && dim != 128) ||
        tokens * (q_heads / kv_heads) >= kMaxDim - 256)
        return FP4_ERR_SHAPE;
    return FP4_OK;
}

// Strides of a tensor map's dimensions (one of a single element has none).
bool map_strides_ok(int64_t tokens, int64_t heads, int64_t token, int64_t head)
{
    constexpr int64_t kMaxStride = int64_t(1) << 38;
    return (tokens <= 1 || (token > 0 && token <= kMaxStride)) && (heads <= 1 || (head > 0 && head <= kMaxStride));
}

// ------------------------------------------------------ products, experts

fp4_status check_gemv(const void* x, const void* w, const void* sw, const void* bias, const void* out, int64_t N, int64_t K)
{
    if (N <= 0 || N > (int64_t(1) << 24) || K <= 0 || K % 32 != 0 || K > 65536)
        return FP4_ERR_SHAPE;
    if (!x || !w || !sw || !out)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(sw, 16) || !aligned(out, 16) || !aligned(bias, 2))
        return FP4_ERR_ALIGNMENT;
    return FP4_OK;
}

fp4_status gemv(const void* x, const uint8_t* w, const uint8_t* sw, float w_global, const void* bias, void* out, int64_t M,
                int64_t N, int64_t K, bool nv, void* stream)
{
    if (M < 0 || M > 8)
        return FP4_ERR_SHAPE;
    if (M == 0)
        return FP4_OK;
    fp4_status st = check_gemv(x, w, sw, bias, out, N, K);
    fp4lin::GemvArgs a = {};
    if (st != FP4_OK || (st = device(&a.status)) != FP4_OK)
        return st;
    a.wait_ns = fp4lin::api_wait_limit_ns();
    a.withhold = fp4lin::api_withhold_signal();
    a.x = x, a.w = w, a.sw = sw, a.bias = bias, a.out = out;
    a.M = static_cast<int>(M), a.N = N, a.K = K;
    a.nv = nv, a.w_global = w_global;
    return from_cuda(fp4lin::launch_gemv(a, static_cast<cudaStream_t>(stream)));
}

fp4_status check_choices(int64_t tokens, int32_t top_k, int64_t width, int64_t stride)
{
    if (tokens < 0 || top_k <= 0 || top_k > 64 || tokens >= kMaxDim || tokens * top_k >= kMaxDim - 16384 || width <= 0 ||
        width % 8 != 0 || width > (int64_t(1) << 20) || stride < 0)
        return FP4_ERR_SHAPE;
    return stride % 8 == 0 ? FP4_OK : FP4_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

size_t fp4_fp8_act_scale_bytes(int64_t M, int64_t K)
{
    if (!fp8_dims_ok(M, K))
        return 0;
    return static_cast<size_t>(fp8_blocks(K) * ((M + 3) / 4 * 4)) * sizeof(float);
}

fp4_status fp4_quant_act_fp8_b128(const void* x_bf16, uint8_t* codes, float* scales, int64_t M, int64_t K, void* stream)
{
    if (!fp8_dims_ok(M, K) || M * fp8_blocks(K) >= kMaxDim)
        return FP4_ERR_SHAPE;
    if (M == 0)
        return FP4_OK;
    if (!x_bf16 || !codes || !scales)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return FP4_ERR_ALIGNMENT;
    const fp4_status st = device();
    if (st != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_quant_act_fp8(x_bf16, codes, scales, M, K, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_quant_weight_fp8_b128(const void* w_bf16, uint8_t* codes, float* scales, int64_t N, int64_t K,
                                     void* stream)
{
    if (!fp8_dims_ok(N, K) || N == 0 || fp8_blocks(N) * fp8_blocks(K) >= kMaxDim)
        return FP4_ERR_SHAPE;
    if (!w_bf16 || !codes || !scales)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(w_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return FP4_ERR_ALIGNMENT;
    const fp4_status st = device();
    if (st != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_quant_weight_fp8(w_bf16, codes, scales, N, K, static_cast<cudaStream_t>(stream)));
}

static fp4_status gemm_fp8(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, const void* bias,
                           void* out, int64_t M, int64_t N, int64_t K, bool early_weights, void* stream)
{
    fp4lin::Fp8GemmArgs g;
    const fp4_status st = device(&g.status);
    if (st != FP4_OK)
        return st;
    g.a = a, g.sa = sa, g.b = b, g.sb = sb, g.bias = bias, g.out = out;
    g.M = M, g.N = N, g.K = K;
    g.wait_ns = fp4lin::api_wait_limit_ns();
    g.early_weights = early_weights;
    return from_cuda(fp4lin::launch_gemm_fp8(g, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_gemm_fp8_b128(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, const void* bias_bf16,
                             void* out_bf16, int64_t M, int64_t N, int64_t K, void* stream)
{
    if (!fp8_shape_ok(M, N, K))
        return FP4_ERR_SHAPE;
    if (M == 0)
        return FP4_OK;
    if (!a || !sa || !b || !sb || !out_bf16)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(sa, 16) || !aligned(b, 16) || !aligned(sb, 4) || !aligned(out_bf16, 16) ||
        (bias_bf16 && !aligned(bias_bf16, 16)))
        return FP4_ERR_ALIGNMENT;
    return gemm_fp8(a, sa, b, sb, bias_bf16, out_bf16, M, N, K, false, stream);
}

size_t fp4_linear_fp8_b128_workspace_size(int64_t M, int64_t N, int64_t K)
{
    if (!fp8_shape_ok(M, N, K) || M == 0)
        return 0;
    return round_up(static_cast<size_t>(M) * K, 256) + round_up(fp4_fp8_act_scale_bytes(M, K), 256);
}

fp4_status fp4_linear_fp8_b128(const void* x_bf16, const uint8_t* b, const float* sb, const void* bias_bf16,
                               void* out_bf16, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    if (!fp8_shape_ok(M, N, K))
        return FP4_ERR_SHAPE;
    if (M == 0)
        return FP4_OK;
    if (!x_bf16 || !b || !sb || !out_bf16 || !workspace ||
        workspace_bytes < fp4_linear_fp8_b128_workspace_size(M, N, K))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(b, 16) || !aligned(sb, 4) || !aligned(out_bf16, 16) ||
        (bias_bf16 && !aligned(bias_bf16, 16)) || !aligned(workspace, 256))
        return FP4_ERR_ALIGNMENT;
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    float* sa = reinterpret_cast<float*>(codes + round_up(static_cast<size_t>(M) * K, 256));
    fp4_status st = device();
    if (st != FP4_OK)
        return st;
    st = from_cuda(fp4lin::launch_quant_act_fp8(x_bf16, codes, sa, M, K, static_cast<cudaStream_t>(stream)));
    if (st != FP4_OK)
        return st;
    // the quantizer is the kernel ahead: the weights were complete before it began
    return gemm_fp8(codes, sa, b, sb, bias_bf16, out_bf16, M, N, K, true, stream);
}

fp4_status fp4_rope_table(float* table, int64_t positions, int32_t rot_dim, double base, const fp4_rope_scaling* scaling,
                          void* stream)
{
    if (positions <= 0 || positions >= kMaxDim || rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > 1024)
        return FP4_ERR_SHAPE;
    if (!table || !(base > 1.0) || !std::isfinite(base))
        return FP4_ERR_INVALID_ARG;
    fp4lin::RopeFrequencies f = {base, fp4lin::kRopeNone, 1.0, 0.0, 0.0, 1.0};
    if (scaling) {
        if (scaling->kind != FP4_ROPE_UNSCALED && scaling->kind != FP4_ROPE_LINEAR && scaling->kind != FP4_ROPE_BY_PARTS)
            return FP4_ERR_INVALID_ARG;
        f.scaling = scaling->kind;
        if (f.scaling != FP4_ROPE_UNSCALED) {
            if (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor))
                return FP4_ERR_INVALID_ARG;
            f.factor = scaling->factor;
        }
        if (f.scaling == FP4_ROPE_BY_PARTS) {
            if (!(scaling->turns_slow > 0.0) || !(scaling->turns_fast >= scaling->turns_slow) ||
                !std::isfinite(scaling->turns_fast) || scaling->original_positions <= 0 ||
                !(scaling->magnitude > 0.0) || !std::isfinite(scaling->magnitude))
                return FP4_ERR_INVALID_ARG;
            // frequency index at which the original context holds a given number of turns; the
            // slow end may lie past the last frequency, rot_dim / 2 - 1
            const double half = rot_dim / 2;
            const double l = static_cast<double>(scaling->original_positions);
            f.low = std::fmax(std::floor(half * std::log(l / (scaling->turns_fast * kTwoPi)) / std::log(base)), 0.0);
            f.high = std::fmin(std::ceil(half * std::log(l / (scaling->turns_slow * kTwoPi)) / std::log(base)), rot_dim - 1.0);
            f.magnitude = scaling->magnitude;
        }
    }
    if (!aligned(table, 16))
        return FP4_ERR_ALIGNMENT;
    const fp4_status st = device();
    if (st != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_rope_table(table, positions, rot_dim, f, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_rope(const void* x_bf16, void* out_bf16, const int32_t* positions, const fp4_rope_params* rope,
                    int64_t tokens, int32_t heads, int32_t head_dim, int64_t x_token_stride, int64_t x_head_stride,
                    int64_t out_token_stride, int64_t out_head_stride, void* stream)
{
    if (tokens < 0 || heads <= 0 || heads > 65536 || head_dim <= 0 || head_dim % 16 != 0 || head_dim > 1024 ||
        tokens >= kMaxDim || tokens * heads * (head_dim / 16) >= (int64_t(1) << 32) - 1024)
        return FP4_ERR_SHAPE;  // 32-bit indexes of 16-element units
    if (tokens == 0)
        return FP4_OK;
    if (!x_bf16 || !out_bf16)
        return FP4_ERR_INVALID_ARG;
    fp4lin::RopeArgs r;
    fp4_status st = check_rope(rope, positions, head_dim, &r);
    if (st != FP4_OK)
        return st;
    if ((st = check_strides(x_bf16, x_token_stride, x_head_stride)) != FP4_OK ||
        (st = check_strides(out_bf16, out_token_stride, out_head_stride)) != FP4_OK)
        return st;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_rope(x_bf16, out_bf16, r, tokens, heads, head_dim, x_token_stride, x_head_stride,
                                         out_token_stride, out_head_stride, static_cast<cudaStream_t>(stream)));
}

size_t fp4_kv_code_bytes(const fp4_kv_cache* c)
{
    if (!c || (c->format != FP4_ACT_MXFP4 && c->format != FP4_ACT_MXFP8))
        return 0;
    const size_t elements = static_cast<size_t>(c->num_pages) * c->kv_heads * c->page_size * c->head_dim;
    return c->format == FP4_ACT_MXFP8 ? elements : elements / 2;
}

size_t fp4_kv_scale_bytes(const fp4_kv_cache* c)
{
    if (!c)
        return 0;
    return static_cast<size_t>(c->num_pages) * c->kv_heads * c->page_size * (c->head_dim / 32);
}

fp4_status fp4_kv_append(const fp4_kv_cache* cache, const void* k_bf16, const void* v_bf16, int64_t tokens,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         const int64_t* slots, const fp4_rope_params* rope, const int32_t* positions, void* stream)
{
    fp4lin::KvCache c;
    fp4_status st = check_cache(cache, &c);
    if (st != FP4_OK)
        return st;
    if (tokens < 0 || tokens >= kMaxDim || tokens * c.heads * (c.dim / 4) >= (int64_t(1) << 32) - 1024)
        return FP4_ERR_SHAPE;  // 32-bit indexes of 8-element vectors
    if (tokens == 0)
        return FP4_OK;
    if (!k_bf16 || !v_bf16 || !slots)
        return FP4_ERR_INVALID_ARG;
    fp4lin::RopeArgs r = {};
    if (rope && (st = check_rope(rope, positions, c.dim, &r)) != FP4_OK)
        return st;
    if ((st = check_strides(k_bf16, k_token_stride, k_head_stride)) != FP4_OK ||
        (st = check_strides(v_bf16, v_token_stride, v_head_stride)) != FP4_OK)
        return st;
    if (!aligned(slots, 8))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_kv_append(c, k_bf16, v_bf16, tokens, k_token_stride, k_head_stride, v_token_stride,
                                              v_head_stride, slots, r, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_kv_read(const fp4_kv_cache* cache, const int32_t* block_table, int64_t block_table_stride,
                       const int32_t* cu_lens, int32_t batch, int64_t rows, void* k_bf16, void* v_bf16, void* stream)
{
    fp4lin::KvCache c;
    fp4_status st = check_cache(cache, &c);
    if (st != FP4_OK)
        return st;
    if (batch <= 0 || rows < 0 || rows >= kMaxDim - 256 || block_table_stride <= 0)
        return FP4_ERR_SHAPE;
    if (rows == 0)
        return FP4_OK;
    if (!block_table || !cu_lens || !k_bf16 || !v_bf16)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(cu_lens, 4) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_kv_read(c, block_table, block_table_stride, cu_lens, batch, rows, k_bf16, v_bf16,
                                            static_cast<cudaStream_t>(stream)));
}

size_t fp4_kv_attention_workspace_size(int32_t batch, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                       int32_t head_dim, int64_t max_seq_len, int32_t max_draft)
{
    if (check_attention_shape(batch, tokens, q_heads, kv_heads, head_dim, max_seq_len, max_draft) != FP4_OK ||
        tokens == 0)
        return 0;
    return fp4lin::kv_attention_workspace_bytes(batch, tokens, q_heads, kv_heads, head_dim, max_seq_len, max_draft);
}

fp4_status fp4_kv_attention(const fp4_kv_cache* cache, const fp4_kv_attention_args* args, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    fp4lin::KvAttentionArgs a = {};
    fp4_status st = check_cache(cache, &a.cache);
    if (st != FP4_OK)
        return st;
    if (!args)
        return FP4_ERR_INVALID_ARG;
    if ((st = check_attention_shape(args->batch, args->tokens, args->q_heads, a.cache.heads, a.cache.dim,
                                    args->max_seq_len, args->max_draft)) != FP4_OK)
        return st;
    if (args->block_table_stride <= 0 || (args->tree_mask && args->mask_words * int64_t(32) < args->max_draft))
        return FP4_ERR_SHAPE;
    if (args->tokens == 0)
        return FP4_OK;
    if (!args->q_bf16 || !args->out_bf16 || !args->block_table || !args->context_lens || !args->q_offsets ||
        !(args->softmax_scale > 0.0f) || !std::isfinite(args->softmax_scale))
        return FP4_ERR_INVALID_ARG;
    const size_t need = fp4lin::kv_attention_workspace_bytes(args->batch, args->tokens, args->q_heads, a.cache.heads,
                                                             a.cache.dim, args->max_seq_len, args->max_draft);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return FP4_ERR_INVALID_ARG;
    if ((st = check_strides(args->q_bf16, args->q_token_stride, args->q_head_stride)) != FP4_OK ||
        (st = check_strides(args->out_bf16, args->out_token_stride, args->out_head_stride)) != FP4_OK)
        return st;
    if (!aligned(args->block_table, 4) || !aligned(args->context_lens, 4) || !aligned(args->q_offsets, 4) ||
        !aligned(args->tree_mask, 4) || !aligned(args->lse, 4) || (need > 0 && !aligned(workspace, 256)))
        return FP4_ERR_ALIGNMENT;
    if ((st = device(&a.status)) != FP4_OK)
        return st;
    a.wait_ns = fp4lin::api_wait_limit_ns();
    a.withhold = fp4lin::api_withhold_signal();
    a.q = args->q_bf16;
    a.out = args->out_bf16;
    a.lse = args->lse;
    a.qt = args->q_token_stride;
    a.qh = args->q_head_stride;
    a.ot = args->out_token_stride;
    a.oh = args->out_head_stride;
    a.block_table = args->block_table;
    a.table_stride = args->block_table_stride;
    a.context_lens = args->context_lens;
    a.q_offsets = args->q_offsets;
    a.tree_mask = args->tree_mask;
    a.mask_words = args->mask_words;
    a.batch = args->batch;
    a.T = args->tokens;
    a.q_heads = args->q_heads;
    a.max_seq = args->max_seq_len;
    a.max_draft = args->max_draft;
    a.scale = args->softmax_scale;
    a.workspace = workspace;
    return from_cuda(fp4lin::launch_kv_attention(a, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_qk_norm_rope(const fp4_qk_norm_args* args, const fp4_rope_params* rope, void* stream)
{
    if (!args)
        return FP4_ERR_INVALID_ARG;
    const fp4_qk_norm_args& g = *args;
    if (g.tokens < 0 || g.tokens >= kMaxDim || g.q_heads <= 0 || g.q_heads > 65536 || g.kv_heads < 0 || g.kv_heads > 65536 ||
        (g.head_dim != 64 && g.head_dim != 128 && g.head_dim != 256) ||
        g.tokens * (g.q_heads + g.kv_heads) * (g.head_dim / 16) >= (int64_t(1) << 32) - 1024)
        return FP4_ERR_SHAPE;  // 32-bit indexes of 16-element units
    if (!(g.eps >= 0.0f) || !std::isfinite(g.eps))
        return FP4_ERR_INVALID_ARG;
    if (g.tokens == 0)
        return FP4_OK;
    if (!g.q_bf16 || !g.q_out_bf16 || !g.q_weight_bf16 || (g.kv_heads > 0 && (!g.k_bf16 || !g.k_out_bf16 || !g.k_weight_bf16)))
        return FP4_ERR_INVALID_ARG;
    fp4lin::HeadNormArgs a = {};
    fp4_status st;
    if (rope && (st = check_rope(rope, g.positions, g.head_dim, &a.rope)) != FP4_OK)
        return st;
    if ((st = check_strides(g.q_bf16, g.q_token_stride, g.q_head_stride)) != FP4_OK ||
        (st = check_strides(g.q_out_bf16, g.q_out_token_stride, g.q_out_head_stride)) != FP4_OK)
        return st;
    if (g.kv_heads > 0 && ((st = check_strides(g.k_bf16, g.k_token_stride, g.k_head_stride)) != FP4_OK ||
                           (st = check_strides(g.k_out_bf16, g.k_out_token_stride, g.k_out_head_stride)) != FP4_OK))
        return st;
    if (!aligned(g.q_weight_bf16, 16) || (g.kv_heads > 0 && !aligned(g.k_weight_bf16, 16)))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    a.part[0] = {g.q_bf16, g.q_out_bf16, g.q_weight_bf16, g.q_token_stride, g.q_head_stride, g.q_out_token_stride, g.q_out_head_stride};
    a.part[1] = {g.k_bf16, g.k_out_bf16, g.k_weight_bf16, g.k_token_stride, g.k_head_stride, g.k_out_token_stride, g.k_out_head_stride};
    a.T = g.tokens;
    a.q_heads = g.q_heads, a.kv_heads = g.kv_heads, a.dim = g.head_dim;
    a.eps = g.eps;
    return from_cuda(fp4lin::launch_head_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t fp4_prompt_attention_workspace_size(int32_t batch, int64_t tokens, int64_t key_tokens, int32_t q_heads,
                                           int32_t kv_heads, int32_t head_dim)
{
    if (check_prompt_shape(batch, tokens, key_tokens, q_heads, kv_heads, head_dim) != FP4_OK || tokens == 0)
        return 0;
    return fp4lin::prompt_attention_workspace_bytes(batch, tokens, key_tokens, q_heads, kv_heads, head_dim);
}

fp4_status fp4_prompt_attention(const fp4_prompt_attention_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!args)
        return FP4_ERR_INVALID_ARG;
    const fp4_prompt_attention_args& g = *args;
    fp4_status st = check_prompt_shape(g.batch, g.tokens, g.key_tokens, g.q_heads, g.kv_heads, g.head_dim);
    if (st != FP4_OK)
        return st;
    if ((g.causal != 0 && g.causal != 1) || !(g.softmax_scale > 0.0f) || !std::isfinite(g.softmax_scale))
        return FP4_ERR_INVALID_ARG;
    if (g.tokens == 0)
        return FP4_OK;
    if (!g.q_bf16 || !g.out_bf16 || !g.q_offsets || !g.k_offsets || (g.key_tokens > 0 && (!g.k_bf16 || !g.v_bf16)))
        return FP4_ERR_INVALID_ARG;
    if ((st = check_strides(g.q_bf16, g.q_token_stride, g.q_head_stride)) != FP4_OK ||
        (st = check_strides(g.out_bf16, g.out_token_stride, g.out_head_stride)) != FP4_OK)
        return st;
    if (!map_strides_ok(g.tokens, g.q_heads, g.q_token_stride, g.q_head_stride))
        return FP4_ERR_SHAPE;
    if (g.key_tokens > 0) {
        if ((st = check_strides(g.k_bf16, g.k_token_stride, g.k_head_stride)) != FP4_OK ||
            (st = check_strides(g.v_bf16, g.v_token_stride, g.v_head_stride)) != FP4_OK)
            return st;
        if (!map_strides_ok(g.key_tokens, g.kv_heads, g.k_token_stride, g.k_head_stride) ||
            !map_strides_ok(g.key_tokens, g.kv_heads, g.v_token_stride, g.v_head_stride))
            return FP4_ERR_SHAPE;
    }
    const size_t need = fp4lin::prompt_attention_workspace_bytes(g.batch, g.tokens, g.key_tokens, g.q_heads, g.kv_heads, g.head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(g.q_offsets, 4) || !aligned(g.k_offsets, 4) || !aligned(g.lse, 4) || (need > 0 && !aligned(workspace, 256)))
        return FP4_ERR_ALIGNMENT;
    fp4lin::PromptArgs a = {};
    if ((st = device(&a.status)) != FP4_OK)
        return st;
    a.q = g.q_bf16, a.k = g.k_bf16, a.v = g.v_bf16, a.out = g.out_bf16, a.lse = g.lse;
    a.qt = g.q_token_stride, a.qh = g.q_head_stride, a.kt = g.k_token_stride, a.kh = g.k_head_stride;
    a.vt = g.v_token_stride, a.vh = g.v_head_stride, a.ot = g.out_token_stride, a.oh = g.out_head_stride;
    a.q_offsets = g.q_offsets, a.k_offsets = g.k_offsets;
    a.T = g.tokens, a.keys = g.key_tokens;
    a.batch = g.batch, a.q_heads = g.q_heads, a.kv_heads = g.kv_heads, a.dim = g.head_dim;
    a.causal = g.causal;
    a.scale = g.softmax_scale;
    a.workspace = workspace;
    a.wait_ns = fp4lin::api_wait_limit_ns();
    a.withhold = fp4lin::api_withhold_signal();
    return from_cuda(fp4lin::launch_prompt_attention(a, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_gemv_mxfp4(const void* x_bf16, const uint8_t* w, const uint8_t* sw, const void* bias_bf16, void* out_bf16,
                          int64_t M, int64_t N, int64_t K, void* stream)
{
    return gemv(x_bf16, w, sw, 1.0f, bias_bf16, out_bf16, M, N, K, false, stream);
}

fp4_status fp4_gemv_nvfp4(const void* x_bf16, const uint8_t* w, const uint8_t* sw, float w_global, const void* bias_bf16,
                          void* out_bf16, int64_t M, int64_t N, int64_t K, void* stream)
{
    return gemv(x_bf16, w, sw, w_global, bias_bf16, out_bf16, M, N, K, true, stream);
}

fp4_status fp4_gemv_mxfp4_experts(const void* x_bf16, const int32_t* expert_ids, int32_t E, int64_t rows, int32_t rows_per_x,
                                  const uint8_t* w, const uint8_t* sw, const void* bias_bf16, void* out_bf16, int64_t N,
                                  int64_t K, void* stream)
{
    if (E <= 0 || E > fp4lin::kMaxGroupedExperts || rows < 0 || rows > 65535 || rows_per_x <= 0)
        return FP4_ERR_SHAPE;
    if (rows == 0)
        return FP4_OK;
    fp4_status st = check_gemv(x_bf16, w, sw, bias_bf16, out_bf16, N, K);
    if (st != FP4_OK)
        return st;
    if (E * N >= kMaxDim - 256)
        return FP4_ERR_SHAPE;  // 32-bit rows
    if (!expert_ids)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(expert_ids, 4))
        return FP4_ERR_ALIGNMENT;
    fp4lin::GemvArgs a = {};
    if ((st = device(&a.status)) != FP4_OK)
        return st;
    a.wait_ns = fp4lin::api_wait_limit_ns();
    a.withhold = fp4lin::api_withhold_signal();
    a.x = x_bf16, a.w = w, a.sw = sw, a.bias = bias_bf16, a.out = out_bf16;
    a.M = static_cast<int>(rows), a.N = N, a.K = K;
    a.w_global = 1.0f;
    a.expert_ids = expert_ids, a.E = E, a.rows_per_x = rows_per_x;
    return from_cuda(fp4lin::launch_gemv(a, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_moe_dispatch(const void* x_bf16, const int32_t* expert_ids, int64_t tokens, int32_t top_k, int32_t E,
                            int64_t width, int64_t x_token_stride, void* sorted_bf16, int32_t* row_offsets, int32_t* row_of,
                            void* stream)
{
    fp4_status st = check_choices(tokens, top_k, width, x_token_stride);
    if (st != FP4_OK)
        return st;
    if (E <= 0 || E > fp4lin::kMaxGroupedExperts)
        return FP4_ERR_SHAPE;
    // (no tokens: the offsets are still written)
    if (!row_offsets || (tokens > 0 && (!x_bf16 || !expert_ids || !sorted_bf16 || !row_of)))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(sorted_bf16, 16) || !aligned(expert_ids, 4) || !aligned(row_offsets, 4) ||
        !aligned(row_of, 4))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_moe_dispatch(x_bf16, expert_ids, tokens, top_k, E, width, x_token_stride, sorted_bf16,
                                                 row_offsets, row_of, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_moe_combine(const void* y_bf16, const int32_t* row_of, const float* weights, int64_t tokens, int32_t top_k,
                           int64_t rows, int64_t width, void* out_bf16, int64_t out_token_stride, void* stream)
{
    fp4_status st = check_choices(tokens, top_k, width, out_token_stride);
    if (st != FP4_OK)
        return st;
    if (rows < 0 || rows >= kMaxDim)
        return FP4_ERR_SHAPE;
    if (tokens == 0)
        return FP4_OK;
    if (!out_bf16 || (rows > 0 && !y_bf16))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(y_bf16, 16) || !aligned(out_bf16, 16) || !aligned(row_of, 4) || !aligned(weights, 4))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_moe_combine(y_bf16, row_of, weights, tokens, top_k, rows, width, out_bf16,
                                                out_token_stride, static_cast<cudaStream_t>(stream)));
}

fp4_status fp4_moe_combine_backward(const void* grad_out_bf16, const void* y_bf16, const int32_t* row_of,
                                    const float* weights, int64_t tokens, int32_t top_k, int64_t rows, int64_t width,
                                    int64_t grad_out_token_stride, void* grad_y_bf16, float* grad_weights, void* stream)
{
    fp4_status st = check_choices(tokens, top_k, width, grad_out_token_stride);
    if (st != FP4_OK)
        return st;
    if (rows < 0 || rows >= kMaxDim)
        return FP4_ERR_SHAPE;
    if (tokens == 0)
        return FP4_OK;
    if (!grad_out_bf16 || (rows > 0 && (!grad_y_bf16 || (grad_weights && !y_bf16))))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(grad_out_bf16, 16) || !aligned(y_bf16, 16) || !aligned(grad_y_bf16, 16) || !aligned(row_of, 4) ||
        !aligned(weights, 4) || !aligned(grad_weights, 4))
        return FP4_ERR_ALIGNMENT;
    if ((st = device()) != FP4_OK)
        return st;
    return from_cuda(fp4lin::launch_moe_combine_backward(grad_out_bf16, y_bf16, row_of, weights, tokens, top_k, rows, width,
                                                         grad_out_token_stride, grad_y_bf16, grad_weights,
                                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
