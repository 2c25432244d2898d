"""The attention block of a decoder layer that a checkpoint keeps in FP8: the
q/k/v projection, rotary positions, the MX-quantized paged cache, attention of
the step's tokens over it, and the output projection -- the library's calls in
the order in which a serving step makes them, on buffers that are allocated
once.

    block = AttentionBlock(w_qkv, w_o, cache, rope, q_heads, max_tokens, max_batch,
                           max_seq_len, max_draft)
    out = block.step(x, positions, slots, block_table, context_lens, q_offsets, tree_mask)

A step's tokens are the drafted tokens of each sequence (one per sequence for
plain decoding, a chain or a tree of them otherwise): their keys and values are
appended to the cache at `slots` and then attended together with the context.
Whole prompts of any length go through

    out = block.prompt(x, positions, slots, q_offsets)

which attends their own keys and values in bf16, as they come from the projection,
and leaves them in the cache for the steps to come.  Everything is enqueued on the current CUDA stream; nothing synchronizes.
"""
from __future__ import annotations

import torch

from . import fp4lin as L


def allocate_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, format: int = L.FP4_ACT_MXFP8) -> L.kv_cache:
    """An empty MX-quantized paged cache on the current device."""
    width = head_dim if format == L.FP4_ACT_MXFP8 else head_dim // 2
    codes = [torch.zeros((num_pages, kv_heads, page_size, width), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((num_pages, kv_heads, page_size, head_dim // 32), dtype=torch.uint8, device="cuda")
              for _ in range(2)]
    return L.kv_cache(codes[0], scales[0], codes[1], scales[1], page_size, format)


class Fp8Linear:
    """y = x W^T (+ bias) with E4M3 weights and a scale per 128 x 128 block: codes
    [N, K] of one byte, scales float32 [N / 128, K / 128] rounded up, bias bf16 [N].
    A layer with one scale for its whole weight has that scale in every block."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None):
        self.codes, self.scales, self.bias = codes, scales, bias
        self.N, self.K = codes.shape
        if codes.element_size() != 1 or not codes.is_contiguous() or not all(
                t.is_cuda for t in (codes, scales, bias) if t is not None):
            raise ValueError("codes are contiguous bytes [N, K]; all are device tensors")
        if scales.dtype != torch.float32 or scales.shape != (-(-self.N // 128), -(-self.K // 128)) or not scales.is_contiguous():
            raise ValueError("scales are contiguous float32, one for each 128 x 128 block")
        if bias is not None and (bias.dtype != torch.bfloat16 or bias.shape != (self.N,) or not bias.is_contiguous()):
            raise ValueError("bias is contiguous bf16 [N]")

    @classmethod
    def from_bf16(cls, w: torch.Tensor, bias: torch.Tensor | None = None) -> "Fp8Linear":
        N, K = w.shape
        if w.dtype != torch.bfloat16 or not w.is_contiguous() or not w.is_cuda:
            raise ValueError("w is a contiguous bf16 device tensor [N, K]")
        codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
        scales = torch.empty((-(-N // 128), -(-K // 128)), dtype=torch.float32, device=w.device)
        L.fp4_quant_weight_fp8_b128(w, codes, scales, N, K)
        return cls(codes, scales, bias)

    def workspace_size(self, M: int) -> int:
        return L.fp4_linear_fp8_b128_workspace_size(M, self.N, self.K)

    def __call__(self, x: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor) -> torch.Tensor:
        if x.dtype is not torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.K or not x.is_contiguous() or not x.is_cuda:
            raise ValueError("x is a contiguous bf16 device tensor [M, K]")
        if out.dtype is not torch.bfloat16 or out.shape != (x.shape[0], self.N) or not out.is_contiguous() or not out.is_cuda:
            raise ValueError("out is a contiguous bf16 device tensor [M, N]")
        L.fp4_linear_fp8_b128(x, self.codes, self.scales, self.bias, out, x.shape[0], self.N, self.K, workspace)
        return out


class AttentionBlock:
    """qkv: Fp8Linear [(q_heads + 2 kv_heads) head_dim, hidden]; o: Fp8Linear
    [hidden, q_heads head_dim]; cache: allocate_cache(...); rope: fp4lin.rope_params.
    max_draft and max_seq_len choose the attention kernel and the cut of the
    contexts: a block for pieces of a prompt decodes single tokens slower than one
    made for them, which may share its cache, weights and rope.
    q_norm, k_norm (both or neither): bf16 [head_dim], the weights of a norm of every
    head of the queries and keys before the rotation; head_dim 64 or 128.
    prompts: allocate what prompt() needs."""

    def __init__(self, qkv: Fp8Linear, o: Fp8Linear, cache: L.kv_cache, rope: L.rope_params, q_heads: int,
                 max_tokens: int, max_batch: int, max_seq_len: int, max_draft: int, q_norm: torch.Tensor | None = None,
                 k_norm: torch.Tensor | None = None, norm_eps: float = 1e-6, prompts: bool = False):
        c = cache.struct
        self.qkv, self.o, self.cache, self.rope = qkv, o, cache, rope
        self.q_heads, self.kv_heads, self.head_dim = q_heads, c.kv_heads, c.head_dim
        if qkv.N != (q_heads + 2 * c.kv_heads) * c.head_dim or o.K != q_heads * c.head_dim:
            raise ValueError("the projections do not fit the heads")
        if (q_norm is None) != (k_norm is None):
            raise ValueError("q_norm and k_norm: both or neither")
        self.q_norm, self.k_norm, self.norm_eps = q_norm, k_norm, norm_eps
        self.max_tokens, self.max_batch = max_tokens, max_batch
        self.max_seq_len, self.max_draft = max_seq_len, max_draft
        self.projected = torch.empty((max_tokens, qkv.N), dtype=torch.bfloat16, device="cuda")
        self.attended = torch.empty((max_tokens, o.K), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty((max_tokens, o.N), dtype=torch.bfloat16, device="cuda")
        linear = max(qkv.workspace_size(max_tokens), o.workspace_size(max_tokens))
        self.linear_ws = torch.empty(linear, dtype=torch.uint8, device="cuda")
        # the size depends on the batch: few long sequences are cut into more parts
        attention = max(L.fp4_kv_attention_workspace_size(b, min(max_tokens, b * max_draft), q_heads, c.kv_heads, c.head_dim,
                                                          max_seq_len, max_draft) for b in range(1, max_batch + 1))
        self.attention_ws = torch.empty(max(attention, 1), dtype=torch.uint8, device="cuda")
        self.prompt_ws = None
        if prompts:
            need = L.fp4_prompt_attention_workspace_size(max_batch, max_tokens, max_tokens, q_heads, c.kv_heads, c.head_dim)
            self.prompt_ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def _project(self, x):
        """The queries, keys and values of x, slices of one buffer."""
        T, hq, hkv, d = x.shape[0], self.q_heads, self.kv_heads, self.head_dim
        qkv = self.qkv(x, self.projected[:T], self.linear_ws)
        return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))

    def step(self, x, positions, slots, block_table, context_lens, q_offsets, tree_mask=None):
        """x: bf16 [tokens, hidden]; positions: int32 [tokens]; slots: int64
        [tokens]; block_table: int32 [batch, pages]; context_lens: int32 [batch];
        q_offsets: int32 [batch + 1]; tree_mask: int32 [tokens, max_draft / 32,
        rounded up] or None.
        Returns bf16 [tokens, hidden], a view of a buffer that the next step reuses.
        More than max_draft tokens of one sequence are an error: where the sum over
        the sequences shows it, a ValueError, otherwise NaN in the rows past the bound."""
        T = x.shape[0]
        if T > self.max_tokens or block_table.shape[0] > self.max_batch:
            raise ValueError("more tokens or sequences than the block was made for")
        if T > block_table.shape[0] * self.max_draft:
            raise ValueError("more tokens than max_draft for each sequence")
        q, k, v = self._project(x)
        if self.q_norm is None:
            L.fp4_rope(q, q, positions, self.rope)
            L.fp4_kv_append(self.cache, k, v, slots, rope=self.rope, positions=positions)
        else:
            L.fp4_qk_norm_rope(q, k, q, k, self.q_norm, self.k_norm, self.norm_eps, positions, self.rope)
            L.fp4_kv_append(self.cache, k, v, slots)
        a = self.attended[:T]
        L.fp4_kv_attention(self.cache, q, a.unflatten(1, (self.q_heads, self.head_dim)), block_table, context_lens, q_offsets,
                           self.max_seq_len, self.max_draft, self.attention_ws, tree_mask=tree_mask)
        return self.o(a, self.out[:T], self.linear_ws)

    def prompt(self, x, positions, slots, q_offsets):
        """Whole prompts, packed: x: bf16 [tokens, hidden]; positions: int32 [tokens];
        slots: int64 [tokens]; q_offsets: int32 [batch + 1], ascending from 0 to tokens.
        Every token sees its sequence up to itself.  The keys are rotated (and normed)
        to bf16, attended as such, and quantized into the cache from there.
        Returns bf16 [tokens, hidden], a view of a buffer that the next call reuses."""
        T = x.shape[0]
        if self.prompt_ws is None:
            raise ValueError("the block was not made for prompts")
        if T > self.max_tokens or q_offsets.numel() - 1 > self.max_batch:
            raise ValueError("more tokens or sequences than the block was made for")
        q, k, v = self._project(x)
        if self.q_norm is None:
            L.fp4_rope(q, q, positions, self.rope)
            L.fp4_rope(k, k, positions, self.rope)
        else:
            L.fp4_qk_norm_rope(q, k, q, k, self.q_norm, self.k_norm, self.norm_eps, positions, self.rope)
        L.fp4_kv_append(self.cache, k, v, slots)
        a = self.attended[:T]
        L.fp4_prompt_attention(q, k, v, a.unflatten(1, (self.q_heads, self.head_dim)), q_offsets, None, self.prompt_ws)
        return self.o(a, self.out[:T], self.linear_ws)
