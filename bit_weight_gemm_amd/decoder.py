"""The attention block of one decoder layer, on the library's entry points.

A step takes the residual stream's rows of a ragged batch (at most 32 new tokens
in all, the product's limit) and runs, in this order:

  QKV product     biloco_gemm_lowrank on the norm's h and its FP4 codes
  cache append    biloco_kv_append: rotation, quantisation, paged append
  attention       biloco_attn_paged over the 8-bit cache
  O product       biloco_gemm_lowrank_quant (quantises the attention's rows)
  norms           biloco_norm_gate_residual: the norm after the block, its
                  residual scale, the norm before the next block and that h's
                  FP4 codes, which the next product takes as they are

No arithmetic happens here.  Buffers are allocated once for the largest step
and every call is on the current stream, so a step can be captured in a graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


@dataclass
class Linear:
    """Operands of one product (include/biloco.h): y [M][N] = x [M][K] W^T."""
    w_codes: torch.Tensor
    w_scales: torch.Tensor
    g: float
    v_packed: torch.Tensor
    u_packed: torch.Tensor
    alpha: torch.Tensor
    N: int
    K: int
    r: int

    def workspace(self, M: int, device) -> torch.Tensor:
        """Zero-filled, for products of up to M rows."""
        n = max(B.biloco_gemm_workspace_bytes(m, self.N, self.K, self.r) for m in range(1, M + 1))
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


class AttentionBlock:
    MAX_TOKENS = 32

    def __init__(self, qkv: Linear, out: Linear, heads: int, kv_heads: int, head_dim: int, cache: tuple,
                 cos_sin: torch.Tensor, post_w: torch.Tensor, next_w: torch.Tensor, *, max_sequences: int,
                 max_kv_len: int, res_scale: float = 1.0, window: int = 0, sinks: int = 0, eps: float = 1e-6,
                 device="cuda"):
        self.width = qkv.K
        if qkv.N != (heads + 2 * kv_heads) * head_dim or out.K != heads * head_dim or out.N != self.width:
            raise ValueError("the products' sizes do not fit the heads")
        self.qkv, self.out, self.heads, self.kv_heads, self.dim = qkv, out, heads, kv_heads, head_dim
        self.cache, self.cos_sin, self.post_w, self.next_w = cache, cos_sin, post_w, next_w
        self.max_sequences, self.max_kv_len, self.res_scale, self.window, self.sinks, self.eps = (
            max_sequences, max_kv_len, res_scale, window, sinks, eps)
        M = self.MAX_TOKENS

        def rows(*shape, dtype=torch.bfloat16):
            return torch.empty((M,) + shape, dtype=dtype, device=device)

        self._qkv, self._q, self._o = rows(qkv.N), rows(heads, head_dim), rows(heads, head_dim)
        self._proj, self._h = rows(self.width), rows(self.width)
        self._o_codes = rows(out.K // 2, dtype=torch.uint8)
        self._o_scales = rows(out.K // 16, dtype=torch.uint8)
        self._codes = rows(self.width // 2, dtype=torch.uint8)
        self._scales = rows(self.width // 16, dtype=torch.uint8)
        self._qkv_ws, self._out_ws = qkv.workspace(M, device), out.workspace(M, device)
        # that of the largest step covers every smaller one
        need = B.biloco_attn_workspace_bytes(max_sequences, M, heads, kv_heads, head_dim, M, max_kv_len)
        self._attn_ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)

    def step(self, h, codes, scales, res, positions, q_start, kv_len, block_table, max_q_len: int):
        """h [T][width] bf16 with its FP4 codes and scales, res [T][width]
        (updated in place) -> (h, codes, scales) of the next block."""
        T, heads, kv, d = h.shape[0], self.heads, self.kv_heads, self.dim
        if T > self.MAX_TOKENS:
            raise ValueError(f"at most {self.MAX_TOKENS} new tokens a step")
        if kv_len.shape[0] > self.max_sequences:      # before the cache changes
            raise ValueError(f"at most {self.max_sequences} sequences a step")
        if T == 0:
            return self._h[:0], self._codes[:0], self._scales[:0]
        a, o = self.qkv, self.out
        y = self._qkv[:T]
        B.biloco_gemm_lowrank(codes, scales, h, a.w_codes, a.w_scales, a.g, a.v_packed, a.u_packed, a.alpha, T, a.N,
                              a.K, a.r, y, self._qkv_ws, self._qkv_ws.numel())
        q = y[:, :heads * d].unflatten(1, (heads, d))
        k = y[:, heads * d:(heads + kv) * d].unflatten(1, (kv, d))
        v = y[:, (heads + kv) * d:].unflatten(1, (kv, d))
        q = B.biloco_kv_append(self.cache, q, k, v, positions, self.cos_sin, q_start, kv_len, block_table, max_q_len,
                               q_out=self._q[:T])
        att = B.biloco_attn_paged(self.cache, q, q_start, kv_len, block_table, max_q_len, self.max_kv_len, d ** -0.5,
                                  window=self.window, sinks=self.sinks, out=self._o[:T], workspace=self._attn_ws)
        B.biloco_gemm_lowrank_quant(att, self._o_codes, self._o_scales, o.w_codes, o.w_scales, o.g, o.v_packed,
                                    o.u_packed, o.alpha, T, o.N, o.K, o.r, self._proj, self._out_ws,
                                    self._out_ws.numel())
        next_codes, next_scales = self._codes[:T], self._scales[:T]
        _, next_h = B.biloco_norm_gate_residual(self._proj[:T], res, self.next_w, post_w=self.post_w,
                                                res_scale=self.res_scale, eps=self.eps, res_out=res, h=self._h[:T],
                                                a_codes=next_codes, a_scales=next_scales)
        return next_h, next_codes, next_scales
