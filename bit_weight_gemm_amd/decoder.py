"""The attention block of one decoder layer, and the choice of tokens behind the last,
on the library's entry points.

A step takes the residual stream's rows of a ragged batch (at most 32 new tokens
in all, the low-rank product's limit) and runs, in this order:

  QKV product     biloco_gemm_lowrank on the norm's h and its FP4 codes
  cache append    biloco_kv_append: rotation, quantisation, paged append
  attention       biloco_attn_paged over the 8-bit cache
  O product       biloco_gemm_lowrank_quant (quantises the attention's rows)
  norms           biloco_norm_gate_residual: the norm after the block, its
                  residual scale, the norm before the next block and that h's
                  FP4 codes, which the next product takes as they are

With MxLinear products (biloco_gemm_mxfp4_quant) a step takes any number of tokens, so
that a prompt is taken in at once, and with `shared` the sequences of a group read their
first tokens once (biloco_attn_shared): several answers to one prompt.  Head turns rows
behind the last block into tokens (biloco_gemm_mxfp4_quant, biloco_sample).

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


@dataclass
class MxLinear:
    """A product whose weight is kept as microscaled 4-bit floats: y [M][N] = Q(x) [M][K] W^T."""
    codes: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def of(cls, w: torch.Tensor) -> "MxLinear":
        """w bf16 or fp32 [N][K]."""
        return cls(*B.biloco_quant_mxfp4(w))

    @property
    def N(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return 2 * self.codes.shape[1]

    def workspace(self, M: int, device) -> torch.Tensor:
        """For products of up to M rows."""
        n = B.biloco_gemm_mxfp4_workspace_bytes(M, self.N, self.K)
        return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


class AttentionBlock:
    MAX_TOKENS = 32      # of a step through a Linear

    def __init__(self, qkv: Linear | MxLinear, out: Linear | MxLinear, heads: int, kv_heads: int, head_dim: int, cache: tuple,
                 cos_sin: torch.Tensor, post_w: torch.Tensor, next_w: torch.Tensor, *, max_sequences: int,
                 max_kv_len: int, res_scale: float = 1.0, window: int = 0, sinks: int = 0, eps: float = 1e-6,
                 max_tokens: int = MAX_TOKENS, max_groups: int = 0, device="cuda"):
        """max_tokens: of a step, more than MAX_TOKENS only through MxLinear products.
        max_groups: of the steps with shared tokens (0: there are none)."""
        self.width = qkv.K
        if qkv.N != (heads + 2 * kv_heads) * head_dim or out.K != heads * head_dim or out.N != self.width:
            raise ValueError("the products' sizes do not fit the heads")
        self.qkv, self.out, self.heads, self.kv_heads, self.dim = qkv, out, heads, kv_heads, head_dim
        self.cache, self.cos_sin, self.post_w, self.next_w = cache, cos_sin, post_w, next_w
        self.max_sequences, self.max_kv_len, self.res_scale, self.window, self.sinks, self.eps = (
            max_sequences, max_kv_len, res_scale, window, sinks, eps)
        self.max_tokens, self.max_groups = max_tokens, max_groups
        if max_tokens > self.MAX_TOKENS and not (isinstance(qkv, MxLinear) and isinstance(out, MxLinear)):
            raise ValueError(f"at most {self.MAX_TOKENS} new tokens a step through a low-rank product")
        M = max_tokens

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
        if max_groups:
            need = max(need, B.biloco_attn_shared_workspace_bytes(max_sequences, M, heads, kv_heads, head_dim, M, max_kv_len,
                                                                  max_groups, max_kv_len))
        self._attn_ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)

    def step(self, h, codes, scales, res, positions, q_start, kv_len, block_table, max_q_len: int, shared=None):
        """h [T][width] bf16 with its FP4 codes and scales (unused by an MxLinear: any), res
        [T][width] (updated in place) -> (h, codes, scales) of the next block.  shared: None,
        or (group_start, shared_len) of biloco_attn_shared, shared tokens up to max_kv_len,
        for which the launch is cut."""
        T, heads, kv, d = h.shape[0], self.heads, self.kv_heads, self.dim
        if T > self.max_tokens:
            raise ValueError(f"at most {self.max_tokens} new tokens a step")
        if kv_len.shape[0] > self.max_sequences:      # before the cache changes
            raise ValueError(f"at most {self.max_sequences} sequences a step")
        if shared is not None and shared[1].shape[0] > self.max_groups:
            raise ValueError(f"at most {self.max_groups} groups a step")
        if T == 0:
            return self._h[:0], self._codes[:0], self._scales[:0]
        a, o = self.qkv, self.out
        y = self._qkv[:T]
        if isinstance(a, MxLinear):
            B.biloco_gemm_mxfp4_quant(h, a.codes, a.scales, y=y, workspace=self._qkv_ws)
        else:
            B.biloco_gemm_lowrank(codes, scales, h, a.w_codes, a.w_scales, a.g, a.v_packed, a.u_packed, a.alpha, T, a.N,
                                  a.K, a.r, y, self._qkv_ws, self._qkv_ws.numel())
        q = y[:, :heads * d].unflatten(1, (heads, d))
        k = y[:, heads * d:(heads + kv) * d].unflatten(1, (kv, d))
        v = y[:, (heads + kv) * d:].unflatten(1, (kv, d))
        q = B.biloco_kv_append(self.cache, q, k, v, positions, self.cos_sin, q_start, kv_len, block_table, max_q_len,
                               q_out=self._q[:T])
        kw = dict(window=self.window, sinks=self.sinks, out=self._o[:T], workspace=self._attn_ws)
        if shared is None:
            att = B.biloco_attn_paged(self.cache, q, q_start, kv_len, block_table, max_q_len, self.max_kv_len, d ** -0.5, **kw)
        else:
            att = B.biloco_attn_shared(self.cache, q, q_start, kv_len, block_table, *shared, max_q_len, self.max_kv_len,
                                       self.max_kv_len, d ** -0.5, **kw)
        if isinstance(o, MxLinear):
            B.biloco_gemm_mxfp4_quant(att.flatten(1), o.codes, o.scales, y=self._proj[:T], workspace=self._out_ws)
        else:
            B.biloco_gemm_lowrank_quant(att, self._o_codes, self._o_scales, o.w_codes, o.w_scales, o.g, o.v_packed,
                                        o.u_packed, o.alpha, T, o.N, o.K, o.r, self._proj, self._out_ws,
                                        self._out_ws.numel())
        next_codes, next_scales = self._codes[:T], self._scales[:T]
        _, next_h = B.biloco_norm_gate_residual(self._proj[:T], res, self.next_w, post_w=self.post_w,
                                                res_scale=self.res_scale, eps=self.eps, res_out=res, h=self._h[:T],
                                                a_codes=next_codes, a_scales=next_scales)
        return next_h, next_codes, next_scales


class Head:
    """Tokens from the rows behind the last block: their product with a weight of V rows,
    fp32 logits, and a draw from each."""

    def __init__(self, weight: MxLinear, *, max_rows: int, device="cuda"):
        self.weight, self.max_rows = weight, max_rows
        self._logits = torch.empty((max_rows, weight.N), dtype=torch.float32, device=device)
        self._token = torch.empty((max_rows,), dtype=torch.int32, device=device)
        self._ws = weight.workspace(max_rows, device)
        self._sample_ws = torch.empty(max(B.biloco_sample_workspace_bytes(max_rows, weight.N), 16), dtype=torch.uint8,
                                      device=device)

    def step(self, h, u, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None):
        """h [R][K] bf16, u fp32 [n] -> tokens int32 [n]: one of each row, or, where R is 1, n of
        that one's.  The rest as for biloco_sample."""
        R, n = h.shape[0], u.shape[0]
        if n > self.max_rows:
            raise ValueError(f"at most {self.max_rows} tokens a step")
        if R != n and R != 1:
            raise ValueError("a row a token, or one row, expected")
        if n == 0:
            return self._token[:0]
        w = self.weight
        logits = B.biloco_gemm_mxfp4_quant(h, w.codes, w.scales, y=self._logits[:R], workspace=self._ws)
        return B.biloco_sample(logits.expand(n, w.N), u, temperature, top_k, top_p, min_p, token=self._token[:n],
                               logprob=logprob, workspace=self._sample_ws)
