"""The attention block's empty steps, the example's refusals (no GPU)."""
import os
import runpy
import sys

import pytest
import torch

from bit_weight_gemm_amd import binding as B
from bit_weight_gemm_amd.decoder import AttentionBlock, Head, Linear, MxLinear

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _block():
    def linear(N, K):
        return Linear(None, None, 1.0, None, None, None, N, K, 16)
    return AttentionBlock(linear(512, 256), linear(256, 256), 4, 2, 64, None, None, None, None, max_sequences=2,
                          max_kv_len=100, device="cpu")


def test_a_step_of_no_tokens_is_empty():
    block = _block()
    x = torch.zeros((0, 256), dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    h, codes, scales = block.step(x, x[:, :128].byte(), x[:, :16].byte(), x, i32[None, :0], i32, i32[:2], i32[:2, None], 1)
    assert (tuple(h.shape), tuple(codes.shape), tuple(scales.shape)) == ((0, 256), (0, 128), (0, 16))
    assert h.dtype == torch.bfloat16 and codes.dtype == scales.dtype == torch.uint8


@pytest.mark.parametrize("args", [["--sequences", "33"], ["--sequences", "0"], ["--steps", "0"], ["--prompt", "-5"]])
def test_example_refuses_what_a_step_cannot_take(args, monkeypatch, capsys):
    path = os.path.join(ROOT, "examples", "decode_block.py")
    monkeypatch.setattr(sys, "argv", [path] + args)
    with pytest.raises(SystemExit) as e:
        runpy.run_path(path, run_name="__main__")
    err = capsys.readouterr().err
    assert e.value.code == 2 and "usage" in err and args[0] in err.splitlines()[-1]


def _mx(N, K):
    return MxLinear(torch.zeros((N, K // 2), dtype=torch.uint8), torch.zeros((N, K // 32), dtype=torch.uint8))


def _mx_block(qkv, out, **kw):
    return AttentionBlock(qkv, out, 4, 2, 64, None, None, None, None, max_sequences=2, max_kv_len=100, device="cpu", **kw)


def test_microscaled_products_take_more_tokens():
    low = Linear(None, None, 1.0, None, None, None, 256, 256, 16)
    block = _mx_block(_mx(512, 256), _mx(256, 256), max_tokens=100)
    assert block._q.shape == (100, 4, 64) and block.qkv.N == 512 and block.qkv.K == 256
    with pytest.raises(ValueError, match="at most 32"):
        _mx_block(_mx(512, 256), low, max_tokens=33)
    x = torch.zeros((101, 256), dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="at most 100 new"):
        block.step(x, None, None, x, i32, i32, i32[:2], i32[:2, None], 1)
    with pytest.raises(ValueError, match="at most 0 groups"):
        block.step(x[:1], None, None, x[:1], i32, i32, i32[:2], i32[:2, None], 1, shared=(i32[:2], i32[:1]))
    h, _, _ = block.step(x[:0], None, None, x[:0], i32, i32, i32[:2], i32[:2, None], 1)
    assert tuple(h.shape) == (0, 256)


def test_head_refusals():
    head = Head(_mx(300, 64), max_rows=4, device="cpu")
    h, u = torch.zeros((5, 64), dtype=torch.bfloat16), torch.zeros(5)
    with pytest.raises(ValueError, match="at most 4"):
        head.step(h, u)
    with pytest.raises(ValueError, match="a row a token"):
        head.step(h[:2], u[:3])
    assert head.step(h[:0], u[:0]).shape == (0,) and head.step(h[:1], u[:0]).shape == (0,)


@pytest.mark.parametrize("heads,kv_heads,sequences,tokens,kv", [(64, 8, 8, 64, 32768), (16, 2, 33, 40, 9000), (40, 40, 3, 700, 4000)])
def test_a_block_holds_the_workspace_of_every_shared_step(heads, kv_heads, sequences, tokens, kv):
    width = heads * 64
    block = AttentionBlock(_mx((heads + 2 * kv_heads) * 64, width), _mx(width, width), heads, kv_heads, 64, None, None, None,
                           None, max_sequences=sequences, max_kv_len=kv, max_tokens=tokens, max_groups=3, device="cpu")
    for b in (1, 2, sequences):
        for t in (1, 2, 7, tokens):
            for q in {1, 2, t}:
                for g in (1, 2, 3):
                    if q <= t:
                        assert B.biloco_attn_shared_workspace_bytes(b, t, heads, kv_heads, 64, q, kv, g, kv) <= block._attn_ws.numel()
