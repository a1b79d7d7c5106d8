"""The attention block's empty steps, the example's refusals (no GPU)."""
import os
import runpy
import sys

import pytest
import torch

from bit_weight_gemm_amd.decoder import AttentionBlock, Linear

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
