"""The attention block's empty steps (no GPU)."""
import torch

from bit_weight_gemm_amd.decoder import AttentionBlock, Linear


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
