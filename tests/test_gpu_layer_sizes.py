"""Decoder-layer calls of more rows than one launch's threads can count are refused, and
write nothing."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,C", [((1 << 26) + 5, 8), ((1 << 24) + 5, 3)])
def test_norm(T, C):
    x = torch.ones((T, C), dtype=torch.bfloat16, device="cuda")
    out, h = (torch.full((T, C), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.ones((C,), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.BilocoError):
        B.biloco_norm_gate_residual(x, x, w, res_out=out, h=h)
    torch.cuda.synchronize()
    assert bool((out == 5).all()) and bool((h == 5).all())
    few = T // 8
    B.biloco_norm_gate_residual(x[:few], x[:few], w, res_out=out[:few], h=h[:few])
    assert bool((out[:few] == 2).all()) and bool((h[:few] == 1).all())
    assert bool((out[few:] == 5).all()) and bool((h[few:] == 5).all())
