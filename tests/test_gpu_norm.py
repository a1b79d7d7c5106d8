"""biloco_norm_gate_residual against the 64-bit formula.

Tolerances.  A row's sum of C squares in fp32 is off by at most
(C / lanes + 2 log2 lanes) roundings of 2^-24, less than 2^-17 of itself for
C <= 32768 over at least 64 lanes, and rsqrt halves that; the other operations
are a handful of roundings.  So n and h are off by 2^-16 relative, r' by
2^-16 (|res| + |res_scale gate n|), before the last rounding: 2^-8 relative for
bf16, 2^-24 for fp32.  h's own error also has r''s share of each element: it is
bounded with |r'| replaced by |res| + |res_scale gate n|.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import layer

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


def _f(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _inputs(T, C, res_dtype, gate, post, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16, scale=1.0, mean=0.0):
        x = torch.zeros(shape[:-1] + (shape[-1] + pad,), dtype=dtype, device="cuda")[..., :shape[-1]]
        x.copy_((torch.randn(shape, generator=g) * scale + mean).to(dtype))
        return x

    x, res = rand(T, C, scale=0.7), rand(T, C, dtype=res_dtype, scale=3.0)
    w = [(torch.randn(C, generator=g) * 0.2 + 1).to(torch.bfloat16).cuda() for _ in range(2)]
    gt = None if gate is None else rand(1 if gate == "row" else T, C, scale=0.5, mean=0.3)
    return x, res, w[0], w[1] if post else None, gt


def _check(T, C, res_dtype=torch.bfloat16, gate=None, post=True, scale=1.0, offset=0.0, pad=0, eps=1e-6,
           inplace=False, codes=False):
    x, res, pre_w, post_w, gt = _inputs(T, C, res_dtype, gate, post, seed=T * 31 + C, pad=pad)
    want_r, want_h, mag = layer.norm_gate_residual(_f(x), _f(res), _f(pre_w), _f(post_w), _f(gt), scale, eps, offset)
    kw = {}
    if codes:
        kw = dict(a_codes=torch.full((T, C // 2), 0x5A, dtype=torch.uint8, device="cuda"),
                  a_scales=torch.full((T, C // 16), 0x33, dtype=torch.uint8, device="cuda"))
    h = torch.full((T, C + pad), 7.0, dtype=torch.bfloat16, device="cuda")[:, :C]
    out = res if inplace else torch.full((T, C + pad), 7.0, dtype=res_dtype, device="cuda")[:, :C]
    r, h = B.biloco_norm_gate_residual(x, res, pre_w, post_w=post_w, gate=gt, res_scale=scale, eps=eps,
                                       w_offset=offset, res_out=out, h=h, **kw)
    torch.cuda.synchronize()
    last = 2.0 ** -8 if res_dtype is torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(_f(r) - want_r) <= REL * mag + last * np.abs(want_r) * (1 + REL))
    w = np.abs(offset + _f(pre_w))
    inv = 1 / np.sqrt((want_r ** 2).mean(1, keepdims=True) + eps)
    assert np.all(np.abs(_f(h) - want_h) <= 2 * REL * mag * inv * w + 2.0 ** -8 * np.abs(want_h) * (1 + REL) + 1e-38)
    if pad:
        for t in (h, r):
            if t is not res:
                whole = t.as_strided((T, C + pad), (C + pad, 1))
                assert bool((whole[:, C:] == 7.0).all())
    if codes:
        c, s = B.biloco_quant_act_fp4(h.contiguous())
        torch.cuda.synchronize()
        assert torch.equal(c, kw["a_codes"]) and torch.equal(s, kw["a_scales"])


@pytest.mark.parametrize("T,C", [(1, 1), (3, 7), (2, 8), (1, 64), (5, 100), (2, 512), (4, 520), (33, 1024), (2, 1030),
                                 (7, 2880), (32, 5120), (2, 8192), (3, 13824), (2, 16384), (1, 16391), (1, 32768),
                                 (1, 32765)])
def test_widths(T, C):
    _check(T, C)


@pytest.mark.parametrize("C", [8, 500, 1000, 2048, 4096, 8192, 16384, 24576])
def test_many_rows(C):
    _check(600, C, gate="token", scale=0.3)


@pytest.mark.parametrize("res_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "row", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("C", [96, 333, 5120])
def test_forms(res_dtype, gate, post, C):
    _check(9, C, res_dtype, gate, post, scale=0.22, offset=1.0)


@pytest.mark.parametrize("pad", [8, 24, 3])
@pytest.mark.parametrize("C", [64, 1025, 5120])
def test_strided_rows(pad, C):
    _check(6, C, torch.float32, "token", pad=pad)
    _check(6, C, torch.bfloat16, "row", pad=pad)


@pytest.mark.parametrize("res_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [72, 71, 8192])
def test_in_place(res_dtype, C):
    _check(40, C, res_dtype, "token", inplace=True)


@pytest.mark.parametrize("T,C,pad", [(1, 32, 0), (32, 5120, 0), (3, 13824, 0), (700, 8192, 0), (2, 32768, 0),
                                     (4, 96, 3), (2, 5120, 1), (2, 16416, 5)])
def test_codes_are_those_of_h(T, C, pad):
    _check(T, C, codes=True, gate="row", pad=pad)


def test_zero_rows():
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    r, h = B.biloco_norm_gate_residual(x, x.clone(), w, post_w=w, eps=1e-6)
    assert bool((r == 0).all()) and bool((h == 0).all())
    r, h = B.biloco_norm_gate_residual(x[:0], x[:0], w)
    assert r.shape == (0, 256)


def test_another_stream_and_replay():
    x, res, pre_w, post_w, gt = _inputs(16, 5120, torch.bfloat16, "token", True)
    r0, h0 = B.biloco_norm_gate_residual(x, res, pre_w, post_w=post_w, gate=gt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r, h = torch.empty_like(res), torch.empty_like(x)
    with torch.cuda.stream(s):
        B.biloco_norm_gate_residual(x, res, pre_w, post_w=post_w, gate=gt, res_out=r, h=h)
    s.synchronize()
    assert torch.equal(r, r0) and torch.equal(h, h0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_norm_gate_residual(x, res, pre_w, post_w=post_w, gate=gt, res_out=r, h=h)
    for _ in range(3):
        r.zero_(), h.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, r0) and torch.equal(h, h0)
