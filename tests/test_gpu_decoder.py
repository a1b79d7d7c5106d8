"""The attention block of bit_weight_gemm_amd/decoder.py: the operators
together, stage by stage against the 64-bit forms.

Each stage is checked on the values that the stage before it really gave it
(read back from the block's buffers), with that stage's own tolerance, so no
error is carried from one to the next.  Prompts taken up in several steps, decode
steps of one token, a sequence that rests, window and sinks.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_weight_gemm_amd import binding as B
from bit_weight_gemm_amd import workloads as wl
from bit_weight_gemm_amd.decoder import AttentionBlock, Linear
from oracle import layer
from util import check_y

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, PAGE = 4, 2, 64, 16
WIDTH = HEADS * DIM


def _linear(N, K, r, seed):
    d = wl.make_inputs(1, K, N, r, seed, g=0.003)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return d, Linear(dev(d["wcodes_packed"]), dev(d["wscales"]), float(d["g"]), B.biloco_pack_signs(dev(d["V"].T)),
                     B.biloco_pack_signs(dev(d["U"].T)), dev(d["alpha"].view(np.int16)), N, K, r)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _product(d, x):
    return oracle.gemm_lowrank(_bits(x), d["wcode"], d["wscales"], d["g"], d["V"], d["U"], d["alpha"])


@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_block_stage_by_stage(window, sinks):
    rng = np.random.default_rng(3)
    dq, qkv = _linear((HEADS + 2 * KV) * DIM, WIDTH, 16, 1)
    do, out = _linear(WIDTH, HEADS * DIM, 16, 2)
    table = rng.permutation(12).astype(np.int32).reshape(3, 4)
    cache = tuple(torch.full_like(t, 0x7F) for t in B.biloco_kv_cache(12, KV, PAGE, DIM))
    ang = np.arange(64)[:, None] * 50.0 ** (-np.arange(DIM // 2) / (DIM // 2))
    cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = [torch.from_numpy(rng.normal(1, 0.1, WIDTH).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2)]
    block = AttentionBlock(qkv, out, HEADS, KV, DIM, cache, torch.from_numpy(cos_sin).cuda(), w[0], w[1],
                           max_sequences=3, max_kv_len=64, res_scale=0.7, window=window, sinks=sinks)
    lens = np.zeros(3, np.int32)
    for new in ([20, 0, 5], [0, 32, 0], [1, 1, 1], [3, 4, 0], [1, 0, 1], [1, 1, 1]):
        T = sum(new)
        print("new tokens", new, flush=True)
        pos = np.concatenate([np.arange(n, n + k) for n, k in zip(lens, new)]).astype(np.int32)[None]
        lens = (lens + new).astype(np.int32)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x = torch.from_numpy(rng.standard_normal((T, WIDTH)).astype(np.float32)).to(torch.bfloat16).cuda()
        codes, scales = B.biloco_quant_act_fp4(x)
        res = x.clone()
        before = tuple(c.cpu().numpy() for c in cache)
        h, hc, hs = block.step(x, codes, scales, res, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(),
                               torch.from_numpy(lens).cuda(), torch.from_numpy(table).cuda(), max(new))
        torch.cuda.synchronize()
        y = block._qkv[:T]
        check_y(y.double().cpu().numpy(), _product(dq, x), "qkv")
        rows = y.float().cpu().numpy()
        q = rows[:, :WIDTH].reshape(T, HEADS, DIM)
        k = rows[:, WIDTH:WIDTH + KV * DIM].reshape(T, KV, DIM)
        v = rows[:, WIDTH + KV * DIM:].reshape(T, KV, DIM)
        axis = np.zeros(DIM // 2, np.uint8)
        q = layer.rotate(q, pos, cos_sin, axis, False, np.float32)
        np.testing.assert_array_equal(block._q[:T].float().cpu().numpy(),
                                      torch.from_numpy(q).to(torch.bfloat16).float().numpy())
        want = layer.append(before, layer.rotate(k, pos, cos_sin, axis, False, np.float32), v, start, lens, table)
        for got, ref in zip(cache, want):
            np.testing.assert_array_equal(got.cpu().numpy() & 127, ref & 127)
        o, _, mag, terms = layer.attend(want, block._q[:T].double().cpu().numpy(), start, lens, table, DIM ** -0.5,
                                        window, sinks)
        e = 2 * (DIM + 8) * 2.0 ** -24 * terms[..., None] + 2.0 ** -20
        got = block._o[:T].double().cpu().numpy()
        assert np.all(np.abs(got - o) <= (2.0 ** -8 + e) * mag + 2.0 ** -8 * np.abs(o))
        att = block._o[:T].reshape(T, HEADS * DIM)
        check_y(block._proj[:T].double().cpu().numpy(), _product(do, att), "out")
        r64, h64, size = layer.norm_gate_residual(block._proj[:T].double().cpu().numpy(), x.double().cpu().numpy(),
                                                  w[1].double().cpu().numpy(), w[0].double().cpu().numpy(),
                                                  res_scale=0.7)
        assert np.all(np.abs(res.double().cpu().numpy() - r64) <= 2.0 ** -16 * size + 2.0 ** -8 * np.abs(r64) * 1.001)
        inv = 1 / np.sqrt((r64 ** 2).mean(1, keepdims=True) + 1e-6)
        bound = 2.0 ** -15 * size * inv * np.abs(w[1].double().cpu().numpy()) + 2.0 ** -8 * np.abs(h64) * 1.001
        assert np.all(np.abs(h.double().cpu().numpy() - h64) <= bound)
        c, s = oracle.quant_act_fp4(_bits(h))
        np.testing.assert_array_equal(hc.cpu().numpy(), c)
        np.testing.assert_array_equal(hs.cpu().numpy(), s)


def test_block_replays_from_a_graph():
    _, qkv = _linear((HEADS + 2 * KV) * DIM, WIDTH, 16, 1)
    _, out = _linear(WIDTH, HEADS * DIM, 16, 2)
    cache = tuple(torch.full_like(t, 0x30) for t in B.biloco_kv_cache(8, KV, PAGE, DIM))
    for t in cache[2:]:
        t.fill_(120)
    ones = torch.ones(WIDTH, dtype=torch.bfloat16, device="cuda")
    cos_sin = torch.ones((64, DIM), device="cuda") * 0.7
    block = AttentionBlock(qkv, out, HEADS, KV, DIM, cache, cos_sin, ones, ones, max_sequences=2, max_kv_len=64)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, WIDTH), generator=g, device="cuda").to(torch.bfloat16)
    codes, scales = B.biloco_quant_act_fp4(x)
    pos = torch.tensor([[17, 30]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([18, 31], dtype=torch.int32, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 4)
    first = tuple(t.clone() for t in cache)

    def step(res):
        for t, c in zip(cache, first):
            t.copy_(c)
        return block.step(x, codes, scales, res, pos, start, lens, table, 1)
    res0 = x.clone()
    h0 = step(res0)[0].clone()
    torch.cuda.synchronize()
    res = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res.copy_(x)
        step(res)
    for _ in range(3):
        block._h.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(block._h[:2], h0) and torch.equal(res, res0)


def test_block_refuses():
    _, qkv = _linear((HEADS + 2 * KV) * DIM, WIDTH, 16, 1)
    _, out = _linear(WIDTH, HEADS * DIM, 16, 2)
    cache = B.biloco_kv_cache(8, KV, PAGE, DIM)
    ones = torch.ones(WIDTH, dtype=torch.bfloat16, device="cuda")
    cos_sin = torch.ones((64, DIM), device="cuda")
    with pytest.raises(ValueError):
        AttentionBlock(qkv, out, HEADS, KV + 1, DIM, cache, cos_sin, ones, ones, max_sequences=2, max_kv_len=64)
    block = AttentionBlock(qkv, out, HEADS, KV, DIM, cache, cos_sin, ones, ones, max_sequences=2, max_kv_len=64)
    x = torch.zeros((33, WIDTH), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        block.step(x, None, None, x, None, None, None, None, 33)
