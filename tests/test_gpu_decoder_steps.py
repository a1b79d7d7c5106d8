"""The attention block's steps of every size in the workspace that the block
allocates: 9 to 32 new tokens of one or a few sequences, whose rows go to the
kernel for many rows.

Tolerance of the attention: that of test_gpu_attn.py, on the block's own q and cache.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from bit_weight_gemm_amd import workloads as wl
from bit_weight_gemm_amd.decoder import AttentionBlock, Linear

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, PAGE = 16, 2, 64, 64
WIDTH = HEADS * DIM


def _linear(N, K, r, seed):
    d = wl.make_inputs(1, K, N, r, seed, g=0.003)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return Linear(dev(d["wcodes_packed"]), dev(d["wscales"]), float(d["g"]), B.biloco_pack_signs(dev(d["V"].T)),
                  B.biloco_pack_signs(dev(d["U"].T)), dev(d["alpha"].view(np.int16)), N, K, r)


def _block(max_sequences, max_kv_len, pages):
    cache = B.biloco_kv_cache(pages, KV, PAGE, DIM)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in cache[:2]:      # E4M3 codes up to 2 in magnitude, either sign
        t.copy_(torch.randint(0, 0x41, t.shape, generator=g, device="cuda", dtype=torch.uint8)
                + 128 * torch.randint(0, 2, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in cache[2:]:
        t.fill_(127)
    ones = torch.ones(WIDTH, dtype=torch.bfloat16, device="cuda")
    angle = torch.arange(max_kv_len, device="cuda", dtype=torch.float64)[:, None] / torch.arange(
        1, DIM // 2 + 1, device="cuda", dtype=torch.float64)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    return AttentionBlock(_linear((HEADS + 2 * KV) * DIM, WIDTH, 16, 1), _linear(WIDTH, WIDTH, 16, 2), HEADS, KV, DIM,
                          cache, cos_sin, ones, ones, max_sequences=max_sequences, max_kv_len=max_kv_len)


def _values(block, table, n):
    """(k, v) of a sequence's first n tokens, fp64 [heads][n][dim]."""
    kc, vc, ks, vs = (t[table[:-(-n // PAGE)].long()] for t in block.cache)
    k = kc.view(torch.float8_e4m3fn).double() * torch.exp2(ks.double() - 127)[..., None, None]
    v = vc.view(torch.float8_e4m3fn).double().transpose(3, 4).flatten(2, 3) * torch.exp2(vs.double() - 127)[..., None, None]
    return k.transpose(0, 1).flatten(1, 2)[:, :n], v.transpose(0, 1).flatten(1, 2)[:, :n]


@pytest.mark.parametrize("new,past", [([16], [3000]), ([13], [700]), ([9], [130]), ([32], [1000]), ([1], [5]),
                                      ([10, 6], [900, 3]), ([15, 0, 1], [500, 20, 64]), ([2, 30], [2000, 0])])
def test_steps_behind_a_context_far_below_the_bound(new, past):
    n, T = len(new), sum(new)
    max_kv = 131072      # the block's bound on lengths
    per = -(-(max(past) + 32) // PAGE)
    block = _block(n, max_kv, n * per)
    table = torch.randperm(n * per, generator=torch.Generator().manual_seed(1)).to(torch.int32).reshape(n, per).cuda()
    lens = [a + b for a, b in zip(past, new)]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pos = np.concatenate([np.arange(a, a + b) for a, b in zip(past, new)]).astype(np.int32)[None]
    x = torch.randn((T, WIDTH), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    codes, scales = B.biloco_quant_act_fp4(x)
    h, _, _ = block.step(x, codes, scales, x.clone(), torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), table, max(new))
    torch.cuda.synchronize()
    assert bool(torch.isfinite(h.float()).all())
    G = HEADS // KV
    for b in range(n):
        k, v = _values(block, table[b], lens[b])
        hidden = torch.arange(lens[b], device="cuda") > torch.arange(past[b], lens[b], device="cuda")[:, None]
        for a in range(HEADS if new[b] else 0):
            q = block._q[start[b]:start[b + 1], a].double()
            s = (q @ k[a // G].T.contiguous() * DIM ** -0.5).masked_fill(hidden, -torch.inf)
            w = torch.softmax(s, 1)
            want, size = w @ v[a // G], w @ v[a // G].abs()
            terms = (q.abs() @ k[a // G].abs().T.contiguous() * DIM ** -0.5).amax(1, keepdim=True)
            e = 2 * (DIM + 8) * 2.0 ** -24 * terms + 2.0 ** -20
            got = block._o[start[b]:start[b + 1], a].double()
            assert bool(((got - want).abs() <= (2.0 ** -8 + e) * size + 2.0 ** -8 * want.abs()).all()), (b, a)


def test_more_sequences_than_the_block_has_workspace_for():
    block = _block(1, 1000, 4)
    x = torch.zeros((2, WIDTH), dtype=torch.bfloat16, device="cuda")
    codes, scales = B.biloco_quant_act_fp4(x)
    before = [t.clone() for t in block.cache]
    i32 = torch.zeros((2,), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="sequences"):
        block.step(x, codes, scales, x.clone(), i32[None], torch.arange(3, dtype=torch.int32, device="cuda"), i32 + 1,
                   torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2), 1)
    torch.cuda.synchronize()
    for t, u in zip(block.cache, before):
        assert torch.equal(t, u)
