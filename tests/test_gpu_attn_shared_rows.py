"""biloco_attn_shared where test_gpu_attn_shared.py does not look: how exact the weights
of shared tokens are, batches of many sequences, lists out of order among them, and odd numbers of heads
and rows, and rows of one tile that see far-apart tokens or none.

Tolerance of the weights.  With e, t and the output's rounding as there, a weight is within 2^-16 of
itself (two bf16 terms, each rounded to 8 significant bits: 2^-8 of 2^-8).  Over n tokens
the products take n / 16 steps of two terms (each at most one truncation to 24 bits, 2^-23:
n / 4 times 2^-24), a lane's sum of weights n / 2 roundings of 2^-24, the joins under 64:
  |o - o64| <= E sum w |v| + 2^-8 (|o64| + E sum w |v|),  E = 2^-16 + e + (3 n / 4 + 64) 2^-24.
Values are chosen so that o64 nearly cancels: there the output's rounding is small
against sum w |v| and E is what is seen.  One term alone, put into the plain form,
has to exceed the bound.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import layer
from test_gpu_attn_shared import Case

pytestmark = pytest.mark.gpu


def _cancel(c, seed):
    """Gives each channel of a group and key/value head two shared tokens whose weighted
    values nearly cancel in one of the group's rows; the others, own ones too, are zero."""
    rng = np.random.default_rng(seed)
    kval, _ = layer.cache_values(c.cache)
    q, G = c.q.double().numpy(), c.hq // c.hk
    c.cache[1][:] = 0
    c.cache[3][:] = 120
    for g0, g1, n in zip(c.group_start[:-1], c.group_start[1:], c.shared):
        for h in range(c.hk):
            for d in range(c.dim):
                b, g = rng.integers(g0, g1), rng.integers(G)
                i = rng.integers(c.new[b])
                at = c.seen[b, :min(n, c.kv_len[b] - c.new[b] + i + 1)]
                s = kval[at // c.page, h, at % c.page] @ q[c.q_start[b] + i, h * G + g] * c.scale
                first = rng.choice(np.argsort(-s)[:max(2, len(s) // 2)])
                other = np.argsort(np.abs(s - s[first]))[1]
                v = rng.uniform(60, 120)
                for j, x in ((first, v), (other, -v * np.exp(s[first] - s[other]))):
                    c.cache[1][at[j] // c.page, h, at[j] % c.page // 8, d, at[j] % 8] = layer.e4m3_encode(np.clip(x, -448, 448))


def _one_term(c):
    """The plain form with weights of a single bf16 term."""
    exp = np.exp
    try:
        np.exp = lambda x: torch.from_numpy(exp(x)).to(torch.bfloat16).double().numpy()
        return c.want(0, 0)[0]
    finally:
        np.exp = exp


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("groups,hq,hk", [
    ([(200, [(1, 201), (1, 230), (2, 300)])], 2, 2),
    ([(513, [(1, 514 + i) for i in range(40)])], 8, 1),      # more rows than a tile's
    ([(640, [(1, 700), (3, 650)]), (64, [(1, 65)] * 3), (130, [(5, 140), (1, 131)])], 16, 2),
    ([(1500, [(1, 1501), (4, 1600)])], 4, 2),      # in pieces
    # sequences of many rows, which share nothing, alone and among others, in pieces
    ([(300, [(40, 400)])], 4, 2), ([(128, [(1, 140), (30, 260), (2, 150)])], 8, 1), ([(1408, [(33, 1500), (34, 1450)])], 4, 2)])
def test_weights_of_shared_tokens(dim, groups, hq, hk):
    c = Case(groups, hq, hk, dim, 32, seed=dim + hq)
    for g, n in enumerate(c.shared):
        c.table[c.group_start[g]:c.group_start[g + 1], :n // 32] = c.table[c.group_start[g], :n // 32]
    _cancel(c, seed=3)
    want, _, size, terms = c.want(0, 0)
    e = 2 * (dim + 8) * 2.0 ** -24 * terms[..., None] + 2.0 ** -20 + 2.0 ** -16
    e = e + (3 * int(c.kv_len.max()) / 4 + 64) * 2.0 ** -24
    bound = e * size + 2.0 ** -8 * (np.abs(want) + e * size)
    assert (np.abs(_one_term(c) - want) > 2 * bound).any()
    o, _ = c.run()
    over = np.abs(o.double().cpu().numpy() - want) - bound
    assert over.max() <= 0, over.max()


def test_lists_out_of_order_that_claim_more_rows_than_32_bits_count():
    """Every second sequence claims all T rows: unspecified values, no access outside the
    arrays, in 2^31 rows of heads and more; a batch that is in order is right again after it."""
    n, T, G, dim = 4096, 17000, 64, 64
    assert np.int64(n // 2 * T * G).astype(np.int32) < 0
    cache = B.biloco_kv_cache(40, 1, 32, dim)
    for t in cache:
        t.fill_(0x38)
    q = torch.randn((T, G, dim), device="cuda").to(torch.bfloat16)
    table = (torch.arange(n * 8, device="cuda", dtype=torch.int32) % 40).reshape(n, 8)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    kv_len, out = torch.full((n,), 200, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    for start in ([0, T] * (n // 2) + [0], [T, 0] * (n // 2) + [T]):
        for groups, lens in ((ints(0, n), ints(128)), (ints(0, n // 3, n), ints(64, 150))):
            B.biloco_attn_shared(cache, q, ints(*start), kv_len, table, groups, lens, 1, 200, 150, 0.125, out=out)
            torch.cuda.synchronize()
    Case([(100, [(1, 140), (1, 101)]), (64, [(1, 70)])], 8, 2, dim, 32, seed=1).check()


def test_more_sequences_and_groups_than_the_table_takes_at_a_time():
    rng = np.random.default_rng(0)
    Case([(int(rng.integers(0, 40)), [(1, int(rng.integers(1, 60)))] * int(rng.integers(0, 4))) for _ in range(1300)], 2, 1, 64, 16,
         seed=5).check()
    Case([(70, [(int(rng.integers(0, 3)), 80) for _ in range(2100)]), (20, [(1, 30)] * 50)], 2, 1, 64, 16, seed=6).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hk,groups", [(1, 1, [(200, [(1, 201)])]), (5, 1, [(130, [(1, 140), (1, 131), (1, 300)])]),
                                          (9, 3, [(700, [(1, 701)] * 4 + [(3, 720)])]), (63, 1, [(90, [(1, 91)])])])
def test_odd_numbers_of_heads_and_rows(dim, hq, hk, groups):
    Case(groups, hq, hk, dim, 32, seed=hq).check()


def _forget(c, window, sinks):
    """Shared pages of which no row sees a token hold NaN codes and scales without a value,
    and every other one of them is named no more."""
    seen = [set() for _ in c.shared]
    group = np.repeat(np.arange(len(c.shared)), np.diff(c.group_start))
    for b, n in enumerate(c.new):
        for p in range(c.kv_len[b] - n, c.kv_len[b]):
            lo = max(0, p - window + 1)
            if p >= 0:
                seen[group[b]].update(j // c.page for j in list(range(min(sinks, lo))) + list(range(lo, p + 1)))
    k, v, ks, vs = c.cache
    forgotten = 0
    for g, n in enumerate(c.shared):
        for i in set(range(n // c.page)) - seen[g]:
            at = c.table[c.group_start[g], i]
            k[at], v[at], ks[at], vs[at] = 0x7F, 0xFF, 255, 255
            if i % 2:
                c.table[c.group_start[g], i] = -1
            forgotten += 1
    return forgotten


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 4), (100, 70), (30, 0), (1, 0)])
@pytest.mark.parametrize("groups", [
    [(640, [(1, 700), (1, 0), (2, 100), (1, 660)])],      # an idle slot, one that ends among the shared tokens
    [(640, [(1, 0), (1, 641)]), (256, [(3, 2), (1, 300), (1, 120)])],
    [(1280, [(1, 1281 + 3 * i if i % 5 else 40 * i) for i in range(30)])],      # several tiles
    [(512, [(1, 2000), (1, 0)]), (512, [(1, 520), (1, 2000), (1, 300)])]])      # windows past the shared tokens
def test_what_no_row_sees_of_the_shared_tokens_may_hold_anything(dim, window, sinks, groups):
    c = Case(groups, 8, 1, dim, 32, seed=window + sinks)
    assert _forget(c, window, sinks) > 0
    c.check(window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
def test_idle_slots_among_answers(dim):
    """Rows that see nothing, in every tile and wave, without a window and with one."""
    c = Case([(700, [(1, 0 if i % 3 == 1 else 705 + i) for i in range(40)]), (300, [(2, 0)] * 9), (64, [(1, 65)])], 8, 1, dim, 16, seed=2)
    for window, sinks in ((0, 0), (128, 0), (128, 9)):
        o, lse = c.check(window, sinks)
        assert not o[1::3][:13].any() and np.isneginf(lse[1::3][:13]).all()
