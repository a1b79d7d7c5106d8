"""biloco_attn_paged where test_gpu_attn.py does not look: how exact the weights of
sequences of few rows are, and the order of many rows' chunks at 128 channels (whole
ones in interleaved order between masked ones, many in one piece).

Tolerance of the few rows.  With e, t and the output's rounding as in
test_gpu_attn.py, a weight is within 2^-16 of itself (two bf16 terms, each rounded to
8 significant bits: 2^-8 of 2^-8), and the sums over n tokens take at most n / 4 + 64
roundings of 2^-24 (a step of the product adds 32 tokens; eight waves are joined):
  |o - o64| <= E sum w |v| + 2^-8 (|o64| + E sum w |v|),  E = 2^-16 + e + (n / 4 + 64) 2^-24.
Values are chosen so that o64 nearly cancels: there the output's rounding is small
against sum w |v| and E is what is seen.  One term alone, put into the plain form,
has to exceed the bound.
"""
import numpy as np
import pytest
import torch

from oracle import layer
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


def _cancel(c, seed):
    """Gives each channel of a sequence and key/value head two tokens whose
    weighted values nearly cancel in one of the rows; the others are zero."""
    rng = np.random.default_rng(seed)
    kval, _ = layer.cache_values(c.cache)
    q, G = c.q.double().numpy(), c.hq // c.hk
    c.cache[1][:] = 0
    c.cache[3][:] = 120
    for b, n in enumerate(c.new):
        for h in range(c.hk if n else 0):
            for d in range(c.dim):
                i, g = rng.integers(n), rng.integers(G)
                seen = np.arange(c.kv_len[b] - n + i + 1)
                s = kval[c.table[b, seen // c.page], h, seen % c.page] @ q[c.q_start[b] + i, h * G + g] * c.scale
                first = rng.choice(np.argsort(-s)[:max(2, len(s) // 2)])
                other = np.argsort(np.abs(s - s[first]))[1] if len(s) > 1 else first
                v = rng.uniform(60, 120)
                for j, x in ((first, v), (other, -v * np.exp(s[first] - s[other]))):
                    if j == other and other == first:
                        continue
                    c.cache[1][c.table[b, j // c.page], h, j % c.page // 8, d, j % 8] = layer.e4m3_encode(np.clip(x, -448, 448))


def _one_term(c):
    """The plain form with weights of a single bf16 term."""
    exp = np.exp
    try:
        np.exp = lambda x: torch.from_numpy(exp(x)).to(torch.bfloat16).double().numpy()
        return layer.attend(c.cache, c.q.double().numpy(), c.q_start, c.kv_len, c.table, c.scale)[0]
    finally:
        np.exp = exp


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_kv", [None, 100000])      # a workgroup an item, and pieces
@pytest.mark.parametrize("new,kv,hq,hk", [([1, 1, 1], [200, 513, 64], 2, 2), ([1, 8, 3], [700, 77, 300], 8, 1),
                                          ([2, 4, 0, 5], [130, 500, 9, 64], 16, 2)])
def test_weights_of_few_rows(dim, max_kv, new, kv, hq, hk):
    c = Case(new, kv, hq, hk, dim, 32, seed=dim + sum(kv), tail=False)
    _cancel(c, seed=3)
    want, _, size, terms = layer.attend(c.cache, c.q.double().numpy(), c.q_start, c.kv_len, c.table, c.scale)
    e = 2 * (dim + 8) * 2.0 ** -24 * terms[..., None] + 2.0 ** -20 + 2.0 ** -16 + (max(kv) / 4 + 64) * 2.0 ** -24
    bound = e * size + 2.0 ** -8 * (np.abs(want) + e * size)
    assert (np.abs(_one_term(c) - want) > 2 * bound).any()
    o, _ = c.run(c.gpu(), max_kv=max_kv)
    over = np.abs(o.double().cpu().numpy() - want) - bound
    assert over.max() <= 0, over.max()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_kv", [1, None])      # one piece, and several
@pytest.mark.parametrize("window,sinks", [(640, 70), (700, 0), (1000, 200), (0, 0), (65, 1)])
def test_whole_chunks_between_masked_ones(dim, max_kv, window, sinks):
    c = Case([150, 70], [1900, 1000], 4, 2, dim, 32, seed=window + dim)
    c.check(window, sinks, max_kv=max_kv)
    # NaN values where chunks are masked for some rows, where every row sees them,
    # among the first tokens and in the window's first and last chunk
    for b, j, h, d in ((0, 3, 0, 1), (0, 69, 1, 63), (0, 1500, 0, 2), (0, 1180, 1, 40), (0, 1110, 0, 33), (0, 1885, 1, 7),
                       (1, 64, 0, 5), (1, 960, 1, 0), (1, 350, 0, 62)):
        c.cache[1][c.table[b, j // 32], h, j % 32 // 8, d, j % 8] = 0x7F
    o, _ = c.check(window, sinks, max_kv=max_kv)
    assert np.isnan(o).any() and not np.isnan(o).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_kv", [1, None])
def test_a_prompt_of_many_chunks(dim, max_kv):
    Case([1700], [1700], 1, 1, dim, 64, seed=31).check(max_kv=max_kv)
    Case([900, 300], [1777, 2111], 2, 1, dim, 128, seed=32).check(max_kv=max_kv)


@pytest.mark.parametrize("new", [[100, 40], [33, 64]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (127, 70), (640, 130), (5000, 4), (3, 5000)])
def test_window_and_sinks_at_128_channels(new, window, sinks):
    Case(new, [700, 300], 4, 2, 128, 16, seed=window + sinks).check(window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 3), (700, 200)])
def test_a_window_far_smaller_than_the_bound(dim, window, sinks):
    Case([20, 9], [1500, 700], 16, 2, dim, 64, seed=window).check(window, sinks, max_kv=131072)
