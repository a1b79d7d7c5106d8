"""biloco_attn_paged against the 64-bit formula.

Tolerances.  Queries, codes and scales are exact in bf16, products exact in
fp32; a score is a sum of `dim` such terms, off by at most dim 2^-24 of the sum
of their magnitudes, so with t = max_j scale sum_d |q_d k_jd| a weight is off by
e = 2 (dim + 8) 2^-24 t + 2^-20 relative (numerator and denominator; the
exponential and the sums' own roundings in the last term).  The weights' rounding
to bf16 adds 2^-8 each, the output's 2^-8 of itself:
  |o - o64| <= (2^-8 + e) sum w |v| + 2^-8 |o64|,   |lse - lse64| <= e + 2^-21 (1 + |lse64|).
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import layer

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, new, kv, hq, hk, dim, page, seed=0, tail=True):
        rng = np.random.default_rng(seed)
        self.new, self.kv_len = np.array(new), np.array(kv, np.int32)
        self.dim, self.page, self.hq, self.hk, self.T = dim, page, hq, hk, int(sum(new))
        need = [max(1, -(-n // page)) for n in kv]
        pool = sum(need) + 2
        order = rng.permutation(pool)
        self.table = np.full((len(kv), max(need) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        k = layer.e4m3_encode(np.clip(rng.standard_normal((pool, hk, page, dim)) * 100, -448, 448))
        v = layer.e4m3_encode(np.clip(rng.standard_normal((pool, hk, page // 8, dim, 8)) * 100, -448, 448))
        ks, vs = (rng.integers(118, 122, (pool, hk)).astype(np.uint8) for _ in range(2))
        if tail:      # whatever lies past the last token, NaN codes and odd scales included
            used = np.zeros((pool, page), bool)
            for b, n in enumerate(kv):
                for j in range(n):
                    used[self.table[b, j // page], j % page] = True
            k = np.where(used[:, None, :, None], k, np.uint8(0x7F))
            u8 = used.reshape(pool, 1, page // 8, 1, 8)
            v = np.where(u8, v, np.uint8(0xFF))
            free = ~used.any(1)
            ks[free], vs[free] = 255, 255
        self.cache = [k, v, ks, vs]
        self.q = torch.from_numpy(rng.standard_normal((self.T, hq, dim)).astype(np.float32)).to(torch.bfloat16)
        self.scale = dim ** -0.5

    def gpu(self):
        return dict(cache=tuple(torch.from_numpy(np.ascontiguousarray(c)).cuda() for c in self.cache),
                    q=self.q.cuda(), q_start=torch.from_numpy(self.q_start).cuda(),
                    kv_len=torch.from_numpy(self.kv_len).cuda(), table=torch.from_numpy(self.table).cuda())

    def run(self, d, window=0, sinks=0, max_q=None, max_kv=None, **kw):
        lse = torch.full((self.T, self.hq), 77.0, device="cuda")
        o = B.biloco_attn_paged(d["cache"], d["q"], d["q_start"], d["kv_len"], d["table"],
                                max_q or max(1, int(self.new.max())), max(1, int(self.kv_len.max())) if max_kv is None
                                else max_kv, self.scale, window=window, sinks=sinks, lse=lse, **kw)
        torch.cuda.synchronize()
        return o, lse

    def check(self, window=0, sinks=0, **kw):
        o, lse = self.run(self.gpu(), window, sinks, **kw)
        want, want_lse, mag, terms = layer.attend(self.cache, self.q.double().numpy(), self.q_start, self.kv_len,
                                                  self.table, self.scale, window, sinks)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        e = 2 * (self.dim + 8) * 2.0 ** -24 * terms + 2.0 ** -20
        bound = (2.0 ** -8 + e[..., None]) * mag + 2.0 ** -8 * np.abs(want)
        assert np.array_equal(np.isnan(o), np.isnan(want))
        assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse))
        ok = ~np.isnan(want)
        worst = (np.abs(o - want)[ok] - bound[ok]).max() if ok.any() else 0.0
        assert worst <= 0, worst
        fin = np.isfinite(want_lse)
        assert np.all(np.abs(lse[fin] - want_lse[fin]) <= e[fin] + 2.0 ** -21 * (1 + np.abs(want_lse[fin])))
        return o, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kv", [[1], [2, 15, 16, 17], [63, 64, 65, 128, 129], [255, 256, 257, 300], [1025, 3, 700]])
def test_single_tokens(dim, page, kv):
    Case([1] * len(kv), kv, 4, 2, dim, page, seed=sum(kv) + page).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (40, 40), (64, 8), (16, 1), (17, 1), (40, 1), (10, 2), (66, 2)])
def test_heads(hq, hk):
    Case([1, 1, 1], [77, 900, 5], hq, hk, 128, 32, seed=hq).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv", [
    ([2], [2]), ([5, 1, 4], [400, 33, 1000]), ([7, 16, 17], [7, 100, 17]), ([33, 64], [33, 500]),
    ([65, 130], [65, 1300]), ([200, 3, 0, 1], [200, 3, 50, 777])])
def test_several_tokens(dim, new, kv):
    Case(new, kv, 8, 2, dim, 32, seed=sum(kv)).check()


@pytest.mark.parametrize("new,kv", [([1, 1], [1500, 40]), ([5, 2], [900, 900]), ([100, 40], [700, 40]),
                                    ([300], [300])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (127, 70), (640, 130), (5000, 4), (3, 5000)])
def test_window_and_sinks(new, kv, window, sinks):
    Case(new, kv, 4, 2, 64, 16, seed=window + sinks).check(window, sinks)


def test_rows_that_see_nothing():
    c = Case([4, 3, 2, 1, 0], [2, 0, 2, 0, 0], 4, 2, 128, 16, seed=1)
    o, lse = c.check()
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(o[4:7] == 0)
    Case([70, 1], [30, 0], 8, 2, 64, 16, seed=1).check()
    Case([1, 1], [0, 2000], 4, 2, 64, 16, seed=1).check()


def test_nan_reaches_only_the_rows_that_see_it():
    c = Case([6, 40, 1], [300, 64, 700], 4, 2, 128, 32, seed=6)
    for b, j, h, d in ((0, 297, 0, 5), (0, 296, 1, 127), (1, 40, 0, 64), (2, 3, 1, 0), (2, 699, 0, 9)):
        c.cache[1][c.table[b, j // 32], h, j % 32 // 8, d, j % 8] = 0x7F
    o, _ = c.check()
    assert np.isnan(o).any() and not np.isnan(o).all()
    c.check(window=50, sinks=2)
    c.check(window=1)
    c.cache[0][c.table[0, 9], 1, 9, 3] = 0xFF      # a key: the whole row of scores it is in
    c.check()


def test_large_scores_and_extreme_scales():
    c = Case([1, 3], [300, 20], 4, 2, 64, 16, seed=2, tail=False)
    c.cache[2][:] = 127      # scores of several thousands: one weight takes all
    c.check()
    c = Case([1, 3], [300, 20], 4, 2, 64, 16, seed=2, tail=False)
    c.cache[2][:] = np.random.default_rng(0).integers(1, 121, c.cache[2].shape)
    c.cache[3][:] = np.random.default_rng(1).integers(60, 180, c.cache[3].shape)
    c.check()


def test_strided_rows_and_outputs():
    c = Case([3, 1], [90, 400], 4, 2, 64, 32, seed=3)
    d = c.gpu()
    o0, lse0 = c.run(d)
    wide = torch.zeros((4, 4 * 64 + 128), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 64:64 + 256].unflatten(1, (4, 64))
    q.copy_(d["q"])
    out = torch.full((4, 4 * 64 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    d["q"] = q
    o, lse = c.run(d, out=out[:, :256].unflatten(1, (4, 64)))
    assert torch.equal(o, o0) and torch.equal(lse, lse0) and bool((out[:, 256:] == 5.0).all())
    o = B.biloco_attn_paged(d["cache"], q, d["q_start"], d["kv_len"], d["table"], 3, 400, c.scale)
    assert torch.equal(o, o0)


@pytest.mark.parametrize("max_kv", [0, 1, 700, 100000])
def test_host_bounds_only_shape_the_launch(max_kv):
    Case([1, 1, 2], [2000, 1, 333], 8, 2, 128, 64, seed=9).check(max_kv=max_kv)


def test_page_ids_outside_the_cache_are_not_read():
    c = Case([1], [200], 2, 1, 64, 16, seed=9)
    d = c.gpu()
    d["table"][0, 3] = 10 ** 8
    d["table"][0, 4] = -7
    c.run(d)      # unspecified values, no access outside the cache


def test_long_context_is_split_and_joined():
    c = Case([1], [33000], 8, 1, 64, 128, seed=11)
    c.check()
    c = Case([1, 1, 1], [9000, 1, 4097], 4, 2, 128, 64, seed=12)
    c.check()


def test_more_sequences_than_lanes():
    kv = [int(x) for x in np.random.default_rng(0).integers(0, 40, 150)]
    kv[100] = 3000
    Case([1 if x % 5 else 0 for x in range(150)], kv, 2, 1, 64, 16, seed=13).check()


@pytest.mark.parametrize("new,kv", [([1, 1], [2500, 60]), ([4, 4], [300, 900]), ([150], [600])])
def test_repeats_and_replays_are_the_same(new, kv):
    c = Case(new, kv, 16, 2, 128, 64, seed=5)
    d = c.gpu()
    o0, lse0 = c.run(d)
    ws = torch.empty(max(16, B.biloco_attn_workspace_bytes(len(kv), c.T, 16, 2, 128, max(new), max(kv))),
                     dtype=torch.uint8, device="cuda").fill_(0xFF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = c.run(d, workspace=ws)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    o, lse = torch.zeros_like(o0), torch.zeros_like(lse0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_attn_paged(d["cache"], d["q"], d["q_start"], d["kv_len"], d["table"], max(new), max(kv), c.scale,
                            out=o, lse=lse, workspace=ws)
    for _ in range(3):
        o.zero_(), lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_offsets_beyond_32_bits(new):
    """The same pages at the end of a cache of more than 2^32 bytes."""
    c = Case(new, [300, 90], 8, 8, 128, 128, seed=21, tail=False)
    d = c.gpu()
    o0, lse0 = c.run(d)
    pages = 33000      # of 128 KiB each
    big = B.biloco_kv_cache(pages, 8, 128, 128)
    assert big[0].numel() > 1 << 32
    n = d["cache"][0].shape[0]
    for t, u in zip(big, d["cache"]):
        t[-n:].copy_(u)
    d["cache"] = big
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - n), d["table"])
    o, lse = c.run(d)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
@pytest.mark.parametrize("max_kv", [None, 100000])      # a workgroup an item, and pieces
def test_sequences_of_different_row_counts(dim, window, sinks, max_kv):
    # 8 to 64 rows of a key/value head: one, two and four groups of waves in one launch
    Case([1, 3, 8, 5, 2, 0, 4, 6], [900, 25, 777, 600, 64, 300, 1, 129], 16, 2, dim, 32, seed=dim + window).check(
        window, sinks, max_kv=max_kv)
