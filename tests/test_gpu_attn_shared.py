"""biloco_attn_shared against the 64-bit formula on the tokens that its definition names.

Tolerances as for biloco_attn_paged: queries, codes and scales are exact in bf16, a
score is a sum of `dim` exact terms, so with t = max_j scale sum_d |q_d k_jd| a weight is
off by e = 2 (dim + 8) 2^-24 t + 2^-20 relative; the weights' rounding to bf16 adds 2^-8
each, the output's 2^-8 of itself:
  |o - o64| <= (2^-8 + e) sum w |v| + 2^-8 |o64|,   |lse - lse64| <= e + 2^-21 (1 + |lse64|).
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import layer

pytestmark = pytest.mark.gpu


class Case:
    """Groups of (shared tokens, [(new tokens, tokens in all), ...])."""

    def __init__(self, groups, hq, hk, dim, page, seed=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hk, self.dim, self.page, self.scale = hq, hk, dim, page, dim ** -0.5
        seqs = [s for _, g in groups for s in g]
        self.new = np.array([n for n, _ in seqs])
        self.kv_len = np.array([k for _, k in seqs], np.int32)
        self.T = int(self.new.sum())
        self.q_start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.group_start = np.cumsum([0] + [len(g) for _, g in groups]).astype(np.int32)
        self.shared = np.array([n for n, _ in groups], np.int32)
        cols = max(max(1, -(-int(max(k, n)) // page)) for n, g in groups for _, k in g) + 1
        pool, used = [], []
        self.table = np.full((len(seqs), cols), -1, np.int32)      # as a kernel reads own tokens
        self.seen = np.full((len(seqs), cols * page), -1, np.int64)      # page * page size + slot of each token
        b = at = 0
        total = sum(-(-n // page) for n, _ in groups) + sum(-(-max(k, 1) // page) for k in self.kv_len) + 3
        order = rng.permutation(total)
        for n, g in groups:
            first = b
            for _, kv in g:
                own = max(0, -(-kv // page) - n // page)      # pages behind the shared whole ones
                if b == first:
                    got = -(-n // page) if n else 0
                    self.table[b, :got] = order[at:at + got]
                    at += got
                    whole = self.table[b, :n // page].copy()
                    head = self.table[b, :got].copy()
                else:
                    # other rows name rubbish where the first one's row is to be read
                    self.table[b, :n // page] = -7 if (b - first) % 2 else whole
                if b != first or n % page == 0:
                    self.table[b, n // page:n // page + own] = order[at:at + own]
                    at += own
                elif own > 1:
                    self.table[b, n // page + 1:n // page + own] = order[at:at + own - 1]
                    at += own - 1
                for j in range(max(kv, 0)):
                    row = head if j < n else self.table[b]
                    self.seen[b, j] = int(row[j // page]) * page + j % page
                b += 1
        pool = total
        k = layer.e4m3_encode(np.clip(rng.standard_normal((pool, hk, page, dim)) * 100, -448, 448))
        v = layer.e4m3_encode(np.clip(rng.standard_normal((pool, hk, page // 8, dim, 8)) * 100, -448, 448))
        ks, vs = (rng.integers(118, 122, (pool, hk)).astype(np.uint8) for _ in range(2))
        used = np.zeros(pool * page, bool)
        used[self.seen[self.seen >= 0]] = True
        used = used.reshape(pool, page)
        # whatever no token names, NaN codes and odd scales included
        k = np.where(used[:, None, :, None], k, np.uint8(0x7F))
        v = np.where(used.reshape(pool, 1, page // 8, 1, 8), v, np.uint8(0xFF))
        ks[~used.any(1)], vs[~used.any(1)] = 255, 255
        self.cache = [k, v, ks, vs]
        self.q = torch.from_numpy(rng.standard_normal((self.T, hq, dim)).astype(np.float32)).to(torch.bfloat16)

    def want(self, window, sinks):
        """By sequences of their own whose pages are single tokens, in the oracle's layout."""
        page, (kc, vc, ks, vs) = self.page, self.cache
        pool, hk = ks.shape
        # tokens as pages of 8 slots of which the first is used
        k1 = np.zeros((pool * page, hk, 8, self.dim), np.uint8)
        v1 = np.zeros((pool * page, hk, 1, self.dim, 8), np.uint8)
        k1[:, :, 0] = kc.transpose(0, 2, 1, 3).reshape(pool * page, hk, self.dim)
        v1[:, :, 0, :, 0] = vc.transpose(0, 2, 4, 1, 3).reshape(pool * page, hk, self.dim)
        kval, vval = layer.cache_values((k1, v1, np.repeat(ks, page, 0), np.repeat(vs, page, 0)))
        T, G = self.T, self.hq // self.hk
        o, mag = np.zeros((T, self.hq, self.dim)), np.zeros((T, self.hq, self.dim))
        lse, terms = np.full((T, self.hq), -np.inf), np.zeros((T, self.hq))
        q = self.q.double().numpy()
        for b, n in enumerate(self.new):
            for i in range(n):
                p, t = self.kv_len[b] - n + i, self.q_start[b] + i
                if p < 0:
                    continue
                lo = max(0, p - window + 1) if window else 0
                seen = np.array(list(range(min(sinks, lo))) + list(range(lo, p + 1)))
                at = self.seen[b, seen]
                for h in range(self.hq):
                    k, v = kval[at, h // G, 0], vval[at, h // G, 0]
                    with np.errstate(invalid="ignore"):
                        s = (k @ q[t, h]) * self.scale
                        w = np.exp(s - s.max())
                        o[t, h], mag[t, h] = (w @ v) / w.sum(), (w @ np.abs(v)) / w.sum()
                        lse[t, h] = s.max() + np.log(w.sum())
                        terms[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * self.scale
        return o, lse, mag, terms

    def args(self):
        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x)).cuda()
        return (tuple(dev(c) for c in self.cache), self.q.cuda(), dev(self.q_start), dev(self.kv_len), dev(self.table),
                dev(self.group_start), dev(self.shared), max(1, int(self.new.max())), max(1, int(self.kv_len.max())),
                int(self.shared.max()), self.scale)

    def run(self, **kw):
        lse = torch.full((self.T, self.hq), 77.0, device="cuda")
        o = B.biloco_attn_shared(*self.args(), lse=lse, **kw)
        torch.cuda.synchronize()
        return o, lse

    def check(self, window=0, sinks=0, **kw):
        o, lse = self.run(window=window, sinks=sinks, **kw)
        want, want_lse, mag, terms = self.want(window, sinks)
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
@pytest.mark.parametrize("shared", [0, 1, 15, 16, 63, 64, 65, 128, 200, 700])
def test_one_group(dim, page, shared):
    Case([(shared, [(1, shared + k) for k in (1, 2, 30, 70, 1)])], 4, 2, dim, page, seed=shared + page).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (40, 40), (64, 8), (16, 1), (17, 1), (40, 1), (10, 2), (60, 1), (66, 2)])
def test_heads(hq, hk):
    Case([(300, [(1, 301), (1, 333), (1, 400)]), (64, [(1, 65)])], hq, hk, 128, 32, seed=hq).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("groups", [
    [(100, [(3, 140), (1, 101), (5, 260), (2, 102)])],
    [(64, [(1, 70)] * 40)],
    [(500, [(2, 600)] * 33), (32, [(1, 64)] * 3), (0, [(4, 50), (1, 1)]), (1000, [(7, 1010)])],
    [(130, [(1, 131 + i) for i in range(70)]), (5, [(1, 6)] * 70)]])
def test_groups_and_several_tokens(dim, groups):
    Case(groups, 8, 2, dim, 32, seed=len(groups)).check()


def test_sequences_that_end_inside_the_shared_tokens():
    """Rows whose position is a shared token's; idle slots; more rows than tokens."""
    Case([(200, [(1, 100), (4, 200), (4, 202), (1, 0), (0, 50), (0, 0), (3, 2), (1, 300)])], 4, 2, 128, 16, seed=3).check()
    Case([(64, [(1, 0), (2, 1)]), (0, [(0, 0)]), (128, [(0, 200)])], 4, 2, 64, 16, seed=4).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (100, 0), (130, 70), (640, 130), (5000, 4), (3, 5000), (40, 260)])
def test_window_and_sinks(window, sinks):
    Case([(250, [(1, 251), (3, 300), (2, 900), (1, 120)]), (40, [(4, 100), (1, 41)])], 4, 2, 64, 16,
         seed=window + sinks).check(window, sinks)
    Case([(700, [(1, 720)] * 40)], 8, 2, 128, 64, seed=window).check(window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
def test_sequences_of_many_rows_among_others(dim):
    """Prompts behind a shared part: they read their own tables, which name the shared pages."""
    c = Case([(128, [(1, 140), (70, 260), (2, 150), (1, 129)]), (64, [(40, 200)])], 8, 2, dim, 32, seed=9)
    c.table[1, :4], c.table[3, :4] = c.table[0, :4], c.table[0, :4]
    c.check()
    c = Case([(64, [(80, 200), (70, 300)])], 8, 2, dim, 32, seed=10)      # none of few
    c.table[1, :2] = c.table[0, :2]
    c.check()


def test_long_shared_part_is_split():
    Case([(9000, [(1, 9001), (1, 9100), (2, 9500)])], 4, 2, 128, 64, seed=11).check()
    Case([(6000, [(1, 6000 + 9 * i + 1) for i in range(40)])], 8, 1, 64, 16, seed=12).check()


def test_nan_reaches_only_the_rows_that_see_it():
    c = Case([(100, [(6, 104), (1, 160), (1, 101)])], 4, 2, 128, 32, seed=6)
    shared, own = c.seen[0, 99], c.seen[1, 150]
    for at, h, d in ((shared, 0, 5), (own, 1, 127)):
        c.cache[1][at // 32, h, at % 32 // 8, d, at % 8] = 0x7F
    o, _ = c.check()
    assert np.isnan(o[1:, 0, 5]).all() and not np.isnan(o[0]).any() and np.isnan(o[6, 2, 127]) and not np.isnan(o[7, 2]).any()


def test_equals_the_paged_call_on_the_same_pages():
    """Tables that name the shared pages: both calls are within one rounding of a weight of one another."""
    c = Case([(512, [(1, 513 + 40 * i) for i in range(12)]), (96, [(2, 200), (1, 97)])], 16, 4, 128, 32, seed=13)
    for b, (first, n) in enumerate([(0, 16)] * 12 + [(12, 3)] * 2):
        c.table[b, :n] = c.table[first, :n]
    o, lse = c.check()
    a = c.args()
    other = torch.empty((c.T, c.hq), device="cuda")
    want = B.biloco_attn_paged(*a[:5], a[7], a[8], c.scale, lse=other)
    e = 2.0 ** -7 * float(want.float().abs().max())
    assert float((torch.from_numpy(o).cuda() - want.double()).abs().max()) <= e
    assert float((torch.from_numpy(lse).cuda() - other.double()).abs().max()) <= 1e-4


def test_one_workspace_serves_smaller_calls():
    ws = torch.full((B.biloco_attn_shared_workspace_bytes(48, 100, 8, 2, 64, 8, 3000, 4, 2000),), 255, dtype=torch.uint8,
                    device="cuda")
    for seed, groups in enumerate(([(2000, [(2, 2100)] * 48)], [(1500, [(1, 1600)])], [(64, [(8, 200)] * 3), (0, [(1, 9)] * 4)],
                                   [(1000, [(1, 1001)] * 2)] * 4)):
        c = Case(groups, 8, 2, 64, 32, seed=seed)
        c.check(workspace=ws)
        c.check(40, 3, workspace=ws)


def test_arrays_that_break_the_rules_stay_inside():
    """Unspecified values, no access outside: lists that are not in order, pages that are not there."""
    c = Case([(128, [(1, 140), (2, 150)]), (64, [(1, 70), (1, 90)])], 8, 2, 128, 32, seed=20)
    for group_start, shared in (([3, 1, 9], [128, 64]), ([-4, 2, 2], [1 << 30, -5]), ([0, 0, 0], [64, 64]), ([2, 2, 4], [32, 0]),
                                ([0, 4, 2], [1 << 29, 40])):
        a = list(c.args())
        a[5], a[6] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (group_start, shared))
        B.biloco_attn_shared(*a)
        a[2] = torch.tensor([0, 3, 1, 9, 2], dtype=torch.int32, device="cuda")
        B.biloco_attn_shared(*a)
        a[4] = torch.full_like(a[4], 1 << 30)
        B.biloco_attn_shared(*a)
        torch.cuda.synchronize()


def test_captured():
    c = Case([(288, [(1, 301 + 7 * i) for i in range(9)]), (64, [(1, 100)] * 3)], 8, 2, 128, 32, seed=21)
    c.table[1:9, :9], c.table[10:, :2] = c.table[0, :9], c.table[9, :2]      # less may be shared than the pages are
    a, kw = c.args(), dict(lse=torch.empty((c.T, c.hq), device="cuda"), out=torch.empty_like(c.q.cuda()))
    kw["workspace"] = torch.empty(B.biloco_attn_shared_workspace_bytes(12, c.T, 8, 2, 128, 1, 400, 2, 288), dtype=torch.uint8,
                                  device="cuda")
    B.biloco_attn_shared(*a[:8], 400, *a[9:], **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_attn_shared(*a[:8], 400, *a[9:], **kw)
    for i in range(4):      # lengths that change between replays
        a[3].copy_(torch.from_numpy(c.kv_len - i))
        a[6].copy_(torch.tensor([288 - 50 * i, 64 - 16 * i], dtype=torch.int32))
        a[1].copy_(torch.randn(c.q.shape).to(torch.bfloat16))
        g.replay()
        got, got_lse = kw["out"].clone(), kw["lse"].clone()
        lse = torch.empty_like(got_lse)
        want = B.biloco_attn_shared(*a[:8], 400, *a[9:], lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_lse, lse)
