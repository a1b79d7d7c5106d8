"""biloco_kv_append against the plain implementation.

The rotation's products and sums are rounded to fp32 one by one, so the fp32
form of the plain implementation has to be met bit for bit: q_out, codes, scale
bytes, and every byte that the call has no business with.  Against 64 bits the
rotated value is off by at most 3 roundings of 2^-24 of |a c| + |b s|, so a code
stands within half a code step plus that of the exact value.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import layer

pytestmark = pytest.mark.gpu


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


class Batch:
    """Sequences with `past` cached and `new` tokens over shuffled pages."""

    def __init__(self, past, new, hq, hk, dim, page, seed=0, rot=None, axes=1, n_pos=4096, fill="random"):
        rng = np.random.default_rng(seed)
        self.rng, self.dim, self.page, self.hq, self.hk = rng, dim, page, hq, hk
        self.past, self.new = np.array(past), np.array(new)
        self.T, self.rot, self.axes = int(sum(new)), dim if rot is None else rot, axes
        need = [max(1, -(-(p + n) // page)) for p, n in zip(past, new)]
        pool = sum(need) + 3
        order = rng.permutation(pool)
        self.table = np.full((len(past), max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = (self.past + self.new).astype(np.int32)
        k = rng.integers(0, 256, (pool, hk, page, dim)).astype(np.uint8)      # NaN codes among them
        v = rng.integers(0, 256, (pool, hk, page // 8, dim, 8)).astype(np.uint8)
        ks, vs = (rng.integers(110, 124, (pool, hk)).astype(np.uint8) for _ in range(2))
        self.cache = (k, v, ks, vs)
        self.x = {n: (rng.standard_normal((self.T, h, dim)) * 2.0).astype(np.float32)
                  for n, h in (("q", hq), ("k", hk), ("v", hk))}
        self.n_pos = n_pos
        ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(self.rot // 2) / max(1, self.rot // 2))
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.positions = rng.integers(0, n_pos, (axes, self.T)).astype(np.int32)
        self.pair_axis = (np.arange(self.rot // 2) * axes // max(1, self.rot // 2)).astype(np.uint8)

    def gpu(self, fused=True):
        d = dict(cache=tuple(torch.from_numpy(c).cuda() for c in self.cache))
        w = (self.hq + 2 * self.hk) * self.dim
        if fused:      # slices of one product's rows
            y = torch.zeros((self.T, w), dtype=torch.bfloat16, device="cuda")
            at = 0
            for n, h in (("q", self.hq), ("k", self.hk), ("v", self.hk)):
                d[n] = y[:, at:at + h * self.dim].unflatten(1, (h, self.dim)) if h else None
                if h:
                    d[n].copy_(_bf16(self.x[n]))
                at += h * self.dim
        else:
            for n in "qkv":
                d[n] = _bf16(self.x[n]).cuda()
        for n in ("positions", "cos_sin", "q_start", "kv_len", "table"):
            d[n] = torch.from_numpy(getattr(self, n)).cuda()
        return d

    def run(self, d, q_out=None, interleaved=False, stream=None, max_q=None):
        q = B.biloco_kv_append(d["cache"], d["q"], d["k"], d["v"], d["positions"], d["cos_sin"] if self.rot else None,
                               d["q_start"], d["kv_len"], d["table"], max_q or max(1, int(self.new.max())),
                               q_out=q_out, pair_axis=self.pair_axis.tobytes() if self.axes > 1 else None,
                               interleaved=interleaved, stream=stream)
        torch.cuda.synchronize()
        return q

    def plain(self, interleaved=False, dtype=np.float32):
        x = {n: _bf16(self.x[n]).float().numpy() for n in "qkv"}
        if self.rot:
            for n in "qk":
                x[n] = layer.rotate(x[n], self.positions, self.cos_sin, self.pair_axis, interleaved, dtype)
        return x, layer.append(self.cache, x["k"], x["v"], self.q_start, self.kv_len, self.table)

    def check(self, interleaved=False, fused=True, **kw):
        d = self.gpu(fused)
        q = self.run(d, interleaved=interleaved, **kw)
        x, want = self.plain(interleaved)
        for name, got, ref in zip(("k codes", "v codes", "k scales", "v scales"), d["cache"], want):
            got = got.cpu().numpy()
            if "codes" in name:      # a NaN's sign is free
                got, ref = np.where(got & 127 == 127, 127, got), np.where(ref & 127 == 127, 127, ref)
            np.testing.assert_array_equal(got, ref, err_msg=name)
        if self.hq:
            np.testing.assert_array_equal(q.float().cpu().numpy(), _bf16(x["q"]).float().numpy())
        return d, want


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("past,new", [
    ([0], [1]), ([5, 16, 31, 127], [1, 1, 1, 1]), ([0, 7, 3], [8, 9, 1]), ([13, 0, 64], [33, 16, 100]),
    ([1, 127, 40], [300, 129, 0]), ([63, 15], [2, 17])])
def test_matches_plain(page, dim, past, new):
    Batch(past, new, 4, 2, dim, page, seed=page + dim + sum(past)).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (40, 40), (64, 8), (5, 1), (0, 3)])
@pytest.mark.parametrize("new", [[1, 1, 1], [20, 1, 70]])
def test_heads(hq, hk, new):
    Batch([3, 64, 17], new, hq, hk, 128, 32, seed=hq).check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,axes", [(128, 128, 1), (128, 64, 2), (64, 64, 3), (64, 16, 1), (128, 112, 4),
                                          (64, 0, 1)])
def test_rotations(interleaved, dim, rot, axes):
    b = Batch([9, 0], [40, 3], 3, 2, dim, 16, seed=rot + axes, rot=rot, axes=axes)
    b.check(interleaved=interleaved)
    if axes > 1:      # axes that alternate from pair to pair
        b.pair_axis = (np.arange(rot // 2) % axes).astype(np.uint8)
        b.check(interleaved=interleaved)


def test_against_64_bits():
    b = Batch([9, 0, 30], [40, 65, 1], 3, 2, 128, 32, seed=5)
    d, _ = b.check()
    x64, _ = b.plain(dtype=np.float64)
    mag = np.abs(_bf16(b.x["k"]).float().numpy()).max() * 2.0      # over |a c| + |b s|
    k, v = layer.cache_values([t.cpu().numpy() for t in d["cache"]])
    ks = d["cache"][2].cpu().numpy()
    for s in range(len(b.past)):
        for i in range(b.new[s]):
            a, t = b.past[s] + i, b.q_start[s] + i
            pg, slot = b.table[s, a // 32], a % 32
            unit = 2.0 ** (ks[pg].astype(float) - 127)[:, None]
            got, want = k[pg, :, slot], x64["k"][t]
            step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(got), 1e-300) / unit)), 2.0 ** -6) * unit / 8
            assert np.all(np.abs(got - want) <= step / 2 + 3 * 2.0 ** -24 * mag)


def test_token_by_token_equals_the_plain_form_step_by_step():
    """A page filled by single tokens of growing size: its scale grows and the
    codes written before move with it."""
    b = Batch([0], [40], 2, 2, 64, 16, seed=3)
    b.x["k"] *= (2.0 ** np.linspace(-12, 9, 40))[:, None, None].astype(np.float32)
    b.x["v"] *= (2.0 ** np.linspace(6, -9, 40))[:, None, None].astype(np.float32)
    d = b.gpu()
    cache = d["cache"]
    for i in range(40):
        one = Batch([i], [1], 2, 2, 64, 16, seed=99)
        one.table, one.cache = b.table, tuple(c.cpu().numpy() for c in cache)
        one.x = {n: b.x[n][i:i + 1] for n in "qkv"}
        e = one.gpu()
        e["cache"] = cache
        one.run(e)
        _, want = one.plain()
        for got, ref in zip(cache, want):
            np.testing.assert_array_equal(got.cpu().numpy() & 127, ref & 127)
    assert cache[2].float().std() > 0


def test_special_values():
    b = Batch([4, 0], [12, 20], 2, 2, 128, 16, seed=8, rot=0)
    b.x["k"][3, 0, 5], b.x["k"][7, 1, 100] = np.inf, np.nan
    b.x["v"][0, 0, 0], b.x["v"][20, 1, 127], b.x["v"][25, 0, 3] = -np.inf, np.nan, 3.38e38
    b.x["v"][14] = 0.0
    b.x["k"][13] = 1e-39
    b.x["k"][16] = -2.9e38
    b.check()
    b.x["k"][:] = 0.0
    b.x["v"][:] = -0.0
    b.check()


def test_positions_outside_the_table_are_nan():
    b = Batch([0], [6], 2, 1, 64, 16, seed=2, axes=2)
    b.positions[0, 1], b.positions[1, 3] = -1, b.n_pos
    d, want = b.check()
    assert np.any((want[0] & 127) == 127)
    q = b.run(b.gpu())
    assert bool(q[1].isnan().any()) and bool(q[3].isnan().any()) and not bool(q[2].isnan().any())


def test_pages_and_tables_outside_the_cache_are_left_alone():
    b = Batch([0, 0], [20, 20], 2, 1, 64, 16, seed=2)
    b.table[0, 1], b.table[1, 0] = 10 ** 6, -5
    d = b.gpu()
    b.run(d)
    k = d["cache"][0].cpu().numpy()
    rest = [p for p in range(k.shape[0]) if p not in (b.table[0, 0], b.table[1, 1])]
    np.testing.assert_array_equal(k[rest], b.cache[0][rest])
    assert not np.array_equal(k[b.table[1, 1]], b.cache[0][b.table[1, 1]])


def test_in_place_and_separate_rows():
    b = Batch([2, 50], [30, 1], 4, 2, 128, 32, seed=4)
    d = b.gpu()
    x, want = b.plain()
    q = b.run(d, q_out=d["q"])      # the product's own rows
    np.testing.assert_array_equal(q.float().cpu().numpy(), _bf16(x["q"]).float().numpy())
    np.testing.assert_array_equal(d["cache"][1].cpu().numpy() & 127, want[1] & 127)
    b.check(fused=False)


def test_nothing_to_do():
    b = Batch([4], [0], 2, 1, 64, 16, seed=4)
    d = b.gpu(fused=False)
    b.run(d)
    for got, was in zip(d["cache"], b.cache):
        np.testing.assert_array_equal(got.cpu().numpy(), was)


def test_another_stream_and_replay():
    b = Batch([2, 50, 7], [1, 1, 1], 8, 2, 128, 32, seed=4)
    d = b.gpu()
    _, want = b.plain()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(s):
        b.run(d, q_out=out)
    s.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_kv_append(d["cache"], d["q"], d["k"], d["v"], d["positions"], d["cos_sin"], d["q_start"], d["kv_len"],
                           d["table"], 1, q_out=out)
    for _ in range(3):
        out.zero_()
        for t, c in zip(d["cache"], b.cache):
            t.copy_(torch.from_numpy(c))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        for got, ref in zip(d["cache"], want):
            np.testing.assert_array_equal(got.cpu().numpy() & 127, ref & 127)


@pytest.mark.parametrize("new", [[1, 1], [150, 3]])
def test_offsets_beyond_32_bits(new):
    """The same pages at the end of a cache of more than 2^32 bytes."""
    b = Batch([100, 7], new, 8, 8, 128, 128, seed=21)
    d = b.gpu()
    pages = 33000      # of 128 KiB each
    big = B.biloco_kv_cache(pages, 8, 128, 128)
    assert big[0].numel() > 1 << 32
    n = d["cache"][0].shape[0]
    for t, u in zip(big, d["cache"]):
        t[-n:].copy_(u)
    q0 = b.run(d)
    small = d["cache"]
    d["cache"] = big
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - n), d["table"])
    q = b.run(d)
    assert torch.equal(q, q0)
    for t, u in zip(big, small):
        assert torch.equal(t[-n:], u)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("kv,new", [([0, 7], [1, 1]), ([3, 40, 0], [5, 2, 3]), ([0, 0, 0], [1, 1, 1]), ([20, 90], [70, 30])])
def test_rows_before_the_first_token_are_not_appended(dim, page, kv, new):
    """Row i of n new ones is token kv_len - n + i; where that is negative (an idle
    slot of a padded batch, for one) its q is rotated and nothing is written, not
    even to the pages that its table row still names."""
    b = Batch([max(0, k - n) for k, n in zip(kv, new)], new, 4, 2, dim, page, seed=sum(kv) + page)
    b.kv_len = np.array(kv, np.int32)
    b.past = b.kv_len - b.new
    b.table[:] = np.where(b.table < 0, b.table.max(), b.table)      # left from earlier sequences
    idle = np.array(kv) == 0
    b.table[idle] = b.table[~idle][0] if (~idle).any() else b.table[idle]
    b.check()
