"""biloco_sample against the 64-bit form.

Tokens are equal, unless the outcome hangs on less than the weights' steps: V weights
are off by at most 2^-45 of the largest each, and the largest is at most the sum compared,
so a border nearer than V 2^-44 of that sum (and of 2^-40 for the exponential's own error)
may fall either way; where it does the row is left out, and there are hardly any.
log-probabilities are rounded once (2^-24) and carry the sum's error.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import answers

pytestmark = pytest.mark.gpu


def _dev(v, dtype=torch.float32):
    return None if v is None else torch.as_tensor(np.asarray(v)).to(dtype).cuda()


def check(x, u, t=None, k=None, p=None, m=None, exact=False):
    """x: a tensor [rows][V]."""
    R, V = x.shape
    lp = torch.full((R,), 9.0, device="cuda")
    tok = B.biloco_sample(x.cuda(), _dev(u), _dev(t), _dev(k, torch.int32), _dev(p), _dev(m), logprob=lp)
    torch.cuda.synchronize()
    tok, lp, xs = tok.cpu().numpy(), lp.double().cpu().numpy(), x.double().cpu().numpy()
    skipped = 0
    for r in range(R):
        def of(v, off):
            return off if v is None else float(np.float32(v[r]))
        with np.errstate(invalid="ignore"):
            want, want_lp, near = answers.sample(xs[r], of(u, 0), of(t, 1.0), 0 if k is None else int(k[r]), of(p, 1.0), of(m, 0.0))
        if tok[r] != want and near < V * 2.0 ** -44 + 2.0 ** -40 and not exact:
            skipped += 1
            continue
        assert tok[r] == want, (r, tok[r], want, near)
        if np.isinf(want_lp):
            assert lp[r] == want_lp
        else:
            assert abs(lp[r] - want_lp) <= 2.0 ** -24 * abs(want_lp) + V * 2.0 ** -44 + 2.0 ** -40
    assert skipped <= max(1, R // 50)
    return tok


def _logits(rng, R, V, dtype, spread=2.0):
    x = rng.standard_normal((R, V)) * spread
    x[np.arange(R), rng.integers(0, V, R)] += 4 * spread
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 63, 64, 65, 511, 512, 1000, 1025, 4099, 20011])
def test_sizes(dtype, V):
    rng = np.random.default_rng(V)
    R = 24
    x = _logits(rng, R, V, dtype)
    u = rng.random(R, np.float32)
    check(x, u)
    check(x, u, t=rng.uniform(0.2, 3, R))
    check(x, u, k=rng.integers(1, max(2, V), R))
    check(x, u, p=rng.uniform(0.1, 0.99, R))
    check(x, u, m=rng.uniform(0.001, 0.5, R))
    check(x, u, t=rng.choice([0.0, 0.5, 1.0, 1.7], R), k=rng.choice([0, 1, 5, 50, V], R), p=rng.choice([0.5, 0.9, 1.0], R),
          m=rng.choice([0.0, 0.02, 0.3], R))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,spread", [(32000, 2.0), (100001, 0.3), (131072, 2.5), (262144, 1.0), (1048575, 3.0)])
def test_many_logits(dtype, V, spread):
    rng = np.random.default_rng(V)
    R = 12
    x = _logits(rng, R, V, dtype, spread)
    u = rng.random(R, np.float32)
    check(x, u)
    check(x, u, k=[0, 1, 2, 50, 1023, 1024, 1025, 2000, 30000, V - 1, V, -3])
    check(x, u, p=[0.0, 0.01, 0.3, 0.5, 0.9, 0.95, 0.99, 0.999, 0.99999, 1.0, 1.5, -1.0])
    check(x, u, t=[0.05, 0.1, 0.3, 0.5, 0.7, 1.0, 1.3, 2.0, 5.0, 50.0, 1e4, 0.0], p=[0.9] * R, k=[0, 3000] * 6)
    check(x, u, m=[0.0, 1e-9, 1e-4, 0.01, 0.1, 0.5, 0.9, 1.0, 2.0, -1.0, 0.3, 0.05], p=[0.99, 1.0] * 6)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties(dtype):
    """Equal logits are taken by index, whatever their number."""
    rng = np.random.default_rng(0)
    R, V = 12, 20000
    x = torch.from_numpy(rng.integers(0, 3, (R, V)).astype(np.float32)).to(dtype)
    u = rng.random(R, np.float32)
    check(x, u, k=[1, 2, 500, 1024, 1025, 4000, 6600, 6700, 8000, 13400, 19999, 20000])
    check(x, u, p=np.linspace(0.05, 0.97, R))
    flat = torch.zeros((R, V), dtype=dtype)
    # all alike: sums are exact, so borders may be met exactly
    got = check(flat, np.arange(R) / 16, exact=True)
    assert list(got) == [int(r / 16 * V) for r in range(R)]
    got = check(flat, np.full(R, 0.999), k=np.arange(1, R + 1) * 1500, exact=True)
    assert list(got) == [int(np.float32(0.999) * (r + 1) * 1500) for r in range(R)]
    check(flat, np.full(R, 0.5), p=np.full(R, 0.5), exact=True)
    signed = flat.clone()
    signed[:, ::2] = -0.0
    check(signed, np.full(R, 0.25), k=np.full(R, 7), exact=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_masked_never_comes(dtype):
    rng = np.random.default_rng(1)
    R, V = 16, 5000
    x = _logits(rng, R, V, dtype)
    x[:, ::3] = -float("inf")
    x[:, 1::3] = float("nan")
    x[3:5] = -float("inf")
    x[5] = float("nan")
    x[6, 17], x[6, 4000] = float("inf"), float("inf")
    x[7, :] = -float("inf")
    x[7, 4999] = -3.0
    x[8] = torch.finfo(dtype).min
    x[9, 5] = torch.finfo(dtype).max
    u = rng.random(R, np.float32)
    for kw in ({}, dict(k=np.full(R, 40)), dict(p=np.full(R, 0.8)), dict(k=np.full(R, 4000), p=np.full(R, 0.99)),
               dict(m=np.full(R, 0.1)), dict(t=np.zeros(R)), dict(t=np.full(R, np.inf)), dict(t=np.full(R, 1e-30))):
        tok = check(x, u, **kw)
        assert list(tok[3:6]) == [-1, -1, -1] and tok[7] == 4999 and tok[6] in (17, 4000)
        assert tok[9] == 5 or np.isinf(kw.get("t", [0.0])[0])      # an infinite temperature makes finite logits alike


def test_numbers_at_the_ends():
    rng = np.random.default_rng(2)
    R, V = 8, 3000
    x = _logits(rng, R, V, torch.float32)
    u = np.array([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan, 0.5, 2.0 ** -149], np.float32)
    for kw in ({}, dict(k=np.full(R, 10)), dict(p=np.full(R, 0.9)), dict(k=np.full(R, 2000))):
        check(x, u, **kw)
    nan = np.full(R, np.nan)
    u = rng.random(R, np.float32)
    check(x, u, t=nan)
    check(x, u, p=nan, m=nan)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_apart_and_rows_alike(dtype):
    rng = np.random.default_rng(3)
    R, V = 10, 1003
    wide = _logits(rng, R, 2 * V + 1, dtype)
    u, k = rng.random(R, np.float32), rng.integers(1, 300, R)
    lead = 16 // wide.element_size()
    whole = wide.cuda()
    tok = B.biloco_sample(whole[:, lead:lead + V], _dev(u), top_k=_dev(k, torch.int32))
    want = check(wide[:, lead:lead + V].contiguous(), u, k=k)
    assert list(tok.cpu().numpy()) == list(want)
    one = wide[:1, :V].contiguous()
    tok = B.biloco_sample(one.cuda().expand(R, V), _dev(u), top_k=_dev(k, torch.int32))
    assert list(tok.cpu().numpy()) == list(check(one.expand(R, V).contiguous(), u, k=k))


def test_draws_follow_the_weights():
    """Evenly spaced u: each token comes as often as its weight says, to one."""
    rng = np.random.default_rng(4)
    V, R = 50, 4096
    x = _logits(rng, 1, V, torch.float32, 1.0)
    u = (np.arange(R) + 0.5) / R
    tok = B.biloco_sample(x.cuda().expand(R, V), _dev(u)).cpu().numpy()
    share = torch.softmax(x[0].double(), 0).numpy() * R
    assert np.all(np.diff(tok) >= 0) and np.all(np.abs(np.bincount(tok, minlength=V) - share) <= 1.001)


def test_no_rows_and_no_logprob():
    assert B.biloco_sample(torch.empty((0, 9), device="cuda"), torch.empty(0, device="cuda")).shape == (0,)
    x = torch.zeros((2, 9), device="cuda")
    x[:, 4] = 50
    assert B.biloco_sample(x, torch.full((2,), 0.5, device="cuda")).tolist() == [4, 4]


@pytest.mark.parametrize("R,V", [(1, 50000), (40, 3000), (300, 9000)])
def test_captured(R, V):
    rng = np.random.default_rng(R)
    x = _logits(rng, R, V, torch.bfloat16).cuda()
    u, p = torch.rand(R, device="cuda"), torch.full((R,), 0.9, device="cuda")
    tok, lp = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    ws = torch.full((max(16, B.biloco_sample_workspace_bytes(R, V)),), 255, dtype=torch.uint8, device="cuda")
    kw = dict(top_p=p, token=tok, logprob=lp, workspace=ws)
    B.biloco_sample(x, u, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_sample(x, u, **kw)
    for i in range(4):
        x.copy_(_logits(np.random.default_rng(100 + i), R, V, torch.bfloat16))
        u.copy_(torch.rand(R))
        g.replay()
        got, got_lp = tok.clone(), lp.clone()
        other = torch.empty(R, device="cuda")
        want = B.biloco_sample(x, u, top_p=p, logprob=other)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_lp, other)


@pytest.mark.parametrize("dtype", DTYPES)
def test_slices_of_odd_rows(dtype):
    """Rows cut over several workgroups: ties, rows and slices without weight, one logit in
    the last slice, infinities, NaN."""
    rng = np.random.default_rng(7)
    R, V = 12, 60003
    x = torch.from_numpy(rng.integers(0, 3, (R, V)).astype(np.float32))
    x[1] = -float("inf")
    x[2] = float("nan")
    x[3] = -float("inf")
    x[3, V - 1] = 1.0
    x[4, [100, V - 2]] = float("inf")
    x[5, ::2] = float("nan")
    x[6, : V // 2] = -float("inf")
    x[7, 10:] = -200.0
    u = rng.random(R, np.float32)
    x = x.to(dtype)
    check(x, u)
    check(x, u, k=[1, 5, 5, 5, 1, 1025, 4000, 3, 20000, 20500, 59999, 60003])
    check(x, u, p=np.linspace(0.05, 0.97, R))
    check(x, u, t=[0.0, 1.0, 0.5, 0.0, 0.7, 2.0, 0.0, 1.0, 0.3, 1.5, 3.0, 0.0], p=[0.8] * R, m=[0.2] * R)
