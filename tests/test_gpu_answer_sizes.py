"""The calls for several answers to one prompt at sizes past what one launch or 32 bits
take: millions of rows or columns, operands and outputs of more than 4 GiB.  Rows and
columns repeat, so that a small call's results are what is wanted of all of them."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu


def _gen(seed=1):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weight(gen, rows, K):
    return (torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8),
            torch.randint(120, 131, (rows, K // 32), generator=gen, device="cuda", dtype=torch.uint8))


def _repeats(y, want, dim=0):
    """y along dim is `want` over and over."""
    n, at = want.shape[dim], 0
    while at < y.shape[dim]:
        part = y.narrow(dim, at, min(64 * n, y.shape[dim] - at))
        times = -(-part.shape[dim] // n)
        assert torch.equal(part, torch.cat([want] * times, dim).narrow(dim, 0, part.shape[dim])), at
        at += part.shape[dim]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_of_millions_of_rows(dtype):
    g, n, V = _gen(), (1 << 22) + 3, 8
    x = torch.randn((4096, V), generator=g, device="cuda").to(dtype)
    u, p, k = (f((4096,), generator=g, device="cuda") for f in (torch.rand, torch.rand, torch.rand))
    t, k = 0.2 + k, (k * 6).to(torch.int32)

    def call(r):
        lp = torch.full((r,), 9.0, device="cuda")
        times = -(-r // 4096)
        return B.biloco_sample(x.repeat(times, 1)[:r], u.repeat(times)[:r], t.repeat(times)[:r], k.repeat(times)[:r],
                               p.repeat(times)[:r], logprob=lp), lp
    want, got = call(4096), call(n)
    for a, b in zip(got, want):
        _repeats(a, b)


@pytest.mark.parametrize("M,N,dtype", [(1, (1 << 27) + 5, torch.bfloat16), (20, (1 << 28) + 37, torch.bfloat16)])
def test_few_rows_to_millions_of_columns(M, N, dtype):
    g, K = _gen(), 32
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = _weight(g, 1 << 16, K)
    want = B.biloco_gemm_mxfp4_quant(x, *w, out_dtype=dtype)
    times = -(-N // (1 << 16))
    got = B.biloco_gemm_mxfp4_quant(x, *(t.repeat(times, 1)[:N] for t in w), out_dtype=dtype)
    assert bool(want.isfinite().all()) and int(want.count_nonzero()) > 0
    _repeats(got, want, 1)


# ---------------------------------------------------------------- more than 4 GiB

def _tiled(t, rows):
    """t's rows over and over."""
    return t.repeat(-(-rows // t.shape[0]), 1)[:rows]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [0, 32])
def test_quantised_rows_and_back(dtype, gap):
    g, rows, K = _gen(), (1 << 20) + 77, 2080
    x = torch.randn((4096, K + gap), generator=g, device="cuda").to(dtype)
    want = B.biloco_quant_mxfp4(x[:, :K])
    got = B.biloco_quant_mxfp4(_tiled(x, rows)[:, :K])
    for a, b in zip(got, want):
        _repeats(a, b)
    out = torch.zeros((rows, K + gap), dtype=dtype, device="cuda")
    B.biloco_dequant_mxfp4(*got, out=out[:, :K])
    _repeats(out[:, :K], B.biloco_dequant_mxfp4(*want, out_dtype=dtype))
    assert not bool(out[:, K:].any())


@pytest.mark.parametrize("M,K", [(5, 8224), (32, 8192), (40, 8224), (300, 8192)])
def test_weights(M, K):
    """In LDS, streamed and tiled; rows of scales that have to be padded."""
    g, N = _gen(), (1 << 20) + 77
    a, w = _weight(g, M, K), _weight(g, 8192, K)
    got = B.biloco_gemm_mxfp4(*a, *(_tiled(t, N) for t in w), out_dtype=torch.float32)
    want = torch.cat([B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32)] * 2, 1)
    # one order of sums for every number of columns, but for K in pieces (as for few tiles)
    if M > 32:
        assert torch.allclose(got[:, :8192], want[:, :8192], rtol=1e-4, atol=float(want.abs().max()) * 1e-5)
        want = got[:, :8192].clone()
    _repeats(got, want[:, :8192].contiguous(), 1)


def test_rows_of_a_product():
    g, M, K, N = _gen(), (1 << 20) + 77, 8224, 70
    a, w = _weight(g, 8192, K), _weight(g, N, K)
    got = B.biloco_gemm_mxfp4(*(_tiled(t, M) for t in a), *w)
    _repeats(got, got[:8192].clone())
    few = B.biloco_gemm_mxfp4(*(t[:200] for t in a), *w)
    assert torch.allclose(got[:200].float(), few.float(), rtol=2.0 ** -7, atol=float(few.float().abs().max()) * 1e-5)


def test_results_of_a_product():
    g, M, N, K = _gen(), 70001, 40003, 64
    a, w = _weight(g, 8192, K), _weight(g, N, K)
    got = B.biloco_gemm_mxfp4(*(_tiled(t, M) for t in a), *w, out_dtype=torch.float32)
    want = B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32)
    for at in range(0, M, 8192):
        n = min(8192, M - at)
        assert torch.equal(got[at:at + n], want[:n]), at


@pytest.mark.parametrize("V", [30000, 1000003])      # a workgroup a row, and slices
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_logits_far_apart(V, dtype):
    g, far = _gen(), (1 << 30) - 3
    x = (torch.randn((3, V), generator=g, device="cuda") * 3).to(dtype)
    room = torch.empty(2 * far + V, dtype=dtype, device="cuda")
    rows = room.as_strided((3, V), (far, 1))
    rows.copy_(x)
    u, p = torch.rand(3, generator=g, device="cuda"), torch.tensor([0.9, 1.0, 0.5], device="cuda")
    lp = [torch.empty(3, device="cuda") for _ in range(2)]
    assert torch.equal(B.biloco_sample(rows, u, top_p=p, logprob=lp[0]), B.biloco_sample(x, u, top_p=p, logprob=lp[1]))
    assert torch.equal(*lp)


@pytest.mark.parametrize("dim", [64, 128])
def test_shared_attention(dim):
    """Pages at the end of a cache of more than 4 GiB; rows of q and o that lie far apart."""
    from test_gpu_attn_shared import Case
    c = Case([(300, [(1, 301), (3, 350), (2, 700)]), (64, [(1, 65)] * 3)], 16, 4, dim, 64, seed=dim)
    a = list(c.args())
    lse = [torch.empty((c.T, c.hq), device="cuda") for _ in range(2)]
    want = B.biloco_attn_shared(*a, lse=lse[0])
    pool = a[0][0].shape[0]
    pages = (1 << 32) // (4 * 64 * dim) + 100
    big = []
    for t in a[0]:
        b = torch.full((pages,) + t.shape[1:], 0x7F, dtype=torch.uint8, device="cuda")
        b[-pool:] = t
        big.append(b)
    a[0], a[4] = tuple(big), torch.where(a[4] >= 0, a[4] + pages - pool, a[4])
    far = 1 << 28
    q, o = (torch.zeros(far * (c.T - 1) + c.hq * dim, dtype=torch.bfloat16, device="cuda").as_strided(
        (c.T, c.hq, dim), (far, dim, 1)) for _ in range(2))
    q.copy_(a[1])
    a[1] = q
    got = B.biloco_attn_shared(*a, lse=lse[1], out=o)
    assert torch.equal(got, want) and torch.equal(*lse)
