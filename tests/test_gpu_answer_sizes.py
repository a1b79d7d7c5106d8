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
