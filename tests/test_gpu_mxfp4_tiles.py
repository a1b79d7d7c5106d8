"""Products of many rows by the kernel that takes them: tiles of 256, tiles of 128, and
tiles of 128 with K in pieces (test_mx_plan_host.py says that these sizes reach them), with
rows, columns and k past the last whole tile, one group of stages and more, NaN blocks at
the ends, rows of y that lie apart.

Against float64 sums of the exact products; tolerance as in test_gpu_mxfp4.py:
  |y - y64| <= (K / 64 + 64) 2^-23 sum |a w| + half a step of y's type.
"""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

LARGE = [(3900, 4001, 288), (3900, 4001, 1120), (3841, 4096, 2080), (4096, 3850, 4096), (3585, 3900, 32), (5000, 6100, 1024),
         (4500, 3400, 5152), (257, 27000, 3200), (27001, 500, 2048)]
SMALL = [(4200, 4111, 288), (8200, 2100, 800), (2001, 2300, 1184), (2100, 2049, 4096), (129, 33000, 160), (1920, 2176, 1024)]
PIECES = [(100, 500, 13824), (600, 1000, 2080), (129, 1000, 4096), (33, 77, 8192), (1000, 1111, 3104)]


def _values(codes, scales):
    t = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    t = torch.cat([t, -t])
    v = torch.stack([t[(codes & 15).int()], t[(codes >> 4).int()]], -1).flatten(1)
    s = torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127))
    return (v.unflatten(1, (-1, 32)) * s[..., None]).flatten(1)


def _compare(y, a, w):
    a, w = _values(*a), _values(*w)
    want, mag = a @ w.T.contiguous(), a.abs() @ w.abs().T.contiguous()
    assert torch.equal(y.isnan(), want.isnan())
    bound = (a.shape[1] / 64 + 64) * 2.0 ** -23 * mag + want.abs() * (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24)
    over = ((y.double() - want).abs() - bound).nan_to_num(-1.0)
    assert float(over.max()) <= 0, float(over.max())


@pytest.mark.parametrize("M,N,K", LARGE + SMALL + PIECES)
def test_tiles(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randn((M, K), generator=g, device="cuda")
    x = (x * (1 + 7 * (torch.rand((K,), generator=g, device="cuda") < 0.03))).to(torch.bfloat16)
    a = B.biloco_quant_mxfp4(x)
    w = B.biloco_quant_mxfp4(torch.randn((N, K), generator=g, device="cuda") * K ** -0.5)
    y = torch.full((M + 1, N + 3), 5.0, device="cuda")
    B.biloco_gemm_mxfp4(*a, *w, y=y[:M, :N])
    assert bool((y[M] == 5).all()) and bool((y[:, N:] == 5).all())
    _compare(y[:M, :N], a, w)
    z = B.biloco_gemm_mxfp4_quant(x, *w)
    assert torch.equal(z, y[:M, :N].to(torch.bfloat16))
    # NaN blocks: the last rows, the last blocks, the first ones
    for t, n in ((a, M), (w, N)):
        t[1][n - 1, K // 32 - 1], t[1][n // 2, 0], t[1][n - 2, K // 64] = 255, 255, 255
    B.biloco_gemm_mxfp4(*a, *w, y=y[:M, :N])
    assert int(y[:M, :N].isnan().sum()) == 3 * (M + N) - 9
    _compare(y[:M, :N], a, w)
