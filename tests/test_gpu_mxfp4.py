"""biloco_quant_mxfp4, biloco_dequant_mxfp4 and the products of such rows, against the
64-bit forms.

Tolerances.  Codes, scales and values are exact.  A product's terms are exact in fp32;
a matrix instruction adds at least 64 of them to a sum and truncates to 24 bits (2^-23
of what it adds, at most); pieces' and waves' sums add at most 64 roundings more:
  |y - y64| <= (K / 64 + 64) 2^-23 sum |a w|, and 2^-8 |y64| for y in bf16 (2^-24 in fp32).
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from oracle import answers

pytestmark = pytest.mark.gpu


def _rows(rng, M, K, dtype=torch.bfloat16):
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 12, (M, 1))) * np.exp2(rng.integers(-6, 6, (1, K)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _same(x, want):
    assert torch.equal(x.cpu(), torch.from_numpy(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,pitch", [(1, 32, 32), (3, 64, 64), (7, 96, 104), (33, 256, 256), (5, 4064, 4096), (300, 544, 544)])
def test_quantise(dtype, M, K, pitch):
    x = _rows(np.random.default_rng(M), M, pitch, dtype).cuda()[:, :K]
    codes, scales = B.biloco_quant_mxfp4(x)
    c, s = answers.quant_mxfp4(x.double().cpu().numpy())
    _same(codes, c)
    _same(scales, s)
    want = torch.from_numpy(answers.values_mxfp4(c, s))
    wide = torch.full((M, pitch), 7.0, dtype=dtype, device="cuda")
    B.biloco_dequant_mxfp4(codes, scales, out=wide[:, :K])
    assert torch.equal(wide[:, :K].double().cpu(), want) and bool((wide[:, K:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_borders(dtype):
    """Every middle between two codes and its neighbours, at scales from the smallest to the largest."""
    near = np.array([0, 0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.96875])
    info = torch.finfo(dtype)
    rows = []
    for e in (0, 1, 2, 60, 125, 126, 127, 128, 200, 251, 252):
        for step in (-1, 0, 1):
            y = np.concatenate([near * (1 + step * info.eps), -near * (1 + step * info.eps), [4.0, -0.0] * 4])
            rows.append(y * 2.0 ** (e - 127))
    x = torch.from_numpy(np.array(rows)).to(dtype)      # subnormal ones are rounded here
    codes, scales = B.biloco_quant_mxfp4(x.cuda())
    c, s = answers.quant_mxfp4(x.double().numpy())
    _same(codes, c)
    _same(scales, s)
    got = B.biloco_dequant_mxfp4(codes, scales, out_dtype=dtype).double().cpu().numpy()
    np.testing.assert_array_equal(got, answers.values_mxfp4(c, s))      # the last block's largest is infinite: NaN


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_that_are_not_finite_or_zero(dtype):
    x = torch.ones((4, 96), dtype=dtype)
    x[0, 40], x[1, 0], x[2, 95] = float("nan"), float("inf"), -float("inf")
    x[3, :64] = 0.0
    x[3, 1] = -0.0
    codes, scales = B.biloco_quant_mxfp4(x.cuda())
    c, s = answers.quant_mxfp4(x.double().numpy())
    _same(codes, c)
    _same(scales, s)
    v = B.biloco_dequant_mxfp4(codes, scales).double().cpu().numpy()
    np.testing.assert_array_equal(v, answers.values_mxfp4(c, s))


def test_values_of_every_byte():
    codes = torch.arange(256, dtype=torch.uint8).reshape(16, 16)
    for e in (0, 1, 2, 126, 127, 128, 252, 253, 254, 255):
        s = torch.full((16, 1), e, dtype=torch.uint8)
        want = answers.values_mxfp4(codes.numpy(), s.numpy())
        for dtype in (torch.bfloat16, torch.float32):
            with np.errstate(over="ignore"):
                limited = want.astype(np.float32).astype(np.float64)      # past the range: infinite in both types
            got = B.biloco_dequant_mxfp4(codes.cuda(), s.cuda(), out_dtype=dtype).double().cpu().numpy()
            np.testing.assert_array_equal(got, limited)


def _operands(seed, M, N, K):
    rng = np.random.default_rng(seed)
    x, w = _rows(rng, M, K).cuda(), _rows(rng, N, K, torch.float32).cuda()
    return x, B.biloco_quant_mxfp4(x), B.biloco_quant_mxfp4(w)


def _compare(y, a, w):
    want, mag = answers.gemm_mxfp4(*((c.cpu().numpy(), s.cpu().numpy()) for c, s in (a, w)))
    K = 2 * a[0].shape[1]
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bound = (K / 64 + 64) * 2.0 ** -23 * mag + np.abs(want) * (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24)
    ok = ~np.isnan(want)
    worst = (np.abs(got - want)[ok] - bound[ok]).max() if ok.any() else 0.0
    assert worst <= 0, worst


@pytest.mark.parametrize("K", [32, 64, 96, 224, 256, 288, 480, 512, 544, 1024, 1312, 4096, 5120])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 32])
def test_few_rows(M, K):
    x, a, w = _operands(K + M, M, 77, K)
    for dtype in (torch.float32, torch.bfloat16):
        _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=dtype), a, w)
    assert torch.equal(B.biloco_gemm_mxfp4(*a, *w), B.biloco_gemm_mxfp4_quant(x, *w))


@pytest.mark.parametrize("N", [1, 15, 16, 31, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("M", [1, 9, 33, 64, 65, 128, 130, 257])
def test_rows_and_columns(M, N):
    K = 288
    x, a, w = _operands(M * N, M, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=dtype), a, w)


@pytest.mark.parametrize("M,N,K", [(33, 77, 32), (40, 200, 96), (48, 130, 256), (100, 100, 544), (70, 512, 2560), (200, 320, 5152),
                                   (200, 640, 13824), (129, 1000, 4096), (600, 900, 2080), (1025, 4100, 352)])
def test_many_rows(M, N, K):
    x, a, w = _operands(M + N + K, M, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=dtype), a, w)
    assert torch.equal(B.biloco_gemm_mxfp4(*a, *w), B.biloco_gemm_mxfp4_quant(x, *w))


@pytest.mark.parametrize("M,N,K", [(4200, 4111, 288), (4096, 4096, 512), (8200, 2100, 800)])
def test_large_tiles(M, N, K):
    x, a, w = _operands(M, M, N, K)
    _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32), a, w)
    _compare(B.biloco_gemm_mxfp4_quant(x, *w), a, w)


@pytest.mark.parametrize("M,N,K", [(1, 50, 96), (20, 40, 1024), (40, 77, 544), (300, 200, 256), (200, 160, 8192)])
@pytest.mark.parametrize("gap", [1, 7, 8, 64])
def test_rows_apart(M, N, K, gap):
    """x, a slice of wider rows; y, whose rows lie apart, is written nowhere else."""
    rng = np.random.default_rng(gap)
    x = _rows(rng, M, K + 64).cuda()[:, 24:K + 24]
    w = B.biloco_quant_mxfp4(_rows(rng, N, K, torch.float32).cuda())
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((M + 1, N + gap), 5.0, dtype=dtype, device="cuda")
        B.biloco_gemm_mxfp4_quant(x, *w, y=y[:M, :N])
        assert bool((y[:, N:] == 5).all()) and bool((y[M] == 5).all())
        _compare(y[:M, :N], B.biloco_quant_mxfp4(x), w)


@pytest.mark.parametrize("M,N,K", [(1, 40, 544), (20, 40, 544), (40, 70, 544), (200, 300, 8192)])
def test_nan_blocks(M, N, K):
    x, a, w = _operands(5, M, N, K)
    a[1][M // 2, K // 32 - 1] = 255
    w[1][N - 3, 0] = 255
    y = B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32)
    _compare(y, a, w)
    assert bool(y[M // 2].isnan().all()) and bool(y[:, N - 3].isnan().all())
    assert int(y.isnan().sum()) == M + N - 1


@pytest.mark.parametrize("M,N,K", [(5, 33, 288), (150, 200, 4096)])
def test_scales_far_apart(M, N, K):
    """Products near the ends of fp32's range."""
    x, a, w = _operands(8, M, N, K)
    a[1][:] = torch.randint(170, 180, a[1].shape, dtype=torch.uint8)
    w[1][:] = torch.randint(180, 190, w[1].shape, dtype=torch.uint8)
    _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32), a, w)
    a[1][:] = torch.randint(70, 80, a[1].shape, dtype=torch.uint8)
    w[1][:] = torch.randint(75, 85, w[1].shape, dtype=torch.uint8)
    _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32), a, w)


def test_one_workspace_serves_fewer_rows():
    N, K = 200, 4096
    ws = torch.full((B.biloco_gemm_mxfp4_workspace_bytes(400, N, K),), 255, dtype=torch.uint8, device="cuda")
    for M in (400, 1, 129, 32, 33, 300, 128):
        x, a, w = _operands(M, M, N, K)
        _compare(B.biloco_gemm_mxfp4_quant(x, *w, workspace=ws), a, w)
        _compare(B.biloco_gemm_mxfp4(*a, *w, workspace=ws), a, w)


def test_no_rows():
    w = B.biloco_quant_mxfp4(torch.ones((40, 64), device="cuda"))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    a = B.biloco_quant_mxfp4(x)
    assert a[0].shape == (0, 32) and a[1].shape == (0, 2)
    assert B.biloco_dequant_mxfp4(*a).shape == (0, 64)
    assert B.biloco_gemm_mxfp4(*a, *w).shape == (0, 40) and B.biloco_gemm_mxfp4_quant(x, *w).shape == (0, 40)


def test_results_do_not_change_between_runs():
    x, a, w = _operands(3, 200, 300, 8192)
    first = B.biloco_gemm_mxfp4_quant(x, *w)
    for _ in range(5):
        assert torch.equal(first, B.biloco_gemm_mxfp4_quant(x, *w))


@pytest.mark.parametrize("M", [4, 200])
def test_captured(M):
    N, K = 320, 4096
    x, a, w = _operands(11, M, N, K)
    y, ws = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty(
        B.biloco_gemm_mxfp4_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    B.biloco_gemm_mxfp4_quant(x, *w, y=y, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.biloco_gemm_mxfp4_quant(x, *w, y=y, workspace=ws)
    for i in range(3):
        x.copy_(_rows(np.random.default_rng(i), M, K).cuda())
        y.zero_()
        g.replay()
        want = B.biloco_gemm_mxfp4_quant(x, *w)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("K", [512, 1536, 5120])
@pytest.mark.parametrize("M", [1, 3, 6, 17, 32])
def test_few_rows_many_columns(M, K):
    """Several tiles a CU, some of them cut between waves; a NaN in the last block of one
    row of W and of A's last row stays in that column and row."""
    N = 16 * 256 * 2 + 16 * 77 + 5
    x, a, w = _operands(K + M, M, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=dtype), a, w)
    assert torch.equal(B.biloco_gemm_mxfp4(*a, *w), B.biloco_gemm_mxfp4_quant(x, *w))
    x[M - 1, K - 1] = float("inf")
    w[1][N - 3, K // 32 - 1] = 255
    y = B.biloco_gemm_mxfp4_quant(x, *w)
    assert bool(y[M - 1].isnan().all()) and bool(y[:, N - 3].isnan().all())
    y[M - 1], y[:, N - 3] = 0, 0
    assert not bool(y.isnan().any())


@pytest.mark.parametrize("M,K", [(16, 16384), (17, 8192), (32, 7168), (32, 8192)])
def test_few_long_rows(M, K):
    """On both sides of what a CU's LDS holds."""
    x, a, w = _operands(K, M, 200, K)
    _compare(B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32), a, w)
    assert torch.equal(B.biloco_gemm_mxfp4(*a, *w), B.biloco_gemm_mxfp4_quant(x, *w))


@pytest.mark.parametrize("M,N,K", [(33, 40, 992), (64, 300, 5152), (130, 129, 1056), (200, 320, 13856), (300, 600, 3040),
                                   (4100, 4100, 1120), (257, 100, 16352)])
def test_rows_of_scales_at_any_address(M, N, K):
    """K / 32 no multiple of 4 or of 32: the last of a row's blocks next to the following
    row's, whose scales are NaN."""
    x, a, w = _operands(K, M, N, K)
    a[1][M // 2, 0] = 255
    w[1][N // 2, 0] = 255
    y = B.biloco_gemm_mxfp4(*a, *w, out_dtype=torch.float32)
    _compare(y, a, w)
    whole = torch.arange(M, device="cuda") != M // 2
    assert not bool(y[whole][:, torch.arange(N, device="cuda") != N // 2].isnan().any())
