"""Sampling of few long rows, which are cut into slices that meet in the workspace: two
streams at once, two graphs, a workspace's size, which the unsliced rows of
test_gpu_answer_streams.py do not touch."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

ROWS, V = 5, 60003


def _inputs(seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((ROWS, V), generator=g, device="cuda") * 3).to(dtype)
    return dict(logits=x, u=torch.rand(ROWS, generator=g, device="cuda"),
                top_p=torch.tensor([0.9, 0.5, 1.0, 0.999, 0.9], device="cuda"),
                top_k=torch.tensor([0, 40, 0, 5000, 3], dtype=torch.int32, device="cuda"),
                temperature=torch.tensor([1.0, 0.7, 0.0, 2.0, 1.5], device="cuda"))


def _call(d, **kw):
    lp = torch.empty(ROWS, device="cuda")
    return B.biloco_sample(**d, logprob=lp, **kw), lp


def test_the_workspace_is_used_and_no_more_than_said():
    d = _inputs(1)
    n = B.biloco_sample_workspace_bytes(ROWS, V)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    want, got = _call(d), _call(d, workspace=ws[:n])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((ws[:n] != 0xA5).any()) and bool((ws[n:] == 0xA5).all())
    # a row by itself, which is cut otherwise, gives the same
    for r in range(ROWS):
        lp = torch.empty(1, device="cuda")
        t = B.biloco_sample(**{k: v[r:r + 1].clone() for k, v in d.items()}, logprob=lp)
        assert torch.equal(t, want[0][r:r + 1]) and torch.equal(lp, want[1][r:r + 1])
    with pytest.raises(B.BilocoError, match="WORKSPACE"):
        _call(d, workspace=ws[:n - 16])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_streams_at_once(dtype):
    ds = [_inputs(3, dtype), _inputs(4, dtype)]
    want = [_call(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(8):
        turn = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                turn.append(_call(d))
        got.append(turn)
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs():
    """Two captured calls, their workspaces in the graphs' pools, replayed in turn on
    logits that change between the replays."""
    ds = [_inputs(5), _inputs(6)]
    for d in ds:
        _call(d)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_call(d))
        graphs.append(g)
    for turn in range(4):
        for i, d in enumerate(ds):
            d["logits"].copy_(_inputs(10 + 2 * turn + i)["logits"])
        for g in graphs:
            g.replay()
        want = [_call(d) for d in ds]      # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn
