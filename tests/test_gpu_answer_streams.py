"""The calls for several answers to one prompt on a stream that is not the current one,
with tensors of a GPU that is not, by two streams at once and from two graphs with
workspaces of their own, and their refusal of small workspaces."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu


def _inputs(seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = B.biloco_kv_cache(400, 2, 16, 64)
    for t in cache:
        t.fill_(0x38)
    cache[0].copy_(torch.randint(0x20, 0x50, cache[0].shape, generator=g, device="cuda", dtype=torch.uint8))
    x, w = rand(200, 2048).to(torch.bfloat16), B.biloco_quant_mxfp4(rand(320, 2048))
    return dict(cache=cache, q=rand(3, 16, 64).to(torch.bfloat16), q_start=ints(0, 1, 2, 3), kv_len=ints(1500, 3000, 1400),
                table=torch.arange(600, dtype=torch.int32, device="cuda").reshape(3, 200) % 400, groups=ints(0, 2, 3),
                shared=ints(1400, 100), x=x, w=w, a=B.biloco_quant_mxfp4(x), logits=rand(5, 20000) * 3,
                u=torch.rand(5, generator=g, device="cuda"), top_p=torch.full((5,), 0.9, device="cuda"))


CALLS = {
    "quant": lambda d, **kw: list(B.biloco_quant_mxfp4(d["x"], **kw)),
    "dequant": lambda d, **kw: [B.biloco_dequant_mxfp4(*d["w"], **kw)],
    "product": lambda d, **kw: [B.biloco_gemm_mxfp4(*d["a"], *d["w"], **kw)],
    "product of rows": lambda d, **kw: [B.biloco_gemm_mxfp4_quant(d["x"], *d["w"], **kw)],
    "few rows": lambda d, **kw: [B.biloco_gemm_mxfp4_quant(d["x"][:3], *d["w"], **kw)],
    "shared": lambda d, **kw: [B.biloco_attn_shared(d["cache"], d["q"], d["q_start"], d["kv_len"], d["table"], d["groups"],
                                                    d["shared"], 1, 3000, 1400, 0.125, **kw)],
    "sample": lambda d, **kw: [B.biloco_sample(d["logits"], d["u"], top_p=d["top_p"], **kw)],
}
MADE = {"quant": 2, "dequant": 1, "product": 2, "product of rows": 2, "few rows": 2, "shared": 2, "sample": 2}


def _pool_of(t):
    """The stream whose allocations t's memory belongs to."""
    at = t.untyped_storage().data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("as_number", [False, True])
def test_allocations_belong_to_the_stream(name, as_number, monkeypatch):
    d = _inputs()
    want = CALLS[name](d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    made, empty = [], torch.empty

    def noted(*a, **kw):
        t = empty(*a, **kw)
        made.append(t)
        return t
    monkeypatch.setattr(torch, "empty", noted)
    got = CALLS[name](d, stream=s.cuda_stream if as_number else s)
    monkeypatch.undo()
    s.synchronize()
    assert torch.cuda.current_stream().cuda_stream != s.cuda_stream
    assert len(made) == MADE[name]      # the workspace among them
    assert [_pool_of(t) for t in made] == [s.cuda_stream] * len(made)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", list(CALLS))
def test_another_gpu_than_the_current_one_is_refused(name, monkeypatch):
    d = _inputs()
    cur = torch.cuda.current_stream()
    outs = [torch.empty_like(t) for t in CALLS[name](d)]
    space = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    kw = dict(quant=lambda: dict(codes=outs[0], scales=outs[1]), dequant=lambda: dict(out=outs[0]),
              shared=lambda: dict(out=outs[0], workspace=space), sample=lambda: dict(token=outs[0], workspace=space)).get(
                  name, lambda: dict(y=outs[0], workspace=space))()
    monkeypatch.setattr(B, "_current_device", lambda: 1)      # as if GPU 1 were current
    with pytest.raises(ValueError, match="current GPU"):
        CALLS[name](d, stream=cur.cuda_stream, **kw)
    monkeypatch.undo()
    CALLS[name](d, stream=cur.cuda_stream, **kw)


@pytest.mark.parametrize("name", list(CALLS))
def test_two_streams_at_once(name):
    """Calls of other data on two streams, each with what it allocates, over and over."""
    ds = [_inputs(3), _inputs(4)]
    want = [CALLS[name](d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(8):
        got.append([CALLS[name](d, stream=s) for d, s in zip(ds, streams)])
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", list(CALLS))
def test_two_graphs(name):
    """Two captured calls, their workspaces in the graphs' pools, replayed in turn."""
    ds = [_inputs(3), _inputs(4)]
    want = [CALLS[name](d) for d in ds]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(CALLS[name](d))
        graphs.append(g)
    for turn in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs:
            g.replay()
        CALLS[name](ds[turn % 2])      # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn


def test_small_workspaces_are_refused():
    d = _inputs()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for name in ("product", "product of rows", "shared", "sample"):
        with pytest.raises(B.BilocoError, match="WORKSPACE|workspace"):
            CALLS[name](d, workspace=small)
