"""The decoder-layer calls on a stream that is not the current one, and with
tensors of a GPU that is not: what a call allocates by itself comes from the stream
it runs on, whose memory no other stream's pending work can still be using;
tensors of another GPU than the current one are refused."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

pytestmark = pytest.mark.gpu


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = B.biloco_kv_cache(400, 2, 16, 64)
    for t in cache:
        t.fill_(0x38)
    return dict(cache=cache, q=rand(2, 16, 64), k=rand(2, 2, 64), v=rand(2, 2, 64), positions=ints(5, 6000)[None],
                cos_sin=torch.ones((6400, 64), device="cuda") * 0.7, q_start=ints(0, 1, 2), kv_len=ints(6, 3000),
                table=torch.arange(400, dtype=torch.int32, device="cuda").reshape(2, 200), x=rand(40, 512),
                w=rand(512))


CALLS = {
    "append": lambda d, **kw: [B.biloco_kv_append(d["cache"], d["q"], d["k"], d["v"], d["positions"], d["cos_sin"],
                                                  d["q_start"], d["kv_len"], d["table"], 1, **kw)],
    "attend": lambda d, **kw: [B.biloco_attn_paged(d["cache"], d["q"], d["q_start"], d["kv_len"], d["table"], 1, 3000,
                                                   0.125, **kw)],
    "norm": lambda d, **kw: list(B.biloco_norm_gate_residual(d["x"], d["x"], d["w"], **kw)),
}


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
    assert len(made) == {"append": 1, "attend": 2, "norm": 2}[name]      # the workspace among them
    assert [_pool_of(t) for t in made] == [s.cuda_stream] * len(made)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", ["current", "default number"])
def test_the_current_stream_by_name(name, stream):
    d = _inputs()
    want = CALLS[name](d)
    torch.cuda.synchronize()
    cur = torch.cuda.current_stream()
    got = CALLS[name](d, stream=cur if stream == "current" else cur.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b) and _pool_of(a) == cur.cuda_stream


@pytest.mark.parametrize("name", list(CALLS))
def test_another_gpu_than_the_current_one_is_refused(name, monkeypatch):
    d = _inputs()
    cur = torch.cuda.current_stream()
    monkeypatch.setattr(B, "_current_device", lambda: 1)      # as if GPU 1 were current
    kw = dict(stream=cur.cuda_stream)
    if name == "attend":
        kw.update(out=torch.empty_like(d["q"]), workspace=torch.empty(
            B.biloco_attn_workspace_bytes(2, 2, 16, 2, 64, 1, 3000), dtype=torch.uint8, device="cuda"))
    elif name == "append":
        kw.update(q_out=torch.empty_like(d["q"]))
    else:
        kw.update(res_out=torch.empty_like(d["x"]), h=torch.empty_like(d["x"]))
    with pytest.raises(ValueError, match="current GPU"):
        CALLS[name](d, **kw)
    monkeypatch.undo()
    CALLS[name](d, **kw)
