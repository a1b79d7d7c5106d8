"""Cases of the operators by which a program answers one prompt several times.

Four operators of that serving loop, each in a plain form of elementary torch
operations (``own = False``) and through the framework's entry points
(``own = True``):

* ``quant``: rows to microscaled 4-bit floats (E2M1 codes, one power-of-two scale
  for 32 of them) and back to the values that these stand for;
* ``product``: rows quantised that way times a weight that is kept that way, for one
  row, a decode batch's logits, and whole prompts;
* ``shared``: attention over the paged 8-bit cache for a batch whose sequences share
  their first tokens in groups, which are read once for the group;
* ``sample``: a token for each row of logits, by temperature, top-k, top-p and
  min-p, from a given random number.

Layouts (those of the entry points):
  codes [rows][K/2], two a byte, the even k in the low nibble; scales
  [rows][K/32]: the byte b stands for 2^(b - 127).
  k_codes [pages][kv_heads][page][dim], v_codes [pages][kv_heads][page/8][dim][8],
  k_scales and v_scales [pages][kv_heads], powers of two likewise.  Sequence b's new
  tokens are rows q_start[b] .. q_start[b+1], the last of its kv_len[b] tokens; token
  a is slot a % page of page block_table[b][a // page].  Sequences group_start[g] ..
  group_start[g+1] - 1 share their first shared_len[g] tokens.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the rows of a decode batch, slices of a wider product's: latency
        dict(name="quantise decode rows", op="quant", rows=32, K=5120, pad=2560, type="bf16"),
        # a layer's weight as a program that loads it quantises it
        dict(name="quantise a weight", op="quant", rows=13824, K=5120, pad=0, type="f32"),
        # one token through a wide layer: latency and the weight's bytes
        dict(name="product, one row", op="product", M=1, N=13824, K=5120, out="bf16"),
        # the logits of a decode batch, an odd number of them
        dict(name="product, logits", op="product", M=32, N=100001, K=5120, out="f32"),
        # what is left of a prompt behind a shared part: too many rows for a decode
        # product, few for a prompt's
        dict(name="product, short prompt", op="product", M=200, N=5120, K=13824, out="bf16"),
        # a whole prompt
        dict(name="product, prompt", op="product", M=4096, N=8192, K=8192, out="bf16"),
        # few answers of a short prompt, no shared heads: latency
        dict(name="shared, four answers", op="shared", batch=4, groups=1, q_max=1, shared=608, own=29, heads=40,
             kv_heads=40, dim=128, page=16, window=0, sinks=0, lens=1),
        # several prompts answered at once with drafted tokens, ragged, heads of 64
        dict(name="shared, groups and drafts", op="shared", batch=24, groups=3, q_max=5, shared=6000, own=700,
             heads=64, kv_heads=8, dim=64, page=32, window=0, sinks=0, lens=2),
        # many answers of one long prompt
        dict(name="shared, many answers", op="shared", batch=64, groups=1, q_max=1, shared=16384, own=1024, heads=64,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, lens=3),
        # one request's token: latency
        dict(name="sample one row", op="sample", rows=1, V=32000, type="f32", temperature="one", k="some", p="some",
             min_p="none"),
        # a decode batch, each request with its own settings, greedy ones among them
        dict(name="sample decode batch", op="sample", rows=32, V=100001, type="f32", temperature="mixed", k="mixed",
             p="mixed", min_p="mixed"),
        # many answers at once, the nucleus of wide logits
        dict(name="sample many rows", op="sample", rows=256, V=128000, type="bf16", temperature="mixed", k="none",
             p="some", min_p="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "shared", "shared", "sample", "sample"])
    if op == "quant":
        K = 32 * _log(rng, 1, 512)
        return dict(op=op, rows=_log(rng, 1, min(65536, 13824 * 5120 // K)), K=K, pad=rng.choice([0, 0, 8 * _log(rng, 1, 512)]),
                    type=rng.choice(["bf16", "f32"]))
    if op == "product":
        K = 32 * _log(rng, 1, 512)
        N = _log(rng, 1, min(131072, 100001 * 5120 // K))
        M = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 64), _log(rng, 64, 8192)])
        M = max(1, min(M, 4096 * 8192 * 8192 // (N * K), 4096 * 8192 // N))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "f32"]))
    if op == "sample":
        V = _log(rng, 2, 262144)
        pick = lambda *a: rng.choice(a)  # noqa: E731
        kind = pick("bf16", "f32")
        most = 256 * 128000 // (V if kind == "bf16" else 2 * V)
        return dict(op=op, rows=_log(rng, 1, max(1, min(512, most))), V=V, type=kind,
                    temperature=pick("one", "mixed"), k=pick("none", "some", "mixed"), p=pick("none", "some", "mixed"),
                    min_p=pick("none", "some", "mixed"))
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10, 40])
    heads = kv_heads * rng.choice([1, 2, 5, 8] if kv_heads <= 10 else [1])
    dim = rng.choice([64, 128, 128])
    batch = _log(rng, 1, 64)
    q_max = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 8, 64)])
    shared, mine = _log(rng, 1, 32768), _log(rng, 1, 4096)
    # no more cached data and no more products than the largest listed case has
    groups = rng.choice([1, 1, rng.randint(1, min(batch, 6))])
    while (batch * (shared + mine + q_max) * kv_heads * dim > 64 * 17408 * 8 * 128 or
           (groups * shared + batch * mine) * kv_heads * dim > 28000 * 8 * 128):
        batch, shared, mine = (batch + 1) // 2, (shared + 1) // 2, (mine + 1) // 2
    while q_max > 1 and batch * q_max * (shared + mine + q_max) * heads * dim > 64 * 17408 * 64 * 128:
        q_max = (q_max + 1) // 2
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    return dict(op=op, batch=batch, groups=min(batch, groups), q_max=q_max, shared=shared,
                own=mine, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]), window=window,
                sinks=rng.choice([0, 4, rng.randint(1, 64)]) if window else 0, lens=rng.randrange(1 << 30))


def _batch(case):
    """(new tokens, tokens with them, group) of each sequence, shared tokens of each group: whole pages."""
    rng, page, groups = random.Random(case["lens"]), case["page"], case["groups"]
    shared = [case["shared"] if g == 0 else _log(rng, 1, case["shared"]) for g in range(groups)]
    shared = [n // page * page for n in shared]
    group = sorted(list(range(groups)) + [rng.randrange(groups) for _ in range(case["batch"] - groups)])
    new, kv = [], []
    for b, g in enumerate(group):
        n = case["q_max"] if b == 0 else rng.randint(1, case["q_max"])
        new.append(n)
        kv.append(shared[g] + n + (case["own"] if b == 0 else _log(rng, 1, case["own"] + 1) - 1))
    return new, kv, group, shared


# ------------------------------------------------------------------ inputs

def _rows(gen, rows, K, dtype, pitch=None):
    """Activations with a few strong channels, or a weight; optionally rows of a wider array."""
    x = torch.randn((rows, pitch or K), generator=gen, device=DEV)
    x *= 1.0 + 7.0 * (torch.rand((x.shape[1],), generator=gen, device=DEV) < 0.03)
    return x.to(dtype)[:, :K]


def _weight(gen, N, K):
    """Codes and scales of a weight."""
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((N, K // 32), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // K)
    for at in range(0, N, step):
        w = torch.randn((min(step, N - at), K), generator=gen, device=DEV) * (K ** -0.5)
        codes[at:at + step], scales[at:at + step] = _quantise(w)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "quant":
        r, K = case["rows"], case["K"]
        s["x"] = _rows(gen, r, K, torch.float32 if case["type"] == "f32" else torch.bfloat16, K + case["pad"])
        s["codes"] = torch.empty((r, K // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((r, K // 32), dtype=torch.uint8, device=DEV)
        s["values"] = torch.empty((r, K), dtype=torch.bfloat16, device=DEV)
        return s
    if case["op"] == "product":
        s["x"] = _rows(gen, case["M"], case["K"], torch.bfloat16)
        s["w_codes"], s["w_scales"] = _weight(gen, case["N"], case["K"])
        s["y"] = torch.empty((case["M"], case["N"]), device=DEV,
                             dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
        return s
    if case["op"] == "sample":
        return _prepare_sample(s, case, gen)
    new, kv, group, shared = _batch(case)
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    own_pages = [-(-(n - shared[g]) // page) for n, g in zip(kv, group)]
    total = sum(n // page for n in shared) + sum(own_pages)
    pool = total + total // 16 + 1
    order = torch.randperm(pool, generator=gen, device=DEV)[:total].to(torch.int32)
    table = torch.full((len(kv), max(-(-n // page) for n in kv)), -1, dtype=torch.int32, device=DEV)
    at, first = 0, []
    for n in shared:
        first.append(order[at:at + n // page])
        at += n // page
    for b, (g, n) in enumerate(zip(group, own_pages)):
        table[b, :len(first[g])] = first[g]
        table[b, len(first[g]):len(first[g]) + n] = order[at:at + n]
        at += n
    start = [0]
    for n in new:
        start.append(start[-1] + n)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    s.update(q_start=ints(start), kv_len=ints(kv), block_table=table, shared_len=ints(shared),
             group_start=ints([sum(g < i for g in group) for i in range(len(shared) + 1)]), tokens=start[-1],
             max_q=max(new), max_kv=max(kv), max_shared=max(shared), scale=d ** -0.5)
    for name, shape in (("k_codes", (pool, hk, page, d)), ("v_codes", (pool, hk, page // 8, d, 8))):
        x = torch.randn(shape, generator=gen, device=DEV).mul_(90.0).clamp_(-448.0, 448.0)
        s[name] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    for name in ("k_scales", "v_scales"):
        s[name] = torch.randint(118, 121, (pool, hk), generator=gen, device=DEV, dtype=torch.uint8)
    s["q"] = torch.randn((s["tokens"], case["heads"], d), generator=gen, device=DEV).to(torch.bfloat16)
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((s["tokens"], case["heads"]), device=DEV)
    return s


def _prepare_sample(s, case, gen):
    r, V = case["rows"], case["V"]

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)
    # most tokens far below a few strong ones, as trained logits lie
    x = torch.randn((r, V), generator=gen, device=DEV) * 2.0 + 9.0 * (rand(r, V) < 30.0 / V) * rand(r, V)
    s["logits"] = x.to(torch.float32 if case["type"] == "f32" else torch.bfloat16)

    def some(kind, values, off):
        return None if kind == "none" else torch.where(rand(r) < 0.3, off, values) if kind == "mixed" else values
    s["temperature"] = None if case["temperature"] == "one" else some("mixed", 0.3 + 1.2 * rand(r), 0.0)
    k = some(case["k"], torch.exp(rand(r) * 6.0).floor(), 0.0)
    s["top_k"] = None if k is None else k.to(torch.int32)
    s["top_p"] = some(case["p"], 0.5 + 0.49 * rand(r), 1.0)
    s["min_p"] = some(case["min_p"], 0.01 + 0.2 * rand(r), 0.0)
    s["u"] = rand(r)
    s["token"], s["logprob"] = torch.empty(r, dtype=torch.int32, device=DEV), torch.empty(r, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_quant(s):
    from bit_weight_gemm_amd import binding as B
    B.biloco_quant_mxfp4(s["x"], codes=s["codes"], scales=s["scales"])
    B.biloco_dequant_mxfp4(s["codes"], s["scales"], out=s["values"])
    return dict(values=s["values"], scales=s["scales"])


def _own_product(s):
    from bit_weight_gemm_amd import binding as B
    if "workspace" not in s:      # as a serving program keeps one
        n = B.biloco_gemm_mxfp4_workspace_bytes(s["case"]["M"], s["case"]["N"], s["case"]["K"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    B.biloco_gemm_mxfp4_quant(s["x"], s["w_codes"], s["w_scales"], y=s["y"], workspace=s["workspace"])
    return s["y"]


def _own_shared(s):
    from bit_weight_gemm_amd import binding as B
    c = s["case"]
    if "workspace" not in s:
        n = B.biloco_attn_shared_workspace_bytes(c["batch"], s["tokens"], c["heads"], c["kv_heads"], c["dim"], s["max_q"],
                                                 s["max_kv"], c["groups"], s["max_shared"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    B.biloco_attn_shared((s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]), s["q"], s["q_start"], s["kv_len"],
                         s["block_table"], s["group_start"], s["shared_len"], s["max_q"], s["max_kv"], s["max_shared"],
                         s["scale"], window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"],
                         workspace=s["workspace"])
    return dict(out=s["out"], lse=s["lse"])


def _own_sample(s):
    from bit_weight_gemm_amd import binding as B
    if "workspace" not in s:
        n = B.biloco_sample_workspace_bytes(s["case"]["rows"], s["case"]["V"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    B.biloco_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                    min_p=s["min_p"], token=s["token"], logprob=s["logprob"], workspace=s["workspace"])
    return dict(token=s["token"], logprob=s["logprob"])


def _pow2(e):
    """2^(e - 127) in 32 bits, for e from 1 to 254."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """Codes and scale bytes: the largest value's exponent less two, magnitudes to nearest, ties to even."""
    x = x.float().unflatten(1, (-1, 32))
    amax = x.abs().amax(-1)
    e = ((amax.view(torch.int32) >> 23) - 2).clamp(0, 252)
    y = x * (_pow2(254 - e.clamp(min=1)) * torch.where(e == 0, 2.0, 1.0))[..., None]
    m = y.abs().clamp(max=6.0)
    step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
    m = torch.round(m / step) * step
    code = torch.where(m < 2.0, 2.0 * m, torch.where(m < 4.0, m + 2.0, 0.5 * m + 4.0)).to(torch.uint8)
    code = (code | (torch.signbit(x).to(torch.uint8) << 3)).flatten(1)
    return code[:, 0::2] | (code[:, 1::2] << 4), e.to(torch.uint8)


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    e2m1 = torch.cat([e2m1, -e2m1])
    v = torch.stack([e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]], -1).flatten(1).unflatten(1, (-1, 32))
    return (v * (_pow2(scales.int().clamp(min=1)) * torch.where(scales == 0, 0.5, 1.0))[..., None]).flatten(1)


def _plain_quant(s):
    codes, scales = _quantise(s["x"])
    s["values"].copy_(_values(codes, scales))
    return dict(values=s["values"], scales=scales)


def _plain_product(s):
    a = _values(*_quantise(s["x"]))
    s["y"].copy_(a @ _values(s["w_codes"], s["w_scales"]).T)
    return s["y"]


def _plain_shared(s):
    c = s["case"]
    hk, g, d, page = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    table = s["block_table"].long().clamp(min=0)
    n, length = table.shape[0], table.shape[1] * page
    k = s["k_codes"][table].view(torch.float8_e4m3fn).float() * _pow2(s["k_scales"][table])[..., None, None]
    k = k.transpose(1, 2).reshape(n, hk, length, d)
    v = s["v_codes"][table].view(torch.float8_e4m3fn).float() * _pow2(s["v_scales"][table])[..., None, None, None]
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(n, hk, length, d)
    j = torch.arange(length, device=DEV)
    live = j < kv[:, None]
    i = torch.arange(s["max_q"], device=DEV)
    count = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp(max=s["tokens"] - 1)             # [B][Q]
    q = s["q"][row].float().reshape(n, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    p = (kv - count)[:, None] + i                                       # [B][Q] positions
    see = live[:, None] & (j <= p[..., None])
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    score = score.reshape(n, hk, g, -1, length).masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - top)
    del score
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.reshape(n, hk, -1, length), v).reshape(n, hk, g, -1, d) / total
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]
    s["out"].copy_(out[b, :, :, i].reshape(s["out"].shape))
    s["lse"].copy_(lse[b, :, :, i].reshape(s["lse"].shape))
    return dict(out=s["out"], lse=s["lse"])


def _plain_sample(s):
    x = s["logits"].double()          # borders between tokens lie close: 64 bits
    r, V = x.shape
    one = torch.ones(r, dtype=torch.float64, device=DEV)

    def param(name, off):
        return (one * off if s[name] is None else s[name].double())[:, None]
    t, k, p, m = param("temperature", 1.0), param("top_k", 0.0), param("top_p", 1.0), param("min_p", 0.0)
    top = x.amax(1, keepdim=True)
    w = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws, rank = w.gather(1, order), torch.arange(V, device=DEV)
    keep = rank < torch.where(k > 0, k, V)
    wk = torch.where(keep, ws, 0.0)
    before = torch.cat([torch.zeros_like(top), wk.cumsum(1)[:, :-1]], 1)
    keep &= (before < p * wk.sum(1, keepdim=True)) | (p >= 1.0)
    keep &= ws >= m
    keep = torch.where(t > 0, keep, rank == 0)
    chosen = torch.where(torch.zeros_like(keep).scatter(1, order, keep), w, 0.0).cumsum(1)
    token = (chosen > s["u"].double()[:, None] * chosen[:, -1:]).int().argmax(1)
    s["token"].copy_(token)
    s["logprob"].copy_((w.gather(1, token[:, None]).log() - w.sum(1, keepdim=True).log())[:, 0])
    return dict(token=s["token"], logprob=s["logprob"])


_OWN = dict(quant=_own_quant, product=_own_product, shared=_own_shared, sample=_own_sample)
_PLAIN = dict(quant=_plain_quant, product=_plain_product, shared=_plain_shared, sample=_plain_sample)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "quant":
        n = case["rows"] * case["K"]
        return dict(bytes=n * (4 if case["type"] == "f32" else 2) + n * 17 // 32 + 2 * n, flops=4 * n)
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=N * K * 17 // 32 + 2 * M * K + M * N * (4 if case["out"] == "f32" else 2), flops=2 * M * N * K)
    if case["op"] == "sample":
        n = case["rows"] * case["V"]
        return dict(bytes=n * (4 if case["type"] == "f32" else 2) + 28 * case["rows"], flops=4 * n)
    new, kv, group, shared = _batch(case)
    hk, d, window, sinks = case["kv_heads"], case["dim"], case["window"], case["sinks"]
    pairs, tokens, reach = 0, 0, [None] * len(shared)
    for n, m, g in zip(new, kv, group):
        for p in range(m - n, m):
            lo = max(0, p - window + 1) if window else 0
            pairs += p + 1 - lo + min(lo, sinks)
        lo = max(0, m - n - window + 1) if window else 0
        tokens += m - max(lo, shared[g]) + max(0, min(sinks, lo) - shared[g])
        reach[g] = lo if reach[g] is None else min(reach[g], lo)
    # a group's shared tokens once: those that any of its sequences sees
    tokens += sum(max(0, n - lo) + min(n, lo, sinks) for n, lo in zip(shared, reach))
    moved = tokens * hk * 2 * d + -(-tokens // case["page"]) * (2 * hk + 4) + sum(new) * case["heads"] * (4 * d + 4)
    return dict(bytes=moved, flops=4 * d * pairs * case["heads"])


# ------------------------------------------------------------------ in 64 bits

def _two_to(n):
    """2^n in 64 bits, from its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_rows(x):
    """Rows as their quantisation stands for, and the scale bytes."""
    y = x.double().reshape(x.shape[0], -1, 32)
    largest = y.abs().amax(2)
    part, e = torch.frexp(largest)
    e = torch.where(largest == 0, -127, e.long() - 3).clamp(min=-127)
    y = y * _two_to(-e)[..., None]
    size = y.abs()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    middle = (grid[1:] + grid[:-1]) / 2
    # past a middle is the next value; on one, that of the even code
    i = torch.bucketize(size, middle, right=False)
    on = (size == middle[i.clamp(max=6)]) & (i < 7)
    i = torch.where(on & (i % 2 == 1), i + 1, i)
    v = torch.copysign(grid[i], y) * _two_to(e)[..., None]
    return v.flatten(1), e + 127


def _exact_weight(codes, scales):
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=DEV)
    for half in range(2):
        c = ((codes >> (4 * half)) & 15).long()
        mag, exp = (c & 1).double(), (c >> 1) & 3
        v = torch.where(exp == 0, mag / 2, (1 + mag / 2) * _two_to(exp - 1))
        out[:, half::2] = torch.where(c >= 8, -v, v)
    return (out.unflatten(1, (-1, 32)) * _two_to(scales.long() - 127)[..., None]).flatten(1)


def _exact_product(s):
    a, _ = _exact_rows(s["x"])
    N, y = s["w_codes"].shape[0], []
    for at in range(0, N, 16384):
        y.append(a @ _exact_weight(s["w_codes"][at:at + 16384], s["w_scales"][at:at + 16384]).T.contiguous())
    return torch.cat(y, 1)


def _exact_shared(s):
    c = s["case"]
    hk, g, d, page = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros((s["tokens"], c["heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["tokens"], c["heads"]), dtype=torch.float64, device=DEV)
    new, lens, _, _ = _batch(c)
    t0 = 0
    for b, (n, kv) in enumerate(zip(new, lens)):
        pages = s["block_table"][b, :-(-kv // page)].long()
        k = s["k_codes"][pages].view(torch.float8_e4m3fn).double() * _two_to(s["k_scales"][pages].long() - 127)[..., None, None]
        v = s["v_codes"][pages].view(torch.float8_e4m3fn).double()
        v = (v * _two_to(s["v_scales"][pages].long() - 127)[..., None, None, None]).transpose(3, 4)
        k, v = (x.reshape(len(pages), hk, page, d).transpose(0, 1).reshape(hk, -1, d)[:, :kv] for x in (k, v))
        j, p = torch.arange(kv, device=DEV), (kv - n + torch.arange(n, device=DEV))[:, None]
        hide = j > p
        if c["window"]:
            hide |= (j <= p - c["window"]) & (j >= c["sinks"])
        hide = hide[:, None].expand(n, g, kv).reshape(n * g, kv)
        for h in range(hk):
            q = s["q"][t0:t0 + n, h * g:(h + 1) * g].double().reshape(n * g, d)
            x = ((q @ k[h].T) * s["scale"]).masked_fill(hide, -math.inf)
            lse[t0:t0 + n, h * g:(h + 1) * g] = torch.logsumexp(x, 1).reshape(n, g)
            out[t0:t0 + n, h * g:(h + 1) * g] = (torch.softmax(x, 1) @ v[h]).reshape(n, g, d)
        t0 += n
    return dict(out=out, lse=lse)


def _exact_sample(s):
    tokens, logprobs = [], []
    for i, row in enumerate(s["logits"].double()):
        def of(name, off):
            return off if s[name] is None else float(s[name][i])
        t, k, p, m = of("temperature", 1.0), int(of("top_k", 0)), of("top_p", 1.0), of("min_p", 0.0)
        full = torch.log_softmax(row / (t if t > 0 else 1.0), 0)
        ids = torch.argsort(row, descending=True, stable=True)
        if not t > 0:
            ids = ids[:1]
        if k > 0:
            ids = ids[:k]
        prob = torch.softmax(full[ids], 0)
        if p < 1.0:
            ids = ids[:max(1, int((prob.cumsum(0) < p).sum()) + 1)]
        ids = ids[full[ids] >= full[ids[0]] + math.log(m)] if m > 0 else ids
        ids = torch.sort(ids)[0]
        upto = torch.exp(full[ids] - full[ids].max()).cumsum(0)
        at = int((upto <= float(s["u"][i]) * float(upto[-1])).sum())
        tokens.append(int(ids[min(at, len(ids) - 1)]))
        logprobs.append(float(full[tokens[-1]]))
    return dict(token=torch.tensor(tokens, dtype=torch.int32), logprob=torch.tensor(logprobs, dtype=torch.float64))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        values, scales = _exact_rows(s["x"])
        return dict(values=values, scales=scales.to(torch.uint8))
    return dict(product=_exact_product, shared=_exact_shared, sample=_exact_sample)[case["op"]](s)
