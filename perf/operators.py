"""Cases of the decoder-layer operators around the low-rank product.

Three operators of one decoder layer's serving step, each in a plain form of
elementary torch operations (``own = False``) and through the framework's
entry points (``own = True``):

* ``append``: rotates q and k (positions with one or several axes), quantises
  k and v to E4M3 with one power-of-two scale per page and head, and writes
  them into a paged cache;
* ``attend``: causal attention of a ragged batch over that cache, optionally
  with a sliding window whose first tokens stay visible;
* ``norm``: the norms after and before a block with the block's gate and
  residual scale between them.

Layouts (those of the entry points):
  k_codes [pages][kv_heads][page][dim], v_codes [pages][kv_heads][page/8][dim][8]
  (eight tokens of one channel are neighbours), k_scales and v_scales
  [pages][kv_heads]: the byte b stands for 2^(b - 127).
  Sequence b's tokens are rows q_start[b] .. q_start[b+1] of the batch and the
  last of its kv_len[b] cached tokens; token a is slot a % page of page
  block_table[b][a // page].
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
N_POS = 1 << 17          # rows of the cos/sin table
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of one sequence, 40 heads of 128 (a layer 5120 wide): latency
        dict(name="append one token", op="append", batch=1, q_max=1, kv_max=613, ragged=0, heads=40,
             kv_heads=40, dim=128, page=16, axes=1, rot=128, interleaved=False, lens=1),
        # a decode batch of 32 at odd lengths, 64 query and 8 key heads (8192 wide)
        dict(name="append decode batch", op="append", batch=32, q_max=1, kv_max=8192, ragged=1, heads=64,
             kv_heads=8, dim=128, page=64, axes=1, rot=128, interleaved=False, lens=2),
        # a prefill of image and text tokens: three position axes, ragged prompts behind cached prefixes
        dict(name="append ragged prefill, 3 axes", op="append", batch=5, q_max=4096, kv_max=6000, ragged=1,
             heads=64, kv_heads=8, dim=128, page=32, axes=3, rot=128, interleaved=False, lens=3),
        # one token over a short context: latency
        dict(name="attend one short", op="attend", batch=1, q_max=1, kv_max=613, ragged=0, heads=40,
             kv_heads=40, dim=128, page=16, window=0, sinks=0, lens=4),
        # one token over a very long context: the axis has to be split
        dict(name="attend one long", op="attend", batch=1, q_max=1, kv_max=131071, ragged=0, heads=64,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, lens=5),
        # a decode batch of very different lengths, idle slots among them, no shared heads
        dict(name="attend ragged decode", op="attend", batch=32, q_max=1, kv_max=8192, ragged=1, heads=40,
             kv_heads=40, dim=128, page=32, window=0, sinks=0, lens=6),
        # streaming decode: a window of 1024 and 4 sink tokens over long contexts
        dict(name="attend window and sinks", op="attend", batch=32, q_max=1, kv_max=32768, ragged=1, heads=64,
             kv_heads=8, dim=128, page=64, window=1024, sinks=4, lens=7),
        # drafted tokens checked together: up to 5 rows a sequence
        dict(name="attend drafted tokens", op="attend", batch=16, q_max=5, kv_max=4100, ragged=1, heads=64,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, lens=8),
        # a whole prompt from empty, no shared heads
        dict(name="attend prompt", op="attend", batch=1, q_max=4096, kv_max=4096, ragged=0, heads=40,
             kv_heads=40, dim=128, page=64, window=0, sinks=0, lens=9),
        # chunks of prompts behind cached prefixes, heads of 64, window and sinks
        dict(name="attend chunks, window and sinks", op="attend", batch=3, q_max=2048, kv_max=12000, ragged=1,
             heads=64, kv_heads=8, dim=64, page=32, window=4096, sinks=16, lens=10),
        # a decode batch's rows between two blocks
        dict(name="norm decode rows", op="norm", tokens=32, width=5120, res="bf16", gate="none", post=True,
             offset=0.0, scale=1.0),
        # a long prompt's rows with a gate a token, residual in 32 bits
        dict(name="norm prompt rows, gated", op="norm", tokens=6001, width=8192, res="f32", gate="token",
             post=True, offset=1.0, scale=0.22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "attend", "norm"])
    if kind == "norm":
        width = rng.choice([_log(rng, 8, 1024) * 16, _log(rng, 100, 16384), 5120, 8192, 13824])
        most = 6001 * 8192 // width
        return dict(op="norm", tokens=_log(rng, 1, min(8192, most)), width=width,
                    res=rng.choice(["bf16", "f32"]), gate=rng.choice(["none", "row", "token"]),
                    post=rng.random() < 0.8, offset=float(rng.choice([0, 1])),
                    scale=rng.choice([1.0, 0.22, 0.7]))
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10, 40])
    heads = kv_heads * rng.choice([1, 2, 5, 8] if kv_heads <= 10 else [1])
    page = rng.choice([16, 32, 64, 128])
    seed = rng.randrange(1 << 30)
    if kind == "append":
        batch = _log(rng, 1, 64)
        q_max = rng.choice([1, 1, _log(rng, 2, 4096)])
        while batch * q_max * (heads + 2 * kv_heads) * dim > 12000 * 80 * 128:
            batch, q_max = (batch + 1) // 2, (q_max + 1) // 2
        axes = rng.choice([1, 1, 2, 3])
        return dict(op="append", batch=batch, q_max=q_max, kv_max=q_max + _log(rng, 1, 8192), ragged=1,
                    heads=heads, kv_heads=kv_heads, dim=dim, page=page, axes=axes,
                    rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, lens=seed)
    q_max = rng.choice([1, 1, rng.randint(2, 12), _log(rng, 16, 4096)])
    batch = _log(rng, 1, 64 if q_max <= 12 else 8)
    kv_max = q_max + _log(rng, 1, 131072 // batch if q_max == 1 else 16384)
    # no more cached data and no more products than the largest listed cases have
    while (batch * kv_max * kv_heads * dim > 32 * 8192 * 40 * 128 or
           batch * q_max * kv_max * heads * dim > 4096 * 2048 * 40 * 128):
        batch, q_max, kv_max = (batch + 1) // 2, (q_max + 1) // 2, (kv_max + 1) // 2
    kv_max = max(kv_max, q_max)
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return dict(op="attend", batch=batch, q_max=q_max, kv_max=kv_max, ragged=1, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, window=window,
                sinks=rng.choice([0, 4, rng.randint(1, 64)]) if window else 0, lens=seed)


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    n, q_max, kv_max = case["batch"], case["q_max"], case["kv_max"]
    if not case["ragged"]:
        return [q_max] * n, [kv_max] * n
    rng = random.Random(case["lens"])
    q, kv = [], []
    for b in range(n):
        if b == 0:
            new, past = q_max, kv_max - q_max
        else:
            new = rng.randint(0 if rng.random() < 0.1 else 1, q_max)
            past = _log(rng, 1, kv_max - q_max + 1) - 1
        q.append(new)
        kv.append(new + past)
    return q, kv


# ------------------------------------------------------------------ inputs

def _e4m3_cache(shape, gen):
    """Codes of a cache as values with a few strong channels leave them, and their scales."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(90.0).clamp_(-448.0, 448.0)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _ragged(case, gen):
    q, kv = _lengths(case)
    page = case["page"]
    need = [max(1, -(-n // page)) for n in kv]
    total = sum(need)
    pool = total + total // 16 + 1
    order = torch.randperm(pool, generator=gen, device=DEV)[:total].to(torch.int32)
    table = torch.full((len(q), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    start = [0]
    for n in q:
        start.append(start[-1] + n)
    s = dict(q_start=torch.tensor(start, dtype=torch.int32, device=DEV),
             kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV), block_table=table,
             q_lens=q, kv_lens=kv, tokens=start[-1], max_q=max(q), max_kv=max(kv), pool=pool)
    h, d = case["kv_heads"], case["dim"]
    s["k_codes"] = _e4m3_cache((pool, h, page, d), gen)
    s["v_codes"] = _e4m3_cache((pool, h, page // 8, d, 8), gen)
    for name in ("k_scales", "v_scales"):
        s[name] = torch.randint(118, 121, (pool, h), generator=gen, device=DEV, dtype=torch.uint8)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        t, c = case["tokens"], case["width"]
        rdt = torch.float32 if case["res"] == "f32" else torch.bfloat16

        def rand(*shape, dtype=torch.bfloat16, scale=1.0, mean=0.0):
            return (torch.randn(shape, generator=gen, device=DEV) * scale + mean).to(dtype)

        s["x"] = rand(t, c, scale=0.6)
        s["res"] = rand(t, c, dtype=rdt, scale=3.0)
        mean = 1.0 - case["offset"]
        s["post_w"] = rand(c, scale=0.1, mean=mean) if case["post"] else None
        s["pre_w"] = rand(c, scale=0.1, mean=mean)
        s["gate"] = {"none": None, "row": (1, c), "token": (t, c)}[case["gate"]]
        if s["gate"] is not None:
            s["gate"] = rand(*s["gate"], scale=0.5, mean=0.5)
        s["res_out"], s["h"] = torch.empty_like(s["res"]), torch.empty_like(s["x"])
        return s
    s.update(_ragged(case, gen))
    t, hq, hk, d = s["tokens"], case["heads"], case["kv_heads"], case["dim"]
    s["out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "attend":
        s["q"] = torch.randn((t, hq, d), generator=gen, device=DEV).to(torch.bfloat16)
        s["lse"] = torch.empty((t, hq), dtype=torch.float32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    # q, k and v are slices of one projection's rows
    y = torch.randn((t, (hq + 2 * hk) * d), generator=gen, device=DEV)
    y *= 1.0 + 4.0 * (torch.rand((y.shape[1],), generator=gen, device=DEV) < 0.03)
    y = y.to(torch.bfloat16)
    s["q"] = y[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = y[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    s["v"] = y[:, (hq + hk) * d:].unflatten(1, (hk, d))
    pairs = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)
    angle = torch.arange(N_POS, device=DEV, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    # text tokens have one position on every axis, image tokens a row and a column
    first = [kv - q for q, kv in zip(s["q_lens"], s["kv_lens"])]
    pos = torch.cat([torch.arange(p, p + n, dtype=torch.int32, device=DEV) for p, n in zip(first, s["q_lens"])])
    more = torch.randint(0, 64, (case["axes"] - 1, t), generator=gen, device=DEV, dtype=torch.int32)
    s["positions"] = torch.cat([pos[None], pos[None] // 2 + more], 0).contiguous()
    # the axes take sections of the pairs, the first the shortest
    a = case["axes"]
    ends = [pairs] if a == 1 else [pairs // (a + 1)] + [pairs * (i + 2) // (a + 1) for i in range(1, a)]
    s["pair_axis"] = bytes(next(i for i, e in enumerate(ends) if p < e) for p in range(pairs))
    s["pair_axis_dev"] = torch.tensor(list(s["pair_axis"]), device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_append(s):
    from bit_weight_gemm_amd import binding as B
    B.biloco_kv_append((s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]), s["q"], s["k"], s["v"],
                       s["positions"], s["cos_sin"], s["q_start"], s["kv_len"], s["block_table"], s["max_q"],
                       q_out=s["out"], pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"])
    return _append_outputs(s)


def _append_outputs(s):
    return dict(q=s["out"], k=s["k_codes"].view(torch.float8_e4m3fn), v=s["v_codes"].view(torch.float8_e4m3fn),
                k_scales=s["k_scales"], v_scales=s["v_scales"])


def _own_attend(s):
    from bit_weight_gemm_amd import binding as B
    c = s["case"]
    if "workspace" not in s:      # as a serving program keeps one
        n = B.biloco_attn_workspace_bytes(c["batch"], s["tokens"], c["heads"], c["kv_heads"], c["dim"],
                                          s["max_q"], s["max_kv"])
        s["workspace"] = torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV)
    B.biloco_attn_paged((s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]), s["q"], s["q_start"],
                        s["kv_len"], s["block_table"], s["max_q"], s["max_kv"], s["scale"],
                        window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"],
                        workspace=s["workspace"])
    return dict(out=s["out"], lse=s["lse"])


def _own_norm(s):
    from bit_weight_gemm_amd import binding as B
    c = s["case"]
    B.biloco_norm_gate_residual(s["x"], s["res"], s["pre_w"], post_w=s["post_w"], gate=s["gate"],
                                res_scale=c["scale"], eps=EPS, w_offset=c["offset"], res_out=s["res_out"],
                                h=s["h"])
    return dict(res=s["res_out"], h=s["h"])


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][heads][dim] in 32 bits; cos and sin [T][rot/2]."""
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _need(amax):
    """The smallest scale byte that brings amax to at most 448."""
    bits = amax.contiguous().view(torch.int32)
    return (((bits + 0x1FFFFF) >> 23) - 8).clamp(1, 254)


def _pow2(e):
    return (e.to(torch.int32) << 23).view(torch.float32)


def _plain_append(s):
    c = s["case"]
    page, rot = c["page"], c["rot"]
    p = s["positions"][s["pair_axis_dev"]].long().T                      # [T][pairs]
    pair = torch.arange(rot // 2, device=DEV)
    cos, sin = s["cos_sin"][p, pair], s["cos_sin"][p, pair + rot // 2]
    s["out"].copy_(_rotate(s["q"].float(), cos, sin, rot, c["interleaved"]))
    start, kv, table = s["q_start"].long(), s["kv_len"].long(), s["block_table"].long()
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    past = kv - (start[1:] - start[:-1])
    a = past[b] + t - start[b]                                          # token's place in its sequence
    pg, slot = table[b, a // page], a % page
    # the one page of a sequence that may hold earlier tokens
    edge = table[torch.arange(len(past), device=DEV), (past // page).clamp(max=table.shape[1] - 1)]
    edge = torch.where(edge < 0, table[:, 0], edge)
    for name, x in (("k", _rotate(s["k"].float(), cos, sin, rot, c["interleaved"])), ("v", s["v"].float())):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        amax = torch.zeros(scales.shape, device=DEV).index_reduce_(0, pg, x.abs().amax(-1), "amax")
        need = _need(amax)
        old = torch.where((past % page > 0)[:, None], scales[edge].int(), 0)
        new = torch.maximum(need[edge], old)
        # earlier tokens of that page in the page's new scale
        kept = codes[edge].view(torch.float8_e4m3fn).float()            # [B][heads][...]
        down = _pow2(127 + old - new).reshape(*old.shape, 1, 1, *([1] if name == "v" else []))
        was = (kept * down).to(torch.float8_e4m3fn).view(torch.uint8)
        at = torch.arange(page, device=DEV)
        at = at[:, None] if name == "k" else at.reshape(page // 8, 1, 8)
        had = at < (past % page).reshape(-1, 1, *([1] * at.dim()))
        grow = (new > old).reshape(down.shape)
        codes[edge] = torch.where(had & grow & (old > 0).reshape(down.shape), was, codes[edge])
        need[edge] = torch.maximum(new, need[edge])
        e = need[pg]                                                    # [T][heads]
        y = (x * _pow2(254 - e)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        if name == "k":
            codes[pg, :, slot] = y
        else:
            codes[pg, :, slot // 8, :, slot % 8] = y
        scales[pg] = e.to(torch.uint8)
    return _append_outputs(s)


def _plain_attend(s):
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
    v = torch.where(live[:, None, :, None], v, 0.0)
    i = torch.arange(s["max_q"], device=DEV)
    count = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp(max=max(0, s["tokens"] - 1))     # [B][Q]
    q = s["q"][row].float().reshape(n, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    p = (kv - count)[:, None] + i                                       # [B][Q] positions
    see = live[:, None] & (j <= p[..., None])
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    score = score.reshape(n, hk, g, -1, length).masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.reshape(n, hk, -1, length), v).reshape(n, hk, g, -1, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]
    s["out"].copy_(out[b, :, :, i].reshape(s["out"].shape))
    s["lse"].copy_(lse[b, :, :, i].reshape(s["lse"].shape))
    return dict(out=s["out"], lse=s["lse"])


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["post_w"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["post_w"].float() + c["offset"])
    if s["gate"] is not None:
        x = x * s["gate"].float()
    r = s["res"].float() + c["scale"] * x
    h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * (s["pre_w"].float() + c["offset"])
    s["res_out"].copy_(r)
    s["h"].copy_(h)
    return dict(res=s["res_out"], h=s["h"])


_OWN = dict(append=_own_append, attend=_own_attend, norm=_own_norm)
_PLAIN = dict(append=_plain_append, attend=_plain_attend, norm=_plain_norm)


# ------------------------------------------------------------------ what a pass cannot do without

def _visible(case, q, kv):
    """(query, token) pairs of one sequence, and the tokens that some query sees."""
    window, sinks = case["window"], case["sinks"]
    first = kv - q
    if not window:
        return sum(first + i + 1 for i in range(q)), kv if q else 0
    pairs = 0
    for p in range(first, kv):
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(lo, sinks)
    lo = max(0, first - window + 1)
    return pairs, (kv - lo + min(lo, sinks)) if q else 0


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["width"]
        r = 4 if case["res"] == "f32" else 2
        gate = {"none": 0, "row": case["width"], "token": n}[case["gate"]]
        return dict(bytes=n * (4 + 2 * r) + 2 * gate + 4 * case["width"], flops=10 * n)
    q, kv = _lengths(case)
    t, hq, hk, d = sum(q), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        scales = sum(-(-(n % case["page"] + m) // case["page"]) for m, n in
                     ((m, n - m) for m, n in zip(q, kv))) * hk * 2
        moved = t * d * (4 * hq + 4 * hk + 2 * hk) + t * (4 * case["rot"] + 4 * case["axes"]) + scales
        return dict(bytes=moved, flops=t * ((hq + hk) * 3 * case["rot"] + 4 * hk * d))
    pairs, tokens = (sum(x) for x in zip(*(_visible(case, m, n) for m, n in zip(q, kv))))
    moved = tokens * hk * (2 * d) + -(-tokens // case["page"]) * (2 * hk + 4) + t * hq * (4 * d + 4)
    return dict(bytes=moved, flops=4 * d * pairs * hq)


# ------------------------------------------------------------------ in 64 bits

def _two_to(n):
    """2^n in 64 bits, from its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x, scale_byte):
    """The E4M3 value nearest to x / 2^(byte - 127), ties to even, in 64 bits."""
    y = x * _two_to(127 - scale_byte.long())
    m = y.abs().clamp(max=448.0)
    step = _two_to(torch.frexp(m.clamp(min=2.0 ** -6))[1] - 4)
    return torch.sign(y) * (torch.round(m / step) * step).clamp(max=448.0)


def _exact_append(s):
    c = s["case"]
    page, rot, half = c["page"], c["rot"], c["rot"] // 2
    out = s["q"].double().clone()
    k = s["k"].double().clone()
    v = s["v"].double()
    for pair in range(half):
        pos = s["positions"][s["pair_axis"][pair]].long()
        cos, sin = s["cos_sin"][pos, pair].double()[:, None], s["cos_sin"][pos, half + pair].double()[:, None]
        i, j = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + half)
        for x in (out, k):
            a, b = x[..., i].clone(), x[..., j].clone()
            x[..., i], x[..., j] = a * cos - b * sin, b * cos + a * sin
    got = dict(q=out)
    table = s["block_table"].cpu()
    for name, x in (("k", k), ("v", v)):
        codes = s[name + "_codes"].view(torch.float8_e4m3fn).double()
        if name == "v":
            codes = codes.transpose(3, 4).flatten(2, 3)                 # [pages][heads][page][dim]
        scales = s[name + "_scales"].long()
        t0 = 0
        for b, (n, kv) in enumerate(zip(s["q_lens"], s["kv_lens"])):
            a = kv - n
            while a < kv:
                pg, lo = int(table[b, a // page]), a % page
                hi = min(page, lo + kv - a)
                rows = x[t0:t0 + hi - lo]                               # [n][heads][dim]
                amax = rows.abs().amax((0, 2))
                part, e = torch.frexp(amax.clamp(min=2.0 ** -140) / 448.0)
                e = (e.long() - (part == 0.5).long() + 127).clamp(1, 254)
                if lo:
                    new = torch.maximum(e, scales[pg])
                    back = codes[pg, :, :lo] * _two_to(scales[pg] - 127)[:, None, None]
                    codes[pg, :, :lo] = _exact_quant(back, new[:, None, None])
                    e = new
                codes[pg, :, lo:hi] = _exact_quant(rows, e[:, None]).transpose(0, 1)
                scales[pg] = e
                t0 += hi - lo
                a += hi - lo
        if name == "v":
            codes = codes.unflatten(2, (-1, 8)).transpose(3, 4).contiguous()
        got[name] = codes
    got.update(k_scales=None, v_scales=None)
    return got


def _exact_attend(s):
    c = s["case"]
    hk, g, d, page = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros((s["tokens"], c["heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((s["tokens"], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (n, kv) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        pages = s["block_table"][b, :-(-kv // page)].long()
        j = torch.arange(kv, device=DEV)
        for h in range(hk if n else 0):
            k = s["k_codes"][pages, h].view(torch.float8_e4m3fn).double()
            k = (k * _two_to(s["k_scales"][pages, h].long() - 127)[:, None, None]).reshape(-1, d)[:kv]
            v = s["v_codes"][pages, h].view(torch.float8_e4m3fn).double()
            v = v * _two_to(s["v_scales"][pages, h].long() - 127)[:, None, None, None]
            v = v.transpose(2, 3).reshape(-1, d)[:kv]
            p = (kv - n + torch.arange(n, device=DEV))[:, None]
            hide = j > p
            if c["window"]:
                hide |= (j <= p - c["window"]) & (j >= c["sinks"])
            for r in range(h * g, (h + 1) * g):
                x = (s["q"][t0:t0 + n, r].double() @ k.T) * s["scale"]
                x = x.masked_fill(hide, -math.inf)
                lse[t0:t0 + n, r] = torch.logsumexp(x, 1)
                out[t0:t0 + n, r] = torch.softmax(x, 1) @ v
        t0 += n
    return dict(out=out, lse=lse)


def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    if s["post_w"] is not None:
        x = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * (s["post_w"].double() + c["offset"])
    if s["gate"] is not None:
        x = x * s["gate"].double()
    r = s["res"].double() + c["scale"] * x
    return dict(res=r, h=r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * (s["pre_w"].double() + c["offset"]))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, norm=_exact_norm)[case["op"]](s)
