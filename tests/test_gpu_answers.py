"""Several answers to one prompt, as a server would run them: the prompt taken in at once
through microscaled products, its last row drawn from once for each answer, then steps of
one token an answer that read the prompt once, each behind the draw before it.

Each operator is held to its 64-bit form on what it was given: the products and the
draws within the tolerances of test_gpu_mxfp4.py and test_gpu_sample.py, the attention
within those of test_gpu_attn_shared.py.
"""
import numpy as np
import pytest
import torch

from bit_weight_gemm_amd import binding as B
from bit_weight_gemm_amd.decoder import AttentionBlock, Head, MxLinear
from oracle import answers

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, PAGE, V = 16, 2, 64, 64, 1003
WIDTH, ANSWERS, PROMPT, MAX_KV = HEADS * DIM, 5, 192, 400
PER = -(-MAX_KV // PAGE)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(11)

        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda") * scale
        self.embed = rand(V, WIDTH).to(torch.bfloat16)
        self.cache = B.biloco_kv_cache(ANSWERS * PER, KV, PAGE, DIM)
        angle = torch.arange(MAX_KV, device="cuda", dtype=torch.float64)[:, None] / torch.arange(
            1, DIM // 2 + 1, device="cuda", dtype=torch.float64)
        ones = torch.ones(WIDTH, dtype=torch.bfloat16, device="cuda")
        self.block = AttentionBlock(MxLinear.of(rand((HEADS + 2 * KV) * DIM, WIDTH, scale=WIDTH ** -0.5)),
                                    MxLinear.of(rand(WIDTH, WIDTH, scale=WIDTH ** -0.5)), HEADS, KV, DIM, self.cache,
                                    torch.cat([angle.cos(), angle.sin()], 1).float(), ones, ones,
                                    max_sequences=ANSWERS, max_kv_len=MAX_KV, max_tokens=PROMPT, max_groups=2)
        self.head = Head(MxLinear.of(rand(V, WIDTH, scale=3 * WIDTH ** -0.5)), max_rows=ANSWERS)
        self.table = torch.randperm(ANSWERS * PER, generator=torch.Generator().manual_seed(3)).to(torch.int32).reshape(ANSWERS, PER)
        self.table[1:, :PROMPT // PAGE] = -1      # the prompt is the first answer's
        self.table = self.table.cuda()
        self.asks = dict(temperature=torch.tensor([0.0, 0.6, 0.9, 1.0, 1.5], device="cuda"), top_k=_ints([0, 3, 50, 0, 200]),
                         top_p=torch.tensor([1.0, 0.9, 0.95, 0.8, 1.0], device="cuda"),
                         min_p=torch.tensor([0.0, 0.0, 0.05, 0.0, 0.01], device="cuda"))
        self.logprob = torch.empty(ANSWERS, device="cuda")

    def take_prompt(self, tokens):
        x = self.embed[tokens]
        return self.block.step(x, None, None, x.clone(), torch.arange(PROMPT, dtype=torch.int32, device="cuda")[None],
                               _ints([0, PROMPT]), _ints([PROMPT]), self.table[:1], PROMPT)[0]

    def draw(self, h, u):
        return self.head.step(h, u, **self.asks, logprob=self.logprob)

    def answer(self, tokens, n, u):
        """Each answer's n-th token taken in, the next one drawn."""
        x = self.embed[tokens.long()]
        at = PROMPT + n
        h, _, _ = self.block.step(x, None, None, x.clone(), _ints([[at] * ANSWERS]), _ints(range(ANSWERS + 1)),
                                  _ints([at + 1] * ANSWERS), self.table, 1, shared=(_ints([0, ANSWERS]), _ints([PROMPT])))
        return x, h, self.draw(h, u)


def _product_holds(x, w, y):
    a = answers.quant_mxfp4(x.double().cpu().numpy())
    want, mag = answers.gemm_mxfp4(a, (w.codes.cpu().numpy(), w.scales.cpu().numpy()))
    K = w.K
    bound = (K / 64 + 64) * 2.0 ** -23 * mag + np.abs(want) * (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24)
    assert bool((np.abs(y.double().cpu().numpy() - want) <= bound).all())


def _draws_hold(s, rows, u, tokens):
    ask = {k: v.double().cpu().numpy() for k, v in s.asks.items()}
    logits, u, got = s.head._logits.double().cpu().numpy(), u.double().cpu().numpy(), tokens.cpu().numpy()
    for i in range(ANSWERS):
        want, lp, near = answers.sample(logits[i if rows > 1 else 0], u[i], ask["temperature"][i], int(ask["top_k"][i]),
                                        ask["top_p"][i], ask["min_p"][i])
        # u is 24 bits of a fixed seed: no border lies as near as the weights' steps
        assert near > V * 2.0 ** -44 + 2.0 ** -40 and got[i] == want, (i, got[i], want, near)
        assert abs(float(s.logprob[i]) - lp) <= 2.0 ** -24 * abs(lp) + V * 2.0 ** -44 + 2.0 ** -40


def _attention_holds(s, n):
    """The block's rows against the cache's values, the prompt through the first table."""
    kc, vc, ks, vs = s.cache
    k = kc.view(torch.float8_e4m3fn).double() * torch.exp2(ks.double() - 127)[..., None, None]
    v = vc.view(torch.float8_e4m3fn).double().transpose(3, 4).flatten(2, 3) * torch.exp2(vs.double() - 127)[..., None, None]
    G, kv_len = HEADS // KV, PROMPT + n + 1
    for b in range(ANSWERS):
        pages = torch.cat([s.table[0, :PROMPT // PAGE], s.table[b, PROMPT // PAGE:]])[:-(-kv_len // PAGE)].long()
        kb, vb = (t[pages].transpose(0, 1).flatten(1, 2)[:, :kv_len] for t in (k, v))
        for a in range(HEADS):
            q = s.block._q[b, a].double()
            w = torch.softmax(kb[a // G] @ q * DIM ** -0.5, 0)
            want, size = w @ vb[a // G], w @ vb[a // G].abs()
            e = 2 * (DIM + 8) * 2.0 ** -24 * (kb[a // G].abs() @ q.abs()).max() * DIM ** -0.5 + 2.0 ** -20
            got = s.block._o[b, a].double()
            assert bool(((got - want).abs() <= (2.0 ** -8 + e) * size + 2.0 ** -8 * want.abs()).all()), (b, a)


def _uniform(seed):
    return torch.rand(ANSWERS, generator=torch.Generator().manual_seed(seed)).cuda()


def test_a_run():
    s = Server()
    prompt = torch.randint(0, V, (PROMPT,), generator=torch.Generator().manual_seed(9)).cuda()
    h = s.take_prompt(prompt)
    _product_holds(s.embed[prompt], s.block.qkv, s.block._qkv[:PROMPT])
    u = _uniform(0)
    tokens = s.draw(h[-1:], u)
    torch.cuda.synchronize()
    _product_holds(h[-1:], s.head.weight, s.head._logits[:1])
    _draws_hold(s, 1, u, tokens)
    for n in range(70):      # into the answers' second pages of their own
        u = _uniform(1 + n)
        x, h, tokens = s.answer(tokens.clone(), n, u)
        if n in (0, 1, 63, 64, 69):
            _product_holds(x, s.block.qkv, s.block._qkv[:ANSWERS])
            _attention_holds(s, n)
            _product_holds(s.block._o[:ANSWERS].flatten(1), s.block.out, s.block._proj[:ANSWERS])
            _product_holds(h, s.head.weight, s.head._logits)
            _draws_hold(s, ANSWERS, u, tokens)
    assert int(tokens.min()) >= 0 and int(tokens.max()) < V


def test_shared_steps_are_those_of_whole_tables():
    """The same step with the prompt's pages in every table and nothing shared."""
    s = Server()
    h = s.take_prompt(torch.arange(PROMPT, device="cuda"))
    tokens = s.draw(h[-1:], _uniform(0)).clone()
    before = [t.clone() for t in s.cache]
    _, _, first = s.answer(tokens, 0, _uniform(1))
    o, cache = s.block._o[:ANSWERS].clone(), [t.clone() for t in s.cache]
    for t, b in zip(s.cache, before):
        t.copy_(b)
    whole = s.table.clone()
    whole[1:, :PROMPT // PAGE] = whole[0, :PROMPT // PAGE]
    x = s.embed[tokens.long()]
    s.block.step(x, None, None, x.clone(), _ints([[PROMPT] * ANSWERS]), _ints(range(ANSWERS + 1)),
                 _ints([PROMPT + 1] * ANSWERS), whole, 1)
    assert all(torch.equal(a, b) for a, b in zip(cache, s.cache))
    # both within their bound of the same value, |o| and sum w |v| at most the largest |v| of
    # the tokens that are there: the prompt's pages, and the first token of each answer's own
    kc, vc, ks, vs = s.cache
    k = kc.view(torch.float8_e4m3fn).double().abs() * torch.exp2(ks.double() - 127)[..., None, None]
    v = vc.view(torch.float8_e4m3fn).double().abs() * torch.exp2(vs.double() - 127)[..., None, None, None]
    prompt, own = whole[0, :PROMPT // PAGE].long(), whole[:, PROMPT // PAGE].long()
    k = torch.maximum(k[prompt].max(), k[own, :, 0].max())
    v = torch.maximum(v[prompt].max(), v[own, :, 0, :, 0].max())
    terms = k.max() * s.block._q[:ANSWERS].double().abs().sum(2).max() * DIM ** -0.5
    e = 2 * (DIM + 8) * 2.0 ** -24 * terms + 2.0 ** -20
    assert bool(((s.block._o[:ANSWERS].double() - o.double()).abs() <= 2 * (2 * 2.0 ** -8 + e) * v.max()).all())


def test_a_captured_step():
    """A step and its draw in a graph, replayed between other work, against the eager ones."""
    s = Server()
    h = s.take_prompt(torch.arange(PROMPT, device="cuda") * 5 % V)
    tokens = s.draw(h[-1:], _uniform(0)).clone()
    before = [t.clone() for t in s.cache]
    u, x = _uniform(1), s.embed[tokens.long()]
    res = x.clone()
    args = (_ints([[PROMPT] * ANSWERS]), _ints(range(ANSWERS + 1)), _ints([PROMPT + 1] * ANSWERS), s.table, 1)
    shared = (_ints([0, ANSWERS]), _ints([PROMPT]))

    def step():
        h, _, _ = s.block.step(x, None, None, res, *args, shared=shared)
        return s.draw(h, u)
    want = step().clone()
    keep = [t.clone() for t in (res, s.head._logits, s.logprob, *s.cache)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        for t, b in zip(s.cache, before):
            t.copy_(b)
        res.copy_(x)
        s.head._token.fill_(-5)
        s.head._logits.fill_(float("nan"))
        s.logprob.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.head._token, want), turn
        assert all(torch.equal(a, b) for a, b in zip((res, s.head._logits, s.logprob, *s.cache), keep)), turn
        s.draw(h[-1:], _uniform(turn))      # other work of the same buffers between the replays
