"""Each check of the tensor binding by its own words: a call that is right but for
its tensors being the host's gets as far as the last check, and every single
wrong argument is turned away before that one (no GPU)."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

LAST = "tensors of one GPU expected"
T, HQ, HK, D, PAGES, PAGE, SEQS, COLS, C = 3, 4, 2, 64, 5, 16, 2, 3, 64


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def strided(t, dim=0):
    """t's shape and type, every other element along dim."""
    s = list(t.shape)
    s[dim] *= 2
    return torch.zeros(s, dtype=t.dtype)[tuple(slice(None, None, 2 if i == dim else 1) for i in range(t.dim()))]


def cache(**kw):
    c = dict(k=u8(PAGES, HK, PAGE, D), v=u8(PAGES, HK, PAGE // 8, D, 8), ks=u8(PAGES, HK), vs=u8(PAGES, HK))
    return tuple({**c, **kw}.values())


RAGGED = dict(q_start=i32(SEQS + 1), kv_len=i32(SEQS), block_table=i32(SEQS, COLS))


def append(**kw):
    a = dict(cache=cache(), q=bf16(T, HQ, D), k=bf16(T, HK, D), v=bf16(T, HK, D), positions=i32(2, T),
             cos_sin=torch.zeros(10, D), **RAGGED, max_q_len=3, q_out=bf16(T, HQ, D), pair_axis=bytes(D // 2), stream=1)
    return B.biloco_kv_append(**{**a, **kw})


def attend(**kw):
    a = dict(cache=cache(), q=bf16(T, HQ, D), **RAGGED, max_q_len=3, max_kv_len=9, scale=0.1, out=bf16(T, HQ, D),
             lse=torch.zeros(T, HQ), workspace=u8(16), stream=1)
    return B.biloco_attn_paged(**{**a, **kw})


def norm(**kw):
    a = dict(x=bf16(T, C), res=bf16(T, C), pre_w=bf16(C), post_w=bf16(C), gate=bf16(T, C), res_out=bf16(T, C),
             h=bf16(T, C), a_codes=u8(T, C // 2), a_scales=u8(T, C // 16), stream=1)
    return B.biloco_norm_gate_residual(**{**a, **kw})


@pytest.mark.parametrize("call,kw", [
    (append, {}), (append, dict(q=None, q_out=None)), (append, dict(cos_sin=None, positions=None, pair_axis=None)),
    (append, dict(pair_axis=None)), (append, dict(q=bf16(T, 2 * HQ * D)[:, HQ * D:].unflatten(1, (HQ, D)))),
    (attend, {}), (attend, dict(lse=None)), (attend, dict(out=bf16(2 * T, HQ, D)[::2])),
    (norm, {}), (norm, dict(post_w=None, gate=None, a_codes=None, a_scales=None)), (norm, dict(gate=bf16(1, C))),
    (norm, dict(res=torch.zeros(T, C), res_out=torch.zeros(T, C))), (norm, dict(x=bf16(T, 2 * C)[:, :C]))])
def test_right_calls_reach_the_last_check(call, kw):
    with pytest.raises(ValueError, match=LAST):
        call(**kw)


CACHE = [(dict(cache=list(cache())), "cache: a tuple"), (dict(cache=cache()[:3]), "cache: a tuple"),
         (dict(cache=cache(ks=None)), "cache: a tensor"), (dict(cache=cache(k=bf16(PAGES, HK, PAGE, D))), "cache: uint8"),
         (dict(cache=cache(v=u8(PAGES, HK, PAGE // 8, D, 8).byte().bool())), "cache: uint8"),
         (dict(cache=cache(k=strided(u8(PAGES, HK, PAGE, D)))), "cache: contiguous"),
         (dict(cache=cache(vs=strided(u8(PAGES, HK), 1))), "cache: contiguous"),
         (dict(cache=cache(k=u8(PAGES, HK, PAGE * D))), "cache: k_codes"),
         (dict(cache=cache(v=u8(PAGES, HK, PAGE, D))), "cache: arrays of one"),
         (dict(cache=cache(v=u8(PAGES - 1, HK, PAGE // 8, D, 8))), "cache: arrays of one"),
         (dict(cache=cache(ks=u8(PAGES, HK + 1))), "cache: arrays of one"),
         (dict(cache=cache(vs=u8(PAGES - 1, HK))), "cache: arrays of one"),
         (dict(q_start=i32(SEQS)), "q_start"), (dict(q_start=i32(SEQS + 1).long()), "q_start"),
         (dict(q_start=strided(i32(SEQS + 1))), "q_start"), (dict(q_start=None), "q_start: a tensor"),
         (dict(kv_len=i32(SEQS + 1)), "kv_len"), (dict(kv_len=i32(SEQS).float()), "kv_len"),
         (dict(kv_len=i32(SEQS, 1)), "kv_len"), (dict(kv_len=[1, 2]), "kv_len: a tensor"),
         (dict(block_table=i32(SEQS * COLS)), "block_table"), (dict(block_table=i32(SEQS, COLS).long()), "block_table"),
         (dict(block_table=strided(i32(SEQS, COLS), 1)), "block_table"),
         (dict(block_table=i32(SEQS + 1, COLS)), "q_start"), (dict(q=bf16(T, HQ * D)), "q: "),
         (dict(q=bf16(T, HQ, D).half()), "q: bf16"), (dict(q=bf16(T, HQ, D // 2)), "q: bf16"),
         (dict(q=strided(bf16(T, HQ, D), 2)), "q: bf16"), (dict(q=strided(bf16(T, HQ, D), 1)), "q: bf16")]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kw,words", CACHE)
def test_cache_and_batch(call, kw, words):
    with pytest.raises(ValueError, match=words):
        call(**kw)


@pytest.mark.parametrize("kw,words", [
    (dict(q_out=bf16(T, HQ, D).float()), "q_out: bf16"), (dict(q_out=bf16(T + 1, HQ, D)), "q_out: bf16"),
    (dict(q_out=bf16(T, HQ + 1, D)), "q_out: bf16"), (dict(q_out=strided(bf16(T, HQ, D), 1)), "q_out: bf16"),
    (dict(q=bf16(T - 1, HQ, D)), "q: bf16"), (dict(k=bf16(T, HK * D)), "k: "), (dict(k=bf16(T, HK + 1, D)), "k: bf16"),
    (dict(k=bf16(T, HK, D).float()), "k: bf16"), (dict(v=bf16(T - 1, HK, D)), "v: bf16"),
    (dict(v=bf16(T, HK, 2 * D)), "v: bf16"),
    (dict(v=strided(bf16(T, HK, D), 2)), "v: bf16"), (dict(v=None), "v: a tensor"),
    (dict(cos_sin=torch.zeros(10 * D)), "cos_sin"),
    (dict(cos_sin=torch.zeros(10, D).double()), "cos_sin"), (dict(cos_sin=torch.zeros(10, 2 * D)[:, :D]), "cos_sin"),
    (dict(positions=None), "positions"), (dict(positions=i32(T)), "positions"), (dict(positions=i32(2, T + 1)), "positions"),
    (dict(positions=i32(2, T).long()), "positions"), (dict(positions=strided(i32(2, T), 1)), "positions"),
    (dict(pair_axis=bytes(D // 2 - 1)), "pair_axis"), (dict(pair_axis=[0] * (D // 2)), "pair_axis"),
    (dict(pair_axis=bytes(1), cos_sin=None), "pair_axis")])
def test_append(kw, words):
    with pytest.raises(ValueError, match=words):
        append(**kw)


@pytest.mark.parametrize("kw,words", [
    (dict(out=bf16(T, HQ, D).float()), "out: bf16"), (dict(out=bf16(T - 1, HQ, D)), "out: bf16"),
    (dict(out=strided(bf16(T, HQ, D), 2)), "out: bf16"), (dict(lse=torch.zeros(T, HQ + 1)), "lse"),
    (dict(lse=torch.zeros(T + 1, HQ)), "lse"), (dict(lse=torch.zeros(T, HQ).double()), "lse"),
    (dict(lse=strided(torch.zeros(T, HQ), 1)), "lse"), (dict(workspace=strided(u8(16))), "workspace")])
def test_attend(kw, words):
    with pytest.raises(ValueError, match=words):
        attend(**kw)


@pytest.mark.parametrize("kw,words", [
    (dict(x=bf16(T * C)), "x: "), (dict(x=bf16(T, C).float()), "x: "), (dict(x=strided(bf16(T, C), 1)), "x: "),
    (dict(res=bf16(T, C).half()), "res: bf16 or fp32"), (dict(res=bf16(T + 1, C)), "res: "),
    (dict(res=bf16(T, C + 1)), "res: "),
    (dict(res_out=torch.zeros(T, C)), "res_out"), (dict(res_out=bf16(T - 1, C)), "res_out"),
    (dict(h=bf16(T, C).float()), "h: "),
    (dict(h=bf16(T, C - 1)), "h: "), (dict(pre_w=bf16(C + 1)), "pre_w"), (dict(pre_w=bf16(C).float()), "pre_w"),
    (dict(pre_w=strided(bf16(C))), "pre_w"), (dict(post_w=bf16(1, C)), "post_w"), (dict(post_w=bf16(C - 1)), "post_w"),
    (dict(gate=bf16(C)), "gate"), (dict(gate=bf16(T - 1, C)), "gate"), (dict(gate=bf16(T, C + 1)), "gate"),
    (dict(gate=bf16(1, C).float()), "gate"), (dict(gate=strided(bf16(1, C), 1)), "gate"),
    (dict(a_codes=u8(T, C)), "a_codes"), (dict(a_codes=u8(T - 1, C // 2)), "a_codes"),
    (dict(a_codes=bf16(T, C // 2)), "a_codes"),
    (dict(a_codes=strided(u8(T, C // 2), 1)), "a_codes"), (dict(a_scales=u8(T, C // 32)), "a_scales"),
    (dict(a_scales=u8(T + 1, C // 16)), "a_scales"), (dict(a_scales=strided(u8(T, C // 16))), "a_scales")])
def test_norm(kw, words):
    with pytest.raises(ValueError, match=words):
        norm(**kw)
