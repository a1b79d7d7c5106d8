"""Refusals of the entry points for several answers to one prompt, in the C ABI and in
the tensor binding, and their workspaces as sizes ask for them (no GPU; the addresses
are never used)."""
import pytest
import torch

from bit_weight_gemm_amd import binding as B

A = 1 << 36      # far-apart, aligned addresses
OK, BAD, UNS, SMALL = B.BILOCO_OK, B.BILOCO_ERR_INVALID_VALUE, B.BILOCO_ERR_UNSUPPORTED, B.BILOCO_ERR_WORKSPACE_TOO_SMALL
NAN, INF = float("nan"), float("inf")


def _call(name, a, kw):
    assert not set(kw) - set(a), kw
    return getattr(B.lib(), name)(*{**a, **kw}.values())


def quant(**kw):      # no rows: a call that passes the checks returns before any launch
    return _call("biloco_quant_mxfp4", dict(x=A, sx=512, fp32=0, M=0, K=512, c=2 * A, s=3 * A, stream=None), kw)


def dequant(**kw):
    return _call("biloco_dequant_mxfp4", dict(c=2 * A, s=3 * A, M=0, K=512, x=A, sx=512, fp32=0, stream=None), kw)


def product(**kw):
    return _call("biloco_gemm_mxfp4", dict(ac=A, asc=2 * A, wc=3 * A, ws=4 * A, M=0, N=300, K=512, y=5 * A, sy=300, fp32=0,
                                           w=6 * A, wb=1 << 40, stream=None), kw)


def product_quant(**kw):
    return _call("biloco_gemm_mxfp4_quant", dict(x=A, sx=512, wc=3 * A, ws=4 * A, M=0, N=300, K=512, y=5 * A, sy=300, fp32=0,
                                                 w=6 * A, wb=1 << 40, stream=None), kw)


def shared(**kw):
    return _call("biloco_attn_shared", dict(
        kc=A, vc=2 * A, ks=3 * A, vs=4 * A, pages=100, hk=8, page=32, dim=128, q=5 * A, sq=8192, hq=64, qs=10 * A, kvl=11 * A,
        bt=12 * A, mp=20, B=4, T=0, mq=1, mkv=1000, gs=16 * A, sl=17 * A, groups=2, msl=500, scale=0.1, win=0, sinks=0,
        o=13 * A, so=8192, lse=14 * A, ws=15 * A, wsb=1 << 40, stream=None), kw)


def sample(**kw):
    return _call("biloco_sample", dict(x=A, sx=1000, fp32=0, n=0, V=1000, t=2 * A, k=3 * A, p=4 * A, m=5 * A, u=6 * A, tok=7 * A,
                                       lp=8 * A, ws=9 * A, wsb=1 << 40, stream=None), kw)


def test_good_calls_pass_the_checks():
    assert quant() == dequant() == product() == product_quant() == shared() == sample() == OK
    assert quant(fp32=1, sx=520, K=32) == dequant(K=1 << 20, sx=1 << 20) == OK
    assert product(N=1, sy=1) == product_quant(sy=301, sx=1024) == OK
    assert shared(lse=None, groups=65535, msl=0) == OK
    assert sample(t=None, k=None, p=None, m=None, lp=None, sx=0, V=(1 << 20) - 1, fp32=1) == OK


ROWS = [(dict(M=-1), BAD), (dict(K=0), BAD), (dict(K=16), BAD), (dict(K=48), BAD), (dict(K=-32), BAD),
        (dict(K=(1 << 20) + 32, sx=1 << 21), UNS), (dict(x=None), BAD), (dict(c=None), BAD), (dict(s=None), BAD), (dict(x=A + 2), BAD),
        (dict(c=2 * A + 8), BAD), (dict(s=3 * A + 1), BAD), (dict(sx=511), BAD), (dict(sx=504), BAD), (dict(sx=516), BAD),
        (dict(sx=1 << 31), UNS), (dict(M=3, c=A + 1024), BAD), (dict(M=3, s=A), BAD)]


@pytest.mark.parametrize("kw,status", ROWS)
def test_rows_refuse(kw, status):
    assert quant(**kw) == dequant(**kw) == status


def test_codes_over_scales():
    assert quant(M=3, s=2 * A + 512) == BAD


GEMM = [(dict(M=-1), BAD), (dict(M=(1 << 30) + 1), UNS), (dict(N=(1 << 30) + 1, sy=(1 << 30) + 8), UNS), (dict(N=0), BAD), (dict(N=-4), BAD), (dict(K=0), BAD), (dict(K=40), BAD), (dict(K=1 << 21), UNS),
        (dict(wc=None), BAD), (dict(ws=None), BAD), (dict(y=None), BAD), (dict(wc=3 * A + 4), BAD), (dict(ws=4 * A + 2), BAD),
        (dict(y=5 * A + 2), BAD), (dict(w=6 * A + 8), BAD), (dict(sy=299), BAD), (dict(sy=1 << 31), UNS),
        (dict(M=40, K=8192, sx=8192, w=None), BAD), (dict(M=40, K=8192, sx=8192, wb=0), SMALL), (dict(M=2, y=3 * A + 64), BAD),
        (dict(M=2, y=4 * A), BAD), (dict(M=40, K=8192, sx=8192, w=5 * A + 16), BAD), (dict(M=40, K=8192, sx=8192, w=3 * A + 16), BAD)]


@pytest.mark.parametrize("kw,status", GEMM)
def test_products_refuse(kw, status):
    own = {k: v for k, v in kw.items() if k != "sx"}
    assert product(**own) == status
    assert product_quant(**{"sx": max(512, kw.get("K", 512)), **kw}) == status


@pytest.mark.parametrize("kw,status", [(dict(ac=None), BAD), (dict(asc=None), BAD), (dict(ac=A + 8), BAD), (dict(asc=2 * A + 1), BAD),
                                       (dict(M=2, y=A), BAD), (dict(M=2, y=2 * A + 16), BAD)])
def test_products_of_codes_refuse(kw, status):
    assert product(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict(x=None), BAD), (dict(x=A + 2), BAD), (dict(sx=511), BAD), (dict(sx=500), BAD),
                                       (dict(sx=1 << 31), UNS), (dict(M=2, y=A + 16), BAD), (dict(M=2, w=A), BAD)])
def test_products_of_rows_refuse(kw, status):
    assert product_quant(**kw) == status


def test_product_workspace():
    need = B.biloco_gemm_mxfp4_workspace_bytes(200, 5120, 13824)
    assert product(M=200, N=5120, sy=5120, K=13824, wb=need // 1000) == SMALL
    assert B.biloco_gemm_mxfp4_workspace_bytes(0, 5120, 13824) == 0
    for bad in ((-1, 5, 32), (1, 0, 32), (1, 5, 33)):
        assert B.lib().biloco_gemm_mxfp4_workspace_bytes(*bad, None) == BAD
        with pytest.raises(B.BilocoError):
            B.biloco_gemm_mxfp4_workspace_bytes(*bad)


@pytest.mark.parametrize("N,K", [(64, 32), (300, 512), (5120, 13824), (8192, 8192), (100001, 5120), (128, 1 << 16)])
def test_product_workspace_covers_fewer_rows(N, K):
    last = 0
    for M in (1, 2, 16, 17, 32, 33, 64, 65, 127, 128, 129, 200, 256, 257, 384, 385, 1000, 2048, 4096, 8191, 60000):
        n = B.biloco_gemm_mxfp4_workspace_bytes(M, N, K)
        assert n >= last
        last = n


@pytest.mark.parametrize("kw,status", [
    (dict(pages=0), BAD), (dict(page=48), UNS), (dict(dim=96), UNS), (dict(hk=0), BAD), (dict(kc=None), BAD), (dict(vs=4 * A + 1), BAD),
    (dict(qs=None), BAD), (dict(kvl=11 * A + 4), BAD), (dict(bt=None), BAD), (dict(mp=0), BAD), (dict(B=-1), BAD), (dict(T=-1), BAD),
    (dict(mq=0), BAD), (dict(B=70000), UNS), (dict(hq=0), BAD), (dict(hq=60), BAD), (dict(mkv=-1), BAD), (dict(scale=0.0), BAD),
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(win=-1), BAD), (dict(sinks=-1), BAD), (dict(win=(1 << 30) + 1), UNS),
    (dict(mkv=(1 << 30) + 1), UNS), (dict(T=1 << 26), UNS), (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=14 * A + 4), BAD),
    (dict(sq=8190), BAD), (dict(so=8000), BAD), (dict(T=2, o=5 * A), BAD), (dict(T=2, lse=5 * A + 32), BAD),
    # its own
    (dict(gs=None), BAD), (dict(sl=None), BAD), (dict(gs=16 * A + 4), BAD), (dict(sl=17 * A + 2), BAD), (dict(groups=0), BAD),
    (dict(groups=-1), BAD), (dict(groups=65536), UNS), (dict(msl=-1), BAD), (dict(msl=(1 << 30) + 1), UNS), (dict(T=4, ws=None), BAD),
    (dict(T=4, wsb=16), SMALL), (dict(T=2, o=16 * A), BAD), (dict(T=2, o=17 * A), BAD), (dict(T=4, ws=16 * A), BAD),
    (dict(T=4, ws=17 * A), BAD)])
def test_shared_refuses(kw, status):
    assert shared(**kw) == status


def test_shared_workspace_covers_smaller_calls():
    def need(b, t, q, kv, g, s):
        return B.biloco_attn_shared_workspace_bytes(b, t, 40, 8, 128, q, kv, g, s)
    axes = [(1, 3, 8, 33, 200), (1, 2, 9, 16, 64, 200, 1000), (1, 4, 9, 64), (64, 2000, 40000), (1, 2, 8, 40), (0, 64, 3000, 40000)]

    def walk(at, i):
        if i == len(axes):
            n = need(*at)
            for j, v in enumerate(at):
                k = axes[j].index(v)
                if k:
                    assert need(*at[:j], axes[j][k - 1], *at[j + 1:]) <= n, (at, j)
            return
        for v in axes[i]:
            walk(at + (v,), i + 1)
    walk((), 0)
    with pytest.raises(B.BilocoError):
        need(1, 1, 1, 64, 0, 0)
    assert B.lib().biloco_attn_shared_workspace_bytes(1, 1, 40, 8, 128, 1, 64, 1, 0, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), BAD), (dict(V=0), BAD), (dict(V=-5), BAD), (dict(V=1 << 20, sx=1 << 20), UNS), (dict(sx=-1), BAD), (dict(sx=1 << 31), UNS),
    (dict(x=None), BAD), (dict(u=None), BAD), (dict(tok=None), BAD), (dict(x=A + 2), BAD), (dict(t=2 * A + 4), BAD),
    (dict(k=3 * A + 4), BAD), (dict(p=4 * A + 4), BAD), (dict(m=5 * A + 4), BAD), (dict(u=6 * A + 4), BAD), (dict(tok=7 * A + 4), BAD),
    (dict(lp=8 * A + 4), BAD), (dict(ws=9 * A + 4), BAD), (dict(n=32, V=100000, sx=100000, wsb=0), SMALL),
    (dict(n=32, V=100000, sx=100000, ws=None), BAD), (dict(n=5, tok=A + 16), BAD), (dict(n=5, lp=6 * A), BAD), (dict(n=5, tok=8 * A), BAD),
    (dict(n=5, tok=3 * A), BAD), (dict(n=32, V=100000, sx=100000, ws=7 * A), BAD), (dict(n=32, V=100000, sx=0, ws=A + 16), BAD)])
def test_sample_refuses(kw, status):
    assert sample(**kw) == status


@pytest.mark.parametrize("V", [1, 1000, 32000, 100001, (1 << 20) - 1])
def test_sample_workspace_covers_fewer_rows(V):
    got = [B.biloco_sample_workspace_bytes(n, V) for n in (0, 1, 2, 3, 15, 16, 17, 31, 32, 64, 127, 128, 129, 256, 1000, 70000)]
    assert got[0] == 0 and got == sorted(got)
    assert B.lib().biloco_sample_workspace_bytes(1, V, None) == BAD


# ---------------------------------------------------------------- the tensor binding

LAST = "tensors of one GPU expected"      # the last check: host tensors that are right in all else
M, N, K, T, HQ, HK, D, PAGES, PAGE, SEQS, COLS, V = 3, 5, 64, 3, 4, 2, 64, 5, 16, 2, 3, 40


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def apart(t, dim=0):
    """t's shape and type, every other element along dim."""
    s = list(t.shape)
    s[dim] *= 2
    return torch.zeros(s, dtype=t.dtype)[tuple(slice(None, None, 2 if i == dim else 1) for i in range(t.dim()))]


def t_quant(**kw):
    return B.biloco_quant_mxfp4(**{**dict(x=bf16(M, K), codes=u8(M, K // 2), scales=u8(M, K // 32), stream=1), **kw})


def t_dequant(**kw):
    return B.biloco_dequant_mxfp4(**{**dict(codes=u8(M, K // 2), scales=u8(M, K // 32), out=f32(M, K), stream=1), **kw})


def t_product(**kw):
    return B.biloco_gemm_mxfp4(**{**dict(a_codes=u8(M, K // 2), a_scales=u8(M, K // 32), w_codes=u8(N, K // 2),
                                         w_scales=u8(N, K // 32), y=bf16(M, N), workspace=u8(16), stream=1), **kw})


def t_product_quant(**kw):
    return B.biloco_gemm_mxfp4_quant(**{**dict(x=bf16(M, K), w_codes=u8(N, K // 2), w_scales=u8(N, K // 32), y=bf16(M, N),
                                               workspace=u8(16), stream=1), **kw})


def t_shared(**kw):
    cache = (u8(PAGES, HK, PAGE, D), u8(PAGES, HK, PAGE // 8, D, 8), u8(PAGES, HK), u8(PAGES, HK))
    return B.biloco_attn_shared(**{**dict(
        cache=cache, q=bf16(T, HQ, D), q_start=i32(SEQS + 1), kv_len=i32(SEQS), block_table=i32(SEQS, COLS), group_start=i32(2),
        shared_len=i32(1), max_q_len=3, max_kv_len=9, max_shared_len=4, scale=0.1, out=bf16(T, HQ, D), lse=f32(T, HQ),
        workspace=u8(16), stream=1), **kw})


def t_sample(**kw):
    return B.biloco_sample(**{**dict(logits=f32(M, V), u=f32(M), temperature=f32(M), top_k=i32(M), top_p=f32(M), min_p=f32(M),
                                     token=i32(M), logprob=f32(M), workspace=u8(16), stream=1), **kw})


@pytest.mark.parametrize("call,kw", [
    (t_quant, {}), (t_quant, dict(x=f32(M, 2 * K)[:, :K])), (t_dequant, {}), (t_dequant, dict(out=bf16(2 * M, K)[::2])),
    (t_product, {}), (t_product, dict(y=f32(M, N + 3)[:, :N])), (t_product_quant, {}), (t_product_quant, dict(x=bf16(2 * M, K)[::2])),
    (t_shared, {}), (t_shared, dict(lse=None)), (t_sample, {}), (t_sample, dict(logits=bf16(1, V).expand(M, V))),
    (t_sample, dict(temperature=None, top_k=None, top_p=None, min_p=None, logprob=None))])
def test_right_tensors_reach_the_last_check(call, kw):
    with pytest.raises(ValueError, match=LAST):
        call(**kw)


@pytest.mark.parametrize("call,kw,words", [
    (t_quant, dict(x=bf16(M, K).half()), "x: "), (t_quant, dict(x=apart(bf16(M, K), 1)), "x: "),
    (t_quant, dict(codes=u8(M, K), scales=u8(M, K // 16)), "codes"), (t_quant, dict(codes=u8(M + 1, K // 2), scales=u8(M + 1, K // 32)), "codes"), (t_quant, dict(scales=u8(M, K // 16)), "scales"),
    (t_quant, dict(codes=apart(u8(M, K // 2), 1)), "codes"), (t_quant, dict(scales=u8(M, K // 32).char()), "scales"),
    (t_dequant, dict(out=f32(M, K).double()), "out"), (t_dequant, dict(out=f32(M + 1, K)), "out"), (t_dequant, dict(out=f32(M, 2 * K)), "out"),
    (t_dequant, dict(codes=u8(M * K // 2, 1)), "codes|scales"), (t_dequant, dict(scales=u8(M, 1)), "scales"),
    (t_product, dict(a_codes=u8(M, K)), "codes|scales"), (t_product, dict(a_scales=u8(M, 1)), "a_scales"),
    (t_product, dict(a_codes=u8(M, K), a_scales=u8(M, K // 16)), "w_codes"), (t_product, dict(w_codes=apart(u8(N, K // 2))), "w_codes"),
    (t_product, dict(w_scales=u8(N + 1, K // 32)), "w_scales"), (t_product, dict(y=bf16(M, N + 1)), "y: "),
    (t_product, dict(y=bf16(M + 1, N)), "y: "), (t_product, dict(y=bf16(M, N).half()), "y: "), (t_product, dict(y=apart(bf16(M, N), 1)), "y: "),
    (t_product, dict(workspace=apart(u8(16))), "workspace"), (t_product, dict(w_codes=None, workspace=u8(16)), "w_codes"),
    (t_product_quant, dict(x=f32(M, K)), "x: "), (t_product_quant, dict(x=bf16(M, 2 * K)), "x: |w_codes"),
    (t_product_quant, dict(x=apart(bf16(M, K), 1)), "x: "), (t_product_quant, dict(y=bf16(M, N - 1)), "y: "),
    (t_product_quant, dict(y=bf16(M - 1, N)), "y: "), (t_product_quant, dict(workspace=None, w_codes=u8(N, K // 2, 1)), "w_codes|INVALID"),
    (t_shared, dict(group_start=i32(1)), "group_start"), (t_shared, dict(group_start=i32(3)), "group_start"),
    (t_shared, dict(group_start=i32(2).long()), "group_start"), (t_shared, dict(group_start=apart(i32(2))), "group_start"),
    (t_shared, dict(shared_len=i32(1, 1)), "shared_len"), (t_shared, dict(shared_len=f32(1)), "shared_len"),
    (t_shared, dict(shared_len=apart(i32(2)), group_start=i32(3)), "shared_len"), (t_shared, dict(shared_len=[3]), "shared_len: a tensor"),
    (t_shared, dict(q=bf16(T, HQ, D).float()), "q: bf16"), (t_shared, dict(out=bf16(T - 1, HQ, D)), "out: bf16"),
    (t_shared, dict(lse=f32(T, HQ + 1)), "lse"), (t_shared, dict(kv_len=i32(SEQS + 1)), "kv_len"),
    (t_shared, dict(block_table=i32(SEQS)), "block_table"), (t_shared, dict(workspace=apart(u8(16))), "workspace"),
    (t_sample, dict(logits=f32(M, V).double()), "logits"), (t_sample, dict(logits=apart(f32(M, V), 1)), "logits"),
    (t_sample, dict(u=f32(M + 1)), "u: "), (t_sample, dict(u=bf16(M)), "u: "), (t_sample, dict(u=None), "u: "),
    (t_sample, dict(temperature=f32(M, 1)), "temperature"), (t_sample, dict(temperature=f32(M).double()), "temperature"),
    (t_sample, dict(top_k=i32(M).long()), "top_k"), (t_sample, dict(top_k=i32(M - 1)), "top_k"), (t_sample, dict(top_p=apart(f32(M))), "top_p"),
    (t_sample, dict(min_p=0.1), "min_p"), (t_sample, dict(token=i32(M).long()), "token"), (t_sample, dict(token=i32(M + 1)), "token"),
    (t_sample, dict(logprob=f32(M, 1)), "logprob"), (t_sample, dict(workspace=apart(u8(16))), "workspace")])
def test_wrong_tensors(call, kw, words):
    with pytest.raises(ValueError, match=words):
        call(**kw)


def test_calls_of_no_rows():
    assert B.biloco_quant_mxfp4(bf16(0, K))[0].shape == (0, K // 2)
    assert B.biloco_dequant_mxfp4(u8(0, K // 2), u8(0, K // 32)).shape == (0, K)
    assert B.biloco_gemm_mxfp4(u8(0, K // 2), u8(0, K // 32), u8(N, K // 2), u8(N, K // 32)).shape == (0, N)
    assert B.biloco_gemm_mxfp4_quant(bf16(0, K), u8(N, K // 2), u8(N, K // 32)).shape == (0, N)
    assert B.biloco_sample(f32(0, V), f32(0)).shape == (0,)


@pytest.mark.parametrize("dim", [64, 128])
def test_shared_workspace_is_made_of_aligned_arrays(dim):
    """Odd numbers of items and rows: every array in it begins at a multiple of 16 bytes,
    and all are multiples of 16 long."""
    for b, hq, hk, q in ((1, 1, 1, 1), (3, 5, 1, 1), (3, 5, 1, 3), (5, 9, 3, 1), (7, 21, 7, 5), (1, 63, 1, 1), (2, 5, 1, 1)):
        assert B.biloco_attn_shared_workspace_bytes(b, b * q, hq, hk, dim, q, 500, 1, 300) % 16 == 0, (b, hq, hk, q)


def test_more_work_than_a_launch_takes_is_refused():
    """Past 2^32 threads, before anything is launched."""
    big = (1 << 30)
    for call in (quant, dequant):
        assert call(M=(1 << 31) - 1, K=1 << 20, sx=1 << 20) == UNS
    for M, N in ((big, big), (1 << 20, 1 << 26), (1000, big), (big, 1000)):
        assert product(M=M, N=N, sy=N, K=32) == product_quant(M=M, N=N, sy=N, K=32, sx=32) == UNS, (M, N)
        with pytest.raises(B.BilocoError, match="UNSUPPORTED|unsupported"):
            B.biloco_gemm_mxfp4_workspace_bytes(M, N, 32)
    assert B.biloco_gemm_mxfp4_workspace_bytes(700, big, 32) > 0      # 3 x 2^22 tiles
    kw = dict(B=65535, hq=40, hk=40, dim=64, sq=2560, so=2560, T=70000)
    assert shared(mq=64, **kw) == UNS
    with pytest.raises(B.BilocoError, match="UNSUPPORTED|unsupported"):
        B.biloco_attn_shared_workspace_bytes(65535, 70000, 40, 40, 64, 64, 1000, 2, 500)
    assert B.biloco_attn_shared_workspace_bytes(65535, 70000, 40, 40, 64, 4, 1000, 2, 500) > 0
