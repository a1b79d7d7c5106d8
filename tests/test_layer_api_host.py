"""Refusals of the decoder-layer entry points: every bad argument is turned
away on the host before any HIP call (no GPU; the addresses are never used)."""
import numpy as np
import pytest

from bit_weight_gemm_amd import binding as B
from oracle import layer

A = 1 << 36      # far-apart, aligned addresses
BAD, UNS, SMALL = B.BILOCO_ERR_INVALID_VALUE, B.BILOCO_ERR_UNSUPPORTED, B.BILOCO_ERR_WORKSPACE_TOO_SMALL

CACHE = dict(kc=A, vc=2 * A, ks=3 * A, vs=4 * A, pages=100, hk=8, page=32, dim=128)
RAGGED = dict(qs=10 * A, kvl=11 * A, bt=12 * A, mp=20, B=4, T=0, mq=1)


def append(**kw):
    # T = 0: a call that passes the checks returns before any launch
    a = dict(CACHE, q=5 * A, sq=10240, k=6 * A, sk=10240, v=7 * A, sv=10240, hq=64, pos=8 * A, axes=1, pa=None,
             cs=9 * A, np_=4096, rot=128, il=0, **RAGGED, qo=13 * A, sqo=8192, stream=None)
    assert not set(kw) - set(a), kw
    return B.lib().biloco_kv_append(*{**a, **kw}.values())


def attend(**kw):
    a = dict(CACHE, q=5 * A, sq=8192, hq=64, **RAGGED, mkv=1000, scale=0.1, win=0, sinks=0, o=13 * A, so=8192,
             lse=14 * A, ws=15 * A, wsb=1 << 30, stream=None)
    assert not set(kw) - set(a), kw
    return B.lib().biloco_attn_paged(*{**a, **kw}.values())


def norm(**kw):
    a = dict(x=A, sx=5120, pw=2 * A, g=3 * A, sg=0, rs=1.0, r=4 * A, sr=5120, f32=0, w=5 * A, eps=1e-6, off=0.0, T=0,
             C=5120, ro=6 * A, sro=5120, h=7 * A, sh=5120, ac=8 * A, asc=9 * A, stream=None)
    assert not set(kw) - set(a), kw
    return B.lib().biloco_norm_gate_residual(*{**a, **kw}.values())


def test_good_calls_pass_the_checks():
    assert append() == attend() == norm() == B.BILOCO_OK
    assert append(hq=0, q=None, qo=None) == B.BILOCO_OK
    assert append(rot=0, pos=None, cs=None, axes=0, np_=0) == B.BILOCO_OK
    assert append(qo=5 * A, sqo=10240) == B.BILOCO_OK
    assert append(pa=bytes([0, 1] * 32), axes=2) == B.BILOCO_OK
    assert attend(lse=None) == B.BILOCO_OK
    assert norm(pw=None, g=None, ac=None, asc=None, ro=4 * A) == B.BILOCO_OK
    assert norm(C=17, ac=None, asc=None, sx=17, sr=19, sro=23, sh=100) == B.BILOCO_OK


CACHE_BAD = [(dict(pages=0), BAD), (dict(hk=0), BAD), (dict(page=0), BAD), (dict(page=48), UNS), (dict(page=8), UNS),
             (dict(page=256), UNS), (dict(dim=0), BAD), (dict(dim=96), UNS), (dict(dim=256), UNS), (dict(hk=2048), UNS),
             (dict(kc=None), BAD), (dict(vc=None), BAD), (dict(ks=None), BAD), (dict(vs=None), BAD),
             (dict(kc=A + 8), BAD), (dict(vs=4 * A + 1), BAD), (dict(qs=None), BAD), (dict(kvl=None), BAD),
             (dict(bt=None), BAD), (dict(bt=12 * A + 4), BAD), (dict(mp=0), BAD), (dict(B=-1), BAD), (dict(T=-1), BAD),
             (dict(mq=0), BAD), (dict(B=70000), UNS), (dict(mp=1 << 26), UNS)]


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_cache_and_batch(kw, status):
    assert append(**kw) == status
    assert attend(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(hq=-1), BAD), (dict(hq=8192, sq=1 << 20, sqo=1 << 20), UNS), (dict(rot=-2), BAD), (dict(rot=130), BAD),
    (dict(rot=5), BAD), (dict(rot=24), UNS), (dict(axes=0), BAD), (dict(axes=5), UNS), (dict(np_=0), BAD),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(pos=None), BAD), (dict(cs=None), BAD),
    (dict(qo=None), BAD), (dict(q=5 * A + 2), BAD), (dict(sq=8184), BAD), (dict(sk=1020), BAD), (dict(sv=1028), BAD),
    (dict(sqo=8196), BAD), (dict(sk=1 << 31), UNS), (dict(pa=bytes([1] * 64)), BAD),
    (dict(pa=bytes([0] * 63 + [2]), axes=2), BAD),
    (dict(vc=A + 16), BAD), (dict(ks=A + 16), BAD), (dict(T=2, kc=6 * A + 16), BAD), (dict(T=2, qo=5 * A + 16), BAD),
    (dict(T=2, qo=5 * A, sqo=10248), BAD), (dict(T=2, vc=5 * A), BAD), (dict(vs=12 * A), BAD), (dict(T=2, qo=A), BAD)])
def test_append_refuses(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), BAD), (dict(hq=60), BAD), (dict(hq=8192, sq=1 << 20, so=1 << 20), UNS), (dict(mkv=-1), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(win=-1), BAD), (dict(sinks=-1), BAD), (dict(win=(1 << 30) + 1), UNS), (dict(mkv=(1 << 30) + 1), UNS),
    (dict(sinks=(1 << 30) + 1), UNS), (dict(T=1 << 26), UNS), (dict(q=None), BAD), (dict(o=None), BAD), (dict(o=13 * A + 2), BAD),
    (dict(lse=14 * A + 4), BAD), (dict(sq=8190), BAD), (dict(so=8000), BAD), (dict(T=2, o=5 * A), BAD),
    (dict(T=2, o=A + 16), BAD), (dict(T=2, lse=5 * A + 32), BAD)])
def test_attend_refuses(kw, status):
    assert attend(**kw) == status


def test_attend_workspace():
    need = B.biloco_attn_workspace_bytes(4, 4, 64, 8, 128, 1, 100000)
    assert need > 0
    assert attend(T=4, mkv=100000, wsb=need - 1) == SMALL
    assert attend(T=4, mkv=100000, ws=None) == BAD
    assert attend(T=4, mkv=100000, ws=A + 16) == BAD
    assert B.biloco_attn_workspace_bytes(0, 0, 64, 8, 128, 1, 1000) == 0
    with pytest.raises(B.BilocoError):
        B.biloco_attn_workspace_bytes(4, 4, 63, 8, 128, 1, 1000)
    assert B.lib().biloco_attn_workspace_bytes(4, 4, 64, 8, 128, 1, 1000, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(C=0), BAD), (dict(C=40000, sx=40000, sr=40000, sro=40000, sh=40000), UNS),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(x=None), BAD), (dict(r=None), BAD), (dict(w=None), BAD),
    (dict(ro=None), BAD), (dict(h=None), BAD), (dict(ac=None), BAD), (dict(asc=None), BAD), (dict(x=A + 2), BAD),
    (dict(sx=5119), BAD), (dict(sr=100), BAD), (dict(sg=8), BAD), (dict(sg=-5120), BAD), (dict(sh=1 << 31), UNS),
    (dict(C=24), BAD), (dict(C=48), UNS), (dict(T=2, h=A), BAD), (dict(T=2, ro=4 * A, sro=5128), BAD),
    (dict(T=2, ro=4 * A + 16), BAD), (dict(T=2, h=4 * A), BAD), (dict(T=2, ac=7 * A + 16), BAD),
    (dict(T=2, asc=5 * A), BAD)])
def test_norm_refuses(kw, status):
    assert norm(**kw) == status


def test_binding_refuses_wrong_tensors():
    import torch
    cache = B.biloco_kv_cache(4, 2, 16, 64, device="cpu")
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    i32 = torch.zeros
    good = dict(q_start=i32(2, dtype=torch.int32), kv_len=i32(1, dtype=torch.int32),
                block_table=i32((1, 2), dtype=torch.int32))

    def call(cache=cache, q=q, **kw):
        B.biloco_attn_paged(cache, q, **{**good, **kw}, max_q_len=1, max_kv_len=1, scale=1.0, stream=1,
                            workspace=torch.zeros(16, dtype=torch.uint8))

    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(kv_len=i32(1, dtype=torch.int64)),
                dict(q_start=i32(3, dtype=torch.int32)), dict(cache=(cache[0], cache[1], cache[2], cache[3][:2])),
                dict(cache=(cache[0], cache[0], cache[2], cache[3])), dict(lse=torch.zeros(1, 3))):
        with pytest.raises(ValueError):
            call(**bad)


def test_plain_formats():
    v = layer.e4m3_values()
    assert v[0x7E] == 448 and v[0x08] == 2.0 ** -6 and v[1] == 2.0 ** -9 and np.isnan(v[0x7F]) and v[0xB8] == -1
    fin = [c for c in range(256) if c & 127 != 127]
    np.testing.assert_array_equal(layer.e4m3_encode(v[fin]), fin)
    assert layer.e4m3_encode(np.array([1.0625, 1.1875, 0.0, -0.0, 2.0 ** -10]))[:2].tolist() == [0x38, 0x3A]
    for amax, byte in ((448.0, 127), (448.0001, 128), (224.0, 126), (0.0, 1), (1.0, 119), (1e-45, 1)):
        assert layer.need_byte(amax) == byte
        assert amax <= 448 * 2.0 ** (byte - 127)


@pytest.mark.parametrize("kw", [
    dict(k=5 * A), dict(v=5 * A), dict(k=5 * A + 16), dict(v=5 * A + 2 * 8192 - 16),       # columns of q's own
    dict(k=5 * A + 2 * 8192, sk=10248), dict(v=5 * A + 2 * 10240, sv=20480),      # other strides: rows meet q's
    dict(k=5 * A - 2 * 1024 + 16), dict(k=5 * A + 2 * 10240 - 16),      # the last columns reach the next row's q
    dict(k=5 * A + 2 * 10240), dict(v=5 * A + 3 * 2 * 10240 + 32)])
def test_append_in_place_refuses_keys_within_the_queries(kw):
    """q_out = q: k and v may be columns of the same rows, but not q's."""
    assert append(**{**dict(T=5, qo=5 * A, sqo=10240), **kw}) == BAD
    assert append(T=0, qo=5 * A, sqo=10240, **kw) == B.BILOCO_OK


def test_append_passes_on_the_error_of_a_truth_value():
    import torch

    class Odd:
        def __bool__(self):
            raise KeyError("odd")
    cache = B.biloco_kv_cache(4, 2, 16, 64, device="cpu")
    kv = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(KeyError, match="odd"):
        B.biloco_kv_append(cache, None, kv, kv, None, None, i32, i32[:1], i32[None], 1, interleaved=Odd(), stream=1)
