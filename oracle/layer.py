"""Plain CPU implementations of the decoder-layer operators (numpy; test
infrastructure, no code shared with the HIP path).

E4M3 (OCP "FN"): codes 0x7F and 0xFF are NaN, the largest value is 448; a
block's scale byte b stands for 2^(b - 127).
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 codes' values in float64."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]


def e4m3_encode(y: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even code; |y| <= 448 or NaN."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)
    with np.errstate(invalid="ignore"):
        hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 1, 126)
        lo = hi - 1
        dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(np.isnan(y), 127, code)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


LARGEST = 448.0 * 2.0 ** 119


def need_byte(amax: float) -> int:
    """Smallest b >= 1 with amax <= 448 * 2^(b - 127)."""
    if amax <= 0:
        return 1
    m, e = np.frexp(float(amax))      # amax = m 2^e, 1/2 <= m < 1; 448 2^t = 0.875 2^(t+9)
    return max(1, int(e - 9 + (1 if m > 0.875 else 0)) + 127)


def rotate(x, positions, cos_sin, pair_axis, interleaved, dtype):
    """x [T][heads][dim]; every product and sum rounded to `dtype`."""
    x = np.array(x, dtype)
    n_pos, rot = cos_sin.shape
    half = rot // 2
    for i in range(half):
        p = positions[pair_axis[i]]
        ok = (p >= 0) & (p < n_pos)
        row = np.where(ok, p, 0)
        c = np.where(ok, cos_sin[row, i], np.nan).astype(dtype)[:, None]
        s = np.where(ok, cos_sin[row, half + i], np.nan).astype(dtype)[:, None]
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., u].copy(), x[..., w].copy()
        with np.errstate(invalid="ignore", over="ignore"):
            x[..., u] = a * c - b * s
            x[..., w] = b * c + a * s
    return x


def append(cache, x_k, x_v, q_start, kv_len, table):
    """Appends rotated keys and values (float arrays [T][heads][dim]) to a copy
    of the cache (k [pages][heads][page][dim], v [pages][heads][page/8][dim][8],
    k_scales, v_scales); returns the new arrays."""
    kc, vc, ks, vs = (np.array(t) for t in cache)
    page = kc.shape[2]
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        past = kv_len[b] - n
        a = max(past, 0)      # rows before token 0 are no tokens
        while a < kv_len[b]:
            pg, lo = table[b, a // page], a % page
            hi = min(page, lo + kv_len[b] - a)
            t0 = q_start[b] + a - past
            for h in range(kc.shape[1]):
                for is_v, x, scales in ((0, x_k, ks), (1, x_v, vs)):
                    rows = np.asarray(x[t0:t0 + hi - lo, h], np.float64)
                    with np.errstate(invalid="ignore"):
                        rows = np.where(np.abs(rows) <= LARGEST, rows, np.nan)
                    fin = np.abs(rows[~np.isnan(rows)])
                    e = need_byte(fin.max() if fin.size else 0.0)
                    block = vc[pg, h].transpose(0, 2, 1).reshape(page, -1) if is_v else kc[pg, h]
                    block = block.copy()
                    if lo:
                        old = int(scales[pg, h])
                        e = max(e, old)
                        if e > old:
                            block[:lo] = e4m3_encode(_VALUES[block[:lo]] * 2.0 ** (old - e))
                    block[lo:hi] = e4m3_encode(rows * 2.0 ** (127 - e))
                    if is_v:
                        vc[pg, h] = block.reshape(page // 8, 8, -1).transpose(0, 2, 1)
                    else:
                        kc[pg, h] = block
                    scales[pg, h] = e
            a += hi - lo
    return kc, vc, ks, vs


def cache_values(cache):
    """(k, v) values [pages][heads][page][dim] in float64."""
    kc, vc, ks, vs = cache
    pages, heads, page, dim = kc.shape
    k = _VALUES[kc] * 2.0 ** (ks.astype(np.float64) - 127)[..., None, None]
    v = _VALUES[vc].transpose(0, 1, 2, 4, 3).reshape(pages, heads, page, dim)
    return k, v * 2.0 ** (vs.astype(np.float64) - 127)[..., None, None]


def attend(cache, q, q_start, kv_len, table, scale, window=0, sinks=0):
    """o [T][q_heads][dim], lse [T][q_heads], and for tolerances the sums of
    |w_j v_j| and the largest sum of |q_d k_jd| * scale of a row."""
    with np.errstate(invalid="ignore"):
        kval, vval = cache_values(cache)
    T, hq, dim = q.shape
    hk, page = cache[0].shape[1], cache[0].shape[2]
    o, mag = np.zeros((T, hq, dim)), np.zeros((T, hq, dim))
    lse, terms = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            p = kv_len[b] - n + i
            if p < 0:
                continue
            lo = max(0, p - window + 1) if window else 0
            seen = [j for j in range(min(sinks, lo))] + list(range(lo, p + 1))
            pages, slots = [table[b, j // page] for j in seen], [j % page for j in seen]
            t = q_start[b] + i
            for h in range(hq):
                k, v = kval[pages, h // (hq // hk), slots], vval[pages, h // (hq // hk), slots]
                with np.errstate(invalid="ignore"):
                    s = (k @ q[t, h]) * scale
                    top = s.max()
                    w = np.exp(s - top)
                    total = w.sum()
                    o[t, h] = (w[:, None] * v).sum(0) / total
                    mag[t, h] = (w[:, None] * np.abs(v)).sum(0) / total
                    lse[t, h] = top + np.log(total)
                    terms[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
    return o, lse, mag, terms


def norm_gate_residual(x, res, pre_w, post_w=None, gate=None, res_scale=1.0, eps=1e-6, w_offset=0.0):
    """(r', h) in float64, and |res| + |res_scale gate n| for tolerances."""
    x, res = np.asarray(x, np.float64), np.asarray(res, np.float64)
    n = x
    if post_w is not None:
        n = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * (w_offset + np.asarray(post_w, np.float64))
    if gate is not None:
        n = n * np.asarray(gate, np.float64)
    r = res + res_scale * n
    h = r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * (w_offset + np.asarray(pre_w, np.float64))
    return r, h, np.abs(res) + np.abs(res_scale * n)
