"""Plain float64 forms of the operators for several answers to one prompt
(microscaled 4-bit rows and products, sampling); test infrastructure."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
_MIDDLE = (E2M1[1:8] + E2M1[:7]) / 2


def quant_mxfp4(x):
    """x [M][K] -> (codes [M][K/2], scale bytes [M][K/32])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, K // 32), np.uint8)
    for m in range(M):
        for b in range(K // 32):
            v = x[m, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[m, b] = 255
                continue
            a = np.abs(v).max()
            e = 0 if a == 0 else max(0, int(np.frexp(a)[1]) - 1 + 125)
            scales[m, b] = e
            y = np.abs(v) / 2.0 ** (e - 127)
            i = np.searchsorted(_MIDDLE, y, side="left")      # the next value past a middle
            on = (i < 7) & (y == _MIDDLE[np.minimum(i, 6)])
            i = np.where(on & (i % 2 == 1), i + 1, i)          # on one: the even code
            codes[m, 32 * b:32 * b + 32] = i + 8 * np.signbit(v)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values_mxfp4(codes, scales):
    v = np.empty((codes.shape[0], 2 * codes.shape[1]))
    v[:, 0::2], v[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, 1)


def gemm_mxfp4(a, w):
    """a and w: (codes, scales).  y, and the sums of the terms' magnitudes."""
    a, w = values_mxfp4(*a), values_mxfp4(*w)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """One row: (token, log-probability, how near the nearest other outcome is, as a share of the sums compared)."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    t, p, m, u = (off if np.isnan(v) else v for v, off in ((t, 0.0), (p, 1.0), (m, 0.0), (u, 0.0)))
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if t <= 0:
        t, k, p, m = 1.0, 1, 1.0, 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(x == top, 0.0, (x - top) / t)
    d = np.where(np.isnan(d), -np.inf, d)
    w = np.exp(d)
    order = np.argsort(-x, kind="stable")
    near = 1.0
    if 0 < k < len(x):
        order = order[:k]
    if p < 1:
        upto = np.cumsum(w[order])
        target = p * upto[-1]
        order = order[:max(1, int(np.searchsorted(upto, target, side="left")) + 1)]
        near = min(near, np.abs(upto - target).min() / upto[-1])
    if m > 0:
        keep = w[order] >= min(m, 1.0)
        near = min(near, np.abs(w[order] - min(m, 1.0))[w[order] != 1.0].min(initial=1.0))
        order = order[keep]
    ids = np.sort(order)
    upto = np.cumsum(w[ids])
    target = max(u, 0.0) * upto[-1]
    at = int(np.searchsorted(upto, target, side="right"))
    if at >= len(ids):
        at = int(np.nonzero(w[ids] > 2.0 ** -45)[0][-1])
    else:
        near = min(near, np.abs(upto - target).min() / upto[-1])
    token = int(ids[at])
    return token, d[token] - np.log(w.sum()), near
