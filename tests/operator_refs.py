"""Plain float64 forms of the operators beside the layer, on the CPU (test infrastructure)."""
from __future__ import annotations

import numpy as np
import torch

U24 = 2.0 ** -24          # half a step of float32
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LADDER = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ routing
def score64(kind, l):
    """Scores of float64 logits [n]; a logit of -inf scores 0."""
    with np.errstate(over="ignore"):
        if kind == "softmax":
            if not len(l) or l.max() == -np.inf:
                return np.zeros_like(l)
            e = np.exp(l - l.max())
            return e / e.sum()
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        return np.sqrt(np.maximum(l, 0.0) + np.log1p(np.exp(-np.abs(l))))


def log_score(kind, l):
    """log of a score up to a constant of the token: ratios of scores that underflow."""
    if kind == "softmax":
        return l
    if kind == "sigmoid":
        return np.where(l < 0, l - np.log1p(np.exp(-np.abs(l))), -np.log1p(np.exp(-np.abs(l))))
    t = np.exp(-np.abs(l))
    with np.errstate(divide="ignore"):
        return 0.5 * np.where(l > -30, np.log(np.maximum(np.maximum(l, 0) + np.log1p(t), 1e-300)), l)


def route(logits, k, score, bias=None, n_groups=1, topk_groups=1, group_score="max", renormalise=True, scale=1.0):
    """(idx [T, k], w [T, k] float64) of float64-convertible logits [T, E]."""
    L = logits.double().numpy()
    T, E = L.shape
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    b = None if bias is None else bias.double().numpy()
    for t in range(T):
        l = np.minimum(L[t], float(np.finfo(np.float32).max))
        l = np.where(np.isnan(l), -np.inf, l)
        live = l > -np.inf
        s = score64(score, l)
        c = l.copy() if b is None else np.where(live, s + b, -np.inf)
        c[np.isnan(c)] = -np.inf
        l = np.where(c > -np.inf, l, -np.inf)
        if n_groups > 1:
            v = c.reshape(n_groups, -1)
            if group_score == "max":
                gs = v.max(1)
            else:
                sc = (s if b is None else s + b).reshape(n_groups, -1)
                sc = np.sort(np.where(v > -np.inf, sc, -np.inf), axis=1)
                second = sc[:, -2] if sc.shape[1] > 1 else np.full(n_groups, -np.inf)
                gs = sc[:, -1] + np.where(second > -np.inf, second, 0.0)
            order = [g for g in np.argsort(-gs, kind="stable") if gs[g] > -np.inf][:topk_groups]
            keep = np.zeros(n_groups, dtype=bool)
            keep[order] = True
            c = np.where(np.repeat(keep, E // n_groups), c, -np.inf)
        best = [e for e in np.argsort(-c, kind="stable") if c[e] > -np.inf][:k]
        idx[t, :len(best)] = best
        if best:
            if renormalise:
                x = log_score(score, l[best])
                x = np.exp(x - x.max())
                w[t, :len(best)] = x / x.sum()
            else:
                w[t, :len(best)] = s[best]
    return idx, w * scale


def permute(idx, E):
    """(offsets [E + 1], sorted_token, sorted_slot, inv_pos) of idx [T, k]; -1 is placed nowhere."""
    T, k = idx.shape
    flat = idx.reshape(-1)
    pairs = np.nonzero(flat >= 0)[0]
    order = pairs[np.argsort(flat[pairs], kind="stable")]
    offsets = np.zeros(E + 1, dtype=np.int64)
    offsets[1:] = np.cumsum(np.bincount(flat[pairs], minlength=E))
    inv = np.full(T * k, -1, dtype=np.int64)
    inv[order] = np.arange(len(order))
    return offsets, order // k, order % k, inv


# ------------------------------------------------------------------ MXFP4
def mx_scale(amax):
    """Scale bytes of block maxima (float64)."""
    m = np.asarray(amax, dtype=np.float64)
    bad = ~np.isfinite(m)
    e = np.frexp(np.where(bad | (m == 0), 1.0, m))[1] - 1
    s = np.maximum(np.where(m == 0, -127, e - 2), -127) + 127
    return np.where(bad, 255, s).astype(np.uint8)


def mx_round(a):
    """Indices on the ladder of magnitudes a (float64): nearest, ties to the even index, saturated."""
    a = np.minimum(np.abs(a), 6.0)
    hi = np.searchsorted(LADDER, a, side="left").clip(0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - LADDER[lo], LADDER[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantize(x):
    """(codes [R, K/2], scales [R, K/32]) of float64 rows."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(2)
    s = mx_scale(amax)
    bad = (s == 255)[:, :, None]
    a = np.where(bad, 0.0, b) / np.ldexp(1.0, np.where(s == 255, 127, s).astype(np.int64) - 127)[:, :, None]
    code = mx_round(a) | (np.signbit(np.where(bad, 1.0, b)) * 8)
    code = np.where(bad, 7, code).reshape(R, K).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def dequantize(codes, scales):
    """float64 values."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], 2 * codes.shape[1])
    v = np.where(c >= 8, -LADDER[c & 7], LADDER[c & 7])
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    with np.errstate(invalid="ignore"):
        return v * np.repeat(f, 32, axis=1)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def product(a, mats, offsets):
    """(out, bound) for float64 rows a [R, K] grouped by offsets and matrices [E, N, K]: one matrix, or
    gate and up.  The bound is on the error of fp32 sums of exact products: K/32 additions and 8 more
    (inside a block the sums are exact or cost less), each off by at most a step, 2^-23, of the sum of
    the magnitudes; the gated form adds what silu(g) * u makes of it (|silu'| <= 1.1) and 16 half steps
    for its own exponential, sum, quotient and product."""
    R, K = a.shape
    N = mats[0].shape[1]
    outs, errs = [], []
    steps = (K / 32 + 8) * 2.0 ** -23
    for m in mats:
        o, s = np.zeros((R, N)), np.zeros((R, N))
        for e in range(m.shape[0]):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            if hi > lo:
                o[lo:hi] = a[lo:hi] @ m[e].T
                s[lo:hi] = np.abs(a[lo:hi]) @ np.abs(m[e]).T
        outs.append(o)
        errs.append(s * steps)
    if len(mats) == 1:
        return outs[0], errs[0]
    (g, u), (dg, du) = outs, errs
    h = silu(g) * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + 16 * U24 * np.abs(h)
