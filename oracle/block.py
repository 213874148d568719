"""Plain CPU oracle of the block operators (numpy, fp64).

TEST INFRASTRUCTURE.  Only the tests may import this module.  It shares no code with the GPU
library.

Every function is the formula of the operator written down, one token after another where that
is the plainest; inputs are taken as exact values.
"""
from __future__ import annotations

import numpy as np

from .fp8 import E4M3_TABLE, encode_scaled

BLOCK = 128


# ---- choice of experts ------------------------------------------------------------------------

def scores(logits, score):
    """s [T][E]; a logit of -infinity (or NaN) has score 0."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isfinite(m), m, 0.0))
        return e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)


def log_scores(logits, score):
    """log s, without underflow, up to a term that a token's experts share."""
    l = np.asarray(logits, np.float64)
    if score == "softmax":
        return l
    with np.errstate(over="ignore"):
        return np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))


def pick_weights(ls):
    """Shares of a token's picks from the logarithms of their scores."""
    if not len(ls) or not np.isfinite(ls.max()):
        return np.zeros(len(ls))
    w = np.exp(ls - ls.max())
    return w / w.sum()


def select(logits, bias, K, score="softmax", groups=1, top_groups=1, group_rank=1, renorm=False, scale=1.0, mask=None):
    """(idx [T][K], gate [T][K]); index -1 and gate 0 where there is no pick."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    s = scores(logits, score)
    idx, gate = np.full((T, K), -1, np.int64), np.zeros((T, K))
    size = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        on = (logits[t] > -np.inf) & (b > -np.inf)
        c = np.where(on, s[t] + np.where(on, b, 0), -np.inf)
        if top_groups < groups:
            val = []
            for g in range(groups):
                top = sorted(c[g * size:(g + 1) * size][on[g * size:(g + 1) * size]], reverse=True)[:group_rank]
                val.append(sum(top) if top else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups]
            c = np.where(np.isin(np.arange(E) // size, kept), c, -np.inf)
        order = [e for e in np.lexsort((np.arange(E), -c))[:K] if c[e] > -np.inf]
        idx[t, :len(order)] = order
        if renorm:
            gate[t, :len(order)] = scale * pick_weights(log_scores(logits[t, order], score))
        else:
            gate[t, :len(order)] = scale * s[t, order]
    return idx, gate


def select_backward(logits, idx, dgate, score="softmax", renorm=False, scale=1.0, aux=None):
    """(dlogits [T][E], mag [T][E]): mag is the same sum with every term's absolute value."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    s = scores(logits, score)
    r = scores(-logits, "sigmoid")  # 1 - s without cancellation
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ks = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E]
        es, dg = idx[t, ks].astype(int), np.asarray(dgate, np.float64)[t, ks]
        if renorm:
            w = pick_weights(log_scores(logits[t, es], score))
            v, a = scale * w * (dg - w @ dg), abs(scale) * w * (np.abs(dg) + w @ np.abs(dg))
            if score == "sigmoid":
                v, a = v * r[t, es], a * r[t, es]
        elif score == "sigmoid":
            v = scale * dg * s[t, es] * np.where(s[t, es] > 0, r[t, es], 0.0)
            a = np.abs(v)
        else:
            v, a = scale * dg, np.abs(scale * dg)
        np.add.at(out[t], es, v)
        np.add.at(mag[t], es, a)
        if score == "softmax" and not renorm:
            out[t], mag[t] = s[t] * (out[t] - s[t] @ out[t]), s[t] * (mag[t] + s[t] @ mag[t])
    if aux is not None:
        out, mag = out + aux, mag + np.abs(aux)
    return out, mag


# ---- norms around a block ---------------------------------------------------------------------

def rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def block_norm(x, y, gate, w_post, w_pre, a, b, eps):
    """(h, z or None)."""
    h = a * x
    if y is not None:
        u = y if w_post is None else y * rms(y, eps) * w_post
        h = h + b * (u if gate is None else gate * u)
    return h, None if w_pre is None else h * rms(h, eps) * w_pre


def block_norm_backward(h, dh, dz, y, gate, w_post, w_pre, a, b, eps):
    """dict of the gradients and, under the same names with "_mag", the sums of the absolute values
    of their terms."""
    zero = np.zeros_like(h)
    dh, dz = zero if dh is None else dh, zero if dz is None else dz
    w = np.zeros(h.shape[1]) if w_pre is None else w_pre
    r = rms(h, eps)
    v = w * dz
    dH = dh + r * (v - h * r * r * (v * h).mean(1, keepdims=True))
    mH = np.abs(dh) + r * (np.abs(v) + np.abs(h) * r * r * np.abs(v * h).mean(1, keepdims=True))
    o = dict(dx=a * dH, dx_mag=abs(a) * mH, dw_pre=(dz * h * r).sum(0), dw_pre_mag=np.abs(dz * h * r).sum(0))
    if y is None:
        return o
    g = 1.0 if gate is None else gate
    du, mu = b * g * dH, np.abs(b * g) * mH
    q = rms(y, eps) if w_post is not None else np.ones_like(r)
    yn = y * q
    u = yn if w_post is None else yn * w_post
    if gate is not None:
        axis = dict(axis=0) if np.ndim(gate) == 1 else dict(axis=1, keepdims=True)
        o["dgate"], o["dgate_mag"] = (b * u * dH).sum(**axis), (np.abs(b * u) * mH).sum(**axis)
    if w_post is None:
        o["dy"], o["dy_mag"] = du, mu
    else:
        o["dw_post"], o["dw_post_mag"] = (du * yn).sum(0), (mu * np.abs(yn)).sum(0)
        t, m = w_post * du, np.abs(w_post) * mu
        o["dy"] = q * (t - yn * (t * yn).mean(1, keepdims=True))
        o["dy_mag"] = q * (m + np.abs(yn) * (m * np.abs(yn)).mean(1, keepdims=True))
    return o


# ---- block FP8 --------------------------------------------------------------------------------

def quantize(v, rows, cols):
    """v [R][C] in blocks of rows x cols: (codes uint8 [R][C], exponents k, one per block)."""
    v = np.asarray(v, np.float64)
    R, C = v.shape
    nr, nc = -(-R // rows), -(-C // cols)
    pad = np.zeros((nr * rows, nc * cols))
    pad[:R, :C] = v
    amax = np.abs(pad).reshape(nr, rows, nc, cols).max((1, 3))
    frac, e = np.frexp(amax)
    k = np.where(amax == 0, 0, np.maximum(np.where(frac <= 0.875, e - 9, e - 8), -127))
    unit = np.exp2(k.astype(np.float64)).repeat(rows, 0).repeat(cols, 1)[:R, :C]
    return encode_scaled(v / unit).reshape(R, C), k


def values(codes, k, rows, cols):
    R, C = codes.shape
    return E4M3_TABLE[codes] * np.exp2(k.astype(np.float64)).repeat(rows, 0).repeat(cols, 1)[:R, :C]


def quantized(v, rows, cols):
    return values(*quantize(v, rows, cols), rows, cols)
