"""Plain CPU oracle of the layer's training operators (fp64, numpy).

TEST INFRASTRUCTURE.  Only the tests may import this module.  It shares no code with the
GPU library.

  balance_loss     load-balance loss per sequence, z loss, counts and the gradient with
                   respect to the logits (counts held fixed)
  gate_backward    d sum <dy, y> / d gate of every pick
  router_backward  gradient of the gates through the softmax to tokens and router weight
  adamw            one AdamW step in fp64; adamw_fp32 the same in fp32 with every operation
                   rounded, and the 8-bit states' codes from it
"""
from __future__ import annotations

import math

import numpy as np


def softmax(logits):
    """(p, logsumexp) per row; a row of -inf has p = 0 and logsumexp -inf."""
    l64 = np.asarray(logits, np.float64)
    top = l64.max(axis=1, keepdims=True)
    live = np.isfinite(top)
    with np.errstate(invalid="ignore", divide="ignore"):
        ex = np.where(live, np.exp(l64 - np.where(live, top, 0.0)), 0.0)
        tot = ex.sum(axis=1, keepdims=True)
        p = np.where(live, ex / np.where(tot > 0, tot, 1.0), 0.0)
        lse = np.where(live[:, 0], top[:, 0] + np.log(np.where(tot > 0, tot, 1.0))[:, 0], -np.inf)
    return p, lse


def balance_loss(logits, idx, balance, z, offsets=None, mask=None):
    """dict(loss [2], load [S,E], prob [S,E], dlogits [T,E], p, seq [T] (-1: does not count))."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    K = idx.shape[1]
    offsets = np.array([0, T]) if offsets is None else np.clip(np.asarray(offsets), 0, T)
    S = offsets.size - 1
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    clean = np.where(keep[:, None], logits, 0.0)
    p, lse = softmax(clean)
    seq = np.full(T, -1)
    for s in range(S):
        for t in range(offsets[s], offsets[s + 1]):
            if keep[t] and np.isfinite(lse[t]):
                seq[t] = s
    load = np.zeros((S, E), np.int64)
    prob = np.zeros((S, E))
    n = np.array([(seq == s).sum() for s in range(S)])
    for s in range(S):
        for t in np.nonzero(seq == s)[0]:
            for e in idx[t]:
                if 0 <= e < E:
                    load[s, e] += 1
        if n[s]:
            prob[s] = p[seq == s].sum(axis=0) / n[s]
    live, total = (n > 0).sum(), n.sum()
    loss = np.zeros(2)
    grad = np.zeros((T, E))
    for s in range(S):
        if not n[s]:
            continue
        f = E * load[s] / (K * n[s])
        loss[0] += balance / live * (f * prob[s]).sum()
        u = balance * (f - 1.0) / (live * n[s])
        rows = seq == s
        grad[rows] = p[rows] * (u - (p[rows] * u).sum(axis=1, keepdims=True))
    rows = seq >= 0
    if z and total:
        loss[1] = z / total * (lse[rows] ** 2).sum()
        grad[rows] += 2 * z / total * lse[rows, None] * p[rows]
    return dict(loss=loss, load=load, prob=prob, dlogits=grad, p=p, seq=seq, n=n)


def gate_backward(x, rows, slot, dy):
    """(dgate [T,K], sum of the products' magnitudes [T,K])."""
    T, K = slot.shape
    out, mag = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = slot[t, k]
            v = x[t] if r < 0 else rows[r] if r < rows.shape[0] else np.zeros_like(x[t])
            out[t, k] = (v * dy[t]).sum()
            mag[t, k] = np.abs(v * dy[t]).sum()
    return out, mag


def dlogits(logits, idx, dgate, aux=None):
    """(dlogits [T,E], p, dp)."""
    p, _ = softmax(logits)
    dp = np.zeros_like(p)
    T, E = p.shape
    for t in range(T):
        for k, e in enumerate(idx[t]):
            if 0 <= e < E:
                dp[t, e] += dgate[t, k]
    dl = p * (dp - (p * dp).sum(axis=1, keepdims=True))
    return (dl if aux is None else dl + aux), p, dp


def router_backward(x, w_router, logits, idx, dgate, aux=None, add=None):
    """dict(dx, dw_router, dlogits) in fp64."""
    if dgate is None:
        dl = np.zeros((x.shape[0], w_router.shape[0])) if aux is None else np.asarray(aux, np.float64)
    else:
        dl = dlogits(logits, idx, np.asarray(dgate, np.float64), aux)[0]
    dx = dl @ w_router
    return dict(dx=dx if add is None else dx + add, dw_router=dl.T @ x, dlogits=dl)


def adamw(w, g, m, v, lr, beta1, beta2, eps, wd, step, grad_scale=1.0):
    """(w, m, v) after one step, fp64."""
    g = np.asarray(g, np.float64) * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return w - lr * wd * w - lr * mh / (np.sqrt(vh) + eps), m, v


# ---- 8-bit states ------------------------------------------------------------------------

M32 = np.uint64(0xFFFFFFFF)


def mix(x):
    """The 32-bit mixing function of the random bits (x: uint64 array of values below 2^32)."""
    x = np.asarray(x, np.uint64) & M32
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x6A09E667)) & M32
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xBB67AE85)) & M32
    return x ^ (x >> np.uint64(16))


def random_bits(seed, step, place, index):
    """32 random bits of the elements `index` of the tensor at `place` of the call's list."""
    index = np.asarray(index, np.uint64)
    key = mix(np.uint64((seed + 0x9E3779B9 * step) & 0xFFFFFFFF))
    hi = index >> np.uint64(32)
    key = mix((key + np.uint64(0x3C6EF373) * np.uint64(place + 1) + np.uint64(0x85A308D3) * hi) & M32)
    return mix((index + key) & M32)


def e4m3_values(codes):
    c = np.asarray(codes).astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    a = np.where(e > 0, (8 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    return np.where(c & 128, -a, a)


def block_exponents(val):
    """k of each block of 128: the smallest integer with max |val| <= 448 * 2^k (0 for zeros)."""
    n = val.size
    b = np.abs(np.pad(np.asarray(val, np.float64), (0, -n % 128))).reshape(-1, 128).max(axis=1)
    k = np.zeros(b.size, np.int64)
    for i, a in enumerate(b):
        if a > 0:
            f, e = math.frexp(a)
            k[i] = max(e - 9 if f <= 0.875 else e - 8, -127)
    return k


def round_random(val, bits16, lowest, ulps=0):
    """(codes uint8, exponents k) of fp32 values, rounded by 16 random bits each: exact
    arithmetic (fp64 holds every product here).  ulps: the quotients are first moved by that
    many fp32 steps away from 0 (the codes an implementation may give whose quotient is off)."""
    val = np.asarray(val, np.float64)
    k = block_exponents(val)
    y = val / 2.0 ** np.repeat(k, 128)[:val.size].astype(np.float64)
    a = (np.abs(y).astype(np.float32).view(np.int32) + np.where(y == 0, 0, ulps)).astype(np.int32)
    a = a.view(np.float32).astype(np.float64)
    # the library's fraction: the 16 bits above a half, out of 2^20 parts of one step
    r = (np.asarray(bits16, np.int64) << 4) + 8
    # subnormal codes: steps of 2^-9; the sum is rounded to fp32 as the library's is
    sub = np.floor((a * 512.0 + r * 2.0 ** -20).astype(np.float32)).astype(np.int64)
    word = a.astype(np.float32).view(np.int32).astype(np.int64)
    nor = ((word + r) >> 20) - 960
    q = np.minimum(np.where(a < 2.0 ** -6, sub, nor), 126)
    if lowest:
        q = np.where((val > 0) & (q == 0), 1, q)
    return (q | np.where(y < 0, 128, 0)).astype(np.uint8), k


def adamw_fp32(w, g, m, v, lr, beta1, beta2, eps, wd, step, grad_scale=1.0):
    """(m, v, sqrt v) of one step with every operation rounded to fp32, as the codes of the
    8-bit states are taken from."""
    f = np.float32
    g = (np.asarray(g, f) * f(grad_scale)).astype(f)
    m = (f(beta1) * np.asarray(m, f)).astype(f) + (f(1.0 - float(f(beta1))) * g).astype(f)
    v = (f(beta2) * np.asarray(v, f)).astype(f) + ((f(1.0 - float(f(beta2))) * g).astype(f) * g).astype(f)
    return m.astype(f), v.astype(f), np.sqrt(v.astype(f))
