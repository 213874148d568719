"""Pins of the training oracle (oracle.train), no GPU: differences of the losses, torch
autograd of independently written forms, closed forms, and the mean of the random rounding."""
import math

import numpy as np
import pytest

from oracle import moe as orc
from oracle import backward as ob
from oracle import train as ot


def picks(rng, T, E, K):
    return np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int64)


def balance_case(seed, T=23, E=7, K=3):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((T, E)), picks(rng, T, E, K), np.array([0, 5, 5, 17, 23]),
            (rng.random(T) > 0.3).astype(np.uint8))


@pytest.mark.parametrize("seed", range(3))
def test_balance_differences(seed):
    lg, idx, off, mask = balance_case(seed)
    r = ot.balance_loss(lg, idx, 0.3, 0.05, off, mask)
    h = 1e-6
    for t in range(lg.shape[0]):
        for e in range(lg.shape[1]):
            a, b = lg.copy(), lg.copy()
            a[t, e] += h
            b[t, e] -= h
            fd = (ot.balance_loss(a, idx, 0.3, 0.05, off, mask)["loss"].sum()
                  - ot.balance_loss(b, idx, 0.3, 0.05, off, mask)["loss"].sum()) / (2 * h)
            assert abs(fd - r["dlogits"][t, e]) <= 1e-8


def test_balance_autograd():
    """torch autograd (fp64) of the loss written with masks and one-hot products."""
    import torch
    lg, idx, off, mask = balance_case(9)
    T, E = lg.shape
    r = ot.balance_loss(lg, idx, 0.3, 0.05, off, mask)
    x = torch.tensor(lg, requires_grad=True)
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    keep = torch.tensor(mask.astype(np.float64))
    hot = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, torch.tensor(idx), torch.ones(T, idx.shape[1], dtype=torch.float64))
    loss, live = 0.0, 0
    for a, b in zip(off, off[1:]):
        n = keep[a:b].sum()
        if n > 0:
            live += 1
            f = E / (idx.shape[1] * n) * (keep[a:b, None] * hot[a:b]).sum(0)
            loss = loss + (f * (keep[a:b, None] * p[a:b]).sum(0) / n).sum()
    bal = 0.3 * loss / live
    zl = 0.05 * (keep * lse ** 2).sum() / keep.sum()
    (bal + zl).backward()
    np.testing.assert_allclose(r["loss"], [bal.item(), zl.item()], rtol=1e-13)
    np.testing.assert_allclose(r["dlogits"], x.grad.numpy(), atol=1e-15)


def test_balance_closed_forms():
    """An even load: loss = coefficient, no gradient; all picks and all mass on one expert: E
    times it; nothing counts: zeros."""
    T, E = 12, 4
    lg = np.zeros((T, E))
    idx = (np.arange(T)[:, None] + np.arange(2)[None]) % E
    r = ot.balance_loss(lg, idx, 0.5, 0.0)
    np.testing.assert_allclose(r["loss"], [0.5, 0.0])
    assert not r["dlogits"].any()
    hot = np.full((T, E), -np.inf)
    hot[:, 2] = 0.0
    r = ot.balance_loss(hot, np.full((T, 1), 2), 0.5, 1.0)
    np.testing.assert_allclose(r["loss"], [0.5 * E, 0.0])
    r = ot.balance_loss(np.full((T, E), -np.inf), idx, 0.5, 1.0)
    assert not r["loss"].any() and not r["load"].any() and not r["dlogits"].any()
    r = ot.balance_loss(np.full((T, E), np.nan), idx, 0.5, 1.0, mask=np.zeros(T, np.uint8))
    assert not r["loss"].any() and not r["load"].any() and not r["dlogits"].any()


def test_whole_layer_differences():
    """sum <dy, y> + losses as a function of x and W_r, the picks and counts held fixed: the
    gate, router and FFN gradients together."""
    rng = np.random.default_rng(3)
    T, d, N, Z, K, I = 9, 6, 3, 2, 3, 5
    E = N + Z
    x, dy = rng.standard_normal((2, T, d))
    wr = rng.standard_normal((E, d)) / math.sqrt(d)
    w = [rng.standard_normal(s) / math.sqrt(d) for s in ((N, I, d), (N, I, d), (N, d, I))]
    idx = picks(rng, T, E, K)
    experts = lambda e: (w[0][e], w[1][e], w[2][e])  # noqa: E731
    load = ot.balance_loss(x @ wr.T, idx, 0.2, 0.1)

    def forward(x, wr):
        p = ot.softmax(x @ wr.T)[0]
        gate = np.take_along_axis(p, idx, axis=1)
        off, perm, slot = orc.permute(idx, N)
        rows = np.zeros((perm.size, d))
        for e in range(N):
            if off[e + 1] > off[e]:
                rows[off[e]:off[e + 1]] = orc.swiglu_expert(x[perm[off[e]:off[e + 1]]], *experts(e))
        y = orc.combine(x, rows, idx, gate, slot, N)
        b = ot.balance_loss(x @ wr.T, idx, 0.2, 0.1)
        assert (b["load"] == load["load"]).all()
        return (dy * y).sum() + b["loss"].sum(), gate, rows, slot

    _, gate, rows, slot = forward(x, wr)
    dgate = ot.gate_backward(x, rows, slot, dy)[0]
    dx_ffn, _ = ob.ffn_backward(x, dy, idx, gate, experts, N)
    r = ot.router_backward(x, wr, x @ wr.T, idx, dgate, aux=load["dlogits"], add=dx_ffn)
    h = 1e-6
    for arr, grad in ((x, r["dx"]), (wr, r["dw_router"])):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + h
            up = forward(x, wr)[0]
            arr[i] = old - h
            dn = forward(x, wr)[0]
            arr[i] = old
            fd = (up - dn) / (2 * h)
            assert abs(fd - grad[i]) <= 1e-6 * (1 + abs(fd)), (i, fd, grad[i])


def test_adamw_against_torch():
    import torch
    rng = np.random.default_rng(4)
    w, g1, g2 = rng.standard_normal((3, 50))
    p = torch.tensor(w.copy(), requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m, v = np.zeros(50), np.zeros(50)
    for step, g in ((1, g1), (2, g2)):
        p.grad = torch.tensor(g)
        opt.step()
        w, m, v = ot.adamw(w, g, m, v, 0.01, 0.9, 0.95, 1e-8, 0.1, step)
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-12)


def test_codes_round_to_neighbours_with_the_right_mean():
    """Over all 2^16 random values a code is the value's lower or upper neighbour, and the mean
    is the value: within 2^-17 of a step, half of the fraction's own grid."""
    vals = np.array([448.0, 447.9, 300.0, 17.3, 1.0, 0.9999, 0.3, 0.0156, 0.0157, 0.011, 0.0003, 0.0, -5.1], np.float32)
    pad = np.zeros(128, np.float32)
    pad[:vals.size] = vals
    got = ot.e4m3_values(ot.round_random(pad, np.zeros(128, np.int64), False)[0])[:vals.size]
    # the smallest fraction: every value rounds down
    grid = np.unique(ot.e4m3_values(np.arange(127)))
    for v, a in zip(vals, got):
        want = np.sign(v) * grid[np.searchsorted(grid, abs(v), side="right") - 1]
        assert a == want, (v, a, want)
    # the mean over all patterns, from the threshold at which the code goes up
    for v in vals:
        if v == 0:
            continue
        pad[:] = 0
        pad[0], pad[1] = v, 448.0
        base = grid[np.searchsorted(grid, abs(v), side="right") - 1]
        above = grid[min(np.searchsorted(grid, abs(v), side="right"), grid.size - 1)]
        a, z = 0, 1 << 16  # first pattern that rounds up
        while a < z:
            mid = (a + z) // 2
            up = abs(ot.e4m3_values(ot.round_random(pad, np.full(128, mid), False)[0])[0]) > base
            a, z = (a, mid) if up else (mid + 1, z)
        mean = base + (above - base) * ((1 << 16) - a) / (1 << 16)
        assert abs(mean - abs(v)) <= (above - base) * 2.0 ** -16 + 1e-12, (v, mean)


def test_lowest_keeps_positive_values_positive():
    val = np.zeros(128, np.float32)
    val[0], val[1], val[2] = 1.0, 1e-30, 0.0
    q, _ = ot.round_random(val, np.zeros(128, np.int64), True)
    assert q[1] == 1 and q[2] == 0


def test_random_bits_are_even():
    """Every bit of the hash over 2^14 neighbouring elements: its mean is within 5 standard
    deviations (5 / (2 sqrt n)) of a half, so are neighbours' and steps' exclusive ors.  The
    two halves, which round m and v of one element, are uncorrelated as fractions (|r| <= 5 /
    sqrt n)."""
    n = 1 << 14
    i = np.arange(n)
    a, b = ot.random_bits(7, 3, 0, i), ot.random_bits(7, 4, 0, i)
    c = ot.random_bits(7, 3, 1, i)
    tol = 5 / (2 * math.sqrt(n))
    for u in (a, b, a ^ b, a ^ c, a[1:] ^ a[:-1]):
        for bit in range(16):
            mean = ((u >> np.uint64(bit)) & np.uint64(1)).astype(np.float64).mean()
            assert abs(mean - 0.5) <= tol * 1.01, bit
    low, high = (a & np.uint64(0xFFFF)).astype(np.float64), (a >> np.uint64(16)).astype(np.float64)
    assert abs(np.corrcoef(low, high)[0, 1]) <= 5 / math.sqrt(n)
    assert np.unique(ot.random_bits(7, 3, 0, i + (1 << 32))).size == n
    assert (ot.random_bits(7, 3, 0, i + (1 << 32)) != a).mean() > 0.99


def test_8bit_states_track_32bit_ones():
    """200 steps of noisy gradients: r = sqrt v in 8 bits stays unbiased (its mean ratio to
    the fp32 state within 2%), where rounding to nearest would hold it still."""
    rng = np.random.default_rng(5)
    n, b2 = 1024, 0.999
    scale = np.exp(rng.uniform(-3, 3, n))
    v32 = (scale ** 2).astype(np.float32)
    q, k = ot.round_random(np.sqrt(v32), rng.integers(0, 1 << 16, n), True)
    for step in range(1, 201):
        g = (0.5 * scale * rng.standard_normal(n)).astype(np.float32)
        v8 = (ot.e4m3_values(q) * 2.0 ** np.repeat(k, 128)[:n]) ** 2
        v8 = b2 * v8 + (1 - b2) * g.astype(np.float64) ** 2
        v32 = b2 * v32 + (1 - b2) * g.astype(np.float64) ** 2
        q, k = ot.round_random(np.sqrt(v8).astype(np.float32), ot.random_bits(1, step, 0, np.arange(n)) >> np.uint64(16), True)
    r8 = ot.e4m3_values(q) * 2.0 ** np.repeat(k, 128)[:n]
    ratio = (r8 / np.sqrt(v32)).mean()
    assert abs(ratio - 1) <= 0.02
